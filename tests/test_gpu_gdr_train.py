"""GPU parity of the gated delta rule's training pair (gdr_forward_ckpt, gdr_backward_ckpt) with
the fp64 oracle, whose backward pass is pinned by finite differences.

Tolerance: every fp32 operand of a product is split into pieces that keep it to 2^-22 or
better and sums are in fp32, so a result is off by a few 2^-24 of the largest terms it sums.
Those are at most of the order of ten times the result's root mean square here (unit keys,
64 tokens a block, 128 channels a row): 10 x 2^-22 = 2.4e-6, within TOL.
"""
import numpy as np
import pytest
import torch

from gdr_inputs import NAMES, make, on_gpu
from oracle import gdr
from parity import HEADS_SEQ, HEADS_STATE, check

pytestmark = pytest.mark.gpu

TOL = 4e-6
SEQ = ("dq", "dk", "dv", "dg", "dbeta")


@pytest.fixture(scope="module")
def lib():
    import rwkv_linear_attention_amd as m
    m.lib()
    return m


def both(lib, inp, scale=None, d_state=True, seed=1, size=1.0, peak=1.0):
    B, T, Hk, K = inp["q"].shape
    H, V = inp["v"].shape[2:]
    gen = torch.Generator().manual_seed(seed)
    d_o = size * torch.randn(B, T, H, V, generator=gen)
    d_s = 0.3 * torch.randn(B, H, K, V, generator=gen) if d_state else None
    used = K ** -0.5 if scale is None else scale
    ref_o, ref_s, _ = gdr.forward(*(inp[n] for n in NAMES), inp["state"], used)
    ref = gdr.backward(*(inp[n] for n in NAMES), inp["state"], d_o, d_s, used)
    d = on_gpu(inp)
    o, s, ckpt, resid = lib.gdr_forward_ckpt(*(d[n] for n in NAMES), d["state"], scale=scale)
    got = lib.gdr_backward_ckpt(d["q"], d["k"], d["g"], d["beta"], ckpt, resid, d_o.cuda(),
                                None if d_s is None else d_s.cuda(), scale=scale)
    tensors = [(o, ref_o, "o", HEADS_SEQ), (s, ref_s, "state", HEADS_STATE),
               *((got[n], ref[n], n, HEADS_SEQ) for n in SEQ),
               (got["d_state_in"], ref["d_state_in"], "d_state_in", HEADS_STATE)]
    for x, want, n, heads in tensors:
        check(x, want, TOL, n, None)
        check(x, want, peak * TOL, n, heads)
    return got


@pytest.mark.parametrize("B,T,Hk,H,K,V,dtype", [
    (1, 1, 1, 1, 64, 64, "bf16"), (2, 5, 1, 2, 64, 64, "fp32"), (1, 31, 2, 2, 128, 64, "bf16"),
    (1, 32, 1, 1, 64, 128, "bf16"), (2, 33, 1, 3, 64, 64, "bf16"), (1, 63, 2, 4, 128, 128, "bf16"),
    (2, 64, 1, 1, 128, 128, "fp32"), (1, 65, 1, 2, 64, 64, "bf16"), (1, 97, 1, 1, 64, 192, "fp32"),
    (1, 130, 2, 2, 128, 256, "bf16"), (2, 300, 1, 2, 64, 64, "bf16")])
def test_against_the_oracle(lib, B, T, Hk, H, K, V, dtype):
    both(lib, make(B, T, Hk, H, K, V, seed=T, dtype=dtype))


@pytest.mark.parametrize("T", [20, 100])
def test_without_states_and_with_a_scale(lib, T):
    both(lib, make(1, T, 1, 2, 64, 64, seed=3, state=False), scale=1.5, d_state=False)


@pytest.mark.parametrize("T", [40, 140])
def test_dropped_states_and_idle_gates(lib, T):
    """No decay and no strength is divided by: g = -inf, beta = 0 and beta = 1 with a unit key."""
    inp = make(2, T, 1, 2, 64, 64, seed=7, dtype="fp32")
    inp["g"][0, T // 2] = float("-inf")
    inp["g"][1, 3] = -300.0
    inp["g"][1, 9] = 0.0
    inp["beta"][0, ::3] = 0.0
    inp["beta"][1] = 1.0
    both(lib, inp, scale=1.0)


def test_states_that_grow(lib):
    """A positive g is no decay, but nothing forbids it.

    The bound of an element counts in root mean squares of its head, over all tokens.  Here the
    states and gradients grow by up to e^0.1 a token, their squares by e^0.2: all but the last
    (or first) 1 / (1 - e^-0.2) = 5.5 of the 100 tokens hold next to nothing, and the elements of
    those that count are sqrt(100 / 5.5) = 4.3 times that mean.  So the bound is 4.3 times TOL for
    single elements, and TOL for a tensor as a whole.
    """
    inp = make(1, 100, 1, 2, 64, 64, seed=25, dtype="fp32")
    inp["g"] = inp["g"].abs().clamp(max=0.1)
    both(lib, inp, peak=4.3)


def test_one_key_over_and_over(lib):
    inp = make(1, 100, 1, 1, 64, 64, seed=8, dtype="bf16", decay=0.1)
    inp["k"][:] = inp["k"][:, :1]
    both(lib, inp, scale=1.0)


def test_checkpointed_forward_is_the_forward(lib):
    d = on_gpu(make(2, 90, 1, 2, 128, 64, seed=4))
    args = [d[n] for n in NAMES]
    o, s = lib.gdr_forward(*args, d["state"])
    o2, s2, ckpt, resid = lib.gdr_forward_ckpt(*args, d["state"])
    assert torch.equal(o, o2) and torch.equal(s, s2)
    assert ckpt.shape == (2, 2, 2, 128 * 64) and resid.shape == o.shape


def test_empty_sequences(lib):
    d = on_gpu(make(2, 0, 1, 2, 64, 64))
    args = [d[n] for n in NAMES]
    for run in (lib.gdr_forward, lib.gdr_step):
        o, s = run(*args, d["state"])
        assert o.shape == (2, 0, 2, 64) and torch.equal(s, d["state"])
        assert not run(*args)[1].any()
    o, s, ckpt, resid = lib.gdr_forward_ckpt(*args, d["state"])
    assert torch.equal(s, d["state"])
    d_s = torch.randn_like(s)
    g = lib.gdr_backward_ckpt(d["q"], d["k"], d["g"], d["beta"], ckpt, resid, torch.empty_like(o), d_s)
    assert torch.equal(g["d_state_in"], d_s)
    g = lib.gdr_backward_ckpt(d["q"], d["k"], d["g"], d["beta"], ckpt, resid, torch.empty_like(o))
    assert not g["d_state_in"].any()


def test_twice_the_same_bits_and_graph_replays(lib):
    ins = [on_gpu(make(1, 150, 2, 4, 64, 64, seed=s)) for s in range(2)]
    for d in ins:
        d["d_o"] = torch.randn(1, 150, 4, 64, generator=torch.Generator().manual_seed(3)).cuda()

    def step(d, bufs=None):
        f, b, work = bufs if bufs else ({}, None, None)
        o, s, ckpt, resid = lib.gdr_forward_ckpt(*(d[n] for n in NAMES), d["state"], **f)
        g = lib.gdr_backward_ckpt(d["q"], d["k"], d["g"], d["beta"], ckpt, resid, d["d_o"], s, grads=b, work=work)
        return o, s, ckpt, resid, g

    eager = [step(d) for d in ins]
    for a, b in zip(eager, (step(d) for d in ins)):
        assert all(torch.equal(a[4][n], b[4][n]) for n in a[4])
    static = {n: x.clone() for n, x in ins[0].items()}
    o, s, ckpt, resid, g = (step(static))
    bufs = ({"o": o, "state_out": s, "ckpt": ckpt, "resid": resid}, g, torch.empty_like(ckpt))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(static, bufs)
    for i in (1, 0, 1):
        for n, x in static.items():
            x.copy_(ins[i][n])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, eager[i][0])
        for n, x in g.items():
            assert torch.equal(x, eager[i][4][n]), n
        step(ins[1 - i])


def test_two_steps_at_once_on_two_streams(lib):
    ins = [on_gpu(make(2, 500, 2, 4, 64, 128, seed=s)) for s in range(2)]
    d_o = torch.randn(2, 500, 4, 128, generator=torch.Generator().manual_seed(3)).cuda()

    def step(d):
        o, s, ckpt, resid = lib.gdr_forward_ckpt(*(d[n] for n in NAMES), d["state"])
        return lib.gdr_backward_ckpt(d["q"], d["k"], d["g"], d["beta"], ckpt, resid, d_o, s)

    want = [step(d) for d in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = []
    for side, d in zip(streams, ins):
        with torch.cuda.stream(side):
            got.append(step(d))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("size", [1e-25, 1e-9, 1e-4, 1e8])
def test_gradients_of_any_size(lib, size):
    """The gradients are linear in d_o: the mean over many tokens makes it small, a loss scale large."""
    inp = make(1, 150, 1, 2, 64, 64, seed=9, dtype="fp32")
    both(lib, inp, d_state=False, size=size)
    both(lib, inp, size=size)    # and beside a d_state_out of its usual size


@pytest.mark.parametrize("T,K,V,dtype", [(33, 64, 64, "bf16"), (70, 128, 64, "fp32"), (65, 128, 128, "bf16")])
def test_guard_bands(lib, T, K, V, dtype):
    """Inputs lie in NaN, outputs in a pattern: nothing beside them is used or written."""
    from test_gpu_gdr import guarded
    d = on_gpu(make(2, T, 1, 2, K, V, seed=T, dtype=dtype))
    d["d_o"] = torch.randn(2, T, 2, V, generator=torch.Generator().manual_seed(1)).cuda()
    names = ("o", "state_out", "ckpt", "resid")
    fwd = dict(zip(names, lib.gdr_forward_ckpt(*(d[n] for n in NAMES), d["state"])))
    want = lib.gdr_backward_ckpt(d["q"], d["k"], d["g"], d["beta"], fwd["ckpt"], fwd["resid"], d["d_o"], d["state"])
    ins = {n: guarded(x, float("nan"))[0] for n, x in d.items()}
    held = {n: guarded(torch.zeros_like(x), -3.25) for n, x in [*fwd.items(), *want.items(), ("work", fwd["ckpt"])]}
    lib.gdr_forward_ckpt(*(ins[n] for n in NAMES), ins["state"], **{n: held[n][0] for n in names})
    got = lib.gdr_backward_ckpt(ins["q"], ins["k"], ins["g"], ins["beta"], held["ckpt"][0], held["resid"][0],
                                ins["d_o"], ins["state"], grads={n: held[n][0] for n in want}, work=held["work"][0])
    for n, x in want.items():
        assert torch.equal(got[n], x), n
    for n, (v, big) in held.items():
        room = (big.numel() - v.numel()) // 2
        assert bool((big[:room] == -3.25).all()) and bool((big[-room:] == -3.25).all()), n


def test_the_state_gradient_in_place(lib):
    d = on_gpu(make(1, 70, 1, 2, 64, 128, seed=5))
    o, s, ckpt, resid = lib.gdr_forward_ckpt(*(d[n] for n in NAMES), d["state"])
    args = (d["q"], d["k"], d["g"], d["beta"], ckpt, resid, torch.ones_like(o))
    want = lib.gdr_backward_ckpt(*args, s)
    grads = {n: torch.empty_like(x) for n, x in want.items()}
    grads["d_state_in"].copy_(s)
    got = lib.gdr_backward_ckpt(*args, grads["d_state_in"], grads=grads)
    for n, x in want.items():
        assert torch.equal(got[n], x), n


def test_gradients_against_differences(lib):
    """The loss's change along a direction, by the forward pass itself.

    A central difference at step h leaves h^2/6 times the third derivative (of order the loss)
    and the forward's own error over h: 1e-6 |loss| / h.  At h = 1e-2 both are below 1e-3."""
    inp = make(1, 80, 1, 2, 64, 64, seed=12, dtype="fp32")
    d = on_gpu(inp)
    gen = torch.Generator().manual_seed(5)
    d_o = torch.randn(1, 80, 2, 64, generator=gen).cuda()
    d_s = torch.randn(1, 2, 64, 64, generator=gen).cuda()

    def run(x):
        return lib.gdr_forward_ckpt(*(x[n] for n in NAMES), x["state"])

    def loss(x):
        o, s = run(x)[:2]
        return float((o.double() * d_o.double()).sum() + (s.double() * d_s.double()).sum())

    _, _, ckpt, resid = run(d)
    got = lib.gdr_backward_ckpt(d["q"], d["k"], d["g"], d["beta"], ckpt, resid, d_o, d_s)
    for n in NAMES + ("state",):
        way = torch.randn(d[n].shape, generator=gen).cuda()
        way /= way.norm()
        h = 1e-2
        ends = [loss({**d, n: d[n] + e * way}) for e in (h, -h)]
        want = (ends[0] - ends[1]) / (2 * h)
        have = float((got["d_state_in" if n == "state" else "d" + n].double() * way.double()).sum())
        size = float(got["d_state_in" if n == "state" else "d" + n].double().norm())
        print(f"  {n}: difference {want:.6f}, gradient {have:.6f}", flush=True)
        assert abs(want - have) < 2e-3 * max(size, 1.0), n


def test_refusals(lib):
    d = on_gpu(make(1, 70, 1, 2, 64, 64))
    args = [d[n] for n in NAMES]
    o, s, ckpt, resid = lib.gdr_forward_ckpt(*args, d["state"])
    back = [d["q"], d["k"], d["g"], d["beta"], ckpt, resid, torch.zeros_like(o)]
    with pytest.raises(ValueError):
        lib.gdr_forward_ckpt(*args, o=torch.empty_like(o).bfloat16())
    with pytest.raises(ValueError):
        lib.gdr_forward_ckpt(*args, ckpt=ckpt[:, :1].contiguous())
    for i, bad in ((4, ckpt[:, :1].contiguous()), (5, resid.bfloat16()), (6, back[6][:, :-1].contiguous()),
                   (2, d["g"].double())):
        with pytest.raises(ValueError):
            lib.gdr_backward_ckpt(*back[:i], bad, *back[i + 1:])
    with pytest.raises(ValueError):
        lib.gdr_backward_ckpt(*back, work=torch.empty(3, device="cuda"))
    with pytest.raises(lib.Wkv7Error):     # the scratch on top of the checkpoints
        lib.gdr_backward_ckpt(*back, work=ckpt)
