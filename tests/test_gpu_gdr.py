"""GPU parity of the gated delta rule (gdr_forward, gdr_step) with the fp64 oracle.

Tolerances (relative L2; see parity.py for the per-head and per-element bounds).  An fp32
result is a sum of products in fp32 (2^-24 each way) in which some operands were split into
pieces that keep them to 2^-22 (two fp16 pieces, 2^-11 each) or 2^-24 (three bf16 pieces).  At
most four such operands stand between an input and an output (the state, the triangular inverse,
the residual and what it adds to the state), 4 x 2^-22 = 1e-6, and the rule does not amplify an
error (unit keys, beta <= 1, decay <= 1).  4e-6 leaves the accumulation of the sums (up to 128
products and 32 tokens, each rounded) three times as much again.  A bf16 output adds half a
step, 2^-8 relative.
"""
import numpy as np
import pytest
import torch

from gdr_inputs import DT, NAMES, make, on_gpu
from oracle import gdr
from parity import HEADS_SEQ, HEADS_STATE, check

pytestmark = pytest.mark.gpu

TOL = 4e-6
BF16 = 2.0 ** -8


@pytest.fixture(scope="module")
def lib():
    import rwkv_linear_attention_amd as m
    m.lib()
    return m


def check_o(o, ref, what):
    bf16 = o.dtype == torch.bfloat16
    check(o, ref, TOL + (BF16 if bf16 else 0.0), what, HEADS_SEQ, BF16 if bf16 else 0.0)


# B, T, Hk, H, K, V, input, output
SHAPES = [(1, 1, 1, 1, 64, 64, "bf16", "fp32"), (2, 5, 2, 4, 64, 64, "bf16", "bf16"),
          (1, 8, 1, 3, 128, 64, "bf16", "fp32"), (2, 9, 2, 2, 64, 128, "fp32", "fp32"),
          (1, 31, 1, 2, 128, 128, "bf16", "fp32"), (2, 32, 1, 1, 128, 192, "bf16", "bf16"),
          (1, 33, 3, 3, 64, 64, "fp32", "bf16"), (3, 64, 2, 6, 64, 64, "bf16", "fp32"),
          (1, 65, 1, 1, 128, 512, "bf16", "fp32"), (1, 100, 2, 2, 128, 128, "fp32", "fp32"),
          (2, 257, 1, 2, 64, 128, "bf16", "fp32"), (1, 700, 2, 2, 128, 64, "bf16", "fp32")]


@pytest.mark.parametrize("B,T,Hk,H,K,V,dtype,out", SHAPES)
@pytest.mark.parametrize("entry", ["forward", "step"])
def test_against_the_oracle(lib, entry, B, T, Hk, H, K, V, dtype, out):
    inp = make(B, T, Hk, H, K, V, seed=T + H, dtype=dtype)
    ref_o, ref_s, _ = gdr.forward(*(inp[n] for n in NAMES), inp["state"], K ** -0.5)
    d = on_gpu(inp)
    run = lib.gdr_forward if entry == "forward" else lib.gdr_step
    o, s = run(*(d[n] for n in NAMES), d["state"], o_dtype=DT[out])
    assert o.dtype == DT[out]
    check_o(o, ref_o, "o")
    check(s, ref_s, TOL, "state", HEADS_STATE)


@pytest.mark.parametrize("B,H,V", [(1, 2, 64), (5, 13, 64), (3, 22, 128), (9, 15, 64)])
def test_every_width_of_a_workgroup(lib, B, H, V):
    """Few heads split into narrower workgroups (1, 2 or 4 waves of 16 columns): rows of each."""
    inp = make(B, 41, 1, H, 64, V, seed=B)
    ref_o, ref_s, _ = gdr.forward(*(inp[n] for n in NAMES), inp["state"], 0.125)
    d = on_gpu(inp)
    o, s = lib.gdr_forward(*(d[n] for n in NAMES), d["state"])
    check_o(o, ref_o, "o")
    check(s, ref_s, TOL, "state", HEADS_STATE)


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("entry", ["forward", "step"])
def test_without_a_state_in_place_and_with_a_scale(lib, entry, T):
    inp = make(2, T, 1, 2, 64, 64, seed=5, state=False)
    d = on_gpu(inp)
    run = lib.gdr_forward if entry == "forward" else lib.gdr_step
    args = [d[n] for n in NAMES]
    ref_o, ref_s, _ = gdr.forward(*(inp[n] for n in NAMES), None, 2.5)
    o, s = run(*args, scale=2.5)
    check_o(o, ref_o, "o")
    check(s, ref_s, TOL, "state", HEADS_STATE)
    first = s.clone()
    o2, s2 = run(*args, s, scale=2.5, state_out=s)     # on from there, in place
    assert s2 is s
    ref_o2, ref_s2, _ = gdr.forward(*(inp[n] for n in NAMES), first, 2.5)
    check_o(o2, ref_o2, "o in place")
    check(s, ref_s2, TOL, "state in place", HEADS_STATE)


@pytest.mark.parametrize("T,lengths", [(7, [0, 7, 3, 1]), (90, [90, 0, 1, 64]), (90, [32, 33, 31, 200]),
                                       (70, [-3, 9, 8, 69])])
def test_lengths(lib, T, lengths):
    inp = make(4, T, 1, 2, 128, 64, seed=T, dtype="bf16")
    ref_o, ref_s, _ = gdr.forward(*(inp[n] for n in NAMES), inp["state"], 128 ** -0.5, lengths)
    for n in NAMES:   # what stands behind a row's end is not used
        for b, L in enumerate(lengths):
            inp[n][b, max(0, min(L, T)):] = float("nan")
    d = on_gpu(inp)
    o = torch.full((4, T, 2, 64), 7.0, device="cuda")
    o, s = lib.gdr_forward(*(d[n] for n in NAMES), d["state"], o=o, lengths=torch.tensor(lengths))
    for b, L in enumerate(lengths):
        L = max(0, min(L, T))
        assert bool((o[b, L:] == 7.0).all())
        if L:
            check_o(o[b:b + 1, :L], ref_o[b:b + 1, :L], f"o of row {b}")
        else:
            assert torch.equal(s[b], d["state"][b])
    check(s, ref_s, TOL, "state", HEADS_STATE)


@pytest.mark.parametrize("B", [11, 64, 70])
def test_many_rows_of_their_own_lengths(lib, B):
    """Rows start by length (up to 64 of them): each must still be its own."""
    lengths = torch.randint(0, 60, (B,), generator=torch.Generator().manual_seed(B))
    lengths[:3] = 17     # ties
    inp = make(B, 57, 1, 2, 64, 64, seed=B)
    ref_o, ref_s, _ = gdr.forward(*(inp[n] for n in NAMES), inp["state"], 0.125, lengths.tolist())
    d = on_gpu(inp)
    o, s = lib.gdr_forward(*(d[n] for n in NAMES), d["state"], o=torch.zeros(B, 57, 2, 64, device="cuda"),
                           lengths=lengths)
    check_o(o, ref_o, "o")
    check(s, ref_s, TOL, "state", HEADS_STATE)


@pytest.mark.parametrize("K,V", [(64, 64), (128, 128)])
def test_verify_commit_chain(lib, K, V):
    """Serving as it is used: prefill, a verify step over drafts, the drafts judged, the states committed, on."""
    B, H, Hk, N, vocab = 3, 4, 2, 4, 1000
    pre, ver, nxt = (make(B, T, Hk, H, K, V, seed=T, dtype="bf16") for T in (50, N + 1, 1))
    ref = {n: gdr.as_f64(x) for n, x in ver.items()}
    dp, dv, dn = on_gpu(pre), on_gpu(ver), on_gpu(nxt)
    _, s0 = lib.gdr_forward(*(dp[n] for n in NAMES), dp["state"])
    o, none, pos = lib.gdr_step(*(dv[n] for n in NAMES), s0, per_position=True, write_state_out=False)
    assert none is None
    gen = torch.Generator().manual_seed(1)
    target = torch.softmax(2 * torch.randn(B, N + 1, vocab, generator=gen), -1).cuda()
    tokens = torch.randint(0, vocab, (B, N), generator=gen, dtype=torch.int32).cuda()
    u = torch.full((B, N), 0.0, device="cuda")
    u[1, 2], u[2, 0] = 1.0, 1.0     # row 1 keeps two drafts, row 2 none (a sure drafter)
    out, kept = lib.draft_verify(target, tokens, u, torch.rand(B, generator=gen).cuda())
    assert kept.tolist() == [N + 1, 3, 1]
    s1 = lib.wkv7_state_commit(pos, kept, s0, state_out=s0.clone())
    _, ref_s0, _ = gdr.forward(*(pre[n] for n in NAMES), pre["state"], K ** -0.5)
    ref_o, _, ref_pos = gdr.forward(*(ref[n] for n in NAMES), ref_s0, K ** -0.5)
    check_o(o, ref_o, "o of the verify step")
    want = np.stack([ref_pos[b, n - 1] for b, n in enumerate(kept.tolist())])
    check(s1, want, TOL, "committed state", HEADS_STATE)
    o2, s2 = lib.gdr_step(*(dn[n] for n in NAMES), s1, state_out=s1)
    ref_o2, ref_s2, _ = gdr.forward(*(nxt[n] for n in NAMES), want, K ** -0.5)
    check_o(o2, ref_o2, "o of the next token")
    check(s2, ref_s2, TOL, "state of the next token", HEADS_STATE)
    lib.wkv7_state_reset(s2, torch.tensor([True, False, True]))
    assert not s2[0].any() and not s2[2].any() and bool(s2[1].any())


@pytest.mark.parametrize("T", [4, 80])
def test_dropped_states_and_idle_gates(lib, T):
    """g = -inf drops the state before a token, beta = 0 writes nothing, beta = 1 with a unit key replaces."""
    inp = make(2, T, 1, 2, 64, 64, seed=11, dtype="fp32")
    inp["g"][0, T // 2] = float("-inf")
    inp["g"][1, 0] = -200.0
    inp["beta"][0, 1] = 0.0
    inp["beta"][1] = 1.0
    ref_o, ref_s, _ = gdr.forward(*(inp[n] for n in NAMES), inp["state"], 1.0)
    d = on_gpu(inp)
    for run in (lib.gdr_forward, lib.gdr_step):
        o, s = run(*(d[n] for n in NAMES), d["state"], scale=1.0)
        check_o(o, ref_o, "o")
        check(s, ref_s, TOL, "state", HEADS_STATE)


@pytest.mark.parametrize("decay", [0.0, 1.0, 30.0])
def test_one_key_over_and_over(lib, decay):
    """Equal keys make the chunk's triangular system as far from the identity as it gets."""
    inp = make(1, 96, 1, 1, 128, 64, seed=2, dtype="bf16", decay=decay)
    inp["k"][:] = inp["k"][:, :1]
    ref_o, ref_s, _ = gdr.forward(*(inp[n] for n in NAMES), inp["state"], 1.0)
    d = on_gpu(inp)
    for run in (lib.gdr_forward, lib.gdr_step):
        o, s = run(*(d[n] for n in NAMES), d["state"], scale=1.0)
        check_o(o, ref_o, "o")
        check(s, ref_s, TOL, "state", HEADS_STATE)


@pytest.mark.parametrize("T", [3, 70])
def test_value_columns_are_apart(lib, T):
    """A NaN in one value channel stays in its column (and, chunked, within its chunk before the token)."""
    inp = make(1, T, 1, 1, 64, 64, seed=6, dtype="fp32")
    d = on_gpu(inp)
    o1, s1 = lib.gdr_forward(*(d[n] for n in NAMES), d["state"])
    at = T // 2 + 5 if T > 9 else 1
    d["v"][0, at, 0, 7] = float("nan")
    o2, s2 = lib.gdr_forward(*(d[n] for n in NAMES), d["state"])
    cols = torch.arange(64, device="cuda") != 7
    assert torch.equal(o1[..., cols], o2[..., cols]) and torch.equal(s1[..., cols], s2[..., cols])
    assert bool(o2[0, at:, 0, 7].isnan().all()) and bool(s2[0, 0, :, 7].isnan().all())
    chunk = at // 32 * 32 if T >= 9 else at
    assert not bool(o2[0, :chunk, 0, 7].isnan().any())


def test_streams_and_graph_replays(lib):
    """On a side stream, and captured: every replay on new inputs against the eager result."""
    shape = (2, 40, 1, 2, 64, 64)
    ins = [on_gpu(make(*shape, seed=s)) for s in range(3)]
    eager = [lib.gdr_forward(*(d[n] for n in NAMES), d["state"]) for d in ins]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, s = lib.gdr_forward(*(ins[1][n] for n in NAMES), ins[1]["state"])
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, eager[1][0]) and torch.equal(s, eager[1][1])
    static = {n: x.clone() for n, x in ins[0].items()}
    o, s = torch.empty_like(eager[0][0]), torch.empty_like(eager[0][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.gdr_forward(*(static[n] for n in NAMES), static["state"], o=o, state_out=s)
    for i in (1, 2, 0, 1):
        for n, x in static.items():
            x.copy_(ins[i][n])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, eager[i][0]) and torch.equal(s, eager[i][1])
        again = lib.gdr_forward(*(ins[i][n] for n in NAMES), ins[i]["state"])
        assert torch.equal(again[0], o)


@pytest.mark.parametrize("scale_s,scale_v", [(1e-40, 3e4), (1e-20, 1.0), (1e25, 1.0), (1e30, 1e30), (0.0, 1e-25),
                                             (1.0, 1e-12), (1e-6, 1e6)])
def test_magnitudes(lib, scale_s, scale_v):
    """The rule is linear in (state, v): any scale of either must come through the matrix cores' pieces."""
    inp = make(2, 100, 1, 2, 64, 64, seed=21, dtype="fp32", decay=0.2)
    inp["state"] = inp["state"] * scale_s
    inp["v"] = inp["v"] * scale_v
    inp["v"][:, 40:] *= 1e-3      # and a change of scale on the way
    inp["v"][1, :, :, 32:] = 0.0  # columns that only decay
    ref_o, ref_s, _ = gdr.forward(*(inp[n] for n in NAMES), inp["state"], 1.0)
    d = on_gpu(inp)
    o, s = lib.gdr_forward(*(d[n] for n in NAMES), d["state"], scale=1.0)
    for b in range(2):     # each half of each row on its own: one may be 1e30 times the other
        for cols in (slice(0, 32), slice(32, 64)):
            if 0 < np.abs(ref_s[b, :, :, cols]).max() < 1e-30:   # fp32 itself has fewer bits from 1e-38 down
                continue
            check(s[b:b + 1, :, :, cols], ref_s[b:b + 1, :, :, cols], TOL, "state", (1,))
            check(o[b:b + 1, :, :, cols], ref_o[b:b + 1, :, :, cols], TOL, "o", (2,))


@pytest.mark.parametrize("how", ["reset", "late", "both"])
def test_a_change_of_scale_at_once(lib, how):
    """A state of 1e6 that is dropped, values that start after some chunks of zeros."""
    inp = make(1, 200, 1, 2, 64, 64, seed=24, dtype="fp32", decay=0.2)
    if how != "late":
        inp["state"] = inp["state"] * 1e6
        inp["g"][:, 70] = float("-inf")
    if how != "reset":
        inp["state"][:, 1] = 0
        inp["v"][:, :90] = 0
        inp["v"][:, 90:] *= 1e-5
    ref_o, ref_s, _ = gdr.forward(*(inp[n] for n in NAMES), inp["state"], 1.0)
    d = on_gpu(inp)
    o, s = lib.gdr_forward(*(d[n] for n in NAMES), d["state"], scale=1.0)
    check(o[:, 96:], ref_o[:, 96:], TOL, "o", (0, 2))
    check(s, ref_s, TOL, "state", HEADS_STATE)


def test_states_that_grow(lib):
    """A positive g is no decay, but nothing forbids it: 0.3 a token multiplies the state by 1e13."""
    inp = make(1, 100, 1, 2, 64, 64, seed=25, dtype="fp32")
    inp["g"] = inp["g"].abs().clamp(max=0.3)
    ref_o, ref_s, _ = gdr.forward(*(inp[n] for n in NAMES), inp["state"], 1.0)
    d = on_gpu(inp)
    o, s = lib.gdr_forward(*(d[n] for n in NAMES), d["state"], scale=1.0)
    check(o, ref_o, TOL, "o", HEADS_SEQ)
    check(s, ref_s, TOL, "state", HEADS_STATE)


@pytest.mark.parametrize("norm", [1e-4, 0.05, 1.4])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_keys_of_other_norms(lib, norm, dtype):
    """Keys that are not normalised take the path with a power of two per row; mixed rows too."""
    inp = make(1, 70, 1, 2, 128, 64, seed=22, dtype=dtype, key_norm=norm)
    inp["q"] = (inp["q"].float() * 30).to(inp["q"].dtype)
    inp["k"][0, 5] = 0
    inp["q"][0, 33] = 0
    ref_o, ref_s, _ = gdr.forward(*(inp[n] for n in NAMES), inp["state"], 1.0)
    d = on_gpu(inp)
    o, s = lib.gdr_forward(*(d[n] for n in NAMES), d["state"], scale=1.0)
    check_o(o, ref_o, "o")
    check(s, ref_s, TOL, "state", HEADS_STATE)


def test_a_long_sequence(lib):
    inp = make(1, 5000, 1, 2, 64, 64, seed=23, decay=0.05)
    ref_o, ref_s, _ = gdr.forward(*(inp[n] for n in NAMES), inp["state"], 0.125)
    d = on_gpu(inp)
    o, s = lib.gdr_forward(*(d[n] for n in NAMES), d["state"])
    check_o(o, ref_o, "o")
    check(s, ref_s, TOL, "state", HEADS_STATE)


def guarded(x, fill, room=4096):
    """x inside a larger allocation filled with `fill` before and behind it."""
    big = torch.full((x.numel() + 2 * room,), fill, dtype=x.dtype, device="cuda")
    view = big[room:room + x.numel()].view(x.shape)
    view.copy_(x)
    return view, big


@pytest.mark.parametrize("T,K,V,dtype", [(5, 128, 64, "bf16"), (33, 64, 64, "bf16"), (61, 128, 128, "fp32")])
def test_guard_bands(lib, T, K, V, dtype):
    """Inputs lie in NaN, outputs in a pattern: nothing beside them is used or written."""
    inp = make(2, T, 1, 2, K, V, seed=T, dtype=dtype)
    d = on_gpu(inp)
    plain_o, plain_s = lib.gdr_forward(*(d[n] for n in NAMES), d["state"])
    ins = [guarded(d[n], float("nan"))[0] for n in NAMES + ("state",)]
    outs = {"o": torch.zeros_like(plain_o), "state_out": torch.zeros_like(plain_s)}
    held = {n: guarded(x, -3.25) for n, x in outs.items()}
    lengths = guarded(torch.tensor([T, T - 2], dtype=torch.int32, device="cuda"), 1 << 30)[0]
    lib.gdr_forward(*ins, **{n: v for n, (v, _) in held.items()})
    assert torch.equal(held["o"][0], plain_o) and torch.equal(held["state_out"][0], plain_s)
    lib.gdr_forward(*ins, lengths=lengths, **{n: v for n, (v, _) in held.items()})
    pos = guarded(torch.zeros(2, T, 2, K, V, device="cuda"), -3.25)
    lib.gdr_step(*ins, state_pos=pos[0], **{n: v for n, (v, _) in held.items()})
    for n, (v, big) in [*held.items(), ("state_pos", pos)]:
        room = (big.numel() - v.numel()) // 2
        assert bool((big[:room] == -3.25).all()) and bool((big[-room:] == -3.25).all()), n
        assert not bool(v.isnan().any()), n


def test_offsets_beyond_32_bits(lib):
    """More than 2^32 elements in the per-position states, and in v and o of a long sequence."""
    H, T = 8192, 66
    inp = on_gpu(make(1, T, 1, 1, 128, 64, seed=31))
    wide = {n: x.repeat(1, 1, *([1, 1] if n in ("q", "k") else [H] + [1] * (x.dim() - 3))) if n != "state"
            else x.repeat(1, H, 1, 1) for n, x in inp.items()}
    _, _, small = lib.gdr_step(*(inp[n] for n in NAMES), inp["state"], per_position=True)
    _, _, pos = lib.gdr_step(*(wide[n] for n in NAMES), wide["state"], per_position=True)
    assert pos.numel() > 2 ** 32
    assert torch.equal(pos[0, :, -1], small[0, :, 0]) and torch.equal(pos[0, -1, H // 2], small[0, -1, 0])
    del pos, wide
    T, H = 2 ** 20 + 64, 64
    gen = torch.Generator(device="cuda").manual_seed(4)
    v = torch.randn(1, T, H, 64, generator=gen, device="cuda", dtype=torch.bfloat16)
    assert v.numel() > 2 ** 32
    q, k = (torch.nn.functional.normalize(torch.randn(1, T, 1, 64, generator=gen, device="cuda"), dim=-1).bfloat16()
            for _ in range(2))
    g = -0.05 * torch.rand(1, T, H, generator=gen, device="cuda")
    beta = torch.rand(1, T, H, generator=gen, device="cuda")
    o, s = lib.gdr_forward(q, k, v, g, beta, o_dtype=torch.bfloat16)
    cut = 2 ** 20       # the same from there on, from the state at the cut (a multiple of the chunk)
    _, mid = lib.gdr_forward(*(x[:, :cut] for x in (q, k, v, g, beta)))
    o2, s2 = lib.gdr_forward(*(x[:, cut:].contiguous() for x in (q, k, v, g, beta)), mid)
    check(s, s2.double().cpu().numpy(), TOL, "state", HEADS_STATE)
    check(o[:, cut:], o2.double().cpu().numpy(), TOL + BF16, "o", HEADS_SEQ, BF16)


def test_refusals(lib):
    d = on_gpu(make(2, 12, 2, 4, 64, 64))
    args = [d[n] for n in NAMES]
    with pytest.raises(ValueError):
        lib.gdr_forward(*args[:2], args[2].transpose(1, 2), *args[3:])
    with pytest.raises(ValueError):
        lib.gdr_forward(args[0], args[1][:, :, :1].contiguous(), *args[2:])
    with pytest.raises(ValueError):
        lib.gdr_forward(*args[:3], args[3].double(), args[4])
    with pytest.raises(TypeError):
        lib.gdr_forward(args[0].half(), args[1].half(), args[2].half(), *args[3:])
    with pytest.raises(ValueError):
        lib.gdr_forward(*args, d["state"][:, :, :32].contiguous())
    with pytest.raises(ValueError):
        lib.gdr_step(*args, o=torch.empty(2, 12, 4, 32, device="cuda"))
    with pytest.raises(ValueError):
        lib.gdr_step(*args, write_state_out=False)
    with pytest.raises(lib.Wkv7Error):   # 96 channels
        x = on_gpu(make(1, 4, 1, 1, 96, 64))
        lib.gdr_forward(*(x[n] for n in NAMES), x["state"])
    with pytest.raises(lib.Wkv7Error):   # o on top of v
        y = on_gpu(make(2, 12, 2, 4, 64, 64, dtype="fp32"))
        lib.gdr_forward(*(y[n] for n in NAMES), o=y["v"])
