"""GPU parity of draft_verify with the fp64 oracle: whole numbers, so equality."""
import numpy as np
import pytest
import torch

from oracle import draft as oracle_draft

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import rwkv_linear_attention_amd as m
    m.lib()
    return m


def make(B, N, vocab, seed=0, dtype=torch.float32, near=0.4):
    gen = torch.Generator().manual_seed(seed)
    base = 3 * torch.randn(B, N + 1, vocab, generator=gen)
    target = torch.softmax(base, -1)
    draft = torch.softmax(base[:, :N] + near * torch.randn(B, N, vocab, generator=gen), -1)
    tokens = torch.zeros(B, N, dtype=torch.int32)
    if N:
        tokens = torch.multinomial(draft.reshape(B * N, vocab), 1, generator=gen).reshape(B, N).to(torch.int32)
    return {"target": target.to(dtype), "draft": draft.to(dtype), "tokens": tokens,
            "u": torch.rand(B, N, generator=gen), "u_draw": torch.rand(B, generator=gen)}


def both(lib, x, sure=False, n_draft=None):
    draft = None if sure else x["draft"]
    as64 = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    want = oracle_draft.verify(as64(x["target"]), x["tokens"].numpy(), as64(x["u"]), as64(x["u_draw"]), as64(draft),
                               n_draft)
    got = lib.draft_verify(x["target"].cuda(), x["tokens"].cuda(), x["u"].cuda(), x["u_draw"].cuda(),
                           draft=None if draft is None else draft.cuda(),
                           n_draft=None if n_draft is None else torch.tensor(n_draft))
    assert got[0].dtype == torch.int32 and got[1].dtype == torch.int32
    np.testing.assert_array_equal(got[1].cpu().numpy(), want[1])
    np.testing.assert_array_equal(got[0].cpu().numpy(), want[0])
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sure", [False, True])
@pytest.mark.parametrize("B,N,vocab", [(1, 1, 1), (2, 3, 7), (5, 4, 63), (4, 2, 64), (3, 1, 65), (3, 5, 1000),
                                       (2, 2, 4096), (6, 3, 65536), (2, 1, 131071), (3, 0, 777), (1, 40, 33)])
def test_against_the_oracle(lib, B, N, vocab, sure, dtype):
    both(lib, make(B, N, vocab, seed=B + vocab, dtype=dtype), sure)


@pytest.mark.parametrize("vocab,dtype", [(140008, torch.bfloat16), (200000, torch.float32), (262147, torch.bfloat16)])
def test_runs_longer_than_one_reading(lib, vocab, dtype):
    x = make(2, 2, vocab, seed=11, dtype=dtype)
    for sure in (False, True):
        both(lib, x, sure)
    x["target"][:, :, ::7] = float("inf")   # stretches that hold what is no probability
    x["draft"][:, :, 5::1001] = -0.0
    both(lib, x)


def test_row_by_row_numbers_of_drafts(lib):
    x = make(6, 3, 500, seed=2, near=0.05)
    both(lib, x, n_draft=[0, 1, 2, 3, -4, 9])
    x["u"][:] = 0.0     # every draft accepted
    _, kept = both(lib, x, n_draft=[0, 1, 2, 3, -4, 9])
    assert kept.tolist() == [1, 2, 3, 4, 1, 4]
    x["u"][:] = 1e30    # every draft refused
    _, kept = both(lib, x)
    assert kept.tolist() == [1] * 6


def test_the_ends_of_the_draw(lib):
    x = make(5, 1, 300, seed=3)
    x["u_draw"] = torch.tensor([0.0, 1.0, 2.0, -1.0, float("nan")])
    x["target"][:, :, :10] = 0.0
    x["target"][:, :, -20:] = 0.0
    both(lib, x)
    x["u"][:] = 0.0
    out, _ = both(lib, x)
    assert out[0, 1] == 10 and out[3, 1] == 10 and out[1, 1] == 279 and out[4, 1] == 279


def test_rows_that_leave_nothing(lib):
    x = make(4, 2, 200, seed=4)
    x["u"][:] = 1e30
    x["draft"][0] = x["target"][0, :2]      # nothing left of max(p - q, 0): p itself
    x["target"][1] = 0.0                    # no mass at all: -1
    x["target"][2] = float("nan")
    out, kept = both(lib, x)
    assert out[1, 0] == -1 and out[2, 0] == -1 and out[0, 0] >= 0 and kept.tolist() == [1] * 4
    both(lib, x, sure=True)


def test_entries_that_are_no_probabilities(lib):
    x = make(3, 2, 400, seed=5)
    x["target"][:, :, 3] = float("inf")
    x["target"][:, :, 4] = float("nan")
    x["target"][:, :, 5] = -1.0
    x["draft"][:, :, 6] = float("nan")
    x["draft"][:, :, 7] = float("inf")
    both(lib, x)
    both(lib, x, sure=True)


def test_tokens_outside_the_vocabulary_are_refused(lib):
    x = make(3, 2, 100, seed=6)
    x["tokens"][0, 0], x["tokens"][1, 1], x["tokens"][2, 0] = -1, 100, 2 ** 30
    x["u"][:] = 0.0
    for sure in (False, True):
        _, kept = both(lib, x, sure)
        assert kept.tolist() == [1, 2, 1]


def test_one_token_with_all_the_mass(lib):
    x = make(4, 1, 70000, seed=7)
    x["target"][:] = 0.0
    for b, at in enumerate((0, 69999, 1093, 1094)):
        x["target"][b, :, at] = 1.0
    out, _ = both(lib, x, sure=True)
    assert sorted(set(out[:, 0].tolist())) == [0, 1093, 1094, 69999]


@pytest.mark.parametrize("vocab,dtype", [(63, torch.float32), (4096, torch.bfloat16), (1001, torch.bfloat16)])
def test_guard_bands_on_a_side_stream(lib, vocab, dtype):
    """Inputs lie in ones and tokens no vocabulary holds, outputs in a pattern; the stream is the caller's."""
    x = make(3, 4, vocab, seed=8, dtype=dtype)
    x["u"][:] = 0.5
    want = [t.cpu() for t in both(lib, x)]

    def guarded(t, fill):
        big = torch.full((t.numel() + 8192,), fill, dtype=t.dtype, device="cuda")
        big[4096:4096 + t.numel()] = t.reshape(-1).cuda()
        return big[4096:4096 + t.numel()].view(t.shape), big

    ins = {n: guarded(t, 1 << 30 if t.dtype == torch.int32 else 1.0)[0] for n, t in x.items()}
    out, kept = guarded(torch.zeros(3, 5, dtype=torch.int32), -7), guarded(torch.zeros(3, dtype=torch.int32), -7)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lib.draft_verify(ins["target"], ins["tokens"], ins["u"], ins["u_draw"], draft=ins["draft"], out=out[0],
                         kept=kept[0])
    side.synchronize()
    assert torch.equal(out[0].cpu(), want[0]) and torch.equal(kept[0].cpu(), want[1])
    for view, big in (out, kept):
        assert bool((big[:4096] == -7).all()) and bool((big[-4096:] == -7).all())


def test_graph_replays(lib):
    xs = [{n: t.cuda() for n, t in make(4, 3, 5000, seed=s).items()} for s in range(3)]
    args = lambda x: (x["target"], x["tokens"], x["u"], x["u_draw"])  # noqa: E731
    eager = [lib.draft_verify(*args(x), draft=x["draft"]) for x in xs]
    static = {n: t.clone() for n, t in xs[0].items()}
    out, kept = torch.empty_like(eager[0][0]), torch.empty_like(eager[0][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.draft_verify(*args(static), draft=static["draft"], out=out, kept=kept)
    for i in (1, 2, 0, 1):
        for n, t in static.items():
            t.copy_(xs[i][n])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[i][0]) and torch.equal(kept, eager[i][1])


def test_refusals(lib):
    x = {n: t.cuda() for n, t in make(2, 3, 64).items()}
    a = (x["target"], x["tokens"], x["u"], x["u_draw"])
    for bad in ((x["target"].cpu(), *a[1:]), (x["target"].transpose(1, 2), *a[1:]),
                (a[0], x["tokens"].long(), *a[2:]), (*a[:2], x["u"][:, :2], a[3]), (*a[:3], x["u_draw"].double())):
        with pytest.raises(ValueError):
            lib.draft_verify(*bad)
    with pytest.raises(ValueError):
        lib.draft_verify(*a, draft=x["draft"].bfloat16())
    with pytest.raises(TypeError):
        lib.draft_verify(x["target"].half(), *a[1:])
    with pytest.raises(lib.Wkv7Error):    # the drawn tokens over the drafted ones
        lib.draft_verify(*a, kept=x["tokens"].reshape(-1)[:2])
