"""The fp64 oracles of the gated delta rule and of draft verification, on the CPU."""
import numpy as np
import pytest

import oracle
from oracle import draft, gdr
from gdr_inputs import NAMES, make


def small(seed=0, B=2, T=7, Hk=2, H=4, K=8, V=6):
    r = np.random.default_rng(seed)
    return {"q": r.normal(size=(B, T, Hk, K)), "k": 0.5 * r.normal(size=(B, T, Hk, K)), "v": r.normal(size=(B, T, H, V)),
            "g": -r.random((B, T, H)), "beta": r.random((B, T, H)), "state": r.normal(size=(B, H, K, V))}


def test_forward_is_wkv7_with_the_erased_direction_tied_to_the_key():
    """At 64 x 64 and one head per key the rule is WKV-7 with w = alpha, a = -alpha beta k, b = k, v = beta v."""
    inp = {n: gdr.as_f64(x) for n, x in make(2, 9, 3, 3, 64, 64, seed=3, dtype="fp32").items()}
    alpha, beta = np.exp(inp["g"])[..., None], inp["beta"][..., None]
    w = np.broadcast_to(alpha, inp["k"].shape).copy()
    o7, s7 = oracle.forward(inp["q"], w, inp["k"], beta * inp["v"], -alpha * beta * inp["k"], inp["k"].copy(), inp["state"],
                           f64_inputs=True)
    o, s, _ = gdr.forward(*(inp[n] for n in NAMES), inp["state"])
    np.testing.assert_allclose(o, o7, rtol=0, atol=1e-13)
    np.testing.assert_allclose(s, s7, rtol=0, atol=1e-13)


def test_lengths_stop_the_rows():
    inp = small()
    o, s, states = gdr.forward(*(inp[n] for n in NAMES), inp["state"], lengths=[0, 4])
    assert not o[0].any() and not o[1, 4:].any()
    np.testing.assert_array_equal(s[0], inp["state"][0])
    np.testing.assert_array_equal(s[1], states[1, 3])


@pytest.mark.parametrize("name", NAMES + ("state",))
def test_gradients_against_differences(name):
    inp, r = small(), np.random.default_rng(9)
    d_o, d_s = r.normal(size=inp["v"].shape), r.normal(size=inp["state"].shape)
    got = gdr.backward(*(inp[n] for n in NAMES), inp["state"], d_o, d_s, scale=0.7)
    got = got["d_state_in" if name == "state" else "d" + name]

    def loss(x):
        o, s, _ = gdr.forward(*((x if n == name else inp[n]) for n in NAMES), x if name == "state" else inp["state"],
                              scale=0.7)
        return (o * d_o).sum() + (s * d_s).sum()

    flat = inp[name].reshape(-1)
    for at in r.choice(flat.size, min(25, flat.size), replace=False):
        e = np.zeros(flat.size)
        e[at] = 1e-6
        e = e.reshape(inp[name].shape)
        want = (loss(inp[name] + e) - loss(inp[name] - e)) / 2e-6
        # differences of a loss of order 1e2 at steps of 1e-6: rounding 1e-14 * 1e2 / 1e-6
        assert abs(got.reshape(-1)[at] - want) < 1e-6 + 1e-6 * abs(want)


def test_drafts_worked_by_hand():
    """Three tokens, two drafts; the numbers are chosen so that every step can be done on paper."""
    target = np.array([[[0.5, 0.25, 0.25], [0.125, 0.375, 0.5], [0.0, 0.5, 0.5]]])
    draft_p = np.array([[[0.25, 0.5, 0.25], [0.5, 0.25, 0.25]]])
    # draft 0 = token 1: 0.5 u < 0.25 for u < 0.5
    out, kept = draft.verify(target, [[1, 0]], [[0.5, 0.0]], [0.0], draft_p)
    assert kept[0] == 1 and list(out[0]) == [0, -1, -1]      # weights (0.25, 0, 0)
    # accepted, then token 0: 0.5 u < 0.125 for u < 0.25; weights (0, 0.125, 0.25)
    out, kept = draft.verify(target, [[1, 0]], [[0.49, 0.25]], [0.3], draft_p)
    assert kept[0] == 2 and list(out[0]) == [1, 1, -1]
    out, kept = draft.verify(target, [[1, 0]], [[0.49, 0.25]], [0.34], draft_p)
    assert list(out[0]) == [1, 2, -1]
    # both accepted: a draw from (0, 0.5, 0.5); the mark itself is not passed
    out, kept = draft.verify(target, [[1, 0]], [[0.0, 0.0]], [0.5], draft_p)
    assert kept[0] == 3 and list(out[0]) == [1, 0, 2]
    # a sure drafter, refused: its token's mass is gone
    out, kept = draft.verify(target, [[1, 0]], [[0.25, 0.0]], [0.99], None)
    assert kept[0] == 1 and list(out[0]) == [2, -1, -1]


def test_verified_tokens_follow_the_target():
    """Over many uniform numbers the first emitted token has the target's distribution, whatever the drafter's."""
    rng, n, vocab = np.random.default_rng(4), 40000, 5
    p, q = rng.dirichlet(np.ones(vocab)), rng.dirichlet(np.ones(vocab))
    tokens = rng.choice(vocab, size=(n, 1), p=q)
    target = np.broadcast_to(p, (n, 2, vocab))
    out, _ = draft.verify(target, tokens, rng.random((n, 1)), rng.random(n), np.broadcast_to(q, (n, 1, vocab)))
    share = np.bincount(out[:, 0], minlength=vocab) / n
    assert np.all(np.abs(share - p) < 5 * np.sqrt(p * (1 - p) / n))  # five standard deviations
