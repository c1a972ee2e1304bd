"""Timed cases of the gated delta rule and of draft verification.

Every case runs one pass of an operator in one of two forms: the plain form below
(elementary torch operations in 32 bits, 64 for the vocabulary sums), or, with
``own`` set, this library's entry points.  The gated delta rule keeps, per batch
row and value head, a [K, V] state S and computes

    S_t = exp(g_t) (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T
    o_t = scale S_t^T q_t

Groups of H / Hk value heads share one query / key head.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
CHUNK = 64
NOTHING = 2.0 ** -7  # what an output row behind its sequence holds before the call


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _seq(name, op, B, T, Hk, H, K, V, dtype="bf16", out="bf16", **more):
    return {"name": name, "op": op, "B": B, "T": T, "Hk": Hk, "H": H, "K": K, "V": V, "dtype": dtype,
            "out": out, **more}


def listed():
    return [
        # a short chat turn, one row: the fewest tokens that go through the chunked pass
        _seq("prefill-short", "prefill", 1, 37, 12, 12, 64, 64),
        # the 0.1B-shaped prefill: few heads, so the walk along the sequence bounds it
        _seq("prefill-0.1B", "prefill", 8, 4096, 12, 12, 64, 64),
        # the 7.2B-wide prefill with 128-channel heads, two value heads to a key head
        _seq("prefill-7.2B", "prefill", 4, 8192, 16, 32, 128, 128),
        # right-padded prompts of unequal lengths, empty rows among them, three value heads to a key head
        _seq("prefill-ragged", "prefill", 7, 1531, 7, 21, 128, 128, ragged=True),
        # fp32 activations (an evaluation run), unequal key and value widths
        _seq("prefill-fp32", "prefill", 2, 513, 6, 6, 64, 128, dtype="fp32", out="fp32"),
        # one stream's next token: launch and latency
        _seq("decode-one", "step", 1, 1, 16, 32, 128, 128),
        # a serving batch's next token: the states' traffic
        _seq("decode-batch", "step", 32, 1, 20, 40, 128, 128),
        # a drafted run of five tokens to verify, the state after each kept for the commit
        _seq("verify-states", "step", 16, 5, 16, 32, 128, 128, per_position=True),
        # a training step of a small model's layer: forward and gradients, few heads
        _seq("train-0.1B", "train", 8, 1024, 12, 12, 64, 64, out="fp32"),
        # a training step with wide heads and shared keys
        _seq("train-7.2B", "train", 2, 4096, 16, 32, 128, 128, out="fp32"),
        # one stream's drafted tokens against a 65536-entry vocabulary
        {"name": "draft-one", "op": "draft", "B": 1, "N": 4, "vocab": 65536, "dtype": "fp32", "ragged": False,
         "greedy": False},
        # a serving batch's drafts, unequal numbers of them
        {"name": "draft-batch", "op": "draft", "B": 64, "N": 4, "vocab": 65536, "dtype": "fp32", "ragged": True,
         "greedy": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "step", "train", "draft"])
    if op == "draft":
        return {"op": op, "B": _log(rng, 1, 64), "N": rng.randint(1, 8), "vocab": _log(rng, 1000, 131072),
                "dtype": rng.choice(["fp32", "bf16"]), "ragged": rng.random() < 0.5, "greedy": rng.random() < 0.3}
    K, V = rng.choice([64, 128]), rng.choice([64, 128, 192, 256])
    Hk = rng.randint(1, 24)
    H = Hk * rng.choice([1, 2, 3])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "step":
        T, per = rng.choice([(1, False), (1, False), (rng.randint(2, 8), True)])
        most = 160e6 / (H * K * V * (T if per else 1))
        return {"op": op, "B": _log(rng, 1, max(1, min(64, most))), "T": T, "Hk": Hk, "H": H, "K": K, "V": V,
                "dtype": dtype, "out": rng.choice(["bf16", "fp32"]), "per_position": per}
    tokens = (2.5e9 if op == "prefill" else 0.9e9) / (H * K * V)  # B T at most, by the largest case's work
    T = _log(rng, 9, max(10, min(8192, tokens)))
    return {"op": op, "B": _log(rng, 1, max(1, min(8, tokens / T))), "T": T, "Hk": Hk, "H": H, "K": K, "V": V,
            "dtype": dtype, "out": "fp32" if op == "train" else rng.choice(["bf16", "fp32"]),
            "ragged": op == "prefill" and rng.random() < 0.4}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=DEV)

    dt = DTYPES[case["dtype"]]
    if case["op"] == "draft":
        B, N, vocab = case["B"], case["N"], case["vocab"]
        # a target peaked like a language model's, and a drafter near it
        base = normal(B, N + 1, vocab) * 3.0
        target = torch.softmax(base, -1)
        near = torch.softmax(base[:, :N] + 0.5 * normal(B, N, vocab), -1)
        tokens = torch.multinomial(near.reshape(B * N, vocab), 1, generator=gen).reshape(B, N).to(torch.int32)
        n_draft = torch.randint(0, N + 1, (B,), generator=gen, device=DEV).to(torch.int32) if case["ragged"] else None
        return {"case": case, "target": target.to(dt), "draft": None if case["greedy"] else near.to(dt),
                "tokens": tokens, "u": uniform(B, N), "u_draw": uniform(B), "n_draft": n_draft}

    B, T, Hk, H, K, V = (case[n] for n in ("B", "T", "Hk", "H", "K", "V"))
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    s = {"case": case, "scale": K ** -0.5,
         "q": unit(normal(B, T, Hk, K)).to(dt), "k": unit(normal(B, T, Hk, K)).to(dt), "v": normal(B, T, H, V).to(dt),
         # log decays -softplus, heads from short to long memories; writing strengths a sigmoid
         "g": -torch.nn.functional.softplus(normal(B, T, H) - 2.0) * torch.exp(-3.0 * uniform(H)),
         "beta": torch.sigmoid(normal(B, T, H)), "state": 0.1 * normal(B, H, K, V), "lengths": None}
    out = DTYPES[case["out"]]
    s["o"] = torch.full((B, T, H, V), NOTHING, dtype=out, device=DEV)
    s["state_out"] = torch.empty_like(s["state"])
    if case.get("ragged"):
        lengths = torch.randint(0, T + 1, (B,), generator=gen, device=DEV)
        lengths[0] = T
        if B > 2:
            lengths[B // 2] = 0
        s["lengths"] = lengths.to(torch.int32)
    if case.get("per_position"):
        s["state_pos"] = torch.empty((B, T, H, K, V), device=DEV)
    if case["op"] == "train":
        s["d_o"] = normal(B, T, H, V)
        s["d_state"] = 0.1 * normal(B, H, K, V)
        chunks = -(-T // CHUNK)
        s["ckpt"] = torch.empty((B, chunks, H, K * V), device=DEV)
        s["resid"] = torch.empty((B, T, H, V), device=DEV)
        s["work"] = torch.empty((B, chunks, H, K * V), device=DEV)
        f32 = {"device": DEV, "dtype": torch.float32}
        s["grads"] = {"dq": torch.empty((B, T, Hk, K), **f32), "dk": torch.empty((B, T, Hk, K), **f32),
                      "dv": torch.empty((B, T, H, V), **f32), "dg": torch.empty((B, T, H), **f32),
                      "dbeta": torch.empty((B, T, H), **f32), "d_state_in": torch.empty((B, H, K, V), **f32)}
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        import rwkv_linear_attention_amd as lib
        if op == "prefill":
            return lib.gdr_forward(state["q"], state["k"], state["v"], state["g"], state["beta"], state["state"],
                                   scale=state["scale"], o=state["o"], state_out=state["state_out"],
                                   lengths=state["lengths"])
        if op == "step":
            return lib.gdr_step(state["q"], state["k"], state["v"], state["g"], state["beta"], state["state"],
                                scale=state["scale"], o=state["o"], state_out=state["state_out"],
                                state_pos=state.get("state_pos"))
        if op == "train":
            o, s, ckpt, resid = lib.gdr_forward_ckpt(
                state["q"], state["k"], state["v"], state["g"], state["beta"], state["state"], scale=state["scale"],
                o=state["o"], state_out=state["state_out"], ckpt=state["ckpt"], resid=state["resid"])
            grads = lib.gdr_backward_ckpt(state["q"], state["k"], state["g"], state["beta"], ckpt, resid,
                                          state["d_o"], state["d_state"], scale=state["scale"],
                                          grads=state["grads"], work=state["work"])
            return o, s, grads
        return lib.draft_verify(state["target"], state["tokens"], state["u"], state["u_draw"],
                                draft=state["draft"], n_draft=state["n_draft"])
    if op == "prefill":
        return _plain_prefill(state)
    if op == "step":
        return _plain_step(state)
    if op == "train":
        return _plain_train(state)
    return _plain_draft(state)


def _heads(x, H):
    """[B, T, Hk, K] to one query / key head per value head, in 32 bits."""
    return x.float().repeat_interleave(H // x.shape[2], dim=2)


def _unit_lower_inverse(M):
    """(I + M)^-1 of strictly lower triangular M: (I - M)(I + M^2)(I + M^4)..."""
    eye = torch.eye(M.shape[-1], device=M.device)
    inv, power = eye - M, M @ M
    for _ in range(int(math.log2(M.shape[-1])) - 1):
        inv, power = inv + inv @ power, power @ power
    return inv


def _chunked(q, k, v, g, beta, S, scale):
    """The rule over chunks of 64 tokens: everything that needs no state at once, then the states chunk by chunk."""
    B, T, H, K = q.shape
    n = -(-T // CHUNK)
    pad = lambda x: torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, n * CHUNK - T))  # noqa: E731
    cut = lambda x: pad(x).reshape(B, n, CHUNK, *x.shape[2:]).transpose(2, 3).contiguous()  # noqa: E731
    q, k, v, g, beta = cut(q) * scale, cut(k), cut(v), cut(g), cut(beta)   # [B, n, H, C, ...]
    total = torch.cumsum(g, -1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    decay = torch.exp((total[..., :, None] - total[..., None, :]).masked_fill(~low, 0.0)) * low
    M = (beta[..., None] * decay * (k @ k.transpose(-1, -2))).tril(-1)
    solve = _unit_lower_inverse(M) * beta[..., None, :]
    U0, W = solve @ v, solve @ (k * torch.exp(total)[..., None])
    A = decay * (q @ k.transpose(-1, -2))
    into, onto = q * torch.exp(total)[..., None], k * torch.exp(total[..., -1:] - total)[..., None]
    last = torch.exp(total[..., -1])[..., None, None]
    outs = []
    for c in range(n):
        U = U0[:, c] - W[:, c] @ S
        outs.append(into[:, c] @ S + A[:, c] @ U)
        S = last[:, c] * S + onto[:, c].transpose(-1, -2) @ U
    o = torch.stack(outs, 1).transpose(2, 3).reshape(B, n * CHUNK, H, v.shape[-1])
    return o[:, :T], S


def _plain_prefill(s):
    H, T = s["case"]["H"], s["case"]["T"]
    g, beta = s["g"], s["beta"]
    if s["lengths"] is not None:  # a token behind its row's end neither decays nor writes
        inside = (torch.arange(T, device=g.device) < s["lengths"][:, None])[..., None]
        g, beta = g * inside, beta * inside
    o, S = _chunked(_heads(s["q"], H), _heads(s["k"], H), s["v"].float(), g, beta, s["state"], s["scale"])
    o = o.to(s["o"].dtype)
    return (o if s["lengths"] is None else torch.where(inside[..., None], o, s["o"])), S


def _plain_step(s):
    H = s["case"]["H"]
    q, k, v, S = _heads(s["q"], H) * s["scale"], _heads(s["k"], H), s["v"].float(), s["state"]
    outs, states = [], []
    for t in range(q.shape[1]):
        S = S * torch.exp(s["g"][:, t])[..., None, None]
        u = s["beta"][:, t, :, None] * (v[:, t] - (k[:, t, :, :, None] * S).sum(-2))
        S = S + k[:, t, :, :, None] * u[..., None, :]
        outs.append((q[:, t, :, :, None] * S).sum(-2))
        states.append(S)
    o = torch.stack(outs, 1).to(s["o"].dtype)
    return (o, S, torch.stack(states, 1)) if "state_pos" in s else (o, S)


def _plain_train(s):
    H = s["case"]["H"]
    leaves = {n: s[n].float().requires_grad_() for n in ("q", "k", "v")}
    leaves |= {n: s[n].clone().requires_grad_() for n in ("g", "beta", "state")}
    o, S = _chunked(_heads(leaves["q"], H), _heads(leaves["k"], H), leaves["v"], leaves["g"], leaves["beta"],
                    leaves["state"], s["scale"])
    grads = torch.autograd.grad((o, S), tuple(leaves.values()), (s["d_o"], s["d_state"]))
    return o.detach(), S.detach(), dict(zip(("dq", "dk", "dv", "dg", "dbeta", "d_state_in"), grads))


def _clean(x):
    """A probability in 64 bits; what is no positive finite number weighs nothing."""
    x = x.double()
    return torch.where((x > 0) & (x < math.inf), x, 0.0)


def _plain_draft(s):
    target, draft, tokens = _clean(s["target"]), s["draft"], s["tokens"]
    B, N = tokens.shape
    given = torch.full((B,), N, device=DEV) if s["n_draft"] is None else s["n_draft"].long()
    at = tokens.long()[..., None]
    if draft is None:  # the drafter is sure of its token
        draft = torch.zeros_like(target[:, :N]).scatter_(-1, at, 1.0)
    else:
        draft = _clean(draft)
    j = torch.arange(N, device=DEV)
    ok = s["u"].double() * draft.gather(-1, at)[..., 0] < target[:, :N].gather(-1, at)[..., 0]
    n = torch.where((j < given[:, None]) & ~ok, j, N).amin(1).minimum(given)
    rows = torch.arange(B, device=DEV)
    p = target[rows, n]
    q = draft[rows, n.clamp(max=N - 1)] * (n < given)[:, None]
    weight = (p - q).clamp(min=0.0)
    weight = torch.where(weight.sum(-1, keepdim=True) > 0, weight, p)
    upto = torch.cumsum(weight, -1)
    last = torch.where(weight > 0, torch.arange(weight.shape[1], device=DEV), -1).amax(1)
    drawn = (upto <= (s["u_draw"].double() * upto[:, -1])[:, None]).sum(1).minimum(last)
    place = torch.arange(N + 1, device=DEV)
    filled = torch.cat([tokens.long(), tokens.new_zeros((B, 1)).long()], 1)
    out = torch.where(place < n[:, None], filled, torch.where(place == n[:, None], drawn[:, None], -1))
    return out.to(torch.int32), (n + 1).to(torch.int32)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    size = {"bf16": 2, "fp32": 4}
    if case["op"] == "draft":
        # the rows drawn from; the probabilities of single tokens are a few bytes
        rows = case["B"] * (1 if case["greedy"] else 2)
        return {"bytes": rows * case["vocab"] * size[case["dtype"]], "flops": 2 * rows * case["vocab"]}
    B, T, Hk, H, K, V = (case[n] for n in ("B", "T", "Hk", "H", "K", "V"))
    e, f = size[case["dtype"]], size[case["out"]]
    ins = B * T * (2 * Hk * K * e + H * V * e + 2 * H * 4)
    states = B * H * K * V * 4
    forward = 6 * B * T * H * K * V  # k S, k u^T and q S, a product and a sum each
    if case["op"] == "train":
        # forward: inputs, o, the states; backward: the inputs again, d_o, five gradients, the states' gradients
        back = ins + B * T * (H * V * 4 + 2 * Hk * K * 4 + H * V * 4 + 2 * H * 4)
        return {"bytes": ins + B * T * H * V * 4 + 4 * states + back, "flops": 3 * forward}
    kept = T * states if case.get("per_position") else 0
    return {"bytes": ins + B * T * H * V * f + 2 * states + kept, "flops": forward}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "draft":
        return _exact_draft(s)
    H, T = case["H"], case["T"]
    group = torch.arange(H, device=DEV) // (H // case["Hk"])
    q, k, v = s["q"].double()[:, :, group], s["k"].double()[:, :, group], s["v"].double()
    alpha, beta = torch.exp(s["g"].double()), s["beta"].double()

    def token(S, t):
        erased = torch.einsum("bhk,bhkv->bhv", k[:, t], S) * alpha[:, t, :, None]
        write = beta[:, t, :, None] * (v[:, t] - erased)
        return torch.addcmul(alpha[:, t, :, None, None] * S, k[:, t, :, :, None], write[:, :, None, :])

    S, o, states = s["state"].double(), [], []
    keep = {0: S} if case["op"] == "train" else None
    lengths = s["lengths"]
    for t in range(T):
        new = token(S, t)
        S = new if lengths is None else torch.where((t < lengths)[:, None, None, None], new, S)
        o.append(torch.einsum("bhk,bhkv->bhv", q[:, t], S) * s["scale"])
        if keep is not None and (t + 1) % CHUNK == 0:
            keep[t + 1] = S
        if case.get("per_position"):
            states.append(S)
    o = torch.stack(o, 1)
    if lengths is not None:
        inside = torch.arange(T, device=DEV) < lengths[:, None]
        o = torch.where(inside[..., None, None], o, NOTHING)
    if case["op"] != "train":
        return (o, S, torch.stack(states, 1)) if case.get("per_position") else (o, S)

    # the adjoint of that loop, the states of each 64 tokens run again from their first
    D, d_o = s["d_state"].double(), s["d_o"].double() * s["scale"]
    dq, dk, dv, dg, dbeta = ([None] * T for _ in range(5))
    for first in range((T - 1) // CHUNK * CHUNK, -1, -CHUNK):
        run_of, R = [keep[first]], keep[first]
        for t in range(first, min(T, first + CHUNK)):
            R = token(R, t)
            run_of.append(R)
        for t in range(min(T, first + CHUNK) - 1, first - 1, -1):
            before, after = run_of[t - first], run_of[t - first + 1]
            dq[t] = torch.einsum("bhkv,bhv->bhk", after, d_o[:, t])
            D = D + q[:, t, :, :, None] * d_o[:, t, :, None, :]
            decayed = alpha[:, t, :, None, None] * before
            miss = v[:, t] - torch.einsum("bhk,bhkv->bhv", k[:, t], decayed)
            pulled = torch.einsum("bhk,bhkv->bhv", k[:, t], D)
            dbeta[t] = (pulled * miss).sum(-1)
            dv[t] = beta[:, t, :, None] * pulled
            dk[t] = (torch.einsum("bhkv,bhv->bhk", D, beta[:, t, :, None] * miss)
                     - torch.einsum("bhkv,bhv->bhk", decayed, dv[t]))
            D = D - k[:, t, :, :, None] * dv[t][:, :, None, :]
            dg[t] = (D * decayed).sum((-1, -2))
            D = alpha[:, t, :, None, None] * D
    shared = lambda x: torch.stack(x, 1).reshape(*s["q"].shape[:3], H // case["Hk"], -1).sum(3)  # noqa: E731
    grads = {"dq": shared(dq), "dk": shared(dk), "dv": torch.stack(dv, 1), "dg": torch.stack(dg, 1),
             "dbeta": torch.stack(dbeta, 1), "d_state_in": D}
    return o, S, grads


def _exact_draft(s):
    """Row by row in numpy, by the definition."""
    numbers = lambda x: None if x is None else x.double().cpu().numpy()  # noqa: E731
    target, draft, u, u_draw = (numbers(s[n]) for n in ("target", "draft", "u", "u_draw"))
    tokens = s["tokens"].cpu().numpy()
    B, N = tokens.shape
    given = np.full(B, N) if s["n_draft"] is None else s["n_draft"].cpu().numpy()
    out, kept = np.full((B, N + 1), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        n = 0
        while n < given[b]:
            q = 1.0 if draft is None else draft[b, n, tokens[b, n]]
            if not u[b, n] * q < target[b, n, tokens[b, n]]:
                break
            out[b, n] = tokens[b, n]
            n += 1
        weight = target[b, n].copy()
        if n < given[b]:
            if draft is None:
                weight[tokens[b, n]] -= 1.0
            else:
                weight -= draft[b, n]
            weight = np.maximum(weight, 0.0)
            if not weight.sum() > 0:
                weight = target[b, n]
        upto = np.cumsum(weight)
        out[b, n] = min(int(np.searchsorted(upto, u_draw[b] * upto[-1], side="right")), int(np.flatnonzero(weight)[-1]))
        kept[b] = n + 1
    return out, kept
