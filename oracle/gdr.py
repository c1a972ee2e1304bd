"""TEST INFRASTRUCTURE ONLY: the gated delta rule in fp64 numpy, token by token.

    S_t = exp(g_t) (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,   o_t = scale S_t^T q_t

It shares no code with the GPU library.  ``backward`` is the reverse-mode adjoint of the
loop in ``forward``, pinned by finite differences.  Arrays: q, k [B, T, Hk, K], v
[B, T, H, V], g and beta [B, T, H], states [B, H, K, V].
"""
from __future__ import annotations

import numpy as np


def as_f64(x):
    if hasattr(x, "detach"):
        x = x.detach().double().cpu().numpy()
    return np.asarray(x, np.float64)


def _spread(x, H):
    return np.repeat(as_f64(x), H // x.shape[2], axis=2)


def forward(q, k, v, g, beta, state=None, scale=1.0, lengths=None):
    """(o, final state, states after each token [B, T, H, K, V]); o behind a row's length is 0."""
    v, g, beta = as_f64(v), as_f64(g), as_f64(beta)
    B, T, H, V = v.shape
    q, k = _spread(q, H), _spread(k, H)
    K = q.shape[3]
    S = np.zeros((B, H, K, V)) if state is None else as_f64(state).copy()
    o = np.zeros((B, T, H, V))
    states = np.zeros((B, T, H, K, V))
    L = np.full(B, T) if lengths is None else np.clip(np.asarray(lengths), 0, T)
    for t in range(T):
        on = t < L
        decayed = np.exp(g[on, t])[..., None, None] * S[on]
        R = v[on, t] - np.einsum("bhk,bhkv->bhv", k[on, t], decayed)
        S[on] = decayed + k[on, t][..., None] * (beta[on, t][..., None] * R)[:, :, None, :]
        o[on, t] = scale * np.einsum("bhk,bhkv->bhv", q[on, t], S[on])
        states[:, t] = S
    return o, S, states


def backward(q, k, v, g, beta, state, d_o, d_state=None, scale=1.0):
    """The gradients as a dict: dq, dk (summed over a group's heads), dv, dg, dbeta, d_state_in."""
    Hk = q.shape[2]
    _, _, states = forward(q, k, v, g, beta, state, scale)
    v, g, beta, d_o = as_f64(v), as_f64(g), as_f64(beta), as_f64(d_o)
    B, T, H, V = v.shape
    q, k = _spread(q, H), _spread(k, H)
    K = q.shape[3]
    first = np.zeros((B, H, K, V)) if state is None else as_f64(state)
    D = np.zeros((B, H, K, V)) if d_state is None else as_f64(d_state).copy()
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dg, dbeta = np.zeros_like(g), np.zeros_like(beta)
    for t in range(T - 1, -1, -1):
        before = states[:, t - 1] if t else first
        alpha = np.exp(g[:, t])[..., None, None]
        decayed = alpha * before
        R = v[:, t] - np.einsum("bhk,bhkv->bhv", k[:, t], decayed)
        b = beta[:, t][..., None]
        dq[:, t] = scale * np.einsum("bhkv,bhv->bhk", states[:, t], d_o[:, t])
        D = D + scale * q[:, t][..., None] * d_o[:, t][:, :, None, :]
        Y = np.einsum("bhk,bhkv->bhv", k[:, t], D)           # gradient of beta R
        dbeta[:, t] = (Y * R).sum(-1)
        dv[:, t] = b * Y
        dk[:, t] = np.einsum("bhkv,bhv->bhk", D, b * R) - np.einsum("bhkv,bhv->bhk", decayed, dv[:, t])
        D = D - k[:, t][..., None] * dv[:, t][:, :, None, :]  # gradient of the decayed state
        dg[:, t] = (D * decayed).sum((-1, -2))
        D = alpha * D
    group = lambda x: x.reshape(B, T, Hk, H // Hk, K).sum(3)  # noqa: E731
    return {"dq": group(dq), "dk": group(dk), "dv": dv, "dg": dg, "dbeta": dbeta, "d_state_in": D}
