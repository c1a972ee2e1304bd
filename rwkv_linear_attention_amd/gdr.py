"""The gated delta rule: the binding of ``include/gdr.h``.

Per batch row b and value head h a [K, V] fp32 state S (row = key channel) follows

    S_t = exp(g_t) (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,   o_t = scale S_t^T q_t

Tensors, all contiguous and on one GPU: q, k [B, T, Hk, K] and v [B, T, H, V], bf16 or
fp32; g (log decays) and beta [B, T, H] fp32; states [B, H, K, V] fp32.  Hk divides H:
value heads h // (H / Hk) share a query / key head.  K is 64 or 128, V a multiple of 64
up to 512.  scale defaults to K ** -0.5.  Calls run on the current stream of the tensors'
device.  Like the rest of this package these functions record no autograd graph: training
code pairs gdr_forward_ckpt with gdr_backward_ckpt.
"""
from __future__ import annotations

import ctypes

import torch

from . import _check, _dt, _int_rows, _out_arg, _ptr, _state_arg, _stream, lib

F32 = (torch.float32,)
BLOCK = 64  # tokens between two checkpoints


def _on(device):
    """The device's own context, where another device is current."""
    if device.index is None or device.index == torch.cuda.current_device():
        return _SAME
    return torch.cuda.device(device)


class _Same:
    def __enter__(self):
        return self

    def __exit__(self, *_):
        return False


_SAME = _Same()


def _check_qk(q, k, g, beta, H):
    if q.dim() != 4:
        raise ValueError(f"q must be [B, T, Hk, K], got {tuple(q.shape)}")
    B, T, Hk, K = q.shape
    dev = q.device
    if not q.is_cuda:
        raise ValueError("inputs must be on the GPU")
    _dt(q)
    if k.shape != q.shape or k.dtype != q.dtype or k.device != dev:
        raise ValueError("q and k must share shape, dtype and device")
    if not (q.is_contiguous() and k.is_contiguous()):
        raise ValueError("inputs must be contiguous")
    if Hk < 1 or H % Hk:
        raise ValueError(f"the {Hk} query / key heads must divide the {H} value heads")
    for name, x in (("g", g), ("beta", beta)):
        _out_arg(x, (B, T, H), dev, name, F32)
    return B, T, Hk, K, dev


def _check_inputs(q, k, v, g, beta):
    if v.dim() != 4:
        raise ValueError(f"v must be [B, T, H, V], got {tuple(v.shape)}")
    H, V = v.shape[2:]
    B, T, Hk, K, dev = _check_qk(q, k, g, beta, H)
    if tuple(v.shape[:2]) != (B, T) or v.dtype != q.dtype or v.device != dev:
        raise ValueError("v must match q in batch, tokens, dtype and device")
    if not v.is_contiguous():
        raise ValueError("inputs must be contiguous")
    return B, T, Hk, H, K, V, dev


def _new(shape, device, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device=device)


def _scale(scale, K):
    return ctypes.c_float(K ** -0.5 if scale is None else float(scale))


def gdr_forward(q, k, v, g, beta, state_in=None, *, scale=None, o_dtype=torch.float32, o=None, state_out=None,
                lengths=None):
    """Parallel pass over the whole sequence.  Returns (o, state_out).

    state_out may be passed as state_in itself to update the state in place.
    With lengths ([B] integers), row b runs its first lengths[b] tokens (clamped
    to [0, T]); o[b, t] for t >= lengths[b] is left as it was.
    """
    B, T, Hk, H, K, V, dev = _check_inputs(q, k, v, g, beta)
    state_in = _state_arg(state_in, B, H, K, dev, "state_in", V)
    state_out = _new((B, H, K, V), dev) if state_out is None else state_out
    _state_arg(state_out, B, H, K, dev, "state_out", V)
    o = _new((B, T, H, V), dev, o_dtype) if o is None else o
    _out_arg(o, (B, T, H, V), dev, "o")
    with _on(dev):
        lengths = None if lengths is None else _int_rows(lengths, B, dev, "lengths")
        _check(lib().gdr_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _dt(q), _ptr(state_in), _ptr(o),
                                 _dt(o), _ptr(state_out), _ptr(lengths), _scale(scale, K), B, T, Hk, H, K, V,
                                 _stream(dev)))
    return o, state_out


def gdr_step(q, k, v, g, beta, state_in=None, *, scale=None, per_position=False, o_dtype=torch.float32, o=None,
             state_out=None, state_pos=None, write_state_out=True):
    """Recurrent pass, token by token.  Returns (o, state_out) or (o, state_out, state_pos).

    With per_position=True, state_pos[:, t] is the state after token t (wkv7_state_commit
    keeps an accepted prefix of them); then write_state_out=False skips the separate final
    state (state_out is None).
    """
    B, T, Hk, H, K, V, dev = _check_inputs(q, k, v, g, beta)
    state_in = _state_arg(state_in, B, H, K, dev, "state_in", V)
    if not write_state_out:
        if not (per_position or state_pos is not None) or state_out is not None:
            raise ValueError("write_state_out=False needs per-position states and no state_out")
    elif state_out is None:
        state_out = _new((B, H, K, V), dev)
    _state_arg(state_out, B, H, K, dev, "state_out", V)
    o = _new((B, T, H, V), dev, o_dtype) if o is None else o
    _out_arg(o, (B, T, H, V), dev, "o")
    if per_position and state_pos is None:
        state_pos = _new((B, T, H, K, V), dev)
    if state_pos is not None:
        _out_arg(state_pos, (B, T, H, K, V), dev, "state_pos", F32)
    with _on(dev):
        _check(lib().gdr_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _dt(q), _ptr(state_in), _ptr(o),
                              _dt(o), _ptr(state_out), _ptr(state_pos), _scale(scale, K), B, T, Hk, H, K, V,
                              _stream(dev)))
    return (o, state_out) if state_pos is None else (o, state_out, state_pos)


def _nblocks(T):
    return -(-T // BLOCK)


def gdr_forward_ckpt(q, k, v, g, beta, state_in=None, *, scale=None, o=None, state_out=None, ckpt=None,
                     resid=None):
    """Forward pass for training: (o, state_out, ckpt, resid), o in fp32.

    ckpt [B, ceil(T/64), H, K*V] fp32 (the state before every 64 tokens, in an order of
    the library's own) and resid [B, T, H, V] fp32 (every token's v - exp(g) S^T k) are what
    gdr_backward_ckpt reads.
    """
    B, T, Hk, H, K, V, dev = _check_inputs(q, k, v, g, beta)
    state_in = _state_arg(state_in, B, H, K, dev, "state_in", V)
    state_out = _new((B, H, K, V), dev) if state_out is None else state_out
    _state_arg(state_out, B, H, K, dev, "state_out", V)
    o = _new((B, T, H, V), dev) if o is None else o
    _out_arg(o, (B, T, H, V), dev, "o", F32)
    ckpt = _new((B, _nblocks(T), H, K * V), dev) if ckpt is None else ckpt
    _out_arg(ckpt, (B, _nblocks(T), H, K * V), dev, "ckpt", F32)
    resid = _new((B, T, H, V), dev) if resid is None else resid
    _out_arg(resid, (B, T, H, V), dev, "resid", F32)
    with _on(dev):
        _check(lib().gdr_forward_ckpt(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _dt(q), _ptr(state_in),
                                      _ptr(o), _ptr(state_out), _ptr(ckpt) if T else None,
                                      _ptr(resid) if T else None, _scale(scale, K), B, T, Hk, H, K, V, _stream(dev)))
    return o, state_out, ckpt, resid


def gdr_backward_ckpt(q, k, g, beta, ckpt, resid, d_o, d_state_out=None, *, scale=None, grads=None, work=None):
    """Gradients of the gated delta rule from what gdr_forward_ckpt kept of the same inputs.

    d_o [B, T, H, V] fp32; d_state_out [B, H, K, V] fp32 or None (zeros).  Returns a dict of
    fp32 gradients: dq, dk [B, T, Hk, K] (summed over each group's value heads), dv
    [B, T, H, V], dg, dbeta [B, T, H] and d_state_in [B, H, K, V]; ``grads`` may pass that
    dict preallocated, ``work`` a scratch tensor of ckpt's shape.
    """
    if d_o.dim() != 4:
        raise ValueError(f"d_o must be [B, T, H, V], got {tuple(d_o.shape)}")
    H, V = d_o.shape[2:]
    B, T, Hk, K, dev = _check_qk(q, k, g, beta, H)
    _out_arg(d_o, (B, T, H, V), dev, "d_o", F32)
    d_state_out = _state_arg(d_state_out, B, H, K, dev, "d_state_out", V)
    _out_arg(ckpt, (B, _nblocks(T), H, K * V), dev, "ckpt", F32)
    _out_arg(resid, (B, T, H, V), dev, "resid", F32)
    shapes = {"dq": (B, T, Hk, K), "dk": (B, T, Hk, K), "dv": (B, T, H, V), "dg": (B, T, H), "dbeta": (B, T, H),
              "d_state_in": (B, H, K, V)}
    if grads is None:
        grads = {n: _new(s, dev) for n, s in shapes.items()}
    for n, s in shapes.items():
        _out_arg(grads[n], s, dev, n, F32)
    work = _new((B, _nblocks(T), H, K * V), dev) if work is None else work
    _out_arg(work, (B, _nblocks(T), H, K * V), dev, "work", F32)
    with _on(dev):
        _check(lib().gdr_backward_ckpt(_ptr(q), _ptr(k), _ptr(g), _ptr(beta), _dt(q), *[_ptr(x) if T else None for x in (ckpt, resid, d_o)],
                                       _ptr(d_state_out), *[_ptr(grads[n]) for n in shapes],
                                       _ptr(work) if T else None, _scale(scale, K), B, T, Hk, H, K, V, _stream(dev)))
    return grads
