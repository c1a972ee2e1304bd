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

import torch

from . import _check, _dt, _int_rows, _out_arg, _state_arg, lib

F32 = (torch.float32,)
BLOCK = 64  # tokens between two checkpoints
_f32 = torch.float32


def _on(device):
    """The device's own context, where another device is current."""
    if device.index == torch._C._cuda_getDevice():
        return _SAME
    return torch.cuda.device(device)


class _Same:
    def __enter__(self):
        return self

    def __exit__(self, *_):
        return False


_SAME = _Same()


def _stream(device):
    return torch._C._cuda_getCurrentRawStream(device.index)


def _p(x):
    return None if x is None else x.data_ptr()


# A serving step is a few microseconds of kernel: each tensor is checked in one expression, and
# only one that fails is looked at again to say why.
def _good(x, shape, dtype, device):
    return x.shape == shape and x.dtype is dtype and x.device == device and x.is_contiguous()


def _check_qk(q, k, g, beta, H):
    if q.dim() != 4:
        raise ValueError(f"q must be [B, T, Hk, K], got {tuple(q.shape)}")
    shape, dev = q.shape, q.device
    B, T, Hk, K = shape
    if not q.is_cuda:
        raise ValueError("inputs must be on the GPU")
    if not (_good(k, shape, q.dtype, dev) and q.is_contiguous()):
        if k.shape != shape or k.dtype != q.dtype or k.device != dev:
            raise ValueError("q and k must share shape, dtype and device")
        raise ValueError("inputs must be contiguous")
    if Hk < 1 or H % Hk:
        raise ValueError(f"the {Hk} query / key heads must divide the {H} value heads")
    gates = (B, T, H)
    if not (_good(g, gates, _f32, dev) and _good(beta, gates, _f32, dev)):
        _out_arg(g, gates, dev, "g", F32)
        _out_arg(beta, gates, dev, "beta", F32)
    return B, T, Hk, K, dev


def _check_inputs(q, k, v, g, beta):
    if v.dim() != 4:
        raise ValueError(f"v must be [B, T, H, V], got {tuple(v.shape)}")
    _, _, H, V = v.shape
    B, T, Hk, K, dev = _check_qk(q, k, g, beta, H)
    if not _good(v, (B, T, H, V), q.dtype, dev):
        if v.shape[0] != B or v.shape[1] != T or v.dtype != q.dtype or v.device != dev:
            raise ValueError("v must match q in batch, tokens, dtype and device")
        raise ValueError("inputs must be contiguous")
    return B, T, Hk, H, K, V, dev


def _state(x, shape, device, name, new=False):
    """A state argument, or (new) a fresh state in the place of None."""
    if x is None:
        return torch.empty(shape, dtype=_f32, device=device) if new else None
    if not _good(x, shape, _f32, device):
        B, H, K, V = shape
        _state_arg(x, B, H, K, device, name, V)
    return x


def _output(x, shape, device, name, dtype=_f32, dtypes=F32):
    """An output argument, or a fresh tensor in the place of None."""
    if x is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if torch.is_tensor(x) and x.dtype in dtypes and _good(x, shape, x.dtype, device):
        return x
    return _out_arg(x, shape, device, name, dtypes)


BOTH = (torch.float32, torch.bfloat16)


def gdr_forward(q, k, v, g, beta, state_in=None, *, scale=None, o_dtype=torch.float32, o=None, state_out=None,
                lengths=None):
    """Parallel pass over the whole sequence.  Returns (o, state_out).

    state_out may be passed as state_in itself to update the state in place.
    With lengths ([B] integers), row b runs its first lengths[b] tokens (clamped
    to [0, T]); o[b, t] for t >= lengths[b] is left as it was.
    """
    B, T, Hk, H, K, V, dev = _check_inputs(q, k, v, g, beta)
    shape = (B, H, K, V)
    state_in = _state(state_in, shape, dev, "state_in")
    state_out = _state(state_out, shape, dev, "state_out", True)
    o = _output(o, (B, T, H, V), dev, "o", o_dtype, BOTH)
    with _on(dev):
        lengths = None if lengths is None else _int_rows(lengths, B, dev, "lengths")
        _check(lib().gdr_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), _dt(q),
                                 _p(state_in), o.data_ptr(), _dt(o), state_out.data_ptr(), _p(lengths),
                                 K ** -0.5 if scale is None else scale, B, T, Hk, H, K, V, _stream(dev)))
    return o, state_out


def gdr_step(q, k, v, g, beta, state_in=None, *, scale=None, per_position=False, o_dtype=torch.float32, o=None,
             state_out=None, state_pos=None, write_state_out=True):
    """Recurrent pass, token by token.  Returns (o, state_out) or (o, state_out, state_pos).

    With per_position=True, state_pos[:, t] is the state after token t (wkv7_state_commit
    keeps an accepted prefix of them); then write_state_out=False skips the separate final
    state (state_out is None).
    """
    B, T, Hk, H, K, V, dev = _check_inputs(q, k, v, g, beta)
    shape = (B, H, K, V)
    state_in = _state(state_in, shape, dev, "state_in")
    if not write_state_out and (not (per_position or state_pos is not None) or state_out is not None):
        raise ValueError("write_state_out=False needs per-position states and no state_out")
    state_out = _state(state_out, shape, dev, "state_out", write_state_out)
    o = _output(o, (B, T, H, V), dev, "o", o_dtype, BOTH)
    if per_position or state_pos is not None:
        state_pos = _output(state_pos, (B, T, H, K, V), dev, "state_pos")
    with _on(dev):
        _check(lib().gdr_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), _dt(q),
                              _p(state_in), o.data_ptr(), _dt(o), _p(state_out), _p(state_pos),
                              K ** -0.5 if scale is None else scale, B, T, Hk, H, K, V, _stream(dev)))
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
    shape = (B, H, K, V)
    state_in = _state(state_in, shape, dev, "state_in")
    state_out = _state(state_out, shape, dev, "state_out", True)
    o = _output(o, (B, T, H, V), dev, "o")
    ckpt = _output(ckpt, (B, _nblocks(T), H, K * V), dev, "ckpt")
    resid = _output(resid, (B, T, H, V), dev, "resid")
    with _on(dev):
        _check(lib().gdr_forward_ckpt(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), _dt(q),
                                      _p(state_in), o.data_ptr(), state_out.data_ptr(), ckpt.data_ptr(),
                                      resid.data_ptr(), K ** -0.5 if scale is None else scale, B, T, Hk, H, K, V,
                                      _stream(dev)))
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
    d_state_out = _state(d_state_out, (B, H, K, V), dev, "d_state_out")
    saved = (B, _nblocks(T), H, K * V)
    _out_arg(ckpt, saved, dev, "ckpt", F32)
    _out_arg(resid, (B, T, H, V), dev, "resid", F32)
    shapes = {"dq": (B, T, Hk, K), "dk": (B, T, Hk, K), "dv": (B, T, H, V), "dg": (B, T, H), "dbeta": (B, T, H),
              "d_state_in": (B, H, K, V)}
    if grads is None:
        grads = dict.fromkeys(shapes)
    grads = {n: _output(grads[n], s, dev, n) for n, s in shapes.items()}
    work = _output(work, saved, dev, "work")
    with _on(dev):
        _check(lib().gdr_backward_ckpt(q.data_ptr(), k.data_ptr(), g.data_ptr(), beta.data_ptr(), _dt(q),
                                       ckpt.data_ptr(), resid.data_ptr(), d_o.data_ptr(), _p(d_state_out),
                                       *[grads[n].data_ptr() for n in shapes], work.data_ptr(),
                                       K ** -0.5 if scale is None else scale, B, T, Hk, H, K, V, _stream(dev)))
    return grads
