"""Verification of drafted tokens: the binding of ``include/draft.h``."""
from __future__ import annotations

import torch

from . import _check, _dt, _int_rows, _out_arg, _ptr, _stream, lib
from .gdr import _on

I32, F32 = (torch.int32,), (torch.float32,)


def draft_verify(target, tokens, u, u_draw, *, draft=None, n_draft=None, out=None, kept=None):
    """Accept drafted tokens and draw the one that follows.  Returns (out, kept).

    target: [B, N+1, vocab] probabilities, bf16 or fp32; tokens: [B, N] int32 drafts; draft:
    [B, N, vocab] the drafter's probabilities like target's, or None for a drafter that is
    sure of its tokens; n_draft: [B] integers, the drafts of each row (None: N); u [B, N]
    and u_draw [B]: fp32 random numbers in [0, 1).

    Draft j is accepted iff u q(x) < p(x); at the first that is not, the drawn token comes
    from max(p - q, 0), behind the last from p.  out [B, N+1] int32 holds the accepted
    drafts, the drawn token, then -1; kept [B] int32 is the number of tokens in out[b] and
    of the verify step's tokens whose states stand: the ``accepted`` of wkv7_state_commit.
    """
    if target.dim() != 3 or not target.is_cuda or not target.is_contiguous():
        raise ValueError("target must be a contiguous [B, N+1, vocab] GPU tensor")
    _dt(target)
    B, N, vocab = target.shape[0], target.shape[1] - 1, target.shape[2]
    dev = target.device
    _out_arg(tokens, (B, N), dev, "tokens", I32)
    _out_arg(u, (B, N), dev, "u", F32)
    _out_arg(u_draw, (B,), dev, "u_draw", F32)
    if draft is not None:
        _out_arg(draft, (B, N, vocab), dev, "draft", (target.dtype,))
    out = torch.empty((B, N + 1), dtype=torch.int32, device=dev) if out is None else out
    _out_arg(out, (B, N + 1), dev, "out", I32)
    kept = torch.empty((B,), dtype=torch.int32, device=dev) if kept is None else kept
    _out_arg(kept, (B,), dev, "kept", I32)
    with _on(dev):
        n_draft = None if n_draft is None else _int_rows(n_draft, B, dev, "n_draft")
        _check(lib().draft_verify(_ptr(target), _ptr(draft) if N else None, _dt(target), _ptr(tokens) if N else None,
                                  _ptr(n_draft), _ptr(u) if N else None, _ptr(u_draw), _ptr(out), _ptr(kept),
                                  B, N, vocab, _stream(dev)))
    return out, kept
