"""Verification of drafted tokens: the binding of ``include/draft.h``."""
from __future__ import annotations

import torch

from . import _check, _dt, _int_rows, _out_arg, lib
from .gdr import _good, _on, _output, _p, _stream

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
    B, places, vocab = target.shape
    N, dev = places - 1, target.device
    if not (_good(tokens, (B, N), torch.int32, dev) and _good(u, (B, N), torch.float32, dev)
            and _good(u_draw, (B,), torch.float32, dev)):
        _out_arg(tokens, (B, N), dev, "tokens", I32)
        _out_arg(u, (B, N), dev, "u", F32)
        _out_arg(u_draw, (B,), dev, "u_draw", F32)
    if draft is not None and not _good(draft, (B, N, vocab), target.dtype, dev):
        _out_arg(draft, (B, N, vocab), dev, "draft", (target.dtype,))
    out = _output(out, (B, places), dev, "out", torch.int32, I32)
    kept = _output(kept, (B,), dev, "kept", torch.int32, I32)
    with _on(dev):
        n_draft = None if n_draft is None else _int_rows(n_draft, B, dev, "n_draft")
        _check(lib().draft_verify(target.data_ptr(), _p(draft), _dt(target), tokens.data_ptr(), _p(n_draft),
                                  u.data_ptr(), u_draw.data_ptr(), out.data_ptr(), kept.data_ptr(), B, N, vocab,
                                  _stream(dev)))
    return out, kept
