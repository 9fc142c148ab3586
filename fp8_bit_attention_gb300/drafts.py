"""Verification of drafted tokens (binding of ``ovc_verify_drafts``): what
follows :func:`paged_attention` of drafted tokens and the model's head, and says
which of them stay."""
from __future__ import annotations

import ctypes

import torch

from . import _abi
from ._abi import check, lib
from .paged import _call, _device, _ints

_byref = ctypes.byref
_TYPES = {torch.float32: _abi.OVC_FP32, torch.bfloat16: _abi.OVC_BF16, torch.float16: _abi.OVC_FP16}


def _floats(x: torch.Tensor, shape: tuple, what: str) -> int:
    if x.dtype != torch.float32 or x.shape != shape or not x.is_contiguous():
        raise ValueError(f"{what} must be a contiguous float32 tensor {list(shape)}, got {x.dtype} {list(x.shape)}")
    return x.data_ptr()


def verify_drafts(target_probs: torch.Tensor, drafts: torch.Tensor, accept_u: torch.Tensor, sample_u: torch.Tensor, *,
                  draft_probs: torch.Tensor | None = None, cu_drafts: torch.Tensor | None = None, stream=None):
    """Verify the N drafted tokens of B sequences and draw the next token of each.

    ``drafts`` int32: [B, n], n for each sequence, or [N] with ``cu_drafts`` int32
    [B+1], sequence b's being ``drafts[cu_drafts[b]:cu_drafts[b+1]]``.  A negative
    draft ends its sequence's (padding).  ``target_probs`` [N + B, V]: the
    verifying model's probabilities, for each sequence a row for each draft and one
    for the token after them; ``draft_probs`` [N, V]: those that the drafts were
    drawn with (None: each was certain).  Both float32, bfloat16 or float16, not
    negative, unit column stride.  ``accept_u`` (shaped like drafts) and
    ``sample_u`` [B]: float32 random numbers in [0, 1).

    Draft x stays if all before it did and ``accept_u * q[x] < p[x]``.  At the
    first that does not, the next token is drawn from max(p - q, 0) (from p where
    that is zero everywhere), after the last from its row of p: the least token
    whose running sum exceeds ``sample_u`` times the total.

    Returns int32 ``tokens`` [N + B], in the order of ``target_probs``: the drafts
    that stayed, the next token (-1 if its row leaves nothing), -1 for the rest;
    and ``accepted`` [B], how many stayed, so that a sequence whose drafts are in
    its cache goes on with ``kv_lens - n + accepted`` tokens."""
    dev = _device(target_probs, drafts, accept_u, sample_u, draft_probs, cu_drafts, stream=stream)
    dtype = _TYPES.get(target_probs.dtype)
    if dtype is None:
        raise TypeError(f"target_probs must be float32, bfloat16 or float16, got {target_probs.dtype}")
    if cu_drafts is None:
        if drafts.dim() != 2:
            raise ValueError(f"drafts must be [sequences, drafts] (or [drafts] with cu_drafts), got {tuple(drafts.shape)}")
        cu, batch = None, drafts.shape[0]
    else:
        if drafts.dim() != 1 or cu_drafts.dim() != 1 or cu_drafts.shape[0] < 1:
            raise ValueError("with cu_drafts [sequences + 1], drafts must be [drafts]")
        batch = cu_drafts.shape[0] - 1
        cu = _ints(cu_drafts, (batch + 1,), "cu_drafts")
    n = drafts.numel()
    pd, pu = _ints(drafts, drafts.shape, "drafts"), _floats(accept_u, drafts.shape, "accept_u")
    ps = _floats(sample_u, (batch,), "sample_u")
    for x, rows, what in ((target_probs, n + batch, "target_probs"), (draft_probs, n, "draft_probs")):
        if x is not None and (x.dim() != 2 or x.shape[0] != rows or x.shape[1] < 1 or (x.shape[1] > 1 and x.stride(1) != 1)):
            raise ValueError(f"{what} must be [{rows}, vocabulary] with unit column stride, got {tuple(x.shape)}")
    if draft_probs is not None and (draft_probs.shape[1] != target_probs.shape[1] or draft_probs.dtype != target_probs.dtype):
        raise ValueError("draft_probs must have the vocabulary and dtype of target_probs")
    desc = _abi.OvcDrafts(batch, n, target_probs.shape[1], cu, pd, target_probs.data_ptr(),
                          None if draft_probs is None or n == 0 else draft_probs.data_ptr(), dtype, target_probs.stride(0),
                          0 if draft_probs is None else draft_probs.stride(0), pu, ps)

    def run(s):
        out = torch.empty(n + 2 * batch, dtype=torch.int32, device=dev)
        if batch:
            at = out.data_ptr()
            check(lib().ovc_verify_drafts(_byref(desc), at, at + 4 * (n + batch), s), "ovc_verify_drafts")
        return out[:n + batch], out[n + batch:]

    return _call(dev, stream, run)


__all__ = ["verify_drafts"]
