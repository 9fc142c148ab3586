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


def _probs(x: torch.Tensor, rows: int, what: str) -> tuple[int, int, int]:
    """Vocabulary, address and row stride."""
    shape = x.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] < 1:
        raise ValueError(f"{what} must be [{rows}, vocabulary], got {tuple(shape)}")
    strides = x.stride()
    if strides[1] != 1 and shape[1] > 1:
        raise ValueError(f"{what} needs unit column stride")
    return shape[1], x.data_ptr(), strides[0]


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
    that stayed, the next token (-1 if its row leaves nothing), -1 for the rest and
    for rows of no sequence; and ``accepted`` [B], how many stayed, so that a
    sequence whose drafts are in its cache goes on with ``kv_lens - n + accepted``
    tokens.  A sequence whose starts descend or leave [0, N] has no rows and accepts
    0; :func:`device_status` reports it (7)."""
    dev = _device(target_probs, drafts, accept_u, sample_u, draft_probs, cu_drafts, stream=stream)
    dtype = _TYPES.get(target_probs.dtype)
    if dtype is None:
        raise TypeError(f"target_probs must be float32, bfloat16 or float16, got {target_probs.dtype}")
    shape = drafts.shape
    if cu_drafts is None:
        if len(shape) != 2:
            raise ValueError(f"drafts must be [sequences, drafts] (or [drafts] with cu_drafts), got {tuple(shape)}")
        cu, batch = None, shape[0]
        n = batch * shape[1]
    else:
        if len(shape) != 1 or cu_drafts.dim() != 1 or cu_drafts.shape[0] < 1:
            raise ValueError("with cu_drafts [sequences + 1], drafts must be [drafts]")
        n, batch = shape[0], cu_drafts.shape[0] - 1
        cu = _ints(cu_drafts, (batch + 1,), "cu_drafts")
    pd, pu = _ints(drafts, shape, "drafts"), _floats(accept_u, shape, "accept_u")
    ps = _floats(sample_u, (batch,), "sample_u")
    vocab, target, stride = _probs(target_probs, n + batch, "target_probs")
    draft, draft_stride = None, 0
    if draft_probs is not None:
        same, draft, draft_stride = _probs(draft_probs, n, "draft_probs")
        if same != vocab or draft_probs.dtype != target_probs.dtype:
            raise ValueError("draft_probs must have the vocabulary and dtype of target_probs")
        if n == 0:
            draft = None
    desc = _abi.OvcDrafts(batch, n, vocab, cu, pd, target, draft, dtype, stride, draft_stride, pu, ps)

    def run(s):
        # two tensors: views of a new one take the host longer than allocating them
        tokens = torch.empty(n + batch, dtype=torch.int32, device=dev)
        accepted = torch.empty(batch, dtype=torch.int32, device=dev)
        if not batch:
            tokens.fill_(-1)
        else:
            check(lib().ovc_verify_drafts(_byref(desc), tokens.data_ptr(), accepted.data_ptr(), s), "ovc_verify_drafts")
        return tokens, accepted

    return _call(dev, stream, run)


__all__ = ["verify_drafts"]
