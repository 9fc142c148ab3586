"""The pages of growing sequences, and tokens moved inside a paged cache
(binding of the ``ovc_kv_pages_*``, ``ovc_kv_copy`` and ``ovc_kv_compact``
calls).

A serving loop lets its sequences grow, writes and attends, and gives back what
it no longer needs; candidates share the pages of what they continue::

    pages = kv_pages(num_pages, num_sequences, pages_per_sequence, page_size=64)
    kv_pages_fork(pages, parents, children)
    src, dst, tokens = kv_pages_reserve(pages, new_lens)
    kv_cache_copy(cache, src, dst, tokens)                 # for the cache of each layer
    ...                                                    # kv_cache_write, paged_attention(q, cache, pages.page_table, pages.kv_lens)
    kv_pages_release(pages, shorter_lens)

As the calls of :mod:`.paged` these are asynchronous on the current stream (or
``stream``), read no device value on the host, and can be captured into a CUDA
graph after one eager call.  They have no gradient.
"""
from __future__ import annotations

import ctypes
import dataclasses

import torch

from . import _abi
from ._abi import check, lib
from .paged import KVCache, _call, _device, _ints

_byref = ctypes.byref


@dataclasses.dataclass(frozen=True, eq=False)
class KVPages:
    """Which pages each sequence holds: contiguous int32 CUDA tensors
    ``page_table`` [sequences, pages per sequence], ``kv_lens`` [sequences] and
    ``refs`` [pages], and the tokens of a page.  Row b's first
    ceil(kv_lens[b] / page) entries are its pages; ``refs[p]`` counts the entries
    that name page p (a program may add to it to keep a page), 0 says that it is
    free.  At most 8192 sequences; ``refs`` is 16-byte aligned.  The first two are
    what :func:`paged_attention` takes."""
    page_table: torch.Tensor
    kv_lens: torch.Tensor
    refs: torch.Tensor
    page: int

    def __post_init__(self):
        _device(self.page_table, self.kv_lens, self.refs)
        t = self.page_table
        if t.dim() != 2 or self.refs.dim() != 1 or 0 in t.shape or self.refs.shape[0] == 0:
            raise ValueError("page_table must be [sequences, pages per sequence] and refs [pages]")
        ptrs = [_ints(t, t.shape, "page_table"), _ints(self.kv_lens, (t.shape[0],), "kv_lens"),
                _ints(self.refs, (self.refs.shape[0],), "refs")]
        if ptrs[2] % 16:
            raise ValueError("refs must be 16-byte aligned")
        if self.page % 16 or not 16 <= self.page <= 1024:
            raise ValueError(f"page size {self.page} is not a multiple of 16 up to 1024")
        if t.shape[0] > 8192:
            raise ValueError(f"{t.shape[0]} sequences: at most 8192 are supported")
        if max(self.refs.shape[0], t.shape[1]) * self.page > 2 ** 31 - 1024:
            raise ValueError(f"{self.refs.shape[0]} pages, {t.shape[1]} a sequence, of {self.page} tokens are not supported")
        desc = _abi.OvcKVPages(t.shape[0], self.refs.shape[0], t.shape[1], self.page, *ptrs)
        object.__setattr__(self, "_ref", _byref(desc))     # the C struct, kept alive by its reference
        object.__setattr__(self, "_rows", t.shape[0])

    @property
    def device(self) -> torch.device:
        return self.refs.device


def kv_pages(num_pages: int, num_sequences: int, pages_per_sequence: int, page_size: int = 64, *, device=None) -> KVPages:
    """The pages of a new cache, all free, and empty sequences, on `device`
    (default: the current CUDA device)."""
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    i32 = dict(dtype=torch.int32, device=dev)
    return KVPages(torch.full((int(num_sequences), int(pages_per_sequence)), -1, **i32),
                   torch.zeros(int(num_sequences), **i32), torch.zeros(int(num_pages), **i32), int(page_size))


def kv_pages_reserve(pages: KVPages, lens: torch.Tensor, *, stream=None):
    """Let sequence b grow to ``lens[b]`` tokens (int32 [sequences]; not larger
    than its length, or negative: it stays).  It takes the lowest free pages, in
    the order of sequences and then of columns; a partly filled last page that
    others hold too is replaced by one of its own, unless all its holders grow in
    this call: then the highest of them keeps it.  A sequence grows only if those
    up to it need no more pages than are free; ``pages.kv_lens`` says which did.

    Returns the copies that replaced pages ask for: pages, their successors and
    tokens, int32 [sequences] each (-1, -1, 0 for the others), as
    :func:`kv_cache_copy` takes them, for the cache of each layer, before new
    tokens are written to it and before the next change of `pages`."""
    dev = _device(pages.refs, lens, stream=stream)
    n = pages._rows
    pl = _ints(lens, (n,), "lens")

    def run(s):
        # three tensors: views of a new one take the host longer than allocating them
        src, dst, tokens = torch.empty_like(lens), torch.empty_like(lens), torch.empty_like(lens)
        check(lib().ovc_kv_pages_reserve(pages._ref, pl, src.data_ptr(), dst.data_ptr(), tokens.data_ptr(), s), "ovc_kv_pages_reserve")
        return src, dst, tokens

    return _call(dev, stream, run)


def kv_pages_release(pages: KVPages, lens: torch.Tensor, *, stream=None) -> None:
    """Let sequence b shrink to ``lens[b]`` tokens (int32 [sequences]; not smaller
    than its length, or negative: it stays) and give back the pages that hold none
    of them."""
    dev = _device(pages.refs, lens, stream=stream)
    pl = _ints(lens, (pages._rows,), "lens")
    check(_call(dev, stream, lambda s: lib().ovc_kv_pages_release(pages._ref, pl, s)), "ovc_kv_pages_release")


def kv_pages_fork(pages: KVPages, parents: torch.Tensor, children: torch.Tensor, *, stream=None) -> None:
    """Make sequence ``children[i]`` (empty) a second holder of what
    ``parents[i]`` holds (int32 [n] each, n at most the sequences; both negative:
    padding).  Nothing is copied; :func:`kv_pages_reserve` separates them as they
    grow.  A child that is not empty or named elsewhere in the lists, or a row
    outside, is skipped and reported by :func:`device_status` (7)."""
    dev = _device(pages.refs, parents, children, stream=stream)
    n = children.shape[0] if children.dim() == 1 else -1
    if not 0 <= n <= pages._rows:
        raise ValueError(f"children must be [n] with n up to {pages._rows}, got {tuple(children.shape)}")
    pp, pc = _ints(parents, (n,), "parents"), _ints(children, (n,), "children")
    if n:
        check(_call(dev, stream, lambda s: lib().ovc_kv_pages_fork(pages._ref, pp, pc, n, s)), "ovc_kv_pages_fork")


def kv_cache_copy(cache: KVCache, src: torch.Tensor, dst: torch.Tensor, tokens: torch.Tensor | None = None, *,
                  source: KVCache | None = None, stream=None) -> None:
    """Copy the first ``tokens[i]`` tokens (default: all) of page ``src[i]`` of
    `source` (default: `cache`; same heads and page size) to page ``dst[i]`` of
    `cache`, keys and values of every head; int32 [n] each.  Negative pages copy
    nothing; pages or numbers of tokens out of range are skipped and reported by
    :func:`device_status` (7).  A page that is written is named by no other entry."""
    dev = _device(cache.k, src, dst, tokens, None if source is None else source.k, stream=stream)
    if source is not None and (source.heads != cache.heads or source.page != cache.page):
        raise ValueError("source must have the cache's heads and page size")
    n = src.shape[0] if src.dim() == 1 else -1
    if n < 0:
        raise ValueError(f"src must be [n], got {tuple(src.shape)}")
    ps, pd = _ints(src, (n,), "src"), _ints(dst, (n,), "dst")
    pt = None if tokens is None else _ints(tokens, (n,), "tokens")
    if n:
        check(_call(dev, stream, lambda s: lib().ovc_kv_copy(cache._ref, None if source is None else source._ref, ps, pd, pt, n, s)),
              "ovc_kv_copy")


def kv_cache_compact(cache: KVCache, pages: KVPages, keep: torch.Tensor, cu_keep: torch.Tensor, *, stream=None) -> None:
    """Move the kept tokens of each sequence together, in place: sequence b's
    token at position ``keep[cu_keep[b] + i]`` goes to position i.  `keep` is int32
    [n], for all heads, or [heads, n], a list for each (unit column stride);
    ``cu_keep`` int32 [sequences + 1].  A sequence's positions ascend strictly and lie below its
    length.  After the cache of every layer, ``kv_pages_release(pages, kept)``
    gives back the pages behind.

    Every page that is written must be the sequence's alone: one with a shared
    page among them is left as it was, in all heads, and reported by :func:`device_status` (7);
    so are positions that do not ascend or lie outside, which are not moved."""
    dev = _device(cache.k, pages.refs, keep, cu_keep, stream=stream)
    if cache.pages != pages.refs.shape[0] or cache.page != pages.page:
        raise ValueError("cache and pages must have the same number of pages and page size")
    if keep.dim() not in (1, 2) or (keep.dim() == 2 and keep.shape[0] != cache.heads):
        raise ValueError(f"keep must be [n] or [{cache.heads}, n], got {tuple(keep.shape)}")
    n, pc = keep.shape[-1], _ints(cu_keep, (pages._rows + 1,), "cu_keep")
    stride = keep.stride(0) if keep.dim() == 2 and cache.heads > 1 else 0
    if keep.dtype != torch.int32 or (n > 1 and keep.stride(-1) != 1) or 0 < stride < n:
        raise ValueError(f"keep must be int32 with unit stride, its lists apart or all the same, got {keep.dtype}, strides {keep.stride()}")
    pk = keep.data_ptr()
    if n:
        check(_call(dev, stream, lambda s: lib().ovc_kv_compact(cache._ref, pages._ref, pk, stride, pc, n, s)), "ovc_kv_compact")


__all__ = ["KVPages", "kv_pages", "kv_pages_reserve", "kv_pages_release", "kv_pages_fork", "kv_cache_copy", "kv_cache_compact"]
