"""The paged FP8 KV cache: quantised as it is written, read back, and attended
by new tokens (binding of the ``ovc_kv_*`` and ``ovc_paged_*`` calls).

A serving loop writes each step's keys and values and attends with its queries::

    cache = kv_cache(num_pages, num_heads, page_size=64)
    kv_cache_write(cache, k, v, slots)                  # k, v [T, heads, 128]
    o = paged_attention(q, cache, page_table, kv_lens, cu_q=cu_q, max_q=n)

Every call is asynchronous on the current stream (or ``stream``) and reads no
device value on the host, so that a step can be captured into a CUDA graph
(after one eager call, which loads the library and sets its per-device state)
and lengths, slots and page tables may change between replays.  The calls have
no gradient.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses

import torch

from . import _abi
from ._abi import check, lib
from .api import _DTYPES, _device_of

_byref = ctypes.byref
_INT32_MAX = 2 ** 31 - 1


@dataclasses.dataclass(frozen=True, eq=False)
class KVCache:
    """A cache's memory: E4M3 codes ``k``, ``v`` uint8 [pages, heads, page, 128]
    and E8M0 scale bytes ``k_scale``, ``v_scale`` uint8 [pages, heads, page]
    (value ``e4m3(code) * 2**(byte - 127)``), contiguous CUDA tensors.  ``page``
    is a multiple of 16, at most 1024.  The token slot ``s`` is row ``s % page``
    of page ``s // page`` in every head."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    def __post_init__(self):
        _device_of(self.k, self.v, self.k_scale, self.v_scale)
        shape = tuple(self.k.shape)
        if len(shape) != 4 or shape[3] != 128 or tuple(self.v.shape) != shape:
            raise ValueError("k and v must both be [pages, heads, page, 128]")
        if tuple(self.k_scale.shape) != shape[:3] or tuple(self.v_scale.shape) != shape[:3]:
            raise ValueError("k_scale and v_scale must be [pages, heads, page] as k and v")
        if shape[2] % 16 or not 16 <= shape[2] <= 1024:
            raise ValueError(f"page size {shape[2]} is not a multiple of 16 up to 1024")
        if 0 in shape or shape[0] * shape[1] * shape[2] > 2 ** 31 - 1024:
            raise ValueError(f"a cache of {shape[0]} pages, {shape[1]} heads and {shape[2]} tokens a page is not supported")
        for x in (self.k, self.v, self.k_scale, self.v_scale):
            if x.dtype != torch.uint8 or not x.is_contiguous() or x.data_ptr() % 16:
                raise ValueError("a cache's tensors must be contiguous, 16-byte aligned uint8")
        desc = _abi.OvcKVCache(shape[0], shape[1], shape[2], self.k.data_ptr(), self.v.data_ptr(),
                               self.k_scale.data_ptr(), self.v_scale.data_ptr())
        object.__setattr__(self, "_ref", _byref(desc))     # the C struct, kept alive by its reference
        object.__setattr__(self, "_shape", shape)

    @property
    def pages(self) -> int:
        return self._shape[0]

    @property
    def heads(self) -> int:
        return self._shape[1]

    @property
    def page(self) -> int:
        return self._shape[2]

    @property
    def device(self) -> torch.device:
        return self.k.device


def kv_cache(num_pages: int, num_heads: int, page_size: int = 64, *, device=None) -> KVCache:
    """A new cache on `device` (default: the current CUDA device); its slots
    hold nothing until they are written."""
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    shape = (int(num_pages), int(num_heads), int(page_size))
    return KVCache(*(torch.empty(s, dtype=torch.uint8, device=dev) for s in (shape + (128,), shape + (128,), shape, shape)))


@contextlib.contextmanager
def _on(dev: torch.device, stream):
    """The tensors' device as the current one, and `stream` (if given) as the
    current stream, so that what a call allocates belongs to it."""
    with torch.cuda.device(dev):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


def _call(dev, stream, fn):
    """fn(stream handle) under the right device and stream; the usual case, the
    current ones, without the cost of the context managers and stream objects."""
    if stream is None and dev.index == torch.cuda.current_device():
        return fn(torch._C._cuda_getCurrentRawStream(dev.index))
    with _on(dev, stream):
        return fn(torch._C._cuda_getCurrentRawStream(dev.index))


def _device(first: torch.Tensor, *others, stream=None) -> torch.device:
    """The device of all of them (None entries skipped), as :func:`_device_of`."""
    dev = first.device
    if stream is None and dev.type == "cuda":
        for x in others:
            if x is not None and x.device != dev:
                break
        else:
            return dev
    return _device_of(first, *others, stream=stream)


def _rows(x: torch.Tensor, what: str, heads: int | None = None) -> _abi.OvcRows:
    shape = x.shape
    if len(shape) != 3 or shape[2] != 128 or (heads is not None and shape[1] != heads):
        raise ValueError(f"{what} must be [tokens, {heads or 'heads'}, 128], got {tuple(shape)}")
    code = _DTYPES.get(x.dtype)
    if code is None:
        raise TypeError(f"{what} must be bfloat16 or float16, got {x.dtype}")
    st, sh, sc = x.stride()
    ptr = x.data_ptr()
    if sc != 1 or st % 8 or sh % 8 or ptr % 16:
        raise ValueError(f"{what} needs unit channel stride, strides that are multiples of 8 and 16-byte alignment")
    return _abi.OvcRows(ptr, code, shape[0], shape[1], st, sh)


def _ints(x: torch.Tensor, shape: tuple, what: str) -> int:
    if x.dtype != torch.int32 or x.shape != shape or not x.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor {list(shape)}, got {x.dtype} {list(x.shape)}")
    return x.data_ptr()


def kv_cache_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, *, stream=None) -> None:
    """Quantise the keys and values of T tokens, ``[T, heads, 128]`` (strided
    views allowed), into the cache: token t into slot ``slots[t]`` (int32
    [T]).  Negative slots are skipped (padding); slots beyond the cache are
    skipped and reported by :func:`device_status` (7).  A slot is given at most
    once per call.  See ``ovc_kv_write`` for the format."""
    dev = _device(cache.k, k, v, slots, stream=stream)
    rk, rv = _rows(k, "k", cache.heads), _rows(v, "v", cache.heads)
    if k.shape != v.shape or k.dtype != v.dtype:
        raise ValueError("k and v must have one shape and dtype")
    ps = _ints(slots, (k.shape[0],), "slots")
    if k.shape[0] == 0:
        return
    check(_call(dev, stream, lambda s: lib().ovc_kv_write(cache._ref, _byref(rk), _byref(rv), ps, s)), "ovc_kv_write")


def kv_cache_read(cache: KVCache, slots: torch.Tensor, *, dtype: torch.dtype = torch.bfloat16, out=None, stream=None):
    """The keys and values of the tokens in ``slots`` (int32 [T]) as a pair of
    `dtype` (bfloat16 or float16) tensors [T, heads, 128], or in the pair `out`,
    whose rows must not overlap.
    Negative slots give zeros; so do slots beyond the cache, which
    :func:`device_status` reports (7)."""
    dev = _device(cache.k, slots, *(out or ()), stream=stream)
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be bfloat16 or float16, got {dtype}")
    if slots.dim() != 1:
        raise ValueError(f"slots must be [tokens], got {tuple(slots.shape)}")
    n = slots.shape[0]
    ps = _ints(slots, (n,), "slots")
    if out is not None:
        for x in out:
            if tuple(x.shape) != (n, cache.heads, 128) or x.dtype != out[0].dtype:
                raise ValueError(f"out must be a pair of [{n}, {cache.heads}, 128] tensors of one dtype")
        if n and out[0].data_ptr() == out[1].data_ptr():
            raise ValueError("out must be two tensors that do not overlap")

    def run(s):
        pair = out if out is not None else tuple(
            torch.empty((n, cache.heads, 128), dtype=dtype, device=dev) for _ in range(2))
        if n:
            rk, rv = (_rows(x, "out", cache.heads) for x in pair)
            check(lib().ovc_kv_read(cache._ref, ps, _byref(rk), _byref(rv), s), "ovc_kv_read")
        return pair[0], pair[1]

    return _call(dev, stream, run)


def _batch(q, cache, page_table, kv_lens, cu_q, max_q, causal, window):
    shape, strides = page_table.shape, page_table.stride()
    if len(shape) != 2 or page_table.dtype != torch.int32 or strides[1] != 1 or shape[1] < 1:
        raise ValueError("page_table must be int32 [sequences, pages] with unit column stride")
    n, width = shape
    tokens, heads, _ = q.shape
    lens = _ints(kv_lens, (n,), "kv_lens")
    if cu_q is None:
        if tokens != n:
            raise ValueError(f"without cu_q each of the {n} sequences has one query row, got {tokens}")
        if max_q not in (None, 1):
            raise ValueError("max_q needs cu_q")
        cu, most = None, 1
    else:
        cu, most = _ints(cu_q, (n + 1,), "cu_q"), min(int(max_q or 0), _INT32_MAX)
    if most < 0:
        raise ValueError("max_q must not be negative")
    if window is not None and (window < 1 or not causal):
        raise ValueError("window must be positive and needs causal")
    if heads % cache.heads or heads == 0:
        raise ValueError(f"{heads} query heads over {cache.heads} KV heads")
    stride = strides[0] if n > 1 else max(strides[0], width)
    return _abi.OvcPagedBatch(n, page_table.data_ptr(), stride, width, lens, cu, most, int(bool(causal)),
                              min(int(window or 0), _INT32_MAX))


def paged_attention_workspace_bytes(q: torch.Tensor, cache: KVCache, page_table: torch.Tensor, kv_lens: torch.Tensor, *,
                                    cu_q: torch.Tensor | None = None, max_q: int | None = None) -> int:
    """Bytes of :func:`paged_attention`'s workspace (0 for no rows)."""
    if q.shape[0] == 0:
        return 0
    rq = _rows(q, "q")
    b = _batch(q, cache, page_table, kv_lens, cu_q, max_q, True, None)
    return int(lib().ovc_paged_attention_workspace_bytes(_byref(rq), cache._ref, _byref(b)))


def paged_attention(q: torch.Tensor, cache: KVCache, page_table: torch.Tensor, kv_lens: torch.Tensor, *,
                    cu_q: torch.Tensor | None = None, max_q: int | None = None, causal: bool = True,
                    window: int | None = None, softmax_scale: float | None = None, out: torch.Tensor | None = None,
                    return_lse: bool = False, workspace: torch.Tensor | None = None, stream=None):
    """Attention of new tokens over a paged cache (``ovc_paged_attention``).

    q ``[T, query heads, 128]`` BF16 or FP16, a multiple of the cache's heads
    (query head i uses KV head i // (query heads / heads)); ``page_table`` int32
    [B, pages] and ``kv_lens`` int32 [B] describe each sequence's cached tokens,
    the new ones among them.  Without ``cu_q`` every sequence has one query row
    (decoding, T = B); with it (int32 [B+1]) sequence b's rows are
    ``q[cu_q[b]:cu_q[b+1]]``, its last tokens.  ``max_q``, the most rows of any
    sequence if known, only chooses between kernels.  ``causal``: a row sees the
    keys up to its own position, with ``window`` only the last `window` of them;
    otherwise all keys of its sequence.  ``softmax_scale``: finite; 1/sqrt(128) if
    not given or not positive.

    Returns O, BF16 shaped like q (with ``return_lse`` also the FP32 [T, query
    heads] natural log-sum-exp of the scaled scores).  A row that sees no key
    gives 0 and -inf.  Rows of no sequence are left as they were (in a new
    output: unset).  Indices outside the cache, the table or q are cut off and
    reported by :func:`device_status` (7); where ``cu_q`` descends, no row is
    written.  ``out`` must not overlap q.  ``workspace`` (uint8, 256-byte aligned,
    :func:`paged_attention_workspace_bytes`) is allocated if not given; calls,
    or captured graphs, that share one must not run at the same time."""
    dev = _device(q, cache.k, page_table, kv_lens, cu_q, out, workspace, stream=stream)
    rq = _rows(q, "q")
    b = _batch(q, cache, page_table, kv_lens, cu_q, max_q, causal, window)
    if out is not None and (out.shape != q.shape or out.dtype != torch.bfloat16):
        raise ValueError("out must be a bfloat16 tensor shaped like q")
    if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous uint8 tensor")

    def run(s):
        o = out if out is not None else torch.empty_like(q, dtype=torch.bfloat16, memory_format=torch.contiguous_format)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=dev) if return_lse else None
        if q.shape[0] and b.B:
            ro = _rows(o, "out")
            L, pq, pb, ws = lib(), _byref(rq), _byref(b), workspace
            if ws is None:
                ws = torch.empty(L.ovc_paged_attention_workspace_bytes(pq, cache._ref, pb), dtype=torch.uint8, device=dev)
            check(L.ovc_paged_attention(pq, cache._ref, pb, float(softmax_scale or 0.0), _byref(ro),
                                        None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.numel(), s),
                  "ovc_paged_attention")
        return (o, lse) if return_lse else o

    return _call(dev, stream, run)


__all__ = ["KVCache", "kv_cache", "kv_cache_write", "kv_cache_read", "paged_attention", "paged_attention_workspace_bytes"]
