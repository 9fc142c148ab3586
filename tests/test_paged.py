"""CPU checks of the paged FP8 cache: its format in the tests' definition, and
the refusals of the C ABI and of the binding, before any device call."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_bit_attention_gb300 as ovc
from fp8_bit_attention_gb300 import _abi

from paged_util import GRID, SCALES, quantise


@pytest.fixture(scope="module")
def lib():
    from fp8_bit_attention_gb300 import build
    build.build()
    return _abi.lib()


def test_definition_against_torch_casts():
    g = np.random.default_rng(1)
    x = (g.standard_normal((300, 128)) * np.exp2(g.integers(-40, 40, (300, 1)))).astype(np.float32)
    codes, byte = quantise(x)
    want = torch.from_numpy(x / SCALES[byte][:, None].astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8)
    assert np.array_equal(codes, want.numpy())
    top = np.abs(GRID[codes]).max(1)
    assert (top > 216).all() and (top <= 448).all()           # the least scale that holds the vector


@pytest.mark.parametrize("amax, byte", [(0.0, 127), (448.0, 127), (448.0 * (1 + 2 ** -7), 128), (224.0, 126),
                                        (1.0, 119), (1e-44, 0), (2.0 ** 127 * 1.984375, 247), (np.inf, 255), (np.nan, 255)])
def test_scale_bytes(amax, byte):
    x = np.zeros((1, 128))
    x[0, 5] = amax
    codes, e = quantise(x)
    assert e[0] == byte
    assert byte != 255 or not codes.any()


def _cache(pages=4, heads=2, page=16, **kw):
    d = dict(pages=pages, heads=heads, page=page, k=0x10000, v=0x20000, k_scale=0x30000, v_scale=0x40000)
    d.update(kw)
    return _abi.OvcKVCache(*(d[f] for f, _ in _abi.OvcKVCache._fields_))


def _rows(T=3, H=2, **kw):
    d = dict(ptr=0x50000, dtype=_abi.OVC_BF16, T=T, H=H, stride_t=H * 128, stride_h=128)
    d.update(kw)
    return _abi.OvcRows(*(d[f] for f, _ in _abi.OvcRows._fields_))


def _batch(B=3, **kw):
    d = dict(B=B, page_table=0x60000, table_stride=8, table_width=8, kv_lens=0x70000, cu_q=0x80000, max_q=0, causal=1, window=0)
    d.update(kw)
    return _abi.OvcPagedBatch(*(d[f] for f, _ in _abi.OvcPagedBatch._fields_))


BAD_CACHES = [dict(pages=0), dict(heads=0), dict(page=8), dict(page=24), dict(page=2048), dict(k=0), dict(v=0x20008),
              dict(k_scale=None), dict(v_scale=0x40004), dict(pages=1 << 27, heads=2, page=16), dict(pages=1 << 62, page=16)]
BAD_ROWS = [dict(T=0), dict(ptr=0), dict(ptr=0x50002), dict(stride_t=260), dict(stride_h=-128), dict(T=1 << 31)]
R, B = ctypes.byref, ctypes.c_void_p


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_bad_caches_are_refused(lib, bad):
    c, r, b = _cache(**bad), _rows(), _batch()
    assert lib.ovc_kv_write(R(c), R(r), R(r), B(0x90000), None) == _abi.OVC_ERR_INVALID_ARG
    assert lib.ovc_kv_read(R(c), B(0x90000), R(r), R(r), None) == _abi.OVC_ERR_INVALID_ARG
    assert lib.ovc_paged_attention_workspace_bytes(R(r), R(c), R(b)) == 0
    assert lib.ovc_paged_attention(R(r), R(c), R(b), 0.0, R(r), None, B(0x100000), 1 << 30, None) == _abi.OVC_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", BAD_ROWS, ids=str)
def test_bad_rows_are_refused(lib, bad):
    c, r, x, b = _cache(), _rows(), _rows(**bad), _batch()
    for k, v in ((x, r), (r, x)):
        assert lib.ovc_kv_write(R(c), R(k), R(v), B(0x90000), None) == _abi.OVC_ERR_INVALID_ARG
        assert lib.ovc_kv_read(R(c), B(0x90000), R(k), R(v), None) == _abi.OVC_ERR_INVALID_ARG
    for q, o in ((x, r), (r, x)):
        assert lib.ovc_paged_attention(R(q), R(c), R(b), 0.0, R(o), None, B(0x100000), 1 << 30, None) == _abi.OVC_ERR_INVALID_ARG


@pytest.mark.parametrize("strides, ok", [((0, 128), False), ((256, 0), False), ((128, 128), False), ((256, 128), True),
                                         ((248, 128), False), ((256, 120), False), ((128, 5 * 128), True),
                                         ((128, 4 * 128), False), ((1 << 40, 136), True), ((136, 1 << 40), True)], ids=str)
def test_outputs_that_overlap_are_refused(lib, strides, ok):
    """5 tokens, 2 heads; the same strides are fine to read from."""
    c, r, o, b = _cache(), _rows(T=5), _rows(T=5, stride_t=strides[0], stride_h=strides[1]), _batch()
    if not ok or not torch.cuda.is_available():
        st = lib.ovc_kv_read(R(c), B(0x90000), R(o), R(o), None)
        assert (st != _abi.OVC_ERR_INVALID_ARG) == ok
        st = lib.ovc_paged_attention(R(r), R(c), R(b), 0.0, R(o), None, B(0x100000), 1 << 30, None)
        assert (st != _abi.OVC_ERR_INVALID_ARG) == ok
    if not torch.cuda.is_available():
        assert lib.ovc_kv_write(R(c), R(o), R(o), B(0x90000), None) != _abi.OVC_ERR_INVALID_ARG


def test_mismatched_arguments_are_refused(lib):
    c, r, b = _cache(), _rows(), _batch()
    bad = _abi.OVC_ERR_INVALID_ARG
    assert lib.ovc_kv_write(None, R(r), R(r), B(0x90000), None) == bad
    assert lib.ovc_kv_write(R(c), None, R(r), B(0x90000), None) == bad
    assert lib.ovc_kv_write(R(c), R(r), R(r), None, None) == bad
    assert lib.ovc_kv_write(R(c), R(r), R(r), B(0x90002), None) == bad
    assert lib.ovc_kv_write(R(c), R(r), R(_rows(T=4)), B(0x90000), None) == bad
    assert lib.ovc_kv_write(R(c), R(r), R(_rows(H=4)), B(0x90000), None) == bad
    assert lib.ovc_kv_write(R(c), R(r), R(_rows(dtype=_abi.OVC_FP16)), B(0x90000), None) == bad
    assert lib.ovc_kv_write(R(c), R(_rows(dtype=5)), R(_rows(dtype=5)), B(0x90000), None) == _abi.OVC_ERR_UNSUPPORTED

    def attend(q=r, c=c, b=b, o=r, lse=None, ws=0x100000, n=1 << 30):
        return lib.ovc_paged_attention(R(q), R(c), R(b), 0.0, R(o), B(lse), B(ws), n, None)

    assert attend(q=_rows(H=3), o=_rows(H=3)) == bad                      # 3 query heads over 2
    assert attend(o=_rows(T=4)) == bad
    assert attend(o=_rows(dtype=_abi.OVC_FP16)) == bad
    assert attend(lse=0xA0002) == bad
    assert attend(ws=None) == bad
    assert attend(ws=0x100010) == bad
    assert attend(n=16) == _abi.OVC_ERR_WORKSPACE_TOO_SMALL
    for kw in (dict(B=0), dict(page_table=None), dict(kv_lens=None), dict(table_width=0), dict(table_stride=7), dict(max_q=-1),
               dict(causal=2), dict(window=-1), dict(causal=0, window=4), dict(cu_q=0x80002), dict(B=2, cu_q=None)):
        assert attend(b=_batch(**kw)) == bad, kw
        assert lib.ovc_paged_attention_workspace_bytes(R(r), R(c), R(_batch(**kw))) == 0, kw
    assert lib.ovc_paged_attention_workspace_bytes(R(r), R(c), R(b)) > 0
    if not torch.cuda.is_available():
        assert attend() in (_abi.OVC_ERR_CUDA, _abi.OVC_ERR_UNSUPPORTED)


def test_binding_refuses_cpu_tensors():
    x = torch.zeros((2, 1, 16, 128), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        ovc.KVCache(x, x, x[..., 0], x[..., 0])


def test_status_string(lib):
    assert b"slot" in lib.ovc_status_string(_abi.OVC_ERR_BAD_INDEX)
