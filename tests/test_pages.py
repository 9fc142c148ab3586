"""CPU checks of the pages of sequences, of moves inside the cache and of the
verification of drafts: the tests' definitions, and the refusals of the C ABI and
of the binding, before any device call."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import fp8_bit_attention_gb300 as ovc
from fp8_bit_attention_gb300 import _abi

from pages_util import Pages, check_verified, verify
from test_paged import BAD_CACHES, _cache, lib  # noqa: F401

R, B = ctypes.byref, ctypes.c_void_p
BAD = _abi.OVC_ERR_INVALID_ARG


def _pages(rows=3, pages=4, width=2, page=16, **kw):
    d = dict(rows=rows, pages=pages, width=width, page=page, page_table=0x10000, kv_lens=0x20000, refs=0x30000)
    d.update(kw)
    return _abi.OvcKVPages(*(d[f] for f, _ in _abi.OvcKVPages._fields_))


def _drafts(**kw):
    d = dict(B=2, N=6, V=100, cu_drafts=0x10000, drafts=0x20000, target=0x30000, draft=0x40000, dtype=_abi.OVC_FP32,
             target_stride=100, draft_stride=100, accept_u=0x50000, sample_u=0x60000)
    d.update(kw)
    return _abi.OvcDrafts(*(d[f] for f, _ in _abi.OvcDrafts._fields_))


# ------------------------------------------------------------ the definitions
def test_definition_keeps_the_state_sound():
    g = np.random.default_rng(1)
    p = Pages(np.full((6, 5), -1), np.zeros(6), np.zeros(17), 16)
    for _ in range(300):
        op = g.integers(3)
        if op == 0:
            before = p.lens.copy()
            src, dst, tokens = p.reserve(before + g.integers(-3, 40, 6))
            assert ((src >= 0) == (dst >= 0)).all() and (tokens[src >= 0] > 0).all()
        elif op == 1:
            p.release(p.lens - g.integers(-5, 50, 6))
        else:
            empty = np.nonzero(p.lens == 0)[0]
            if len(empty) and p.lens.any():
                p.fork([int(p.lens.argmax())] * len(empty), empty)
        assert p.sound()
        for b in range(6):     # what a row may write to next is its own
            if p.lens[b] % 16 and op == 0 and p.lens[b] > before[b]:
                assert p.refs[p.table[b, p.lens[b] // 16]] == 1


def test_verified_tokens_are_distributed_as_the_target():
    """One draft drawn from q, accepted or replaced: P(token) = p exactly."""
    g = np.random.default_rng(2)
    p, q = g.random((2, 5)), g.random((1, 5))
    p, q = p / p.sum(1, keepdims=True), q / q.sum(1, keepdims=True)
    got = np.zeros(5)
    for x in range(5):
        stay = min(1.0, p[0, x] / q[0, x])
        got[x] += q[0, x] * stay
        (i, w), = verify(p, q, [x], [0, 1], [1.0 - 1e-12], [0.0])
        assert (i == 1) == (stay == 1.0)
        if i == 0:
            got += q[0, x] * (1 - stay) * w / w.sum()
    assert np.allclose(got, p[0], rtol=0, atol=1e-12)


def test_checked_tokens_lie_at_their_place():
    w = np.array([0.0, 0.5, 0.0, 0.25, 0.25])
    for u, t in itertools.product((0.0, 0.25, 0.6, 0.75 - 1e-9, 0.9, 1.0), range(5)):
        right = 1 if u < 0.5 else 3 if u < 0.75 else 4
        try:
            check_verified(np.array([t]), [0], [], [0, 0], [u], [(0, w)])
            ok = True
        except AssertionError:
            ok = False
        assert ok == (t == right), (u, t)


# ------------------------------------------------------------------- refusals
BAD_PAGES = [dict(rows=0), dict(rows=8193), dict(pages=0), dict(width=0), dict(page=8), dict(page=24), dict(page=2048), dict(page_table=0),
             dict(kv_lens=0x20002), dict(refs=None), dict(refs=0x30004), dict(pages=1 << 27), dict(width=1 << 27), dict(rows=1 << 31)]


@pytest.mark.parametrize("bad", BAD_PAGES, ids=str)
def test_bad_pages_are_refused(lib, bad):  # noqa: F811
    p = _pages(**bad)
    assert lib.ovc_kv_pages_reserve(R(p), B(0x1000), B(0x2000), B(0x3000), B(0x4000), None) == BAD
    assert lib.ovc_kv_pages_release(R(p), B(0x1000), None) == BAD
    assert lib.ovc_kv_pages_fork(R(p), B(0x1000), B(0x2000), 1, None) == BAD
    c = _cache(pages=p.pages, page=p.page)
    assert lib.ovc_kv_compact(R(c), R(p), B(0x1000), 0, B(0x2000), 5, None) == BAD


def test_bad_lists_are_refused(lib):  # noqa: F811
    p, c = _pages(), _cache()
    for x in (None, 0x1002):
        for i in range(4):
            args = [B(x if i == j else 0x1000 * (j + 1)) for j in range(4)]
            assert lib.ovc_kv_pages_reserve(R(p), *args, None) == BAD
        assert lib.ovc_kv_pages_release(R(p), B(x), None) == BAD
        assert lib.ovc_kv_pages_fork(R(p), B(x), B(0x2000), 1, None) == BAD
        assert lib.ovc_kv_pages_fork(R(p), B(0x1000), B(x), 1, None) == BAD
        assert lib.ovc_kv_copy(R(c), None, B(x), B(0x2000), None, 1, None) == BAD
        assert lib.ovc_kv_copy(R(c), None, B(0x1000), B(x), None, 1, None) == BAD
        assert lib.ovc_kv_compact(R(c), R(p), B(x), 0, B(0x2000), 5, None) == BAD
        assert lib.ovc_kv_compact(R(c), R(p), B(0x1000), 0, B(x), 5, None) == BAD
    assert lib.ovc_kv_copy(R(c), None, B(0x1000), B(0x2000), B(0x3002), 1, None) == BAD
    for n in (0, -1, 4):
        assert lib.ovc_kv_pages_fork(R(p), B(0x1000), B(0x2000), n, None) == BAD
    for n in (0, -1, 1 << 31):
        assert lib.ovc_kv_copy(R(c), None, B(0x1000), B(0x2000), None, n, None) == BAD
        assert lib.ovc_kv_compact(R(c), R(p), B(0x1000), 0, B(0x2000), n, None) == BAD
    for stride in (4, -1):
        assert lib.ovc_kv_compact(R(c), R(p), B(0x1000), stride, B(0x2000), 5, None) == BAD
    for other in (dict(heads=3), dict(page=32), dict(k=0x10008)):
        assert lib.ovc_kv_copy(R(c), R(_cache(**other)), B(0x1000), B(0x2000), None, 1, None) == BAD
    for other in (dict(pages=5), dict(page=32), dict(heads=32768)):
        assert lib.ovc_kv_compact(R(_cache(**other)), R(p), B(0x1000), 0, B(0x2000), 5, None) == BAD
    assert lib.ovc_kv_pages_release(None, B(0x1000), None) == BAD
    assert lib.ovc_kv_compact(None, R(p), B(0x1000), 0, B(0x2000), 5, None) == BAD


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_bad_caches_are_not_copied(lib, bad):  # noqa: F811
    c = _cache(**bad)
    assert lib.ovc_kv_copy(R(c), None, B(0x1000), B(0x2000), None, 1, None) == BAD
    assert lib.ovc_kv_copy(R(_cache()), R(c), B(0x1000), B(0x2000), None, 1, None) == BAD


@pytest.mark.parametrize("bad", [dict(B=0), dict(B=1 << 24), dict(N=-1), dict(V=0), dict(V=1 << 31), dict(N=1 << 31),
                                 dict(cu_drafts=0x10002), dict(cu_drafts=None, N=7), dict(drafts=0), dict(drafts=0x20001),
                                 dict(target=0), dict(target=0x30002), dict(draft=0x40002), dict(accept_u=0),
                                 dict(sample_u=0), dict(sample_u=0x60002), dict(target_stride=-1), dict(draft_stride=-1)], ids=str)
def test_bad_drafts_are_refused(lib, bad):  # noqa: F811
    assert lib.ovc_verify_drafts(R(_drafts(**bad)), B(0x1000), B(0x2000), None) == BAD


def test_drafts_outputs_and_types(lib):  # noqa: F811
    for t, a in ((None, 0x2000), (0x1000, None), (0x1002, 0x2000), (0x1000, 0x2001)):
        assert lib.ovc_verify_drafts(R(_drafts()), B(t), B(a), None) == BAD
    assert lib.ovc_verify_drafts(None, B(0x1000), B(0x2000), None) == BAD
    assert lib.ovc_verify_drafts(R(_drafts(dtype=3)), B(0x1000), B(0x2000), None) == _abi.OVC_ERR_UNSUPPORTED
    assert lib.ovc_verify_drafts(R(_drafts(dtype=_abi.OVC_BF16, target=0x30001)), B(0x1000), B(0x2000), None) == BAD
    if not torch.cuda.is_available():
        for kw in (dict(), dict(dtype=_abi.OVC_FP16, target=0x30002), dict(cu_drafts=None), dict(draft=None),
                   dict(N=0, drafts=None, accept_u=None)):
            assert lib.ovc_verify_drafts(R(_drafts(**kw)), B(0x1000), B(0x2000), None) in (_abi.OVC_ERR_CUDA, _abi.OVC_ERR_UNSUPPORTED)


def test_other_calls_take_no_fp32(lib):  # noqa: F811
    from test_paged import _rows
    x = _rows(dtype=_abi.OVC_FP32)
    assert lib.ovc_kv_write(R(_cache()), R(x), R(x), B(0x90000), None) == _abi.OVC_ERR_UNSUPPORTED


def test_bindings_refuse_cpu_tensors():
    i = torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ovc.KVPages(i, i[0], i[0], 16)
    p = torch.zeros((4, 10))
    with pytest.raises(ValueError, match="CUDA"):
        ovc.verify_drafts(p, i[:, :1], p[:2, :1], p[0, :2])
