"""GPU tests of the paged FP8 cache and of attention over it, against the
definition in 64 bits (paged_util)."""
import math

import numpy as np
import pytest
import torch

import fp8_bit_attention_gb300 as ovc

from paged_util import attention, error_bounds, quantise, values

pytestmark = pytest.mark.gpu

BAD_INDEX = 7


@pytest.fixture(scope="module", autouse=True)
def _build():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()
    ovc.device_status()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _poisoned(pages, heads, page):
    """A cache whose unwritten slots hold the worst: NaN codes, NaN and huge scales."""
    c = ovc.kv_cache(pages, heads, page)
    c.k.fill_(0x7F)
    c.v.fill_(0xFF)
    c.k_scale.fill_(255)
    c.v_scale.fill_(254)
    return c


class Case:
    """A filled cache, its sequences and queries."""

    def __init__(self, q_lens, kv_lens, heads, group, page, dtype=torch.bfloat16, seed=0, k_mul=1.0, v_spread=0):
        g = _gen(seed)
        self.q_lens, self.kv_lens, self.group = list(q_lens), list(kv_lens), group
        used = [-(-n // page) for n in kv_lens]
        pages = sum(used) + 2
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        width = max(1, max(used)) + 1
        self.cache = _poisoned(pages, heads, page)
        self.table = torch.full((len(kv_lens), width), -77, dtype=torch.int32, device="cuda")   # what lies behind is not read
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = order[at:at + n]
            at += n
        total = sum(kv_lens)
        self.k = (_randn(g, total, heads, 128) * k_mul + _randn(g, heads, 128)).to(dtype)
        v = _randn(g, total, heads, 128)
        if v_spread:
            v = v * torch.exp2(torch.randint(-v_spread, v_spread + 1, (total, heads, 1), generator=g, device="cuda").float())
        self.v = v.to(dtype)
        self.slots = torch.cat([self.slot(b, torch.arange(n, device="cuda")) for b, n in enumerate(kv_lens)] +
                               [_i32([])]).to(torch.int32)
        if total:
            ovc.kv_cache_write(self.cache, self.k, self.v, self.slots)
        self.q = _randn(g, sum(q_lens), heads * group, 128).to(dtype)
        self.lens = _i32(kv_lens)
        self.cu = _i32(np.concatenate([[0], np.cumsum(q_lens)]))

    def slot(self, b, t):
        return (self.table[b, (t // self.cache.page)] * self.cache.page + t % self.cache.page).to(torch.int32)

    def dense(self):
        """K and V of each sequence as the cache holds them, in 64 bits."""
        c, out, at = self.cache, [], 0
        for n in self.kv_lens:
            s = self.slots[at:at + n].long()
            at += n
            p, r = s // c.page, s % c.page
            out.append((values(c.k[p, :, r], c.k_scale[p, :, r]), values(c.v[p, :, r], c.v_scale[p, :, r])))
        return out

    def run(self, **kw):
        if "cu_q" not in kw:
            kw.update(cu_q=self.cu, max_q=max(self.q_lens))
        return ovc.paged_attention(self.q, self.cache, self.table, self.lens, **kw)

    def check(self, got, lse=None, rows=None, **kw):
        o, ref_lse, av, sq = attention(self.q, self.dense(), self.q_lens, self.kv_lens, self.group, **kw)
        eo, el = error_bounds(o, ref_lse, av, sq)
        assert torch.isfinite(got).all()
        bad = (got.double() - o).abs() > eo
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} values, worst {float(((got.double() - o).abs() / eo).max()):.2f} bounds"
        if lse is not None:
            assert torch.equal(lse == -math.inf, ref_lse == -math.inf)
            d = torch.where(lse == -math.inf, 0.0, (lse.double() - ref_lse).abs())
            assert (d <= el).all(), f"log-sum off by {float((d / el).max()):.2f} bounds"
        assert ovc.device_status() == 0


# ------------------------------------------------------------------ the cache
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens, heads, page", [(1, 1, 16), (37, 3, 48), (1000, 8, 64), (5, 7, 1024)])
def test_write_and_read_back(dtype, tokens, heads, page):
    g = _gen(tokens)
    x = _randn(g, tokens, heads, 384) * torch.exp2(torch.randint(-12, 12, (tokens, heads, 1), generator=g, device="cuda").float())
    x = x.to(dtype)
    k, v = x[..., 128:256], x[..., 256:]                     # strided views
    pages = -(-tokens // page) + 2
    c = _poisoned(pages, heads, page)
    before = [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:tokens].to(torch.int32)
    skip = torch.zeros(tokens, dtype=torch.bool, device="cuda")
    skip[3::7] = True
    slots = torch.where(skip, -1 - slots, slots)
    ovc.kv_cache_write(c, k, v, slots)
    s = slots[~skip].long()
    for x, codes, scale, old_codes, old_scale in ((k, c.k, c.k_scale, before[0], before[2]), (v, c.v, c.v_scale, before[1], before[3])):
        want, byte = quantise(x[~skip].double().cpu().numpy())
        old_codes[s // page, :, s % page] = torch.from_numpy(want).cuda()
        old_scale[s // page, :, s % page] = torch.from_numpy(byte).cuda()
        assert torch.equal(codes, old_codes) and torch.equal(scale, old_scale)      # and every other slot as it was
    for out_type in (torch.bfloat16, torch.float16):
        rk, rv = ovc.kv_cache_read(c, slots, dtype=out_type)
        for got, codes, scale in ((rk, c.k, c.k_scale), (rv, c.v, c.v_scale)):
            assert got.dtype == out_type and not got[skip].any()
            want = values(codes[s // page, :, s % page], scale[s // page, :, s % page])
            assert torch.equal(got[~skip], want.to(torch.float32).to(out_type))
    assert ovc.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_write_special_values(dtype):
    info = torch.finfo(dtype)
    x = torch.zeros((12, 1, 128), device="cuda")
    x[1, 0, 3] = info.max
    x[2, 0, 3] = info.tiny
    x[3, 0, :] = info.tiny * 2.0 ** -3
    x[4] = 448.0
    x[5, 0, 9] = 450.0
    x[6, 0, 7] = math.inf
    x[7, 0, 7] = -math.inf
    x[8, 0, 7] = math.nan
    x[9, 0, :64], x[9, 0, 64:] = info.max, -info.tiny
    x[10] = torch.arange(128, device="cuda") * 2.0 ** -9 / 2     # subnormal codes and ties
    x[10, 0, 127] = 400.0
    x[11] = -0.0
    x = x.to(dtype)
    c = _poisoned(1, 1, 16)
    ovc.kv_cache_write(c, x, x.flip(0), _i32(range(12)))
    codes, byte = quantise(x.double().cpu().numpy())
    assert np.array_equal(c.k[0, 0, :12].cpu().numpy(), codes[:, 0]) and np.array_equal(c.k_scale[0, 0, :12].cpu().numpy(), byte[:, 0])
    assert torch.equal(c.v[0, 0, :12], c.k[0, 0, :12].flip(0)) and torch.equal(c.v_scale[0, 0, :12], c.k_scale[0, 0, :12].flip(0))
    k, _ = ovc.kv_cache_read(c, _i32(range(12)), dtype=dtype)
    want = values(c.k[0, :, :12], c.k_scale[0, :, :12]).transpose(0, 1).float().to(dtype)
    assert torch.equal(torch.isnan(k), torch.isnan(want)) and torch.isnan(k[6:9]).all()
    assert torch.equal(torch.nan_to_num(k), torch.nan_to_num(want))


def test_slots_beyond_the_cache_are_skipped_and_reported():
    c = _poisoned(2, 2, 16)
    x = torch.ones((4, 2, 128), dtype=torch.bfloat16, device="cuda")
    ovc.kv_cache_write(c, x, x, _i32([0, 31, 32, 2 ** 31 - 1]))
    assert ovc.device_status() == BAD_INDEX and ovc.device_status() == 0
    assert (c.k == 0x7F).sum() == 30 * 2 * 128
    k, v = ovc.kv_cache_read(c, _i32([0, 32, 31, -5]))
    assert ovc.device_status() == BAD_INDEX and ovc.device_status() == 0
    assert (k[[0, 2]] == 1).all() and (v[[0, 2]] == 1).all() and not k[[1, 3]].any() and not v[[1, 3]].any()


def test_empty_calls():
    c = _poisoned(1, 2, 16)
    none = torch.empty((0, 2, 128), dtype=torch.float16, device="cuda")
    ovc.kv_cache_write(c, none, none, _i32([]))
    k, v = ovc.kv_cache_read(c, _i32([]), dtype=torch.float16)
    assert k.shape == v.shape == (0, 2, 128)
    table = torch.zeros((3, 1), dtype=torch.int32, device="cuda")
    o, lse = ovc.paged_attention(none, c, table, _i32([0, 0, 0]), cu_q=_i32([0, 0, 0, 0]), return_lse=True)
    assert o.shape == (0, 2, 128) and lse.shape == (0, 2)


# -------------------------------------------------------------- the attention
DECODE = [
    # kv_lens, heads, group, page
    ([1], 1, 1, 16),
    ([17], 2, 7, 16),
    ([5, 0, 33, 64, 1], 3, 4, 32),
    ([1000, 31, 257], 2, 8, 48),
    ([4097, 2, 513], 1, 16, 64),
    ([300, 900], 2, 17, 128),
    ([2000], 1, 33, 16),
    ([777, 64], 1, 100, 1024),
    ([65, 9000, 1234, 128] * 8, 4, 3, 64),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kv_lens, heads, group, page", DECODE)
def test_single_tokens(kv_lens, heads, group, page, dtype):
    c = Case([1] * len(kv_lens), kv_lens, heads, group, page, dtype, seed=len(kv_lens) + group)
    o, lse = c.run(cu_q=None, return_lse=True)
    c.check(o, lse)
    o2, lse2 = c.run(cu_q=None, return_lse=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)         # the same call gives the same bits


CHUNKS = [
    # q_lens, kv_lens, heads, group, page
    ([2], [2], 1, 1, 16),
    ([4, 4, 4], [100, 4, 3], 2, 2, 16),                # the last: more rows than tokens
    ([8, 1, 3], [777, 64, 500], 1, 4, 32),
    ([33], [33], 2, 1, 64),
    ([100, 0, 7], [1000, 50, 0], 2, 3, 48),
    ([128, 129], [128, 1000], 1, 2, 64),
    ([300, 1, 2], [300, 2000, 1999], 2, 7, 16),
    ([257], [5000], 1, 8, 128),
    ([511, 64], [600, 4100], 3, 1, 256),
    ([20, 1, 1, 1, 30], [20, 900, 1, 33, 4000], 2, 16, 64),
    ([3], [40000], 2, 5, 64),
]


@pytest.mark.parametrize("mode", ["causal", "window", "all"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("q_lens, kv_lens, heads, group, page", CHUNKS)
def test_chunks(q_lens, kv_lens, heads, group, page, dtype, mode):
    c = Case(q_lens, kv_lens, heads, group, page, dtype, seed=sum(q_lens))
    kw = {"causal": dict(), "window": dict(window=45), "all": dict(causal=False)}[mode]
    o, lse = c.run(return_lse=True, **kw)
    c.check(o, lse, **kw)
    o2, lse2 = c.run(return_lse=True, **kw)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("window", [1, 16, 31, 128, 1000, 10 ** 6])
@pytest.mark.parametrize("q_len", [1, 5, 200])
def test_windows(q_len, window):
    c = Case([q_len, q_len], [1500, q_len], 2, 4, 32, seed=window)
    c.check(c.run(window=window), window=window)


@pytest.mark.parametrize("q_len", [1, 300])
@pytest.mark.parametrize("scale", [0.01, 1.0])
def test_softmax_scale(q_len, scale):
    c = Case([q_len], [700], 1, 4, 16, seed=3)
    o, lse = c.run(softmax_scale=scale, return_lse=True)
    c.check(o, lse, scale=scale)


@pytest.mark.parametrize("q_len", [1, 4, 200])
def test_values_of_very_different_size(q_len):
    """Token scales that spread over 2^24, and keys that leave most weights tiny."""
    c = Case([q_len], [1111], 2, 3, 16, seed=9, k_mul=3.0, v_spread=12)
    o, lse = c.run(return_lse=True)
    c.check(o, lse)


@pytest.mark.parametrize("max_q", [None, 1, 4000])
def test_max_q_only_chooses(max_q):
    c = Case([40, 1, 90], [500, 300, 90], 2, 4, 32, seed=4)
    c.check(c.run(cu_q=c.cu, max_q=max_q))


def test_one_row_each_with_and_without_cu_q():
    c = Case([1, 1, 1], [500, 33, 2000], 2, 4, 32, seed=5)
    assert torch.equal(c.run(cu_q=None), c.run())


@pytest.mark.parametrize("q_len", [3, 150])
@pytest.mark.parametrize("which", ["k", "v"])
def test_nan_tokens_reach_only_the_rows_that_see_them(q_len, which):
    kv, at = 300, 300 - q_len + q_len // 2
    c = Case([q_len, q_len], [kv, kv], 2, 2, 32, seed=6)
    x = getattr(c, which)
    x[at, 1, 77] = math.nan
    x[kv + at, 0, 3] = math.inf
    ovc.kv_cache_write(c.cache, c.k, c.v, c.slots)
    o = c.run()
    row = at - (kv - q_len)
    want = torch.zeros((2 * q_len, 4), dtype=torch.bool, device="cuda")
    want[row:q_len, 2:] = True
    want[q_len + row:, :2] = True
    assert torch.equal(torch.isnan(o).all(-1), want) and torch.equal(torch.isnan(o).any(-1), want)
    clean = Case([q_len, q_len], [kv, kv], 2, 2, 32, seed=6)
    ref, ref_lse, av, sq = attention(clean.q, clean.dense(), clean.q_lens, clean.kv_lens, 2)
    eo, _ = error_bounds(ref, ref_lse, av, sq)
    assert ((o.double() - ref).abs() <= eo)[~want].all()
    # a window that has moved past the token is clean too
    w = c.run(window=1)
    assert int(torch.isnan(w).any(-1).sum()) == 4


@pytest.mark.parametrize("q_len", [1, 100])
def test_nan_queries(q_len):
    c = Case([q_len], [200], 1, 4, 16, seed=7)
    c.q[q_len - 1, 2, 5] = math.nan
    o = c.run()
    want = torch.zeros(o.shape[:2], dtype=torch.bool, device="cuda")
    want[q_len - 1, 2] = True
    assert torch.equal(torch.isnan(o).any(-1), want) and torch.equal(torch.isnan(o).all(-1), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("q_len", [1, 100])
def test_infinite_queries(q_len, dtype):
    """Also where every score would be minus infinity."""
    c = Case([q_len], [200], 1, 4, 16, dtype, seed=18)
    c.k[:, :, 5] = -1.0
    ovc.kv_cache_write(c.cache, c.k, c.v, c.slots)
    c.q[0, 1, 5] = math.inf
    c.q[q_len - 1, 2, 5] = -math.inf
    o, lse = c.run(return_lse=True)
    want = torch.zeros(o.shape[:2], dtype=torch.bool, device="cuda")
    want[0, 1] = want[q_len - 1, 2] = True
    assert torch.equal(torch.isnan(o).all(-1), want) and torch.equal(torch.isnan(o).any(-1), want)
    assert torch.equal(torch.isnan(lse), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("q_len", [4, 100])
def test_rows_without_keys_are_zero_whatever_they_hold(q_len, dtype):
    c = Case([q_len, q_len], [q_len - 3, 0], 1, 4, 16, dtype, seed=24)
    c.q[:3] = math.nan
    c.q[q_len:] = math.inf
    o, lse = c.run(return_lse=True)
    empty = torch.cat([torch.arange(3), torch.arange(q_len, 2 * q_len)]).cuda()
    assert (o[empty] == 0).all() and (lse[empty] == -math.inf).all()
    assert torch.isfinite(o[3:q_len]).all() and torch.isfinite(lse[3:q_len]).all()


@pytest.mark.parametrize("max_q", [1, 64])
def test_descending_row_starts_write_nothing(max_q):
    """Taken one by one, such sequences have 200 times q's rows, and work beyond 2^31 places."""
    c = Case([2000], [3000], 8, 8, 1024, seed=25)
    n = 400
    cu = _i32([2000 * (i % 2) for i in range(n + 1)])
    table = torch.zeros((n, 2048), dtype=torch.int32, device="cuda")
    out = torch.full(c.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lens = _i32([2 ** 21] * n)
    ovc.paged_attention(c.q, c.cache, table, lens, cu_q=cu, max_q=max_q, out=out)
    assert ovc.device_status() == BAD_INDEX and ovc.device_status() == 0
    assert (out == 7.0).all()


@pytest.mark.parametrize("window", [2 ** 31 - 1, 10 ** 12])
def test_windows_beyond_every_length(window):
    c = Case([300, 2, 40], [250, 900, 40], 1, 2, 16, seed=19)     # the first: more rows than tokens
    assert torch.equal(c.run(window=window), c.run())
    c.check(c.run(window=window))


@pytest.mark.parametrize("q_len", [1, 30])
def test_many_short_sequences(q_len):
    """More sequences than a CTA has threads, some without rows or tokens."""
    n = 700
    q_lens = [q_len if b % 7 else 0 for b in range(n)]
    kv_lens = [0 if b % 11 == 0 else max(q_lens[b], (b * 37) % 150) for b in range(n)]
    c = Case(q_lens, kv_lens, 2, 2, 16, seed=20)
    o, lse = c.run(return_lse=True)
    c.check(o, lse)


@pytest.mark.parametrize("q_len", [1, 64])
def test_page_tables_far_wider_than_the_sequences(q_len):
    """2^31 tokens' worth of page table, of which the lengths use a little."""
    c = Case([q_len] * 2, [3000, 500], 8, 2, 16, seed=21)
    wide = torch.empty((2, 1 << 27), dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    o = ovc.paged_attention(c.q, c.cache, wide, c.lens, cu_q=c.cu, max_q=q_len)
    c.check(o)


def test_calls_on_two_streams_at_once():
    cases = [Case([q] * 3, [900, 5000, 77], 2, 4, 32, seed=22 + q) for q in (1, 50)]
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(20):
        for i, (c, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                ovc.kv_cache_write(c.cache, c.k, c.v, c.slots)
                got[i].append(c.run())
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        assert all(torch.equal(w, o) for o in outs)
    assert ovc.device_status() == 0


@pytest.mark.parametrize("q_len", [1, 90])
def test_rows_of_no_sequence_keep_what_they_held(q_len):
    c = Case([q_len, q_len], [200, 60], 2, 2, 16, seed=8)
    q = torch.cat([c.q[:5], c.q, c.q[:7]])
    if q_len < 5:
        q = torch.cat([c.q[:1]] * 5 + [c.q] + [c.q[:1]] * 7)
    out = torch.full_like(q, 3.0, dtype=torch.bfloat16)
    got = ovc.paged_attention(q, c.cache, c.table, c.lens, cu_q=c.cu + 5, max_q=q_len, out=out)
    assert got is out and (out[:5] == 3).all() and (out[-7:] == 3).all()
    assert torch.equal(out[5:-7], c.run())


@pytest.mark.parametrize("q_len", [1, 70])
def test_strided_queries_and_output(q_len):
    c = Case([q_len] * 3, [100, 300, 500], 2, 4, 32, seed=11)
    wide = torch.zeros((3 * q_len, 20, 128), dtype=torch.bfloat16, device="cuda")
    wide[:, 5:13] = c.q
    big = torch.zeros((3 * q_len, 10, 256), dtype=torch.bfloat16, device="cuda")
    out = big[:, 1:9, 64:192]
    table = torch.full((3, 50), 10 ** 9, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = c.table
    got = ovc.paged_attention(wide[:, 5:13], c.cache, table[:, :c.table.shape[1]], c.lens, cu_q=c.cu, max_q=q_len, out=out)
    assert torch.equal(got, c.run())
    big[:, 1:9, 64:192] = 0
    assert not big.any()


@pytest.mark.parametrize("start, stride_t, stride_h", [(8, 0, 128), (0, 8, 128), (0, 0, 136)])
@pytest.mark.parametrize("q_len", [1, 200])
def test_rows_at_16_bytes(q_len, start, stride_t, stride_h):
    """Rows of q, of the output, of both at odd multiples of 16 bytes."""
    c = Case([q_len] * 2, [2100, 300], 2, 4, 32, seed=23)
    want = c.run()
    n, h = c.q.shape[:2]

    def odd(x, fill):
        flat = torch.full((start + n * (stride_h * h + stride_t),), fill, dtype=torch.bfloat16, device="cuda")
        y = flat.as_strided((n, h, 128), (stride_h * h + stride_t, stride_h, 1), start)
        return flat, y.copy_(x) if x is not None else y

    _, q = odd(c.q, 0.0)
    flat, out = odd(None, 7.0)
    for args in (dict(), dict(out=out)):
        got = ovc.paged_attention(q, c.cache, c.table, c.lens, cu_q=c.cu, max_q=q_len, **args)
        assert torch.equal(got, want)
    out.fill_(7.0)
    assert (flat == 7.0).all()                       # nothing between the rows was touched
    got = ovc.paged_attention(c.q, c.cache, c.table, c.lens, cu_q=c.cu, max_q=q_len, out=out)
    assert torch.equal(got, want)


@pytest.mark.parametrize("q_len, group", [(1, 8), (1, 16), (3, 8), (40, 8)])
def test_one_long_sequence_over_all_sms(q_len, group):
    c = Case([q_len], [70001], 1, group, 16, seed=26)
    o, lse = c.run(return_lse=True)
    c.check(o, lse)


@pytest.mark.parametrize("q_len", [1, 100])
def test_bad_pages_and_lengths_are_reported(q_len):
    c = Case([q_len, q_len], [400, 400], 2, 2, 16, seed=12)
    good = c.run()
    for bad in (-1, c.cache.pages, 2 ** 31 - 1, -2 ** 31):
        keep = int(c.table[0, 3])
        c.table[0, 3] = bad
        o = c.run()
        assert ovc.device_status() == BAD_INDEX and ovc.device_status() == 0
        assert torch.equal(o[q_len:], good[q_len:])
        c.table[0, 3] = keep
    for lens in ([10 ** 9, 400], [-5, 400]):
        c.lens = _i32(lens)
        c.run()
        assert ovc.device_status() == BAD_INDEX
    c.lens = _i32([400, 400])
    for cu in ([0, q_len, 10 ** 9], [-4, q_len, 2 * q_len], [0, 2 * q_len, q_len]):
        c.run(cu_q=_i32(cu), max_q=q_len)
        assert ovc.device_status() == BAD_INDEX
    assert torch.equal(c.run(), good) and ovc.device_status() == 0


@pytest.mark.parametrize("q_len", [1, 64])
def test_caches_beyond_32_bit_offsets(q_len):
    heads, page = 2, 64
    pages = (1 << 32) // (heads * page * 128) + 1000          # 4 GiB of codes and some more
    c = ovc.kv_cache(pages, heads, page)
    n = 3 * page - 5
    g = _gen(13)
    table = _i32([[pages - 1, 3, pages - 500]])
    t = torch.arange(n, device="cuda")
    slots = (table[0, t // page] * page + t % page).to(torch.int32)
    k, v = (_randn(g, n, heads, 128).to(torch.bfloat16) for _ in range(2))
    ovc.kv_cache_write(c, k, v, slots)
    rk, rv = ovc.kv_cache_read(c, slots)
    for x, got in ((k, rk), (v, rv)):
        codes, byte = quantise(x.double().cpu().numpy())
        assert torch.equal(values(torch.from_numpy(codes), torch.from_numpy(byte)), got.double().cpu())
    q = _randn(g, q_len, 2 * heads, 128).to(torch.bfloat16)
    o = ovc.paged_attention(q, c, table, _i32([n]), cu_q=_i32([0, q_len]), max_q=q_len)
    ref = attention(q, [(rk.double(), rv.double())], [q_len], [n], 2)
    eo, _ = error_bounds(*ref)
    assert ((o.double() - ref[0]).abs() <= eo).all()
    assert ovc.device_status() == 0


# ------------------------------------------------- streams, graphs, a whole run
@pytest.mark.parametrize("q_len", [1, 80])
def test_explicit_stream_and_workspace(q_len):
    c = Case([q_len] * 2, [3000, 700], 2, 4, 64, seed=14)
    want = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    need = ovc.paged_attention_workspace_bytes(c.q, c.cache, c.table, c.lens, cu_q=c.cu, max_q=q_len)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")       # holds NaN: nothing is read before it is written
    ws = ws[-ws.data_ptr() % 256:][:need]
    s.wait_stream(torch.cuda.current_stream())
    got = c.run(stream=s, workspace=ws)
    k, v = ovc.kv_cache_read(c.cache, c.slots, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    assert torch.equal(k, ovc.kv_cache_read(c.cache, c.slots)[0])
    with pytest.raises(ovc.OvcError):
        c.run(workspace=ws[:need - 256] if need > 256 else ws[:16])


@pytest.mark.parametrize("q_len", [1, 40])
def test_captured_steps_follow_new_lengths(q_len):
    """A decoding loop's step (write, then attend) captured once and replayed
    with new tokens, slots and lengths equals the eager calls; a second graph
    over the same workspace does too, replayed in turn."""
    heads, group, page, width = 2, 4, 16, 64
    cache, eager = _poisoned(140, heads, page), _poisoned(140, heads, page)
    g = _gen(15)
    table = torch.randperm(140, generator=g, device="cuda")[:2 * width].view(2, width).to(torch.int32).contiguous()
    rows = 2 * q_len
    q, k, v = (torch.zeros((rows, n, 128), dtype=torch.bfloat16, device="cuda") for n in (heads * group, heads, heads))
    slots, lens = torch.full((rows,), -1, dtype=torch.int32, device="cuda"), _i32([0, 0])
    cu = _i32([0, q_len, 2 * q_len])
    ws = torch.empty(ovc.paged_attention_workspace_bytes(q, cache, table, lens, cu_q=cu, max_q=q_len), dtype=torch.uint8, device="cuda")

    def step(c, **kw):
        ovc.kv_cache_write(c, k, v, slots)
        return ovc.paged_attention(q, c, table, lens, cu_q=cu, max_q=q_len, **kw)

    step(cache)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(cache, workspace=ws))
        graphs.append(graph)
    have = [0, 300]
    for i in range(5):
        have = [n + q_len for n in have]
        for x in (q, k, v):
            x.copy_(_randn(g, *x.shape))
        t = torch.cat([torch.arange(n - q_len, n, device="cuda") for n in have])
        b = torch.arange(2, device="cuda").repeat_interleave(q_len)
        slots.copy_(table[b, t // page] * page + t % page)
        if i == 0:                                   # what sequence 1 already holds
            old = torch.arange(300, device="cuda")
            os_ = (table[1, old // page] * page + old % page).to(torch.int32)
            ok = _randn(g, 300, heads, 128).to(torch.bfloat16)
            for c in (cache, eager):
                ovc.kv_cache_write(c, ok, ok, os_)
        lens.copy_(_i32(have))
        graphs[i % 2].replay()
        got = outs[i % 2].clone()
        assert torch.equal(got, step(eager))
    assert torch.equal(cache.k, eager.k) and torch.equal(cache.v_scale, eager.v_scale)
    assert ovc.device_status() == 0


def test_prefill_in_chunks_equals_one_call():
    """A prompt written and attended in chunks of odd sizes, then decoded: each
    step's rows as attention over the whole sequence gives them."""
    heads, group, page, n = 2, 4, 32, 900
    c = Case([n], [n], heads, group, page, seed=16)
    ref = attention(c.q, c.dense(), [n], [n], group)
    eo, el = error_bounds(*ref)
    fresh = _poisoned(c.cache.pages, heads, page)
    at = 0
    for step in (257, 1, 300, 1, 1, 31, 200, 109):
        sl = slice(at, at + step)
        at += step
        ovc.kv_cache_write(fresh, c.k[sl], c.v[sl], c.slots[sl])
        o, lse = ovc.paged_attention(c.q[sl], fresh, c.table, _i32([at]), cu_q=_i32([0, step]), max_q=step, return_lse=True)
        assert ((o.double() - ref[0][sl]).abs() <= eo[sl]).all()
        assert ((lse.double() - ref[1][sl]).abs() <= el[sl]).all()
    assert at == n and ovc.device_status() == 0


# ------------------------------------------------------------------- refusals
def test_refusals():
    c = Case([2, 3], [20, 30], 2, 2, 16, seed=17)
    q, t, n, cu = c.q, c.table, c.lens, c.cu
    bad = [
        dict(q=q.float()), dict(q=q[:, :3]), dict(q=q[..., :64]), dict(q=q[:, :, ::2]), dict(q=q.cpu()), dict(table=t.long()),
        dict(table=t[:1]), dict(n=n.long()), dict(n=n[:1]), dict(cu=cu[:2]), dict(cu=cu.long()), dict(cu=None), dict(window=0),
        dict(window=3, causal=False), dict(max_q=-1), dict(out=torch.empty_like(q[:2])), dict(out=torch.empty_like(q).half()),
        dict(out=torch.empty_like(q, device="cpu")), dict(workspace=torch.empty(1 << 20, device="cuda")),
        dict(workspace=torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 28)),
    ]
    for kw in bad:
        a = dict(q=q, table=t, n=n, cu=cu) | kw
        with pytest.raises((ValueError, TypeError)):
            ovc.paged_attention(a.pop("q"), c.cache, a.pop("table"), a.pop("n"), cu_q=a.pop("cu"), **a)
    k = c.k
    for args in ((k.float(), k.float(), c.slots), (k, k[:, :1], c.slots), (k, k.half(), c.slots), (k, k, c.slots.long()),
                 (k, k, c.slots[:3]), (k[..., :64], k[..., :64], c.slots), (k.cpu(), k.cpu(), c.slots.cpu())):
        with pytest.raises((ValueError, TypeError)):
            ovc.kv_cache_write(c.cache, *args)
    with pytest.raises(TypeError):
        ovc.kv_cache_read(c.cache, c.slots, dtype=torch.float32)
    with pytest.raises(ValueError):
        ovc.kv_cache_read(c.cache, c.slots.view(1, -1))
    with pytest.raises(ValueError):
        ovc.kv_cache_read(c.cache, c.slots, out=(k, k[:2]))
    with pytest.raises(ovc.OvcError):
        ovc.kv_cache_read(c.cache, c.slots, out=(k.clone(), k[:1].clone().expand_as(k)))
    with pytest.raises(ovc.OvcError):
        ovc.paged_attention(q, c.cache, t, n, cu_q=cu, out=torch.empty_like(q[:1]).expand_as(q))
    for shape in ((2, 1, 24), (2, 1, 2048), (0, 1, 16), (1 << 27, 1, 16)):
        with pytest.raises((ValueError, RuntimeError)):
            ovc.KVCache(*(torch.empty(1, dtype=torch.uint8, device="cuda").expand(*s) for s in (shape + (128,), shape + (128,), shape, shape)))
    assert ovc.device_status() == 0
