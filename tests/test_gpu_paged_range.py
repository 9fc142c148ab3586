"""GPU tests of the paged cache's attention at the ends of its number range,
against the definition in 64 bits (paged_util)."""
import math

import pytest
import torch

import fp8_bit_attention_gb300 as ovc

from paged_util import attention, error_bounds
from test_gpu_paged import Case

pytestmark = pytest.mark.gpu

# Query rows of a sequence and query heads per KV head: the kernels' tiles of 8
# and 16 rows, 128 rows or fewer, several tiles of 256.
ROWS = [(3, 2), (4, 4), (9, 8), (80, 8)]


@pytest.fixture(scope="module", autouse=True)
def _build():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()
    ovc.device_status()


def _rewrite(c):
    ovc.kv_cache_write(c.cache, c.k, c.v, c.slots)


# ------------------------------------------------------------- sizes of values
@pytest.mark.parametrize("size", [1e-6, 1e-8, 1e-30])
@pytest.mark.parametrize("which", ["every fifth", "the first 400", "all but 20"])
@pytest.mark.parametrize("q_len, group", ROWS)
def test_zero_vectors_among_small_values(q_len, group, which, size):
    """A value vector of zeros adds nothing, whatever its scale byte (127) says."""
    n = 1500
    c = Case([q_len], [n], 2, group, 32, seed=31, k_mul=0.3)
    t = torch.arange(n, device="cuda")
    zero = {"every fifth": t % 5 == 3, "the first 400": t < 400, "all but 20": (t < 500) | (t >= 520)}[which]
    c.v = c.v * size
    c.v[zero] = 0.0
    c.v[zero & (t % 2 == 0)] = -0.0
    _rewrite(c)
    o, lse = c.run(return_lse=True)
    c.check(o, lse)
    assert (o != 0).any(-1).all()


def _check(c, o, lse, rows=None, terms=False, scale=None, **kw):
    """c.check for some rows.  With `terms`, a key's term may also be off by
    2^-20 of its row's largest, p * 448 * 2^(e-127): a weight keeps that much
    of the row's range, however the sizes of its values spread."""
    dense = c.dense()
    ref, ref_lse, av, sq = attention(c.q, dense, c.q_lens, c.kv_lens, c.group, scale=scale, **kw)
    eo, el = error_bounds(ref, ref_lse, av, sq)
    if terms:
        big = [(k, v.abs().amax(-1, keepdim=True).expand_as(v) * 2.0) for k, v in dense]     # 448 * 2^(e-127) at most
        most = torch.zeros_like(av[..., 0])
        for j in range(max(c.kv_lens)):
            one = [(k, torch.where((torch.arange(k.shape[0], device="cuda") == j)[:, None, None], v, 0.0)) for k, v in big]
            most = torch.maximum(most, attention(c.q, one, c.q_lens, c.kv_lens, c.group, scale=scale, **kw)[2].amax(-1))
        eo = eo + 2.0 ** -20 * max(c.kv_lens) * most.unsqueeze(-1)
    rows = slice(None) if rows is None else rows
    assert torch.isfinite(o[rows]).all()
    bad = ((o.double() - ref).abs() > eo)[rows]
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} values, worst {float(((o.double() - ref).abs() / eo)[rows].max()):.2f} bounds"
    d = torch.where(ref_lse == -math.inf, 0.0, (lse.double() - ref_lse).abs())
    assert (d <= el)[rows].all(), f"log-sum off by {float((d / el)[rows].max()):.2f} bounds"
    assert ovc.device_status() == 0


@pytest.mark.parametrize("huge", [1e30, 3e38])
@pytest.mark.parametrize("q_len, group", ROWS)
def test_a_huge_value_reaches_only_the_rows_that_see_it(q_len, group, huge):
    n = 1500
    at = n - q_len + q_len // 2 + 1
    c = Case([q_len], [n], 2, group, 32, seed=32)
    c.v[at, 0, 5] = huge
    c.v[at, 1, 99] = -huge
    _rewrite(c)
    o, lse = c.run(return_lse=True)
    before = slice(0, at - (n - q_len))
    _check(c, o, lse, before)
    seen = o[at - (n - q_len):]
    assert torch.isfinite(seen).all() and (seen[:, :group, 5] > 0).all() and (seen[:, group:, 99] < 0).all()


@pytest.mark.parametrize("q_len, group", ROWS)
def test_a_huge_value_before_the_window(q_len, group):
    n = 1500
    c = Case([q_len], [n], 2, group, 32, seed=33)
    c.v[n - q_len - 60] = 1e37
    _rewrite(c)
    o, lse = c.run(return_lse=True, window=60)
    _check(c, o, lse, window=60)


@pytest.mark.parametrize("weight", [-80.0, -60.0])
@pytest.mark.parametrize("q_len, group", ROWS)
def test_a_huge_value_with_a_weight_of_nearly_nothing(q_len, group, weight):
    """Its term is far below the others', or among them."""
    n = 700
    c = Case([q_len], [n], 2, group, 32, seed=34, k_mul=0.3)
    c.q[..., 0] = 32.0
    c.k[..., 0] = 0.0
    c.k[300, :, 0] = weight * math.sqrt(128.0) / 32.0
    c.k[300, :, 1:] = 0.0
    c.v[300] *= 2.0 ** 80
    _rewrite(c)
    o, lse = c.run(return_lse=True)
    _check(c, o, lse, terms=True)


@pytest.mark.parametrize("spread", [40, 100])
@pytest.mark.parametrize("q_len, group", ROWS)
def test_values_of_every_size(q_len, group, spread):
    c = Case([q_len, q_len], [600, 333], 2, group, 32, seed=35, k_mul=2.0, v_spread=spread)
    o, lse = c.run(return_lse=True)
    _check(c, o, lse, terms=True)
    o2, lse2 = c.run(return_lse=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


# ------------------------------------------------------------- sizes of scores
@pytest.mark.parametrize("scale", [1e-30, 1e-44])
@pytest.mark.parametrize("q_len, group", ROWS)
def test_scales_next_to_nothing(q_len, group, scale):
    """All weights alike: each row's mean of the values that it sees."""
    c = Case([q_len], [700], 2, group, 32, seed=38)
    c.q = c.q * 2.0 ** -20
    o, lse = c.run(return_lse=True, softmax_scale=scale)
    _check(c, o, lse, scale=scale)
    o, lse = c.run(return_lse=True, softmax_scale=scale, window=100)
    _check(c, o, lse, scale=scale, window=100)


@pytest.mark.parametrize("power", [6, 24, 36, 100])
@pytest.mark.parametrize("most, mul", [(4, 1.0), (7, 1.5)])
@pytest.mark.parametrize("q_len, group", ROWS)
def test_scores_far_apart(q_len, group, most, mul, power):
    """Scores of whole multiples of mul * 2^power / sqrt(128): beyond power 6 a row gives
    the mean of the values at its largest one.  Equal scores have to stay equal, and
    the largest has to have the weight 1, however large it is."""
    n = 700
    c = Case([q_len], [n], 2, group, 32, seed=40)
    k = torch.randint(-most, most + 1, (n, 2), device="cuda", generator=torch.Generator("cuda").manual_seed(41))
    c.k[:] = 0.0
    c.k[..., 3] = k.to(c.k.dtype)
    sign = torch.where(c.q[..., 3] < 0, -1.0, 1.0)
    c.q[:] = 0.0
    c.q[..., 3] = sign * mul * 2.0 ** power
    _rewrite(c)
    o, lse = c.run(return_lse=True)
    # distances to the largest score from whole numbers: in the definition's own
    # 64 bits they would be lost beside scores of 2^100
    s = sign.double().unsqueeze(-1) * k.double().T.repeat_interleave(group, 0)           # [rows, heads, keys]
    seen = torch.arange(n, device="cuda") <= torch.arange(n - q_len, n, device="cuda").view(-1, 1, 1)
    s = torch.where(seen, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    unit = mul * 2.0 ** power / math.sqrt(128.0)
    w = torch.exp((s - top) * unit)
    total = w.sum(-1)
    v = c.dense()[0][1].repeat_interleave(group, 1)
    ref, av = (torch.einsum("thj,jhd->thd", w / total.unsqueeze(-1), x) for x in (v, v.abs()))
    ref_lse = top.squeeze(-1) * unit + total.log()
    # Scores share the factor's and their own last rounding, 2^-23: distances of up
    # to 14 units are off by 2^-19 of a unit, which matters while weights are left.
    ds = torch.full_like(ref_lse, 2.0 ** -19 * unit if power == 6 else 0.0)
    eo, _ = error_bounds(ref, ref_lse, av, 2.0 ** 15 * ds)
    assert ((o.double() - ref).abs() <= eo).all()
    assert ((lse.double() - ref_lse).abs() <= ds + 2.0 ** -20 + 2.0 ** -21 * ref_lse.abs()).all()
    assert ovc.device_status() == 0


# --------------------------------------------------------------- sizes of keys
@pytest.mark.parametrize("power", [118, -118])
@pytest.mark.parametrize("q_len, group", ROWS)
def test_large_keys_and_small_queries(q_len, group, power):
    """Scores of ordinary size, whatever the sizes they come from."""
    c = Case([q_len], [700], 2, group, 32, seed=36)
    c.k = c.k * 2.0 ** power
    c.q = c.q * 2.0 ** -power
    _rewrite(c)
    o, lse = c.run(return_lse=True)
    c.check(o, lse)


@pytest.mark.parametrize("q_len, group", ROWS)
def test_a_huge_key_reaches_only_the_rows_that_see_it(q_len, group):
    """Later rows have a single weight, or that token's is 0."""
    n = 700
    at = n - q_len + q_len // 2 + 1
    row = at - (n - q_len)
    c = Case([q_len], [n], 2, group, 32, seed=37)
    c.k[at] = 0.0
    c.k[at, :, 9] = 1e37
    c.q[..., 9] = torch.where(c.q[..., 9] < 0, -1.0, 1.0)
    _rewrite(c)
    o, lse = c.run(return_lse=True)
    _check(c, o, lse, slice(0, row))
    k, v = c.dense()[0]
    only = v[at].repeat_interleave(group, 0).unsqueeze(0).expand(q_len - row, -1, -1)
    up = c.q[row:, :, 9] > 0
    assert torch.equal(o[row:][up].double(), only[up].float().to(torch.bfloat16).double())
    # where it has no weight: the definition without it
    c.k[at, :, 9] = -1e37
    c.q[..., 9] = c.q[..., 9].abs()
    _rewrite(c)
    o, lse = c.run(return_lse=True)
    c.k[at, :, 9] = -2000.0
    _rewrite(c)
    _check(c, o, lse)


# --------------------------------------------------------------- sizes of queries
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("q_len, group", ROWS)
def test_a_query_channel_far_above_the_others(q_len, group, dtype):
    """The large channel's keys are small.  A query element is off by what lies
    below 2^-18 of its row's largest: half a subnormal step of E4M3, 2^-10, where
    the largest is scaled to between 224 and 448, is 2^-17.8 of it.  Each score is
    off by that much times scale * sum |k| more."""
    c = Case([q_len], [700], 2, group, 32, dtype, seed=39)
    c.q[..., 7] *= 2.0 ** 8
    c.k[..., 7] *= 2.0 ** -8
    _rewrite(c)
    o, lse = c.run(return_lse=True)
    dense = c.dense()
    ref, ref_lse, av, sq = attention(c.q, dense, c.q_lens, c.kv_lens, c.group)
    amax = c.q.double().abs().amax(-1)
    k1 = dense[0][0].abs().sum(-1).amax(0).repeat_interleave(group)
    more = 2.0 ** -17.8 * amax * k1 / math.sqrt(128.0)
    eo, el = error_bounds(ref, ref_lse, av, sq + 2.0 ** 15 * more)
    assert ((o.double() - ref).abs() <= eo).all() and ((lse.double() - ref_lse).abs() <= el).all()


# ------------------------------------------------------------ all of it at once
def _largest_terms(c, dense, causal=True, window=None):
    """max_j p_j * 448 * 2^(e_j - 127) of every row (at most: twice the largest
    magnitude of the vector), NaN tokens left out."""
    out, at = [], 0
    for (k, v), ql, kl in zip(dense, c.q_lens, c.kv_lens):
        x = c.q[at:at + ql].double()
        at += ql
        k, big = (t.repeat_interleave(c.group, 1) for t in (torch.nan_to_num(k), 2.0 * torch.nan_to_num(v).abs().amax(-1)))
        s = torch.einsum("thd,jhd->thj", x, k) / math.sqrt(128.0)
        j, pos = torch.arange(kl, device="cuda"), torch.arange(kl - ql, kl, device="cuda").unsqueeze(1)
        seen = (j <= pos) if causal else torch.ones((ql, kl), dtype=torch.bool, device="cuda")
        if window:
            seen = seen & (j > pos - window)
        p = torch.softmax(torch.where(seen.unsqueeze(1), s, -math.inf), -1)
        out.append((p * big.T).amax(-1))
    return torch.cat(out)


@pytest.mark.parametrize("mode", ["causal", "window", "all"])
@pytest.mark.parametrize("dtype, spread", [(torch.bfloat16, 40), (torch.float16, 12)])
@pytest.mark.parametrize("q_lens, group", [((1, 3), 2), ((4, 4), 4), ((9, 2), 8), ((70, 150), 4)])
def test_wide_values_and_nan_tokens_in_long_sequences(q_lens, group, dtype, spread, mode):
    """Parts cut between CTAs, zero vectors and tokens that are not finite among
    values of every size."""
    kw = {"causal": dict(), "window": dict(window=301), "all": dict(causal=False)}[mode]
    lens = [6000, 2111]
    c = Case(q_lens, lens, 2, group, 48, dtype, seed=42, k_mul=2.0, v_spread=spread)
    c.v[::7] = 0.0
    rows = sum(q_lens)
    if mode != "all":
        c.v[lens[0] - q_lens[0] // 2 - 1, 0, 3] = math.inf      # the last rows of the first sequence see it
        c.k[sum(lens) - 1, 1, 77] = math.nan                    # the last row of the second
    _rewrite(c)
    o, lse = c.run(return_lse=True, **kw)
    dense = c.dense()
    ref, ref_lse, av, sq = attention(c.q, dense, c.q_lens, c.kv_lens, group, **kw)
    want = torch.isnan(ref).any(-1) | torch.isnan(ref_lse)
    assert torch.equal(torch.isnan(o).any(-1), want) and torch.equal(torch.isnan(o).all(-1), want)
    assert int(want.sum()) == (0 if mode == "all" else group * (q_lens[0] // 2 + 1 + 1))
    eo, el = error_bounds(ref, ref_lse, av, sq)
    seen = 301 if mode == "window" else max(lens)
    eo = eo + 2.0 ** -20 * seen * _largest_terms(c, dense, **kw).unsqueeze(-1)
    ok = ~want
    assert ((o.double() - ref).abs() <= eo)[ok].all() and ((lse.double() - ref_lse).abs() <= el)[ok].all()
    o2, lse2 = c.run(return_lse=True, **kw)
    assert torch.equal(o.nan_to_num(), o2.nan_to_num()) and torch.equal(lse.nan_to_num(), lse2.nan_to_num())
    assert o.shape[0] == rows and ovc.device_status() == 0


@pytest.mark.parametrize("q_len, group", ROWS)
def test_fp16_queries_over_a_huge_bf16_key(q_len, group):
    n = 700
    at = n - q_len + q_len // 2 + 1
    c = Case([q_len], [n], 2, group, 32, seed=43)
    c.k[at] = 3e38
    c.v[at] = -3e38
    _rewrite(c)
    c.q = c.q.half()
    o, lse = c.run(return_lse=True)
    _check(c, o, lse, slice(0, at - (n - q_len)))
