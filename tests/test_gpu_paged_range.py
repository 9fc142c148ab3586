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
