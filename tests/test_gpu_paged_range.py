"""GPU tests of the paged cache's attention at the ends of its number range,
against the definition in 64 bits (paged_util)."""

import pytest
import torch

import fp8_bit_attention_gb300 as ovc

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
