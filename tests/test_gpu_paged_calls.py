"""GPU tests of how the paged cache's calls report and refuse."""
import pytest
import torch

import fp8_bit_attention_gb300 as ovc

from gpu_util import inputs, to_dev

pytestmark = pytest.mark.gpu

TIMEOUT, BAD_INDEX = 5, 7


@pytest.fixture(scope="module", autouse=True)
def _build():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()
    ovc.device_status()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_each_status_is_reported_in_its_turn():
    """A wait that ran out (the probe's, whose products are left out) and a slot
    beyond the cache: one call reports one of them and leaves the other."""
    prep = ovc.prepare(*to_dev(*inputs(1, 1, 256, seed=1)))
    ovc.attention_probe(prep, skip_mma=True, wait_timeout_ns=20_000_000)
    c = ovc.kv_cache(2, 1, 16)
    x = torch.ones((1, 1, 128), dtype=torch.bfloat16, device="cuda")
    ovc.kv_cache_write(c, x, x, _i32([32]))
    assert [ovc.device_status() for _ in range(3)] == [TIMEOUT, BAD_INDEX, 0]
    ovc.kv_cache_write(c, x, x, _i32([32]))
    assert [ovc.device_status() for _ in range(2)] == [BAD_INDEX, 0]


def test_one_tensor_for_keys_and_values_is_refused():
    """Each of its rows would hold parts of both."""
    c = ovc.kv_cache(2, 3, 16)
    x = torch.ones((5, 3, 128), dtype=torch.bfloat16, device="cuda")
    slots = _i32([1, 2, 3, 4, 20])
    ovc.kv_cache_write(c, x, 2 * x, slots)
    pair = torch.zeros((5, 6, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        ovc.kv_cache_read(c, slots, out=(pair[:, :3], pair[:, :3]))
    k, v = ovc.kv_cache_read(c, slots, out=(pair[:, :3], pair[:, 3:]))
    assert (k == 1).all() and (v == 2).all() and ovc.device_status() == 0
    none = pair[:0, :3]
    ovc.kv_cache_read(c, _i32([]), out=(none, none))
