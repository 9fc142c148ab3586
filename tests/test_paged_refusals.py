"""CPU checks of refusals of the paged calls, before any device call."""
import ctypes
import math

import pytest
import torch

from fp8_bit_attention_gb300 import _abi

from test_paged import _batch, _cache, _rows, lib  # noqa: F401

R, B = ctypes.byref, ctypes.c_void_p


@pytest.mark.parametrize("scale, ok", [(math.nan, False), (math.inf, False), (3e38, False), (2e38, True), (1e-44, True),
                                       (0.0, True), (-1.0, True), (-math.inf, True)])
def test_softmax_scales_that_are_not_finite_are_refused(lib, scale, ok):  # noqa: F811
    """3e38 is finite, but not times log2(e)."""
    if ok and torch.cuda.is_available():
        pytest.skip("would launch on addresses that are none")
    st = lib.ovc_paged_attention(R(_rows()), R(_cache()), R(_batch()), scale, R(_rows()), None, B(0x100000), 1 << 30, None)
    assert (st == _abi.OVC_ERR_INVALID_ARG) == (not ok)
