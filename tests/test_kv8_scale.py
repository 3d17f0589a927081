"""Attention's scale without a GPU: refused where it leaves fp32 in units of log2."""
import ctypes as C

import pytest

from tests.test_kv8_refusals import _cache


@pytest.mark.parametrize("scale", [3e38, -3e38, 2.4e38])
def test_scales_that_leave_fp32(tq_lib, scale):
    B, L = tq_lib.binding, tq_lib.binding.lib
    c = C.byref(_cache(B))
    assert L.tq_kv8_attention(c, 0, 1, None, 256, 1, 1, 4, 256, B.TQ_BF16, 512, 128, scale, 1, 0, 256,
                              None, 256, 1 << 30, None) == B.TQ_ERR_ARG
