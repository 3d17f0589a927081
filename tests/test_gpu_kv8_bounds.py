"""Counts that do not fit what the host said, rows that no sequence owns, numbers at
the ends of fp32's range."""
import math

import pytest
import torch

from tests.test_gpu_kv8 import (PEAK, assert_near, check_attention, cu_of, dense, fill, gen, ints,
                                make_cache, values, visible)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_append_tiny_values(tq_lib, cuda, fmt):
    """Maxima down to fp32's last bit, where max / M is a few units of 2^-149 itself:
    codes within their range, values within half a step (of the scale as it is
    held), signs kept."""
    units = [1, 63, 64, 127, 178, 190, 254, 255, 448, 500, 1000, 4000, 2 ** 15 + 1, 2 ** 20 + 77]
    n = len(units)
    c = make_cache(tq_lib, cuda, fmt, heads=1, page=16, slots=n, max_pages=1, pages=n)
    x = torch.zeros(n, 1, 128, dtype=torch.float64)
    for i, u in enumerate(units):
        x[i, 0, 0], x[i, 0, 1], x[i, 0, 2] = u, -u, u // 3
    x = (x * 2.0 ** -149).float().to(cuda)
    one = ints([1] * n, cuda)
    c.reserve(ints(range(n), cuda), one)
    c.append(0, x, x, cu_of([1] * n, cuda), 1)
    c.status()
    for i in range(n):
        s = float(c.kscale[0, int(c.table[i, 0]), 0].double())
        got, want = values(c, "k", 0, i, 1)[0, 0], x[i, 0].cpu().double()
        assert s * PEAK[fmt] >= float(want.max()) * (1 - 2.0 ** -23)
        assert float(got.abs().max()) <= float(want.max()) + s / 2 * (32 if fmt == "e4m3" else 1)
        step = s / 2 if fmt == "i8" else (want.abs() * 2.0 ** -4).clamp_min(s * 2.0 ** -10)
        # (the reciprocal of the scale: 2^-23 of a code)
        assert ((got - want).abs() <= step * (1 + 2.0 ** -10) + s * PEAK[fmt] * 2.0 ** -22).all(), units[i]
        assert (got * want >= 0).all()
