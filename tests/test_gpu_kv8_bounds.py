"""Counts that do not fit what the host said, rows that no sequence owns, numbers at
the ends of fp32's range."""
import math

import pytest
import torch

from tests.test_gpu_kv8 import (PEAK, assert_near, check_attention, cu_of, dense, fill, gen, ints,
                                make_cache, values, visible)

pytestmark = pytest.mark.gpu


def refused(tq_lib, c):
    with pytest.raises(tq_lib.TQError) as e:
        c.status()
    assert e.value.status == tq_lib.binding.TQ_ERR_ARG
    c.status()


def dirty(n):
    """Memory that a call may be handed holds anything."""
    torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("counts,max_q", [([1, 7], 1), ([2, 1], 1), ([5, 300], 4)])
def test_attention_counts_above_max_q(tq_lib, cuda, counts, max_q):
    """Computed all the same, or refused: never left as the memory was."""
    lens = [90, 400]
    c = fill(tq_lib, cuda, "i8", 2, 128, 32, lens)
    q = torch.randn(sum(counts), 8, 128, generator=gen(1)).to(torch.bfloat16).to(cuda)
    dirty(q.numel() * 2)
    lse = torch.full((sum(counts), 8), 7.0, device=cuda)
    out = c.attention(0, q, cu_of(counts, cuda), max_q, lse=lse)
    assert not (out.view(torch.int16) == 0x7F7F).any()
    refused(tq_lib, c)
    assert (out == 0).all() and (lse == -math.inf).all()
    check_attention(c, q, counts, lens)  # and afterwards it works


@pytest.mark.parametrize("counts", [[1, 1], [40, 60]])
def test_attention_counts_beyond_q(tq_lib, cuda, counts):
    """cu that names more tokens than q has: refused."""
    lens = [90, 400]
    c = fill(tq_lib, cuda, "i8", 2, 128, 32, lens)
    q = torch.randn(sum(counts) - 1, 8, 128, generator=gen(1)).to(torch.bfloat16).to(cuda)
    out = c.attention(0, q, cu_of(counts, cuda), max(counts))
    refused(tq_lib, c)
    assert (out == 0).all()


@pytest.mark.parametrize("counts,max_new,short", [([40, 3], 3, 0), ([2, 1], 1, 0), ([3, 5], 5, 1),
                                                  ([3, 5], 5, 5), ([3, 5], 5, 7)])
def test_append_counts_above_max_new(tq_lib, cuda, counts, max_new, short):
    """More tokens than the host said, or than k has: refused, and later calls wait
    for status()."""
    c = make_cache(tq_lib, cuda, page=16, slots=2, max_pages=4, pages=8)
    c.reserve(ints([0, 1], cuda), ints(counts, cuda))
    c.status()
    x = torch.randn(sum(counts) - short, 2, 128, device=cuda).to(torch.bfloat16)
    c.append(0, x, x, cu_of(counts, cuda), max_new)
    refused(tq_lib, c)


@pytest.mark.parametrize("max_count", [1, 7, 40])
def test_read_more_than_max_count(tq_lib, cuda, max_count):
    """Every token that cu names is read, and rows behind them are 0."""
    lens = [90, 33]
    c = fill(tq_lib, cuda, "e4m3", 2, 64, 16, lens)
    counts, begin, total = [60, 33], [20, 0], 130
    want = [torch.cat([values(c, name, 0, i, b + n)[:, b:].transpose(0, 1)
                       for i, (b, n) in enumerate(zip(begin, counts))]) for name in "kv"]
    dirty(total * 2 * 64 * 4)
    dirty(total * 2 * 64 * 4)
    got = c.read(0, ints(begin, cuda), cu_of(counts, cuda), total, max_count, dtype=torch.float32)
    for g, w in zip(got, want):
        assert ((g[:93].cpu().double() - w).abs() <= w.abs() * 2.0 ** -23).all()
        assert (g[93:] == 0).all()
    for cu, most in (([0], 4), ([0, 0, 0], 0)):
        dirty(total * 2 * 64 * 4)
        dirty(total * 2 * 64 * 4)
        n = len(cu) - 1
        got = c.read(0, ints(begin[:n], cuda), ints(cu, cuda), total, most, dtype=torch.float32)
        assert all((g == 0).all() for g in got)


@pytest.mark.parametrize("counts,max_q", [([1, 1], 1), ([3, 1], 4), ([64, 30], 64), ([1, 100], 100)])
def test_attention_rows_behind(tq_lib, cuda, counts, max_q):
    """A padded q: the rows behind the last sequence's are 0 in an output that the
    call allocates, and stay as they were in one that is given."""
    lens = [90, 400]
    c = fill(tq_lib, cuda, "i8", 2, 64, 32, lens)
    used = sum(counts)
    q = torch.randn(used + 37, 8, 64, generator=gen(1)).to(torch.bfloat16).to(cuda)
    dirty(q.numel() * 2)
    out = c.attention(0, q, cu_of(counts, cuda), max_q)
    keep = torch.full_like(q, 3.0)
    c.attention(0, q, cu_of(counts, cuda), max_q, out=keep)
    c.status()
    assert (out[used:] == 0).all() and (keep[used:] == 3.0).all()
    assert torch.equal(out[:used], keep[:used])
    at = 0
    for i, (m, n) in enumerate(zip(counts, lens)):
        ref, bound, _ = dense(q[at:at + m].cpu(), values(c, "k", 0, i, n), values(c, "v", 0, i, n),
                              visible(m, n, True, 0), 64 ** -0.5)
        assert_near(out[at:at + m], ref, bound)
        at += m
    for cu, most in (([0], 4), ([0, 0, 0], 0), ([0, 0, 0], max_q)):  # entries without tokens
        dirty(q.numel() * 2)
        assert (c.attention(0, q, ints(cu, cuda), most) == 0).all()


@pytest.mark.parametrize("count", [1, 3, 40])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_lse_of_a_bad_query(tq_lib, cuda, count, bad):
    """A row whose query is not finite: NaN, in the log sum as well; the others as
    without it."""
    c = fill(tq_lib, cuda, "i8", 1, 128, 64, [300])
    q = torch.randn(count, 4, 128, generator=gen(1)).to(torch.bfloat16).to(cuda)
    cu = cu_of([count], cuda)
    good, lse0 = c.attention(0, q, cu, count, lse=(l := torch.zeros(count, 4, device=cuda))), l
    q[count - 1, 2, 5] = bad
    lse = torch.zeros(count, 4, device=cuda)
    out = c.attention(0, q, cu, count, lse=lse)
    c.status()
    hit = torch.zeros(count, 4, dtype=torch.bool, device=cuda)
    hit[count - 1, 2] = True
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(out[~hit], good[~hit]) and torch.equal(lse[~hit], lse0[~hit])


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
