"""Attention over the 8-bit cache where value scales differ widely: what a row does
not see, or hardly weighs, has no say in how precisely the rest is summed."""
import math

import pytest
import torch

from tests.test_gpu_kv8 import PEAK, U, cu_of, fill, gen, ints, make_cache, values, visible

pytestmark = pytest.mark.gpu


def scales(cache, slot, n):
    """[heads, n] fp64 value scales of a slot's tokens."""
    ids = cache.table[slot, torch.arange(n, device=cache.device) // cache.page].long()
    return cache.vscale[0][ids].cpu().double().T


def check(c, fmt, q, counts, lens, causal=True, window=0, scale=None, skip=(0, 0)):
    """Against fp64, relative to what each row sees; skip: last rows of each sequence
    that are not looked at.

    Bound.  Logits as in the other tests: a sum of d exact products and a few
    scalings, off by (d + 9) 2^-23 B with B = max sum |q k| scale; a probability by
    twice that and 2^-21.  Probability times scale is rounded to a half, 2^-11, with
    the row's largest such product at 2^5 at least: what falls below halves' normal
    range is off by 2^-25, 2^-30 of that largest product, times a code.  fp32 sums of
    n terms: n 2^-24; the result's own rounding."""
    dev, scale = c.device, c.d ** -0.5 if scale is None else scale
    out = c.attention(0, q, cu_of(counts, dev), max(counts), causal=causal, window=window, scale=scale)
    c.status()
    at = 0
    for i, (m, n, less) in enumerate(zip(counts, lens, skip)):
        assert torch.isfinite(out[at:at + m - less]).all()
        k, v, s = values(c, "k", 0, i, n), values(c, "v", 0, i, n), scales(c, i, n)
        see = visible(m, n, causal, window)
        for h in range(q.shape[1]):
            g = h // (q.shape[1] // c.heads)
            qq = q[at:at + m, h].cpu().double()
            p = torch.softmax((qq @ k[g].T * scale).masked_fill(~see, -math.inf), 1)
            ref, mass = p @ v[g], p @ v[g].abs()
            B = float((qq.abs() @ k[g].abs().T).max()) * abs(scale)
            rel = 2 * (c.d + 9) * 2.0 ** -23 * B + 2.0 ** -21 + 2.0 ** -11 + n * 2.0 ** -24
            bound = rel * mass + n * 2.0 ** -30 * PEAK[fmt] * (p * s[g]).amax(1, keepdim=True)
            bound = bound + U[q.dtype] * (ref.abs() + bound) + 2.0 ** -25 * (q.dtype == torch.float16)
            far = (out[at:at + m, h].cpu().double() - ref).abs()
            ratio = (far / (bound + 1e-38))[:m - less]
            assert (ratio <= 1).all(), (i, h, float(ratio.max()))
        at += m
    return out


@pytest.mark.parametrize("factor", [2.0 ** 26, 2.0 ** 60, 2.0 ** 110])
@pytest.mark.parametrize("fmt,dt,d,page,counts", [
    ("i8", "bf16", 128, 16, [129, 60]), ("e4m3", "f16", 64, 16, [300, 129]), ("i8", "f16", 128, 64, [200, 90])])
def test_scales_of_later_pages(tq_lib, cuda, fmt, dt, d, page, counts, factor):
    """A later page's large values do not show in the rows before it, which are bit
    for bit what they are without them; the rows that see them are right where the
    type holds their results."""
    lens = [300, 129]
    c = fill(tq_lib, cuda, fmt, 2, d, page, lens)
    dtype = torch.bfloat16 if dt == "bf16" else torch.float16
    q = torch.randn(sum(counts), 4, d, generator=gen(1)).to(dtype).to(cuda)
    plain = c.attention(0, q, cu_of(counts, cuda), max(counts))
    tail = []
    for i, n in enumerate(lens):
        last = (n - 1) // page
        c.vscale[0, int(c.table[i, last])] *= factor
        tail.append(n - last * page)
    out = check(c, fmt, q, counts, lens, skip=tail if dt == "f16" else (0, 0))
    at = 0
    for m, t in zip(counts, tail):
        assert torch.equal(out[at:at + m - t], plain[at:at + m - t])
        at += m


@pytest.mark.parametrize("counts,window", [([1, 1], 9), ([2, 3], 20), ([30, 64], 33)])
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_scales_outside_the_window(tq_lib, cuda, fmt, counts, window):
    """Pages that lie outside every row's window, in the tiles that hold it too."""
    lens = [300, 129]
    c = fill(tq_lib, cuda, fmt, 2, 128, 16, lens)
    for i, (m, n) in enumerate(zip(counts, lens)):
        first = max(0, n - m - window + 1) // 16  # the first page that a row sees
        for p in range(first):
            c.vscale[0, int(c.table[i, p])] *= 2.0 ** 40
    q = torch.randn(sum(counts), 4, 128, generator=gen(2)).to(torch.bfloat16).to(cuda)
    check(c, fmt, q, counts, lens, window=window)


@pytest.mark.parametrize("counts", [[1, 1], [3, 2], [90, 129]])
@pytest.mark.parametrize("fmt,d", [("i8", 128), ("e4m3", 64)])
def test_scales_spread(tq_lib, cuda, fmt, d, counts):
    """Scales over 80 powers of two, some 0, all visible."""
    lens = [300, 129]
    c = fill(tq_lib, cuda, fmt, 2, d, 16, lens)
    g = gen(3)
    e = torch.randint(-40, 41, c.vscale.shape, generator=g)
    c.vscale.copy_(2.0 ** e.float() * (torch.rand(e.shape, generator=g) > 0.1))
    q = torch.randn(sum(counts), 4, d, generator=g).to(torch.bfloat16).to(cuda)
    for causal in (True, False):
        check(c, fmt, q, counts, lens, causal=causal)


@pytest.mark.parametrize("count", [1, 40])
@pytest.mark.parametrize("sink_scale", [None, 0.0, 1e-30])
def test_attention_sink(tq_lib, cuda, count, sink_scale):
    """One key takes nearly all of a row's weight and adds nothing; the rest, at
    2^-25 of it and less each, makes the result."""
    n = 20000
    c = fill(tq_lib, cuda, "i8", 1, 128, 64, [n])
    c.v.copy_(c.v.abs().clamp(20, 100))
    page = int(c.table[0, 0])
    c.k[0, page, 0, 0] = 100
    c.v[0, page, 0, 0] = 0
    c.kscale.fill_(0.01)
    if sink_scale is not None:
        c.vscale[0, page] = sink_scale
    q = torch.randn(count, 2, 128, generator=gen(4)) * 0.2 + 0.3
    # the sink's logit: scale sum(q); the others' spread about 0
    scale = 18.0 / 38.4
    check(c, "i8", q.to(torch.float16).to(cuda), [count], [n], scale=scale)


def test_a_later_infinity(tq_lib, cuda):
    """An infinite value of the last token, held as 2^127, leaves the results of the
    rows that do not see its page as they are."""
    g = gen(5)
    k, v = (torch.randn(100, 2, 128, generator=g).to(torch.bfloat16).to(cuda) for _ in "kv")
    q = torch.randn(100, 4, 128, generator=g).to(torch.bfloat16).to(cuda)
    got = []
    for last in (1.0, math.inf):
        c = make_cache(tq_lib, cuda, "i8", page=16, slots=1, max_pages=8, pages=8)
        v[99] = last
        c.reserve(ints([0], cuda), ints([100], cuda))
        c.append(0, k, v, cu_of([100], cuda), 100)
        got.append(c.attention(0, q, cu_of([100], cuda), 100)[:96])
    assert torch.equal(*got)


@pytest.mark.parametrize("count", [1, 40])
def test_small_query_coordinates(tq_lib, cuda, count):
    """A query's small coordinates count beside large ones: the large ones' keys are
    0, so the logits are the small ones' alone."""
    n = 200
    c = fill(tq_lib, cuda, "i8", 1, 128, 64, [n])
    c.k[..., :64] = 0
    q = torch.randn(count, 2, 128, generator=gen(6))
    q[..., 64:] *= 2.0 ** -20
    q[..., :64] = 1.0
    check(c, "i8", q.to(torch.bfloat16).to(cuda), [count], [n], scale=2.0 ** 20)


@pytest.mark.parametrize("count", [1, 3, 40])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("top", [1e3, 3e7, 1e9, 1e12, -1e9, 1e30])
def test_large_logits(tq_lib, cuda, count, page, top):
    """One key's logit is twice as large as any other's, up to 1e30: the result is its
    value, to the rounding of a probability of 1 times a scale (2^-11) and the type's."""
    n = 300
    c = fill(tq_lib, cuda, "i8", 1, 128, page, [n], scale_range=(0.9, 1.1))
    sign = 1 if top > 0 else -1
    c.k.copy_(c.k.abs().clamp(1, 50) * sign)
    c.kscale.fill_(0.01)
    at = int(c.table[0, 70 // page]), 70 % page
    c.k[0, at[0], 0, at[1]] = 100 * sign
    q = torch.ones(count, 2, 128, dtype=torch.bfloat16, device=cuda)
    lse = torch.zeros(count, 2, device=cuda)
    out = c.attention(0, q, cu_of([count], cuda), count, scale=top / 128, lse=lse)
    c.status()
    want = values(c, "v", 0, 0, n)[0, 70]
    if top < 0:  # (the sign of the codes and of the scale: the logits are positive)
        assert (lse > 0).all()
    far = (out.cpu().double() - want).abs()
    assert (far <= want.abs() * (2.0 ** -11 + U[torch.bfloat16]) * (1 + 2.0 ** -8) + 1e-12).all()
    assert ((lse.cpu().double() / abs(top) - 1).abs() <= 2.0 ** -18).all()


@pytest.mark.parametrize("count", [1, 3, 40])
@pytest.mark.parametrize("at", [0, 70, 200, 299])
@pytest.mark.parametrize("top", [3e7, 1e9, 1e12])
def test_a_large_logit_among_small_ones(tq_lib, cuda, count, at, top):
    """One key's logit, wherever it lies, is the only large one."""
    n = 300 + count
    c = fill(tq_lib, cuda, "i8", 1, 128, 64, [n], scale_range=(0.9, 1.1))
    c.k.zero_()
    c.kscale.fill_(0.01)
    c.k[0, int(c.table[0, at // 64]), 0, at % 64] = 100
    q = torch.ones(count, 2, 128, dtype=torch.bfloat16, device=cuda)
    out = c.attention(0, q, cu_of([count], cuda), count, scale=top / 128)
    c.status()
    want = values(c, "v", 0, 0, n)[0, at]
    far = (out.cpu().double() - want).abs()
    assert (far <= want.abs() * (2.0 ** -11 + U[torch.bfloat16]) * (1 + 2.0 ** -8) + 1e-12).all()
