"""The 8-bit paged cache and the rotary positions on the GPU, against plain
implementations in 64 bits.  Tolerances are derived where they stand."""
import itertools
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

CODE = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn}
PEAK = {"i8": 127.0, "e4m3": 448.0}
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def ints(v, device, dtype=torch.int32):
    return torch.tensor(list(v), dtype=dtype, device=device)


def cu_of(counts, device):
    return ints([0] + list(itertools.accumulate(counts)), device)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def values(cache, name, layer, slot, n):
    """[heads, n, d] fp64 values of a slot, on the CPU."""
    ids = cache.table[slot, :-(-n // cache.page)].long()
    codes = getattr(cache, name)[layer].view(torch.uint8)[ids].cpu().view(cache.k.dtype).double()
    x = codes * getattr(cache, name + "scale")[layer][ids].cpu().double()[..., None, None]
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


# ------------------------------------------------------------------ rope

def rope_ref(x, pos, r, transpose):
    """fp64 from the parameters' own frequencies: the angle's fraction of a turn in
    exact integers."""
    p, out = r.params, x.double().clone()
    for i in range(p.rot // 2):
        turn = torch.tensor([((int(t) * p.turns[i]) % 2 ** 64) / 2 ** 64 for t in pos],
                            dtype=torch.float64)
        c, s = torch.cos(2 * math.pi * turn)[:, None], torch.sin(2 * math.pi * turn)[:, None]
        s = -s if transpose else s
        a, b = (i, i + p.rot // 2) if p.layout == 0 else (2 * i, 2 * i + 1)
        x1, x2 = x[..., a].double(), x[..., b].double()
        out[..., a] = p.amplitude * (x1 * c - x2 * s)
        out[..., b] = p.amplitude * (x2 * c + x1 * s)
    return out


def rope_bound(x, r, ref):
    """One rounding to the type, on top of the fp32 arithmetic: the angle within
    1/8 turn and its 2-ulp sine and cosine (2^-25 pi/4 + 2^-23), amplitude, two
    products and a sum (4 roundings of 2^-24), of terms up to |x1| + |x2|."""
    big = x.double().abs().amax(-1, keepdim=True) * 2 * max(1.0, abs(r.params.amplitude))
    return ref.abs() * U[x.dtype] + big * 2.0 ** -21 + 2.0 ** -24 * (x.dtype == torch.float16)


@pytest.mark.parametrize("T,heads,d,rot,layout", [
    (1, 1, 128, 128, "half"), (7, 5, 64, 32, "interleaved"), (33, 32, 128, 64, "half"),
    (3, 2, 128, 6, "half"), (3, 2, 80, 20, "interleaved"), (5, 1, 6, 2, "half"),
    (300, 3, 256, 256, "half"), (2, 3, 128, 0, "half"), (17, 9, 96, 96, "interleaved")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_rope(tq_lib, cuda, T, heads, d, rot, layout, dtype):
    g = gen(T + d + rot)
    r = tq_lib.Rope(d, rot, base=1e4, layout=layout, amplitude=1.25)
    x = torch.randn(T, heads, d, generator=g).to(dtype)
    pos = torch.randint(0, 1 << 20, (T,), generator=g)
    pos[0] = 0
    if T > 2:
        pos[1], pos[2] = -5, (1 << 40) + 12345
    for transpose in (False, True):
        ref = rope_ref(x, pos.tolist(), r, transpose)
        got = r.apply(x.to(cuda), pos.to(cuda), transpose=transpose)
        assert got.dtype == dtype
        assert ((got.cpu().double() - ref).abs() <= rope_bound(x, r, ref)).all()
        # coordinates behind rot are copied
        assert torch.equal(got[..., rot:].cpu(), x[..., rot:])
        same = x.to(cuda)
        r.apply(same, pos.to(cuda), out=same, transpose=transpose)
        assert torch.equal(same, got)


def test_rope_strides_and_offsets(tq_lib, cuda):
    """Slices of a packed projection, odd offsets, transposed heads."""
    g = gen(3)
    r = tq_lib.Rope(64, layout="half")
    big = torch.randn(20, 7 * 64 + 3, generator=g).to(torch.bfloat16).to(cuda)
    pos = torch.arange(20, device=cuda)
    for off in (0, 1, 3, 8):
        x = big[:, off:off + 5 * 64].unflatten(1, (5, 64))
        ref = rope_ref(x.cpu(), range(20), r, False)
        assert ((r.apply(x, pos).cpu().double() - ref).abs() <= rope_bound(x.cpu(), r, ref)).all()
    x = torch.randn(5, 20, 64, generator=g).to(cuda).transpose(0, 1)
    ref = rope_ref(x.cpu(), range(20), r, False)
    assert ((r.apply(x, pos).cpu().double() - ref).abs() <= rope_bound(x.cpu(), r, ref)).all()
    out = torch.full((20, 5, 80), 7.0, device=cuda)
    r.apply(x, pos, out=out[..., :64])
    assert ((out[..., :64].cpu().double() - ref).abs() <= rope_bound(x.cpu(), r, ref)).all()
    assert (out[..., 64:] == 7.0).all()
    assert r.apply(x[:0], pos[:0]).shape == (0, 5, 64)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_gradient(tq_lib, cuda, layout):
    """Against the formula and against differences: the map is linear, so a
    central difference of step 1 is the derivative up to fp32's roundings."""
    g = gen(9)
    r = tq_lib.Rope(64, 32, layout=layout, amplitude=0.5)
    x = torch.randn(6, 2, 64, generator=g).to(cuda).requires_grad_()
    pos = torch.tensor([0, 1, 5, 1000, 70000, 131071], device=cuda)
    w = torch.randn(6, 2, 64, generator=g).to(cuda)
    (r(x, pos) * w).sum().backward()
    ref = rope_ref(w.cpu(), pos.tolist(), r, True)
    assert ((x.grad.cpu().double() - ref).abs() <= rope_bound(w.cpu(), r, ref)).all()
    for t, h, i in ((0, 0, 0), (3, 1, 7), (4, 0, 31), (5, 1, 40)):
        e = torch.zeros_like(w)
        e[t, h, i] = 1.0
        d = ((r.apply(x.detach() + e, pos) - r.apply(x.detach() - e, pos)).double() * w).sum() / 2
        # values up to 4 in both terms, 64 of them at most differ: 64 x 4 x 2^-21
        assert abs(float(d) - float(x.grad[t, h, i])) <= 2.0 ** -13


def test_rope_second_gradient(tq_lib, cuda):
    """The gradient of a squared gradient: g = R^T (w (R x)) with elementwise w, so
    d(sum g u)/dx = R^T (w (R u)), by the map's own forms."""
    g = gen(10)
    r = tq_lib.Rope(64, 64, layout="half")
    x, u, w = (torch.randn(3, 2, 64, generator=g).to(cuda) for _ in range(3))
    x.requires_grad_()
    pos = torch.tensor([3, 77, 5000], device=cuda)
    y = r(x, pos)
    first, = torch.autograd.grad((0.5 * w * y * y).sum(), x, create_graph=True)
    second, = torch.autograd.grad((first * u).sum(), x)
    # each map is within 2^-21 of its largest terms (rope_bound); two maps of values
    # up to 16 and a product: 16 x 2 x 2 x 2^-21
    want = r.apply(w * r.apply(u, pos), pos, transpose=True)
    assert ((second - want).abs() <= 2.0 ** -15).all()


# ------------------------------------------------------------------ append and read

def make_cache(tq_lib, dev, fmt="i8", layers=1, heads=2, d=128, page=64, slots=4, max_pages=8,
               pages=40, seed=0):
    """An empty cache whose pools hold random bytes (never-written rows)."""
    c = tq_lib.KV8Cache.empty(layers, pages, heads, d, slots, max_pages, page=page, dtype=CODE[fmt],
                              device=dev)
    for t in (c.k, c.v):
        t.view(torch.uint8).random_(0, 256, generator=torch.Generator(device=dev).manual_seed(seed))
    return c


def half_step(code, fmt):
    """Half the distance between neighbouring codes at a code's value."""
    if fmt == "i8":
        return torch.full_like(code, 0.5)
    e = torch.floor(torch.log2(code.abs().clamp_min(2.0 ** -6)))
    return 2.0 ** (e - 4)


def check_codes(cache, fmt, rows, name, slot, first, what):
    """Rows [heads, n, d] fp64 from position `first` lie within half a step of
    the codes: a quotient of fp32 numbers (2^-24), of keys turned in fp32
    (2^-21 of the largest coordinate): 2^-20 of the largest code."""
    n = rows.shape[1]
    got = values(cache, name, 0, slot, first + n)[:, first:]
    ids = cache.table[slot, torch.arange(first, first + n, device=cache.device) // cache.page].long()
    s = getattr(cache, name + "scale")[0][ids].cpu().double().T[..., None]  # [heads, n, 1]
    code = torch.where(s > 0, got / s, 0.0)
    x = torch.where(s > 0, rows / s, 0.0)
    assert (code.abs() <= PEAK[fmt] * (1 + 2 ** -20)).all(), what
    slack = PEAK[fmt] * 2.0 ** -20
    # at a power of two the steps below are half as wide, so the far half decides
    assert ((code - x).abs() <= half_step(code, fmt) * (1 + 2 ** -12) + slack).all(), what


@pytest.mark.parametrize("fmt,dtype,d,page,layout,rot", [
    ("i8", torch.bfloat16, 128, 64, "half", 128), ("e4m3", torch.float16, 64, 16, "interleaved", 32),
    ("i8", torch.float32, 128, 128, "interleaved", 128), ("e4m3", torch.bfloat16, 128, 32, "half", 40),
    ("i8", torch.float16, 64, 32, None, 0)])
def test_append_and_read(tq_lib, cuda, fmt, dtype, d, page, layout, rot):
    g = gen(d + page)
    c = make_cache(tq_lib, cuda, fmt, heads=3, d=d, page=page, slots=5, max_pages=10, pages=60)
    rope = tq_lib.Rope(d, rot, layout=layout) if layout else None
    slots = ints([3, 0, 4], cuda)
    kept = {i: {"k": [], "v": []} for i in (3, 0, 4)}
    scales = {}
    for step, counts in enumerate([(page + 5, 3, 2 * page), (1, 1, 1), (7, page, 1), (1, 0, 2)]):
        T = sum(counts)
        k, v = (torch.randn(T, 3, d, generator=g) * (step + 1) for _ in "kv")
        k, v = k.to(dtype), v.to(dtype)
        c.reserve(slots, ints(counts, cuda))
        c.append(0, k.to(cuda), v.to(cuda), cu_of(counts, cuda), max(counts), slots=slots, rope=rope)
        c.status()
        at = 0
        for slot, n in zip((3, 0, 4), counts):
            old = sum(x.shape[1] for x in kept[slot]["k"])
            kk = k[at:at + n]
            kk = rope_ref(kk, range(old, old + n), rope, False) if rope else kk.double()
            kept[slot]["k"].append(kk.transpose(0, 1))
            kept[slot]["v"].append(v[at:at + n].double().transpose(0, 1))
            at += n
            if n:  # the tokens of this step: one rounding
                for name in "kv":
                    check_codes(c, fmt, kept[slot][name][-1], name, slot, old, (step, slot, name))
    for slot in (3, 0, 4):
        n = sum(x.shape[1] for x in kept[slot]["k"])
        assert int(c.lens[slot]) == n
        for name in "kv":
            rows = torch.cat(kept[slot][name], 1)
            ids = c.table[slot, :-(-n // page)].long()
            s = getattr(c, name + "scale")[0][ids].cpu().double()
            for p in range(len(ids)):  # the scale of a page: its largest row, to fp32
                top = rows[:, p * page:(p + 1) * page].abs().amax((1, 2)) / PEAK[fmt]
                assert ((s[p] - top).abs() <= top * 2.0 ** -20).all()
            # all tokens: a step of the first rounding and of each that followed; a
            # page sees one for every append into it, 4 at most
            got = values(c, name, 0, slot, n)
            per = s.T[:, torch.arange(n) // page][..., None]
            far = (got - rows).abs()
            if fmt == "i8":
                assert (far <= per * 4 * 0.51).all()
            else:  # half a step of 2^-3 relative, or of 2^-9 absolute
                assert (far <= 4 * (rows.abs() * 2.0 ** -4 * 1.3 + per * 2.0 ** -9)).all()
    # read back: the codes' values, rounded once more
    begin, counts = [2, 0, page - 1], [page, 4, page + 3]
    rk, rv = c.read(0, ints(begin, cuda), cu_of(counts, cuda), sum(counts), max(counts), slots=slots,
                    dtype=dtype)
    at = 0
    for slot, b, n in zip((3, 0, 4), begin, counts):
        for name, r in (("k", rk), ("v", rv)):
            ref = values(c, name, 0, slot, b + n)[:, b:].transpose(0, 1)
            got = r[at:at + n].cpu().double()
            tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
            assert ((got - ref).abs() <= ref.abs() * (U[dtype] + 2.0 ** -23) + tiny).all()
        at += n


def test_append_leaves_other_rows(tq_lib, cuda):
    """Rows behind the last token, other pages and other layers keep their bytes."""
    c = make_cache(tq_lib, cuda, "i8", layers=2, page=32, slots=2, max_pages=4, pages=9)
    before = c.k.clone(), c.v.clone()
    c.reserve(ints([1], cuda), ints([40], cuda))
    x = torch.randn(40, 2, 128, device=cuda)
    c.append(1, x, x, cu_of([40], cuda), 40, slots=ints([1], cuda))
    ids = c.table[1, :2].tolist()
    assert ids == [0, 1]
    for old, new in zip(before, (c.k, c.v)):
        assert torch.equal(old[0], new[0]) and torch.equal(old[1, 2:], new[1, 2:])
        assert torch.equal(old[1, 1, :, 8:], new[1, 1, :, 8:])
        assert not torch.equal(old[1, 1, :, :8], new[1, 1, :, :8])


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_append_special_values(tq_lib, cuda, fmt):
    c = make_cache(tq_lib, cuda, fmt, page=16, slots=3, max_pages=2, pages=6)
    x = torch.zeros(3, 2, 128, device=cuda)
    x[1, 0, 5], x[1, 0, 6], x[1, 1, 3] = float("nan"), 2.0, -4.0  # NaN: as 0
    x[2, 0, 9], x[2, 0, 10] = float("inf"), 1.0                    # inf: as 2^127
    one = ints([1, 1, 1], cuda)
    c.reserve(ints([0, 1, 2], cuda), one)
    c.append(0, x, x, cu_of([1, 1, 1], cuda), 1)
    k, _ = c.read(0, ints([0, 0, 0], cuda), cu_of([1, 1, 1], cuda), 3, 1, dtype=torch.float32)
    assert (k[0] == 0).all() and (c.kscale[0, c.table[0, 0].long()] == 0).all()
    assert k[1, 0, 5] == 0 and k[1, 0, 6] == 2.0 and k[1, 1, 3] == -4.0
    assert abs(float(k[2, 0, 9]) / 2.0 ** 127 - 1) <= 2.0 ** -22 and k[2, 0, 10] == 0
    assert bool(torch.isfinite(k).all())
    # zeros first, then a value: the scale of zeros is 0, and the zeros stay
    c.reserve(ints([0], cuda), ints([1], cuda))
    y = torch.full((1, 2, 128), 3.0, device=cuda)
    c.append(0, y, y, cu_of([1], cuda), 1, slots=ints([0], cuda))
    k, v = c.read(0, ints([0], cuda), cu_of([2], cuda), 2, 2, slots=ints([0], cuda), dtype=torch.float32)
    assert (k[0] == 0).all() and ((k[1] - 3.0).abs() <= 3.0 * 2 ** -23).all() and torch.equal(k, v)


def test_append_strided_and_unaligned(tq_lib, cuda):
    """Slices of a packed projection, at 16-byte boundaries and off them, give the
    same bytes as their contiguous copies."""
    r = tq_lib.Rope(64, 48, layout="interleaved")
    packed = torch.randn(50, 6 * 64 + 8, device=cuda).to(torch.bfloat16)
    for off in (0, 8, 1):
        got = []
        for dense in (False, True):
            c = make_cache(tq_lib, cuda, "i8", d=64, page=32, slots=2, max_pages=3, pages=6)
            k = packed[:, off:off + 128].unflatten(1, (2, 64))
            v = packed[:, off + 128:off + 256].unflatten(1, (2, 64))
            if dense:
                k, v = k.contiguous(), v.contiguous()
            c.reserve(ints([0, 1], cuda), ints([17, 33], cuda))
            c.append(0, k, v, cu_of([17, 33], cuda), 33, rope=r)
            got.append((c.k.clone(), c.v.clone(), c.kscale.clone(), c.vscale.clone()))
        assert all(torch.equal(a, b) for a, b in zip(*got)), off


def test_absent_pages_are_passed_over(tq_lib, cuda):
    """Slots out of range and table entries that name no page: nothing is
    touched, reads give 0, attention sees only what is there."""
    c = make_cache(tq_lib, cuda, "e4m3", page=16, slots=3, max_pages=4, pages=8)
    c.reserve(ints([0, 1], cuda), ints([40, 20], cuda))
    x = torch.randn(60, 2, 128, device=cuda).to(torch.bfloat16)
    c.append(0, x, x, cu_of([40, 20], cuda), 40, slots=ints([0, 1], cuda))
    want = c.read(0, ints([0], cuda), cu_of([16], cuda), 16, 16, slots=ints([0], cuda))
    for absent in (-1, 8, 1 << 30):
        c.table[0, 1] = absent
        state = [t.view(torch.uint8) for t in (c.k, c.v, c.kscale, c.vscale)]  # (NaN codes too)
        before = [t.clone() for t in state]
        slots = ints([0, 99, -7], cuda)
        cu = cu_of([40, 3, 2], cuda)
        k, v = c.read(0, ints([0, 0, 0], cuda), cu, 45, 40, slots=slots)
        assert torch.equal(k[:16], want[0]) and torch.equal(v[:16], want[1])
        assert (k[16:32] == 0).all() and (k[40:] == 0).all() and (v[40:] == 0).all()
        q = torch.randn(45, 4, 128, device=cuda).to(torch.bfloat16)
        out = c.attention(0, q, cu, 40, slots=slots, causal=False)
        assert torch.isfinite(out).all() and (out[40:] == 0).all()
        keep = [j for j in range(40) if not 16 <= j < 32]
        kk, vv = (values_at(c, n, 0, keep) for n in "kv")
        ref = dense(q[:40].cpu(), kk, vv, torch.ones(40, len(keep), dtype=torch.bool), 128 ** -0.5)
        assert_near(out[:40], *ref)
        y = torch.randn(45, 2, 128, device=cuda).to(torch.bfloat16)
        c.append(0, y[16:32], y[16:32], cu_of([0, 16], cuda), 16, slots=ints([1, 77], cuda))
        assert all(torch.equal(a, b) for a, b in zip(before, state))


def values_at(c, name, slot, keep):
    rows = []
    for j in keep:
        p = int(c.table[slot, j // c.page])
        x = getattr(c, name)[0, p, :, j % c.page].cpu().double()
        rows.append(x * getattr(c, name + "scale")[0, p].cpu().double()[:, None])
    return torch.stack(rows, 1)


# ------------------------------------------------------------------ attention

def dense(q, k, v, see, scale):
    """fp64 attention of q [m, hq, d] over k, v [h, n, d]; see [m, n].  Returns
    out, its bound and the log sums.

    Bound.  A logit is an exact product sum rounded in fp32: at most d + 8
    additions and scalings of up to sum |q k| scale, so |dl| <= (d + 8) 2^-23 B,
    and B 2^-24 more for the row's unit; a probability moves by 2 |dl| + 2^-21
    (two exponentials' 2^-22), and is rounded to a half, 2^-11, or where it falls
    below halves' normal range by 2^-25 of the largest value scale x code.  All
    of it acts on sum p |v|; fp32 sums of n terms add n 2^-24 of that, and the
    result is rounded to its type."""
    m, hq, d = q.shape
    g = hq // k.shape[0]
    n = k.shape[1]
    out, bound = torch.zeros(m, hq, d, dtype=torch.float64), torch.zeros(m, hq, d, dtype=torch.float64)
    lse = torch.full((m, hq), -math.inf, dtype=torch.float64)
    if n and m:
        for h in range(hq):
            qq, kk, vv = q[:, h].double(), k[h // g], v[h // g]
            l = (qq @ kk.T * scale).masked_fill(~see, -math.inf)
            some = see.any(1)
            p = torch.where(some[:, None], torch.softmax(l, 1), 0.0)
            out[:, h] = p @ vv
            lse[:, h] = torch.logsumexp(l, 1)
            B = float((qq.abs() @ kk.abs().T).max()) * abs(scale)
            delta = 2 * (d + 9) * 2.0 ** -23 * B + 2.0 ** -21 + 2.0 ** -11 + n * 2.0 ** -24
            bound[:, h] = delta * (p @ vv.abs()) + n * 2.0 ** -25 * float(vv.abs().max())
    bound += U[q.dtype] * (out.abs() + bound) + (2.0 ** -25 if q.dtype == torch.float16 else 0.0)
    return out, bound, lse


def assert_near(got, ref, bound, lse=None):
    far = (got.cpu().double() - ref).abs()
    assert torch.isfinite(got).all()
    assert (far <= bound).all(), float((far / bound.clamp_min(1e-300)).max())


def visible(m, n, causal, window):
    pos, j = torch.arange(n - m, n)[:, None], torch.arange(n)[None]
    see = (j <= pos) if causal else torch.ones(m, n, dtype=torch.bool)
    return see & (j > pos - window) if window else see


def fill(tq_lib, dev, fmt, heads, d, page, lens, seed=5, scale_range=(0.5, 1.5), layers=1):
    """A cache of random codes at scattered pages; unwritten rows any bytes."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    c = make_cache(tq_lib, dev, fmt, layers, heads, d, page, len(lens), max(max(need), 1) + 1, pages, seed)
    g = gen(seed)
    ids = torch.randperm(pages, generator=g).tolist()
    unit = 40.0 if fmt == "i8" else 120.0
    for i, n in enumerate(lens):
        mine = [ids.pop() for _ in range(need[i])]
        c.table[i, :need[i]] = ints(mine, dev) if mine else c.table[i, :0]
        c.refs[mine] = 1
        for at, p in enumerate(mine):
            rows = min(page, n - at * page)
            for t in (c.k, c.v):
                x = torch.randn(layers, heads, rows, d, generator=g) * unit
                x = x.round().clamp(-127, 127) if fmt == "i8" else x.clamp(-448, 448)
                t.view(torch.uint8)[:, p, :, :rows] = x.to(c.k.dtype).view(torch.uint8).to(dev)
    lo, hi = scale_range
    for t in (c.kscale, c.vscale):
        t.copy_((torch.rand(t.shape, generator=g) * (hi - lo) + lo) / unit)
    c.lens.copy_(ints(lens, dev))
    return c


def check_attention(c, q, counts, lens, causal=True, window=0, scale=None, slots=None, layer=0):
    dev = c.device
    lse = torch.full(q.shape[:2], 7.0, device=dev)
    out = c.attention(layer, q, cu_of(counts, dev), max(counts), slots=slots, causal=causal,
                      window=window, scale=scale, lse=lse)
    c.status()
    at = 0
    for i, (m, n) in enumerate(zip(counts, lens)):
        slot = i if slots is None else int(slots[i])
        k, v = values(c, "k", layer, slot, n), values(c, "v", layer, slot, n)
        ref, bound, rl = dense(q[at:at + m].cpu(), k, v, visible(m, n, causal, window),
                               c.d ** -0.5 if scale is None else scale)
        if m:
            assert_near(out[at:at + m], ref, bound)
            got = lse[at:at + m].cpu().double()
            assert torch.equal(got == -math.inf, rl == -math.inf)
            some = rl > -math.inf
            assert ((got - rl)[some].abs() <= 1e-4 + 2.0 ** -20 * rl[some].abs()).all()
        at += m
    return out


CASES = [
    # fmt, dtype, heads, group, d, page, lens, counts, causal, window
    ("i8", "bf16", 2, 4, 128, 64, [1, 2, 31, 32, 33, 64, 65, 500], [1] * 8, True, 0),
    ("e4m3", "f16", 3, 1, 64, 16, [15, 16, 17, 48, 200], [1] * 5, True, 0),
    ("e4m3", "bf16", 1, 7, 128, 32, [5, 100, 33], [2, 3, 1], True, 0),
    ("i8", "f16", 2, 16, 64, 128, [129, 1000], [1, 4], True, 0),
    ("i8", "bf16", 2, 3, 128, 16, [70, 150, 40, 300], [70, 33, 1, 129], True, 0),
    ("e4m3", "f16", 1, 8, 64, 64, [260, 90], [130, 90], True, 0),
    ("e4m3", "bf16", 2, 2, 128, 64, [300, 77], [20, 77], True, 50),
    ("i8", "bf16", 2, 2, 64, 32, [300, 1, 64], [1, 1, 1], True, 1),
    ("i8", "f16", 2, 2, 128, 32, [130, 65], [65, 65], False, 0),
    # rows that see nothing: empty slots, more queries than tokens, no queries
    ("i8", "bf16", 2, 4, 128, 64, [0, 3, 10, 64], [1, 5, 0, 2], True, 0),
    ("e4m3", "bf16", 2, 4, 64, 16, [0, 3, 0, 20], [4, 40, 0, 70], True, 7),
    ("i8", "bf16", 1, 128, 128, 64, [200], [2], True, 0),
]


@pytest.mark.parametrize("fmt,dt,heads,group,d,page,lens,counts,causal,window", CASES)
def test_attention(tq_lib, cuda, fmt, dt, heads, group, d, page, lens, counts, causal, window):
    c = fill(tq_lib, cuda, fmt, heads, d, page, lens)
    dtype = torch.bfloat16 if dt == "bf16" else torch.float16
    q = torch.randn(sum(counts), heads * group, d, generator=gen(1)).to(dtype).to(cuda)
    check_attention(c, q, counts, lens, causal, window)


@pytest.mark.parametrize("fmt,counts", [("i8", [1, 1, 1]), ("e4m3", [2, 1, 1]), ("i8", [200, 1, 300])])
def test_attention_long(tq_lib, cuda, fmt, counts):
    """Lengths that are cut over many warps, beside short ones."""
    lens = [9001, 40, 3333]
    c = fill(tq_lib, cuda, fmt, 2, 128, 64, lens)
    q = torch.randn(sum(counts), 8, 128, generator=gen(2)).to(torch.bfloat16).to(cuda)
    check_attention(c, q, counts, lens)


@pytest.mark.parametrize("heads,group,lens,counts", [
    (1, 8, [60000], [1]), (1, 3, [20000, 5000, 9], [1, 4, 1]), (2, 16, [40000], [1]),
    (3, 1, [7000, 7001, 31, 2500, 64], [1, 1, 1, 1, 1]), (1, 1, [30000, 31000], [12, 1])])
def test_attention_over_many_blocks(tq_lib, cuda, heads, group, lens, counts):
    """Items over many blocks, two and more of them in a block, short ones between."""
    c = fill(tq_lib, cuda, "i8", heads, 64, 64, lens)
    q = torch.randn(sum(counts), heads * group, 64, generator=gen(2)).to(torch.bfloat16).to(cuda)
    first = check_attention(c, q, counts, lens)
    for _ in range(3):
        assert torch.equal(first, check_attention(c, q, counts, lens))


def test_attention_many_entries(tq_lib, cuda):
    """More entries than threads of a block, most of them without queries."""
    lens = [(i * 7) % 90 for i in range(700)]
    counts = [1 if i % 3 else 0 for i in range(700)]
    c = fill(tq_lib, cuda, "i8", 1, 64, 32, lens)
    q = torch.randn(sum(counts), 2, 64, generator=gen(2)).to(torch.float16).to(cuda)
    check_attention(c, q, counts, lens)


@pytest.mark.parametrize("counts", [[1, 1], [40, 70]])
def test_attention_scales_and_extremes(tq_lib, cuda, counts):
    """Block scales over many powers of two, queries large and tiny, a peaked
    softmax, a negative scale, zero scales."""
    lens = [300, 129]
    c = fill(tq_lib, cuda, "i8", 2, 128, 16, lens)
    g = gen(4)
    c.vscale.copy_(2.0 ** torch.randint(-20, 6, c.vscale.shape, generator=g).float())
    c.kscale.copy_(2.0 ** torch.randint(-12, -4, c.kscale.shape, generator=g).float())
    q = torch.randn(sum(counts), 4, 128, generator=g)
    for factor, scale in ((1.0, None), (1e30, 1e-31), (1e-30, 1e29), (30.0, None), (1.0, -0.3), (0.0, 1.0)):
        check_attention(c, (q * factor).to(torch.bfloat16).to(cuda), counts, lens, scale=scale)
    c.vscale.zero_()
    out = check_attention(c, q.to(torch.bfloat16).to(cuda), counts, lens)
    assert (out == 0).all()


def test_attention_slots_layers_strides_and_rows_behind(tq_lib, cuda):
    lens = [100, 7, 64, 250]
    c = fill(tq_lib, cuda, "e4m3", 2, 64, 32, lens, layers=3)
    packed = torch.randn(60, 5 * 64 + 64, generator=gen(6)).to(torch.bfloat16).to(cuda)
    q = packed[:, 64:64 + 256].unflatten(1, (4, 64))
    slots = ints([3, 0, 3], cuda)  # a slot twice is a batch of two
    counts = [1, 2, 1]
    for layer in (2, 0):
        out = check_attention(c, q[:4], counts, [lens[3], lens[0], lens[3]], slots=slots, layer=layer)
    # rows behind the last entry's stay as they were
    keep = torch.full((60, 4, 64), 3.0, dtype=torch.bfloat16, device=cuda)
    lse = torch.full((60, 4), 5.0, device=cuda)
    got = c.attention(0, q, cu_of(counts, cuda), 2, slots=slots, out=keep, lse=lse)
    assert torch.equal(got[:4], out) and (keep[4:] == 3.0).all() and (lse[4:] == 5.0).all()
    assert not torch.equal(lse[:4], torch.full_like(lse[:4], 5.0))


def test_attention_masked_rubbish(tq_lib, cuda):
    """NaN and extreme codes in the rows behind a slot's end change nothing."""
    lens, counts = [33, 100], [1, 40]
    got = []
    for byte in (0x00, 0x7F, 0xFF, 0x7E):
        c = fill(tq_lib, cuda, "e4m3", 2, 128, 64, lens)
        for i, n in enumerate(lens):
            p = int(c.table[i, n // 64])
            for t in (c.k, c.v):
                t.view(torch.uint8)[:, p, :, n % 64:] = byte
        q = torch.randn(41, 4, 128, generator=gen(8)).to(torch.bfloat16).to(cuda)
        got.append(c.attention(0, q, cu_of(counts, cuda), 40))
    assert all(torch.equal(got[0], x) for x in got[1:])
    assert torch.isfinite(got[0]).all()


@pytest.mark.parametrize("counts", [[1, 1, 1], [64, 100, 1]])
def test_attention_repeats_bit_for_bit(tq_lib, cuda, counts):
    lens = [5000, 321, 64]
    c = fill(tq_lib, cuda, "i8", 4, 128, 64, lens)
    q = torch.randn(sum(counts), 16, 128, generator=gen(8)).to(torch.bfloat16).to(cuda)
    first = c.attention(0, q, cu_of(counts, cuda), max(counts))
    for _ in range(5):
        assert torch.equal(first, c.attention(0, q, cu_of(counts, cuda), max(counts)))


@pytest.mark.parametrize("counts", [[2], [1, 3], [0, 7]])
def test_attention_padded_batch(tq_lib, cuda, counts):
    """q may be longer than the batch, and max_q larger than any count: every
    token of the batch is computed, what lies behind stays."""
    lens = [90, 300][:len(counts)]
    c = fill(tq_lib, cuda, "i8", 2, 64, 32, lens)
    total, used = 100 * len(counts), sum(counts)
    q = torch.randn(total, 8, 64, generator=gen(3)).to(torch.bfloat16).to(cuda)
    want = check_attention(c, q[:used], counts, lens)
    for max_q in (max(counts), 50, 100, 200):
        out = torch.full_like(q, 3.0)
        c.attention(0, q, cu_of(counts, cuda), max_q, out=out)
        c.status()
        at = 0
        for i, (m, n) in enumerate(zip(counts, lens)):
            k, v = values(c, "k", 0, i, n), values(c, "v", 0, i, n)
            ref, bound, _ = dense(q[at:at + m].cpu(), k, v, visible(m, n, True, 0), 64 ** -0.5)
            assert_near(out[at:at + m], ref, bound)
            at += m
        assert (out[used:] == 3.0).all()
        assert want.shape[0] == used


def test_attention_unaligned_queries(tq_lib, cuda):
    """Packed projections whose rows do not begin at 16 bytes, one token and one
    head among them (their strides count for nothing)."""
    c = fill(tq_lib, cuda, "i8", 1, 64, 32, [90])
    packed = torch.randn(4, 387, generator=gen(3)).to(torch.bfloat16).to(cuda)
    for q in (packed[:1, :256].unflatten(1, (4, 64)), packed[:, 3:67].unsqueeze(1),
              packed[:3, 1:257].unflatten(1, (4, 64)), packed[2:3, 64:128].unsqueeze(1)):
        check_attention(c, q, [q.shape[0]], [90])


@pytest.mark.parametrize("counts", [[5, 1], [90, 70]])
def test_attention_widest_window(tq_lib, cuda, counts):
    """Windows beyond every length, up to the largest int, hide nothing; more
    queries than tokens among them."""
    lens = [3, 200]
    c = fill(tq_lib, cuda, "i8", 2, 128, 64, lens)
    q = torch.randn(sum(counts), 4, 128, generator=gen(3)).to(torch.bfloat16).to(cuda)
    want = check_attention(c, q, counts, lens)
    for window in (1 << 20, 2 ** 31 - 1):
        got = c.attention(0, q, cu_of(counts, cuda), max(counts), window=window)
        assert torch.equal(got, want)


# ------------------------------------------------------------------ pages

class Model:
    """The page rules, one slot after another, in plain Python; a page is known by
    the content that was put into it."""

    def __init__(self, slots, max_pages, pages, page):
        self.table = [[] for _ in range(slots)]
        self.len, self.refs = [0] * slots, [0] * pages
        self.page, self.max = page, max_pages

    def reserve(self, slots, counts):
        free = [p for p, r in enumerate(self.refs) if r == 0]
        plan, refs = [], list(self.refs)
        for s, n in zip(slots, counts):
            if n < 0 or self.len[s] + n > self.max * self.page:
                return "ARG", []
            need = -(-(self.len[s] + n) // self.page) - len(self.table[s])
            cow = n > 0 and self.len[s] % self.page > 0 and refs[self.table[s][-1]] > 1
            if cow:
                refs[self.table[s][-1]] -= 1
            plan.append((s, n, need, cow))
        if sum(p[2] + p[3] for p in plan) > len(free):
            return "PAGES", []
        copies = []
        for s, n, need, cow in plan:
            if cow:
                src, dst = self.table[s][-1], free.pop(0)
                copies.append((src, dst))
                self.table[s][-1] = dst
                self.refs[src] -= 1
                self.refs[dst] = 1
            for _ in range(need):
                p = free.pop(0)
                self.refs[p] = 1
                self.table[s].append(p)
            self.len[s] += n
        return "OK", copies

    def fork(self, parents, children):
        if len(set(children)) < len(children) or set(children) & set(parents) or any(self.len[c] for c in children):
            return "ARG"
        for p, c in zip(parents, children):
            self.table[c] = list(self.table[p])
            self.len[c] = self.len[p]
            for x in self.table[p]:
                self.refs[x] += 1
        return "OK"

    def truncate(self, slots, lens):
        if len(set(slots)) < len(slots) or min(lens) < 0:
            return "ARG"
        for s, n in zip(slots, lens):
            n = min(n, self.len[s])
            while len(self.table[s]) > -(-n // self.page):
                self.refs[self.table[s].pop()] -= 1
            self.len[s] = n
        return "OK"

    def compact(self):
        live = [p for p, r in enumerate(self.refs) if r > 0]
        holes = [p for p in range(len(live)) if self.refs[p] == 0]
        move = dict(zip([p for p in live if p >= len(live)], holes))
        for a, b in move.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.table = [[move.get(p, p) for p in t] for t in self.table]
        return list(move.items())

    def same(self, c):
        table = torch.full((len(self.table), self.max), -1, dtype=torch.int32)
        for i, t in enumerate(self.table):
            table[i, :len(t)] = torch.tensor(t, dtype=torch.int32)
        assert torch.equal(c.table.cpu(), table)
        assert c.lens.tolist() == self.len and c.refs.tolist() == self.refs


def expect(tq_lib, c, what):
    if what == "OK":
        c.status()
    else:
        with pytest.raises(tq_lib.TQError) as e:
            c.status()
        assert e.value.status == getattr(tq_lib.binding, "TQ_ERR_" + what)


@pytest.mark.parametrize("seed,page,pages,slots", [(0, 16, 30, 12), (1, 64, 200, 40), (2, 32, 5000, 300),
                                                   (3, 128, 9, 7)])
def test_pages_random_walk(tq_lib, cuda, seed, page, pages, slots):
    """Random steps against the plain rules, errors among them: tables, counts,
    lengths, statuses and the pages' contents."""
    import random
    r = random.Random(seed)
    c = make_cache(tq_lib, cuda, "i8", layers=2, heads=1, d=64, page=page, slots=slots, max_pages=6,
                   pages=pages)
    c.kscale.uniform_()
    c.vscale.uniform_()
    m = Model(slots, 6, pages, page)
    pools = [t.clone() for t in (c.k, c.v, c.kscale, c.vscale)]
    seen = set()
    for step in range(60):
        kind = r.choice(["reserve", "reserve", "fork", "truncate", "compact"])
        n = r.randint(1, slots)
        pick = r.sample(range(slots), n)
        moves, what = [], "OK"
        if kind == "reserve":
            counts = [r.choice([0, 1, 1, page, r.randint(0, 2 * page)]) for _ in pick]
            if r.random() < 0.1:
                counts[0] = r.choice([-1, 6 * page + 1])
            what, moves = m.reserve(pick, counts)
            c.reserve(ints(pick, cuda), ints(counts, cuda))
        elif kind == "fork":
            empty = [s for s in range(slots) if m.len[s] == 0]
            full = [s for s in range(slots) if m.len[s] > 0]
            if not empty or not full:
                continue
            kids = r.sample(empty, r.randint(1, len(empty)))
            if r.random() < 0.15:
                kids[0] = r.choice(full + kids[-1:])
            parents = [r.choice(full) for _ in kids]
            what = m.fork(parents, kids)
            c.fork(ints(parents, cuda), ints(kids, cuda))
        elif kind == "truncate":
            lens = [r.choice([0, 0, r.randint(0, 6 * page)]) for _ in pick]
            if r.random() < 0.1:
                lens[-1] = -1
            if r.random() < 0.1 and n > 1:
                pick[0] = pick[1]
            what = m.truncate(pick, lens)
            c.truncate(ints(pick, cuda), ints(lens, cuda))
        else:
            moves = m.compact()
            c.compact()
        seen.add((kind, what))
        expect(tq_lib, c, what)
        m.same(c)
        for t in pools:
            old = t.clone()
            for a, b in moves:
                t[:, b] = old[:, a]
        for t, now in zip(pools, (c.k, c.v, c.kscale, c.vscale)):
            assert torch.equal(t, now), (step, kind)
    assert ("reserve", "OK") in seen and ("compact", "OK") in seen


def test_pages_device_refusals(tq_lib, cuda):
    c = make_cache(tq_lib, cuda, page=16, slots=4, max_pages=4, pages=6)
    c.reserve(ints([0, 1], cuda), ints([20, 16], cuda))
    c.status()
    state = [t.clone() for t in (c.table, c.lens, c.refs, c.k, c.v)]

    def refused(call, what, *lists):
        call(*(ints(x, cuda) for x in lists))
        expect(tq_lib, c, what)
        assert all(torch.equal(a, b) for a, b in zip(state, (c.table, c.lens, c.refs, c.k, c.v)))
    refused(c.reserve, "ARG", [0, 0], [1, 1])        # a slot twice
    refused(c.reserve, "ARG", [4, 2], [1, 1])        # out of range
    refused(c.reserve, "ARG", [-1, 2], [1, 1])
    refused(c.reserve, "ARG", [2, 0], [1, -1])       # a negative count
    refused(c.reserve, "ARG", [2, 0], [1, 45])       # beyond the table
    refused(c.reserve, "ARG", [0], [2 ** 31 - 1])
    refused(c.reserve, "PAGES", [2, 3], [33, 16])    # 3 + 1 of 3
    refused(c.fork, "ARG", [0], [1])                 # the child holds pages
    refused(c.fork, "ARG", [0, 1], [2, 2])           # a child twice
    refused(c.fork, "ARG", [0, 2], [2, 3])           # a child that is a parent
    refused(c.fork, "ARG", [0], [0])
    refused(c.fork, "ARG", [9], [2])
    refused(c.fork, "ARG", [0], [-2])
    refused(c.truncate, "ARG", [0, 0], [1, 1])
    refused(c.truncate, "ARG", [0, 5], [1, 1])
    refused(c.truncate, "ARG", [0, 1], [1, -1])
    c.reserve(ints([2, 3], cuda), ints([32, 16], cuda))  # and after them it goes on
    c.status()
    assert (c.refs == 1).all()


@pytest.mark.parametrize("n", [255, 256, 257, 1025, 3000])
def test_pages_list_lengths(tq_lib, cuda, n):
    """Lists around the lengths at which the checks change their way: the plain
    rules, copies on write of one page by many, and a repeated slot at either end."""
    c = make_cache(tq_lib, cuda, "i8", layers=1, heads=1, d=64, page=16, slots=n + 2, max_pages=3,
                   pages=2 * n + 8)
    m = Model(n + 2, 3, 2 * n + 8, 16)

    def both(kind, a, b, what="OK"):
        got = getattr(m, kind)(a, b) if what == "OK" else what
        assert (got[0] if isinstance(got, tuple) else got) == what
        getattr(c, kind)(ints(a, cuda), ints(b, cuda))
        expect(tq_lib, c, what)
        m.same(c)
    both("reserve", [n, n + 1], [20, 7])
    kids = list(range(n))
    both("fork", [n if i % 3 else n + 1 for i in kids], kids)
    both("reserve", kids[::-1], [i % 5 for i in kids])
    for bad in (kids[:-1] + [0], [kids[-1]] + kids[1:]):
        both("truncate", bad, [0] * n, "ARG")
        both("reserve", bad, [1] * n, "ARG")
    both("truncate", kids, [0] * n)
    both("fork", [n] * (n - 1) + [0], kids, "ARG")   # a parent among the children
    both("fork", [n] * n, kids[:-1] + [0], "ARG")
    both("fork", [n] * n, kids)


# ------------------------------------------------------------------ together

def test_engine_steps(tq_lib, cuda):
    """Prompts, sampling from a fork, single tokens, drafts given up, compaction:
    every layer's attention against the cache's contents in 64 bits, and the
    contents against the tokens."""
    torch.manual_seed(0)
    L, H, G, d, page = 2, 2, 4, 128, 16
    c = make_cache(tq_lib, cuda, "i8", layers=L, heads=H, d=d, page=page, slots=6, max_pages=12, pages=60)
    rope = tq_lib.Rope(d, base=1e4)
    kept = {s: [[] for _ in range(L)] for s in range(6)}

    def step(slots, counts):
        T = sum(counts)
        start = [int(c.lens[s]) for s in slots]
        ds, cu = ints(slots, cuda), cu_of(counts, cuda)
        c.reserve(ds, ints(counts, cuda))
        c.status()
        pos = torch.cat([torch.arange(a, a + n) for a, n in zip(start, counts)]).to(cuda)
        for layer in range(L):
            q, k, v = (torch.randn(T, h, d, device=cuda).to(torch.bfloat16) for h in (H * G, H, H))
            c.append(layer, k, v, cu, max(counts), slots=ds, rope=rope)
            q = rope.apply(q, pos)
            at = 0
            for s, a, n in zip(slots, start, counts):
                kk = rope_ref(k[at:at + n].cpu(), range(a, a + n), rope, False)
                kept[s][layer] = kept[s][layer][:a] + [(kk[t], v[at + t].cpu().double()) for t in range(n)]
                at += n
            check_attention(c, q, counts, [int(c.lens[s]) for s in slots], slots=ds, layer=layer)

    def contents():
        for s in range(6):
            n = int(c.lens[s])
            for layer in range(L if n else 0):
                for name, which in (("k", 0), ("v", 1)):
                    rows = torch.stack([x[which] for x in kept[s][layer][:n]], 1)
                    got = values(c, name, layer, s, n)
                    ids = c.table[s, torch.arange(n, device=cuda) // page].long()
                    per = getattr(c, name + "scale")[layer][ids].cpu().double().T[..., None]
                    # half a step for the first rounding and each growth of the scale
                    # behind it; 16 tokens grow it 15 times at most
                    assert ((got - rows).abs() <= per * 8.5).all()
                    assert ((got - rows).abs().mean() <= 0.6 * per.mean())

    step([0, 1, 2], [50, 16, 33])
    c.fork(ints([0, 0, 1], cuda), ints([3, 4, 5], cuda))
    for a, b in ((0, 3), (0, 4), (1, 5)):
        kept[b] = [list(x) for x in kept[a]]
    step([0, 1, 2, 3, 4, 5], [1] * 6)
    step([4, 0, 5], [5, 5, 3])             # drafts ...
    c.truncate(ints([4, 0], cuda), ints([53, 52], cuda))  # ... of which some are given up
    step([0, 1, 2, 3, 4, 5], [1] * 6)
    c.truncate(ints([1, 3], cuda), ints([0, 0], cuda))
    c.compact()
    c.status()
    assert int((c.refs > 0).sum()) == int(c.refs.nonzero().max()) + 1
    step([5, 4, 2, 0], [1, 20, 1, 2])
    contents()


def test_calls_in_a_graph_and_on_other_streams(tq_lib, cuda):
    """A decode step captured and replayed with new inputs gives what the eager
    calls give; two graphs of one cache keep workspaces of their own."""
    lens = [300, 45, 64]

    def fresh():
        return fill(tq_lib, cuda, "i8", 2, 128, 64, lens)
    a, b = fresh(), fresh()
    for c in (a, b):  # room for the tokens to come
        c.refs[c.refs.numel() - 3:] = 0
        used = set(c.table[c.table >= 0].tolist())
        for p in range(c.pages):
            c.refs[p] = int(p in used)
    slots, ones, cu = ints([0, 1, 2], cuda), ints([1, 1, 1], cuda), cu_of([1, 1, 1], cuda)
    k, v = (torch.zeros(3, 2, 128, dtype=torch.bfloat16, device=cuda) for _ in "kv")
    q, pos = torch.zeros(3, 8, 128, dtype=torch.bfloat16, device=cuda), torch.zeros(3, dtype=torch.int64, device=cuda)
    rope = tq_lib.Rope(128)

    def step(c):
        c.reserve(slots, ones)
        c.append(0, k, v, cu, 1, slots=slots, rope=rope)
        return c.attention(0, rope.apply(q, pos), cu, 1, slots=slots)
    warm = fresh()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(warm)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(a)
        graphs.append((g, out))
    for i in range(6):
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, generator=gen(i)))
        pos.copy_(a.lens)
        g, out = graphs[i % 2]
        g.replay()
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            want = step(b)
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        assert torch.equal(a.lens, b.lens) and torch.equal(a.table, b.table)
        ids = a.table[a.table >= 0].long()
        assert torch.equal(a.kscale[0, ids], b.kscale[0, ids])


@pytest.mark.parametrize("counts", [[1, 1, 1], [3, 1, 2], [200, 1, 64]])
def test_attention_replayed_and_side_by_side(tq_lib, cuda, counts):
    """Items joined across blocks: a captured call replayed over changing queries,
    on a side stream while eager calls run on others, gives what a call alone gives."""
    lens = [30000, 5000, 700]
    c = fill(tq_lib, cuda, "i8", 2, 128, 64, lens)
    total = sum(counts)
    cu, q = cu_of(counts, cuda), torch.zeros(total, 8, 128, dtype=torch.bfloat16, device=cuda)
    qs = [torch.randn(total, 8, 128, generator=gen(i)).to(torch.bfloat16).to(cuda) for i in range(4)]
    want = [c.attention(0, x, cu, max(counts)) for x in qs]
    c.status()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = c.attention(0, q, cu, max(counts))
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for i in range(12):
        got = []
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                if k == 0:
                    q.copy_(qs[i % 4])
                    g.replay()
                else:
                    got.append(((i + k) % 4, c.attention(0, qs[(i + k) % 4], cu, max(counts))))
        torch.cuda.synchronize()
        assert torch.equal(out, want[i % 4]), i
        assert all(torch.equal(x, want[j]) for j, x in got), i
    c.status()
