"""The 8-bit cache and the rotary positions without a GPU: every refusal comes
before any device work, and the host-side tables are right."""
import ctypes as C
import math

import pytest

BIG = (1 << 64) - 1


def _cache(B, **kw):
    c = dict(d=128, heads=2, page=64, format=B.TQ_KV_I8, layers=1, slots=4, max_pages=8, pages=16,
             d_k=256, d_v=256, d_kscale=256, d_vscale=256, d_table=256, d_len=256, d_refs=256)
    c.update(kw)
    return B.tq_kv8_t(**c)


@pytest.mark.parametrize("kw,status", [
    (dict(d=96), "UNSUPPORTED"), (dict(page=48), "UNSUPPORTED"), (dict(page=256), "UNSUPPORTED"),
    (dict(format=2), "ARG"), (dict(heads=0), "ARG"), (dict(layers=0), "ARG"), (dict(slots=0), "ARG"),
    (dict(max_pages=0), "ARG"), (dict(pages=0), "ARG"), (dict(pages=1 << 26), "UNSUPPORTED"),
    (dict(max_pages=1 << 25), "UNSUPPORTED"), (dict(d_k=None), "ARG"), (dict(d_v=264), "ARG"),
    (dict(d_table=None), "ARG"), (dict(d_refs=None), "ARG"), (dict(d_vscale=None), "ARG")])
def test_cache_geometry(tq_lib, kw, status):
    B, L = tq_lib.binding, tq_lib.binding.lib
    c, want = C.byref(_cache(B, **kw)), getattr(B, "TQ_ERR_" + status)
    assert L.tq_kv8_workspace_bytes(B.TQ_KV8_OP_PAGES, c, 1, 0, 0, 0) == BIG
    assert L.tq_kv8_reserve(c, 1, 256, 256, 256, 1 << 30, None) == want
    assert L.tq_kv8_fork(c, 1, 256, 256, 256, 1 << 30, None) == want
    assert L.tq_kv8_truncate(c, 1, 256, 256, 256, 1 << 30, None) == want
    assert L.tq_kv8_compact(c, 256, 1 << 30, None) == want
    assert L.tq_kv8_append(c, 0, 1, None, 256, 1, 1, 256, 256, B.TQ_BF16, 256, 128, None, None) == want
    assert L.tq_kv8_read(c, 0, 1, None, 256, 256, 1, 1, 256, 256, B.TQ_BF16, None) == want
    assert L.tq_kv8_attention(c, 0, 1, None, 256, 1, 1, 4, 256, B.TQ_BF16, 512, 128, 0.1, 1, 0, 256,
                              None, 256, 1 << 30, None) == want


def test_page_calls(tq_lib):
    B, L = tq_lib.binding, tq_lib.binding.lib
    c = C.byref(_cache(B))
    for fn in (L.tq_kv8_reserve, L.tq_kv8_fork, L.tq_kv8_truncate):
        assert fn(c, -1, 256, 256, 256, 1 << 30, None) == B.TQ_ERR_ARG
        assert fn(c, 4097, 256, 256, 256, 1 << 30, None) == B.TQ_ERR_UNSUPPORTED
        assert fn(c, 2, None, 256, 256, 1 << 30, None) == B.TQ_ERR_ARG
        assert fn(c, 2, 256, None, 256, 1 << 30, None) == B.TQ_ERR_ARG
        assert fn(c, 2, 256, 256, None, 1 << 30, None) == B.TQ_ERR_WORKSPACE
        assert fn(c, 2, 256, 256, 256, 16, None) == B.TQ_ERR_WORKSPACE
        assert fn(c, 0, None, None, None, 0, None) == B.TQ_OK
    assert L.tq_kv8_compact(c, 256, 16, None) == B.TQ_ERR_WORKSPACE
    assert L.tq_kv8_compact(c, None, 1 << 30, None) == B.TQ_ERR_WORKSPACE
    assert L.tq_kv8_workspace_bytes(B.TQ_KV8_OP_PAGES, c, 4097, 0, 0, 0) == BIG
    assert L.tq_kv8_workspace_bytes(9, c, 1, 0, 0, 0) == BIG
    assert 0 < L.tq_kv8_workspace_bytes(B.TQ_KV8_OP_PAGES, c, 0, 0, 0, 0) < BIG


def test_token_calls(tq_lib):
    B, L = tq_lib.binding, tq_lib.binding.lib
    c = C.byref(_cache(B))

    def append(layer=0, ns=1, slots=None, cu=256, total=1, new=1, k=256, v=256, dt=B.TQ_BF16, r=None):
        return L.tq_kv8_append(c, layer, ns, slots, cu, total, new, k, v, dt, 256, 128, r, None)
    assert append(layer=1) == B.TQ_ERR_ARG and append(layer=-1) == B.TQ_ERR_ARG
    assert append(ns=-1) == B.TQ_ERR_ARG and append(total=-1) == B.TQ_ERR_ARG
    assert append(new=-1) == B.TQ_ERR_ARG and append(dt=3) == B.TQ_ERR_ARG
    assert append(ns=5) == B.TQ_ERR_ARG  # more entries than slots, without a list
    assert append(cu=None) == B.TQ_ERR_ARG and append(k=None) == B.TQ_ERR_ARG
    assert append(v=None) == B.TQ_ERR_ARG
    r = B.tq_rope_params_t()
    assert append(r=C.byref(r)) == B.TQ_ERR_ARG  # never built
    B.tq_build_rope(64, 64, 1e4, 0, 0, 1, 1, 0, 1, 1, r)
    assert append(r=C.byref(r)) == B.TQ_ERR_ARG  # another d
    for kw in (dict(ns=0), dict(total=0), dict(new=0)):
        assert append(**kw) == B.TQ_OK

    def read(layer=0, ns=1, begin=256, cu=256, total=1, new=1, k=256, dt=B.TQ_F32):
        return L.tq_kv8_read(c, layer, ns, None, begin, cu, total, new, k, 256, dt, None)
    assert read(layer=1) == B.TQ_ERR_ARG and read(dt=7) == B.TQ_ERR_ARG
    assert read(begin=None) == B.TQ_ERR_ARG and read(cu=None) == B.TQ_ERR_ARG
    assert read(k=264) == B.TQ_ERR_ARG and read(ns=5) == B.TQ_ERR_ARG
    assert read(ns=0) == B.TQ_OK and read(total=0) == B.TQ_OK

    def attn(layer=0, ns=1, cu=256, total=1, mq=1, hq=4, q=256, dt=B.TQ_BF16, ts=512, hs=128,
             scale=0.1, causal=1, window=0, out=256, ws=256, wn=1 << 30):
        return L.tq_kv8_attention(c, layer, ns, None, cu, total, mq, hq, q, dt, ts, hs, scale,
                                  causal, window, out, None, ws, wn, None)
    assert attn(layer=1) == B.TQ_ERR_ARG and attn(ns=5) == B.TQ_ERR_ARG
    assert attn(dt=B.TQ_F32) == B.TQ_ERR_ARG and attn(scale=float("nan")) == B.TQ_ERR_ARG
    assert attn(scale=float("inf")) == B.TQ_ERR_ARG and attn(causal=2) == B.TQ_ERR_ARG
    assert attn(window=-1) == B.TQ_ERR_ARG and attn(causal=0, window=4) == B.TQ_ERR_ARG
    assert attn(hq=3) == B.TQ_ERR_UNSUPPORTED and attn(hq=2 * 129) == B.TQ_ERR_UNSUPPORTED
    assert attn(hq=0) == B.TQ_ERR_ARG and attn(q=264) == B.TQ_ERR_ARG
    assert attn(ts=500) == B.TQ_ERR_ARG and attn(hs=100) == B.TQ_ERR_ARG
    assert attn(cu=None) == B.TQ_ERR_ARG and attn(out=None) == B.TQ_ERR_ARG
    assert attn(total=0) == B.TQ_OK and attn(mq=0) == B.TQ_OK and attn(ns=0) == B.TQ_OK
    n = L.tq_kv8_workspace_bytes(B.TQ_KV8_OP_ATTENTION, c, 1, 1, 1, 4)
    assert 0 < n < BIG
    assert L.tq_kv8_workspace_bytes(B.TQ_KV8_OP_ATTENTION, c, 1, 1, 1, 3) == BIG
    assert L.tq_kv8_workspace_bytes(B.TQ_KV8_OP_ATTENTION, c, 1, -1, 1, 4) == BIG


def test_attention_row_count(tq_lib):
    """Rows (tokens x group) count in 32 bits."""
    B, L = tq_lib.binding, tq_lib.binding.lib
    c = C.byref(_cache(B))
    for heads_q, total in ((2, 1 << 31), (256, 1 << 24), (8, 1 << 29)):
        assert L.tq_kv8_attention(c, 0, 1, None, 256, total, 1, heads_q, 256, B.TQ_BF16, 512, 128, 0.1, 1,
                                  0, 256, None, 256, 1 << 60, None) == B.TQ_ERR_UNSUPPORTED


def test_structs_match_the_header(tq_lib, tmp_path):
    import os
    import subprocess
    B = tq_lib.binding
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = "#include <stdio.h>\n#include <stddef.h>\n#include \"tq.h\"\nint main(void) {\n"
    for t in ("tq_kv8_t", "tq_rope_params_t"):
        src += f"  printf(\"%zu\\n\", sizeof({t}));\n"
        src += "".join(f"  printf(\"%zu\\n\", offsetof({t}, {f}));\n"
                       for f, _ in getattr(B, t)._fields_)
    (tmp_path / "l.c").write_text(src + "  return 0;\n}\n")
    subprocess.check_call(["gcc", "-I", os.path.join(root, "include"), str(tmp_path / "l.c"), "-o",
                           str(tmp_path / "l")])
    got = [int(v) for v in subprocess.check_output([str(tmp_path / "l")]).split()]
    want = []
    for t in (B.tq_kv8_t, B.tq_rope_params_t):
        want += [C.sizeof(t)] + [getattr(t, f).offset for f, _ in t._fields_]
    assert got == want


def test_rope_refusals(tq_lib):
    B, L = tq_lib.binding, tq_lib.binding.lib
    r = B.tq_rope_params_t()

    def build(d=128, rot=128, base=1e4, layout=0, scaling=0, factor=1.0, ctx=1.0, low=0.0, high=1.0,
              amp=1.0, p=C.byref(r)):
        return L.tq_build_rope(d, rot, base, layout, scaling, factor, ctx, low, high, amp, p)
    assert build(p=None) == B.TQ_ERR_ARG and build(layout=2) == B.TQ_ERR_ARG
    assert build(scaling=4) == B.TQ_ERR_ARG and build(base=1.0) == B.TQ_ERR_ARG
    assert build(base=float("nan")) == B.TQ_ERR_ARG and build(amp=float("inf")) == B.TQ_ERR_ARG
    assert build(d=127) == B.TQ_ERR_UNSUPPORTED and build(d=258) == B.TQ_ERR_UNSUPPORTED
    assert build(rot=130) == B.TQ_ERR_UNSUPPORTED and build(rot=3) == B.TQ_ERR_UNSUPPORTED
    assert build(scaling=1, factor=0.5) == B.TQ_ERR_ARG
    assert build(scaling=2, factor=2.0, rot=2) == B.TQ_ERR_UNSUPPORTED
    assert build(scaling=3, factor=2.0, ctx=0.0) == B.TQ_ERR_ARG
    assert build(scaling=3, factor=2.0, low=2.0, high=2.0) == B.TQ_ERR_ARG
    assert build() == B.TQ_OK

    def rope(T=1, heads=1, x=256, dt=B.TQ_F32, pos=256, out=512, ts=128, ots=128, tr=0, p=C.byref(r)):
        return L.tq_rope(p, T, heads, x, ts, 128, dt, pos, out, ots, 128, tr, None)
    assert rope(p=None) == B.TQ_ERR_ARG and rope(T=-1) == B.TQ_ERR_ARG
    assert rope(heads=0) == B.TQ_ERR_ARG and rope(dt=3) == B.TQ_ERR_ARG
    assert rope(tr=2) == B.TQ_ERR_ARG and rope(x=None) == B.TQ_ERR_ARG
    assert rope(pos=None) == B.TQ_ERR_ARG and rope(out=256, ots=256) == B.TQ_ERR_ARG
    assert rope(p=C.byref(B.tq_rope_params_t())) == B.TQ_ERR_ARG
    assert rope(heads=1 << 20) == B.TQ_ERR_UNSUPPORTED
    assert rope(T=0, x=None) == B.TQ_OK


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "parts"])
@pytest.mark.parametrize("d,rot,base", [(128, 128, 1e4), (64, 32, 5e5), (256, 256, 1e6), (8, 6, 3.0)])
def test_rope_frequencies(tq_lib, scaling, d, rot, base):
    """turns / 2^64 is f / 2 pi by the rule, to fp64's precision (the pow and the
    few products around it: 8 roundings of 2^-53) and half a unit of 2^-63."""
    r = tq_lib.Rope(d, rot, base=base, scaling=scaling, factor=4.0, ctx=4096, low=1.0, high=32.0)
    for i in range(rot // 2):
        b = base * 4.0 ** (rot / (rot - 2)) if scaling == "ntk" else base
        f = math.exp(-2 * i / rot * math.log(b))
        if scaling == "linear":
            f /= 4.0
        if scaling == "parts":
            g = min(1.0, max(0.0, (4096 * f / (2 * math.pi) - 1.0) / 31.0))
            f = f * g + f / 4.0 * (1 - g)
        # exp(x log b): an argument of up to 14 in fp64 adds 14 2^-53
        want = f / (2 * math.pi)
        assert abs(r.params.turns[i] / 2 ** 64 - want) <= 24 * 2 ** -53 * want + 2 ** -63


def test_wrapper_checks(tq_lib):
    import torch
    with pytest.raises(ValueError):
        tq_lib.Rope(128, layout="other")
    with pytest.raises(ValueError):
        tq_lib.Rope(128, scaling="other")
    with pytest.raises(tq_lib.TQError):
        tq_lib.Rope(128, rot=129)

    def parts(**kw):
        t = dict(k=torch.zeros(1, 4, 2, 16, 64, dtype=torch.int8),
                 v=torch.zeros(1, 4, 2, 16, 64, dtype=torch.int8),
                 kscale=torch.zeros(1, 4, 2), vscale=torch.zeros(1, 4, 2),
                 table=torch.zeros(3, 5, dtype=torch.int32), lens=torch.zeros(3, dtype=torch.int32),
                 refs=torch.zeros(4, dtype=torch.int32))
        t.update(kw)
        return t
    for bad in (dict(v=torch.zeros(1, 4, 2, 16, 64)), dict(kscale=torch.zeros(1, 4, 3)),
                dict(table=torch.zeros(2, 5, dtype=torch.int32)), dict(refs=torch.zeros(4)),
                dict(lens=torch.zeros(3, dtype=torch.int64)), dict(k=torch.zeros(4, 2, 16, 64)),
                dict(table=torch.zeros(5, 3, dtype=torch.int32).T)):
        with pytest.raises(ValueError):
            tq_lib.KV8Cache(**parts(**bad))
    with pytest.raises(tq_lib.TQError):  # a page of 24 tokens
        tq_lib.KV8Cache(**parts(k=torch.zeros(1, 4, 2, 24, 64, dtype=torch.int8),
                                v=torch.zeros(1, 4, 2, 24, 64, dtype=torch.int8)))
