"""Torch-facing wrapper of the 8-bit paged KV cache and the rotary positions:
owns the device tensors and forwards every call to libtq on the current stream
of the tensors' device.  Lists of slots, counts and cumulative lengths are int32
device tensors; nothing here waits for the device."""
import contextlib

import torch

from . import _binding as B
from .quantizer import Workspace

_DTYPES = {torch.float32: B.TQ_F32, torch.bfloat16: B.TQ_BF16, torch.float16: B.TQ_F16}
_FORMATS = {torch.int8: B.TQ_KV_I8, torch.float8_e4m3fn: B.TQ_KV_E4M3}
_LAYOUTS = {"half": B.TQ_ROPE_HALF, "interleaved": B.TQ_ROPE_INTERLEAVED}
_SCALINGS = {"none": B.TQ_ROPE_PLAIN, "linear": B.TQ_ROPE_LINEAR, "ntk": B.TQ_ROPE_NTK,
             "parts": B.TQ_ROPE_PARTS}
_SAME = contextlib.nullcontext()


def _on(device):
    """The device as the current one (the streams are its own)."""
    if device.type != "cuda":
        raise ValueError(f"expected a CUDA tensor, got one on {device}")
    if device.index is None or device.index == torch.cuda.current_device():
        return _SAME
    return torch.cuda.device(device)


def _stream(device):
    return torch.cuda.current_stream(device).cuda_stream


def _ints(t, name, n, device, dtype=torch.int32):
    """A contiguous [n] index tensor's address."""
    if t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or t.device != device:
        raise ValueError(f"{name}: expected [{n}] {dtype} on {device}, got {tuple(t.shape)} "
                         f"{t.dtype} on {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t.data_ptr()


def _rows(x, heads, d, name):
    """x [T, heads, d] with contiguous heads: itself, or a copy."""
    if x.dim() != 3 or (heads is not None and x.shape[1] != heads) or x.shape[2] != d:
        raise ValueError(f"{name}: expected [T, {'heads' if heads is None else heads}, {d}], got "
                         f"{tuple(x.shape)}")
    if x.dtype not in _DTYPES:
        raise TypeError(f"{name}: unsupported dtype {x.dtype}; expected float32, bfloat16 or "
                        f"float16")
    return x if x.stride(2) == 1 else x.contiguous()


class _RopeFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, pos, rope):
        ctx.rope = rope
        ctx.save_for_backward(pos)
        return rope.apply(x, pos)

    @staticmethod
    def backward(ctx, g):
        return ctx.rope.apply(g, ctx.saved_tensors[0], transpose=True), None, None


class Rope:
    """Rotary positions of the first `rot` coordinates of a head of d (all by
    default): layout "half" pairs i with i + rot/2, "interleaved" 2i with 2i + 1.
    scaling: "none", "linear" (factor), "ntk" (factor) or "parts" (factor, ctx,
    low, high); amplitude multiplies the rotated coordinates (include/tq.h)."""

    def __init__(self, d, rot=None, base=10000.0, layout="half", scaling="none", factor=1.0,
                 ctx=1.0, low=0.0, high=1.0, amplitude=1.0):
        if layout not in _LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}, got {layout!r}")
        if scaling not in _SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}, got {scaling!r}")
        self.d, self.rot = int(d), int(d if rot is None else rot)
        self.params = B.tq_rope_params_t()
        B.tq_build_rope(self.d, self.rot, float(base), _LAYOUTS[layout], _SCALINGS[scaling],
                        float(factor), float(ctx), float(low), float(high), float(amplitude),
                        self.params)

    def apply(self, x, pos, out=None, transpose=False):
        """x [T, heads, d] turned to positions pos [T] int64 (transpose: by the
        transposed matrix, the gradient).  out may be x (contiguous heads)."""
        x = _rows(x, None, self.d, "x")
        T, heads = x.shape[0], x.shape[1]
        dev = x.device
        if out is None:
            out = torch.empty((T, heads, self.d), dtype=x.dtype, device=dev)
        elif out.shape != x.shape or out.dtype != x.dtype or out.device != dev or out.stride(2) != 1:
            raise ValueError("out: expected x's shape, type and device, contiguous heads")
        with _on(dev):
            B.tq_rope(self.params, T, heads, x.data_ptr(), x.stride(0), x.stride(1),
                      _DTYPES[x.dtype], _ints(pos, "pos", T, dev, torch.int64), out.data_ptr(),
                      out.stride(0), out.stride(1), int(transpose), _stream(dev))
        return out

    def __call__(self, x, pos):
        """apply(x, pos) with a gradient."""
        return _RopeFn.apply(x, pos, self)


class KV8Cache:
    """A paged KV cache in 8 bits over an engine's own tensors:

    k, v            [layers, pages, heads, page, d] int8 or float8_e4m3fn codes
    kscale, vscale  [layers, pages, heads] float32
    table           [slots, max_pages] int32 page ids (-1: none)
    lens, refs      [slots], [pages] int32

    KV8Cache.empty(...) allocates them.  A step of an engine: reserve (room for
    the new tokens, lengths move on), then layer by layer append and attention.
    Page calls check on the device; status() waits and raises what the last one
    found."""

    def __init__(self, k, v, kscale, vscale, table, lens, refs):
        if k.dim() != 5 or k.dtype not in _FORMATS:
            raise ValueError("k: expected [layers, pages, heads, page, d] int8 or float8_e4m3fn")
        layers, pages, heads, page, d = k.shape
        want = {"v": (v, k.shape, k.dtype), "kscale": (kscale, k.shape[:3], torch.float32),
                "vscale": (vscale, k.shape[:3], torch.float32),
                "table": (table, (lens.shape[0], table.shape[-1]), torch.int32),
                "lens": (lens, (lens.shape[0],), torch.int32), "refs": (refs, (pages,), torch.int32)}
        for name, (t, shape, dtype) in {"k": (k, k.shape, k.dtype), **want}.items():
            if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != k.device:
                raise ValueError(f"{name}: expected {tuple(shape)} {dtype} on {k.device}, got "
                                 f"{tuple(t.shape)} {t.dtype} on {t.device}")
            if not t.is_contiguous():
                raise ValueError(f"{name}: expected a contiguous tensor")
        self.k, self.v, self.kscale, self.vscale = k, v, kscale, vscale
        self.table, self.lens, self.refs = table, lens, refs
        self.layers, self.pages, self.heads, self.page, self.d = layers, pages, heads, page, d
        self.slots, self.device = lens.shape[0], k.device
        self.c = B.tq_kv8_t(d, heads, page, _FORMATS[k.dtype], layers, self.slots, table.shape[1],
                            pages, k.data_ptr(), v.data_ptr(), kscale.data_ptr(),
                            vscale.data_ptr(), table.data_ptr(), lens.data_ptr(), refs.data_ptr())
        if B.tq_kv8_workspace_bytes(B.TQ_KV8_OP_PAGES, self.c, 0, 0, 0, 0) == (1 << 64) - 1:
            raise B.TQError("tq_kv8_workspace_bytes", B.TQ_ERR_UNSUPPORTED)
        self._ws = {}  # per stream: calls of one stream follow one another
        self._ws_need = {}
        self._last = None

    @classmethod
    def empty(cls, layers, pages, heads, d, slots, max_pages, page=64, dtype=torch.int8,
              device="cuda"):
        """An empty cache: all pages free, all slots of length 0."""
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        codes = (layers, pages, heads, page, d)

        def new(shape, dtype, fill):
            return torch.full(shape, fill, dtype=dtype, device=dev)
        return cls(torch.empty(codes, dtype=dtype, device=dev),
                   torch.empty(codes, dtype=dtype, device=dev),
                   new(codes[:3], torch.float32, 0.0), new(codes[:3], torch.float32, 0.0),
                   new((slots, max_pages), torch.int32, -1), new((slots,), torch.int32, 0),
                   new((pages,), torch.int32, 0))

    def _workspace(self, *key):
        """(address, bytes, stream) for a call on the current stream."""
        stream = _stream(self.device)
        need = self._ws_need.get(key)
        if need is None:
            op, n, total, max_q, heads_q = key
            need = B.tq_kv8_workspace_bytes(op, self.c, n, total, max_q, heads_q)
            if len(self._ws_need) > 4096:
                self._ws_need.clear()
            self._ws_need[key] = need
        if torch.cuda.is_current_stream_capturing():
            # the graph's own memory: graphs that run side by side share nothing
            self._last = ws = torch.empty(max(need, 256), dtype=torch.uint8, device=self.device)
            return ws.data_ptr(), need, stream
        ws = self._ws.get(stream)
        if ws is None:
            ws = self._ws[stream] = Workspace(self.device)
        ptr, size = ws.get(need)
        self._last = ws.buf
        return ptr, size, stream

    # ---- pages

    def _list(self, fn, a, b, names):
        n = a.shape[0]
        pa, pb = (_ints(t, name, n, self.device) for t, name in zip((a, b), names))
        with _on(self.device):
            fn(self.c, n, pa, pb, *self._workspace(B.TQ_KV8_OP_PAGES, n, 0, 0, 0))

    def reserve(self, slots, counts):
        """Room for counts[i] more tokens in slots[i]; lens move on."""
        self._list(B.tq_kv8_reserve, slots, counts, ("slots", "counts"))

    def fork(self, parents, children):
        """children[i] (empty) becomes a copy of parents[i], sharing its pages."""
        self._list(B.tq_kv8_fork, parents, children, ("parents", "children"))

    def truncate(self, slots, lens):
        """slots[i] keeps its first lens[i] tokens; 0 frees the slot."""
        self._list(B.tq_kv8_truncate, slots, lens, ("slots", "lens"))

    def compact(self):
        """Live pages move to the front of the pool."""
        with _on(self.device):
            B.tq_kv8_compact(self.c, *self._workspace(B.TQ_KV8_OP_PAGES, 0, 0, 0, 0))

    def status(self):
        """Waits for the stream and raises what the last page or attention call
        found on the device."""
        if self._last is None:
            return
        with _on(self.device):
            rc = B.tq_device_status(self._last.data_ptr(), _stream(self.device))
        if rc != B.TQ_OK:
            raise B.TQError("tq_device_status", rc)

    # ---- tokens

    def _batch(self, slots, cu):
        ns = cu.shape[0] - 1
        return (ns, None if slots is None else _ints(slots, "slots", ns, self.device),
                _ints(cu, "cu", ns + 1, self.device))

    def append(self, layer, k, v, cu, max_new, slots=None, rope=None):
        """Writes k, v [total, heads, d] as the last cu[i+1] - cu[i] (at most
        max_new) tokens of every slot; rope turns the keys to their positions."""
        k, v = _rows(k, self.heads, self.d, "k"), _rows(v, self.heads, self.d, "v")
        if v.dtype != k.dtype or v.shape != k.shape or k.device != self.device or v.device != self.device:
            raise ValueError("k, v: expected one shape and type, on the cache's device")
        if v.stride() != k.stride():
            k, v = k.contiguous(), v.contiguous()
        ns, ps, pc = self._batch(slots, cu)
        with _on(self.device):
            B.tq_kv8_append(self.c, layer, ns, ps, pc, k.shape[0], max_new, k.data_ptr(),
                            v.data_ptr(), _DTYPES[k.dtype], k.stride(0), k.stride(1),
                            None if rope is None else rope.params, _stream(self.device))

    def read(self, layer, begin, cu, total, max_count, slots=None, dtype=torch.bfloat16):
        """(k, v) [total, heads, d] of tokens begin[i] .. begin[i] + cu[i+1] - cu[i]."""
        ns, ps, pc = self._batch(slots, cu)
        shape = (total, self.heads, self.d)
        k = torch.empty(shape, dtype=dtype, device=self.device)
        v = torch.empty(shape, dtype=dtype, device=self.device)
        with _on(self.device):
            B.tq_kv8_read(self.c, layer, ns, ps, _ints(begin, "begin", ns, self.device), pc, total,
                          max_count, k.data_ptr(), v.data_ptr(), _DTYPES[dtype],
                          _stream(self.device))
        return k, v

    def attention(self, layer, q, cu, max_q, slots=None, scale=None, causal=True, window=0,
                  out=None, lse=None):
        """Attention of q [total, heads_q, d] (bfloat16 or float16), the last
        cu[i+1] - cu[i] (at most max_q) tokens of every slot, over the slot's
        tokens: [total, heads_q, d].  scale defaults to 1/sqrt(d); window > 0: a
        token sees the last `window` keys, itself included; lse: [total, heads_q]
        float32, filled where given."""
        q = _rows(q, None, self.d, "q")
        if q.device != self.device:
            raise ValueError(f"q: expected a tensor on {self.device}")
        if q.data_ptr() % 16 or q.stride(0) % 8 or q.stride(1) % 8:
            q = q.contiguous() if not q.is_contiguous() else q.clone()
        total, heads_q = q.shape[0], q.shape[1]
        if out is None:
            out = torch.empty((total, heads_q, self.d), dtype=q.dtype, device=self.device)
        elif (out.shape != q.shape or out.dtype != q.dtype or out.device != self.device or
              not out.is_contiguous()):
            raise ValueError("out: expected q's shape, type and device, contiguous")
        if lse is not None and (lse.shape != q.shape[:2] or lse.dtype != torch.float32 or
                                lse.device != self.device or not lse.is_contiguous()):
            raise ValueError("lse: expected [total, heads_q] float32, contiguous")
        ns, ps, pc = self._batch(slots, cu)
        with _on(self.device):
            B.tq_kv8_attention(self.c, layer, ns, ps, pc, total, max_q, heads_q, q.data_ptr(),
                               _DTYPES[q.dtype], q.stride(0), q.stride(1),
                               self.d ** -0.5 if scale is None else float(scale), int(causal),
                               window, out.data_ptr(), None if lse is None else lse.data_ptr(),
                               *self._workspace(B.TQ_KV8_OP_ATTENTION, ns, total, max_q, heads_q))
        return out
