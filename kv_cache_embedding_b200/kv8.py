"""Torch-facing wrapper of the 8-bit paged KV cache and the rotary positions:
owns the device tensors and forwards every call to libtq on the current stream
of the tensors' device (the checks, outputs and workspaces are the native
module's, _kv8).  Lists of slots, counts and cumulative lengths are int32 device
tensors; nothing here waits for the device but KV8Cache.status()."""
import ctypes

import torch

from . import _binding as B

N = None  # the native module


def _native():
    """Loads _kv8.so, built beside libtq.so for one version of torch; the rest of
    the package does without it."""
    global N
    if N is None:
        hint = "run `python kv_cache_embedding_b200/build.py`"
        try:
            from . import _kv8 as module
        except ImportError as e:
            raise ImportError(f"_kv8.so does not load ({e}); {hint}") from e
        if module.built_for != f"built for torch {torch.__version__}":
            raise ImportError(f"_kv8.so is {module.built_for}, this is {torch.__version__}; {hint}")
        module.init(B.TQError)
        N = module
    return N


_FORMATS = {torch.int8: B.TQ_KV_I8, torch.float8_e4m3fn: B.TQ_KV_E4M3}
_LAYOUTS = {"half": B.TQ_ROPE_HALF, "interleaved": B.TQ_ROPE_INTERLEAVED}
_SCALINGS = {"none": B.TQ_ROPE_PLAIN, "linear": B.TQ_ROPE_LINEAR, "ntk": B.TQ_ROPE_NTK,
             "parts": B.TQ_ROPE_PARTS}


_words = {}  # device: words that no cache has had yet


def _status_word(device):
    """A zero on the device that every stream can use at once: a kernel that writes it
    would be waited for on one stream alone.  Copies from pageable memory are complete
    when they return; one in 256 caches pays for it."""
    if device.type != "cuda" or torch.cuda.is_current_stream_capturing():
        return torch.zeros(1, dtype=torch.int32, device=device)
    words = _words.setdefault(device, [])
    while True:
        try:
            return words.pop()
        except IndexError:
            words.extend(torch.zeros(256, dtype=torch.int32).to(device).split(1))


class _RopeFn(torch.autograd.Function):
    """A linear map: its gradient is the transposed one, again with a gradient."""

    @staticmethod
    def forward(ctx, x, pos, rope, transpose):
        ctx.rope, ctx.transpose = rope, transpose
        ctx.save_for_backward(pos)
        return rope.apply(x, pos, transpose=transpose)

    @staticmethod
    def backward(ctx, g):
        return _RopeFn.apply(g, ctx.saved_tensors[0], ctx.rope, not ctx.transpose), None, None, None


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
        self._h = _native().rope_params(ctypes.addressof(self.params))

    def apply(self, x, pos, out=None, transpose=False):
        """x [T, heads, d] turned to positions pos [T] int64 (transpose: by the
        transposed matrix), with a gradient.  Into out, which may be x (contiguous
        heads), without one: tensors that require it are refused."""
        y = N.rope(self._h, x, pos, out, transpose)
        return _RopeFn.apply(x, pos, self, bool(transpose)) if y is None else y

    def __call__(self, x, pos):
        return self.apply(x, pos)


class KV8Cache:
    """A paged KV cache in 8 bits over an engine's own tensors:

    k, v            [layers, pages, heads, page, d] int8 or float8_e4m3fn codes
    kscale, vscale  [layers, pages, heads] float32
    table           [slots, max_pages] int32 page ids (-1: none)
    lens, refs      [slots], [pages] int32

    KV8Cache.empty(...) allocates them.  A step of an engine: reserve (room for
    the new tokens, lengths move on), then layer by layer append and attention.
    The calls check on the device.  From the first one that is refused there (or
    times out) until status() has raised it, further calls leave the cache as it
    is: the step's append writes nothing, its attention gives zeros.  Where a
    reserve was refused the step can simply be repeated; lengths are as they were
    before it."""

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
        self._status = _status_word(k.device)
        self.c = B.tq_kv8_t(d, heads, page, _FORMATS[k.dtype], layers, self.slots, table.shape[1],
                            pages, k.data_ptr(), v.data_ptr(), kscale.data_ptr(),
                            vscale.data_ptr(), table.data_ptr(), lens.data_ptr(), refs.data_ptr(),
                            self._status.data_ptr())
        # the workspaces live there, one a stream
        self._h = _native().cache(ctypes.addressof(self.c), self._status)

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

    # ---- pages

    def reserve(self, slots, counts):
        """Room for counts[i] more tokens in slots[i]; lens move on."""
        N.pages(self._h, 0, slots, counts)

    def fork(self, parents, children):
        """children[i] (empty) becomes a copy of parents[i], sharing its pages."""
        N.pages(self._h, 1, parents, children)

    def truncate(self, slots, lens):
        """slots[i] keeps its first lens[i] tokens; 0 frees the slot."""
        N.pages(self._h, 2, slots, lens)

    def compact(self):
        """Live pages move to the front of the pool."""
        N.compact(self._h)

    def status(self):
        """Waits for the device (calls on every stream and replayed graphs) and raises
        the first refusal or time-out since the last status(); after that the cache
        can be used again.  Not during a capture."""
        N.status(self._h)

    # ---- tokens

    def append(self, layer, k, v, cu, max_new, slots=None, rope=None):
        """Writes k, v [total, heads, d] as the last cu[i+1] - cu[i] (at most
        max_new) tokens of every slot; rope turns the keys to their positions.  No
        gradient: tensors that require one are refused (attention's too)."""
        N.append(self._h, layer, k, v, cu, max_new, slots, None if rope is None else rope._h)

    def read(self, layer, begin, cu, total, max_count, slots=None, dtype=torch.bfloat16):
        """(k, v) [total, heads, d] of tokens begin[i] .. begin[i] + cu[i+1] - cu[i]
        (max_count: as many at most, a hint); 0 where there is no such token, and
        behind cu[-1]."""
        return N.read(self._h, layer, begin, cu, total, max_count, slots, dtype)

    def attention(self, layer, q, cu, max_q, slots=None, scale=None, causal=True, window=0,
                  out=None, lse=None):
        """Attention of q [total, heads_q, d] (bfloat16 or float16), the last
        cu[i+1] - cu[i] (at most max_q) tokens of every slot, over the slot's
        tokens: [total, heads_q, d].  Rows of q behind cu[-1] are 0 in the result, or
        stay as they were in an `out` (contiguous, q's own memory or none of it) that is
        given.  scale defaults to 1/sqrt(d); window > 0: a
        token sees the last `window` keys, itself included; lse: [total, heads_q]
        float32, filled where given."""
        return N.attention(self._h, layer, q, cu, max_q, slots, scale, causal, window, out, lse)
