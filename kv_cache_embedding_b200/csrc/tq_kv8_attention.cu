// Attention over the 8-bit paged cache, few query rows: for every row (query
// token, query head) of a slot,
//   l_j = scale s_k(j) <q, c_k(j)>,   out = sum_j softmax(l)_j s_v(j) c_v(j).
//
// Numerics.  Codes are exact halves; a query row times a power of two is a row
// of halves (row_unit), so <q, c> is a sum of exact products in fp32.  The
// block scales never touch the codes: s_k multiplies the logit, s_v the
// probability, which is rounded to a half relative to the running largest s_v
// (one rounding of 2^-11; the running maximum, sum and output are fp32).
//
// Work.  Reading the cache is the cost (2 d bytes a token and KV head for up to
// 16 rows), so every warp is a stream of its own: it takes an equal, contiguous
// share of all (entry, head, 32-key tile) steps of the batch --
// ragged lengths included -- and keeps kStages tiles of K and V in flight by TMA
// into its private ring; warps meet only where an item's steps are cut, and
// there k_attn_merge joins the parts in the order of their keys.  Products are
// m16n8k16 MMAs on half fragments made in registers from the codes (K: plain
// ldmatrix, coordinates permuted alike on both sides; V: transposing ldmatrix of
// byte pairs, the halves sorted out by byte permutes).
#include <cmath>
#include <mutex>

#include "tq_kv8_attention.cuh"

namespace tq {
namespace kv8 {

using namespace sm100;

int code_map(CUtensorMap* m, const void* base, int d, int64_t rows, int box) {
    typedef CUresult (*Fn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                           const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                           CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                           CUtensorMapFloatOOBfill);
    static Fn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<Fn>(p);
    });
    if (!fn) return TQ_ERR_CUDA;
    const cuuint64_t gdim[2] = {(cuuint64_t)d, (cuuint64_t)rows};
    const cuuint64_t gstride[1] = {(cuuint64_t)d};
    const cuuint32_t bdim[2] = {(cuuint32_t)d, (cuuint32_t)box};
    const cuuint32_t estride[2] = {1, 1};
    if (fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), gdim, gstride, bdim,
           estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
           d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return TQ_ERR_CUDA;
    return TQ_OK;
}

namespace {

constexpr int kTile = 32;     // keys a step
constexpr int kRows = 16;     // query rows of an item (MMA M)
constexpr int kWarps = 8;
constexpr int kStages = 3;
constexpr int kThreads = 32 * kWarps;

// Workspace: [status word (256 B) | a status word a block | a Cut a warp | per
// warp two parts: (m, L) of 16 rows, 16 x d sums].  Part 2u: the end of an item
// that warp u did not begin; 2u + 1: the beginning of one that it does not end.
struct Parts {
    int* status;
    int* block_status;
    Cut* cut;
    float2* ml;
    float* o;
};

template <int D>
struct alignas(1024) WarpSmem {
    uint8_t k[kStages][kTile * D];
    uint8_t v[kStages][kTile * D];
};
template <int D>
struct Smem {
    WarpSmem<D> w[kWarps];
    float scale[kWarps][kStages][4];  // K of both halves of a tile, V of both; K -inf: no page
    uint64_t full[kWarps][kStages];
    int64_t pre[kThreads + 1];        // steps before each thread's run of entries
    int abort;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Byte offset of the 16-byte chunk ch of row r in a swizzled tile.
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int ch) {
    return D == 128 ? (uint32_t)(r * 128 + ((ch ^ (r & 7)) << 4))
                    : (uint32_t)(r * 64 + ((ch ^ ((r >> 1) & 3)) << 4));
}

// Steps of batch entry i: heads x tiles (one tile at least, so that rows without
// keys are written); none where it has no rows, or too many for this kernel.
struct Span {
    Entry e;
    int tile0, tiles;
    int64_t steps;
};
__device__ __forceinline__ Span span_of(const Attn& a, int i) {
    Span s;
    s.e = entry_of(a, i);
    s.tile0 = first_key(a, s.e) / kTile;
    s.tiles = max(1, (s.e.len + kTile - 1) / kTile - s.tile0);
    const int64_t rows = (int64_t)s.e.qn * a.group;
    s.steps = rows > 0 && rows <= a.few ? (int64_t)a.v.heads * s.tiles : 0;
    return s;
}

// Where step g lies.
struct Place {
    Span s;
    int entry, head, t;  // t: tile within the item
    __device__ __forceinline__ void open(int64_t rem) {
        head = (int)(rem / s.tiles);
        t = (int)(rem - (int64_t)head * s.tiles);
    }
    __device__ __forceinline__ bool next(int heads) {  // false: the entry is through
        if (++t < s.tiles) return true;
        t = 0;
        return ++head < heads;
    }
};

template <int FMT, int D, typename T>
__global__ __launch_bounds__(kThreads, 1) void k_attn_rows(const Attn a, const __grid_constant__ CUtensorMap kmap,
                                                           const __grid_constant__ CUtensorMap vmap,
                                                           const Parts parts) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem<D>& sm = *reinterpret_cast<Smem<D>*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
    constexpr int CH = D / 16;  // 16-byte chunks of a code row
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = warp * gridDim.x + blockIdx.x;  // short work spreads over the SMs
    const int64_t umax = (int64_t)gridDim.x * kWarps;
    WarpSmem<D>& ws = sm.w[warp];
    volatile int* abort = &sm.abort;
    grid_begin();

    // ---- the batch's steps: a run of entries a thread, prefix over the block
    const int run = (a.ns + kThreads - 1) / kThreads;
    {
        int64_t mine = 0;
        for (int i = threadIdx.x * run; i < min(a.ns, (int)(threadIdx.x + 1) * run); ++i)
            mine += span_of(a, i).steps;
        if (threadIdx.x == 0) sm.abort = 0;
        if (lane < kStages) mbar_init(&sm.full[warp][lane], 1);
        fence_mbar_init();
        int64_t inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        sm.pre[threadIdx.x + 1] = inc;
        __syncthreads();
        int64_t before = 0;
        for (int w = 0; w < warp; ++w) before += sm.pre[32 * w + 32];
        __syncthreads();
        sm.pre[threadIdx.x + 1] = inc + before;
        if (threadIdx.x == 0) sm.pre[0] = 0;
        __syncthreads();
    }
    const int64_t total = sm.pre[kThreads];
    const int64_t units = min(umax, total);
    int64_t g0 = 0, g1 = 0;
    if (unit < units) {
        g0 = unit * total / units;
        g1 = (unit + 1) * total / units;
    }
    if (lane == 0) parts.cut[unit].parts = 0;

    auto locate = [&](int64_t g, Place& p) {
        int lo = 0, hi = kThreads;  // the run that holds step g
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sm.pre[mid] <= g) lo = mid;
            else hi = mid;
        }
        int64_t rem = g - sm.pre[lo];
        int i = lo * run;
        while (true) {
            p.s = span_of(a, i);
            if (rem < p.s.steps) break;
            rem -= p.s.steps;
            ++i;
        }
        p.entry = i;
        p.open(rem);
    };

    // ---- producer: tile loads kStages - 1 ahead.  Lane j < 4 serves half j & 1
    // of the tile (pages of 16 end inside it), K (j < 2) or V.
    Place pp = {};
    int64_t gp = g0;
    int pstage = 0;
    const int box = min(a.v.page, kTile);
    const int nbox = kTile / box;
    float pend = 0.f;   // the last produced tile's scale, on its way
    int pend_stage = -1;
    auto settle = [&]() {
        if (pend_stage >= 0 && lane < 4) sm.scale[warp][pend_stage][lane] = pend;
        pend_stage = -1;
    };
    auto produce = [&]() {
        settle();
        if (gp >= g1) return;
        uint64_t* bar = &sm.full[warp][pstage];
        if (lane == 0) mbar_arrive_expect_tx(bar, 2 * kTile * D);
        __syncwarp();
        if (lane < 4) {
            const int hf = lane & 1, isv = lane >> 1;
            const int key = (pp.s.tile0 + pp.t) * kTile + hf * 16;
            int pid = -1;
            if (key < pp.s.e.len) pid = page_of(a.v, pp.s.e.slot, key >> a.v.page_log2);
            const int64_t ph = (int64_t)max(pid, 0) * a.v.heads + pp.head;
            if (hf < nbox) {
                // an absent page reads as zeros: rows behind the tensor
                const int row = pid >= 0 ? (int)((ph << a.v.page_log2) + (key & (a.v.page - 1))) : a.rows;
                uint8_t* dst = (isv ? ws.v[pstage] : ws.k[pstage]) + hf * box * D;
                tma_load_2d(dst, isv ? &vmap : &kmap, 0, row, bar);
            }
            pend = pid < 0 ? (isv ? 0.f : -INFINITY) : (isv ? a.vs : a.ks)[ph];
        }
        pend_stage = pstage;
        pstage = pstage + 1 == kStages ? 0 : pstage + 1;
        if (++gp < g1 && !pp.next(a.v.heads)) {
            // the following entry with steps
            int i = pp.entry;
            do {
                pp.s = span_of(a, ++i);
            } while (pp.s.steps == 0);
            pp.entry = i;
            pp.open(0);
        }
    };

    Place p = {};
    bool ok = true;
    if (g0 < g1) {
        locate(g0, pp);
        p = pp;
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) produce();
    }
    int stage = 0;
    uint32_t phase = 0;
    const int c2 = lane & 3, r0 = lane >> 2;
    // ldmatrix row of this lane: row lane % 8 of matrix lane / 8
    const int lrow = lane & 7, lmat = lane >> 3;

    for (int64_t g = g0; g < g1 && ok;) {
        // ---- an item, or this warp's part of it: tiles p.t .. t_end of its s.tiles
        const int64_t left = g1 - g;
        const int t_begin = p.t;
        const int t_end = (int)min((int64_t)p.s.tiles, t_begin + left);
        const Entry e = p.s.e;
        const int nrows = e.qn * a.group;
        // rows r0 and r0 + 8 of this thread: query token, and the last key it sees
        uint32_t qf[CH][4];
        float sl[2], m[2] = {-INFINITY, -INFINITY}, L[2] = {0.f, 0.f};
        int lim[2], low[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = r0 + 8 * u;
            const int ri = min(r, nrows - 1), tq = ri / a.group, hq = ri - tq * a.group;
            const T* q = (const T*)a.q + (e.c0 + tq) * a.q_ts + (int64_t)(p.head * a.group + hq) * a.q_hs;
            const int pos = e.len - e.qn + tq;
            lim[u] = a.causal ? min(pos, e.len - 1) : e.len - 1;
            low[u] = below_window(a, pos);
            float x[CH][4], top = 0.f;
#pragma unroll
            for (int ch = 0; ch < CH; ++ch) {
                const Pack<T, 4> v = *reinterpret_cast<const Pack<T, 4>*>(q + 16 * ch + 4 * c2);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    x[ch][k] = to_f(v.v[k]);
                    top = fmaxf(top, fabsf(x[ch][k]));
                }
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float unit_q = row_unit(top);
            sl[u] = a.scale_log2 / unit_q;
#pragma unroll
            for (int ch = 0; ch < CH; ++ch) {
                qf[ch][u] = pack_half2(x[ch][0] * unit_q, x[ch][1] * unit_q);
                qf[ch][u + 2] = pack_half2(x[ch][2] * unit_q, x[ch][3] * unit_q);
            }
        }
        // keys below `clear` and above `low_any` need no mask for any row
        const int clear = a.causal ? min(e.len - e.qn, e.len - 1) : e.len - 1;
        const int low_any = a.window > 0 ? e.len - 1 - a.window : -1;
        float o[2 * CH][4];  // chunk, parity: coordinates 16 ch + 4 c2 + 2 {0, 1} + parity
#pragma unroll
        for (int i = 0; i < 2 * CH; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
        float R = 0.f;  // running largest value scale: o is in units of it

        for (int t = t_begin; t < t_end; ++t) {
            const int key0 = (p.s.tile0 + t) * kTile;
            settle();
            if (!mbar_wait(&sm.full[warp][stage], phase, abort, kWaitNs)) ok = false;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const float4 sc = *reinterpret_cast<const float4*>(sm.scale[warp][stage]);
            // ---- logits: 4 blocks of 8 keys
            float s[4][4];
            const uint32_t kb = smem_u32(ws.k[stage]);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
#pragma unroll
                for (int k = 0; k < 4; ++k) s[b][k] = 0.f;
#pragma unroll
                for (int c = 0; c < CH; c += 4) {
                    uint32_t w[4];
                    ldsm4(kb + swz<D>(8 * b + lrow, c + lmat), w);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t lo, hi;
                        codes_to_half<FMT>(w[k], lo, hi);
                        mma16816(s[b], qf[c + k], lo, hi);
                    }
                }
            }
            const bool masked = key0 + kTile - 1 > clear || key0 <= low_any || sc.x == -INFINITY ||
                                sc.y == -INFINITY;
            float mx[2] = {m[0], m[1]};
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const float ks = b < 2 ? sc.x : sc.y;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int u = k >> 1;
                    float l = s[b][k] * (sl[u] * ks);
                    if (masked) {
                        const int key = key0 + 8 * b + 2 * c2 + (k & 1);
                        if (key > lim[u] || key <= low[u] || ks == -INFINITY) l = -INFINITY;
                    }
                    s[b][k] = l;
                    mx[u] = fmaxf(mx[u], l);
                }
            }
            float alpha[2];
            const float vmax = fmaxf(sc.z, sc.w);
            const float shrink = vmax > R ? R / vmax : 1.f;
            R = fmaxf(R, vmax);
            // (scales below fp32's normal range have no reciprocal: their values count as 0)
            const float inv = R >= 1.17549435e-38f ? 1.f / R : 0.f;
            const float w0 = sc.z * inv, w1 = sc.w * inv;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 1));
                mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 2));
                const float base = mx[u] == -INFINITY ? 0.f : mx[u];
                alpha[u] = ex2(m[u] - base);
                m[u] = mx[u];
                mx[u] = base;
                L[u] *= alpha[u];
                alpha[u] *= shrink;
            }
            uint32_t pf[2][4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const float w = b < 2 ? w0 : w1;
                float pr[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    pr[k] = ex2(s[b][k] - mx[k >> 1]);
                    L[k >> 1] += pr[k];
                }
                pf[b >> 1][2 * (b & 1)] = pack_half2(pr[0] * w, pr[1] * w);
                pf[b >> 1][2 * (b & 1) + 1] = pack_half2(pr[2] * w, pr[3] * w);
            }
            if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
                for (int i = 0; i < 2 * CH; ++i) {
                    o[i][0] *= alpha[0];
                    o[i][1] *= alpha[0];
                    o[i][2] *= alpha[1];
                    o[i][3] *= alpha[1];
                }
            }
            // e4m3 rows behind the slot's end may hold NaN codes, and 0 NaN is NaN
            if (FMT == TQ_KV_E4M3 && key0 + kTile > e.len) {
                for (int i = lane; i < kTile * CH; i += 32)
                    if (key0 + i / CH >= e.len)
                        *reinterpret_cast<uint4*>(ws.v[stage] + 16 * i) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
            }
            // ---- values: 16 keys x 32 coordinates a load
            const uint32_t vb = smem_u32(ws.v[stage]);
#pragma unroll
            for (int k16 = 0; k16 < 2; ++k16) {
#pragma unroll
                for (int c = 0; c < CH; c += 2) {
                    uint32_t w[4];  // keys 0-7 | 8-15 of chunk c, then of chunk c + 1
                    ldsm4t(vb + swz<D>(16 * k16 + 8 * (lmat & 1) + lrow, c + (lmat >> 1)), w);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t e0, e1, d0, d1;
                        codes_to_half_02<FMT>(w[2 * h], e0, d0);
                        codes_to_half_02<FMT>(w[2 * h + 1], e1, d1);
                        mma16816(o[2 * (c + h)], pf[k16], e0, e1);
                        mma16816(o[2 * (c + h) + 1], pf[k16], d0, d1);
                    }
                }
            }
            __syncwarp();  // every lane is done with the stage
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1;
            }
            produce();
        }
        if (!ok) break;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            L[u] += __shfl_xor_sync(0xffffffffu, L[u], 1);
            L[u] += __shfl_xor_sync(0xffffffffu, L[u], 2);
        }
        const bool begins = t_begin == 0, ends = t_end == p.s.tiles;
        if (begins && ends) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = r0 + 8 * u;
                if (r >= nrows) continue;
                const int64_t tok = e.c0 + r / a.group;
                const int hq = p.head * a.group + r % a.group;
                const float n = L[u] > 0.f ? R / L[u] : (L[u] == 0.f ? 0.f : L[u]);
                T* out = (T*)a.out + (tok * a.heads_q + hq) * D;
#pragma unroll
                for (int ch = 0; ch < CH; ++ch) {
                    Pack<T, 4> v;
                    from_f(o[2 * ch][2 * u] * n, v.v[0]);
                    from_f(o[2 * ch + 1][2 * u] * n, v.v[1]);
                    from_f(o[2 * ch][2 * u + 1] * n, v.v[2]);
                    from_f(o[2 * ch + 1][2 * u + 1] * n, v.v[3]);
                    *reinterpret_cast<Pack<T, 4>*>(out + 16 * ch + 4 * c2) = v;
                }
                if (a.lse && c2 == 0)
                    a.lse[tok * a.heads_q + hq] = L[u] > 0.f ? (m[u] + log2f(L[u])) * 0.69314718056f : m[u];
            }
        } else {
            const int64_t slot = 2 * (int64_t)unit + (begins ? 1 : 0);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = r0 + 8 * u;
                if (r >= nrows) continue;
                if (c2 == 0) parts.ml[slot * kRows + r] = make_float2(m[u], L[u]);
                float* dst = parts.o + (slot * kRows + r) * D;
#pragma unroll
                for (int ch = 0; ch < CH; ++ch)
                    *reinterpret_cast<float4*>(dst + 16 * ch + 4 * c2) =
                        make_float4(o[2 * ch][2 * u] * R, o[2 * ch + 1][2 * u] * R,
                                    o[2 * ch][2 * u + 1] * R, o[2 * ch + 1][2 * u + 1] * R);
            }
            if (begins && lane == 0) {
                const int64_t last = g + p.s.tiles - 1;  // the item's last step: its warp
                Cut c;
                c.parts = (int)(((last + 1) * units - 1) / total) - unit + 1;
                c.rows = nrows;
                c.head = p.head;
                c.pad = 0;
                c.row0 = e.c0 * a.group;
                parts.cut[unit] = c;
            }
        }
        g += t_end - t_begin;
        if (g < g1) {
            p.t = p.s.tiles - 1;
            if (!p.next(a.v.heads)) {
                int i = p.entry;
                do {
                    p.s = span_of(a, ++i);
                } while (p.s.steps == 0);
                p.entry = i;
                p.open(0);
            }
        }
    }
    if (!ok) {
        // gave up: no copy of this warp's ring may land after it has left
        *abort = 1;
        for (int s = 0; s < kStages; ++s) mbar_wait(&sm.full[warp][s], phase, abort, kWaitNs);
    }
    __syncthreads();
    if (threadIdx.x == 0) parts.block_status[blockIdx.x] = sm.abort ? TQ_ERR_DEVICE_TIMEOUT * 1000 - 80 : 0;
}

// Joins the parts of the items that were cut: block (u, r) row r of the item
// that begins in warp u and does not end there.  4 warps take every fourth part.
template <int D, typename T>
__global__ __launch_bounds__(128) void k_attn_merge(const Attn a, const Parts parts, int blocks) {
    const int u = blockIdx.x, r = blockIdx.y;
    grid_begin();
    if (u == 0 && r == 0) {  // the call's status
        int st = 0;
        for (int i = threadIdx.x; i < blocks; i += 128) st = min(st, parts.block_status[i]);
        st = __syncthreads_or(st);
        if (threadIdx.x == 0) *parts.status = st ? TQ_ERR_DEVICE_TIMEOUT * 1000 - 80 : 0;
    }
    const Cut c = parts.cut[u];
    if (c.parts == 0 || r >= c.rows) return;
    __shared__ float s_ml[4][2];
    __shared__ float s_o[4][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int E = D / 32;
    // part i of the item: 2u + 1 first, then 2 (u + i)
    auto slot = [&](int i) { return i == 0 ? 2 * (int64_t)u + 1 : 2 * (int64_t)(u + i); };
    float m = -INFINITY;
    for (int i = threadIdx.x; i < c.parts; i += 128) m = fmaxf(m, parts.ml[slot(i) * kRows + r].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) s_ml[warp][0] = m;
    __syncthreads();
    m = fmaxf(fmaxf(s_ml[0][0], s_ml[1][0]), fmaxf(s_ml[2][0], s_ml[3][0]));
    const float base = m == -INFINITY ? 0.f : m;
    float L = 0.f, acc[E];
#pragma unroll
    for (int k = 0; k < E; ++k) acc[k] = 0.f;
#pragma unroll 4
    for (int i = warp; i < c.parts; i += 4) {
        const float2 ml = parts.ml[slot(i) * kRows + r];
        const float w = ex2(ml.x - base);
        L = fmaf(w, ml.y, L);
        const float* src = parts.o + (slot(i) * kRows + r) * D + lane * E;
        float x[E];
        if (E == 4) *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(src);
        else *reinterpret_cast<float2*>(x) = *reinterpret_cast<const float2*>(src);
#pragma unroll
        for (int k = 0; k < E; ++k) acc[k] = fmaf(w, x[k], acc[k]);
    }
    if (lane == 0) s_ml[warp][1] = L;
#pragma unroll
    for (int k = 0; k < E; ++k) s_o[warp][lane * E + k] = acc[k];
    __syncthreads();
    L = s_ml[0][1] + s_ml[1][1] + s_ml[2][1] + s_ml[3][1];
    const int64_t ri = c.row0 + r, tok = ri / a.group;
    const int hq = c.head * a.group + (int)(ri % a.group);
    const float n = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
    if (threadIdx.x < D) {
        const float x = s_o[0][threadIdx.x] + s_o[1][threadIdx.x] + s_o[2][threadIdx.x] + s_o[3][threadIdx.x];
        from_f(x * n, ((T*)a.out)[(tok * a.heads_q + hq) * D + threadIdx.x]);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[tok * a.heads_q + hq] = L > 0.f ? (m + log2f(L)) * 0.69314718056f : m;
}

constexpr int kMaxBlocks = 148;  // the workspace's size

// The most steps that a call of these sizes can have (its lengths lie on the
// device); blocks: one an SM, fewer where the tables are too short to fill them.
int64_t most_steps(const tq_kv8_t* c, int ns) {
    return ((int64_t)c->max_pages * c->page + kTile - 1) / kTile * ns * c->heads;
}
int64_t blocks_for(const tq_kv8_t* c, int ns) {
    const int64_t steps = most_steps(c, ns);
    return steps < kMaxBlocks ? (steps < 1 ? 1 : steps) : kMaxBlocks;
}

// Which kernels a call launches: an entry of up to kRows rows takes the few-rows
// kernel.  The counts of a batch lie on the device; where total_q is ns times
// max_q every entry has max_q tokens (or the batch is padded), and beyond kRows
// the prompt kernel takes all entries.
bool any_few(const tq_kv8_t* c, int ns, int64_t total_q, int max_q, int heads_q) {
    return (int64_t)max_q * (heads_q / c->heads) <= kRows || total_q < (int64_t)ns * max_q;
}
bool any_many(const tq_kv8_t* c, int max_q, int heads_q) {
    return (int64_t)max_q * (heads_q / c->heads) > kRows;
}

template <int D>
Parts carve(void* ws, int64_t blocks, size_t* bytes) {
    const int64_t units = blocks * kWarps;
    Parts p;
    char* at = (char*)ws;
    p.status = (int*)at;
    at += 256;
    p.block_status = (int*)at;
    at += align256(blocks * 4);
    p.cut = (Cut*)at;
    at += align256(units * sizeof(Cut));
    p.ml = (float2*)at;
    at += align256(2 * units * kRows * sizeof(float2));
    p.o = (float*)at;
    at += align256(2 * units * kRows * D * 4);
    *bytes = (size_t)(at - (char*)ws);
    return p;
}

template <int FMT, int D, typename T>
int launch(const Attn& a, const CUtensorMap& km, const CUtensorMap& vm, const Parts& p, int blocks,
           int cuts, int rows, cudaStream_t s) {
    constexpr int smem = (int)sizeof(Smem<D>) + 1024;
    int rc = allow_smem<k_attn_rows<FMT, D, T>>(smem);
    if (!rc) rc = launch_behind(k_attn_rows<FMT, D, T>, dim3(blocks), kThreads, smem, s, a, km, vm, p);
    if (!rc)
        rc = launch_behind(k_attn_merge<D, T>, dim3((unsigned)cuts, (unsigned)rows), 128, 0, s, a, p, blocks);
    return rc;
}

template <int D>
int dispatch(const tq_kv8_t* c, const Attn& a, const CUtensorMap& km, const CUtensorMap& vm,
             const Parts& p, int blocks, int cuts, int rows, int q_dtype, cudaStream_t s) {
    if (c->format == TQ_KV_I8)
        return q_dtype == TQ_BF16
                   ? launch<TQ_KV_I8, D, __nv_bfloat16>(a, km, vm, p, blocks, cuts, rows, s)
                   : launch<TQ_KV_I8, D, __half>(a, km, vm, p, blocks, cuts, rows, s);
    return q_dtype == TQ_BF16
               ? launch<TQ_KV_E4M3, D, __nv_bfloat16>(a, km, vm, p, blocks, cuts, rows, s)
               : launch<TQ_KV_E4M3, D, __half>(a, km, vm, p, blocks, cuts, rows, s);
}

Parts carve_for(const tq_kv8_t* c, void* ws, int64_t blocks, size_t* bytes) {
    return c->d == 128 ? carve<128>(ws, blocks, bytes) : carve<64>(ws, blocks, bytes);
}

}  // namespace

// [status word | the few-rows kernel's parts | the prompt kernel's parts]
size_t attention_workspace(const tq_kv8_t* c, int ns, int64_t total_q, int max_q, int heads_q) {
    size_t few = 256, many = 0;
    if (any_few(c, ns, total_q, max_q, heads_q)) carve_for(c, nullptr, blocks_for(c, ns), &few);
    if (any_many(c, max_q, heads_q))
        prompt_carve(c, nullptr, prompt_blocks(c, ns, total_q, heads_q), &many);
    return few + many;
}

}  // namespace kv8
}  // namespace tq

using namespace tq;

extern "C" int tq_kv8_attention(const tq_kv8_t* c, int layer, int ns, const int32_t* d_slots,
                                const int32_t* d_cu, int64_t total_q, int max_q, int heads_q,
                                const void* d_q, int q_dtype, int64_t q_ts, int64_t q_hs, float scale,
                                int causal, int window, void* d_out, float* d_lse, void* d_ws,
                                size_t ws_bytes, void* stream) {
    int status;
    if (!kv8::valid(c, &status)) return status;
    if (layer < 0 || layer >= c->layers || ns < 0 || total_q < 0 || max_q < 0 || heads_q < 1)
        return TQ_ERR_ARG;
    if (q_dtype != TQ_BF16 && q_dtype != TQ_F16) return TQ_ERR_ARG;
    if (causal < 0 || causal > 1 || window < 0 || (window > 0 && !causal) || !std::isfinite(scale))
        return TQ_ERR_ARG;
    if (!d_slots && ns > c->slots) return TQ_ERR_ARG;
    if (heads_q % c->heads || heads_q / c->heads > 128) return TQ_ERR_UNSUPPORTED;
    if (ns == 0 || total_q == 0 || max_q == 0) return TQ_OK;
    if (!d_cu || !d_q || !d_out || (((uintptr_t)d_q | (uintptr_t)d_out) & 15u) || q_ts % 8 || q_hs % 8)
        return TQ_ERR_ARG;
    if (!d_ws || ws_bytes < kv8::attention_workspace(c, ns, total_q, max_q, heads_q))
        return TQ_ERR_WORKSPACE;
    kv8::Attn a;
    a.v = kv8::view(c);
    a.ns = ns;
    a.group = heads_q / c->heads;
    a.heads_q = heads_q;
    a.causal = causal;
    a.window = window;
    a.slots = d_slots;
    a.cu = d_cu;
    a.total_q = total_q;
    a.q = d_q;
    a.q_ts = q_ts;
    a.q_hs = q_hs;
    a.scale_log2 = scale * 1.44269504089f;
    a.ks = c->d_kscale + layer * kv8::layer_scales(c);
    a.vs = c->d_vscale + layer * kv8::layer_scales(c);
    a.out = d_out;
    a.lse = d_lse;
    a.rows = c->pages * c->heads * c->page;
    cudaStream_t s = (cudaStream_t)stream;
    const bool few = kv8::any_few(c, ns, total_q, max_q, heads_q);
    a.few = few ? kv8::kRows : 0;
    size_t at = 256;
    if (few) {
        const int box = c->page < kv8::kTile ? c->page : kv8::kTile;
        CUtensorMap km, vm;
        int rc = kv8::code_map(&km, (const char*)c->d_k + layer * kv8::layer_bytes(c), c->d, a.rows, box);
        if (!rc) rc = kv8::code_map(&vm, (const char*)c->d_v + layer * kv8::layer_bytes(c), c->d, a.rows, box);
        if (rc) return rc;
        const int blocks = (int)kv8::blocks_for(c, ns);
        const kv8::Parts p = kv8::carve_for(c, d_ws, blocks, &at);
        const int64_t steps = kv8::most_steps(c, ns);
        const int cuts = (int)(steps < blocks * kv8::kWarps ? steps : blocks * kv8::kWarps);
        const int64_t most = (int64_t)max_q * a.group;
        const int rows = (int)(most < kv8::kRows ? most : kv8::kRows);
        rc = c->d == 128 ? kv8::dispatch<128>(c, a, km, vm, p, blocks, cuts, rows, q_dtype, s)
                         : kv8::dispatch<64>(c, a, km, vm, p, blocks, cuts, rows, q_dtype, s);
        if (rc) return rc;
    }
    if (!kv8::any_many(c, max_q, heads_q)) return TQ_OK;
    size_t bytes;
    const int blocks = kv8::prompt_blocks(c, ns, total_q, heads_q);
    kv8::PromptParts p = kv8::prompt_carve(c, (char*)d_ws + at, blocks, &bytes);
    p.status = (int*)d_ws;
    p.keep_status = few;
    return kv8::launch_prompt(c, layer, a, p, blocks, q_dtype, s);
}
