// Attention over the 8-bit paged cache, few query rows: for every row (query
// token, query head) of a slot,
//   l_j = scale s_k(j) <q, c_k(j)>,   out = sum_j softmax(l)_j s_v(j) c_v(j).
//
// Numerics.  Codes are exact halves; a query row times a power of two is a row
// of halves (row_unit), so <q, c> is a sum of exact products in fp32.  The
// block scales never touch the codes: s_k multiplies the logit, s_v the
// probability, and the product is rounded to a half (2^-11) in units of its own
// row's, a power of two by which the row's largest product so far is at 2^10 at least:
// what is smaller than halves' normal range is off by 2^-35 of that largest one, and
// keys that the row does not see have no part in it.  (The unit is kept relative to the
// reference of the logits, which may be so large that their last bits are whole units.)
// Maximum, sum and output are fp32.
//
// Work.  Reading the cache is the cost (2 d bytes a token and KV head for up to
// 16 rows), so every warp is a stream of its own: it takes an equal, contiguous
// share of all (entry, head, 32-key tile) steps of the batch --
// ragged lengths included -- and keeps kStages tiles of K and V in flight by TMA
// into its private ring; warps meet only where an item's steps are cut (joining
// the parts, below).  Products are
// m16n8k16 MMAs with the codes as the A operand (16 keys, then 16 coordinates)
// and the query rows as the 8 columns: a code is converted once for all rows, and
// 8 rows cost half of what 16 do.  Fragments are made in registers from the codes
// (K: plain ldmatrix, coordinates permuted alike on both sides; V: transposing
// ldmatrix of byte pairs, the halves sorted out by byte permutes).
//
// Measured: 4 x 131072 keys x 8 heads of 128, one token of 32 heads: 191 us, 5.6 TB/s
// (a copy runs at 6.55); 64 ragged sequences 104 us, 5.2 TB/s; one sequence of 500
// keys 9.5 us, a chain of lookups, two tiles of dependent instructions and the join.
// With 8 warps of 16 rows and lookups in line: 233, 122 and 10.4 us.  16 rows are bound
// by issue and by what is spilled of 168 registers: 184 us for keys that one token reads
// in 95 (16 x 16384).
#include <atomic>
#include <chrono>
#include <cmath>
#include <mutex>

#include "kv8_bind.h"
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
constexpr int kRows = 16;     // query rows of an item, at most
constexpr int kWarps = 12;
constexpr int kThreads = 32 * kWarps;
constexpr int kItemTiles = 4 * kWarps;  // see "sharing out"
constexpr float kStart = 11.f;  // a row's largest product: at 2^(kStart - 1) at least
template <int D>
constexpr int kStages = D == 128 ? 2 : 4;  // 16 KB of a warp's ring

// Sharing out.  A small batch (no more items than blocks, none of more than
// kItemTiles tiles) takes a block an item.  Otherwise every warp takes an equal,
// contiguous share of the steps; few steps keep only the first `busy` warps of each
// block at work, so that they spread over the SMs.  "Unit" u is warp u % busy of
// block u / busy.
//
// Joining.  A block's parts of an item meet in shared memory (the ring of a warp
// that is through), or in the workspace where their warp goes on with another item
// (slot w of warp w of the grid).  Where the item lies within the block that is its
// result; of an item across blocks each block leaves one sum in the workspace (slot
// 2b: the end or middle of an item that block b did not begin, 2b + 1 the beginning
// of one).  A block sets its flag behind its sum of the one item that goes on beyond
// it, and the block in which the item ends waits for the flags of the others --
// blocks before it, which are dispatched before it -- and joins.  A flag is set to
// the call's nonce and taken back by the joining block, so a workspace needs no
// preparation and a replayed graph finds none set.  The order of the sum is that of
// the keys.
//
// Workspace: [status word (256 B) | a flag a block | (m, L) of 16 rows and 16 x d
// sums: a slot a warp, then two a block].
struct Parts {
    int* status;
    uint64_t* flag;
    float2* ml;
    float* o;
    uint64_t nonce;
};

// A block's parts of an item.
struct Job {
    int64_t row0;   // the item's first row of the entry's (token x group) rows, from token 0
    int64_t first;  // the unit that begins the item
    int parts;      // warps of the block that hold a part; 0: no job
    int rows, head;
    bool begins, ends;  // in this block
};

template <int D>
struct alignas(1024) WarpSmem {
    uint8_t k[kStages<D>][kTile * D];
    uint8_t v[kStages<D>][kTile * D];
};
template <int D>
struct Smem {
    WarpSmem<D> w[kWarps];
    float scale[kWarps][kStages<D>][4];  // K of both halves of a tile, V of both; K -inf: no page
    uint64_t full[kWarps][kStages<D>];
    int64_t pre[kThreads + 1];           // steps before each thread's run of entries
    int items[kThreads + 1];             // items before it
    int64_t warp_steps[kWarps];
    int warp_items[kWarps], warp_most[kWarps];
    float2 ml[kWarps][kRows];            // of the part that a warp leaves in its ring
    Job job[kWarps + 1];                 // of the items that a warp begins; the last: begun before the block
    int outside[kWarps];                 // this warp left the end of an item in the workspace
    int beyond;                          // an item goes on behind the block
    int used;                            // tokens that entries own
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
// An 8 x 8 matrix of halves, transposed.
__device__ __forceinline__ uint32_t movm(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
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
        head = (int)quot(rem, s.tiles);
        t = (int)(rem - (int64_t)head * s.tiles);
    }
    __device__ __forceinline__ bool next(int heads) {  // false: the entry is through
        if (++t < s.tiles) return true;
        t = 0;
        return ++head < heads;
    }
};

__device__ __forceinline__ void set_flag(uint64_t* p, uint64_t x) {
    asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(x) : "memory");
}
__device__ __forceinline__ uint64_t get_flag(const uint64_t* p) {
    uint64_t x;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(x) : "l"(p) : "memory");
    return x;
}
template <int D>
struct Sum {
    float m, L, acc[D / 32];  // coordinates lane * D / 32 ..
};
// Every `step`-th of n parts of a row, from part i0 on: a warp.  ml(i), o(i):
// where part i lies.
template <int D, typename Ml, typename O>
__device__ __forceinline__ Sum<D> sum_parts(int n, int i0, int step, int lane, Ml ml, O o) {
    constexpr int E = D / 32;
    Sum<D> s;
    s.m = -INFINITY;
    s.L = 0.f;
#pragma unroll
    for (int k = 0; k < E; ++k) s.acc[k] = 0.f;
    for (int c0 = i0; c0 < n; c0 += 32 * step) {  // 32 parts: (m, L) of one a lane
        const int mine = c0 + lane * step;
        const float2 x = mine < n ? ml(mine) : make_float2(-INFINITY, 0.f);
        float m = fmaxf(s.m, x.x);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
        const float base = m == -INFINITY ? 0.f : m;
        const float w = ex2(x.x - base), old = ex2(s.m - base);
        float L = w * x.y;
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) L += __shfl_xor_sync(0xffffffffu, L, k);
        s.L = fmaf(s.L, old, L);
        s.m = m;
#pragma unroll
        for (int k = 0; k < E; ++k) s.acc[k] *= old;
        const int cnt = min(32, (n - c0 + step - 1) / step);
#pragma unroll 8
        for (int i = 0; i < cnt; ++i) {
            const float* src = o(c0 + i * step) + lane * E;
            float y[E];
            if (E == 4) *reinterpret_cast<float4*>(y) = *reinterpret_cast<const float4*>(src);
            else *reinterpret_cast<float2*>(y) = *reinterpret_cast<const float2*>(src);
            const float f = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
            for (int k = 0; k < E; ++k) s.acc[k] = fmaf(f, y[k], s.acc[k]);
        }
    }
    return s;
}
template <int D, typename T>
__device__ __forceinline__ void write_row(const Attn& a, const Job& job, int r, const Sum<D>& s, int lane) {
    constexpr int E = D / 32;
    const int t = r / a.group;  // row0 is a token's first row
    const int64_t tok = quot(job.row0, a.group) + t;
    const int hq = job.head * a.group + r - t * a.group;
    const float n = s.L > 0.f ? 1.f / s.L : (s.L == 0.f ? 0.f : s.L);
    Pack<T, E> y;
#pragma unroll
    for (int k = 0; k < E; ++k) from_f(s.acc[k] * n, y.v[k]);
    *reinterpret_cast<Pack<T, E>*>((T*)a.out + (tok * a.heads_q + hq) * D + lane * E) = y;
    if (a.lse && lane == 0)
        a.lse[tok * a.heads_q + hq] = s.L > 0.f ? (s.m + log2f(s.L)) * 0.69314718056f : s.L == 0.f ? -INFINITY : s.L;
}

// NB: blocks of 8 query rows.
template <int FMT, int D, int NB, typename T>
__global__ __launch_bounds__(kThreads, 1) void k_attn_rows(const Attn a, const __grid_constant__ CUtensorMap kmap,
                                                           const __grid_constant__ CUtensorMap vmap,
                                                           const Parts parts) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem<D>& sm = *reinterpret_cast<Smem<D>*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
    constexpr int CH = D / 16;  // 16-byte chunks of a code row
    constexpr int NS = kStages<D>;
    // registers are short: a row's limits are formed where a mask is (64 sequences: 104
    // against 107 us; 16 x 16384 keys 93 against 96; where they are not short it loses)
    constexpr bool kLean = NB == 1 && D == 128;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int self = blockIdx.x * kWarps + warp;
    WarpSmem<D>& ws = sm.w[warp];
    volatile int* abort = &sm.abort;
    if (threadIdx.x == 0) {
        sm.abort = 0;
        sm.beyond = 0;
    }
    if (lane == 0) {
        sm.job[warp].parts = 0;
        sm.job[kWarps].parts = 0;
        sm.outside[warp] = 0;
    }
    if (threadIdx.x == 64) sm.used = INT32_MAX;
    if (lane < NS) mbar_init(&sm.full[warp][lane], 1);
    fence_mbar_init();
    if (threadIdx.x == 0) {
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
    }
    grid_begin();
    int held = pending(a.v);
    if (a.behind && threadIdx.x == 64) sm.used = max(a.cu[a.ns], 0);
    // (blocks are dispatched in order, and one that gives up has waited for a second)
    if (blockIdx.x == 0 && threadIdx.x == 0) *parts.status = held;

    // ---- the batch's steps and items: a run of entries a thread, prefixes over the block
    const int run = (a.ns + kThreads - 1) / kThreads;
    {
        int64_t steps = 0;
        int items = 0, most = 0;
        for (int i = threadIdx.x * run; i < min(a.ns, (int)(threadIdx.x + 1) * run); ++i) {
            const Span s = span_of(a, i);
            if (misfit(a, i, s.e)) held = held ? held : TQ_ERR_ARG;
            steps += s.steps;
            items = min(items + (s.steps > 0 ? a.v.heads : 0), 1 << 20);
            most = max(most, s.steps > 0 ? s.tiles : 0);
        }
        most = __reduce_max_sync(0xffffffffu, most);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, steps, o);
            const int y = __shfl_up_sync(0xffffffffu, items, o);
            if (lane >= o) {
                steps += x;
                items += y;
            }
        }
        if (lane == 31) {
            sm.warp_steps[warp] = steps;
            sm.warp_items[warp] = items;
            sm.warp_most[warp] = most;
        }
        if (__syncthreads_or(held)) {
            if (blockIdx.x == 0 && held == TQ_ERR_ARG) {
                *parts.status = held;
                leave_status(a.v, held);
            }
            empty_rows<D, T>(a);
            zero_behind<D, T>(a, sm.used);
            return;
        }
        for (int w = 0; w < warp; ++w) {
            steps += sm.warp_steps[w];
            items += sm.warp_items[w];
        }
        sm.pre[threadIdx.x + 1] = steps;
        sm.items[threadIdx.x + 1] = items;
        if (threadIdx.x == 0) sm.pre[0] = sm.items[0] = 0;
        __syncthreads();
    }
    const int64_t total = sm.pre[kThreads];
    int most = 0;
    for (int w = 0; w < kWarps; ++w) most = max(most, sm.warp_most[w]);
    const bool by_item = sm.items[kThreads] <= (int)gridDim.x && most <= kItemTiles;
    const int runs = (a.ns + run - 1) / run;

    Place p = {};
    int busy = 1;
    int64_t g0 = 0, g1 = 0, units = 0, unit = 0, base = 0, rest = 0;
    if (by_item) {
        if ((int)blockIdx.x < sm.items[kThreads]) {
            int lo = 0, hi = runs;  // the run that holds this block's item
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (sm.items[mid] <= (int)blockIdx.x) lo = mid;
                else hi = mid;
            }
            int rem = blockIdx.x - sm.items[lo];
            p.entry = lo * run;
            while (true) {
                p.s = span_of(a, p.entry);
                const int n = p.s.steps > 0 ? a.v.heads : 0;
                if (rem < n) break;
                rem -= n;
                ++p.entry;
            }
            p.head = rem;
            busy = min(kWarps, p.s.tiles);
            if (warp < busy) {
                g0 = (unsigned)(warp * p.s.tiles) / (unsigned)busy;
                g1 = (unsigned)((warp + 1) * p.s.tiles) / (unsigned)busy;
                p.t = (int)g0;
            }
        }
        unit = (int64_t)blockIdx.x * busy + warp;
    } else {
        busy = (int)min((int64_t)kWarps, quot(total + gridDim.x - 1, gridDim.x));
        units = min((int64_t)gridDim.x * busy, total);
        unit = (int64_t)blockIdx.x * busy + warp;
        // the first `rest` units take base + 1 steps, the others base
        base = quot(total, units);
        rest = total - base * units;
        if (warp < busy && unit < units) {
            g0 = unit * base + min(unit, rest);
            g1 = g0 + base + (unit < rest ? 1 : 0);
            int lo = 0, hi = runs;  // the run that holds step g0
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (sm.pre[mid] <= g0) lo = mid;
                else hi = mid;
            }
            int64_t rem = g0 - sm.pre[lo];
            p.entry = lo * run;
            while (true) {
                p.s = span_of(a, p.entry);
                if (rem < p.s.steps) break;
                rem -= p.s.steps;
                ++p.entry;
            }
            p.open(rem);
        }
    }
    // a block's two sums lie behind the warps' slots
    auto block_slot = [&](int b) { return (int64_t)gridDim.x * kWarps + 2 * b; };
    // the unit that takes a step
    auto owner = [&](int64_t step) {
        const int64_t head = rest * (base + 1);
        return step < head ? quot(step, base + 1) : rest + quot(step - head, base);
    };
    // On to the next step's place, over entries without steps.
    auto advance = [&](Place& p) {
        if (p.next(a.v.heads)) return;
        int i = p.entry;
        do {
            p.s = span_of(a, ++i);
        } while (p.s.steps == 0);
        p.entry = i;
        p.open(0);
    };

    // ---- producer: tile loads NS - 1 ahead, page ids one further, scales into
    // shared memory one tile later: nothing waits for a lookup.  Lane j < 4 serves
    // half j & 1 of the tile (pages of 16 end inside it), K (j < 2) or V.
    Place pp = p;
    int64_t gp = g0;
    uint32_t np = 0;  // tiles produced
    const int box = min(a.v.page, kTile), nbox = kTile / box;
    const int hf = lane & 1, isv = lane >> 1;
    int pid = -1;       // page of this lane's half of the next tile
    float pend = 0.f;   // the last produced tile's scale, on its way
    int pend_stage = -1;
    auto lookup = [&]() {
        if (lane < 4) {
            const int key = (pp.s.tile0 + pp.t) * kTile + hf * 16;
            pid = key < pp.s.e.len ? page_of(a.v, pp.s.e.slot, key >> a.v.page_log2) : -1;
        }
    };
    auto settle = [&]() {
        if (pend_stage >= 0 && lane < 4) sm.scale[warp][pend_stage][lane] = pend;
        pend_stage = -1;
        __syncwarp();  // all lanes read the scales next, also where no tile is left to produce
    };
    auto produce = [&]() {
        settle();
        if (gp >= g1) return;
        const int st = np % NS;
        uint64_t* bar = &sm.full[warp][st];
        if (lane == 0) mbar_arrive_expect_tx(bar, 2 * kTile * D);
        __syncwarp();
        if (lane < 4) {
            const int key = (pp.s.tile0 + pp.t) * kTile + hf * 16;
            const int64_t ph = (int64_t)max(pid, 0) * a.v.heads + pp.head;
            if (hf < nbox) {
                // an absent page reads as zeros: rows behind the tensor
                const int row = pid >= 0 ? (int)((ph << a.v.page_log2) + (key & (a.v.page - 1))) : a.rows;
                uint8_t* dst = (isv ? ws.v[st] : ws.k[st]) + hf * box * D;
                tma_load_2d(dst, isv ? &vmap : &kmap, 0, row, bar);
            }
            pend = pid < 0 ? (isv ? 0.f : -INFINITY) : (isv ? a.vs : a.ks)[ph];
        }
        pend_stage = st;
        ++np;
        if (++gp < g1) {
            advance(pp);
            lookup();
        }
    };

    bool ok = true;
    if (g0 < g1) {
        lookup();
#pragma unroll
        for (int s = 0; s < NS - 1; ++s) produce();
    }
    uint32_t nc = 0;  // tiles consumed
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
        // the query rows as MMA columns: this thread loads row 8 nb + r0, and keeps
        // the sums of rows 8 nb + 2 c2 + {0, 1}: column 2 nb + {0, 1}
        uint32_t qf[NB][CH][2];
        float sl[2 * NB], m[2 * NB], up[2 * NB], L[2 * NB];  // o in units of 2^(m - up), L of 2^m
        int lim[2 * NB], low[2 * NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int ri = min(8 * nb + r0, nrows - 1), tq = ri / a.group, hq = ri - tq * a.group;
            const T* q = (const T*)a.q + (e.c0 + tq) * a.q_ts + (int64_t)(p.head * a.group + hq) * a.q_hs;
            Pack<T, 4> v[CH];
#pragma unroll
            for (int ch = 0; ch < CH; ++ch) v[ch] = *reinterpret_cast<const Pack<T, 4>*>(q + 16 * ch + 4 * c2);
            float top = 0.f;
#pragma unroll
            for (int ch = 0; ch < CH; ++ch)
#pragma unroll
                for (int k = 0; k < 4; ++k) top = fmaxf(top, fabsf(to_f(v[ch].v[k])));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float unit_q = row_unit(top);
#pragma unroll
            for (int ch = 0; ch < CH; ++ch) {
                qf[nb][ch][0] = pack_half2(to_f(v[ch].v[0]) * unit_q, to_f(v[ch].v[1]) * unit_q);
                qf[nb][ch][1] = pack_half2(to_f(v[ch].v[2]) * unit_q, to_f(v[ch].v[3]) * unit_q);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int u = 2 * nb + j, r = min(8 * nb + 2 * c2 + j, nrows - 1);
                const int pos = e.len - e.qn + r / a.group;
                sl[u] = a.scale_log2 / __shfl_sync(0xffffffffu, unit_q, 4 * (2 * c2 + j));
                lim[u] = kLean ? pos : a.causal ? min(pos, e.len - 1) : e.len - 1;
                low[u] = below_window(a, pos);
                m[u] = kNoKey;
                up[u] = 0.f;
                L[u] = 0.f;
            }
        }
        // keys below `clear` and above `low_any` need no mask for any row
        const int clear = a.causal ? min(e.len - e.qn, e.len - 1) : e.len - 1;
        const int low_any = below_window(a, e.len - 1);
        float o[NB][CH][4];  // coordinates 16 ch + 2 r0 + {0, 1} of the columns {0, 1}: [coordinate][column]
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[nb][i][k] = 0.f;

        for (int t = t_begin; t < t_end; ++t) {
            const int key0 = (p.s.tile0 + t) * kTile;
            produce();
            const int stage = nc % NS;
            if (!mbar_wait(&sm.full[warp][stage], (nc / NS) & 1, abort, kWaitNs)) ok = false;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ++nc;
            const float4 sc = *reinterpret_cast<const float4*>(sm.scale[warp][stage]);
            // ---- logits: 2 blocks of 16 keys; s[..][k]: key r0 + 8 (k / 2), column k & 1
            float s[NB][2][4];
            const uint32_t kb = smem_u32(ws.k[stage]);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[nb][b][k] = 0.f;
#pragma unroll
                for (int c = 0; c < CH; c += 2) {
                    uint32_t w[4];  // keys 0-7 | 8-15 of chunk c, then of chunk c + 1
                    ldsm4(kb + swz<D>(16 * b + 8 * (lmat & 1) + lrow, c + (lmat >> 1)), w);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t f[4];
                        codes_to_half<FMT>(w[2 * h], f[0], f[2]);
                        codes_to_half<FMT>(w[2 * h + 1], f[1], f[3]);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) mma16816(s[nb][b], f, qf[nb][c + h][0], qf[nb][c + h][1]);
                    }
                }
            }
            const bool masked = key0 + kTile - 1 > clear || key0 <= low_any || sc.x == -INFINITY ||
                                sc.y == -INFINITY;
            const float vs[2] = {sc.z, sc.w}, es[2] = {scale_exp(sc.z), scale_exp(sc.w)};
            float top[2 * NB];  // the largest logits
            bool grown = false;
            const float room = kRoom - fmaxf(es[0], es[1]);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                top[2 * nb] = top[2 * nb + 1] = -INFINITY;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const float ks = b == 0 ? sc.x : sc.y;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int u = 2 * nb + (k & 1);
                        float l = s[nb][b][k] * (sl[u] * ks);
                        if (masked) {
                            const int key = key0 + 16 * b + r0 + 8 * (k >> 1);
                            const bool hidden = kLean ? key >= e.len || (a.causal && key > lim[u]) ||
                                                            key <= below_window(a, lim[u])
                                                      : key > lim[u] || key <= low[u];
                            if (hidden || ks == -INFINITY) l = -INFINITY;
                        }
                        s[nb][b][k] = l;
                        top[u] = fmaxf(top[u], l);
                    }
                }
#pragma unroll
                for (int u = 2 * nb; u < 2 * nb + 2; ++u) {
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) top[u] = fmaxf(top[u], __shfl_xor_sync(0xffffffffu, top[u], x));
                    const float d = top[u] - m[u];
                    grown |= (d > kGrow) | (d + up[u] > room);
                }
            }
            if (__any_sync(0xffffffffu, grown)) {  // units follow, and the sums in them
#pragma unroll
                for (int u = 0; u < 2 * NB; ++u) {
                    const float m0 = m[u];
                    if (top[u] - m0 > kGrow) m[u] = ceilf(top[u]);
                    float topv = top[u] - m[u] + es[0];
                    if (es[0] != es[1]) {  // (the same in all tiles that one page holds)
                        topv = -INFINITY;
#pragma unroll
                        for (int b = 0; b < 2; ++b)
                            topv = fmaxf(topv, fmaxf(s[u >> 1][b][u & 1], s[u >> 1][b][2 + (u & 1)]) - m[u] + es[b]);
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) topv = fmaxf(topv, __shfl_xor_sync(0xffffffffu, topv, x));
                    }
                    const float follow = up[u] + (m[u] - m0);
                    up[u] = new_up(follow, topv, kStart);
                    L[u] *= ex2(m0 - m[u]);
                    const float f = ex2(up[u] - follow);
#pragma unroll
                    for (int i = 0; i < CH; ++i) {
                        o[u >> 1][i][u & 1] *= f;
                        o[u >> 1][i][2 + (u & 1)] *= f;
                    }
                }
            }
            uint32_t pf[NB][2][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const float2 lift = make_float2(pow2(up[2 * nb]), pow2(up[2 * nb + 1]));
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    float2 pr[2], l2 = make_float2(L[2 * nb], L[2 * nb + 1]);
                    const float2 mm = make_float2(-m[2 * nb], -m[2 * nb + 1]);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        pr[k] = __fadd2_rn(make_float2(s[nb][b][2 * k], s[nb][b][2 * k + 1]), mm);
                        pr[k].x = ex2(pr[k].x);
                        pr[k].y = ex2(pr[k].y);
                        l2 = __fadd2_rn(l2, pr[k]);
                        // (the scale last: a hidden page's may be anything, and meets zeros)
                        pr[k] = __fmul2_rn(__fmul2_rn(pr[k], lift), make_float2(vs[b], vs[b]));
                        // keys x columns, transposed into the B operand
                        pf[nb][b][k] = movm(pack_half2(pr[k].x, pr[k].y));
                    }
                    L[2 * nb] = l2.x;
                    L[2 * nb + 1] = l2.y;
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
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int c = 0; c < CH; c += 2) {
                    uint32_t x[4];  // keys 0-7 | 8-15 of chunk c, then of chunk c + 1
                    ldsm4t(vb + swz<D>(16 * b + 8 * (lmat & 1) + lrow, c + (lmat >> 1)), x);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t f[4];  // even coordinates, odd ones; the same of keys 8-15
                        codes_to_half_02<FMT>(x[2 * h], f[0], f[1]);
                        codes_to_half_02<FMT>(x[2 * h + 1], f[2], f[3]);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) mma16816(o[nb][c + h], f, pf[nb][b][0], pf[nb][b][1]);
                    }
                }
            }
            __syncwarp();  // every lane is done with the stage
        }
        if (!ok) break;
        const bool begins = t_begin == 0, ends = t_end == p.s.tiles;
        // where a part goes: units first .. last share the item
        const int64_t block0 = (int64_t)blockIdx.x * busy;
        int64_t first = block0, last = block0 + busy - 1;
        if (!by_item && !(begins && ends)) {
            const int64_t start = g - t_begin;
            first = begins ? unit : owner(start);
            last = ends ? unit : owner(start + p.s.tiles - 1);
        }
        const bool in_ring = g + (t_end - t_begin) == g1;  // nothing more comes into the ring
        float2* part_ml = in_ring ? sm.ml[warp] : parts.ml + (int64_t)self * kRows;
        float* part_o = in_ring ? reinterpret_cast<float*>(&ws) : parts.o + (int64_t)self * kRows * D;
#pragma unroll
        for (int u = 0; u < 2 * NB; ++u) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) L[u] += __shfl_xor_sync(0xffffffffu, L[u], x);
            const int r = 8 * (u >> 1) + 2 * c2 + (u & 1), j = u & 1, nb = u >> 1;
            if (r >= nrows) continue;
            const float size = pow2(-up[u]);
            if (begins && ends) {
                const int64_t tok = e.c0 + r / a.group;
                const int hq = p.head * a.group + r % a.group;
                const float n = L[u] > 0.f ? 1.f / L[u] : (L[u] == 0.f ? 0.f : L[u]);
                T* out = (T*)a.out + (tok * a.heads_q + hq) * D + 2 * r0;
#pragma unroll
                for (int ch = 0; ch < CH; ++ch) {
                    Pack<T, 2> v;
                    from_f(o[nb][ch][j] * size * n, v.v[0]);
                    from_f(o[nb][ch][2 + j] * size * n, v.v[1]);
                    *reinterpret_cast<Pack<T, 2>*>(out + 16 * ch) = v;
                }
                if (a.lse && r0 == 0)
                    a.lse[tok * a.heads_q + hq] =
                        L[u] > 0.f ? (m[u] + log2f(L[u])) * 0.69314718056f : L[u] == 0.f ? -INFINITY : L[u];
            } else {
                if (r0 == 0) part_ml[r] = make_float2(m[u], L[u]);
                float* dst = part_o + r * D + 2 * r0;
#pragma unroll
                for (int ch = 0; ch < CH; ++ch)
                    *reinterpret_cast<float2*>(dst + 16 * ch) =
                        make_float2(o[nb][ch][j] * size, o[nb][ch][2 + j] * size);
            }
        }
        if (lane == 0 && !(begins && ends)) {
            const int64_t block1 = block0 + busy;  // behind the block's units
            if (begins || (warp == 0 && g == g0)) {
                Job job;
                job.first = first;
                job.parts = (int)(min(last, block1 - 1) - max(first, block0) + 1);
                job.rows = nrows;
                job.head = p.head;
                job.row0 = e.c0 * a.group;
                job.begins = first >= block0;
                job.ends = last < block1;
                sm.job[begins ? warp : kWarps] = job;
            }
            if (!in_ring) sm.outside[warp] = 1;
            if (last >= block1 && warp == busy - 1) sm.beyond = 1;
        }
        g += t_end - t_begin;
        if (g < g1) {
            p.t = p.s.tiles - 1;
            advance(p);
        }
    }
    if (!ok) {
        // gave up: no copy into this warp's ring may land after it has left
        *abort = 1;
        int none = 0;
        for (; nc < np; ++nc) mbar_wait(&sm.full[warp][nc % NS], (nc / NS) & 1, &none, kWaitNs);
    }
    __syncthreads();

    // ---- joining: the block's parts, a warp a row
    uint32_t jobs = __ballot_sync(0xffffffffu, lane <= kWarps && sm.job[min(lane, kWarps)].parts > 0);
    bool across = false;
    for (int at = 0; jobs; jobs &= jobs - 1) {
        const int which = __ffs(jobs) - 1, w0 = which % kWarps;
        const Job& job = sm.job[which];
        const int n = job.parts, tail = w0 + n - 1;
        // the last part may lie in the workspace (but not where its warp began the item)
        const bool outside = sm.outside[tail] && (n > 1 || !job.begins);
        const int64_t far = ((int64_t)blockIdx.x * kWarps + tail) * kRows;
        const bool whole = job.begins && job.ends;
        across |= !whole;
        for (int r = (warp + kWarps - at) % kWarps; r < job.rows; r += kWarps) {
            const Sum<D> s = sum_parts<D>(
                n, 0, 1, lane,
                [&](int j) { return outside && j == n - 1 ? parts.ml[far + r] : sm.ml[w0 + j][r]; },
                [&](int j) -> const float* {
                    return outside && j == n - 1 ? parts.o + (far + r) * D
                                                 : reinterpret_cast<const float*>(&sm.w[w0 + j]) + r * D;
                });
            if (whole) {
                write_row<D, T>(a, job, r, s, lane);
            } else {
                const int64_t to = (block_slot(blockIdx.x) + (job.begins ? 1 : 0)) * kRows + r;
                if (lane == 0) parts.ml[to] = make_float2(s.m, s.L);
                float* dst = parts.o + to * D + lane * (D / 32);
#pragma unroll
                for (int k = 0; k < D / 32; ++k) dst[k] = s.acc[k];
            }
        }
        at = (at + job.rows) % kWarps;
    }
    if (across) {  // (the same for all warps)
        __syncthreads();
        if (threadIdx.x == 0 && sm.beyond) set_flag(&parts.flag[blockIdx.x], parts.nonce);
        const Job job = sm.job[kWarps];
        if (job.parts && job.ends) {  // an item of earlier blocks ends here
            const int b0 = (int)quot(job.first, busy), n = (int)blockIdx.x - b0 + 1;
            if (warp == 0) {
                const uint64_t t0 = globaltimer();
                bool all;
                do {
                    all = true;
                    for (int i = b0 + lane; i < (int)blockIdx.x; i += 32) all &= get_flag(&parts.flag[i]) == parts.nonce;
                    all = __all_sync(0xffffffffu, all);
                } while (!all && __all_sync(0xffffffffu, globaltimer() - t0 < kWaitNs));
                if (!all) sm.abort = 1;
                for (int i = b0 + lane; i < (int)blockIdx.x; i += 32) parts.flag[i] = 0;
            }
            __syncthreads();
            struct alignas(16) Row {  // acc is read 16 bytes at a time
                float acc[D], m, L;
            };
            static_assert(sizeof(Row) * kWarps <= sizeof(sm.w), "the rings hold the warps' sums");
            Row* rows = reinterpret_cast<Row*>(sm.w);
            const int per = max(1, kWarps / job.rows);  // warps that share a row
            for (int r0 = 0; r0 < job.rows && !sm.abort; r0 += kWarps / per) {
                const int r = r0 + warp / per, sub = warp % per;
                const bool mine = warp / per < kWarps / per && r < job.rows;
                auto at = [&](int i) { return (block_slot(b0 + i) + (i == 0 ? 1 : 0)) * kRows + r; };
                Sum<D> s;
                if (mine)
                    s = sum_parts<D>(
                        n, sub, per, lane, [&](int i) { return __ldcg(&parts.ml[at(i)]); },
                        [&](int i) -> const float* { return parts.o + at(i) * D; });
                if (per > 1) {
                    if (mine) {
                        if (lane == 0) {
                            rows[warp].m = s.m;
                            rows[warp].L = s.L;
                        }
#pragma unroll
                        for (int k = 0; k < D / 32; ++k) rows[warp].acc[lane * (D / 32) + k] = s.acc[k];
                    }
                    __syncthreads();
                    if (mine && sub == 0)
                        s = sum_parts<D>(
                            per, 0, 1, lane, [&](int i) { return make_float2(rows[warp + i].m, rows[warp + i].L); },
                            [&](int i) -> const float* { return rows[warp + i].acc; });
                    __syncthreads();
                }
                if (mine && sub == 0) write_row<D, T>(a, job, r, s, lane);
            }
        }
    }
    if (sm.used < a.total_q) zero_behind<D, T>(a, sm.used);
    if (threadIdx.x == 0 && sm.abort) {
        *parts.status = TQ_ERR_DEVICE_TIMEOUT * 1000 - 80;
        leave_status(a.v, TQ_ERR_DEVICE_TIMEOUT * 1000 - 80);
    }
}

constexpr int kMaxBlocks = 148;  // the workspace's size
constexpr float kLog2e = 1.44269504089f;

// The most steps that a call of these sizes can have (its lengths lie on the
// device); blocks: one an SM, fewer where the tables are too short to fill them.
int64_t blocks_for(const tq_kv8_t* c, int ns) {
    const int64_t steps = ((int64_t)c->max_pages * c->page + kTile - 1) / kTile * ns * c->heads;
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
    Parts p = {};
    char* at = (char*)ws;
    p.status = (int*)at;
    at += 256;
    p.flag = (uint64_t*)at;
    at += align256(blocks * 8);
    p.ml = (float2*)at;
    at += align256((units + 2 * blocks) * kRows * sizeof(float2));
    p.o = (float*)at;
    at += align256((units + 2 * blocks) * kRows * D * 4);
    *bytes = (size_t)(at - (char*)ws);
    return p;
}

template <int FMT, int D, int NB, typename T>
int launch(const Attn& a, const CUtensorMap& km, const CUtensorMap& vm, const Parts& p, int blocks,
           cudaStream_t s) {
    constexpr int smem = (int)sizeof(Smem<D>) + 1024;
    static_assert(smem <= 232448, "shared memory of a block");
    int rc = allow_smem<k_attn_rows<FMT, D, NB, T>>(smem);
    return rc ? rc : launch_behind(k_attn_rows<FMT, D, NB, T>, dim3(blocks), kThreads, smem, s, a, km, vm, p);
}

template <int FMT, int D, typename T>
int launch_rows(const Attn& a, const CUtensorMap& km, const CUtensorMap& vm, const Parts& p, int blocks,
                int rows, cudaStream_t s) {
    return rows <= 8 ? launch<FMT, D, 1, T>(a, km, vm, p, blocks, s)
                     : launch<FMT, D, 2, T>(a, km, vm, p, blocks, s);
}

template <int D>
int dispatch(const tq_kv8_t* c, const Attn& a, const CUtensorMap& km, const CUtensorMap& vm,
             const Parts& p, int blocks, int rows, int q_dtype, cudaStream_t s) {
    if (c->format == TQ_KV_I8)
        return q_dtype == TQ_BF16 ? launch_rows<TQ_KV_I8, D, __nv_bfloat16>(a, km, vm, p, blocks, rows, s)
                                  : launch_rows<TQ_KV_I8, D, __half>(a, km, vm, p, blocks, rows, s);
    return q_dtype == TQ_BF16 ? launch_rows<TQ_KV_E4M3, D, __nv_bfloat16>(a, km, vm, p, blocks, rows, s)
                              : launch_rows<TQ_KV_E4M3, D, __half>(a, km, vm, p, blocks, rows, s);
}

// A value that no earlier call has left in a workspace.
uint64_t new_nonce() {
    static std::atomic<uint64_t> next{
        (uint64_t)std::chrono::system_clock::now().time_since_epoch().count() * 0xD1342543DE82EF95ull ^
        (uint64_t)(uintptr_t)&next};
    const uint64_t x = next.fetch_add(0x9E3779B97F4A7C15ull);  // an odd step: all values in turn
    return x ? x : next.fetch_add(0x9E3779B97F4A7C15ull);      // (0: a flag that was taken back)
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
    return tq_kv8_attention_rows(c, layer, ns, d_slots, d_cu, total_q, max_q, heads_q, d_q, q_dtype, q_ts,
                                 q_hs, scale, causal, window, d_out, 0, d_lse, d_ws, ws_bytes, stream);
}

extern "C" int tq_kv8_attention_rows(const tq_kv8_t* c, int layer, int ns, const int32_t* d_slots,
                                     const int32_t* d_cu, int64_t total_q, int max_q, int heads_q,
                                     const void* d_q, int q_dtype, int64_t q_ts, int64_t q_hs, float scale,
                                     int causal, int window, void* d_out, int zero_behind, float* d_lse,
                                     void* d_ws, size_t ws_bytes, void* stream) {
    int status;
    if (!kv8::valid(c, &status)) return status;
    if (layer < 0 || layer >= c->layers || ns < 0 || total_q < 0 || max_q < 0 || heads_q < 1)
        return TQ_ERR_ARG;
    if (q_dtype != TQ_BF16 && q_dtype != TQ_F16) return TQ_ERR_ARG;
    if (causal < 0 || causal > 1 || window < 0 || (window > 0 && !causal) ||
        !std::isfinite(scale * kv8::kLog2e))
        return TQ_ERR_ARG;
    if (!d_slots && ns > c->slots) return TQ_ERR_ARG;
    if (heads_q % c->heads || heads_q / c->heads > 128) return TQ_ERR_UNSUPPORTED;
    // rows (tokens x group) count in 32 bits
    if (total_q > (((int64_t)1 << 31) - (1 << 16)) / (heads_q / c->heads)) return TQ_ERR_UNSUPPORTED;
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
    a.scale_log2 = scale * kv8::kLog2e;
    a.ks = c->d_kscale + layer * kv8::layer_scales(c);
    a.vs = c->d_vscale + layer * kv8::layer_scales(c);
    a.out = d_out;
    a.behind = zero_behind;
    a.lse = d_lse;
    a.rows = c->pages * c->heads * c->page;
    cudaStream_t s = (cudaStream_t)stream;
    const bool few = kv8::any_few(c, ns, total_q, max_q, heads_q);
    const int64_t most = (int64_t)max_q * a.group;
    a.max_q = kv8::any_many(c, max_q, heads_q) ? INT32_MAX : max_q;
    a.few = few ? (int)(most < kv8::kRows ? most : kv8::kRows) : 0;
    size_t at = 256;
    if (few) {
        const int box = c->page < kv8::kTile ? c->page : kv8::kTile;
        CUtensorMap km, vm;
        int rc = kv8::code_map(&km, (const char*)c->d_k + layer * kv8::layer_bytes(c), c->d, a.rows, box);
        if (!rc) rc = kv8::code_map(&vm, (const char*)c->d_v + layer * kv8::layer_bytes(c), c->d, a.rows, box);
        if (rc) return rc;
        const int blocks = (int)kv8::blocks_for(c, ns);
        kv8::Parts p = kv8::carve_for(c, d_ws, blocks, &at);
        p.nonce = kv8::new_nonce();
        rc = c->d == 128 ? kv8::dispatch<128>(c, a, km, vm, p, blocks, a.few, q_dtype, s)
                         : kv8::dispatch<64>(c, a, km, vm, p, blocks, a.few, q_dtype, s);
        if (rc) return rc;
    }
    if (!kv8::any_many(c, max_q, heads_q)) return TQ_OK;
    if (few) a.behind = 0;  // (done)
    size_t bytes;
    const int blocks = kv8::prompt_blocks(c, ns, total_q, heads_q);
    kv8::PromptParts p = kv8::prompt_carve(c, (char*)d_ws + at, blocks, &bytes);
    p.status = (int*)d_ws;
    p.keep_status = few;
    return kv8::launch_prompt(c, layer, a, p, blocks, q_dtype, s);
}
