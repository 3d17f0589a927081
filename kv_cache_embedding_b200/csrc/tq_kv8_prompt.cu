// Attention over the 8-bit paged cache, many query rows (prompts, chunks behind
// a prefix, drafts): the sums of tq_kv8_attention.cu on the sm_100a tensor cores.
//
//   S = Q C_k^T   (rows x 128 keys),   P = 2^(S s_k s_q - m),   O += (P s_v 2^u) C_v
//
// with the codes C as exact halves, Q a row of halves times a power of two, s_k
// and s_v one number per 16 keys (a page at least).  m and u are the row's own: whole
// numbers by which the largest P of the keys that it sees is near 1, and the largest
// P s_v 2^u, which is rounded to a half (2^-11), at 2^5 at least: what is smaller than
// halves' normal range is off by 2^-30 of that one, and no page that the row does not
// see has a part in it.  Sums are fp32.
//
// A CTA runs items of 256 rows (two stages of 128) of one entry and KV head over
// tiles of 128 keys; the steps (item x tile) of the whole batch are shared out
// evenly, contiguously, over one CTA an SM, so ragged and causal batches balance
// and a long context with few rows fills the machine; the items that are cut are
// joined by k_prompt_merge.  Warps:
//   0-3, 4-7  softmax of stage 0, 1: a thread a row, half a tile (64 keys) at a time.
//             Loads its query row, turns S (tensor memory) into P in place, rescales
//             O only when the row's largest product has grown by more than 2^8 (u then
//             follows; the product is below 2^15 meanwhile, inside a half's range),
//             writes the result.
//   8-11      codes -> halves: from the TMA ring (128 keys x d bytes) into the
//             swizzled operand tiles of K (K-major) and V (the same rows, read
//             MN-major), with the tile's scales.
//   12, 15    issue the MMAs of stage 0, 1: per half O += P V, then S of the half
//             two further, so the softmax finds its next S complete.
//   13        the TMA loads, a page table lookup a box, a tile ahead.
//   14        walks the CTA's share and hands the others its items through a short
//             ring: lengths, divisions and lookups are off their path.
// Every wait is bounded (1 s); a warp that gives up sets the abort flag and the
// call's status.
//
// Measured (4096 tokens x 32 heads of 128 over 16384 keys, causal): 1055 us, 911
// TFLOP/s.  Latency bounds it: two stages' half tiles are some 1000 cycles of
// exponentials and 1000 of MMAs and take 2100, with half of the issue slots and 43 % of
// the tensor pipe in use; one softmax warp a scheduler and stage runs a chain S ->
// maximum -> exponentials -> P.  Tried and slower: a quarter or half of the exponentials
// as polynomials on the FMA pipe (1087 and 1181 us against 1040), whole tiles (1101),
// one warp for both stages' MMAs (1189).
#include "tq_kv8_attention.cuh"
#include "tq_score_common.cuh"

namespace tq {
namespace kv8 {

using namespace sm100;
using sc::ffma2;

namespace {

constexpr int kPT = 128;            // keys a tile
constexpr int kPH = 64;             // keys a half of a tile: what a stage works on at a time
constexpr int kPM = 128;            // rows a stage
constexpr int kPRows = 2 * kPM;     // rows an item
constexpr int kPThreads = 512;
constexpr int kGroups = kPT / 16;   // scale groups of a tile
constexpr int kRing = 4;            // tiles whose scales are kept
constexpr int kWorks = 4;           // items that are handed out ahead
constexpr uint32_t kTmemCols = 512;
constexpr float kStart = 6.f;       // a row's largest product: at 2^(kStart - 1) at least

// A CTA's piece of an item, as the warps get it.
struct Work {
    int slot, len, head;
    int pos0;         // position of the entry's first query: len - its queries
    int row0, rows;   // first of the item's rows (token x group), their number; 0: no more work
    int t0, t, t_end, nt;  // first tile of the item; the CTA's tiles t .. t_end of its nt
    int parts;        // CTAs that hold the item, where it begins here and goes on
    int64_t c0;       // the entry's first query token
};

template <int D>
struct PSmem {
    uint8_t q[2][kPM * D * 2];    // stages' queries: 64-coordinate blocks of 128 rows x 128 B
    uint8_t kv[4][kPT * D * 2];   // K of even, odd tiles, V of even, odd tiles
    uint8_t raw[2][kPT * D];      // codes as they arrive: K, V
    float kscale[kRing][kGroups], vscale[kRing][kGroups], vexp[kRing][kGroups];  // s_k, s_v, its exponent
    uint32_t absent[kRing];       // 16-key groups without a page
    Work work[kWorks];
    uint64_t raw_full[2], raw_empty[2], kv_full[4], kv_empty[4];
    uint64_t q_full[2], s_full[2][2], p_full[2][2], o_done[2][2], mma_done[2];  // [stage][half]
    uint64_t work_full[kWorks], work_empty[kWorks];
    uint32_t tmem_base;
    int abort;
};

// (rows of a call, tokens x group, count in 32 bits)
__device__ __forceinline__ int parts_of(const Attn& a, const Entry& e) {
    const int rows = e.qn * a.group;
    return rows > a.few ? (rows + kPRows - 1) / kPRows : 0;
}
// First tile and number of tiles of a part (one at least: rows without keys are
// written too).
__device__ __forceinline__ void tiles_of(const Attn& a, const Entry& e, int part, int& t0, int& nt) {
    const int first = (unsigned)(part * kPRows) / (unsigned)a.group;
    const int last = min(e.qn - 1, (int)(((unsigned)(part + 1) * kPRows - 1) / (unsigned)a.group));
    const int end = a.causal ? min(e.len, e.len - e.qn + last + 1) : e.len;
    const int beg = below_window(a, e.len - e.qn + first) + 1;
    t0 = beg / kPT;
    nt = max(1, (end + kPT - 1) / kPT - t0);
}
// Tiles of all parts of a head: part i, i + step, ..
__device__ __forceinline__ int64_t tiles_per_head(const Attn& a, const Entry& e, int i, int step) {
    int64_t n = 0;
    for (const int m = parts_of(a, e); i < m; i += step) {
        int t0, nt;
        tiles_of(a, e, i, t0, nt);
        n += nt;
    }
    return n;
}
__device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// Bits 0 .. n (none for n < 0).
__device__ __forceinline__ uint32_t first_bits(int n) {
    return n < 0 ? 0u : n >= 31 ? 0xFFFFFFFFu : (2u << n) - 1u;
}
__device__ __forceinline__ float max16(const uint32_t* s) {
    auto f = [&](int i) { return __uint_as_float(s[i]); };
    const float a = max3(max3(f(0), f(1), f(2)), f(3), f(4)), b = max3(max3(f(5), f(6), f(7)), f(8), f(9));
    return max3(max3(a, f(10), f(11)), max3(b, f(12), f(13)), fmaxf(f(14), f(15)));
}

template <int FMT, int D, typename T>
__global__ __launch_bounds__(kPThreads, 1) void k_attn_prompt(const Attn a,
                                                              const __grid_constant__ CUtensorMap kmap,
                                                              const __grid_constant__ CUtensorMap vmap,
                                                              const PromptParts parts) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    PSmem<D>& sm = *reinterpret_cast<PSmem<D>*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
    constexpr int CH = D / 16;   // 16-code chunks of a row
    constexpr uint32_t kBlock = kPM * 128;  // bytes of such a block
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort = &sm.abort;
    const int unit = blockIdx.x;
    grid_begin();

    // ---- the batch's steps: a run of entries a thread (few entries: a warp an
    // entry), prefix over the block
    int64_t* pre = reinterpret_cast<int64_t*>(sm.kv);  // (before the operands are)
    const int run = (a.ns + kPThreads - 1) / kPThreads;
    {
        int64_t mine = 0;
        bool bad = false;
        if (a.ns <= 32) {
            for (int i = warp; i < a.ns; i += kPThreads / 32) {
                const Entry e = entry_of(a, i);
                bad |= misfit(a, i, e);
                const int64_t n = warp_sum(tiles_per_head(a, e, lane, 32));
                if (lane == 0) pre[kPThreads + 1 + i] = a.v.heads * n;
            }
            __syncthreads();
            if ((int)threadIdx.x < a.ns) mine = pre[kPThreads + 1 + threadIdx.x];
        } else {
            for (int i = threadIdx.x * run; i < min(a.ns, (int)(threadIdx.x + 1) * run); ++i) {
                const Entry e = entry_of(a, i);
                bad |= misfit(a, i, e);
                mine += a.v.heads * tiles_per_head(a, e, 0, 1);
            }
        }
        if (threadIdx.x == 0) {
            sm.abort = 0;
            for (int i = 0; i < 2; ++i) {
                mbar_init(&sm.raw_full[i], 1);
                mbar_init(&sm.raw_empty[i], 4);
                mbar_init(&sm.q_full[i], 4);
                for (int h = 0; h < 2; ++h) {
                    mbar_init(&sm.s_full[i][h], 1);
                    mbar_init(&sm.p_full[i][h], 4);
                    mbar_init(&sm.o_done[i][h], 1);
                }
            }
            for (int i = 0; i < 4; ++i) {
                mbar_init(&sm.kv_full[i], 4);
                mbar_init(&sm.kv_empty[i], 2);
            }
            for (int i = 0; i < kWorks; ++i) {
                mbar_init(&sm.work_full[i], 1);
                mbar_init(&sm.work_empty[i], 15);  // all warps but the one that fills it
            }
            mbar_init(&sm.mma_done[0], 1);
            mbar_init(&sm.mma_done[1], 1);
            fence_mbar_init();
            prefetch_tmap(&kmap);
            prefetch_tmap(&vmap);
            parts.cut[unit].parts = 0;
        }
        int64_t inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        int64_t* sums = pre + kPThreads + 40;
        if (lane == 31) sums[warp] = inc;
        bad = __syncthreads_or(bad);
        if (__syncthreads_or(bad || (threadIdx.x == 0 && pending(a.v)))) {  // (k_prompt_merge writes the rows)
            if (threadIdx.x == 0) parts.block_status[unit] = bad ? TQ_ERR_ARG : 0;
            return;
        }
        for (int w = 0; w < warp; ++w) inc += sums[w];
        pre[threadIdx.x + 1] = inc;
        if (threadIdx.x == 0) pre[0] = 0;
        __syncthreads();
    }
    // the first `rest` CTAs take base + 1 steps, the others base
    const int64_t total = pre[kPThreads];
    const int units = (int)min((int64_t)gridDim.x, total);
    const int64_t base = units ? quot(total, units) : 0, rest = total - base * units;
    const int64_t g0 = unit < units ? unit * base + min((int64_t)unit, rest) : 0;
    const int64_t g1 = unit < units ? g0 + base + (unit < rest ? 1 : 0) : 0;
    int entry = 0;
    int64_t rem = 0;  // step g0 is step `rem` of entry `entry` and those behind it
    if (warp == 14 && g0 < g1) {
        int lo = 0, hi = (a.ns + run - 1) / run;  // the run of entries that holds step g0
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] <= g0) lo = mid;
            else hi = mid;
        }
        rem = g0 - pre[lo];
        entry = lo * run;
    }
    if (warp == 12) {
        tmem_alloc(&sm.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();  // also: nobody reads `pre` any more
    tc_fence_after();
    const uint32_t tbase = sm.tmem_base;

    auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool ok = mbar_wait(bar, parity, abort, kWaitNs);
        if (!__all_sync(0xffffffffu, ok)) {
            *abort = 1;
            return false;
        }
        return true;
    };

    // the n-th piece of work
    auto get = [&](uint32_t n) { return wait(&sm.work_full[n % kWorks], n / kWorks & 1); };
    auto done_with = [&](uint32_t n) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.work_empty[n % kWorks]);
    };

    if (warp < 8) {
        // ================================================== softmax, a row a thread
        const int st = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lane_addr = tbase + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t o_col = lane_addr + 2 * kPT + st * D;
        uint32_t tile = 0, halves = 0;  // tiles so far; halves of tiles that this stage has seen
        bool ok = true;
        for (uint32_t n = 0; ok && (ok = get(n)); ++n) {
            const Work& w = sm.work[n % kWorks];
            if (w.rows == 0) break;
            const int t_begin = w.t, t_end = w.t_end;
            if (st * kPM >= w.rows) {  // the item has one stage
                tile += t_end - t_begin;
                done_with(n);
                continue;
            }
            const bool valid = st * kPM + row < w.rows;
            const unsigned ri = w.row0 + (valid ? st * kPM + row : 0);
            const int tq = ri / (unsigned)a.group, hq = w.head * a.group + (int)(ri - tq * a.group);
            const int64_t tok = w.c0 + tq;
            // ---- the query row, as halves
            float sl;
            {
                const T* q = (const T*)a.q + tok * a.q_ts + (int64_t)hq * a.q_hs;
                Pack<T, 8> x[D / 8];
                float top = 0.f;
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    if (valid) {
                        x[c] = *reinterpret_cast<const Pack<T, 8>*>(q + 8 * c);
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k) from_f(0.f, x[c].v[k]);
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(to_f(x[c].v[k])));
                }
                // (a negative scale turns the row's sign, so that the factor of S is >= 0)
                const float unit_q = row_unit(top);
                const float f = a.scale_log2 < 0.f ? -unit_q : unit_q;
                sl = fabsf(a.scale_log2) / unit_q;
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    uint4 o;
                    o.x = half2_bits(to_f(x[c].v[0]) * f, to_f(x[c].v[1]) * f);
                    o.y = half2_bits(to_f(x[c].v[2]) * f, to_f(x[c].v[3]) * f);
                    o.z = half2_bits(to_f(x[c].v[4]) * f, to_f(x[c].v[5]) * f);
                    o.w = half2_bits(to_f(x[c].v[6]) * f, to_f(x[c].v[7]) * f);
                    *reinterpret_cast<uint4*>(sm.q[st] + (c >> 3) * kBlock + row * 128 +
                                              (((c & 7) ^ (row & 7)) << 4)) = o;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.q_full[st]);
            }
            const int pos = w.pos0 + tq, len = w.len;
            const int lim = valid && a.causal ? min(pos, len - 1) : len - 1;
            const int low = valid ? below_window(a, pos) : -1;
            // L is in units of 2^m, O of 2^(m - up), lift is 2^up
            float m = kNoKey, up = 0.f, lift = 1.f;
            float2 L2 = make_float2(0.f, 0.f);
            const uint32_t first = halves, last = halves + 2 * (t_end - t_begin);
            for (int key0 = (w.t0 + t_begin) * kPT; halves < last; key0 += kPH) {
                const int h = halves & 1, rg = (tile + ((halves - first) >> 1)) & (kRing - 1);
                const uint32_t s_col = lane_addr + st * kPT + h * kPH;
                if (!wait(&sm.s_full[st][h], halves >> 1 & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t s[2][32];
                tmem_ld32(s_col, s[0]);
                float cg[4], tg[4];  // of 16 keys: the factor of S, the largest logit
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    cg[g] = sl * sm.kscale[rg][4 * h + g];
                    tg[g] = -INFINITY;
                }
                const uint32_t absent = sm.absent[rg] >> 4 * h & 15u;
                // a half tile that a mask touches, or with rows whose logits may pass 2^22
                // (rows that are not finite aside): there logits are rounded before m is taken
                // off.  What the fused product of the other way keeps of such would be whole
                // units
                const float most = fmaxf(max3(cg[0], cg[1], cg[2]), cg[3]);
                const bool far = most > 4194304.f / (65536.f * code_max<FMT>() * D) && most < 1e25f;
                const bool masked = __any_sync(0xffffffffu, key0 + kPH - 1 > lim || key0 <= low || absent || far);
                // 32 keys are on their way while the 32 before them are looked at
                if (masked) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        tmem_wait_ld();
                        if (c < 1) tmem_ld32(s_col + 32, s[1]);
                        // the keys that the row sees, a bit each
                        const uint32_t see = first_bits(lim - (key0 + 32 * c)) & ~first_bits(low - (key0 + 32 * c)) &
                                             ~((absent >> 2 * c & 1u) * 0xFFFFu | (absent >> (2 * c + 1) & 1u) * 0xFFFF0000u);
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float x = see >> i & 1u ? __uint_as_float(s[c][i]) * cg[2 * c + i / 16] : -INFINITY;
                            s[c][i] = __float_as_uint(x);
                            tg[2 * c + i / 16] = fmaxf(tg[2 * c + i / 16], x);
                        }
                    }
#pragma unroll
                    for (int g = 0; g < 4; ++g) cg[g] = 1.f;
                } else {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        tmem_wait_ld();
                        if (c < 1) tmem_ld32(s_col + 32, s[1]);
                        tg[2 * c] = max16(&s[c][0]) * cg[2 * c];
                        tg[2 * c + 1] = max16(&s[c][16]) * cg[2 * c + 1];
                    }
                }
                // the references follow when what they are of has grown out of their range.
                // (All relative to m: logits may be so large that their last bits are whole
                // units.  The first test takes every key for one of the largest scale.)
                const float* ve = &sm.vexp[rg][4 * h];
                const float room = kRoom - fmaxf(max3(ve[0], ve[1], ve[2]), ve[3]);
                const float top = fmaxf(max3(tg[0], tg[1], tg[2]), tg[3]), d = top - m;
                float shrink = 1.f;
                if ((d > kGrow) | (d + up > room)) {
                    const float m0 = m;
                    m = fmaxf(m, ceilf(top));
                    const float topv =
                        fmaxf(max3(tg[0] - m + ve[0], tg[1] - m + ve[1], tg[2] - m + ve[2]), tg[3] - m + ve[3]);
                    const float f = ex2(m0 - m), follow = up + (m - m0);
                    L2.x *= f;
                    L2.y *= f;
                    up = new_up(follow, topv, kStart);
                    lift = pow2(up);
                    shrink = ex2(up - follow);
                }
                if (halves > first && __any_sync(0xffffffffu, shrink != 1.f)) {
                    // O holds all halves before this one when the last one's MMAs are done
                    if (!wait(&sm.o_done[st][(halves - 1) & 1], ((halves - 1) >> 1) & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t o[16];
                        tmem_ld16(o_col + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * shrink);
                        tmem_st16(o_col + c, o);
                    }
                }
                const float base = -m;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t p[16];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int g = 2 * c + k;
                        // (a hidden page's may be anything: it meets zeros)
                        const float vw = fminf(sm.vscale[rg][4 * h + g] * lift, kLargestFloat);
                        const float2 cc = make_float2(cg[g], cg[g]), bb = make_float2(base, base);
                        const float2 ww = make_float2(vw, vw);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float2 x = make_float2(__uint_as_float(s[c][16 * k + 2 * i]),
                                                   __uint_as_float(s[c][16 * k + 2 * i + 1]));
                            x = ffma2(x, cc, bb);
                            x.x = ex2(x.x);
                            x.y = ex2(x.y);
                            L2 = __fadd2_rn(L2, x);
                            x = __fmul2_rn(x, ww);
                            p[8 * k + i] = half2_bits(x.x, x.y);
                        }
                    }
                    tmem_st16(s_col + 16 * c, p);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_full[st][h]);
                ++halves;
            }
            tile += t_end - t_begin;
            for (int h = 0; h < 2; ++h) ok = ok && wait(&sm.o_done[st][h], ((halves - 1) >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            const float L = L2.x + L2.y;
            const bool begins = t_begin == 0, ends = t_end == w.nt;
            const float size = 1.f / lift;
            if (begins && ends) {
                const float f = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
                T* out = (T*)a.out + (tok * a.heads_q + hq) * D;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(o_col + c, o);
                    tmem_wait_ld();
                    if (valid) {
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            Pack<T, 8> y;
#pragma unroll
                            for (int k = 0; k < 8; ++k) from_f(__uint_as_float(o[8 * h + k]) * size * f, y.v[k]);
                            *reinterpret_cast<Pack<T, 8>*>(out + c + 8 * h) = y;
                        }
                    }
                }
                if (a.lse && valid)
                    a.lse[tok * a.heads_q + hq] = L > 0.f ? (m + log2f(L)) * 0.69314718056f : (L == 0.f ? -INFINITY : L);
            } else {
                const int64_t slot = 2 * (int64_t)unit + (begins ? 1 : 0);
                const int64_t pr = slot * kPRows + st * kPM + row;
                if (valid) parts.ml[pr] = make_float2(m, L);
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(o_col + c, o);
                    tmem_wait_ld();
                    if (valid) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            *reinterpret_cast<float4*>(parts.o + pr * D + c + k) =
                                make_float4(__uint_as_float(o[k]) * size, __uint_as_float(o[k + 1]) * size,
                                            __uint_as_float(o[k + 2]) * size, __uint_as_float(o[k + 3]) * size);
                    }
                }
                if (begins && st == 0 && row == 0) {
                    Cut c;
                    c.parts = w.parts;
                    c.rows = w.rows;
                    c.head = w.head;
                    c.pad = 0;
                    c.row0 = w.c0 * a.group + w.row0;
                    parts.cut[unit] = c;
                }
            }
            tc_fence_before();  // O is read before the next item's MMAs write it
            done_with(n);
        }
    } else {
        if (warp < 12) {
            // ============================================== codes -> halves
            const int tid = threadIdx.x - 256;
            uint32_t tile = 0, n_raw = 0;
            bool ok = true;
            for (uint32_t n = 0; ok && (ok = get(n)); ++n) {
                const Work& w = sm.work[n % kWorks];
                if (w.rows == 0) break;
                const int t_end = w.t_end, len = w.len, slot = w.slot, head = w.head, tile0 = w.t0;
                // thread g < 8: s_k of the next tile's 16-key group g; 8..15: s_v; NaN: no page
                auto load_scale = [&](int t) {
                    float x = 0.f;
                    if (tid < 16) {
                        const int key = (tile0 + t) * kPT + 16 * (tid & 7);
                        const int pid = key < len ? page_of(a.v, slot, key >> a.v.page_log2) : -1;
                        if (pid >= 0) x = (tid < 8 ? a.ks : a.vs)[(int64_t)pid * a.v.heads + head];
                        else x = tid < 8 ? -1.f : 0.f;
                    }
                    return x;
                };
                float next = load_scale(w.t);
                for (int t = w.t; t < t_end && ok; ++t, ++tile) {
                    const int key0 = (tile0 + t) * kPT;
                    const float sc = next;
                    if (t + 1 < t_end) next = load_scale(t + 1);
#pragma unroll 1
                    for (int isv = 0; isv < 2; ++isv) {
                        const int buf = 2 * isv + (tile & 1);
                        const uint32_t b = n_raw & 1, ph = (n_raw >> 1) & 1;
                        if (!wait(&sm.raw_full[b], ph) ||
                            (tile >= 2 && !wait(&sm.kv_empty[buf], ((tile >> 1) - 1) & 1))) {
                            ok = false;
                            break;
                        }
                        ++n_raw;
                        if (isv == 0 && warp == 8) {
                            const int rg = tile & (kRing - 1);
                            const uint32_t gone = __ballot_sync(0xffffffffu, tid < 8 && sc < 0.f);
                            if (tid < 8) sm.kscale[rg][tid] = fmaxf(sc, 0.f);
                            else if (tid < 16) {
                                sm.vscale[rg][tid - 8] = sc;
                                sm.vexp[rg][tid - 8] = scale_exp(sc);
                            }
                            if (tid == 0) sm.absent[rg] = gone;
                        }
                        const uint8_t* src = sm.raw[b];
                        uint8_t* dst = sm.kv[buf];
                        // chunk c of rows r0, r0 + 128 / CH, ..: the swizzles do not change
                        const int c = tid % CH, r0 = tid / CH, c0 = (c & 3) * 2;
                        const uint32_t from = r0 * D + ((D == 128 ? c ^ (r0 & 7) : c ^ ((r0 >> 1) & 3)) << 4);
                        const uint32_t to = (c >> 2) * kBlock + r0 * 128;
                        // the second block's lanes write in the other order: no bank twice
                        const uint32_t swap = c >= 4;
                        const uint32_t p0 = to + (((c0 + swap) ^ (r0 & 7)) << 4);
                        const uint32_t p1 = to + (((c0 + 1 - swap) ^ (r0 & 7)) << 4);
                        uint4 x[CH];
#pragma unroll
                        for (int i = 0; i < CH; ++i) {
                            x[i] = *reinterpret_cast<const uint4*>(src + from + i * (128 / CH) * D);
                            // rows behind the slot's end: 0 (e4m3 rubbish may be NaN)
                            if (FMT == TQ_KV_E4M3 && key0 + r0 + i * (128 / CH) >= len) x[i] = make_uint4(0, 0, 0, 0);
                        }
#pragma unroll
                        for (int i = 0; i < CH; ++i) {
                            uint4 y0, y1;
                            codes_to_half<FMT>(x[i].x, y0.x, y0.y);
                            codes_to_half<FMT>(x[i].y, y0.z, y0.w);
                            codes_to_half<FMT>(x[i].z, y1.x, y1.y);
                            codes_to_half<FMT>(x[i].w, y1.z, y1.w);
                            *reinterpret_cast<uint4*>(dst + p0 + i * (128 / CH) * 128) = swap ? y1 : y0;
                            *reinterpret_cast<uint4*>(dst + p1 + i * (128 / CH) * 128) = swap ? y0 : y1;
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&sm.kv_full[buf]);
                            mbar_arrive(&sm.raw_empty[b]);
                        }
                    }
                }
                done_with(n);
            }
        } else if (warp == 12 || warp == 15) {
            // ============================================== MMAs of a stage
            const int st = warp == 15;
            constexpr uint32_t kQK = idesc_f16(0, kPM, kPH);
            constexpr uint32_t kPV = idesc_f16(0, kPM, D) | (1u << 16);  // B MN-major
            constexpr uint32_t kQBytes = kPM * D * 2;
            const uint32_t qb = smem_u32(sm.q[st]), kvb = smem_u32(sm.kv[0]);
            const uint32_t s_col = tbase + st * kPT, o_col = tbase + 2 * kPT + st * D;
            uint32_t tile = 0, n_q = 0, n_t = 0;  // all tiles; items and tiles of the stage
            bool ok = true;
            // (an offset within an operand adds to its descriptor, in units of 16 bytes)
            auto qk = [&](uint32_t u, int h) {  // S of half h of tile u
                const uint64_t q = smem_desc_kmajor_sw128(qb);
                const uint64_t kd = smem_desc_kmajor_sw128(kvb + (u & 1) * kQBytes + h * kPH * 128);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = ((k >> 2) * kBlock + (k & 3) * 32) / 16;
                        mma_f16_ss(s_col + h * kPH, q + off, kd + off, kQK, k > 0);
                    }
                    tc_commit(&sm.s_full[st][h]);
                }
            };
            auto pv = [&](uint32_t u, int h, bool first) {
                const uint64_t v = smem_desc_mnmajor_sw128(kvb + (2 + (u & 1)) * kQBytes + h * kPH * 128, kBlock);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kPH / 16; ++k)
                        mma_f16_ts(o_col, s_col + h * kPH + 8 * k, v + k * 2048 / 16, kPV, !(first && k == 0));
                    tc_commit(&sm.o_done[st][h]);
                }
            };
            for (uint32_t n = 0; ok && (ok = get(n)); ++n) {
                const Work& w = sm.work[n % kWorks];
                const int tiles = w.t_end - w.t, rows = w.rows;
                if (rows == 0) break;
                done_with(n);
                if (st * kPM >= rows) {  // not for this stage: its consent to every tile's release
                    for (int t = 0; t < tiles && ok; ++t, ++tile)
                        for (uint32_t b = tile & 1; b < 4 && ok; b += 2) {
                            ok = wait(&sm.kv_full[b], (tile >> 1) & 1);
                            if (ok && lane == 0) mbar_arrive(&sm.kv_empty[b]);
                        }
                    continue;
                }
                ok = wait(&sm.q_full[st], n_q++ & 1) && wait(&sm.kv_full[tile & 1], (tile >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
                qk(tile, 0);
                qk(tile, 1);
                if (elect_one()) tc_commit(&sm.kv_empty[tile & 1]);
                // S of a half is two halves ahead of P V: its softmax never waits for it
                for (int t = 0; t < tiles && ok; ++t, ++tile, ++n_t) {
                    const bool more = t + 1 < tiles;
                    ok = wait(&sm.kv_full[2 + (tile & 1)], (tile >> 1) & 1);
                    for (int h = 0; h < 2 && ok; ++h) {
                        ok = wait(&sm.p_full[st][h], n_t & 1);
                        if (!ok) break;
                        tc_fence_after();
                        pv(tile, h, t == 0 && h == 0);
                        if (!more) continue;
                        if (h == 0) ok = wait(&sm.kv_full[(tile + 1) & 1], ((tile + 1) >> 1) & 1);
                        if (ok) qk(tile + 1, h);
                    }
                    if (ok && elect_one()) {
                        tc_commit(&sm.kv_empty[2 + (tile & 1)]);
                        if (more) tc_commit(&sm.kv_empty[(tile + 1) & 1]);
                    }
                }
            }
            // all MMAs are done before tensor and shared memory go
            if (elect_one()) tc_commit(&sm.mma_done[st]);
            __syncwarp();
            int none = 0;
            mbar_wait(&sm.mma_done[st], 0, &none, kWaitNs);
            __syncwarp();
        } else if (warp == 13) {
            // ============================================== TMA
            const int box = a.v.page, nbox = kPT / box;
            uint32_t c = 0;  // copies of a tile's K or V
            bool ok = true;
            for (uint32_t n = 0; ok && (ok = get(n)); ++n) {
                const Work& w = sm.work[n % kWorks];
                if (w.rows == 0) break;
                const int t_end = w.t_end, len = w.len, slot = w.slot, head = w.head, tile0 = w.t0;
                auto lookup = [&](int t) {
                    const int key = (tile0 + t) * kPT + lane * box;
                    return lane < nbox && key < len ? page_of(a.v, slot, key >> a.v.page_log2) : -1;
                };
                int t = w.t, next = lookup(t);
                done_with(n);
                for (; t < t_end && ok; ++t) {
                    // (a page that is not there: rows behind the tensor, zeros)
                    const int row = next >= 0 ? (int)(((int64_t)next * a.v.heads + head) << a.v.page_log2) : a.rows;
                    if (t + 1 < t_end) next = lookup(t + 1);
                    for (int isv = 0; isv < 2; ++isv, ++c) {
                        const uint32_t b = c & 1;
                        if (c >= 2 && !wait(&sm.raw_empty[b], ((c >> 1) - 1) & 1)) {
                            ok = false;
                            break;
                        }
                        if (lane == 0) mbar_arrive_expect_tx(&sm.raw_full[b], kPT * D);
                        __syncwarp();
                        if (lane < nbox)
                            tma_load_2d(sm.raw[b] + lane * box * D, isv ? &vmap : &kmap, 0, row, &sm.raw_full[b]);
                    }
                }
            }
            if (!ok) {  // no copy may land after the block has gone
                int none = 0;
                for (uint32_t i = c >= 2 ? c - 2 : 0; i < c; ++i)
                    mbar_wait(&sm.raw_full[i & 1], (i >> 1) & 1, &none, kWaitNs);
            }
        } else if (warp == 14) {
            // ============================================== the CTA's share, item by item
            Entry e = {};
            int head = 0, part = 0, m = 0, t = 0;
            bool ok = true;
            if (g0 < g1) {
                int64_t per_head;
                while (true) {
                    e = entry_of(a, entry);
                    per_head = warp_sum(tiles_per_head(a, e, lane, 32));
                    if (rem < per_head * a.v.heads) break;
                    rem -= per_head * a.v.heads;
                    ++entry;
                }
                m = parts_of(a, e);
                head = (int)quot(rem, per_head);
                rem -= head * per_head;
                for (;; part += 32) {  // 32 parts at a time
                    int t0, nt = 0;
                    if (part + lane < m) tiles_of(a, e, part + lane, t0, nt);
                    int64_t inc = nt;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
                        if (lane >= o) inc += y;
                    }
                    const uint32_t past = __ballot_sync(0xffffffffu, inc > rem);
                    if (past) {
                        const int k = __ffs(past) - 1;
                        t = (int)(rem - (__shfl_sync(0xffffffffu, inc, k) - __shfl_sync(0xffffffffu, nt, k)));
                        part += k;
                        break;
                    }
                    rem -= __shfl_sync(0xffffffffu, inc, 31);
                }
            }
            uint32_t n = 0;
            for (int64_t g = g0; ok; ++n) {
                Work w = {};
                if (g < g1) {
                    w.slot = e.slot;
                    w.len = e.len;
                    w.head = head;
                    w.pos0 = e.len - e.qn;
                    w.row0 = part * kPRows;
                    w.rows = min(kPRows, e.qn * a.group - w.row0);
                    w.c0 = e.c0;
                    tiles_of(a, e, part, w.t0, w.nt);
                    w.t = t;
                    w.t_end = (int)min((int64_t)w.nt, t + (g1 - g));
                    if (t == 0 && w.t_end < w.nt) {
                        const int64_t last = g + w.nt - 1, head1 = rest * (base + 1);  // the item's last step: its CTA
                        w.parts = (int)(last < head1 ? quot(last, base + 1) : rest + quot(last - head1, base)) - unit + 1;
                    }
                }
                ok = n < kWorks || wait(&sm.work_empty[n % kWorks], (n / kWorks - 1) & 1);
                if (!ok) break;
                if (lane == 0) {
                    sm.work[n % kWorks] = w;
                    mbar_arrive(&sm.work_full[n % kWorks]);
                }
                if (w.rows == 0) break;
                g += w.t_end - t;
                t = 0;
                if (g < g1 && ++part == m) {
                    part = 0;
                    if (++head == a.v.heads) {
                        head = 0;
                        do {
                            e = entry_of(a, ++entry);
                            m = parts_of(a, e);
                        } while (m == 0);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tmem_dealloc(tbase, kTmemCols);
    if (threadIdx.x == 0) parts.block_status[unit] = sm.abort ? TQ_ERR_DEVICE_TIMEOUT * 1000 - 81 : 0;
}

// Joins the parts of the items that were cut: blocks (u, y) the item that begins
// in CTA u, a warp a row, 4 coordinates a lane (d = 128) or 2.  Where the call was
// refused or the cache's status is set it writes rows that see no key; rows behind the
// last entry's are its work too.
template <int D, typename T>
__global__ __launch_bounds__(256) void k_prompt_merge(const Attn a, const PromptParts parts, int blocks) {
    const int u = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_begin();
    if (a.behind && blockIdx.y == 0) zero_behind<D, T>(a, max(a.cu[a.ns], 0));
    const bool bad = parts.block_status[0] == TQ_ERR_ARG;  // (all blocks', then)
    const int held = pending(a.v);
    if (u == 0 && blockIdx.y == 0) {
        int st = 0;
        for (int i = threadIdx.x; i < blocks; i += 256) st |= parts.block_status[i] != 0;
        st = __syncthreads_or(st);
        const int status = bad ? TQ_ERR_ARG : st ? TQ_ERR_DEVICE_TIMEOUT * 1000 - 81 : held;
        // (the few-rows kernel of the call has set the word; a time-out stands)
        if (threadIdx.x == 0 && (st || !parts.keep_status)) *parts.status = status;
        if (threadIdx.x == 0 && st) leave_status(a.v, status);
    }
    const Cut c = parts.cut[u];
    if (held || bad) empty_rows<D, T>(a);
    if (held || bad || c.parts == 0) return;
    constexpr int E = D / 32;
    auto slot = [&](int i) { return i == 0 ? 2 * (int64_t)u + 1 : 2 * (int64_t)(u + i); };
    for (int r = blockIdx.y * 8 + warp; r < c.rows; r += gridDim.y * 8) {
        float m = -INFINITY;
        for (int i = lane; i < c.parts; i += 32) m = fmaxf(m, parts.ml[slot(i) * kPRows + r].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float base = m == -INFINITY ? 0.f : m;
        float L = 0.f, acc[E];
#pragma unroll
        for (int k = 0; k < E; ++k) acc[k] = 0.f;
#pragma unroll 2
        for (int i = 0; i < c.parts; ++i) {
            const int64_t pr = slot(i) * kPRows + r;
            const float2 ml = parts.ml[pr];
            const float f = ex2(ml.x - base);
            L = fmaf(f, ml.y, L);
            const float* src = parts.o + pr * D + lane * E;
            float x[E];
            if (E == 4) *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(src);
            else *reinterpret_cast<float2*>(x) = *reinterpret_cast<const float2*>(src);
#pragma unroll
            for (int k = 0; k < E; ++k) acc[k] = fmaf(f, x[k], acc[k]);
        }
        const int64_t ri = c.row0 + r, tok = ri / a.group;
        const int hq = c.head * a.group + (int)(ri - tok * a.group);
        const float n = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
        T* out = (T*)a.out + (tok * a.heads_q + hq) * D + lane * E;
        Pack<T, E> y;
#pragma unroll
        for (int k = 0; k < E; ++k) from_f(acc[k] * n, y.v[k]);
        *reinterpret_cast<Pack<T, E>*>(out) = y;
        if (a.lse && lane == 0)
            a.lse[tok * a.heads_q + hq] = L > 0.f ? (m + log2f(L)) * 0.69314718056f : (L == 0.f ? -INFINITY : L);
    }
}

template <int FMT, int D, typename T>
int go(const Attn& a, const CUtensorMap& km, const CUtensorMap& vm, const PromptParts& p, int blocks,
       cudaStream_t s) {
    constexpr int smem = (int)sizeof(PSmem<D>) + 1024;
    static_assert(smem <= 232448, "shared memory of a block");
    int rc = allow_smem<k_attn_prompt<FMT, D, T>>(smem);
    if (!rc) rc = launch_behind(k_attn_prompt<FMT, D, T>, dim3(blocks), kPThreads, smem, s, a, km, vm, p);
    if (!rc) rc = launch_behind(k_prompt_merge<D, T>, dim3((unsigned)blocks, 16), 256, 0, s, a, p, blocks);
    return rc;
}

template <int D>
int go_d(const tq_kv8_t* c, const Attn& a, const CUtensorMap& km, const CUtensorMap& vm,
         const PromptParts& p, int blocks, int q_dtype, cudaStream_t s) {
    if (c->format == TQ_KV_I8)
        return q_dtype == TQ_BF16 ? go<TQ_KV_I8, D, __nv_bfloat16>(a, km, vm, p, blocks, s)
                                  : go<TQ_KV_I8, D, __half>(a, km, vm, p, blocks, s);
    return q_dtype == TQ_BF16 ? go<TQ_KV_E4M3, D, __nv_bfloat16>(a, km, vm, p, blocks, s)
                              : go<TQ_KV_E4M3, D, __half>(a, km, vm, p, blocks, s);
}

}  // namespace

int prompt_blocks(const tq_kv8_t* c, int ns, int64_t total_q, int heads_q) {
    const int64_t tiles = ((int64_t)c->max_pages * c->page + kPT - 1) / kPT;
    const int64_t most = tiles * (total_q * (heads_q / c->heads) / kPRows + ns) * c->heads;
    return (int)(most < 148 ? (most < 1 ? 1 : most) : 148);
}

PromptParts prompt_carve(const tq_kv8_t* c, void* ws, int blocks, size_t* bytes) {
    PromptParts p;
    char* at = (char*)ws;
    p.status = nullptr;
    p.keep_status = 0;
    p.block_status = (int*)at;
    at += align256(blocks * 4);
    p.cut = (Cut*)at;
    at += align256(blocks * sizeof(Cut));
    p.ml = (float2*)at;
    at += align256((size_t)2 * blocks * kPRows * sizeof(float2));
    p.o = (float*)at;
    at += align256((size_t)2 * blocks * kPRows * c->d * 4);
    *bytes = (size_t)(at - (char*)ws);
    return p;
}

int launch_prompt(const tq_kv8_t* c, int layer, const Attn& a, const PromptParts& p, int blocks,
                  int q_dtype, cudaStream_t s) {
    CUtensorMap km, vm;
    int rc = code_map(&km, (const char*)c->d_k + layer * layer_bytes(c), c->d, a.rows, c->page);
    if (!rc) rc = code_map(&vm, (const char*)c->d_v + layer * layer_bytes(c), c->d, a.rows, c->page);
    if (rc) return rc;
    return c->d == 128 ? go_d<128>(c, a, km, vm, p, blocks, q_dtype, s)
                       : go_d<64>(c, a, km, vm, p, blocks, q_dtype, s);
}

}  // namespace kv8
}  // namespace tq
