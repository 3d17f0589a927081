// The 8-bit paged KV cache: geometry, writing tokens and reading them back.
//
// Write (tq_kv8_append): for every page and head that new tokens fall into,
//   s = max(s0, max |x| / M)   (s0: the scale of the tokens there already, if any;
//                               below fp32's normal range the quotient is rounded up)
//   code = rnd(x / s),         old codes: rnd(code s0 / s) where s > s0,
// keys turned to their positions first (fp32, not rounded in between).
//
// A block owns whole (slot, page, head)s of K or V, so the page's maximum is a
// block reduction and nothing is written twice: new rows are loaded once into
// registers, turned, reduced, rounded and stored; the page's old rows are touched
// only when the scale grows.  Bound by issue slots and by its loads' latency at half
// of the warps for prompts (28105 tokens x 8 heads of 128, bf16 to e4m3: 55 us, 3.2
// TB/s, 66 us with half of each key turned; 512 threads of one item beat 256 of two,
// 53 against 65, and 4 heads a block one head, 53 against 78), by the chain length ->
// table -> scale for single tokens (4.6 us for 64).
#include "tq_kv8.cuh"
#include "tq_rope.cuh"

namespace tq {
namespace kv8 {

bool valid(const tq_kv8_t* c, int* status) {
    *status = TQ_ERR_ARG;
    if (!c) return false;
    if (c->format != TQ_KV_I8 && c->format != TQ_KV_E4M3) return false;
    *status = TQ_ERR_UNSUPPORTED;
    if (c->d != 64 && c->d != 128) return false;
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return false;
    *status = TQ_ERR_ARG;
    if (c->heads < 1 || c->layers < 1 || c->slots < 1 || c->max_pages < 1 || c->pages < 1)
        return false;
    *status = TQ_ERR_UNSUPPORTED;
    // rows of a layer, and a slot's tokens, count in 32 bits
    if ((int64_t)c->pages * c->heads >= ((int64_t)1 << 31) / c->page) return false;
    if ((int64_t)c->max_pages * c->page >= (int64_t)1 << 31 || c->heads > 65535) return false;
    *status = TQ_ERR_ARG;
    if (!c->d_k || !c->d_v || !c->d_kscale || !c->d_vscale || !c->d_table || !c->d_len || !c->d_refs)
        return false;
    if (((uintptr_t)c->d_k | (uintptr_t)c->d_v) & 15u) return false;
    *status = TQ_OK;
    return true;
}

namespace {

// ---- write ------------------------------------------------------------------

struct AppendArgs {
    View v;
    const int32_t* slots;
    const int32_t* cu;
    int ppb;  // pages a slot's new tokens can touch
    int hb;   // heads a block
    int max_new;
    int64_t total;
    const void *x[2];
    int64_t x_ts, x_hs;
    uint8_t* codes[2];
    float* scale[2];
    int rope;
};

constexpr float kLargest = 1.7014118e38f;  // 2^127

// The cache's status on its way into shared memory (a register would be spilled).
__device__ __forceinline__ void pending_to(int32_t* s, const View& v) {
    if (v.status)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;"
                     ::"r"((uint32_t)__cvta_generic_to_shared(s)), "l"(v.status) : "memory");
    else
        *s = 0;
}

// The larger one of a and |b|, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("{\n\t.reg .f32 t;\n\tabs.f32 t, %2;\n\tmax.NaN.f32 %0, %1, t;\n\t}" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A block writes `hb` heads of one page, one after another: an item of a thread
// (two runs of VEC coordinates of a row, half the turned or the other part apart)
// is the same in every head, so its angles are formed once, and the next head's
// rows are on their way while this one's are rounded.  VEC = 8 (16-byte accesses)
// or 1; NI items a thread; ROPE: 0 none, 1 half layout, 2 interleaved.
template <typename T, int FMT, int VEC, int NI, int ROPE>
__global__ __launch_bounds__(VEC == 8 ? 1024 : 256) void k_append(
    const AppendArgs a, const __grid_constant__ tq_rope_params_t rope) {
    __shared__ uint32_t s_red[2][32];
    __shared__ int32_t s_held;
    grid_begin();
    const View& v = a.v;
    const int seq = blockIdx.x / a.ppb, pj = blockIdx.x - seq * a.ppb;
    const int kv = blockIdx.z;
    const int slot = slot_of(v, a.slots, seq);
    const int64_t c0 = max(a.cu[seq], 0);
    const int count = (int)(min((int64_t)a.cu[seq + 1], a.total) - c0);
    if (slot < 0) return;
    if (count > a.max_new || a.cu[seq + 1] > a.total) {  // not what the host launched for
        if (threadIdx.x == 0) leave_status(v, TQ_ERR_ARG);
        return;
    }
    if (count <= 0) return;
    const int len = length_of(v, slot);
    // tokens before the slot's first position have no place
    const int start = max(len - count, 0), skip = max(count - len, 0);
    const int page0 = start >> v.page_log2;
    const int lo_pos = max(start, (page0 + pj) << v.page_log2);
    const int hi_pos = min(len, (page0 + pj + 1) << v.page_log2);
    if (lo_pos >= hi_pos) return;
    const int pid = page_of(v, slot, page0 + pj);
    if (pid < 0) return;
    const int row0 = lo_pos & (v.page - 1), rows = hi_pos - lo_pos;
    const int h0 = blockIdx.y * a.hb, h1 = min(v.heads, h0 + a.hb);
    const int64_t ph0 = (int64_t)pid * v.heads;
    const T* x = (const T*)a.x[kv] + (c0 + skip + lo_pos - start) * a.x_ts + h0 * a.x_hs;
    const bool turn = ROPE && kv == 0;

    const int shift = (v.d == 128 ? 6 : 5) - (VEC == 8 ? 3 : 0);  // log2 of the items of a row
    const int n = rows << shift, half = rope.rot / 2;
    using P = Pack<T, VEC>;
    const T* src[NI];   // the first run of the item in the next head
    int o1[NI], gap[NI];  // its coordinate, the second run's distance
    P p1[NI], p2[NI];
    bool on[NI], pair[NI];
    float2 cs[VEC == 8 ? NI : 1][VEC];
    auto fetch = [&]() {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if (!on[i]) continue;
            p1[i] = *reinterpret_cast<const P*>(src[i]);
            p2[i] = *reinterpret_cast<const P*>(src[i] + gap[i]);
            src[i] += a.x_hs;
        }
    };
    // amplitude (cos, sin) of the item's pairs: coordinates o1 + e and o1 + gap + e
    // (half layout), or neighbours, those of the first run and then of the second
    auto angles = [&](int i, float2 (&w)[VEC]) {
        const int64_t pos = lo_pos + ((threadIdx.x + i * blockDim.x) >> shift);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            int k = o1[i] + e;
            if (ROPE == 2)
                k = VEC == 1 ? o1[i] / 2 : e < VEC / 2 ? o1[i] / 2 + e : (o1[i] + gap[i] - VEC) / 2 + e;
            float c = 1.f, s = 0.f;
            if (k < half) rope_angle(rope.turns[k], pos, c, s);
            w[e] = make_float2(rope.amplitude * c, rope.amplitude * s);
        }
    };
    // pair e of an interleaved item is turned (its coordinates lie within rot)
    auto turned = [&](int i, int e) {
        return VEC == 1 ? o1[i] < rope.rot : (e < VEC / 2 ? o1[i] + 2 * e : o1[i] + gap[i] + 2 * e - VEC) < rope.rot;
    };
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int it = threadIdx.x + i * blockDim.x;
        on[i] = it < n;
        const int row = it >> shift, m = (it - (row << shift)) * VEC;
        pair[i] = ROPE == 1 && turn && m < half;
        const int from = ROPE == 1 && turn ? rope.rot : 0;  // coordinates that are left to the plain items
        o1[i] = pair[i] || from == 0 ? m : from + m - half;
        gap[i] = pair[i] ? half : (v.d - from) / 2;
        if (VEC == 1 && ROPE == 2) {  // a neighbour pair
            o1[i] = 2 * m;
            gap[i] = 1;
        }
        src[i] = x + row * a.x_ts + o1[i];
    }
    if (threadIdx.x == 0) pending_to(&s_held, v);
    fetch();
    if (VEC == 8 && ROPE && turn) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (on[i] && (ROPE == 2 || pair[i])) angles(i, cs[VEC == 8 ? i : 0]);
    }

    for (int h = h0; h < h1; ++h) {
        const int64_t ph = ph0 + h;
        const float s_old = row0 > 0 ? a.scale[kv][ph] : 0.f;
        float val[NI][2 * VEC];
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if (!on[i]) continue;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                val[i][e] = to_f(p1[i].v[e]);
                val[i][VEC + e] = to_f(p2[i].v[e]);
            }
            if (turn && (ROPE == 2 || pair[i])) {
                if (VEC == 1) angles(i, cs[0]);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int i1 = ROPE == 1 ? e : 2 * e, i2 = ROPE == 1 ? VEC + e : 2 * e + 1;
                    const float2 w = cs[VEC == 8 ? i : 0][e];
                    const float x1 = val[i][i1], x2 = val[i][i2];
                    if (ROPE == 1 || turned(i, e)) {
                        val[i][i1] = x1 * w.x - x2 * w.y;
                        val[i][i2] = x2 * w.x + x1 * w.y;
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 2 * VEC; ++e) top = max_nan(top, val[i][e]);
        }
        if (h + 1 < h1) fetch();
        if (!(top <= kLargest)) {  // NaN: 0; up to 2^127, so that scale x code stays finite
            top = 0.f;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                if (!on[i]) continue;
#pragma unroll
                for (int e = 0; e < 2 * VEC; ++e) {
                    const float y = val[i][e];
                    val[i][e] = y == y ? fminf(fmaxf(y, -kLargest), kLargest) : 0.f;
                    top = fmaxf(top, fabsf(val[i][e]));
                }
            }
        }
        // (floats >= 0 are ordered as their bits are)
        uint32_t* red = s_red[h & 1];
        const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = most;
        if (h == h0 && threadIdx.x == 0) asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        const int held = h == h0 ? s_held : 0;
        const uint32_t lane = threadIdx.x & 31;
        top = __uint_as_float(__reduce_max_sync(0xffffffffu, lane < blockDim.x / 32 ? red[lane] : 0u));
        if (held) return;  // (before the first store)
        float s = fmaxf(s_old, __fdiv_rn(top, code_max<FMT>()));
        float up = 1.f, inv = s > 0.f ? __frcp_rn(s) : 0.f;
        if (s < 1.17549435e-38f) {  // below fp32's normal range:
            // a few units of 2^-149 are rounded up, so that no code leaves its range;
            if (fmaf(s, code_max<FMT>(), -top) < 0.f) s = __uint_as_float(__float_as_uint(s) + 1);
            up = 18446744073709551616.f;  // a reciprocal may overflow: all times 2^64
            inv = s > 0.f ? __frcp_rn(s * up) : 0.f;
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int e = 0; e < 2 * VEC; ++e) val[i][e] *= up;
        }
        if (threadIdx.x == 0) a.scale[kv][ph] = s;
        uint8_t* codes = a.codes[kv] + (ph << v.page_log2) * v.d;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if (!on[i]) continue;
            const int row = (threadIdx.x + i * blockDim.x) >> shift;
            uint8_t* c1 = codes + (row0 + row) * v.d + o1[i];
            uint8_t* c2 = c1 + gap[i];
            if (VEC == 8) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = encode4<FMT>(val[i][4 * e % (2 * VEC)], val[i][(4 * e + 1) % (2 * VEC)],
                                        val[i][(4 * e + 2) % (2 * VEC)], val[i][(4 * e + 3) % (2 * VEC)], inv);
                *reinterpret_cast<uint2*>(c1) = make_uint2(w[0], w[1]);
                *reinterpret_cast<uint2*>(c2) = make_uint2(w[2], w[3]);
            } else {
                const uint32_t w = encode4<FMT>(val[i][0], val[i][1], 0.f, 0.f, inv);
                *c1 = (uint8_t)w;
                *c2 = (uint8_t)(w >> 8);
            }
        }
        if (row0 > 0 && s > s_old) {  // the page's old rows, for the new scale
            const float f = s_old * up * inv;
            uint4* w = reinterpret_cast<uint4*>(codes);
            const int nw = row0 * v.d / 16;
            for (int i0 = threadIdx.x; i0 < nw; i0 += 4 * blockDim.x) {
                uint4 c[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (i0 + e * (int)blockDim.x < nw) c[e] = w[i0 + e * blockDim.x];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (i0 + e * (int)blockDim.x >= nw) continue;
                    uint32_t y[4] = {c[e].x, c[e].y, c[e].z, c[e].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float z[4];
                        decode4<FMT>(y[k], z);
                        y[k] = encode4<FMT>(z[0], z[1], z[2], z[3], f);
                    }
                    w[i0 + e * blockDim.x] = make_uint4(y[0], y[1], y[2], y[3]);
                }
            }
        }
    }
}

template <typename T, int FMT, int VEC, int NI>
int append_go(AppendArgs a, const tq_rope_params_t& r, int ns, int threads, cudaStream_t s) {
    const int64_t gx = (int64_t)ns * a.ppb;
    if (gx > 0x7fffffff) return TQ_ERR_UNSUPPORTED;
    // heads a block: as many as leave every SM 16 blocks
    const int64_t share = gx * a.v.heads * 2 / (148 * 16);
    a.hb = (int)(share < 1 ? 1 : share > 8 ? 8 : share);
    const int parts = (a.v.heads + a.hb - 1) / a.hb;
    a.hb = (a.v.heads + parts - 1) / parts;
    const dim3 grid((unsigned)gx, (unsigned)parts, 2);
    auto kernel = !a.rope || r.rot == 0 ? k_append<T, FMT, VEC, NI, 0>
                  : r.layout == TQ_ROPE_HALF ? k_append<T, FMT, VEC, NI, 1> : k_append<T, FMT, VEC, NI, 2>;
    return launch_behind(kernel, grid, threads, 0, s, a, r);
}

// Threads and items a thread for the most rows that a block can get.
template <typename T, int FMT>
int append_fmt(const AppendArgs& a, const tq_rope_params_t& r, int ns, int max_new, bool wide,
               cudaStream_t s) {
    const int rows = max_new < a.v.page ? max_new : a.v.page;
    if (wide) {
        const int items = rows * a.v.d / 16;
        if (items <= 128) return append_go<T, FMT, 8, 1>(a, r, ns, 128, s);
        return append_go<T, FMT, 8, 1>(a, r, ns, items <= 256 ? 256 : items <= 512 ? 512 : 1024, s);
    }
    const int items = rows * a.v.d / 2;
    if (items <= 256) return append_go<T, FMT, 1, 1>(a, r, ns, 256, s);
    return append_go<T, FMT, 1, 32>(a, r, ns, 256, s);
}

template <typename T>
int append_type(const tq_kv8_t* c, const AppendArgs& a, const tq_rope_params_t& r, int ns,
                int max_new, cudaStream_t s) {
    bool wide = ((uintptr_t)a.x[0] | (uintptr_t)a.x[1]) % 16 == 0 && a.x_ts % 8 == 0 &&
                a.x_hs % 8 == 0;
    // a half-layout pair block is 8 + 8 coordinates
    if (a.rope && r.layout == TQ_ROPE_HALF && r.rot % 16) wide = false;
    return c->format == TQ_KV_I8 ? append_fmt<T, TQ_KV_I8>(a, r, ns, max_new, wide, s)
                                 : append_fmt<T, TQ_KV_E4M3>(a, r, ns, max_new, wide, s);
}

// ---- read -------------------------------------------------------------------

constexpr int kReadThreads = 256;
constexpr int kReadItems = 4;  // of 16 codes, a thread

// A block reads `tokens` tokens of one slot, all heads, K or V: 16 codes an item.
// (and, of an entry with more tokens than the launch was sized for, every bps-th such
// run behind it).  The lookups of a thread's items, then their codes, are on their way
// together.  Rows that no entry owns become 0.
// 28306 tokens x 8 heads of 128, e4m3 to bf16: 38 us, 4.6 TB/s, 70 % of the copy rate;
// the divisions that find an item's token, head and chunk are the rest.
template <typename T, int FMT>
__global__ __launch_bounds__(kReadThreads) void k_read(View v, const int32_t* slots, const int32_t* begin,
                                                       const int32_t* cu, int ns, int bps, int tokens, int64_t total,
                                                       const uint8_t* kc, const uint8_t* vc, const float* ks,
                                                       const float* vs, T* out_k, T* out_v) {
    grid_begin();
    const int seq = blockIdx.x / bps, blk = blockIdx.x - seq * bps;
    const int slot = slot_of(v, slots, seq);
    const int64_t c0 = max(cu[seq], 0), c1 = min((int64_t)cu[seq + 1], total);
    const int used = max(cu[ns], 0);
    const int64_t b0 = begin[seq];
    const int held = v.status ? *v.status : 0;  // (through L1: nothing here has to agree on it)
    int len = slot >= 0 ? length_of(v, slot) : 0;
    if (held) len = 0;
    const int chunks = v.d / 16, per = v.heads * chunks;
    const bool is_v = blockIdx.y != 0;
    T* out = is_v ? out_v : out_k;
    if (!out) return;
    const uint8_t* codes = is_v ? vc : kc;
    const float* scales = is_v ? vs : ks;
    for (int64_t first = (int64_t)blk * tokens; first < c1 - c0; first += (int64_t)bps * tokens) {
        const int64_t b = b0 + first;
        const int n = (int)min((int64_t)tokens, c1 - c0 - first) * per;
        // (items of a block are neighbours in the output: token, head, chunk)
        Pack<T, 8>* dst = reinterpret_cast<Pack<T, 8>*>(out + (c0 + first) * v.heads * v.d);
        for (int i0 = threadIdx.x; i0 < n; i0 += kReadItems * kReadThreads) {
            int pid[kReadItems];
#pragma unroll
            for (int e = 0; e < kReadItems; ++e) {
                const int i = i0 + e * kReadThreads;
                pid[e] = -1;
                if (i < n) {
                    const int64_t pos = b + i / per;
                    if (pos >= 0 && pos < len) pid[e] = page_of(v, slot, (int)(pos >> v.page_log2));
                }
            }
            uint4 w[kReadItems];
            float s[kReadItems];
#pragma unroll
            for (int e = 0; e < kReadItems; ++e) {
                const int i = i0 + e * kReadThreads;
                w[e] = make_uint4(0, 0, 0, 0);
                s[e] = 0.f;
                if (pid[e] >= 0) {
                    const int t = i / per, hc = i - t * per, h = hc / chunks, ch = hc - h * chunks;
                    const int64_t ph = (int64_t)pid[e] * v.heads + h;
                    w[e] = *reinterpret_cast<const uint4*>(
                        codes + ((ph << v.page_log2) + ((b + t) & (v.page - 1))) * v.d + 16 * ch);
                    s[e] = scales[ph];
                }
            }
#pragma unroll
            for (int e = 0; e < kReadItems; ++e) {
                const int i = i0 + e * kReadThreads;
                if (i >= n) continue;
                const uint32_t ww[4] = {w[e].x, w[e].y, w[e].z, w[e].w};
                Pack<T, 8> o[2];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float x[4];
                    decode4<FMT>(ww[k], x);
#pragma unroll
                    for (int j = 0; j < 4; ++j) from_f(s[e] * x[j], o[k / 2].v[4 * (k & 1) + j]);
                }
                dst[2 * (int64_t)i] = o[0];
                dst[2 * (int64_t)i + 1] = o[1];
            }
        }
    }
    Pack<T, 8> zero;
#pragma unroll
    for (int j = 0; j < 8; ++j) from_f(0.f, zero.v[j]);
    for (int64_t t = (int64_t)used + blockIdx.x; t < total; t += gridDim.x)
        for (int i = threadIdx.x; i < 2 * per; i += kReadThreads)
            reinterpret_cast<Pack<T, 8>*>(out + t * v.heads * v.d)[i] = zero;
}

template <typename T>
int read_type(const tq_kv8_t* c, int layer, int ns, const int32_t* slots, const int32_t* begin,
              const int32_t* cu, int64_t total, int max_new, void* k, void* v, cudaStream_t s) {
    // a batch of items a thread, or fewer tokens a block where that leaves SMs idle
    const int per = c->heads * c->d / 16;
    int64_t tokens = kReadItems * kReadThreads / per, fill = (int64_t)ns * max_new / (148 * 4);
    if (tokens > fill) tokens = fill;
    tokens = tokens < 1 ? 1 : (tokens > max_new ? max_new : tokens);
    const int64_t bps = (max_new + tokens - 1) / tokens;
    if (bps * ns > 0x7fffffff) return TQ_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)(bps * ns), 2);
    const uint8_t* kc = (const uint8_t*)c->d_k + layer * layer_bytes(c);
    const uint8_t* vc = (const uint8_t*)c->d_v + layer * layer_bytes(c);
    const float* ks = c->d_kscale + layer * layer_scales(c);
    const float* vs = c->d_vscale + layer * layer_scales(c);
    return launch_behind(c->format == TQ_KV_I8 ? k_read<T, TQ_KV_I8> : k_read<T, TQ_KV_E4M3>, grid,
                         kReadThreads, 0, s, view(c), slots, begin, cu, ns, (int)bps, (int)tokens, total, kc, vc,
                         ks, vs, (T*)k, (T*)v);
}

}  // namespace
}  // namespace kv8
}  // namespace tq

using namespace tq;

extern "C" size_t tq_kv8_workspace_bytes(int op, const tq_kv8_t* c, int n, int64_t total, int max_q,
                                         int heads_q) {
    int status;
    if (!kv8::valid(c, &status) || n < 0) return (size_t)-1;
    if (op == TQ_KV8_OP_PAGES) return n > 4096 ? (size_t)-1 : kv8::pages_workspace(c, n);
    if (op == TQ_KV8_OP_ATTENTION) {
        if (total < 0 || max_q < 0 || heads_q < 1 || heads_q % c->heads) return (size_t)-1;
        return kv8::attention_workspace(c, n, total, max_q, heads_q);
    }
    return (size_t)-1;
}

extern "C" int tq_kv8_append(const tq_kv8_t* c, int layer, int ns, const int32_t* d_slots,
                             const int32_t* d_cu, int64_t total, int max_new, const void* d_k,
                             const void* d_v, int x_dtype, int64_t x_ts, int64_t x_hs,
                             const tq_rope_params_t* r, void* stream) {
    int status;
    if (!kv8::valid(c, &status)) return status;
    if (layer < 0 || layer >= c->layers || ns < 0 || total < 0 || max_new < 0) return TQ_ERR_ARG;
    if (x_dtype != TQ_F32 && x_dtype != TQ_BF16 && x_dtype != TQ_F16) return TQ_ERR_ARG;
    if (r && (!rope_valid(r) || r->d != c->d)) return TQ_ERR_ARG;
    if (!d_slots && ns > c->slots) return TQ_ERR_ARG;
    if (ns == 0 || total == 0 || max_new == 0) return TQ_OK;
    if (!d_cu || !d_k || !d_v) return TQ_ERR_ARG;
    kv8::AppendArgs a;
    a.v = kv8::view(c);
    a.slots = d_slots;
    a.cu = d_cu;
    a.ppb = (int)(((int64_t)max_new + c->page - 2) / c->page + 1);
    if (a.ppb > c->max_pages) a.ppb = c->max_pages;
    a.max_new = max_new;
    a.total = total;
    a.x[0] = d_k;
    a.x[1] = d_v;
    a.x_ts = x_ts;
    a.x_hs = x_hs;
    a.codes[0] = (uint8_t*)c->d_k + layer * kv8::layer_bytes(c);
    a.codes[1] = (uint8_t*)c->d_v + layer * kv8::layer_bytes(c);
    a.scale[0] = c->d_kscale + layer * kv8::layer_scales(c);
    a.scale[1] = c->d_vscale + layer * kv8::layer_scales(c);
    a.rope = r != nullptr;
    const tq_rope_params_t none = {};
    cudaStream_t s = (cudaStream_t)stream;
    switch (x_dtype) {
        case TQ_F32: return kv8::append_type<float>(c, a, r ? *r : none, ns, max_new, s);
        case TQ_BF16: return kv8::append_type<__nv_bfloat16>(c, a, r ? *r : none, ns, max_new, s);
        default: return kv8::append_type<__half>(c, a, r ? *r : none, ns, max_new, s);
    }
}

extern "C" int tq_kv8_read(const tq_kv8_t* c, int layer, int ns, const int32_t* d_slots,
                           const int32_t* d_begin, const int32_t* d_cu, int64_t total, int max_new,
                           void* d_k, void* d_v, int dtype, void* stream) {
    int status;
    if (!kv8::valid(c, &status)) return status;
    if (layer < 0 || layer >= c->layers || ns < 0 || total < 0 || max_new < 0) return TQ_ERR_ARG;
    if (dtype != TQ_F32 && dtype != TQ_BF16 && dtype != TQ_F16) return TQ_ERR_ARG;
    if (!d_slots && ns > c->slots) return TQ_ERR_ARG;
    if (ns == 0 || total == 0 || max_new == 0 || (!d_k && !d_v)) return TQ_OK;
    if (!d_begin || !d_cu || (((uintptr_t)d_k | (uintptr_t)d_v) & 15u)) return TQ_ERR_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    switch (dtype) {
        case TQ_F32: return kv8::read_type<float>(c, layer, ns, d_slots, d_begin, d_cu, total, max_new, d_k, d_v, s);
        case TQ_BF16: return kv8::read_type<__nv_bfloat16>(c, layer, ns, d_slots, d_begin, d_cu, total, max_new, d_k, d_v, s);
        default: return kv8::read_type<__half>(c, layer, ns, d_slots, d_begin, d_cu, total, max_new, d_k, d_v, s);
    }
}
