// The 8-bit paged KV cache: geometry, writing tokens and reading them back.
//
// Write (tq_kv8_append): for every page and head that new tokens fall into,
//   s = max(s0, max |x| / M)   (s0: the scale of the tokens there already, if any)
//   code = rnd(x / s),         old codes: rnd(code s0 / s) where s > s0,
// keys turned to their positions first (fp32, not rounded in between).
//
// A block owns one (slot, page, head) of K or V, so the page's maximum is a
// block reduction and nothing is written twice: its new rows are loaded once
// into registers (16 elements an item), turned, reduced, rounded and stored;
// the page's old rows are touched only when the scale grows.  Bound by HBM for
// prompts, by the chain length -> table -> scale for single tokens.
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
    int64_t total;
    const void *x[2];
    int64_t x_ts, x_hs;
    uint8_t* codes[2];
    float* scale[2];
    int rope;
};

constexpr float kLargest = 1.7014118e38f;  // 2^127

// The larger one, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// NI items of 2 VEC elements a thread; VEC = 8 (16-byte accesses) or 1.
template <typename T, int FMT, int VEC, int NI>
__global__ __launch_bounds__(256) void k_append(const AppendArgs a,
                                                const __grid_constant__ tq_rope_params_t rope) {
    __shared__ float s_red[8];
    grid_begin();
    const View& v = a.v;
    const int seq = blockIdx.x / a.ppb, pj = blockIdx.x - seq * a.ppb;
    const int h = blockIdx.y, kv = blockIdx.z;
    const int slot = slot_of(v, a.slots, seq);
    if (slot < 0) return;
    const int64_t c0 = max(a.cu[seq], 0);
    const int count = (int)(min((int64_t)a.cu[seq + 1], a.total) - c0);
    const int len = length_of(v, slot);
    if (count <= 0) return;
    // tokens before the slot's first position have no place
    const int start = max(len - count, 0), skip = max(count - len, 0);
    const int page0 = start >> v.page_log2;
    const int lo_pos = max(start, (page0 + pj) << v.page_log2);
    const int hi_pos = min(len, (page0 + pj + 1) << v.page_log2);
    if (lo_pos >= hi_pos) return;
    const int pid = page_of(v, slot, page0 + pj);
    if (pid < 0) return;
    const int row0 = lo_pos & (v.page - 1), rows = hi_pos - lo_pos;
    const int64_t ph = (int64_t)pid * v.heads + h;
    uint8_t* codes = a.codes[kv] + (ph << v.page_log2) * v.d;
    const T* x = (const T*)a.x[kv] + (c0 + skip + lo_pos - start) * a.x_ts + h * a.x_hs;
    const float s_old = row0 > 0 ? a.scale[kv][ph] : 0.f;
    const bool turn = kv == 0 && a.rope;

    const int per = v.d / (2 * VEC);  // items of a row
    const int n = rows * per;
    const int rot = turn ? rope.rot : 0, half = rot / 2;
    const bool halves = turn && rope.layout == TQ_ROPE_HALF;
    float val[NI][2 * VEC];
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int it = threadIdx.x + i * blockDim.x;
        if (it < n) {
            const int row = it / per, m = it - row * per;
            // the two runs of the item: a half-layout pair block, or neighbours
            const bool pair = halves && m * VEC < half;
            const int o1 = pair ? m * VEC : 2 * m * VEC;
            const int o2 = pair ? m * VEC + half : o1 + VEC;
            const T* xr = x + row * a.x_ts;
            if (VEC == 8) {
                const Pack<T, VEC> p1 = *reinterpret_cast<const Pack<T, VEC>*>(xr + o1);
                const Pack<T, VEC> p2 = *reinterpret_cast<const Pack<T, VEC>*>(xr + o2);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    val[i][e] = to_f(p1.v[e]);
                    val[i][VEC + e] = to_f(p2.v[e]);
                }
            } else {
                val[i][0] = to_f(xr[o1]);
                val[i][1] = to_f(xr[o2]);
            }
            if (turn) {
                const int64_t pos = lo_pos + row;
                if (pair || VEC == 1) {
                    if (pair || (!halves && o1 < rot)) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            float c, s;
                            rope_angle(rope.turns[pair ? m * VEC + e : m], pos, c, s);
                            const float x1 = val[i][e], x2 = val[i][VEC + e];
                            val[i][e] = rope.amplitude * (x1 * c - x2 * s);
                            val[i][VEC + e] = rope.amplitude * (x2 * c + x1 * s);
                        }
                    }
                } else if (!halves) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {  // pairs of the 2 VEC neighbours
                        if (o1 + 2 * e < rot) {
                            float c, s;
                            rope_angle(rope.turns[m * VEC + e], pos, c, s);
                            const float x1 = val[i][(2 * e) % (2 * VEC)], x2 = val[i][(2 * e + 1) % (2 * VEC)];
                            val[i][(2 * e) % (2 * VEC)] = rope.amplitude * (x1 * c - x2 * s);
                            val[i][(2 * e + 1) % (2 * VEC)] = rope.amplitude * (x2 * c + x1 * s);
                        }
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 2 * VEC; ++e) top = max_nan(top, fabsf(val[i][e]));
        }
    }
    if (!(top <= kLargest)) {  // NaN: 0; up to 2^127, so that scale x code stays finite
        top = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if ((int)(threadIdx.x + i * blockDim.x) >= n) continue;
#pragma unroll
            for (int e = 0; e < 2 * VEC; ++e) {
                const float y = val[i][e];
                val[i][e] = y == y ? fminf(fmaxf(y, -kLargest), kLargest) : 0.f;
                top = fmaxf(top, fabsf(val[i][e]));
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = top;
    __syncthreads();
    for (int w = 0; w < (int)blockDim.x / 32; ++w) top = fmaxf(top, s_red[w]);
    const float s = fmaxf(s_old, __fdiv_rn(top, code_max<FMT>()));
    if (threadIdx.x == 0) a.scale[kv][ph] = s;
    // (below fp32's normal range a reciprocal may overflow: all times 2^64)
    const float up = s < 1.17549435e-38f ? 18446744073709551616.f : 1.f;
    const float inv = s > 0.f ? __frcp_rn(s * up) : 0.f;
    if (up != 1.f) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int e = 0; e < 2 * VEC; ++e) val[i][e] *= up;
    }

#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int it = threadIdx.x + i * blockDim.x;
        if (it < n) {
            const int row = it / per, m = it - row * per;
            const bool pair = halves && m * VEC < half;
            const int o1 = pair ? m * VEC : 2 * m * VEC;
            const int o2 = pair ? m * VEC + half : o1 + VEC;
            uint8_t* cr = codes + (row0 + row) * v.d;
            if (VEC == 8) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = encode4<FMT>(val[i][4 * e % (2 * VEC)], val[i][(4 * e + 1) % (2 * VEC)],
                                        val[i][(4 * e + 2) % (2 * VEC)], val[i][(4 * e + 3) % (2 * VEC)], inv);
                *reinterpret_cast<uint2*>(cr + o1) = make_uint2(w[0], w[1]);
                *reinterpret_cast<uint2*>(cr + o2) = make_uint2(w[2], w[3]);
            } else {
                const uint32_t w = encode4<FMT>(val[i][0], val[i][1], 0.f, 0.f, inv);
                cr[o1] = (uint8_t)w;
                cr[o2] = (uint8_t)(w >> 8);
            }
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
                    float x[4];
                    decode4<FMT>(y[k], x);
                    y[k] = encode4<FMT>(x[0], x[1], x[2], x[3], f);
                }
                w[i0 + e * blockDim.x] = make_uint4(y[0], y[1], y[2], y[3]);
            }
        }
    }
}

template <typename T, int FMT, int VEC, int NI>
int append_go(const AppendArgs& a, const tq_rope_params_t& r, int ns, int threads, cudaStream_t s) {
    const int64_t gx = (int64_t)ns * a.ppb;
    if (gx > 0x7fffffff) return TQ_ERR_UNSUPPORTED;
    return launch_behind(k_append<T, FMT, VEC, NI>, dim3((unsigned)gx, (unsigned)a.v.heads, 2), threads, 0,
                         s, a, r);
}

// Threads and items a thread for the most rows that a block can get.
template <typename T, int FMT>
int append_fmt(const AppendArgs& a, const tq_rope_params_t& r, int ns, int max_new, bool wide,
               cudaStream_t s) {
    const int rows = max_new < a.v.page ? max_new : a.v.page;
    if (wide) {
        const int items = rows * a.v.d / 16;
        if (items <= 128) return append_go<T, FMT, 8, 1>(a, r, ns, 128, s);
        if (items <= 256) return append_go<T, FMT, 8, 1>(a, r, ns, 256, s);
        if (items <= 512) return append_go<T, FMT, 8, 2>(a, r, ns, 256, s);
        return append_go<T, FMT, 8, 4>(a, r, ns, 256, s);
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
// The lookups of a thread's items, then their codes, are on their way together.
template <typename T, int FMT>
__global__ __launch_bounds__(kReadThreads) void k_read(View v, const int32_t* slots, const int32_t* begin,
                                                       const int32_t* cu, int bps, int tokens, int64_t total,
                                                       const uint8_t* kc, const uint8_t* vc, const float* ks,
                                                       const float* vs, T* out_k, T* out_v) {
    grid_begin();
    const int seq = blockIdx.x / bps, blk = blockIdx.x - seq * bps;
    const int slot = slot_of(v, slots, seq);
    const int64_t c0 = max(cu[seq], 0), c1 = min((int64_t)cu[seq + 1], total);
    const int64_t b = (int64_t)begin[seq] + (int64_t)blk * tokens;
    const int len = slot >= 0 ? length_of(v, slot) : 0;
    const int nt = (int)min((int64_t)tokens, c1 - c0 - (int64_t)blk * tokens);
    if (nt <= 0) return;
    const int chunks = v.d / 16, per = v.heads * chunks, n = nt * per;
    const bool is_v = blockIdx.y != 0;
    T* out = is_v ? out_v : out_k;
    if (!out) return;
    const uint8_t* codes = is_v ? vc : kc;
    const float* scales = is_v ? vs : ks;
    // (items of a block are neighbours in the output: token, head, chunk)
    Pack<T, 8>* dst = reinterpret_cast<Pack<T, 8>*>(out + (c0 + (int64_t)blk * tokens) * v.heads * v.d);
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

template <typename T>
int read_type(const tq_kv8_t* c, int layer, int ns, const int32_t* slots, const int32_t* begin,
              const int32_t* cu, int64_t total, int max_new, void* k, void* v, cudaStream_t s) {
    // a batch of items a thread, or fewer tokens a block where that leaves SMs idle
    const int per = c->heads * c->d / 16;
    int64_t tokens = kReadItems * kReadThreads / per, fill = (int64_t)ns * max_new / (148 * 2);
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
                         kReadThreads, 0, s, view(c), slots, begin, cu, (int)bps, (int)tokens, total, kc, vc,
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
