// Rotary positions: for token t, head h and each pair (x1, x2) of the first
// `rot` coordinates, with angle p f_i at position p,
//   y1 = a (x1 cos - x2 sin),   y2 = a (x2 cos + x1 sin)
// (transposed: sin -> -sin), the coordinates behind copied.
//
// One pass over the data: a block takes whole tokens, forms their rot/2 cosines
// and sines once in shared memory (all heads of a token share them; no table in
// global memory, no limit on the position) and turns the heads with 16-byte
// accesses where strides and widths allow them.  Bound by HBM for many tokens
// (16383 x 32 x 128 fp32: 102 us, 5.3 TB/s), by the launch for few (64 x 32 x 128
// bf16: 2.2 us).
#include <cmath>

#include "tq_launch.cuh"
#include "tq_rope.cuh"

namespace tq {

bool rope_valid(const tq_rope_params_t* r) {
    return r && r->d >= 2 && r->d <= 256 && r->d % 2 == 0 && r->rot >= 0 && r->rot <= r->d &&
           r->rot % 2 == 0 && (r->layout == TQ_ROPE_HALF || r->layout == TQ_ROPE_INTERLEAVED);
}

namespace {

constexpr int kRT = 256;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f(float v, __half& o) { o = __float2half_rn(v); }

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
};

// VEC: elements per access (16 bytes, or 1).  SPLIT: an item is two runs of VEC
// elements, the half layout's pairs (i, i + rot/2) or with VEC = 1 an interleaved
// pair; otherwise one run.  A thread loads a batch of items before it waits for
// the angles, so the data are on their way meanwhile (and for many tokens 64 bytes
// a thread are in flight).
template <typename T, int VEC, bool SPLIT>
__global__ __launch_bounds__(kRT) void k_rope(const __grid_constant__ tq_rope_params_t r, int64_t T_,
                                              int heads, const T* x, int64_t x_ts, int64_t x_hs,
                                              const int64_t* pos, T* out, int64_t out_ts,
                                              int64_t out_hs, int transpose, int tokens, int in_place) {
    extern __shared__ float2 s_cs[];  // [tokens][rot/2]: a cos, a sin
    grid_begin();
    using P = Pack<T, VEC>;
    constexpr int N = SPLIT ? 2 : 4;  // items of a batch
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int nt = (int)min((int64_t)tokens, T_ - t0);
    const int half = r.rot / 2;
    const int turned = SPLIT ? half / VEC : r.rot / VEC;
    const int items = turned + (in_place ? 0 : (r.d - r.rot) / VEC);
    const int per = heads * items, n = nt * per;
    int64_t p0 = 0;
    if ((int)threadIdx.x < nt * half) p0 = pos[t0 + threadIdx.x / half];
    for (int i0 = threadIdx.x, first = 1; first || i0 - (int)threadIdx.x < n; i0 += N * kRT, first = 0) {
        P a[N], b[N];
        int64_t at[N];
        int o1[N], o2[N], m[N], tok[N];  // m: first pair of a turned item, -1: copied
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int i = i0 + e * kRT;
            if (i >= n) continue;
            const int t = i / per, hi = i - t * per, h = hi / items, it = hi - h * items;
            const T* xr = x + (t0 + t) * x_ts + h * x_hs;
            at[e] = (t0 + t) * out_ts + h * out_hs;
            tok[e] = t;
            if (it >= turned) {
                m[e] = -1;
                o1[e] = r.rot + (it - turned) * VEC;
            } else if (SPLIT) {
                m[e] = it * VEC;
                o1[e] = r.layout == TQ_ROPE_HALF ? m[e] : 2 * m[e];
                o2[e] = r.layout == TQ_ROPE_HALF ? m[e] + half : 2 * m[e] + 1;
                b[e] = *reinterpret_cast<const P*>(xr + o2[e]);
            } else {
                o1[e] = it * VEC;
                m[e] = it * VEC / 2;
            }
            a[e] = *reinterpret_cast<const P*>(xr + o1[e]);
        }
        if (first) {
            for (int i = threadIdx.x; i < nt * half; i += kRT) {
                const int t = i / half, k = i - t * half;
                float c, s;
                rope_angle(r.turns[k], i == (int)threadIdx.x ? p0 : pos[t0 + t], c, s);
                s_cs[i] = make_float2(c * r.amplitude, (transpose ? -s : s) * r.amplitude);
            }
            __syncthreads();
        }
#pragma unroll
        for (int e = 0; e < N; ++e) {
            if (i0 + e * kRT >= n) continue;
            if (m[e] >= 0) {
                const float2* cs = s_cs + tok[e] * half + m[e];
                if (SPLIT) {
#pragma unroll
                    for (int k = 0; k < VEC; ++k) {
                        const float x1 = to_f(a[e].v[k]), x2 = to_f(b[e].v[k]);
                        const float2 w = cs[k];
                        from_f(x1 * w.x - x2 * w.y, a[e].v[k]);
                        from_f(x2 * w.x + x1 * w.y, b[e].v[k]);
                    }
                    *reinterpret_cast<P*>(out + at[e] + o2[e]) = b[e];
                } else {
#pragma unroll
                    for (int k = 0; k + 1 < VEC; k += 2) {
                        const float x1 = to_f(a[e].v[k]), x2 = to_f(a[e].v[k + 1]);
                        const float2 w = cs[k / 2];
                        from_f(x1 * w.x - x2 * w.y, a[e].v[k]);
                        from_f(x2 * w.x + x1 * w.y, a[e].v[k + 1]);
                    }
                }
            }
            *reinterpret_cast<P*>(out + at[e] + o1[e]) = a[e];
        }
    }
}

template <typename T>
int launch(const tq_rope_params_t& r, int64_t T_, int heads, const void* x, int64_t x_ts,
           int64_t x_hs, const int64_t* pos, void* out, int64_t out_ts, int64_t out_hs,
           int transpose, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const bool wide = r.d % V == 0 && (r.layout == TQ_ROPE_HALF ? r.rot / 2 : r.rot) % V == 0 &&
                      ((uintptr_t)x | (uintptr_t)out) % 16 == 0 && x_ts % V == 0 && x_hs % V == 0 &&
                      out_ts % V == 0 && out_hs % V == 0;
    const int in_place = x == out;
    // about two accesses a thread and block: whole tokens, one at least
    const int per = heads * (wide ? r.d / V : r.d);
    int tokens = per >= 2 * kRT ? 1 : (2 * kRT + per - 1) / per;
    if (tokens > 16) tokens = 16;
    const int64_t blocks = (T_ + tokens - 1) / tokens;
    if (blocks > 0x7fffffff) return TQ_ERR_UNSUPPORTED;
    const size_t smem = (size_t)tokens * (r.rot / 2) * sizeof(float2);
    auto kernel = !wide ? k_rope<T, 1, true>
                  : r.layout == TQ_ROPE_HALF ? k_rope<T, V, true> : k_rope<T, V, false>;
    return launch_behind(kernel, dim3((unsigned)blocks), kRT, smem, s, r, T_, heads, (const T*)x, x_ts, x_hs,
                         pos, (T*)out, out_ts, out_hs, transpose, tokens, in_place);
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" int tq_build_rope(int d, int rot, double base, int layout, int scaling, double factor,
                             double ctx, double low, double high, double amplitude,
                             tq_rope_params_t* r) {
    if (!r || (layout != TQ_ROPE_HALF && layout != TQ_ROPE_INTERLEAVED)) return TQ_ERR_ARG;
    if (scaling < TQ_ROPE_PLAIN || scaling > TQ_ROPE_PARTS) return TQ_ERR_ARG;
    if (d < 2 || d > 256 || d % 2 || rot < 0 || rot > d || rot % 2) return TQ_ERR_UNSUPPORTED;
    if (!std::isfinite(base) || base <= 1.0 || !std::isfinite(amplitude) ||
        !std::isfinite((float)amplitude))
        return TQ_ERR_ARG;
    if (scaling != TQ_ROPE_PLAIN && (!std::isfinite(factor) || factor < 1.0)) return TQ_ERR_ARG;
    if (scaling == TQ_ROPE_NTK && rot < 4) return TQ_ERR_UNSUPPORTED;
    if (scaling == TQ_ROPE_PARTS && (!std::isfinite(ctx) || ctx <= 0.0 || !std::isfinite(low) ||
                                     !std::isfinite(high) || low >= high))
        return TQ_ERR_ARG;
    // (long double: 64 bits of mantissa, for positions far out)
    const long double two_pi = 6.283185307179586476925286766559L;
    tq_rope_params_t p = {};
    p.d = d;
    p.rot = rot;
    p.layout = layout;
    p.amplitude = (float)amplitude;
    long double b = base;
    if (scaling == TQ_ROPE_NTK) b *= std::pow((long double)factor, (long double)rot / (rot - 2));
    if (b > 1.7976931348623157e308L) return TQ_ERR_ARG;
    for (int i = 0; i < rot / 2; ++i) {
        long double f = std::pow(b, -2.0L * i / rot);
        if (scaling == TQ_ROPE_LINEAR) f /= factor;
        if (scaling == TQ_ROPE_PARTS) {
            long double g = (ctx * f / two_pi - low) / ((long double)high - low);
            g = g < 0.0L ? 0.0L : (g > 1.0L ? 1.0L : g);
            f *= g + (1.0L - g) / factor;
        }
        // 0 < f <= 1 radian: below 1/6 turn
        p.turns[i] = (uint64_t)std::llrint(std::ldexp(f / two_pi, 64));
    }
    *r = p;
    return TQ_OK;
}

extern "C" int tq_rope(const tq_rope_params_t* r, int64_t T, int heads, const void* d_x,
                       int64_t x_ts, int64_t x_hs, int x_dtype, const int64_t* d_pos, void* d_out,
                       int64_t out_ts, int64_t out_hs, int transpose, void* stream) {
    if (!r || T < 0 || heads < 1 || transpose < 0 || transpose > 1) return TQ_ERR_ARG;
    if (x_dtype != TQ_F32 && x_dtype != TQ_BF16 && x_dtype != TQ_F16) return TQ_ERR_ARG;
    if (!rope_valid(r)) return TQ_ERR_ARG;
    if (T == 0) return TQ_OK;
    if (!d_x || !d_pos || !d_out) return TQ_ERR_ARG;
    if (d_x == d_out && (x_ts != out_ts || x_hs != out_hs)) return TQ_ERR_ARG;
    // a block indexes its tokens' heads in 32 bits
    if ((int64_t)heads * r->d > ((int64_t)1 << 26)) return TQ_ERR_UNSUPPORTED;
    cudaStream_t s = (cudaStream_t)stream;
    switch (x_dtype) {
        case TQ_F32: return launch<float>(*r, T, heads, d_x, x_ts, x_hs, d_pos, d_out, out_ts, out_hs, transpose, s);
        case TQ_BF16: return launch<__nv_bfloat16>(*r, T, heads, d_x, x_ts, x_hs, d_pos, d_out, out_ts, out_hs, transpose, s);
        default: return launch<__half>(*r, T, heads, d_x, x_ts, x_hs, d_pos, d_out, out_ts, out_hs, transpose, s);
    }
}
