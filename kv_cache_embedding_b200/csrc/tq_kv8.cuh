// The 8-bit paged KV cache inside the kernels: geometry, code conversions.
#pragma once

#include <cuda_fp8.h>

#include "tq_internal.cuh"
#include "tq_launch.cuh"

namespace tq {
namespace kv8 {

// A layer of the cache by value (kernel parameter).
struct View {
    int d, heads, page, page_log2, slots, max_pages, pages;
    const int32_t* table;
    const int32_t* len;
    int32_t* status;  // may be null
};

// tq_kv8_t's limits; null pointers where `pointers` is set.
bool valid(const tq_kv8_t* c, int* status);

inline int log2_of(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }

inline View view(const tq_kv8_t* c) {
    View v;
    v.d = c->d;
    v.heads = c->heads;
    v.page = c->page;
    v.page_log2 = log2_of(c->page);
    v.slots = c->slots;
    v.max_pages = c->max_pages;
    v.pages = c->pages;
    v.table = c->d_table;
    v.len = c->d_len;
    v.status = c->d_status;
    return v;
}

// Bytes (codes) and scales of one layer of one pool.
inline int64_t layer_bytes(const tq_kv8_t* c) {
    return (int64_t)c->pages * c->heads * c->page * c->d;
}
inline int64_t layer_scales(const tq_kv8_t* c) { return (int64_t)c->pages * c->heads; }

// The cache's status: 0 where nothing has gone wrong.  A block looks at it once (one
// barrier, or one thread): a call on another stream may set it meanwhile.
__device__ __forceinline__ int pending(const View& v) {
    return v.status ? *(const volatile int32_t*)v.status : 0;
}
// The first one stands.
__device__ __forceinline__ void leave_status(const View& v, int status) {
    if (v.status) atomicCAS(v.status, 0, status);
}

// Slot of batch entry i, or -1; its length, limited to what its table can name.
__device__ __forceinline__ int slot_of(const View& v, const int32_t* slots, int i) {
    const int s = slots ? slots[i] : i;
    return (unsigned)s < (unsigned)v.slots ? s : -1;
}
__device__ __forceinline__ int length_of(const View& v, int slot) {
    const int64_t most = (int64_t)v.max_pages << v.page_log2;
    const int n = v.len[slot];
    return n < 0 ? 0 : (int)(n < most ? n : most);
}
// Page id of page j of a slot, or -1.
__device__ __forceinline__ int page_of(const View& v, int slot, int j) {
    const int p = v.table[(int64_t)slot * v.max_pages + j];
    return (unsigned)p < (unsigned)v.pages ? p : -1;
}

// Four int8 codes (a word) -> two half2 (bytes 0, 1 | bytes 2, 3), exact: with
// the sign bit flipped a byte is x + 128, and 0x64 above it makes the half
// 1024 + x + 128.
__device__ __forceinline__ uint32_t hsub2_1152(uint32_t h) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(0x64806480u));
    return r;
}
// e4m3 pair (16 bits) -> half2, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t v) {
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(v));
    return r;
}
template <int FMT>
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if (FMT == TQ_KV_I8) {
        w ^= 0x80808080u;
        lo = hsub2_1152(__byte_perm(w, 0x64646464u, 0x4140));
        hi = hsub2_1152(__byte_perm(w, 0x64646464u, 0x4342));
    } else {
        lo = e4m3x2_to_half2(w);
        hi = e4m3x2_to_half2(w >> 16);
    }
}
// The same with bytes (0, 2) and (1, 3) paired.
template <int FMT>
__device__ __forceinline__ void codes_to_half_02(uint32_t w, uint32_t& b02, uint32_t& b13) {
    if (FMT == TQ_KV_I8) {
        w ^= 0x80808080u;
        b02 = hsub2_1152(__byte_perm(w, 0x64646464u, 0x4240));
        b13 = hsub2_1152(__byte_perm(w, 0x64646464u, 0x4341));
    } else {
        w = __byte_perm(w, 0u, 0x3120);
        b02 = e4m3x2_to_half2(w);
        b13 = e4m3x2_to_half2(w >> 16);
    }
}

template <int FMT>
__host__ __device__ constexpr float code_max() { return FMT == TQ_KV_I8 ? 127.f : 448.f; }

// The nearest codes of four quotients x / s (ties to even): x times the fp32
// reciprocal, off by 2^-23 of itself, so a code differs from the exact quotient's
// only where that lies as close to the middle between two codes.  |x| <= s
// code_max but for 2^-24 of it, so that nothing leaves the codes' range.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(float x0, float x1, float x2, float x3, float inv) {
    if (FMT == TQ_KV_I8) {
        // behind 1.5 2^23 the last bits of a sum are the integer, rounded by the addition
        const uint32_t a = __float_as_uint(fmaf(x0, inv, 12582912.f)), b = __float_as_uint(fmaf(x1, inv, 12582912.f));
        const uint32_t c = __float_as_uint(fmaf(x2, inv, 12582912.f)), d = __float_as_uint(fmaf(x3, inv, 12582912.f));
        return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
    }
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x0 * inv, x1 * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x2 * inv, x3 * inv), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}
__device__ __forceinline__ float2 half2_to_f(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2*>(&h)); }
// Four codes' values, exact.
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t w, float (&x)[4]) {
    uint32_t lo, hi;
    codes_to_half<FMT>(w, lo, hi);
    const float2 a = half2_to_f(lo), b = half2_to_f(hi);
    x[0] = a.x;
    x[1] = a.y;
    x[2] = b.x;
    x[3] = b.y;
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f(float v, __half& o) { o = __float2half_rn(v); }

template <typename T, int VEC>
struct alignas((sizeof(T) * VEC) < 16 ? (sizeof(T) * VEC) : 16) Pack {
    T v[VEC];
};

// Attention workspaces (tq_kv8_attention.cu).
size_t attention_workspace(const tq_kv8_t* c, int ns, int64_t total_q, int max_q, int heads_q);
size_t pages_workspace(const tq_kv8_t* c, int n);

}  // namespace kv8
}  // namespace tq
