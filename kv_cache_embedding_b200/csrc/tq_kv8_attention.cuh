// Attention over the 8-bit paged cache: what its kernels share.
#pragma once

#include <cuda.h>

#include "tq_kv8.cuh"
#include "tq_sm100.cuh"

namespace tq {
namespace kv8 {

// One call (kernel parameter).
struct Attn {
    View v;
    int ns, group, heads_q, causal, window;
    const int32_t* slots;
    const int32_t* cu;
    int64_t total_q;
    const void* q;
    int64_t q_ts, q_hs;
    float scale_log2;  // scale * log2(e)
    const float *ks, *vs;  // [pages][heads] of the layer
    void* out;
    float* lse;
    int behind;  // rows behind the last entry's become 0
    int rows;  // rows of the layer's pools: pages * heads * page
    int max_q; // tokens of an entry at most, where the prompt kernel is not launched
    int few;   // entries of up to `few` query rows (tokens x group) run on the few-rows
               // kernel, the others on the prompt kernel (0: all of them)
};

// An item that its CTA begins and others go on with: who joins what.
struct Cut {
    int parts;       // CTAs that share the item which begins here; 0: none
    int rows, head;  // its rows and KV head
    int pad;
    int64_t row0;    // its first row of the entry's (token x group) rows, from token 0
};

// The prompt kernel's workspace.  Part 2u: the end of an item that CTA u did not
// begin; 2u + 1: the beginning of one that it does not end.
struct PromptParts {
    int* status;
    int keep_status;   // the few-rows kernel runs before and owns the word
    int* block_status;
    Cut* cut;
    float2* ml;        // (m, L) of 256 rows a part
    float* o;          // 256 x d a part
};
int prompt_blocks(const tq_kv8_t* c, int ns, int64_t total_q, int heads_q);
PromptParts prompt_carve(const tq_kv8_t* c, void* ws, int blocks, size_t* bytes);
int launch_prompt(const tq_kv8_t* c, int layer, const Attn& a, const PromptParts& p, int blocks,
                  int q_dtype, cudaStream_t s);

// A batch entry as the kernels see it.
struct Entry {
    int slot, len, qn;
    int64_t c0;  // first query token
};
__device__ __forceinline__ Entry entry_of(const Attn& a, int i) {
    Entry e;
    e.slot = slot_of(a.v, a.slots, i);
    const int64_t c0 = a.cu[i], c1 = min((int64_t)a.cu[i + 1], a.total_q);
    e.c0 = c0;
    e.qn = c0 >= 0 && c1 > c0 ? (int)(c1 - c0) : 0;
    e.len = e.slot >= 0 ? length_of(a.v, e.slot) : 0;
    return e;
}
// A batch that does not fit the call's sizes, which the host cannot see: more tokens
// than q has, or an entry that none of the launched kernels takes.
__device__ __forceinline__ bool misfit(const Attn& a, int i, const Entry& e) {
    return a.cu[i + 1] > a.total_q || e.qn > a.max_q;
}

// A refused call, or one that finds the cache's status set: no row sees a key.  (All of
// the grid's threads; a block that saw the word before it was set may write rows too.)
template <int D, typename T>
__device__ __forceinline__ void empty_rows(const Attn& a) {
    const int64_t t0 = max(a.cu[0], 0), rows = (min((int64_t)a.cu[a.ns], a.total_q) - t0) * a.heads_q;
    const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    const int64_t at = block * blockDim.x + threadIdx.x, step = (int64_t)gridDim.x * gridDim.y * blockDim.x;
    uint4* out = reinterpret_cast<uint4*>((T*)a.out + t0 * a.heads_q * D);
    for (int64_t i = at; i < rows * (D / 8); i += step) out[i] = make_uint4(0, 0, 0, 0);
    if (a.lse)
        for (int64_t i = at; i < rows; i += step) a.lse[t0 * a.heads_q + i] = -INFINITY;
}

// Rows behind the last entry's (all of the grid's threads; the first kernel of a call).
template <int D, typename T>
__device__ __forceinline__ void zero_behind(const Attn& a, int used) {
    const int64_t row = (int64_t)a.heads_q * (D / 8);  // 16-byte pieces of a token
    const int64_t at = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, step = (int64_t)gridDim.x * blockDim.x;
    uint4* out = reinterpret_cast<uint4*>(a.out);
    for (int64_t i = used * row + at; i < a.total_q * row; i += step) out[i] = make_uint4(0, 0, 0, 0);
}

// First key that any query of the entry sees.
__device__ __forceinline__ int first_key(const Attn& a, const Entry& e) {
    return a.window > 0 ? (int)max((int64_t)0, (int64_t)e.len - e.qn - a.window + 1) : 0;
}
// The last key that the query at position pos does not see for the window.
__device__ __forceinline__ int below_window(const Attn& a, int pos) {
    return a.window > 0 ? (int)max((int64_t)-1, (int64_t)pos - a.window) : -1;
}

// Quotient of non-negative numbers; 64-bit division is a subroutine of some
// hundred cycles, and the numbers mostly fit 32.
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
    return ((uint64_t)a | (uint64_t)b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The exponent e of a value scale, 2^e <= s < 2^(e + 1) (below fp32's normal range
// -127, an upper bound still); -infinity for 0.  2^e of a whole number from -126 to 127:
// behind 1.5 2^23 the last bits of a sum are the integer.
__device__ __forceinline__ float scale_exp(float s) {
    return s > 0.f ? (float)((int)(__float_as_uint(s) >> 23) - 127) : -INFINITY;
}
__device__ __forceinline__ float pow2(float e) { return __uint_as_float(__float_as_uint(e + 12583039.f) << 23); }
constexpr float kLargestFloat = 3.40282347e38f;

// Units of a row: probabilities are 2^(l - m), their products with the value scales are
// summed as P s_v 2^up.  m and up are whole numbers that follow when a probability
// passes 2^kGrow or a product 2^kRoom (a half ends at 2^16).  Before a row's first key m
// is kNoKey: what there is of sums is multiplied by 0 then.
constexpr float kGrow = 8.f, kRoom = 14.f, kNoKey = -1e38f;
// From up, the change of m and the largest log2 (P s_v) + m - m_new among new keys (off
// by up to one), the new up; start: where the largest product is put.  (A row whose
// values are far below its probabilities: as far as fp32 goes.)
__device__ __forceinline__ float new_up(float follow, float top, float start) {
    return fminf(top + follow > kRoom ? start - ceilf(top) : follow, 100.f);
}

// The power of two that brings a row's largest magnitude into [2^15, 2^16), the top
// of a half's range: with it a row of bf16 is a row of halves, exact down to 2^-32 of
// the largest and within 2^-40 of it below; a row of f16 is never divided, so exact.
// (A row below 2^-111 comes to less: 2^126 is the largest unit.)
__device__ __forceinline__ float row_unit(float top) {
    int e = (int)(__float_as_uint(top) >> 23);
    e = min(max(e, 16), 254);
    return __uint_as_float((uint32_t)(269 - e) << 23);
}

constexpr uint64_t kWaitNs = 1000000000ull;

// Tensor map of a layer's code rows: [pages * heads * page][d] bytes, boxes of
// `box` rows, swizzled over a whole row (128 or 64 bytes).
int code_map(CUtensorMap* m, const void* base, int d, int64_t rows, int box);

}  // namespace kv8
}  // namespace tq
