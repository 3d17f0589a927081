// Page operations of the 8-bit cache: reserve (with copy on write), fork,
// truncate, compact.
//
// Each is a plan by ONE block (a list of at most 4096 slots, the reference
// counts of the pool), which checks everything before it changes anything and
// hands out pages in ascending order by prefix sums -- no atomics decide an
// order, so a result is the same every time -- and, where pages move, one copy
// kernel over (page pair, layer, K or V) whose pairs and their number it reads
// from the workspace.  The plan is bound by a few dependent passes over lists
// that sit in L2 (3 us; 8 with copies to plan), the copies by HBM (5.3 TB/s).
#include "tq_kv8.cuh"

namespace tq {
namespace kv8 {

constexpr int kPT = 1024;      // threads of the plan
constexpr int kMaxList = 4096;
constexpr int kPer = kMaxList / kPT;

// [status, pair count (int32 x 2) | pairs: src, dst [m] each | marks [slots] |
//  free pages / remap [pages]], m = max(n, pages / 2 for compact)
struct PagesWs {
    int* head;
    int32_t *src, *dst, *marks, *ids;
};

static size_t pairs_of(const tq_kv8_t* c, int n) {
    const size_t half = (size_t)c->pages / 2 + 1;  // compact: at most half the pages move
    return (size_t)n > half ? (size_t)n : half;
}

size_t pages_workspace(const tq_kv8_t* c, int n) {
    return 256 + 2 * align256(pairs_of(c, n) * 4) + align256((size_t)c->slots * 4) +
           align256((size_t)c->pages * 4);
}

static PagesWs carve(const tq_kv8_t* c, int n, void* ws) {
    PagesWs w;
    char* p = (char*)ws;
    w.head = (int*)p;
    p += 256;
    w.src = (int32_t*)p;
    p += align256(pairs_of(c, n) * 4);
    w.dst = (int32_t*)p;
    p += align256(pairs_of(c, n) * 4);
    w.marks = (int32_t*)p;
    p += align256((size_t)c->slots * 4);
    w.ids = (int32_t*)p;
    return w;
}

namespace {

// Exclusive prefix sum over the block's threads; total in *all.  `tmp`: 33 words.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* tmp, int64_t* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) tmp[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        const int64_t w = tmp[lane];
        int64_t s = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        tmp[lane] = s - w;
        if (lane == 31) tmp[32] = s;
    }
    __syncthreads();
    const int64_t r = tmp[warp] + inc - x;
    *all = tmp[32];
    __syncthreads();
    return r;
}

// Thread 0 gives a plan up: the status that held already, or a new one.
__device__ __forceinline__ void refuse(const View& v, const PagesWs& w, int held, int status) {
    w.head[0] = held ? held : status;
    if (!held) leave_status(v, status);
}

__device__ __forceinline__ int pages_for(const View& v, int64_t tokens) {
    return (int)((tokens + v.page - 1) >> v.page_log2);
}

// Whether a slot is twice in the list, or one of `others` (may be null) is in it.
// Short lists are compared entry by entry in shared memory; a long one is counted
// in the workspace (marks: one word a slot, any contents).  Ends with a barrier.
constexpr int kShortList = 256;
__device__ __forceinline__ bool repeated(const View& v, const int32_t* slots, const int32_t* others, int n,
                                         int32_t* marks) {
    __shared__ int32_t s_list[kShortList];
    bool bad = false;
    if (n <= kShortList) {
        const int i = threadIdx.x % kShortList;
        if ((int)threadIdx.x < n) s_list[i] = slots[i];
        const int other = others && i < n ? others[i] : 0;
        __syncthreads();
        if (i < n)
            for (int j = threadIdx.x / kShortList; j < n; j += kPT / kShortList)
                bad |= (j != i && s_list[j] == s_list[i]) || (others && s_list[j] == other);
        return __syncthreads_or(bad) != 0;
    }
    for (int i = threadIdx.x; i < n; i += kPT) {
        if ((unsigned)slots[i] < (unsigned)v.slots) marks[slots[i]] = 0;
        if (others && (unsigned)others[i] < (unsigned)v.slots) marks[others[i]] = 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPT)
        if ((unsigned)slots[i] < (unsigned)v.slots) bad |= atomicAdd(&marks[slots[i]], 1) != 0;
    __syncthreads();
    if (others)
        for (int i = threadIdx.x; i < n; i += kPT)
            if ((unsigned)others[i] < (unsigned)v.slots) bad |= marks[others[i]] != 0;
    return __syncthreads_or(bad) != 0;
}

__global__ __launch_bounds__(kPT) void k_reserve(View v, int32_t* table, int32_t* len,
                                                 int32_t* refs, int n,
                                                 const int32_t* slots,
                                                 const int32_t* counts, PagesWs w) {
    __shared__ int64_t tmp[33];
    __shared__ int32_t s_held[kMaxList];  // the shared page that entry i writes into, or -1
    __shared__ int32_t s_base[kMaxList];  // first of the entry's new pages
    grid_begin();
    const int per = (n + kPT - 1) / kPT;  // entries of a thread
    const int held_status = threadIdx.x == 0 ? pending(v) : 0;
    bool bad = repeated(v, slots, nullptr, n, w.marks) || held_status;
    if (threadIdx.x == 0) w.head[1] = 0;
    int at[kPer], more[kPer], need[kPer];
    bool shared_page = false;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int i = threadIdx.x * per + e;  // neighbours: list order is thread order
        at[e] = more[e] = need[e] = 0;
        int held = -1;
        if (e < per && i < n) {
            const int s = slots[i], add = counts[i];
            if ((unsigned)s >= (unsigned)v.slots || add < 0) {
                bad = true;
            } else {
                at[e] = length_of(v, s);
                more[e] = add;
                if ((int64_t)at[e] + add > ((int64_t)v.max_pages << v.page_log2)) bad = true;
                else need[e] = pages_for(v, (int64_t)at[e] + add) - pages_for(v, at[e]);
                if (add > 0 && (at[e] & (v.page - 1))) {
                    held = page_of(v, s, at[e] >> v.page_log2);
                    if (held >= 0 && refs[held] <= 1) held = -1;
                    shared_page |= held >= 0;
                }
            }
        }
        if (e < per && i < n) s_held[i] = held;
    }
    // an entry copies unless the entries before it leave it the last holder
    unsigned copy = 0;
    if (__syncthreads_or(shared_page)) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int i = threadIdx.x * per + e;
            if (e < per && i < n && s_held[i] >= 0) {
                int before = 0;
                for (int j = 0; j < i; ++j) before += s_held[j] == s_held[i];
                if (refs[s_held[i]] - before > 1) {
                    copy |= 1u << e;
                    ++need[e];
                }
            }
        }
    }
    int64_t mine = 0, total, ncopy;
#pragma unroll
    for (int e = 0; e < kPer; ++e) mine += need[e];
    int64_t base = block_scan(mine, tmp, &total);
    const int64_t cbase = block_scan(__popc(copy), tmp, &ncopy);
    // the lowest `total` free pages
    int64_t found = 0;
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) refuse(v, w, held_status, TQ_ERR_ARG);
        return;
    }
    for (int64_t p0 = 0; p0 < v.pages && found < total; p0 += 4 * kPT) {
        int flag[4], cnt = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t p = p0 + threadIdx.x * 4 + e;
            flag[e] = p < v.pages && refs[p] == 0;
            cnt += flag[e];
        }
        int64_t got;
        int64_t o = found + block_scan(cnt, tmp, &got);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (flag[e]) {
                if (o < total) w.ids[o] = (int32_t)(p0 + threadIdx.x * 4 + e);
                ++o;
            }
        found += got;
    }
    if (found < total) {
        if (threadIdx.x == 0) refuse(v, w, 0, TQ_ERR_PAGES);
        return;
    }
    __syncthreads();
    // hand them out
    int64_t b = base, ci = cbase;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int i = threadIdx.x * per + e;
        if (e < per && i < n) {
            const int s = slots[i];
            if (copy >> e & 1u) {
                const int dst = w.ids[b], src = s_held[i];
                table[(int64_t)s * v.max_pages + (at[e] >> v.page_log2)] = dst;
                refs[dst] = 1;
                atomicSub(&refs[src], 1);
                w.src[ci] = src;
                w.dst[ci] = dst;
                ++ci;
            }
            s_base[i] = (int32_t)b + (copy >> e & 1u);
            b += need[e];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x >> 5; i < n; i += kPT / 32) {  // a warp an entry
        const int s = slots[i], from = length_of(v, s);
        const int p0 = pages_for(v, from), p1 = pages_for(v, (int64_t)from + counts[i]);
        for (int p = p0 + (threadIdx.x & 31); p < p1; p += 32) {
            const int id = w.ids[s_base[i] + p - p0];
            table[(int64_t)s * v.max_pages + p] = id;
            refs[id] = 1;
        }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int i = threadIdx.x * per + e;
        if (e < per && i < n) len[slots[i]] = at[e] + more[e];
    }
    if (threadIdx.x == 0) {
        w.head[0] = TQ_OK;
        w.head[1] = (int)ncopy;
    }
}

__global__ __launch_bounds__(kPT) void k_fork(View v, int32_t* table, int32_t* len, int32_t* refs,
                                              int n, const int32_t* parents,
                                              const int32_t* children, PagesWs w) {
    grid_begin();
    const int held = threadIdx.x == 0 ? pending(v) : 0;
    bool bad = repeated(v, children, parents, n, w.marks) || held;
    for (int i = threadIdx.x; i < n; i += kPT) {
        const int p = parents[i], c = children[i];
        if ((unsigned)p >= (unsigned)v.slots || (unsigned)c >= (unsigned)v.slots) bad = true;
        else bad |= len[c] != 0;
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) refuse(v, w, held, TQ_ERR_ARG);
        return;
    }
    for (int i = threadIdx.x >> 5; i < n; i += kPT / 32) {
        const int ps = parents[i], cs = children[i], from = length_of(v, ps);
        for (int p = threadIdx.x & 31; p < pages_for(v, from); p += 32) {
            const int id = page_of(v, ps, p);
            table[(int64_t)cs * v.max_pages + p] = id;
            if (id >= 0) atomicAdd(&refs[id], 1);
        }
        if ((threadIdx.x & 31) == 0) len[cs] = from;
    }
    if (threadIdx.x == 0) w.head[0] = TQ_OK;
}

__global__ __launch_bounds__(kPT) void k_truncate(View v, int32_t* table, int32_t* len,
                                                  int32_t* refs, int n,
                                                  const int32_t* slots,
                                                  const int32_t* lens, PagesWs w) {
    grid_begin();
    const int held = threadIdx.x == 0 ? pending(v) : 0;
    bool bad = repeated(v, slots, nullptr, n, w.marks) || held;
    for (int i = threadIdx.x; i < n; i += kPT)
        bad |= (unsigned)slots[i] >= (unsigned)v.slots || lens[i] < 0;
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) refuse(v, w, held, TQ_ERR_ARG);
        return;
    }
    for (int i = threadIdx.x >> 5; i < n; i += kPT / 32) {
        const int s = slots[i], had = length_of(v, s), keep = min(had, lens[i]);
        for (int p = pages_for(v, keep) + (threadIdx.x & 31); p < pages_for(v, had); p += 32) {
            const int id = page_of(v, s, p);
            table[(int64_t)s * v.max_pages + p] = -1;
            if (id >= 0) atomicSub(&refs[id], 1);
        }
        __syncwarp();
        if ((threadIdx.x & 31) == 0) len[s] = keep;
    }
    if (threadIdx.x == 0) w.head[0] = TQ_OK;
}

// Thread t looks after pages [t run, (t + 1) run): one prefix sum places all of
// its movers and holes.
__global__ __launch_bounds__(kPT) void k_compact(View v, int32_t* refs, PagesWs w) {
    __shared__ int64_t tmp[33];
    grid_begin();
    const int64_t run = ((int64_t)v.pages + kPT - 1) / kPT;
    const int64_t p0 = min((int64_t)v.pages, threadIdx.x * run), p1 = min((int64_t)v.pages, p0 + run);
    const int held = threadIdx.x == 0 ? pending(v) : 0;
    int64_t live = 0, L, moves;
    for (int64_t p = p0; p < p1; ++p) live += refs[p] > 0;
    if (__syncthreads_or(held)) {
        if (threadIdx.x == 0) w.head[0] = held;
        return;
    }
    block_scan(live, tmp, &L);
    int64_t movers = 0, holes = 0;
    for (int64_t p = p0; p < p1; ++p) {
        const bool on = refs[p] > 0;
        movers += on && p >= L;
        holes += !on && p < L;
    }
    int64_t m = block_scan(movers, tmp, &moves);
    int64_t k = block_scan(holes, tmp, &moves);
    for (int64_t p = p0; p < p1; ++p) {
        const bool on = refs[p] > 0;
        if (on && p >= L) w.src[m++] = (int32_t)p;
        if (!on && p < L) w.dst[k++] = (int32_t)p;
        if (!on && p >= L) w.ids[p] = (int32_t)p;  // held by nobody: stays
    }
    __syncthreads();
    for (int64_t i = threadIdx.x; i < moves; i += kPT) {
        const int s = w.src[i], d = w.dst[i];
        w.ids[s] = d;
        refs[d] = refs[s];
        refs[s] = 0;
    }
    if (threadIdx.x == 0) {
        w.head[0] = TQ_OK;
        w.head[1] = (int)moves;
        w.head[2] = (int)L;
    }
}

// Copies w.head[1] page pairs over all layers and pools: a block a piece of
// kPiece bytes of one (pair, layer, pool), 4 16-byte loads a thread in flight.
// REMAP (compact): the tables' entries >= L follow.
constexpr int kCT = 256, kPiece = kCT * 16 * 4;

template <bool REMAP>
__global__ __launch_bounds__(kCT) void k_copy_pages(const int* head,
                                                    const int32_t* src,
                                                    const int32_t* dst,
                                                    const int32_t* remap, int layers,
                                                    int pages, int heads, int64_t page_bytes,
                                                    uint8_t* k, uint8_t* v, float* ks, float* vs,
                                                    int32_t* table, int64_t entries) {
    grid_begin();
    if (head[0] != TQ_OK) return;
    const int pairs = head[1];
    const int64_t pieces = (page_bytes + kPiece - 1) / kPiece;
    const int64_t units = (int64_t)pairs * layers * 2 * pieces;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t piece = u % pieces;
        int64_t r = u / pieces;
        const int pool = (int)(r & 1);
        r >>= 1;
        const int layer = (int)(r % layers), pr = (int)(r / layers);
        const int64_t s = (int64_t)layer * pages + src[pr], d = (int64_t)layer * pages + dst[pr];
        uint8_t* base = pool ? v : k;
        const uint4* from = reinterpret_cast<const uint4*>(base + s * page_bytes + piece * kPiece);
        uint4* to = reinterpret_cast<uint4*>(base + d * page_bytes + piece * kPiece);
        const int n16 = (int)min((int64_t)kPiece, page_bytes - piece * kPiece) / 16;
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if ((int)threadIdx.x + i * kCT < n16) x[i] = from[threadIdx.x + i * kCT];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if ((int)threadIdx.x + i * kCT < n16) to[threadIdx.x + i * kCT] = x[i];
        if (piece == 0) {
            float* sc = pool ? vs : ks;
            for (int h = threadIdx.x; h < heads; h += kCT) sc[d * heads + h] = sc[s * heads + h];
        }
    }
    if (REMAP) {
        const int L = head[2];
        for (int64_t i = (int64_t)blockIdx.x * kCT + threadIdx.x; i < entries; i += (int64_t)gridDim.x * kCT) {
            const int id = table[i];
            // a live page behind the front has moved; other entries name nothing
            if (id >= L && id < pages) table[i] = remap[id];
        }
    }
}

template <bool REMAP>
int copy_pages(const tq_kv8_t* c, const PagesWs& w, int64_t most, cudaStream_t s) {
    const int64_t page_bytes = (int64_t)c->heads * c->page * c->d;
    const int64_t pieces = (page_bytes + kPiece - 1) / kPiece;
    const int64_t entries = REMAP ? (int64_t)c->slots * c->max_pages : 0;
    int64_t blocks = most * c->layers * 2 * pieces;
    if (blocks < (entries + kCT - 1) / kCT) blocks = (entries + kCT - 1) / kCT;
    if (blocks > 148 * 8) blocks = 148 * 8;
    return launch_behind(k_copy_pages<REMAP>, dim3((unsigned)blocks), kCT, 0, s, w.head, w.src, w.dst, w.ids,
                         c->layers, c->pages, c->heads, page_bytes, (uint8_t*)c->d_k, (uint8_t*)c->d_v,
                         c->d_kscale, c->d_vscale, c->d_table, entries);
}

// The checks that the list operations share.
int check_list(const tq_kv8_t* c, int n, const int32_t* a, const int32_t* b, void* ws,
               size_t ws_bytes) {
    int status;
    if (!valid(c, &status)) return status;
    if (n < 0) return TQ_ERR_ARG;
    if (n > kMaxList) return TQ_ERR_UNSUPPORTED;
    if (n > 0 && (!a || !b)) return TQ_ERR_ARG;
    if (n > 0 && (!ws || ws_bytes < pages_workspace(c, n))) return TQ_ERR_WORKSPACE;
    return TQ_OK;
}

}  // namespace
}  // namespace kv8
}  // namespace tq

using namespace tq;

extern "C" int tq_kv8_reserve(const tq_kv8_t* c, int n, const int32_t* d_slots,
                              const int32_t* d_counts, void* d_ws, size_t ws_bytes, void* stream) {
    int rc = kv8::check_list(c, n, d_slots, d_counts, d_ws, ws_bytes);
    if (rc || n == 0) return rc;
    const kv8::PagesWs w = kv8::carve(c, n, d_ws);
    cudaStream_t s = (cudaStream_t)stream;
    rc = launch_behind(kv8::k_reserve, dim3(1), kv8::kPT, 0, s, kv8::view(c), c->d_table, c->d_len,
                                  c->d_refs, n, d_slots, d_counts, w);
    return rc ? rc : kv8::copy_pages<false>(c, w, n, s);
}

extern "C" int tq_kv8_fork(const tq_kv8_t* c, int n, const int32_t* d_parents,
                           const int32_t* d_children, void* d_ws, size_t ws_bytes, void* stream) {
    const int rc = kv8::check_list(c, n, d_parents, d_children, d_ws, ws_bytes);
    if (rc || n == 0) return rc;
    return launch_behind(kv8::k_fork, dim3(1), kv8::kPT, 0, (cudaStream_t)stream, kv8::view(c), c->d_table,
                         c->d_len, c->d_refs, n, d_parents, d_children, kv8::carve(c, n, d_ws));
}

extern "C" int tq_kv8_truncate(const tq_kv8_t* c, int n, const int32_t* d_slots,
                               const int32_t* d_lens, void* d_ws, size_t ws_bytes, void* stream) {
    const int rc = kv8::check_list(c, n, d_slots, d_lens, d_ws, ws_bytes);
    if (rc || n == 0) return rc;
    return launch_behind(kv8::k_truncate, dim3(1), kv8::kPT, 0, (cudaStream_t)stream, kv8::view(c), c->d_table,
                         c->d_len, c->d_refs, n, d_slots, d_lens, kv8::carve(c, n, d_ws));
}

extern "C" int tq_kv8_compact(const tq_kv8_t* c, void* d_ws, size_t ws_bytes, void* stream) {
    int rc = kv8::check_list(c, 0, nullptr, nullptr, d_ws, ws_bytes);
    if (rc) return rc;
    if (!d_ws || ws_bytes < kv8::pages_workspace(c, 0)) return TQ_ERR_WORKSPACE;
    const kv8::PagesWs w = kv8::carve(c, 0, d_ws);
    cudaStream_t s = (cudaStream_t)stream;
    rc = launch_behind(kv8::k_compact, dim3(1), kv8::kPT, 0, s, kv8::view(c), c->d_refs, w);
    return rc ? rc : kv8::copy_pages<true>(c, w, c->pages / 2 + 1, s);
}
