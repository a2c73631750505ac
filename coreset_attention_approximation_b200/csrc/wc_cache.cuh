// wc_cache.cuh — what the paged-cache kernels share: the kernels' view of the
// cache, checked lengths and page lookups, the even division of the batch's
// key tiles over the thread blocks, and asynchronous row loads.
#pragma once

#include <math_constants.h>

#include "wc_common.cuh"
#include "wc_internal.h"

namespace wc {
namespace cache {

struct View {
    const int32_t* table;   // [B][max_pages]
    int B, hq, hkv, group;
    int d, dv;
    int page, n_pages, max_pages, cap;   // cap = max_pages * page
    uint32_t page_mul; int page_shift;   // t / page = t * page_mul >> page_shift for 0 <= t < 2^31
    int dtype, esize;
    uint32_t k_page, k_token, v_page, v_token;   // bytes
    int64_t k_head, v_head;
    double beta;
};

// Workspace of the cache calls (256-byte aligned regions).
struct Layout {
    size_t status;    // int32 first device error
    size_t marks;     // int32[n_pages]  references to each page (evict)
    size_t lens;      // int32[2][B]     lengths before and after (evict)
    size_t parts;     // float[units + workers][rows][dv]  partial rows (attend)
    size_t parts_lm;  // float2[units + workers][rows]     their normalisers and references
    size_t cparts;    // float[units][coreset splits][rows][dv]
    size_t cparts_lm; // float2[units][coreset splits][rows]
    size_t logits;    // float[B][hq][cap]  logits in log2 units (attend with accumulation)
    size_t end;
};

// Workers (warps) of one attention launch over the pages, at most (the partial rows are sized for them).
constexpr int kMaxWorkers = 148 * 12;
constexpr int kCoresetBlocks = 148 * 2;   // and over the coresets, beside one a unit

int rows_of(const View& s);   // query rows of one unit of the attention's work
wc_status make_view(const wc_cache* in, View* o);
Layout make_layout(const View& s, bool accumulate);

struct AttendArgs {
    View s;
    const void* Q; int64_t q_batch, q_head;      // strides in elements
    bool q_pairs;                                // pairs of a row's elements are aligned together
    const char* kp; const char* vp;
    const int32_t* lens;
    const void* Ks; const float* W; const int32_t* rank; int r;   // coreset, or r = 0
    float* out; float* lse; float* scores;       // lse, scores may be null
    float* parts; float* cparts; float* logits;
    float2* parts_lm; float2* cparts_lm;
    int* status;
    int rows, row_tiles;   // query rows of one unit of work; units per (sequence, kv head)
    int csplits, csplit_len;
    int blocks;            // blocks for the pages' tiles; those behind them take the coreset
    int workers;           // their warps
    float qscale;          // beta * log2(e)
};

wc_status launch_attend(const AttendArgs& a, cudaStream_t st);

// ---------------------------------------------------------------- device side

// A sequence's length, held to [0, cap]; one outside is recorded.
__device__ __forceinline__ int checked_len(const int32_t* lens, int b, int cap, int* status) {
    int n = __ldg(lens + b);
    if (n < 0 || n > cap) {
        record_status(status, WC_ERR_BOUNDS);
        n = n < 0 ? 0 : cap;
    }
    return n;
}

// t / page by a multiplication (the quotient is needed once a step for every key).
__device__ __forceinline__ int page_of(const View& s, int t) {
    return (int)(((uint64_t)(uint32_t)t * s.page_mul) >> s.page_shift);
}

// Page of token t of sequence b, or -1 (recorded) where the table's entry is no page.
__device__ __forceinline__ int checked_page(const View& s, const int32_t* table, int b, int t_page, int* status) {
    const int p = __ldg(table + (int64_t)b * s.max_pages + t_page);
    if ((unsigned)p >= (unsigned)s.n_pages) {
        record_status(status, WC_ERR_BOUNDS);
        return -1;
    }
    return p;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ const char* shfl_ptr(const char* p, int from) {
    return reinterpret_cast<const char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(p), from));
}
// The same where `go`, by a predicate (never a branch).
__device__ __forceinline__ void cp_async16_if(bool go, uint32_t dst, const void* src) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}" ::"r"(dst),
                 "l"(src), "r"((int)go)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Programmatic dependent launch: lets the stream's next kernel start its
// blocks, and waits until the kernel before this one is complete.
__device__ __forceinline__ void grid_dependents_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Division of the batch's work.  The keys of every unit (sequence, kv head,
// row tile of its group's queries) are cut into tiles; all T tiles stand in one
// row, ordered by unit, and each of C <= T workers (a warp) takes one stretch
// of T / C tiles, the first T % C of them one more.  Workers then have equal
// work whatever the lengths are.  A unit that spans several workers leaves one
// partial row set per worker; the set of unit u from worker c has slot u + c,
// which no other pair has: along the row of tiles each next set has a larger
// u, a larger c or both.
struct Share {
    int per, more;    // T / C, T % C
    __device__ __forceinline__ Share(int tiles, int workers) : per(tiles / workers), more(tiles - per * workers) {}
    __device__ __forceinline__ int first(int c) const { return c * per + min(c, more); }
    __device__ __forceinline__ int worker(int t) const {
        const int big = more * (per + 1);
        return t < big ? t / (per + 1) : more + (t - big) / per;
    }
};

// Tiles of the batch, the workers that get some, and a sequence with the
// tiles before it: the want_b-th, or the one that holds worker c's first tile.
struct Place {
    int total, workers;
    int before, b;
};

// All threads of the block call it; `sh` holds 2 ints + one per warp.  The
// host has seen to it that the tiles of full tables stay below 2^31.
template <int THREADS>
__device__ Place find_place(const View& s, const int32_t* lens, int tile, int per_tile, int workers, int c, int want_b,
                            int* status, int* sh) {
    const int per = (s.B + THREADS - 1) / THREADS;
    const int b0 = threadIdx.x * per, b1 = min(b0 + per, s.B);
    int sum = 0;
    for (int b = b0; b < b1; ++b) sum += (checked_len(lens, b, s.cap, status) + tile - 1) / tile * per_tile;
    int incl = sum;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) sh[2 + warp] = incl;
    if (threadIdx.x == 0) { sh[0] = 0; sh[1] = s.B; }
    __syncthreads();
    int base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) base += sh[2 + w];
        total += sh[2 + w];
    }
    incl += base;
    Place p;
    p.total = total;
    p.workers = min(workers, total);
    const int first = c < p.workers ? Share(total, p.workers).first(c) : total;
    const bool mine = want_b >= 0 ? (want_b >= b0 && want_b < b1) : (first >= incl - sum && first < incl);
    if (mine) {
        int at = incl - sum, b = b0;
        for (; b < b1; ++b) {
            const int n = (checked_len(lens, b, s.cap, status) + tile - 1) / tile * per_tile;
            if (want_b >= 0 ? b == want_b : first < at + n) break;
            at += n;
        }
        sh[0] = at;
        sh[1] = b;
    }
    __syncthreads();
    p.before = sh[0];
    p.b = sh[1];
    return p;
}

}  // namespace cache
}  // namespace wc
