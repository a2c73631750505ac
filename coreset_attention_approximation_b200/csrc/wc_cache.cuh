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
    int dtype, esize;
    int64_t k_page, k_head, k_token, v_page, v_head, v_token;   // bytes
    double beta;
};

// Workspace of the cache calls (256-byte aligned regions).
struct Layout {
    size_t status;    // int32 first device error
    size_t marks;     // int32[n_pages]  references to each page (evict)
    size_t lens;      // int32[2][B]     lengths before and after (evict)
    size_t parts;     // float[units + blocks][rows][c1_row(dv)]  partial rows (attend)
    size_t cparts;    // float[B * hkv * row tiles][coreset splits][rows][c1_row(dv)]
    size_t logits;    // float[B][hq][cap]  logits in log2 units (attend with accumulation)
    size_t end;
};

// Blocks of one attention launch over the pages, at most (the partial rows are sized for them).
constexpr int kMaxBlocks = 148 * 4;
constexpr int kCoresetBlocks = 148 * 2;   // and over the coresets, beside one a unit

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
    int* status;
    int rows, row_tiles;   // query rows of one unit of work; units per (sequence, kv head)
    int csplits, csplit_len;
    int blocks;            // blocks that share the pages' tiles
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

// Page of token t of sequence b, or -1 (recorded) where the table's entry is no page.
__device__ __forceinline__ int checked_page(const View& s, const int32_t* table, int b, int t_page, int* status) {
    const int p = __ldg(table + (int64_t)b * s.max_pages + t_page);
    if ((unsigned)p >= (unsigned)s.n_pages) {
        record_status(status, WC_ERR_BOUNDS);
        return -1;
    }
    return p;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    const int n = valid ? 16 : 0;   // 0: the 16 bytes are filled with zeros and src is not read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
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
// row tile of its group's queries) are cut into tiles; all tiles stand in one
// row, ordered by unit, and block c of C takes tiles [T c / C, T (c + 1) / C)
// (C at most T, so that every block has a tile and leaves its partial rows).
// Blocks then have equal work whatever the lengths are.  A unit that spans
// several blocks leaves one partial row set per block; the set of unit u from
// block c has slot u + c, which no other pair has: along the row of tiles each
// next set has a larger u, a larger c or both.
struct Range { int64_t first, last; };
__device__ __forceinline__ int64_t block_first(int64_t tiles, int c, int blocks) { return tiles * c / blocks; }
// Block that holds tile t.
__device__ __forceinline__ int block_of(int64_t t, int64_t tiles, int blocks) {
    int c = (int)((t * blocks) / tiles);
    while (c + 1 < blocks && block_first(tiles, c + 1, blocks) <= t) ++c;
    while (c > 0 && block_first(tiles, c, blocks) > t) --c;
    return c;
}

// Tiles of all sequences together, of those before sequence `want_b`, and the
// sequence that holds tile block_first(tiles, c) with the tiles before it.
// All threads of a block call it; `sh` holds 4 int64 + one per warp.
struct Place {
    int64_t total;    // tiles of the whole batch
    int64_t before;   // tiles before the sequence
    int b;            // the sequence
    int blocks;       // blocks with tiles
};

template <int THREADS>
__device__ Place find_place(const View& s, const int32_t* lens, int tile, int per_tile, int c, int blocks, int want_b,
                            int* status, int64_t* sh) {
    const int per = (s.B + THREADS - 1) / THREADS;
    const int b0 = threadIdx.x * per, b1 = min(b0 + per, s.B);
    int64_t sum = 0;
    for (int b = b0; b < b1; ++b)
        sum += (int64_t)((checked_len(lens, b, s.cap, status) + tile - 1) / tile) * per_tile;
    int64_t incl = sum;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) sh[4 + warp] = incl;
    if (threadIdx.x == 0) { sh[1] = 0; sh[2] = s.B; }
    __syncthreads();
    int64_t base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) base += sh[4 + w];
        total += sh[4 + w];
    }
    incl += base;
    if (blocks > total) blocks = (int)total;
    const int64_t first = c < blocks ? block_first(total, c, blocks) : total;
    const bool mine = want_b >= 0 ? (want_b >= b0 && want_b < b1) : (first >= incl - sum && first < incl);
    if (mine) {
        int64_t at = incl - sum;
        int b = b0;
        for (; b < b1; ++b) {
            const int64_t n = (int64_t)((checked_len(lens, b, s.cap, status) + tile - 1) / tile) * per_tile;
            if (want_b >= 0 ? b == want_b : first < at + n) break;
            at += n;
        }
        sh[1] = at;
        sh[2] = b;
    }
    __syncthreads();
    Place p;
    p.total = total;
    p.before = sh[1];
    p.b = (int)sh[2];
    p.blocks = blocks;
    __syncthreads();
    return p;
}

}  // namespace cache
}  // namespace wc
