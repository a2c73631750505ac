// wc_cache.cuh — what the paged-cache kernels share: the kernels' view of the
// cache, checked lengths and page lookups, the even division of the batch's
// key tiles over the warps, asynchronous copies and dependent launches.
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
    size_t status;    // int32 first device error; 64 bytes on, int32[2]: the half of `marks` in use (evict)
    size_t marks;     // int32[2][n_pages]  references to each page (evict)
    size_t lens;      // int32[2][B]     lengths before and after (evict)
    size_t parts;     // float[units + warps][rows][dv]  partial rows (attend)
    size_t parts_lm;  // float2[units + warps][rows]     their normalisers and references
    size_t cparts;    // float[units][coreset splits][rows][dv]
    size_t cparts_lm; // float2[units][coreset splits][rows]
    size_t logits;    // float[B][hq][cap]  logits in log2 units (attend with accumulation)
    size_t end;
};

// Warps of one attention launch over the pages, at most: what an SM holds of the kernel for that type and width.
inline int max_warps(const View& s) {
    const int w = s.d > s.dv ? s.d : s.dv;
    return 148 * (s.dtype == WC_BF16 ? (w <= 64 ? 16 : w <= 128 ? 8 : 6) : 12);
}
constexpr int kCoresetBlocks = 148 * 4;   // and over the coresets, beside one a unit

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
    int blocks;            // of the pages' kernel
    float qscale;          // beta * log2(e)
};

wc_status launch_attend(const AttendArgs& a, cudaStream_t st);

// Launches a kernel that may start before the stream's kernel ahead of it has
// ended (programmatic dependent launch): it calls grid_dependency_wait before
// it reads or writes anything of the caller's.
template <typename... A>
bool launch(void (*kern)(A...), int64_t grid, int threads, int smem, cudaStream_t st, A... args) {
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess;
}

// ---------------------------------------------------------------- device side

// A sequence's length, held to [0, cap]; one outside is recorded.
__device__ __forceinline__ int checked_len(const int32_t* lens, int b, int cap, int* status) {
    int n = lens[b];
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
    const int p = table[(int64_t)b * s.max_pages + t_page];
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
// blocks, and waits until the kernel before this one is complete.  (No load of
// these kernels is a read-only-cache load: the compiler may move such a load up
// past the wait.)
__device__ __forceinline__ void grid_dependents_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Division of the batch's work.  The keys of every unit (sequence, kv head,
// row tile of its group's queries) are cut into tiles, all tiles stand in one
// row, ordered by unit, with kUnitCost empty places before each unit's, and each
// warp takes one stretch of `per` places, so that all have equal work whatever
// the lengths are.  (The empty places stand for what a unit costs beside its
// tiles, its queries and its partial rows: without them a warp that meets a
// sequence of a few tokens has a unit at every tile and ends long after the
// others, 52 us against 31 in a batch of 64 with such a one.)
// A unit that spans several stretches leaves one set of partial rows for each;
// the set of unit u from stretch c has slot u + c, which no other pair has: along
// the row each next set has a larger u, a larger c or both.
// (The SMs do not get equal shares of the memory's rate: the slowest warp ends
// at 1.15 times the mean.  Measured and not kept: four fifths of the work divided
// so and the rest in short stretches that warps take from a counter; going on to
// another stretch stalls a warp for longer than the evenness saves, 94 -> 106 us
// for four sequences of 32768 tokens.)
constexpr int kPlaces = 1024;      // places in the row that a block holds: every sequence's, or every n-th one's
constexpr int kUnitCost = 4;       // in tiles (of 1, 2, 4, 8 measured)
// Places of one unit of n tokens.
__host__ __device__ __forceinline__ int64_t unit_places(int n, int tile) { return n > 0 ? ((int64_t)n + tile - 1) / tile + kUnitCost : 0; }
struct Share {
    int total, per, count;   // places, places of a stretch, stretches
    __device__ __forceinline__ Share(int places, int warps)
        : total(places), per(max((places + warps - 1) / warps, 1)), count((places + per - 1) / per) {}
    __device__ __forceinline__ int first(int c) const { return c * per; }
    __device__ __forceinline__ int last(int c) const { return first(c) + min(per, total - first(c)); }
    __device__ __forceinline__ int of(int t) const { return t / per; }
};

// Places of the batch and those before sequence want_b (where >= 0); where pre
// is not null, those before every step-th sequence go there.  All threads of the
// block call it; `sh` holds an int and one per warp.  The host has seen to it
// that the places of full tables and the warps together stay below 2^31.
struct Place { int total, before; };

template <int THREADS>
__device__ Place scan_tiles(const View& s, const int32_t* lens, int tile, int per_tile, int want_b, int* pre, int step,
                            int* status, int* sh) {
    const int per = (s.B + THREADS - 1) / THREADS;
    const int b0 = threadIdx.x * per, b1 = min(b0 + per, s.B);
    int sum = 0;
    for (int b = b0; b < b1; ++b) sum += (int)unit_places(checked_len(lens, b, s.cap, status), tile) * per_tile;
    int incl = sum;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) sh[1 + warp] = incl;
    __syncthreads();
    int at = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) at += sh[1 + w];
        total += sh[1 + w];
    }
    if (pre || (want_b >= b0 && want_b < b1))
        for (int b = b0; b < b1; ++b) {
            if (pre && b % step == 0) pre[b / step] = at;
            if (b == want_b) sh[0] = at;
            at += (int)unit_places(checked_len(lens, b, s.cap, status), tile) * per_tile;
        }
    __syncthreads();
    return Place{total, want_b >= 0 ? sh[0] : 0};
}

}  // namespace cache
}  // namespace wc
