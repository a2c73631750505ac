// cache.cu — the paged cache's C ABI (include/wildcat.h): argument checks,
// workspace layout, append and evict.  The attention is in cache_attend.cu.
#include <math.h>
#include <nvtx3/nvToolsExt.h>

#include "wc_cache.cuh"

namespace wc {
namespace cache {
namespace {

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// A pool's strides: dense where all are 0, else multiples of 16 bytes that
// keep the rows apart along every axis longer than 1.
bool strides_ok(const wc_cache& c, int width, int esize, int64_t page, int64_t head, int64_t token) {
    const int64_t unit = 16 / esize;
    if (page < 0 || head < 0 || token < 0 || page % unit || head % unit || token % unit) return false;
    return (c.page == 1 || token >= width) && (c.hkv == 1 || head >= width) && (c.n_pages == 1 || page >= width);
}

}  // namespace

wc_status make_view(const wc_cache* in, View* o) {
    if (!in) return WC_ERR_INVALID;
    const wc_cache& c = *in;
    if (c.batch < 1 || c.batch > 65535 || c.hkv < 1 || c.hkv > 65535 || c.hq < 1 || c.hq % c.hkv) return WC_ERR_INVALID;
    if ((int64_t)c.batch * c.hq > (1 << 24)) return WC_ERR_INVALID;
    if (c.d < 8 || c.d > 256 || c.d % 8 || c.dv < 8 || c.dv > 256 || c.dv % 8) return WC_ERR_INVALID;
    if (c.dtype != WC_F32 && c.dtype != WC_BF16) return WC_ERR_INVALID;
    if (c.page < 1 || c.page > 65536 || c.n_pages < 1 || c.max_pages < 1) return WC_ERR_INVALID;
    if ((int64_t)c.max_pages * c.page > (1 << 30)) return WC_ERR_INVALID;
    if (!(c.scale >= 0.f) || !isfinite(c.scale)) return WC_ERR_INVALID;
    o->B = c.batch; o->hq = c.hq; o->hkv = c.hkv; o->group = c.hq / c.hkv;
    o->d = c.d; o->dv = c.dv;
    o->page = c.page; o->n_pages = c.n_pages; o->max_pages = c.max_pages; o->cap = c.max_pages * c.page;
    o->dtype = c.dtype; o->esize = c.dtype == WC_BF16 ? 2 : 4;
    o->beta = c.scale > 0.f ? (double)c.scale : 1.0 / sqrt((double)c.d);
    o->table = nullptr;
    if (!c.k_page && !c.k_head && !c.k_token && !c.v_page && !c.v_head && !c.v_token) {
        o->k_token = c.d; o->k_head = (int64_t)c.page * c.d; o->k_page = c.hkv * o->k_head;
        o->v_token = c.dv; o->v_head = (int64_t)c.page * c.dv; o->v_page = c.hkv * o->v_head;
    } else {
        if (!strides_ok(c, c.d, o->esize, c.k_page, c.k_head, c.k_token)) return WC_ERR_INVALID;
        if (!strides_ok(c, c.dv, o->esize, c.v_page, c.v_head, c.v_token)) return WC_ERR_INVALID;
        o->k_page = c.k_page; o->k_head = c.k_head; o->k_token = c.k_token;
        o->v_page = c.v_page; o->v_head = c.v_head; o->v_token = c.v_token;
    }
    o->k_page *= o->esize; o->k_head *= o->esize; o->k_token *= o->esize;
    o->v_page *= o->esize; o->v_head *= o->esize; o->v_token *= o->esize;
    return WC_OK;
}

// Query rows of one unit of the attention's work.
static int rows_of(const View& s) {
    if (s.dtype == WC_BF16) return s.group > 8 ? 16 : s.group > 4 ? 8 : 4;
    return s.group >= 5 ? 8 : s.group >= 3 ? 4 : s.group;
}

// Coreset rows of one block: whole 64-row steps, about kCoresetBlocks blocks over all units (at
// most units + kCoresetBlocks, which the workspace holds).
static int coreset_split_len(const View& s, int r, int row_tiles) {
    const int64_t units = (int64_t)s.B * s.hkv * row_tiles, steps = (r + 63) / 64;
    const int64_t want = (kCoresetBlocks + units - 1) / units, splits = want < steps ? want : steps;
    return (int)((steps + splits - 1) / splits) * 64;
}

Layout make_layout(const View& s, bool accumulate) {
    Layout L;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + bytes, kWsAlign);
        return at;
    };
    const int rows = rows_of(s), tiles = (s.group + rows - 1) / rows;
    const size_t units = (size_t)s.B * s.hkv * tiles, set = sizeof(float) * rows * c1_row(s.dv);
    L.status = take(256);
    L.marks = take(sizeof(int32_t) * (size_t)s.n_pages);
    L.lens = take(sizeof(int32_t) * 2 * (size_t)s.B);
    L.parts = take((units + kMaxBlocks) * set);
    L.cparts = take((units + kCoresetBlocks) * set);
    L.logits = take(accumulate ? sizeof(float) * (size_t)s.B * s.hq * s.cap : 0);
    L.end = off;
    return L;
}

namespace {

// ------------------------------------------------------------------ append

struct AppendArgs {
    View s;
    const char* K; const char* V;
    int64_t k_batch, k_head, k_row, v_batch, v_head, v_row;   // bytes
    const int32_t* pos; const int32_t* count;
    char* kp; char* vp;
    float* scores;
    int t;
    int* status;
};

constexpr int kAppendThreads = 256;

// One warp a row (sequence, new row, kv head): its key and its value in 16-byte
// pieces.  A plain copy, bound by the bytes it moves.
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const AppendArgs a) {
    const View& s = a.s;
    const int64_t rows = (int64_t)s.B * a.t * s.hkv;
    const int lane = threadIdx.x & 31;
    const int ck = s.d * s.esize / 16, cv = s.dv * s.esize / 16;
    for (int64_t i = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5); i < rows;
         i += (int64_t)gridDim.x * (kAppendThreads / 32)) {
        const int h = (int)(i % s.hkv);
        const int64_t bj = i / s.hkv;
        const int j = (int)(bj % a.t), b = (int)(bj / a.t);
        const int n = a.count ? __ldg(a.count + b) : a.t;
        if (n < 0 || n > a.t) record_status(a.status, WC_ERR_BOUNDS);
        if (j >= n) continue;
        const int64_t at = (int64_t)__ldg(a.pos + b) + j;
        if (at < 0 || at >= s.cap) {
            record_status(a.status, WC_ERR_BOUNDS);
            continue;
        }
        const int tp = (int)at / s.page, slot = (int)at - tp * s.page;
        const int pg = checked_page(s, s.table, b, tp, a.status);
        if (pg < 0) continue;
        const uint4* ks = reinterpret_cast<const uint4*>(a.K + b * a.k_batch + h * a.k_head + j * a.k_row);
        const uint4* vs = reinterpret_cast<const uint4*>(a.V + b * a.v_batch + h * a.v_head + j * a.v_row);
        uint4* kd = reinterpret_cast<uint4*>(a.kp + pg * s.k_page + h * s.k_head + slot * s.k_token);
        uint4* vd = reinterpret_cast<uint4*>(a.vp + pg * s.v_page + h * s.v_head + slot * s.v_token);
        for (int c = lane; c < ck + cv; c += 32) {
            if (c < ck) kd[c] = ks[c];
            else vd[c - ck] = vs[c - ck];
        }
        if (a.scores && lane == 0) a.scores[((int64_t)b * s.hkv + h) * s.cap + at] = 0.f;
    }
}

// ------------------------------------------------------------------ evict

struct EvictArgs {
    View s;
    int keep, sink, recent;
    char* kp; char* vp;
    const int32_t* into;      // null: the sequence's own pages
    const int32_t* lens; const float* scores;
    float* scores_into;       // may be scores
    int32_t* idx; int32_t* lens_out;
    int32_t* marks; int32_t* ws_lens;
    int* status;
};

// References to every page: one for each page a sequence's tokens use, one for
// each page of `into` that it will write.
__global__ void cache_mark_kernel(const EvictArgs a) {
    const View& s = a.s;
    const int b = blockIdx.y;
    const int len = checked_len(a.lens, b, s.cap, a.status), kept = min(len, a.keep);
    const int used = (len + s.page - 1) / s.page, written = a.into ? (kept + s.page - 1) / s.page : 0;
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < used + written; i += gridDim.x * blockDim.x) {
        const int32_t* row = (i < used ? s.table : a.into) + (int64_t)b * s.max_pages;
        const int p = row[i < used ? i : i - used];
        if ((unsigned)p < (unsigned)s.n_pages) atomicAdd(a.marks + p, 1);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.ws_lens[2 * b] = len;
        a.ws_lens[2 * b + 1] = kept;
    }
}

// Order-preserving bits of a score: larger score, larger key; NaN as -inf, -0 as 0.
__device__ __forceinline__ uint32_t score_key(float x) {
    if (isnan(x)) x = -CUDART_INF_F;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kSelectThreads = 1024;

// Inclusive sum over the block's threads; sh holds one int per warp and stays
// the block's own until the next call's first barrier.
__device__ __forceinline__ int block_scan(int v, int* sh, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();
    if (lane == 31) sh[warp] = v;
    __syncthreads();
    int w = lane < kSelectThreads / 32 ? sh[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += u;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    return v + (warp > 0 ? before : 0);
}

// The kept positions of one (sequence, kv head): a radix select of the
// threshold score in three passes over the keys (11, 11 and 10 bits, a
// histogram each), then the positions in order.
__global__ void __launch_bounds__(kSelectThreads) cache_select_kernel(const EvictArgs a) {
    __shared__ int hist[2048];
    __shared__ int sh[32];
    __shared__ uint32_t s_bin;
    __shared__ int s_left;
    const View& s = a.s;
    const int h = blockIdx.x % s.hkv, b = blockIdx.x / s.hkv, tid = threadIdx.x;
    const int len = a.ws_lens[2 * b], kept = a.ws_lens[2 * b + 1];
    int32_t* idx = a.idx + ((int64_t)b * s.hkv + h) * a.keep;
    for (int i = kept + tid; i < a.keep; i += kSelectThreads) idx[i] = -1;
    if (len <= a.keep) {
        for (int i = tid; i < kept; i += kSelectThreads) idx[i] = i;
        return;
    }
    const float* x = a.scores + ((int64_t)b * s.hkv + h) * s.cap;
    const int first = a.sink, last = len - a.recent;
    const int want = a.keep - a.sink - a.recent;   // of the positions [first, last); fewer than there are
    uint32_t prefix = 0, mask = 0;
    int left = want;
    if (want > 0) {
        const int shifts[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
        for (int pass = 0; pass < 3; ++pass) {
            const int bins = 1 << bits[pass];
            for (int i = tid; i < 2048; i += kSelectThreads) hist[i] = 0;
            __syncthreads();
            for (int i = first + tid; i < last; i += kSelectThreads) {
                const uint32_t k = score_key(x[i]);
                if ((k & mask) == prefix) atomicAdd(&hist[(k >> shifts[pass]) & (bins - 1)], 1);
            }
            __syncthreads();
            // from the top bin down: the bin in which the `left`-th key lies
            const int hi = bins - 1 - 2 * tid, n1 = hi >= 0 ? hist[hi] : 0, n0 = hi >= 1 ? hist[hi - 1] : 0;
            int total;
            const int incl = block_scan(n1 + n0, sh, &total), before = incl - n1 - n0;
            if (before < left && left <= incl) {
                const bool up = left <= before + n1;
                s_bin = up ? hi : hi - 1;
                s_left = left - before - (up ? 0 : n1);
            }
            __syncthreads();
            prefix |= s_bin << shifts[pass];
            mask |= (uint32_t)(bins - 1) << shifts[pass];
            left = s_left;
            __syncthreads();
        }
    }
    // keys above `prefix` are kept, and the first `left` equal to it
    int base = 0, ties = 0;
    for (int at = 0; at < len; at += kSelectThreads) {
        const int i = at + tid;
        int above = 0, tie = 0;
        if (i < len) {
            if (i < first || i >= last) above = 1;
            else if (want > 0) {
                const uint32_t k = score_key(x[i]);
                above = k > prefix;
                tie = k == prefix;
            }
        }
        int total;
        const int incl = block_scan(above | tie << 16, sh, &total);
        const int tie_rank = ties + (incl >> 16) - tie;              // ties before this one
        const int tie_before = min(tie_rank, left) - min(ties, left);  // of them kept, in this stretch
        if (above || (tie && tie_rank < left)) idx[base + (incl & 0xffff) - above + tie_before] = i;
        const int all_ties = total >> 16;
        base += (total & 0xffff) + min(ties + all_ties, left) - min(ties, left);
        ties += all_ties;
    }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveBytes = 64 * 1024;   // rows staged at a time

// Whether a sequence's move is refused, and the reason recorded: a page
// outside the pool, or a page to be written that is named more than once.
__device__ bool refused(const EvictArgs& a, int b, int len, int kept) {
    const View& s = a.s;
    const int used = (len + s.page - 1) / s.page, written = (kept + s.page - 1) / s.page;
    int bad = 0;
    const bool moves = a.into || len > kept;
    for (int i = threadIdx.x; i < used; i += blockDim.x) {
        const int p = s.table[(int64_t)b * s.max_pages + i];
        if ((unsigned)p >= (unsigned)s.n_pages) bad |= 1;
        else if (!a.into && moves && i < written && a.marks[p] != 1) bad |= 2;
    }
    if (a.into)
        for (int i = threadIdx.x; i < written; i += blockDim.x) {
            const int p = a.into[(int64_t)b * s.max_pages + i];
            if ((unsigned)p >= (unsigned)s.n_pages) bad |= 1;
            else if (a.marks[p] != 1) bad |= 2;
        }
    const int any1 = __syncthreads_or(bad & 1), any2 = __syncthreads_or(bad & 2);
    if ((any1 || any2) && threadIdx.x == 0) record_status(a.status, any1 ? WC_ERR_BOUNDS : WC_ERR_INVALID);
    return any1 || any2;
}

// Moves the kept rows of one (sequence, kv head).  blockIdx.z: 0 keys, 1
// values, 2 scores.  In place the target of kept row j is position j and its
// source idx[j] >= j, so a block that works upwards, reading a stretch of rows
// whole before it writes it, never writes a row that is still to be read.
__global__ void __launch_bounds__(kMoveThreads) cache_move_kernel(const EvictArgs a) {
    extern __shared__ __align__(16) char stage[];
    const View& s = a.s;
    const int h = blockIdx.x, b = blockIdx.y, what = blockIdx.z, tid = threadIdx.x;
    const int len = a.ws_lens[2 * b], kept = a.ws_lens[2 * b + 1];
    const bool no = refused(a, b, len, kept);
    int32_t* idx = a.idx + ((int64_t)b * s.hkv + h) * a.keep;
    if (what == 2) {
        if (h == 0 && tid == 0) a.lens_out[b] = no ? len : kept;
        if (no)   // (the blocks that move keys and values are refused too and do not read idx)
            for (int j = tid; j < a.keep; j += kMoveThreads) idx[j] = -1;
        if (!no && (len > kept || a.scores_into != a.scores)) {
            const float* from = a.scores + ((int64_t)b * s.hkv + h) * s.cap;
            float* to = a.scores_into + ((int64_t)b * s.hkv + h) * s.cap;
            float* sh = reinterpret_cast<float*>(stage);
            constexpr int kChunk = kMoveBytes / 4;
            for (int j0 = 0; j0 < kept; j0 += kChunk) {
                const int n = min(kChunk, kept - j0);
                for (int j = tid; j < n; j += kMoveThreads) sh[j] = from[idx[j0 + j]];
                __syncthreads();
                for (int j = tid; j < n; j += kMoveThreads) to[j0 + j] = sh[j];
                __syncthreads();
            }
        }
        return;
    }
    if (no || (len <= kept && !a.into)) return;
    const int row_bytes = (what ? s.dv : s.d) * s.esize, ch = row_bytes / 16;
    char* pool = (what ? a.vp : a.kp) + h * (what ? s.v_head : s.k_head);
    const int64_t page_st = what ? s.v_page : s.k_page, token_st = what ? s.v_token : s.k_token;
    const int32_t* from = s.table + (int64_t)b * s.max_pages;
    const int32_t* to = (a.into ? a.into : s.table) + (int64_t)b * s.max_pages;
    const int rows = kMoveBytes / row_bytes;
    uint4* sh = reinterpret_cast<uint4*>(stage);
    for (int j0 = 0; j0 < kept; j0 += rows) {
        const int n = min(rows, kept - j0) * ch;
        for (int i = tid; i < n; i += kMoveThreads) {
            const int j = i / ch, c = i - j * ch, at = idx[j0 + j], tp = at / s.page;
            sh[i] = reinterpret_cast<const uint4*>(pool + from[tp] * page_st + (at - tp * s.page) * token_st)[c];
        }
        __syncthreads();
        for (int i = tid; i < n; i += kMoveThreads) {
            const int j = i / ch, c = i - j * ch, at = j0 + j, tp = at / s.page;
            reinterpret_cast<uint4*>(pool + to[tp] * page_st + (at - tp * s.page) * token_st)[c] = sh[i];
        }
        __syncthreads();
    }
}

wc_status launch_evict(const EvictArgs& a, cudaStream_t st) {
    const View& s = a.s;
    if (cudaMemsetAsync(a.marks, 0, sizeof(int32_t) * (size_t)s.n_pages, st) != cudaSuccess) return WC_ERR_CUDA;
    const int per = (s.max_pages + 255) / 256;
    cache_mark_kernel<<<dim3(per < 32 ? per : 32, s.B), 256, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return WC_ERR_CUDA;
    cache_select_kernel<<<s.B * s.hkv, kSelectThreads, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return WC_ERR_CUDA;
    if (cudaFuncSetAttribute(cache_move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMoveBytes) != cudaSuccess)
        return WC_ERR_CUDA;
    cache_move_kernel<<<dim3(s.hkv, s.B, 3), kMoveThreads, kMoveBytes, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? WC_OK : WC_ERR_CUDA;
}

struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
};

wc_status check_cache_ws(const Layout& L, void* ws, size_t ws_bytes) {
    if (!ws || !aligned(ws, kWsAlign)) return WC_ERR_INVALID;
    return ws_bytes < L.end ? WC_ERR_WORKSPACE : WC_OK;
}

}  // namespace
}  // namespace cache
}  // namespace wc

using namespace wc;
using namespace wc::cache;

extern "C" {

size_t wc_cache_workspace_bytes(const wc_cache* cache, int32_t accumulate) {
    View s;
    if (make_view(cache, &s) != WC_OK || (accumulate != 0 && accumulate != 1)) return 0;
    return cache::make_layout(s, accumulate != 0).end;
}

wc_status wc_cache_append(const wc_cache* cache, int32_t t, const void* K, const wc_row_strides* k_strides,
                          const void* V, const wc_row_strides* v_strides, const int32_t* pos, const int32_t* count,
                          void* k, void* v, const int32_t* table, float* scores, void* ws, size_t ws_bytes,
                          void* stream) {
    NvtxRange nvtx_range("wc_cache_append");
    AppendArgs a{};
    wc_status e = make_view(cache, &a.s);
    if (e != WC_OK) return e;
    if (t < 0) return WC_ERR_INVALID;
    if (!pos || !k || !v || !table || !aligned(k, 16) || !aligned(v, 16) || !aligned(pos, 4) || !aligned(count, 4) ||
        !aligned(table, 4) || !aligned(scores, 4))
        return WC_ERR_INVALID;
    if ((e = check_cache_ws(cache::make_layout(a.s, false), ws, ws_bytes)) != WC_OK) return e;
    if (t == 0) return WC_OK;
    if (!K || !V || !k_strides || !v_strides || !aligned(K, 16) || !aligned(V, 16)) return WC_ERR_INVALID;
    const int es = a.s.esize, unit = 16 / es;
    for (const wc_row_strides* r : {k_strides, v_strides})
        if (r->batch % unit || r->head % unit || r->row % unit) return WC_ERR_INVALID;
    a.s.table = table;
    a.K = static_cast<const char*>(K); a.V = static_cast<const char*>(V);
    a.k_batch = k_strides->batch * es; a.k_head = k_strides->head * es; a.k_row = k_strides->row * es;
    a.v_batch = v_strides->batch * es; a.v_head = v_strides->head * es; a.v_row = v_strides->row * es;
    a.pos = pos; a.count = count;
    a.kp = static_cast<char*>(k); a.vp = static_cast<char*>(v);
    a.scores = scores; a.t = t;
    a.status = static_cast<int*>(ws);
    const int64_t rows = (int64_t)a.s.B * t * a.s.hkv, per = kAppendThreads / 32;
    const int64_t grid = (rows + per - 1) / per;
    cache_append_kernel<<<(unsigned)(grid < 148 * 64 ? grid : 148 * 64), kAppendThreads, 0,
                          static_cast<cudaStream_t>(stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? WC_OK : WC_ERR_CUDA;
}

wc_status wc_cache_attend(const wc_cache* cache, const void* Q, int64_t q_batch, int64_t q_head, const void* k,
                          const void* v, const int32_t* table, const int32_t* lens, int32_t r, const void* Ks,
                          const float* W, const int32_t* rank, float* out, float* lse, float* scores, void* ws,
                          size_t ws_bytes, void* stream) {
    NvtxRange nvtx_range("wc_cache_attend");
    AttendArgs a{};
    wc_status e = make_view(cache, &a.s);
    if (e != WC_OK) return e;
    if (r < 0 || r > 4096 || (r > 0 && (!Ks || !W || !aligned(Ks, 16) || !aligned(W, 4) || !aligned(rank, 4))))
        return WC_ERR_INVALID;
    if (!Q || !k || !v || !table || !lens || !out || !aligned(Q, a.s.esize) || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(table, 4) || !aligned(lens, 4) || !aligned(out, 4) || !aligned(lse, 4) || !aligned(scores, 4))
        return WC_ERR_INVALID;
    const cache::Layout L = cache::make_layout(a.s, scores != nullptr);
    if ((e = check_cache_ws(L, ws, ws_bytes)) != WC_OK) return e;
    char* w = static_cast<char*>(ws);
    a.s.table = table;
    a.Q = Q; a.q_batch = q_batch; a.q_head = q_head;
    a.kp = static_cast<const char*>(k); a.vp = static_cast<const char*>(v);
    a.lens = lens;
    a.Ks = Ks; a.W = W; a.rank = r > 0 ? rank : nullptr; a.r = r;
    a.out = out; a.lse = lse; a.scores = scores;
    a.parts = reinterpret_cast<float*>(w + L.parts);
    a.cparts = reinterpret_cast<float*>(w + L.cparts);
    a.logits = scores ? reinterpret_cast<float*>(w + L.logits) : nullptr;
    a.status = static_cast<int*>(ws);
    a.rows = rows_of(a.s);
    a.row_tiles = (a.s.group + a.rows - 1) / a.rows;
    if (r > 0) {
        a.csplit_len = coreset_split_len(a.s, r, a.row_tiles);
        a.csplits = (r + a.csplit_len - 1) / a.csplit_len;
    }
    a.qscale = (float)(a.s.beta * 1.4426950408889634);
    return cache::launch_attend(a, static_cast<cudaStream_t>(stream));
}

wc_status wc_cache_evict(const wc_cache* cache, int32_t keep, int32_t sink, int32_t recent, void* k, void* v,
                         const int32_t* table, const int32_t* into, const int32_t* lens, const float* scores,
                         float* scores_into, int32_t* idx, int32_t* lens_out, void* ws, size_t ws_bytes,
                         void* stream) {
    NvtxRange nvtx_range("wc_cache_evict");
    EvictArgs a{};
    wc_status e = make_view(cache, &a.s);
    if (e != WC_OK) return e;
    if (keep < 1 || keep > a.s.cap || sink < 0 || recent < 0 || (int64_t)sink + recent > keep) return WC_ERR_INVALID;
    if (!k || !v || !table || !lens || !scores || !idx || !lens_out || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(table, 4) || !aligned(into, 4) || !aligned(lens, 4) || !aligned(scores, 4) ||
        !aligned(scores_into, 4) || !aligned(idx, 4) || !aligned(lens_out, 4))
        return WC_ERR_INVALID;
    const cache::Layout L = cache::make_layout(a.s, false);
    if ((e = check_cache_ws(L, ws, ws_bytes)) != WC_OK) return e;
    char* w = static_cast<char*>(ws);
    a.s.table = table;
    a.keep = keep; a.sink = sink; a.recent = recent;
    a.kp = static_cast<char*>(k); a.vp = static_cast<char*>(v);
    a.into = into == table ? nullptr : into;
    a.lens = lens; a.scores = scores;
    a.scores_into = scores_into ? scores_into : const_cast<float*>(scores);
    a.idx = idx; a.lens_out = lens_out;
    a.marks = reinterpret_cast<int32_t*>(w + L.marks);
    a.ws_lens = reinterpret_cast<int32_t*>(w + L.lens);
    a.status = static_cast<int*>(ws);
    return launch_evict(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
