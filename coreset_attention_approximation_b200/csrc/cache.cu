// cache.cu — the paged cache's C ABI (include/wildcat.h): argument checks,
// workspace layout, append and evict.  The attention is in cache_attend.cu.
#include <cooperative_groups.h>
#include <math.h>
#include <nvtx3/nvToolsExt.h>

#include <atomic>

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
    // m = floor(2^(31+s) / page) + 1 with 2^(s-1) < page <= 2^s: m page - 2^(31+s) <= page <= 2^s, so the
    // product is off by less than one part in 2^31 and the quotient exact below 2^31
    int sh = 0;
    while ((1 << sh) < c.page) ++sh;
    o->page_mul = (uint32_t)((1ull << (31 + sh)) / (uint64_t)c.page + 1);
    o->page_shift = 31 + sh;
    o->dtype = c.dtype; o->esize = c.dtype == WC_BF16 ? 2 : 4;
    o->beta = c.scale > 0.f ? (double)c.scale : 1.0 / sqrt((double)c.d);
    o->table = nullptr;
    int64_t k_page = c.k_page, k_token = c.k_token, v_page = c.v_page, v_token = c.v_token;
    o->k_head = c.k_head;
    o->v_head = c.v_head;
    if (!c.k_page && !c.k_head && !c.k_token && !c.v_page && !c.v_head && !c.v_token) {
        k_token = c.d; o->k_head = (int64_t)c.page * c.d; k_page = c.hkv * o->k_head;
        v_token = c.dv; o->v_head = (int64_t)c.page * c.dv; v_page = c.hkv * o->v_head;
    } else {
        if (!strides_ok(c, c.d, o->esize, c.k_page, c.k_head, c.k_token)) return WC_ERR_INVALID;
        if (!strides_ok(c, c.dv, o->esize, c.v_page, c.v_head, c.v_token)) return WC_ERR_INVALID;
    }
    const int64_t most = 0xffffffffll / o->esize;   // the kernels multiply 32 bits by 32
    if (k_page > most || k_token > most || v_page > most || v_token > most) return WC_ERR_UNSUPPORTED;
    o->k_page = (uint32_t)(k_page * o->esize); o->k_token = (uint32_t)(k_token * o->esize);
    o->v_page = (uint32_t)(v_page * o->esize); o->v_token = (uint32_t)(v_token * o->esize);
    o->k_head *= o->esize;
    o->v_head *= o->esize;
    return WC_OK;
}

// Query rows of one unit of the attention's work.
int rows_of(const View& s) {
    if (s.dtype == WC_BF16) return s.group > 8 ? 16 : s.group > 4 ? 8 : 4;
    return s.group >= 5 ? 8 : s.group >= 3 ? 4 : s.group;
}

// Coreset rows of one block: whole 64-row steps, about kCoresetBlocks blocks over all units (at
// most units + kCoresetBlocks, which the workspace holds).
int coreset_split_len(const View& s, int r, int row_tiles) {
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
    const size_t units = (size_t)s.B * s.hkv * tiles, set = sizeof(float) * rows * s.dv, lm = sizeof(float2) * rows;
    L.status = take(256);
    L.marks = take(sizeof(int32_t) * 2 * (size_t)s.n_pages);
    L.lens = take(sizeof(int32_t) * 2 * (size_t)s.B);
    L.parts = take((units + max_warps(s)) * set);
    L.parts_lm = take((units + max_warps(s)) * lm);
    L.cparts = take((units + kCoresetBlocks) * set);
    L.cparts_lm = take((units + kCoresetBlocks) * lm);
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

constexpr int kCopyThreads = 256;
constexpr int kCopyRows = 16;    // rows of one warp's step

// Where 16 rows come from and go to: lane j < 16 holds row j's addresses.
struct RowCopy {
    const char *ks, *vs;
    char *kd, *vd;
    bool ok;
};

// One warp copies 16 key rows and 16 value rows in 16-byte pieces, four pieces a
// lane in flight; rows that are not `ok` are skipped.  A copy, bound by the
// bytes it moves; the addresses of 16 rows are worked out once, a row a lane
// (one row a warp, each with its own lookups, reached half of the rate).
__device__ __forceinline__ void copy_rows(const RowCopy& r, int ck, int cv) {
    const int lane = threadIdx.x & 31;
    const uint32_t live = __ballot_sync(0xffffffffu, r.ok) & 0xffffu;
    if (!live) return;
    const int n = 32 - __clz(live);                  // rows up to the last live one
    // x / c for x < 16 * 64 and c <= 64 as (x * ceil(2^16 / c)) >> 16: off by less than 1024 / 2^16 < 1 / c
    const uint32_t mk = (65535u + ck) / ck, mv = (65535u + cv) / cv;
    const int nk = n * ck, total = nk + n * cv;
    for (int base = 0; base < total; base += 128) {
        uint4 x[4];
        char* to[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = base + u * 32 + lane;
            const bool key = i < nk;
            const uint32_t j = key ? i : i - nk;
            const int row = min((int)((j * (key ? mk : mv)) >> 16), kCopyRows - 1);
            const int at = (int)j - row * (key ? ck : cv);
            // one shuffle a pointer: a lane's source and target are both of its row
            const char* ks = shfl_ptr(r.ks, row);
            const char* vs = shfl_ptr(r.vs, row);
            const char* kd = shfl_ptr(r.kd, row);
            const char* vd = shfl_ptr(r.vd, row);
            const bool go = i < total && ((live >> row) & 1);
            to[u] = go ? const_cast<char*>(key ? kd : vd) + at * 16 : nullptr;
            if (go) x[u] = *reinterpret_cast<const uint4*>((key ? ks : vs) + at * 16);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (to[u]) *reinterpret_cast<uint4*>(to[u]) = x[u];
    }
}

// One warp per 16 new rows of one (sequence, kv head).
__global__ void __launch_bounds__(kCopyThreads) cache_append_kernel(const AppendArgs a) {
    grid_dependency_wait();
    grid_dependents_launch();
    const View& s = a.s;
    const int lane = threadIdx.x & 31, groups = (a.t + kCopyRows - 1) / kCopyRows;
    const int64_t items = (int64_t)s.B * s.hkv * groups;
    for (int64_t i = (int64_t)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); i < items;
         i += (int64_t)gridDim.x * (kCopyThreads / 32)) {
        const int64_t unit = i / groups;
        const int j = (int)(i - unit * groups) * kCopyRows + lane, b = (int)(unit / s.hkv), h = (int)(unit - (int64_t)b * s.hkv);
        int n = a.count ? a.count[b] : a.t;
        if (n < 0 || n > a.t) {
            record_status(a.status, WC_ERR_BOUNDS);
            n = min(max(n, 0), a.t);
        }
        RowCopy r{nullptr, nullptr, nullptr, nullptr, false};
        if (lane < kCopyRows && j < n) {
            const int64_t at = (int64_t)a.pos[b] + j;
            if (at < 0 || at >= s.cap) {
                record_status(a.status, WC_ERR_BOUNDS);
            } else {
                const int tp = page_of(s, (int)at), slot = (int)at - tp * s.page;
                const int pg = checked_page(s, s.table, b, tp, a.status);
                if (pg >= 0) {
                    r.ks = a.K + b * a.k_batch + h * a.k_head + j * a.k_row;
                    r.vs = a.V + b * a.v_batch + h * a.v_head + j * a.v_row;
                    r.kd = a.kp + (int64_t)pg * s.k_page + h * s.k_head + (int64_t)slot * s.k_token;
                    r.vd = a.vp + (int64_t)pg * s.v_page + h * s.v_head + (int64_t)slot * s.v_token;
                    r.ok = true;
                    if (a.scores) a.scores[((int64_t)b * s.hkv + h) * s.cap + at] = 0.f;
                }
            }
        }
        __syncwarp();
        copy_rows(r, s.d * s.esize / 16, s.dv * s.esize / 16);
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
    int32_t* marks;           // int32[2][n_pages], see mark_pages
    int32_t* phase;           // which half this call uses; and a copy for the move
    int32_t* ws_lens;
    int* status;
};

// Order-preserving bits of a score: larger score, larger key; NaN as -inf, -0 as 0.
__device__ __forceinline__ uint32_t score_key(float x) {
    if (isnan(x)) x = -CUDART_INF_F;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kSelectThreads = 512;
constexpr int kSelectBins = 2048 / kSelectThreads;   // of a thread
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kSelectCluster = 8;             // blocks that may share one (sequence, kv head)
constexpr int kSelectSlice = 4096;            // positions of a block before another one joins it
constexpr int kSelectHeld = 40960;            // keys a block holds in shared memory, at most,
constexpr int kSelectHeldMany = 12288;        // and where there are more blocks than SMs (three an SM then)

// References to the pages of sequence b: one for each page its tokens use, one
// for each page of `into` that it will write.  The counts start at 0: of two
// halves the calls use one after the other, and each call clears the half that
// the next will use (its last readers are done), which spares a launch.
__device__ __forceinline__ void mark_pages(const EvictArgs& a, int32_t* marks, int b, int len, int kept, int first,
                                           int step) {
    const View& s = a.s;
    const int used = (len + s.page - 1) / s.page, written = a.into ? (kept + s.page - 1) / s.page : 0;
    for (int i = first; i < used + written; i += step) {
        const int32_t* row = (i < used ? s.table : a.into) + (int64_t)b * s.max_pages;
        const int p = row[i < used ? i : i - used];
        if ((unsigned)p < (unsigned)s.n_pages) atomicAdd(marks + p, 1);
    }
}

// Inclusive sum over the block's threads; sh holds one int per warp.
__device__ __forceinline__ int block_scan(int v, int* sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) sh[warp] = v;
    __syncthreads();
    int w = lane < kSelectWarps ? sh[lane] : 0;
#pragma unroll
    for (int o = 1; o < kSelectWarps; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += u;
    }
    const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    return v + (warp > 0 ? before : 0);
}

// The kept positions of one (sequence, kv head), by a cluster of 1 to 8 blocks,
// each with a stretch of the positions.  The threshold score (the want-th
// largest of those that compete) comes from a radix select in three passes (11,
// 11 and 10 bits of the ordered keys): each block counts its own keys, every
// block adds the cluster's histograms through distributed shared memory and
// finds the same bin; a bin that is kept whole ends the search.  Then each warp counts what it keeps of its own stretch,
// and writes the positions in order behind those of the warps before it.  The
// keys are read from memory once and held in shared memory where they fit.
// Bound by the latency of the passes (a few barriers each) for the lengths of
// real caches.
template <int RANKS>
__global__ void __launch_bounds__(kSelectThreads, 3) cache_select_kernel(const EvictArgs a, int held) {
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ __align__(16) int hist[3][2048];   // (read four at a time)
    __shared__ int sh[kSelectWarps];
    __shared__ int2 counts[kSelectWarps];
    __shared__ int2 block_counts;
    __shared__ uint32_t s_bin;
    __shared__ int s_left, s_whole;
    grid_dependency_wait();
    grid_dependents_launch();
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    constexpr int ranks = RANKS;
    const int rank = RANKS > 1 ? (int)cluster.block_rank() : 0;
    auto sync_all = [&] {   // the cluster's blocks
        if (RANKS > 1) cluster.sync();
        else __syncthreads();
    };
    auto of_rank = [&](auto* p, int r) { return RANKS > 1 ? cluster.map_shared_rank(p, r) : p; };
    const View& s = a.s;
    const int unit = blockIdx.x / ranks, h = unit % s.hkv, b = unit / s.hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int len = checked_len(a.lens, b, s.cap, a.status), kept = min(len, a.keep);
    const int half = *a.phase & 1;
    for (int64_t i = (int64_t)blockIdx.x * kSelectThreads + tid; i < s.n_pages; i += (int64_t)gridDim.x * kSelectThreads)
        a.marks[(int64_t)(half ^ 1) * s.n_pages + i] = 0;
    if (blockIdx.x == 0 && tid == 0) a.phase[1] = half;
    if (h == 0) {
        mark_pages(a, a.marks + (int64_t)half * s.n_pages, b, len, kept, rank * kSelectThreads + tid,
                   ranks * kSelectThreads);
        if (rank == 0 && tid == 0) {
            a.ws_lens[2 * b] = len;
            a.ws_lens[2 * b + 1] = kept;
        }
    }
    int32_t* idx = a.idx + (int64_t)unit * a.keep;
    for (int i = kept + rank * kSelectThreads + tid; i < a.keep; i += ranks * kSelectThreads) idx[i] = -1;
    if (len <= a.keep) {
        for (int i = rank * kSelectThreads + tid; i < kept; i += ranks * kSelectThreads) idx[i] = i;
        return;   // every block of the cluster does
    }
    const float* x = a.scores + (int64_t)unit * s.cap;
    const int per = ((len + ranks - 1) / ranks + 31) / 32 * 32;
    const int lo = min(rank * per, len), hi = min(lo + per, len);
    const int first = a.sink, last = len - a.recent;   // the positions that compete
    const int want = a.keep - a.sink - a.recent;       // of them kept: fewer than there are
    const bool hold = per <= held;
    for (int i = tid; i < 3 * 2048; i += kSelectThreads) (&hist[0][0])[i] = 0;
    auto key = [&](int i) { return hold ? keys[i - lo] : score_key(x[i]); };
    if (hold)
#pragma unroll 4
        for (int i = lo + tid; i < hi; i += kSelectThreads) keys[i - lo] = score_key(x[i]);
    uint32_t prefix = 0, mask = 0;
    int left = want;
    bool whole = false;
    __syncthreads();
    if (want > 0) {
        const int shifts[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
#pragma unroll
        for (int pass = 0; pass < 3; ++pass) {
            if (whole) break;   // (the same in every block: each added the same counts)
            const int bins = 1 << bits[pass];
            for (int i = max(lo, first) + tid; i < min(hi, last); i += kSelectThreads) {
                const uint32_t k = key(i);
                if ((k & mask) == prefix) atomicAdd(&hist[pass][(k >> shifts[pass]) & (bins - 1)], 1);
            }
            sync_all();
            // from the top bin down: the bin in which the `left`-th key lies; a thread has kSelectBins of
            // them, from bin `low` up, and takes every block's counts, all loads in flight
            const int low = bins - kSelectBins * (tid + 1);
            int n[kSelectBins], sum = 0;
#pragma unroll
            for (int i = 0; i < kSelectBins; ++i) n[i] = 0;
            if (low >= 0) {
#pragma unroll
                for (int i = 0; i < kSelectBins; i += 4) {
                    int4 v[RANKS];
#pragma unroll
                    for (int r = 0; r < RANKS; ++r)
                        v[r] = *reinterpret_cast<const int4*>(of_rank(&hist[pass][low + i], r));
#pragma unroll
                    for (int r = 0; r < RANKS; ++r) {
                        n[i] += v[r].x, n[i + 1] += v[r].y, n[i + 2] += v[r].z, n[i + 3] += v[r].w;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kSelectBins; ++i) sum += n[i];
            const int incl = block_scan(sum, sh);
            int before = incl - sum;
            if (before < left && left <= incl) {
#pragma unroll
                for (int i = kSelectBins - 1; i >= 0; --i) {
                    if (before < left && left <= before + n[i]) {
                        s_bin = low + i;
                        s_left = left - before;
                        s_whole = left - before == n[i];
                    }
                    before += n[i];
                }
            }
            __syncthreads();
            prefix |= s_bin << shifts[pass];
            mask |= (uint32_t)(bins - 1) << shifts[pass];
            left = s_left;
            whole = s_whole != 0;   // all of the bin are kept: its keys need not be told apart (mostly after two passes)
        }
    }
    // kept: the positions that do not compete, the keys above `prefix` and, of those equal to it, the first
    // `left`, or, where the bin is kept whole, the keys from `prefix` up
    const int span = ((hi - lo + kSelectWarps - 1) / kSelectWarps + 31) / 32 * 32;
    const int w0 = min(lo + warp * span, hi), w1 = min(w0 + span, hi);
    auto judge = [&](int i, bool& above, bool& tie) {
        above = tie = false;
        if (i >= w1) return;
        if (i < first || i >= last) above = true;
        else if (want > 0) {
            const uint32_t k = key(i);
            above = whole ? k >= prefix : k > prefix;
            tie = !whole && k == prefix;
        }
    };
    // (a bit for each of the first 32 rounds keeps what was found for the second time over)
    uint32_t were_above = 0, were_tie = 0;
    int n_above = 0, n_tie = 0, round = 0;
    for (int i = w0; i < w1; i += 32, ++round) {
        bool above, tie;
        judge(i + lane, above, tie);
        if (round < 32) were_above |= (uint32_t)above << round, were_tie |= (uint32_t)tie << round;
        n_above += __popc(__ballot_sync(0xffffffffu, above));
        n_tie += __popc(__ballot_sync(0xffffffffu, tie));
    }
    if (lane == 0) counts[warp] = make_int2(n_above, n_tie);
    __syncthreads();
    if (warp == 0) {   // the counts before each warp, and the block's
        const int2 own = lane < kSelectWarps ? counts[lane] : make_int2(0, 0);
        int2 c = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, c.x, o), v = __shfl_up_sync(0xffffffffu, c.y, o);
            if (lane >= o) c.x += u, c.y += v;
        }
        if (lane < kSelectWarps) counts[lane] = make_int2(c.x - own.x, c.y - own.y);
        if (lane == 31) block_counts = c;
    }
    sync_all();
    int2 blocks[RANKS];
#pragma unroll
    for (int r = 0; r < RANKS; ++r) blocks[r] = r < rank ? *of_rank(&block_counts, r) : make_int2(0, 0);
    int above_before = counts[warp].x, ties_before = counts[warp].y;
#pragma unroll
    for (int r = 0; r < RANKS; ++r) above_before += blocks[r].x, ties_before += blocks[r].y;
    int at = above_before + min(ties_before, left);
    round = 0;
    for (int i = w0; i < w1; i += 32, ++round) {
        bool above, tie;
        if (round < 32) above = (were_above >> round) & 1, tie = (were_tie >> round) & 1;
        else judge(i + lane, above, tie);
        const uint32_t below = (1u << lane) - 1, ties = __ballot_sync(0xffffffffu, tie);
        const bool keep = above || (tie && ties_before + __popc(ties & below) < left);
        const uint32_t keeps = __ballot_sync(0xffffffffu, keep);
        if (keep) idx[at + __popc(keeps & below)] = i + lane;
        at += __popc(keeps);
        ties_before += __popc(ties);
    }
    if (RANKS > 1) cluster.sync();   // no block leaves while another may read its shared memory
}

constexpr int kMoveThreads = 256;
constexpr int kMoveBytes = 64 * 1024;   // in place: bytes staged at a time
constexpr int kMoveBytesInto = 16 * 1024;   // into other pages: of scores (the rows need none, and more blocks fit)
constexpr int kMoveSlice = 64;          // in place: bytes of a row that one block moves

// Whether a sequence's move is refused, and the reason recorded: a page
// outside the pool, or a page to be written that is named more than once.
__device__ bool refused(const EvictArgs& a, int b, int len, int kept) {
    const View& s = a.s;
    const int32_t* marks = a.marks + (int64_t)a.phase[1] * s.n_pages;
    const int used = (len + s.page - 1) / s.page, written = (kept + s.page - 1) / s.page;
    int bad = 0;
    const bool moves = a.into || len > kept;
    for (int i = threadIdx.x; i < used; i += blockDim.x) {
        const int p = s.table[(int64_t)b * s.max_pages + i];
        if ((unsigned)p >= (unsigned)s.n_pages) bad |= 1;
        else if (!a.into && moves && i < written && marks[p] != 1) bad |= 2;
    }
    if (a.into)
        for (int i = threadIdx.x; i < written; i += blockDim.x) {
            const int p = a.into[(int64_t)b * s.max_pages + i];
            if ((unsigned)p >= (unsigned)s.n_pages) bad |= 1;
            else if (marks[p] != 1) bad |= 2;
        }
    if (!__syncthreads_or(bad)) return false;
    const int outside = __syncthreads_or(bad & 1);
    if (threadIdx.x == 0) record_status(a.status, outside ? WC_ERR_BOUNDS : WC_ERR_INVALID);
    return true;
}

// One int32, whole, where another block may write or read it at the same time.
__device__ __forceinline__ int load_relaxed(const int32_t* p) {
    int x;
    asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(x) : "l"(p) : "memory");
    return x;
}
__device__ __forceinline__ void store_relaxed(int32_t* p, int x) {
    asm volatile("st.relaxed.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(x) : "memory");
}

// The scores of one (sequence, kv head), a stretch read whole before it is
// written (see move_in_place), its lengths, and -1 in idx where refused.
__device__ void move_scores(const EvictArgs& a, int b, int h, int len, int kept, bool no, char* stage) {
    const View& s = a.s;
    const int64_t unit = (int64_t)b * s.hkv + h;
    int32_t* idx = a.idx + unit * a.keep;
    if (h == 0 && threadIdx.x == 0) a.lens_out[b] = no ? len : kept;
    if (no) {   // (blocks that move rows may read idx at the same time: see cache_move_kernel)
        for (int j = threadIdx.x; j < a.keep; j += kMoveThreads) store_relaxed(idx + j, -1);
        return;
    }
    if (len <= kept && a.scores_into == a.scores) return;
    const float* from = a.scores + unit * s.cap;
    float* to = a.scores_into + unit * s.cap;
    float* sh = reinterpret_cast<float*>(stage);
    const int chunk = (a.into ? kMoveBytesInto : kMoveBytes) / 4;
    for (int j0 = 0; j0 < kept; j0 += chunk) {
        const int n = min(chunk, kept - j0);
#pragma unroll 4
        for (int j = threadIdx.x; j < n; j += kMoveThreads) sh[j] = from[idx[j0 + j]];
        __syncthreads();
        for (int j = threadIdx.x; j < n; j += kMoveThreads) to[j0 + j] = sh[j];
        __syncthreads();
    }
}

// In place: 64 bytes of every kept row of one (sequence, kv head) per block.
// The target of kept row j is position j and its source idx[j] >= j, so a
// block that works upwards, reading a stretch of rows whole before it writes
// it, never writes a row that is still to be read.  The slices let eight
// blocks and more share a head whose rows have to move in order.  (The whole
// eviction of 32 ragged sequences to 2048 tokens takes 110 us so, 98 us into other
// pages; of one sequence of 32768 to 1024, 22.6 and 20.6 us.)
__device__ void move_in_place(const EvictArgs& a, int b, int h, int slice, int kept, char* stage) {
    const View& s = a.s;
    const int kslices = (s.d * s.esize + kMoveSlice - 1) / kMoveSlice;
    const bool key = slice < kslices;
    const int off = (key ? slice : slice - kslices) * kMoveSlice, row_bytes = (key ? s.d : s.dv) * s.esize;
    const int ch = min(kMoveSlice, row_bytes - off) / 16;
    char* pool = (key ? a.kp + h * s.k_head : a.vp + h * s.v_head) + off;
    const int64_t page_st = key ? s.k_page : s.v_page, token_st = key ? s.k_token : s.v_token;
    const int32_t* table = s.table + (int64_t)b * s.max_pages;
    const int32_t* idx = a.idx + ((int64_t)b * s.hkv + h) * a.keep;
    constexpr int kRows = kMoveBytes / kMoveSlice;
    const int piece = threadIdx.x & 3;      // a thread's 16 bytes of the slice
    for (int j0 = 0; j0 < kept; j0 += kRows) {
        const int n = min(kRows, kept - j0);
        if (piece < ch)
#pragma unroll 4
            for (int j = threadIdx.x >> 2; j < n; j += kMoveThreads / 4) {
                const int at = idx[j0 + j], tp = page_of(s, at);
                cp_async16((uint32_t)__cvta_generic_to_shared(stage + j * kMoveSlice + piece * 16),
                           pool + table[tp] * page_st + (at - tp * s.page) * token_st + piece * 16);
            }
        cp_async_commit();
        cp_async_wait<0>();
        __syncthreads();
        if (piece < ch)
            for (int j = threadIdx.x >> 2; j < n; j += kMoveThreads / 4) {
                const int at = j0 + j, tp = page_of(s, at);
                *reinterpret_cast<uint4*>(pool + table[tp] * page_st + (at - tp * s.page) * token_st + piece * 16) =
                    *reinterpret_cast<const uint4*>(stage + j * kMoveSlice + piece * 16);
            }
        __syncthreads();
    }
}

// Moves the kept rows and their scores.  blockIdx.z = sequence, y = kv head;
// x = 0 takes the scores, the others the rows: in place a slice each, into
// other pages 128 rows each (a warp 16 of them), where the order is free.
__global__ void __launch_bounds__(kMoveThreads) cache_move_kernel(const EvictArgs a) {
    extern __shared__ __align__(16) char stage[];
    grid_dependency_wait();
    const View& s = a.s;
    const int h = blockIdx.y, b = blockIdx.z, part = blockIdx.x;
    const int len = a.ws_lens[2 * b], kept = a.ws_lens[2 * b + 1];
    if (part == 0 && h == 0 && b == 0 && threadIdx.x == 0) a.phase[0] = a.phase[1] ^ 1;
    constexpr int kBlockRows = kMoveThreads / 32 * kCopyRows;
    if (part > 0 && (a.into ? (part - 1) * kBlockRows >= kept : len <= kept)) return;
    // Where a lane's row comes from and goes to, on its way while the pages are checked.  The sequence may
    // be refused, and then the block that takes the scores writes -1 over idx, before or after this block reads
    // it: only a position of the sequence is looked up (and nothing of it is used once this block has found the
    // refusal itself).  In place, rows are read from idx behind the check alone.
    const int lane = threadIdx.x & 31, j = (part - 1) * kBlockRows + (threadIdx.x >> 5) * kCopyRows + lane;
    RowCopy r{nullptr, nullptr, nullptr, nullptr, false};
    int at = -1;
    if (part > 0 && a.into && lane < kCopyRows && j < kept) at = load_relaxed(a.idx + ((int64_t)b * s.hkv + h) * a.keep + j);
    if ((unsigned)at < (unsigned)len) {
        const int tp = page_of(s, at), slot = at - tp * s.page;
        const int to = page_of(s, j), to_slot = j - to * s.page;
        const int64_t from_page = s.table[(int64_t)b * s.max_pages + tp], to_page = a.into[(int64_t)b * s.max_pages + to];
        r.ks = a.kp + from_page * s.k_page + h * s.k_head + (int64_t)slot * s.k_token;
        r.vs = a.vp + from_page * s.v_page + h * s.v_head + (int64_t)slot * s.v_token;
        r.kd = a.kp + to_page * s.k_page + h * s.k_head + (int64_t)to_slot * s.k_token;
        r.vd = a.vp + to_page * s.v_page + h * s.v_head + (int64_t)to_slot * s.v_token;
        r.ok = true;
    }
    const bool no = refused(a, b, len, kept);
    if (part == 0) move_scores(a, b, h, len, kept, no, stage);
    else if (no) return;
    else if (a.into) copy_rows(r, s.d * s.esize / 16, s.dv * s.esize / 16);
    else move_in_place(a, b, h, part - 1, kept, stage);
}

// The kernels' shared-memory limits, once per device.
wc_status evict_setup() {
    static std::atomic<uint64_t> done{0};   // a bit per device number (the first 64; the others set it each time)
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return WC_ERR_CUDA;
    if (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1)) return WC_OK;
    for (auto kern : {cache_select_kernel<1>, cache_select_kernel<2>, cache_select_kernel<4>, cache_select_kernel<8>})
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelectHeld * 4) != cudaSuccess)
            return WC_ERR_CUDA;
    if (cudaFuncSetAttribute(cache_move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMoveBytes) != cudaSuccess)
        return WC_ERR_CUDA;
    if (dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
    return WC_OK;
}

wc_status launch_evict(const EvictArgs& a, cudaStream_t st) {
    const View& s = a.s;
    wc_status e = evict_setup();
    if (e != WC_OK) return e;
    // blocks of one (sequence, kv head): one for each kSelectSlice positions, while there are at most four an SM
    const int64_t units = (int64_t)s.B * s.hkv;
    int ranks = 1;
    while (ranks < kSelectCluster && 2 * ranks * units <= 4 * 148 && (int64_t)ranks * kSelectSlice < s.cap) ranks *= 2;
    if (units * ranks > INT32_MAX || s.hkv > 65535) return WC_ERR_UNSUPPORTED;
    const int per = ((s.cap + ranks - 1) / ranks + 31) / 32 * 32;
    const int most = units * ranks > 148 ? kSelectHeldMany : kSelectHeld, held = per < most ? per : most;
    cudaLaunchAttribute at[2]{};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = ranks;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(units * ranks));
    cfg.blockDim = dim3(kSelectThreads);
    cfg.dynamicSmemBytes = (size_t)held * 4;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    auto select = ranks == 1 ? cache_select_kernel<1> : ranks == 2 ? cache_select_kernel<2>
                : ranks == 4 ? cache_select_kernel<4> : cache_select_kernel<8>;
    if (cudaLaunchKernelEx(&cfg, select, a, held) != cudaSuccess) return WC_ERR_CUDA;
    const int slices = (s.d * s.esize + kMoveSlice - 1) / kMoveSlice + (s.dv * s.esize + kMoveSlice - 1) / kMoveSlice;
    const int rows = kMoveThreads / 32 * kCopyRows;
    cfg.gridDim = dim3(1 + (a.into ? (a.keep + rows - 1) / rows : slices), s.hkv, s.B);
    cfg.blockDim = dim3(kMoveThreads);
    cfg.dynamicSmemBytes = a.into ? kMoveBytesInto : kMoveBytes;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cache_move_kernel, a) == cudaSuccess ? WC_OK : WC_ERR_CUDA;
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
    if (t < 0 || t > (1 << 30)) return WC_ERR_INVALID;
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
    const int64_t items = (int64_t)a.s.B * a.s.hkv * ((t + (int64_t)kCopyRows - 1) / kCopyRows);
    const int64_t grid = (items + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
    return launch(cache_append_kernel, grid < 148 * 64 ? grid : 148 * 64, kCopyThreads, 0,
                  static_cast<cudaStream_t>(stream), a) ? WC_OK : WC_ERR_CUDA;
}

wc_status wc_cache_attend(const wc_cache* cache, const void* Q, int64_t q_batch, int64_t q_head, const void* k,
                          const void* v, const int32_t* table, const int32_t* lens, int32_t r, const void* Ks,
                          const float* W, const int32_t* rank, float* out, float* lse, float* scores, void* ws,
                          size_t ws_bytes, void* stream) {
    NvtxRange nvtx_range("wc_cache_attend");
    AttendArgs a{};
    wc_status e = make_view(cache, &a.s);
    if (e != WC_OK) return e;
    if (r < 0 || r > 4096 || (r > 0 && (!Ks || !W || !aligned(Ks, 16) || !aligned(W, 16) || !aligned(rank, 4))))
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
    a.parts_lm = reinterpret_cast<float2*>(w + L.parts_lm);
    a.cparts_lm = reinterpret_cast<float2*>(w + L.cparts_lm);
    a.logits = scores ? reinterpret_cast<float*>(w + L.logits) : nullptr;
    a.status = static_cast<int*>(ws);
    a.q_pairs = aligned(Q, 2 * a.s.esize) && q_batch % 2 == 0 && q_head % 2 == 0;
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
    a.phase = reinterpret_cast<int32_t*>(w + L.status + 64);
    a.ws_lens = reinterpret_cast<int32_t*>(w + L.lens);
    a.status = static_cast<int*>(ws);
    return launch_evict(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
