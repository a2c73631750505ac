// cache_attend.cu — attention of one new token per sequence over a paged
// cache, optionally together with a weighted coreset:
//   L = sum_i a_i + sum_s a'_s W[s, dv],   a = exp(beta <q, k>)
//   out = (sum_i a_i v_i + sum_s a'_s W[s, :dv]) / L
// One pass over the keys and values with a running maximum per query row (in
// log2 units, so one multiplication by beta log2(e) is folded into the query):
// a partial result is (O, l, m) with O = sum 2^(x - m) v, l = sum 2^(x - m).
// The key tiles of the whole batch are divided over the warps (Share in
// wc_cache.cuh), whatever the lengths; a warp streams its tiles through a ring
// of its own in shared memory, on from one sequence or head to the next, and
// never waits for another.  The coreset is a kernel of its own ahead of it, whose
// blocks and the pages' do not fit an SM together: a pages' block starts as the
// coreset's blocks leave.  A last kernel joins the partial rows, in order of the stretches and of
// the coreset's splits.
//
// The kernels overlap by programmatic dependent launch: each may start before
// the one ahead of it has ended, lets the next start once it knows that the
// stream's earlier work is complete, and waits before it reads what the one
// ahead wrote.  The pages' kernel reads nothing of the coreset's; it waits for
// it at its end, so that its own end means both to the join.
#include <atomic>
#include <mutex>

#include "wc_cache.cuh"

namespace wc {
namespace cache {
namespace {

constexpr int kSimtWarps = 4;

// A running row's reference is set this far (in log2 units) above the largest
// logit, and moves only when a logit passes it: most steps are spared the
// rescaling.  Above and not below it, so that no weight exceeds 1 and a value's
// product with it overflows only where the value does (weights of up to 2^8
// overflowed from |v| = 2^120 on); a weight underflows below 2^-118 of the largest.
constexpr float kAhead = 8.f;

// Pairs of fp32 values in one 64-bit register, added and multiplied as one:
// half the instructions where the issue of sums is what bounds a loop.
__device__ __forceinline__ uint64_t pair_of(float x, float y) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
    return p;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
    uint64_t p;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(x), "l"(y));
    return p;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
    uint64_t p;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(x), "l"(y));
    return p;
}
// x y + z
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
    uint64_t p;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p) : "l"(x), "l"(y), "l"(z));
    return p;
}
__device__ __forceinline__ float2 halves(uint64_t p) {
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p));
    return v;
}

// Logits of NT staged fp32 keys against RG query rows: lane = (key, part of d).
// Every lane ends with its key's whole sums.
template <int RG, int NT>
__device__ __forceinline__ void tile_logits(const char* krows, int k_row, const float* q, int d, float s[RG]) {
    const int lane = threadIdx.x & 31, key = lane % NT, part = lane / NT;
    const char* row = krows + key * k_row;
    uint64_t sum[RG];
#pragma unroll
    for (int g = 0; g < RG; ++g) sum[g] = 0;
#pragma unroll 4
    for (int c = part; c < d / 4; c += 32 / NT) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(row + c * 16);
#pragma unroll
        for (int g = 0; g < RG; ++g) {
            const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(q + g * d + c * 4);
            sum[g] = fma2(x.x, y.x, sum[g]);
            sum[g] = fma2(x.y, y.y, sum[g]);
        }
    }
#pragma unroll
    for (int g = 0; g < RG; ++g) {
        const float2 v = halves(sum[g]);
        s[g] = v.x + v.y;
    }
#pragma unroll
    for (int o = NT; o < 32; o <<= 1)
#pragma unroll
        for (int g = 0; g < RG; ++g) s[g] += __shfl_xor_sync(0xffffffffu, s[g], o);
}

// A warp's way through its tiles: the stretch, the unit (sequence b, kv head h,
// row tile rt) and the tile k of its `tiles`.
struct Walk {
    int left;          // places to the end of the stretch, from this tile's on
    int stretch;
    int b, h, rt, k, tiles, len;
    // to the first tile of stretch c; pre: the places before every step-th sequence
    __device__ __forceinline__ void start(const AttendArgs& a, const Share& share, const int* pre, int step, int c,
                                          int tile) {
        stretch = c;
        left = 0;
        b = h = rt = k = tiles = len = 0;
        if (c >= share.count) return;
        int t = share.first(c);
        left = share.last(c) - t;
        const int per_tile = a.s.hkv * a.row_tiles;
        int lo = 0, hi = (a.s.B + step - 1) / step;   // the last of them with no more than t places before it
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (pre[mid] <= t) lo = mid;
            else hi = mid;
        }
        t -= pre[lo];
        int places = 0;
        for (b = lo * step;; ++b) {
            len = checked_len(a.lens, b, a.s.cap, a.status);
            places = (int)unit_places(len, tile);
            if (t < places * per_tile) break;
            t -= places * per_tile;
        }
        tiles = places - kUnitCost;
        const int unit = t / places;
        k = t - unit * places - kUnitCost;
        if (k < 0) {   // in the places before its tiles
            left += k;
            k = 0;
        }
        h = unit / a.row_tiles;
        rt = unit - h * a.row_tiles;
    }
    // tiles first, first + n, ... of one unit (short caches: a block has a unit)
    __device__ __forceinline__ void one(const AttendArgs& a, int unit, int first, int tile) {
        stretch = 0;
        const int pair = unit / a.row_tiles;
        rt = unit - pair * a.row_tiles;
        b = pair / a.s.hkv;
        h = pair - b * a.s.hkv;
        len = checked_len(a.lens, b, a.s.cap, a.status);
        tiles = (len + tile - 1) / tile;
        k = first;
        left = tiles - first;
    }
    // past n tiles of this unit, to the next unit behind its last one (true then)
    __device__ __forceinline__ bool skip(const AttendArgs& a, int n, int tile) {
        left -= n;
        k += n;
        if (left <= 0 || k < tiles) return false;
        left -= kUnitCost;
        if (left <= 0) return false;
        k = 0;
        if (++rt == a.row_tiles) {
            rt = 0;
            if (++h == a.s.hkv) {
                h = 0;
                do len = checked_len(a.lens, ++b, a.s.cap, a.status);
                while (len == 0);
                tiles = (len + tile - 1) / tile;
            }
        }
        return true;
    }
    // row of the unit's first partial row
    __device__ __forceinline__ int64_t part_row(const AttendArgs& a) const {
        return ((int64_t)(b * a.s.hkv + h) * a.row_tiles + rt + stretch) * a.rows;
    }
};

// A warp's ring of stages in shared memory.  A stage holds the key rows of one
// step's KEYS keys, then their value rows, of DP elements each; the 16-byte
// pieces of a row stand XOR-swizzled by the row, so that eight rows at one
// column lie in eight different bank groups.  (Rows padded by 16 bytes would do
// that too, but pieces that arrive at unaligned 128-byte groups take two writes
// each: 8 % slower throughout.)  Rows come by 16-byte asynchronous copies, a row
// to 32 lanes or fewer.  Where a page holds whole steps, a lane's sources are
// one base and a fixed stride apart, and no copy needs more than an addition
// for its address: with addresses of their own the copies took half of all
// instructions, and one bulk copy a row, issued lane by lane, 16 cycles each.
template <int KEYS, int DP, int ESIZE, int STAGES>
struct Ring {
    static constexpr int kRow = DP * ESIZE, kStage = 2 * KEYS * kRow;
    static constexpr int kBytes = STAGES * kStage;
    static constexpr int kChunks = DP * ESIZE / 16;                  // pieces of a row
    static constexpr int kPass = kChunks < 32 ? 32 / kChunks : 1;    // rows of one warp-wide copy
    static constexpr int kParts = kChunks < 32 ? 1 : kChunks / 32;   // copies a row takes
    uint32_t mem;            // the ring at this lane's first row
    int row0, ch;            // this lane's first row of a step and its piece
    bool whole;              // a page holds whole steps
    const char *k, *v;       // this lane's places in page 0 of the unit at hand
    // the next step: its page as the table has it (of this lane's key, where not whole), the slot in it, the keys
    int page, slot, keys;

    __device__ __forceinline__ void init(const AttendArgs& a, char* memory) {
        const View& s = a.s;
        const int lane = threadIdx.x & 31;
        row0 = lane / kChunks % kPass;
        ch = lane % (kChunks < 32 ? kChunks : 32);
        mem = (uint32_t)__cvta_generic_to_shared(memory) + row0 * kRow;
        whole = s.page % KEYS == 0;
        // columns past the width are never copied and count as zeros
        if (s.d < DP || s.dv < DP)
            for (int i = lane; i < kBytes / 16; i += 32) reinterpret_cast<uint4*>(memory)[i] = make_uint4(0, 0, 0, 0);
        __syncwarp();
    }
    // Where this lane's piece of a row stands in it.
    __device__ __forceinline__ uint32_t place(int row) const { return (ch ^ (row & 7)) * 16; }
    // The unit that w is in.
    __device__ __forceinline__ void enter(const AttendArgs& a, const Walk& w) {
        const View& s = a.s;
        k = a.kp + w.h * s.k_head + (whole ? row0 * (int64_t)s.k_token + ch * 16 : 0);
        v = a.vp + w.h * s.v_head + (whole ? row0 * (int64_t)s.v_token + ch * 16 : 0);
    }
    // Reads the table for the step at w; nothing here waits for the entry, so
    // that it is on its way while the step before is computed.
    __device__ __forceinline__ void locate(const AttendArgs& a, const Walk& w) {
        const View& s = a.s;
        keys = 0;
        if (w.left <= 0) return;
        const int first = w.k * KEYS, key = first + (whole ? 0 : (threadIdx.x & 31) % KEYS);
        keys = min(KEYS, w.len - first);
        const int tp = page_of(s, min(key, w.len - 1));
        slot = key - tp * s.page;
        page = s.table[(int64_t)w.b * s.max_pages + tp];
    }
    // Starts the copies of the located step and returns a bit for each key that
    // is there.  A value row that is not is filled with zeros (its weight is 0,
    // and 0 times what lay there may not be).
    __device__ __forceinline__ uint32_t fetch(const AttendArgs& a, int stage) {
        const View& s = a.s;
        const uint32_t kd = mem + stage * kStage, vd = kd + KEYS * kRow;
        const int ck = s.d * ESIZE / 16, cv = s.dv * ESIZE / 16;
        const uint32_t all = (uint32_t)((1ull << KEYS) - 1);
        const bool good = (unsigned)page < (unsigned)s.n_pages;
        const uint32_t pg = good ? page : 0;
        const char* ks = k + (uint64_t)pg * s.k_page + (uint64_t)(uint32_t)slot * s.k_token;
        const char* vs = v + (uint64_t)pg * s.v_page + (uint64_t)(uint32_t)slot * s.v_token;
        if (whole && good && keys == KEYS) {
#pragma unroll
            for (int i = 0; i < KEYS / kPass; ++i) {
#pragma unroll
                for (int p = 0; p < kParts; ++p) {
                    const uint32_t off = i * kPass * kRow + p * 512 + place(i * kPass + row0);
                    cp_async16_if(ch + p * 32 < ck, kd + off, ks + p * 512);
                    cp_async16_if(ch + p * 32 < cv, vd + off, vs + p * 512);
                }
                ks += kPass * (uint64_t)s.k_token;
                vs += kPass * (uint64_t)s.v_token;
            }
            return all;
        }
        if (!good) record_status(a.status, WC_ERR_BOUNDS);
        uint32_t live = keys >= KEYS ? all : (1u << keys) - 1;
        if (whole) live = good ? live : 0u;
        else live &= __ballot_sync(0xffffffffu, good);
#pragma unroll 1
        for (int i = 0; i < KEYS / kPass; ++i) {
            const int row = i * kPass + row0;
            const char *kr = ks + i * kPass * (int64_t)s.k_token, *vr = vs + i * kPass * (int64_t)s.v_token;
            if (!whole) {
                kr = shfl_ptr(ks, row) + ch * 16;
                vr = shfl_ptr(vs, row) + ch * 16;
            }
            const bool there = (live >> row) & 1;
#pragma unroll
            for (int p = 0; p < kParts; ++p) {
                const uint32_t off = i * kPass * kRow + p * 512 + place(row);
                cp_async16_if(there && ch + p * 32 < ck, kd + off, kr + p * 512);
                cp_async16_if(there && ch + p * 32 < cv, vd + off, vr + p * 512);
                if (!there && ch + p * 32 < cv)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vd + off), "r"(0) : "memory");
            }
        }
        return live;
    }
};

// No key was summed (every one masked, or none there).  A NaN among the logits
// leaves l NaN and is no such row.
__device__ __forceinline__ bool nothing(float m, float l) { return m == -CUDART_INF_F && l == 0.f; }

// log of the normaliser l 2^m.
__device__ __forceinline__ float log_sum(float m, float l) {
    return nothing(m, l) ? m : (float)(((double)m + log2((double)l)) * 0.69314718055994530942);
}

// Joins a coreset block's warps (shared, [warps][RG][dv + 2]) into partial rows.
template <int RG, int WARPS>
__device__ __forceinline__ void join_warps(const AttendArgs& a, const float* merge, int index, int rows) {
    const int dv = a.s.dv, ld = dv + 2;
    for (int g = 0; g < rows; ++g) {
        const float* r = merge + g * ld;
        float m = -CUDART_INF_F;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) m = fmaxf(m, r[w * RG * ld + dv]);
        const float ref = m == -CUDART_INF_F ? 0.f : m;
        float f[WARPS], l = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            f[w] = ex2(r[w * RG * ld + dv] - ref);
            l += f[w] * r[w * RG * ld + dv + 1];
        }
        const int64_t row = (int64_t)index * a.rows + g;
        float* to = a.cparts + row * dv;
        for (int c = threadIdx.x; c < dv; c += WARPS * 32) {
            float o = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) o = fmaf(f[w], r[w * RG * ld + c], o);
            to[c] = o;
        }
        if (threadIdx.x == 0) a.cparts_lm[row] = make_float2(l, m);
    }
}

// fp32 query rows of one unit into shared memory, scaled to log2 units;
// rows past the group are zero.
template <int RG, int WARPS>
__device__ __forceinline__ void load_queries(const AttendArgs& a, int b, int g0, int rows, float* q) {
    const float* src = static_cast<const float*>(a.Q) + b * a.q_batch + (int64_t)g0 * a.q_head;
    for (int i = threadIdx.x; i < RG * a.s.d; i += WARPS * 32) {
        const int g = i / a.s.d, c = i - g * a.s.d;
        q[i] = g < rows ? src[g * a.q_head + c] * a.qscale : 0.f;
    }
}

// ---------------------------------------------------------------- tensor cores

__device__ __forceinline__ void ldmatrix4(uint32_t r[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4t(uint32_t r[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// a b, 16 x 8 x 16, bf16 in, fp32 sums.
__device__ __forceinline__ void mma16816_new(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%10,%10,%10,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// c += a b.
__device__ __forceinline__ void mma16816(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The three bf16 terms of a pair of weights x >= 0, x = t0 + t1 + t2: the upper 8
// bits of x, of the rest and of the rest of that (one rounded term alone, half a
// step or 2^-9 relative, would be the largest error of the whole attention, whose
// output is fp32).  Cut off, not rounded, so that no term is negative, and none is
// below kLeast = 2^-126: an infinite value then meets only positive factors and
// its column is infinite, as by the definition (0 inf and inf - inf are NaN).  A
// weight that is 0 because it is below 2^-126 grows by that much at most; rows that
// are not there are zeros.  NaN stays NaN.
constexpr uint32_t kLeast = 0x00800080u;   // a pair of bf16 2^-126
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t t[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(t[i]) : "r"(__byte_perm(a, b, 0x7632)), "r"(kLeast));
        x -= __uint_as_float(a & 0xffff0000u);
        y -= __uint_as_float(b & 0xffff0000u);
    }
}

// The bf16 query fragments of one unit for 16-row tiles: rows quad and, where
// kRows = 16, quad + 8; with fewer rows, row quad % kRows (rows past the group
// are zeros).
template <int DP, int kRows>
struct QueryFragments {
    static constexpr int kRegs = kRows == 16 ? 4 : 2;
    uint32_t q[DP / 16][kRegs];
    __device__ __forceinline__ void load(const AttendArgs& a, int b, int g0, int rows) {
        const int lane = threadIdx.x & 31, quad = lane >> 2, pair = lane & 3;
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.Q) + b * a.q_batch + (int64_t)g0 * a.q_head;
        auto two = [&](int row, int col) {
            uint32_t v = 0;
            if (row < rows && col < a.s.d) {
                const __nv_bfloat16* p = src + row * a.q_head + col;
                if (a.q_pairs) v = *reinterpret_cast<const uint32_t*>(p);
                else v = (uint32_t)__bfloat16_as_ushort(p[0]) | (uint32_t)__bfloat16_as_ushort(p[1]) << 16;
            }
            return v;
        };
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
            const int col = k * 16 + pair * 2;
            if (kRows == 16) {
                q[k][0] = two(quad, col), q[k][1] = two(quad + 8, col);
                q[k][kRegs - 2] = two(quad, col + 8), q[k][kRegs - 1] = two(quad + 8, col + 8);
            } else {
                q[k][0] = two(quad % kRows, col);
                q[k][1] = two(quad % kRows, col + 8);
            }
        }
    }
    // x += the k-th 16 columns against 8 keys
    __device__ __forceinline__ void step(float x[4], int k, uint32_t b0, uint32_t b1) const {
        if (kRows == 16) mma16816(x, q[k][0], q[k][1], q[k][kRegs - 2], q[k][kRegs - 1], b0, b1);
        else mma16816(x, q[k][0], q[k][0], q[k][1], q[k][1], b0, b1);
    }
};

constexpr int kCoresetWarps = 4;

// Shared memory of one coreset block, in bytes: two stages a warp of NT keys
// and their rows of W (as they lie in memory, dv + 1 values each, and up to 12
// bytes before them).  The warps' sums go where the stages were.  The end
// leaves room for a lane that reads its columns past dv (and drops them).
template <typename T, int NT, int RG, int DP>
struct CoresetSmem {
    int k_row, w, stage, q, p, total;
    __host__ __device__ CoresetSmem(int d, int dv) {
        k_row = sizeof(T) == 2 ? DP * 2 + 16 : (d / 4 % 2 ? d * 4 : d * 4 + 16);   // an odd number of 16-byte units
        w = NT * k_row;
        stage = (w + 12 + NT * (dv + 1) * 4 + 15) / 16 * 16;
        const int stages = kCoresetWarps * 2 * stage, merge = kCoresetWarps * RG * (dv + 2) * 4;
        q = ((stages > merge ? stages : merge) + 15) / 16 * 16;
        p = q + (sizeof(T) == 2 ? 0 : RG * d * 4);
        total = p + kCoresetWarps * NT * RG * 8 + 512;
    }
};

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// One block of the coreset's share: rows [first, last) of unit (b, h)'s
// coreset against RG query rows, NT at a time for each warp.  W is fp32 with
// rows of dv + 1 values, which have no 16-byte alignment; a step's rows lie side
// by side, so the 16-byte pieces that hold them are copied (4-byte copies took
// 1.3 times as long over all), the last few values one by one.  A lane holds
// columns lane, lane + 32, ... and the row's last value is its weight in the
// normaliser.  The logits of bf16 keys on tensor cores, the sums in fp32 on
// CUDA cores: W's values cancel one another.  8 x 1024 rows of 8 heads take 16.9 us
// (cold, 3.0 TB/s): each warp has only four steps of 720 instructions, and with
// 3.3 warps a scheduler (96 registers, 52 KB of stages a block) the latencies of a
// step's loads, shuffles and sums are not covered (a scheduler issues in half of
// its active cycles).
template <typename T, int RG, int NT, int DP>
__global__ void __launch_bounds__(kCoresetWarps * 32) cache_coreset_kernel(const AttendArgs a) {
    constexpr int WARPS = kCoresetWarps, COLS = DP / 32;
    constexpr bool kTensor = sizeof(T) == 2;     // logits on tensor cores
    static_assert(!kTensor || NT == 8, "a step is one column octet of the product");
    extern __shared__ __align__(128) char smem[];
    grid_dependency_wait();
    grid_dependents_launch();
    const View& s = a.s;
    const int index = blockIdx.x;
    const CoresetSmem<T, NT, RG, DP> L(s.d, s.dv);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* q = reinterpret_cast<float*>(smem + L.q);
    uint64_t* p = reinterpret_cast<uint64_t*>(smem + L.p) + warp * NT * RG;   // a step's weights, each twice
    char* stages = smem + warp * 2 * L.stage;
    const int split = index % a.csplits, unit = index / a.csplits;
    const int rt = unit % a.row_tiles, h = unit / a.row_tiles % s.hkv, b = unit / a.row_tiles / s.hkv;
    const int rows = min(a.rows, s.group - rt * a.rows);
    int n = a.rank ? a.rank[b * s.hkv + h] : a.r;
    if (n < 0 || n > a.r) {
        record_status(a.status, WC_ERR_BOUNDS);
        n = n < 0 ? 0 : a.r;
    }
    const int first = split * a.csplit_len, last = min(first + a.csplit_len, n);
    const int64_t base = ((int64_t)b * s.hkv + h) * a.r;
    const int ck = s.d * (int)sizeof(T) / 16;
    auto load = [&](int stage, int at) {
        const int live = min(NT, last - at);
        if (live > 0) {
            const uint32_t kd = (uint32_t)__cvta_generic_to_shared(stages + stage * L.stage), wd = kd + L.w;
            const char* k = static_cast<const char*>(a.Ks) + (base + at) * s.d * (int64_t)sizeof(T);
            constexpr int kChunks = DP * (int)sizeof(T) / 16;
#pragma unroll
            for (int i = 0; i < NT * kChunks; i += 32) {
                const int row = (i + lane) / kChunks, c = (i + lane) % kChunks;
                cp_async16_if(row < live && c < ck, kd + row * L.k_row + c * 16, k + (row * ck + c) * 16);
            }
            const int64_t w0 = (base + at) * (s.dv + 1), w1 = w0 + live * (s.dv + 1);   // values [w0, w1) of W
            const int pieces = (int)(w1 / 4 - w0 / 4);
            for (int i = lane; i < pieces; i += 32) cp_async16(wd + i * 16, a.W + (w0 / 4 + i) * 4);
            if (lane < (int)(w1 & 3)) cp_async4(wd + pieces * 16 + lane * 4, a.W + (w1 / 4) * 4 + lane);
        }
        cp_async_commit();
    };
    if (kTensor && s.d < DP) {   // columns past the width are never copied and count as zeros
        for (int i = lane; i < L.stage / 8; i += 32) reinterpret_cast<uint4*>(stages)[i] = make_uint4(0, 0, 0, 0);
        __syncwarp();
    }
    int at = first + warp * NT;
    load(0, at);
    const int g0 = h * s.group + rt * a.rows;
    QueryFragments<kTensor ? DP : 16, kTensor ? RG : 4> qf;
    if (kTensor) qf.load(a, b, g0, rows);
    else load_queries<RG, WARPS>(a, b, g0, rows, q);
    __syncthreads();
    constexpr int kRefs = !kTensor ? RG : RG == 16 ? 2 : 1;   // references a lane holds: of all rows, or of its own
    float m[kRefs], l[RG];
#pragma unroll
    for (int r = 0; r < kRefs; ++r) m[r] = -CUDART_INF_F;
    uint64_t o[RG][COLS / 2];   // columns lane + 64 i and 32 further on
#pragma unroll
    for (int g = 0; g < RG; ++g) {
        l[g] = 0.f;
#pragma unroll
        for (int i = 0; i < COLS / 2; ++i) o[g][i] = 0;
    }
    auto rescale = [&](int g, float f) {
        l[g] *= f;
#pragma unroll
        for (int i = 0; i < COLS / 2; ++i) o[g][i] = mul2(o[g][i], pair_of(f, f));
    };
    for (int stage = 0; at < last; at += WARPS * NT, stage ^= 1) {
        load(stage ^ 1, at + WARPS * NT);
        cp_async_wait<1>();
        __syncwarp();
        const char* krows = stages + stage * L.stage;
        const float* wrows = reinterpret_cast<const float*>(krows + L.w) + (int)(((base + at) * (s.dv + 1)) & 3);
        const int live = min(NT, last - at);
        if constexpr (kTensor) {
            // a lane: keys 2 pair and 2 pair + 1 of row quad (and quad + 8)
            const int quad = lane >> 2, pair = lane & 3;
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            const uint32_t kd = (uint32_t)__cvta_generic_to_shared(krows) + (lane & 7) * L.k_row + (lane >> 3) * 16;
#pragma unroll
            for (int k = 0; k < DP / 32; ++k) {
                uint32_t f[4];
                ldmatrix4(f, kd + k * 64);
                qf.step(x, 2 * k, f[0], f[1]);
                qf.step(x, 2 * k + 1, f[2], f[3]);
            }
#pragma unroll
            for (int r = 0; r < kRefs; ++r) {
                float y[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) y[e] = pair * 2 + e < live ? x[2 * r + e] * a.qscale : -CUDART_INF_F;
                float top = fmaxf(y[0], y[1]);
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const bool grow = top > m[r];
                if (__any_sync(0xffffffffu, grow)) {
                    const float f = grow ? ex2(m[r] - (top + kAhead)) : 1.f;
                    if (grow) m[r] = top + kAhead;
#pragma unroll
                    for (int g = 0; g < (RG < 8 ? RG : 8); ++g) rescale((g + 8 * r) % RG, __shfl_sync(0xffffffffu, f, g * 4));
                }
                const float ref = m[r] == -CUDART_INF_F ? 0.f : m[r];
                if (quad < RG)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float w = ex2(y[e] - ref);
                        p[(pair * 2 + e) * RG + quad + 8 * r] = pair_of(w, w);
                    }
            }
        } else {
            float x[RG];
            tile_logits<RG, NT>(krows, L.k_row, q, s.d, x);
            const int key = lane % NT;
#pragma unroll
            for (int g = 0; g < RG; ++g) {
                const float v = key < live ? x[g] : -CUDART_INF_F;
                float top = v;
#pragma unroll
                for (int e = 1; e < NT; e <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, e));
                if (top > m[g % kRefs]) {
                    const float f = ex2(m[g % kRefs] - top);
                    m[g % kRefs] = top;
                    rescale(g, f);
                }
                const float w = ex2(v - (m[g % kRefs] == -CUDART_INF_F ? 0.f : m[g % kRefs]));
                if (lane < NT) p[key * RG + g] = pair_of(w, w);
            }
        }
        __syncwarp();
        auto add_row = [&](int j) {
            const float* w = wrows + j * (s.dv + 1);
            uint64_t y[COLS / 2];
#pragma unroll
            for (int i = 0; i < COLS / 2; ++i) y[i] = pair_of(w[lane + 64 * i], w[lane + 64 * i + 32]);   // (past dv: dropped)
            const float z = w[s.dv];
#pragma unroll
            for (int g = 0; g < RG; ++g) {
                const uint64_t e = p[j * RG + g];
                l[g] = fmaf(halves(e).x, z, l[g]);
#pragma unroll
                for (int i = 0; i < COLS / 2; ++i) o[g][i] = fma2(e, y[i], o[g][i]);
            }
        };
        if (live == NT) {
#pragma unroll
            for (int j = 0; j < NT; ++j) add_row(j);
        } else {
#pragma unroll 1
            for (int j = 0; j < live; ++j) add_row(j);
        }
        __syncwarp();
    }
    cp_async_wait<0>();
    __syncthreads();
    float* merge = reinterpret_cast<float*>(smem);
    const int ld = s.dv + 2;
#pragma unroll
    for (int g = 0; g < RG; ++g) {
        float* row = merge + (warp * RG + g) * ld;
#pragma unroll
        for (int i = 0; i < COLS / 2; ++i) {
            const float2 v = halves(o[g][i]);
            const int c = lane + 64 * i;
            if (c < s.dv) row[c] = v.x;
            if (c + 32 < s.dv) row[c + 32] = v.y;
        }
        if (lane == (kTensor ? g % 8 * 4 : 0)) {   // (the lane that holds the row's reference)
            row[s.dv] = m[kTensor ? g / 8 : g % kRefs];
            row[s.dv + 1] = l[g];
        }
    }
    __syncthreads();
    join_warps<RG, WARPS>(a, merge, index, rows);
}

// Short caches: joins the sums that a block's warps left in shared memory for
// the one unit that the block has, writes the rows, and adds the step's weights
// to the scores.  lm: (normaliser, reference) by warp and row; there[w]: warp w
// had tiles; piece(w, g, c): four of its sums.
template <int WARPS, int ROWS, typename Piece>
__device__ void finish_unit(const AttendArgs& a, const Walk& u, int64_t row0, int rows, const float2 (*lm)[ROWS],
                            const int* there, float2* refs, Piece piece) {
    const View& s = a.s;
    const int c4 = s.dv / 4;
    for (int i = threadIdx.x; i < rows * c4; i += WARPS * 32) {
        const int g = i / c4, c = i - g * c4;
        float m = -CUDART_INF_F, l = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
            if (there[w]) m = fmaxf(m, lm[w][g].y);
        const float ref = m == -CUDART_INF_F ? 0.f : m;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
            if (there[w]) {
                const float f = ex2(lm[w][g].y - ref);
                const float4 v = piece(w, g, c);
                l = fmaf(f, lm[w][g].x, l);
                o.x = fmaf(f, v.x, o.x), o.y = fmaf(f, v.y, o.y), o.z = fmaf(f, v.z, o.z), o.w = fmaf(f, v.w, o.w);
            }
        const bool none = nothing(m, l);
        float* to = a.out + (row0 + g) * s.dv + c * 4;
        to[0] = none ? 0.f : o.x / l, to[1] = none ? 0.f : o.y / l;
        to[2] = none ? 0.f : o.z / l, to[3] = none ? 0.f : o.w / l;
        if (c == 0) {
            if (a.lse) a.lse[row0 + g] = log_sum(m, l);
            refs[g] = make_float2(ref, none ? 0.f : 1.f / l);
        }
    }
    if (!a.logits) return;
    __syncthreads();   // (also orders the block's own logits before their reading)
    float* out = a.scores + ((int64_t)u.b * s.hkv + u.h) * s.cap;
    for (int key = threadIdx.x; key < u.len; key += WARPS * 32) {
        float sum = 0.f;
        for (int g = 0; g < rows; ++g) sum = fmaf(ex2(a.logits[(row0 + g) * s.cap + key] - refs[g].x), refs[g].y, sum);
        out[key] += sum;
    }
}

// fp32 pages, on CUDA cores (their products keep 24 bits): 8 keys a step, two or
// three stages a warp.  For the logits a lane holds one key and a quarter of the
// width, for the values four columns (and, where fewer than 32 lanes cover the
// width, every second key).  DP: d and dv rounded up to 64, 128 or 256.  Long
// passes are bound by bytes (4 x 32768 tokens of 128-wide heads: 169 us, 6.35 TB/s).
// Few bytes a warp are not: 57 MB of ragged 64-wide heads take 16.8 us (3.3 TB/s),
// where a step moves 4 KB behind a chain of shuffles, 2^x and shared memory, 400
// instructions, and a scheduler issues in 39 % of its cycles.
constexpr int kSimtKeys = 8;
template <int DP> constexpr int kSimtStages = DP > 64 ? 2 : 3;

template <int DP> using SimtRing = Ring<kSimtKeys, DP, 4, kSimtStages<DP>>;
template <int DP, int RG>
struct SimtSmem {
    static constexpr int q = SimtRing<DP>::kBytes, p = q + RG * DP * 4, warp = p + kSimtKeys * RG * 8;
    static constexpr int total = kSimtWarps * warp;
};

// SHORT: a block has one unit, its warps the unit's tiles in turn, and no join follows.
template <int DP, int RG, bool SHORT>
__global__ void __launch_bounds__(kSimtWarps * 32) cache_attend_simt_kernel(const AttendArgs a) {
    constexpr int KEYS = kSimtKeys, kChunks = DP / 4;
    constexpr int kGroups = kChunks < 32 ? 32 / kChunks : 1;      // key groups of the value sums
    constexpr int kCols = kChunks < 32 ? 1 : kChunks / 32;        // a lane's column quadruples
    using L = SimtSmem<DP, RG>;
    extern __shared__ __align__(128) char smem[];
    __shared__ int place_sh[1 + kSimtWarps], pre[SHORT ? 1 : kPlaces];
    __shared__ float2 lm_sh[kSimtWarps][RG], refs[RG];
    __shared__ int there[kSimtWarps];
    constexpr int kStride = SHORT ? kSimtWarps : 1;
    if (!a.csplits) grid_dependency_wait();   // (with a coreset its kernel has waited)
    grid_dependents_launch();
    const View& s = a.s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    char* mem = smem + warp * L::warp;
    float* q = reinterpret_cast<float*>(mem + L::q);
    uint64_t* p = reinterpret_cast<uint64_t*>(mem + L::p);   // a step's weights, each twice (as a pair)
    Walk now, ahead;
    if (SHORT) {
        now.one(a, blockIdx.x, warp, KEYS);
        if (lane == 0) there[warp] = now.left > 0;
    } else {
        const int step = (s.B + kPlaces - 1) / kPlaces;
        const Place at = scan_tiles<kSimtWarps * 32>(s, a.lens, KEYS, s.hkv * a.row_tiles, -1, pre, step, a.status, place_sh);
        now.start(a, Share(at.total, a.blocks * kSimtWarps), pre, step, blockIdx.x * kSimtWarps + warp, KEYS);
    }
    const Walk unit = now;
    ahead = now;
    SimtRing<DP> ring;
    ring.init(a, mem);
    constexpr int kStages = kSimtStages<DP>;
    uint32_t masks = 0;   // the live keys of the steps in the ring, a byte each, the next one lowest after a fetch
    auto fetch = [&](int stage) {   // the next step's copies; where the one after it is
        masks >>= 8;
        if (ahead.left > 0) {
            masks |= ring.fetch(a, stage) << (8 * (kStages - 1));
            if (ahead.skip(a, kStride, KEYS)) ring.enter(a, ahead);
            ring.locate(a, ahead);
        }
        cp_async_commit();
    };
    ring.enter(a, ahead);
    ring.locate(a, ahead);
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) fetch(i);
    const int key = lane % KEYS, part = lane / KEYS;
    int stage = 0;
    while (now.left > 0) {
        // the share of one unit: steps now.k up to `last`
        const int rows = min(a.rows, s.group - now.rt * a.rows), g0 = now.h * s.group + now.rt * a.rows;
        const int start = now.k, last = min(now.tiles, now.k + now.left);
        const int64_t row0 = (int64_t)now.b * s.hq + g0, part_row = now.part_row(a);
        const float* src = static_cast<const float*>(a.Q) + now.b * a.q_batch + (int64_t)g0 * a.q_head;
#pragma unroll 4
        for (int i = lane; i < RG * DP; i += 32) {
            const int g = i / DP, col = i % DP;
            q[i] = g < rows && col < s.d ? src[g * a.q_head + col] * a.qscale : 0.f;
        }
        float m[RG], l[RG];
        uint64_t o[RG][kCols * 2];
#pragma unroll
        for (int g = 0; g < RG; ++g) {
            m[g] = -CUDART_INF_F;
            l[g] = 0.f;
#pragma unroll
            for (int i = 0; i < kCols * 2; ++i) o[g][i] = 0;
        }
        for (int at_k = start; at_k < last; at_k += kStride) {
        cp_async_wait<kStages - 2>();
        __syncwarp();
        fetch(stage == 0 ? kStages - 1 : stage - 1);   // the stage that the last step read is free
        const uint32_t mask = masks & 0xff;
        const char* krows = mem + stage * SimtRing<DP>::kStage;
        const char* vrows = krows + KEYS * SimtRing<DP>::kRow;
        uint64_t xx[RG];
#pragma unroll
        for (int g = 0; g < RG; ++g) xx[g] = 0;
#pragma unroll 8
        for (int i = 0; i < kChunks / 4; ++i) {
            const int ch = part + 4 * i;
            const ulonglong2 k4 = *reinterpret_cast<const ulonglong2*>(krows + key * SimtRing<DP>::kRow + (ch ^ key) * 16);
#pragma unroll
            for (int g = 0; g < RG; ++g) {
                const ulonglong2 q4 = *reinterpret_cast<const ulonglong2*>(q + g * DP + ch * 4);
                xx[g] = fma2(k4.x, q4.x, xx[g]);
                xx[g] = fma2(k4.y, q4.y, xx[g]);
            }
        }
        float x[RG];
#pragma unroll
        for (int g = 0; g < RG; ++g) {
            const float2 v = halves(xx[g]);
            x[g] = v.x + v.y;
        }
        const bool ok = (mask >> key) & 1;
        const int pos = at_k * KEYS + key;
#pragma unroll
        for (int g = 0; g < RG; ++g) {
            x[g] += __shfl_xor_sync(0xffffffffu, x[g], 8);
            x[g] += __shfl_xor_sync(0xffffffffu, x[g], 16);
            if (!ok) x[g] = -CUDART_INF_F;
            if (a.logits && part == 0 && pos < now.len && g < rows)
                a.logits[(row0 + g) * s.cap + pos] = x[g];
            float top = x[g];
#pragma unroll
            for (int e = 1; e < KEYS; e <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, e));
            if (top > m[g]) {
                const float f = ex2(m[g] - (top + kAhead));   // 0 where nothing was summed yet
                m[g] = top + kAhead;
                l[g] *= f;
#pragma unroll
                for (int i = 0; i < kCols * 2; ++i) o[g][i] = mul2(o[g][i], pair_of(f, f));
            }
            // nothing but masked keys so far: the reference is 0, every weight 2^-inf = 0
            const float w = ex2(x[g] - (m[g] == -CUDART_INF_F ? 0.f : m[g]));
            if (part == 0) {
                l[g] += w;
                p[key * RG + g] = pair_of(w, w);
            }
        }
        __syncwarp();
#pragma unroll
        for (int j0 = 0; j0 < KEYS; j0 += kGroups) {
            const int j = j0 + (kGroups > 1 ? lane / kChunks : 0);
            uint64_t w[RG];
#pragma unroll
            for (int g = 0; g < RG; ++g) w[g] = p[j * RG + g];
#pragma unroll
            for (int n = 0; n < kCols; ++n) {
                const int ch = (kGroups > 1 ? lane % kChunks : lane) + n * 32;
                const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(vrows + j * SimtRing<DP>::kRow + (ch ^ (j & 7)) * 16);
#pragma unroll
                for (int g = 0; g < RG; ++g) {
                    o[g][n * 2] = fma2(w[g], y.x, o[g][n * 2]);
                    o[g][n * 2 + 1] = fma2(w[g], y.y, o[g][n * 2 + 1]);
                }
            }
        }
        __syncwarp();
        stage = stage + 1 == kStages ? 0 : stage + 1;
        }
        // finished rows where the share is the whole unit, else partial rows
        const bool whole = !SHORT && start == 0 && last == now.tiles && !a.csplits && !a.logits;
#pragma unroll
        for (int g = 0; g < RG; ++g) {
#pragma unroll
            for (int e = 1; e < 32; e <<= 1) l[g] += __shfl_xor_sync(0xffffffffu, l[g], e);
            float v[kCols * 4];
#pragma unroll
            for (int i = 0; i < kCols * 2; ++i) {
                const float2 u = halves(o[g][i]);
                v[2 * i] = u.x, v[2 * i + 1] = u.y;
            }
#pragma unroll
            for (int e = 32 / kGroups; e < 32; e <<= 1)
#pragma unroll
                for (int i = 0; i < kCols * 4; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], e);
            if (g >= rows) continue;
            const bool none = nothing(m[g], l[g]);
            float* to = SHORT ? reinterpret_cast<float*>(mem) + g * s.dv   // (the ring is idle)
                      : whole ? a.out + (row0 + g) * s.dv : a.parts + (part_row + g) * s.dv;
#pragma unroll
            for (int n = 0; n < kCols; ++n) {
                const int col = (lane + n * 32) * 4;
                if (lane < 32 / kGroups && col < s.dv)
#pragma unroll
                    for (int e = 0; e < 4; ++e) to[col + e] = whole ? (none ? 0.f : v[n * 4 + e] / l[g]) : v[n * 4 + e];
            }
            if (lane == 0) {
                if (SHORT) lm_sh[warp][g] = make_float2(l[g], m[g]);
                else if (!whole) a.parts_lm[part_row + g] = make_float2(l[g], m[g]);
                else if (a.lse) a.lse[row0 + g] = log_sum(m[g], l[g]);
            }
        }
        if (SHORT) break;
        now.skip(a, last - start, KEYS);
    }
    if (SHORT) {
        __syncthreads();
        const int g0 = unit.h * s.group + unit.rt * a.rows;
        finish_unit<kSimtWarps, RG>(a, unit, (int64_t)unit.b * s.hq + g0, min(a.rows, s.group - unit.rt * a.rows), lm_sh,
                                    there, refs, [&](int w, int g, int c) {
                                        return *reinterpret_cast<const float4*>(smem + w * L::warp + (g * s.dv + c * 4) * 4);
                                    });
        return;
    }
    if (a.csplits) grid_dependency_wait();
}

constexpr int kMmaKeys = 16;     // keys of one warp's step
// Stages of a warp's ring, and warps of a block: what fits two blocks an SM (one for the widest rows).
template <int DP> constexpr int kMmaStages = DP > 128 ? 2 : 3;
template <int DP> constexpr int kMmaWarps = DP > 128 ? 6 : 4;

// Four columns of a warp's sums as they stand in shared memory (see the kernel's end).
template <int DP>
__device__ __forceinline__ float4 sums_at(const float* sums, int row, int c) {
    return *reinterpret_cast<const float4*>(sums + row * DP + ((c / 2 ^ (row & 7)) * 4 + (c & 1) * 2) * 2);
}

template <int DP> using MmaRing = Ring<kMmaKeys, DP, 2, kMmaStages<DP>>;

// bf16 pages on tensor cores (mma.sync: a group's 1 to 16 query rows fill one
// 16-row tile at most, and the pass is bound by the bytes of the keys and
// values, so the wider tcgen05 tiles would only hold more padding).  A warp
// takes 16 keys a step.  DP: d and dv rounded up to 64, 128 or 256.
// SETS: how the weights' three terms meet the 16 rows of the value product.
//   1  up to 4 query rows, each four times in the tile (r, r + 4, r + 8, r + 12):
//      the copies carry the terms, so one product adds all three
//   2  up to 8 rows, each twice: two products
//   3  up to 16 rows: three products
// DP = 256 needs more than the 255 registers there are and spills up to 628 bytes
// a thread: 2 x 32768 tokens 106 us, 5.0 TB/s (128-wide heads of as many bytes 92 us).
// SHORT: as above.
template <int DP, int SETS, bool SHORT>
__global__ void __launch_bounds__(kMmaWarps<DP> * 32) cache_attend_mma_kernel(const AttendArgs a) {
    using bf16 = __nv_bfloat16;
    constexpr int kRows = SETS == 1 ? 4 : SETS == 2 ? 8 : 16;
    constexpr int KEYS = kMmaKeys, kRow = MmaRing<DP>::kRow;
    constexpr int kStages = kMmaStages<DP>, kBlockWarps = kMmaWarps<DP>;
    constexpr int kMine = SETS == 3 ? 2 : 1;               // rows of a lane
    extern __shared__ __align__(128) char smem[];
    __shared__ int place_sh[1 + kBlockWarps], pre[SHORT ? 1 : kPlaces];
    __shared__ float2 lm_sh[kBlockWarps][kRows], refs[kRows];
    __shared__ int there[kBlockWarps];   // SHORT: 0, or 1 + where in its ring a warp's sums are
    constexpr int kStride = SHORT ? kBlockWarps : 1;
    if (!a.csplits) grid_dependency_wait();   // (with a coreset its kernel has waited)
    grid_dependents_launch();
    const View& s = a.s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = lane >> 2, pair = lane & 3;           // fragment row and column pair
    Walk now, ahead;
    if (SHORT) {
        now.one(a, blockIdx.x, warp, KEYS);
        if (lane == 0) there[warp] = now.left > 0;
    } else {
        const int step = (s.B + kPlaces - 1) / kPlaces;
        const Place at = scan_tiles<kBlockWarps * 32>(s, a.lens, KEYS, s.hkv * a.row_tiles, -1, pre, step, a.status, place_sh);
        now.start(a, Share(at.total, a.blocks * kBlockWarps), pre, step, blockIdx.x * kBlockWarps + warp, KEYS);
    }
    const Walk unit = now;
    ahead = now;
    MmaRing<DP> ring;
    char* mem = smem + warp * MmaRing<DP>::kBytes;
    const uint32_t stages = (uint32_t)__cvta_generic_to_shared(mem);
    ring.init(a, mem);
    uint64_t masks = 0;   // the live keys of the steps in the ring, 16 bits each, the next one lowest after a fetch
    auto fetch = [&](int stage) {   // the next step's copies; where the one after it is
        masks >>= 16;
        if (ahead.left > 0) {
            masks |= (uint64_t)ring.fetch(a, stage) << (16 * (kStages - 1));
            if (ahead.skip(a, kStride, KEYS)) ring.enter(a, ahead);
            ring.locate(a, ahead);
        }
        cp_async_commit();
    };
    ring.enter(a, ahead);
    ring.locate(a, ahead);
#pragma unroll 1
    for (int p = 0; p < kStages - 1; ++p) fetch(p);
    int stage = 0;
    while (now.left > 0) {
        // the share of one unit: steps now.k up to `last`
        const int rows = min(a.rows, s.group - now.rt * a.rows), g0 = now.h * s.group + now.rt * a.rows;
        const int start = now.k, last = min(now.tiles, now.k + now.left);
        const int64_t row0 = (int64_t)now.b * s.hq + g0, part_row = now.part_row(a);
        QueryFragments<DP, kRows> q;                       // (as they are: the logits are scaled in fp32)
        q.load(a, now.b, g0, rows);
        uint64_t o[DP / 8][2];                             // pairs of fp32 sums: row quad, row quad + 8
        float m[kMine], l[kMine];
#pragma unroll
        for (int n = 0; n < DP / 8; ++n) o[n][0] = o[n][1] = 0;
#pragma unroll
        for (int i = 0; i < kMine; ++i) m[i] = -CUDART_INF_F, l[i] = 0.f;
        for (int at_k = start; at_k < last; at_k += kStride) {
        cp_async_wait<kStages - 2>();
        __syncwarp();
        const uint32_t kd = stages + stage * MmaRing<DP>::kStage, vd = kd + KEYS * kRow;
        fetch(stage == 0 ? kStages - 1 : stage - 1);       // the stage that the last step read is free
        const uint32_t mask = (uint32_t)masks & 0xffffu;
        // logits: keys 0..7 in x[0], 8..15 in x[1]
        float x[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
        {
            const int row = (lane & 7) + ((lane >> 4) << 3);
            const uint32_t base = kd + row * kRow;
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) {
                uint32_t f[4];
                ldmatrix4(f, base + (((2 * k + ((lane >> 3) & 1)) ^ (row & 7)) << 4));
                q.step(x[0], k, f[0], f[1]);
                q.step(x[1], k, f[2], f[3]);
            }
        }
        uint32_t w[kMine][2][3];                           // weights' terms: [row][key octet][term]
#pragma unroll
        for (int r = 0; r < kMine; ++r) {
            float y[4];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    y[2 * n + e] = x[n][2 * r + e] * a.qscale;
            if (mask != 0xffffu)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!((mask >> (e / 2 * 8 + pair * 2 + e % 2)) & 1)) y[e] = -CUDART_INF_F;
            if (a.logits && quad + 8 * r < rows) {
                const int pos = at_k * KEYS;
                float* to = a.logits + (row0 + quad + 8 * r) * s.cap + pos;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int key = n * 8 + pair * 2 + e;
                        if (pos + key < now.len) to[key] = y[2 * n + e];
                    }
            }
            float top = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const bool grow = top > m[r];
            if (__any_sync(0xffffffffu, grow)) {
                const float f = grow ? ex2(m[r] - (top + kAhead)) : 1.f;
                if (grow) m[r] = top + kAhead;
                l[r] *= f;
                const uint64_t ff = pair_of(f, f);
#pragma unroll
                for (int n = 0; n < DP / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (SETS != 3 || e == r) o[n][e] = mul2(o[n][e], ff);
            }
            const float ref = m[r] == -CUDART_INF_F ? 0.f : m[r];   // only masked keys so far: weights 2^-inf = 0
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = ex2(y[e] - ref);
            l[r] += (y[0] + y[1]) + (y[2] + y[3]);
            split_bf16(y[0], y[1], w[r][0]);
            split_bf16(y[2], y[3], w[r][1]);
        }
        // values
        {
            const int row = lane & 15;
            const uint32_t base = vd + row * kRow;
            uint32_t p0 = 0, p1 = 0, p2 = 0, p3 = 0;
            if (SETS == 1) {   // rows 0-3: term 0, 8-11: term 1, 4-7: term 2, 12-15: as good as nothing
                const bool up = quad < 4;
                p0 = up ? w[0][0][0] : w[0][0][2]; p1 = up ? w[0][0][1] : kLeast;
                p2 = up ? w[0][1][0] : w[0][1][2]; p3 = up ? w[0][1][1] : kLeast;
            }
#pragma unroll
            for (int n = 0; n < DP / 16; ++n) {
                uint32_t f[4];
                ldmatrix4t(f, base + (((2 * n + (lane >> 4)) ^ (row & 7)) << 4));
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    // The product of the 16 keys by itself, then an ordinary fp32 addition: the
                    // tensor cores' own accumulation does not round to nearest, and over the
                    // thousands of steps of a long cache its errors all point one way
                    // (4.3e-6 of the output at 131072 keys, 0.7e-6 so).
                    float z[4];
                    const uint32_t b0 = f[2 * u], b1 = f[2 * u + 1];
                    if (SETS == 1) {
                        mma16816_new(z, p0, p1, p2, p3, b0, b1);
                    } else if (SETS == 2) {
                        mma16816_new(z, w[0][0][0], w[0][0][1], w[0][1][0], w[0][1][1], b0, b1);
                        mma16816(z, w[0][0][2], kLeast, w[0][1][2], kLeast, b0, b1);
                    } else {
                        mma16816_new(z, w[0][0][0], w[kMine - 1][0][0], w[0][1][0], w[kMine - 1][1][0], b0, b1);
                        mma16816(z, w[0][0][1], w[kMine - 1][0][1], w[0][1][1], w[kMine - 1][1][1], b0, b1);
                        mma16816(z, w[0][0][2], w[kMine - 1][0][2], w[0][1][2], w[kMine - 1][1][2], b0, b1);
                    }
                    o[2 * n + u][0] = add2(o[2 * n + u][0], pair_of(z[0], z[1]));
                    o[2 * n + u][1] = add2(o[2 * n + u][1], pair_of(z[2], z[3]));
                }
            }
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
        __syncwarp();
        }
        // finished rows where the share is the whole unit, else partial rows
        const bool whole = !SHORT && start == 0 && last == now.tiles && !a.csplits && !a.logits;
        // The sums go through the stage that was read last (free until the next fetch): pairs of columns at
        // row quad (quad + 8), XOR-swizzled, then out in 16-byte pieces.  Straight from the fragments the
        // code is five times as long, and a warp that runs it once waits for its instructions.
        float* out_sh = reinterpret_cast<float*>(mem + (stage == 0 ? kStages - 1 : stage - 1) * MmaRing<DP>::kStage);
#pragma unroll
        for (int n = 0; n < DP / 8; ++n)
#pragma unroll
            for (int r = 0; r < kMine; ++r)
                *reinterpret_cast<uint64_t*>(out_sh + (quad + 8 * r) * DP + ((n ^ quad) * 4 + pair) * 2) =
                    SETS == 3 ? o[n][r] : add2(o[n][0], o[n][1]);
#pragma unroll
        for (int r = 0; r < kMine; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            const int g = quad + 8 * r;
            if (pair == 0 && g < rows) {
                if (SHORT) lm_sh[warp][g] = make_float2(l[r], m[r]);
                else if (!whole) a.parts_lm[part_row + g] = make_float2(l[r], m[r]);
                else if (a.lse) a.lse[row0 + g] = log_sum(m[r], l[r]);
            }
        }
        if (SHORT) {
            if (lane == 0) there[warp] = 1 + (int)(reinterpret_cast<char*>(out_sh) - mem);
            break;
        }
        __syncwarp();
        const int c4 = s.dv / 4, pieces = rows * c4;
        float* to = whole ? a.out + row0 * s.dv : a.parts + part_row * s.dv;
#pragma unroll 1
        for (int i0 = 0; i0 < pieces; i0 += 32) {
            const int i = min(i0 + lane, pieces - 1), g = i / c4, c = i - g * c4;
            float4 v = sums_at<DP>(out_sh, g, c);
            if (SETS == 1) {   // the copies of the rows carried the third term
                const float4 u = sums_at<DP>(out_sh, g + 4, c);
                v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
            }
            if (whole) {
                float sum = __shfl_sync(0xffffffffu, l[0], (g & 7) * 4), top = __shfl_sync(0xffffffffu, m[0], (g & 7) * 4);
                if (SETS == 3) {
                    const float sum1 = __shfl_sync(0xffffffffu, l[kMine - 1], (g & 7) * 4);
                    const float top1 = __shfl_sync(0xffffffffu, m[kMine - 1], (g & 7) * 4);
                    if (g >= 8) sum = sum1, top = top1;
                }
                const bool none = nothing(top, sum);
                v.x = none ? 0.f : v.x / sum, v.y = none ? 0.f : v.y / sum;
                v.z = none ? 0.f : v.z / sum, v.w = none ? 0.f : v.w / sum;
            }
            if (i0 + lane < pieces) {
                float* p = to + (int64_t)g * s.dv + c * 4;   // (out need not be aligned to more than a value)
                if (whole) p[0] = v.x, p[1] = v.y, p[2] = v.z, p[3] = v.w;
                else *reinterpret_cast<float4*>(p) = v;
            }
        }
        __syncwarp();
        if (s.d < DP || s.dv < DP) {   // columns past the width are zeros again
            for (int i = lane; i < MmaRing<DP>::kStage / 16; i += 32)
                reinterpret_cast<uint4*>(out_sh)[i] = make_uint4(0, 0, 0, 0);
            __syncwarp();
        }
        now.skip(a, last - start, KEYS);
    }
    if (SHORT) {
        __syncthreads();
        const int g0 = unit.h * s.group + unit.rt * a.rows;
        finish_unit<kBlockWarps, kRows>(
            a, unit, (int64_t)unit.b * s.hq + g0, min(a.rows, s.group - unit.rt * a.rows), lm_sh, there, refs,
            [&](int w, int g, int c) {
                const float* sums = reinterpret_cast<const float*>(smem + w * MmaRing<DP>::kBytes + (there[w] - 1));
                float4 v = sums_at<DP>(sums, g, c);
                if (SETS == 1) {
                    const float4 u = sums_at<DP>(sums, g + 4, c);
                    v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
                }
                return v;
            });
        return;
    }
    if (a.csplits) grid_dependency_wait();
}

// Joins the partial rows of every query row, and adds the step's weights to
// the scores.  The first blocks take `cols` columns of a query row each: the
// sets' weights 2^(m - M) into shared memory, a set a thread, then the sums,
// four columns a thread and the sets spread over the rest (there are up to
// hundreds of sets and few rows, and what counts is the loads in flight).  With
// scores, the others (`chunks` for each sequence and kv head, which bounds them where
// the tables are far larger than the lengths) take kScoreKeys positions at a time:
// the rows' references and normalisers first (a warp a row), then the logits
// that the pages' kernel left, 2^(x - m) / L summed over the group's rows.
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinSets = 1024;   // sets whose weights are held at a time
constexpr int kScoreKeys = 2048;
constexpr int kScoreRows = 64;    // rows whose references are held at a time

__global__ void __launch_bounds__(kJoinThreads, 4) cache_join_kernel(const AttendArgs a, int tile, int warps, int cols, int chunks) {
    __shared__ int place_sh[1 + kJoinWarps];
    __shared__ __align__(16) float4 sums[kJoinThreads];
    __shared__ float weight[kJoinSets];
    __shared__ float red[kJoinWarps];
    __shared__ float refs[kScoreRows][2];
    const View& s = a.s;
    const int per_tile = s.hkv * a.row_tiles, dv = s.dv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per_seq = cols ? s.hq * ((dv + cols - 1) / cols) : (s.hq + kJoinWarps - 1) / kJoinWarps;
    const int row_blocks = s.B * per_seq;
    const bool score = (int)blockIdx.x >= row_blocks;
    int b, hq0, key0 = 0, col0 = 0;
    if (!score) {
        b = blockIdx.x / per_seq;
        const int i = blockIdx.x - b * per_seq;
        hq0 = cols ? i % s.hq : i * kJoinWarps + warp;
        col0 = cols ? i / s.hq * cols : 0;
    } else {
        const int i = blockIdx.x - row_blocks, unit = i / chunks;
        b = unit / s.hkv;
        hq0 = (unit - b * s.hkv) * s.group;
        key0 = (i - unit * chunks) * kScoreKeys;
    }
    const int len = checked_len(a.lens, b, s.cap, a.status);
    if (score && key0 >= len) return;
    const int key_first = key0;
    const Place at = scan_tiles<kJoinThreads>(s, a.lens, tile, per_tile, b, nullptr, 1, a.status, place_sh);
    const Share share(at.total, warps);
    const int tiles = (len + tile - 1) / tile;
    // rows of partial sums of query row hq: first of the pages' (one per stretch), then of the coreset's
    int64_t page0 = 0, core0 = 0;
    int n_pages = 0, n = 0;
    auto find_sets = [&](int hq) {
        const int h = hq / s.group, g = hq - h * s.group, rt = g / a.rows, in_unit = g - rt * a.rows;
        const int in_b = h * a.row_tiles + rt;
        n_pages = 0;
        if (tiles > 0) {
            const int t0 = at.before + in_b * (tiles + kUnitCost) + kUnitCost;
            const int c0 = share.of(t0), c1 = share.of(t0 + tiles - 1);
            if (c0 == c1 && !a.csplits && !a.logits) return false;   // finished by the warp itself
            page0 = ((int64_t)b * per_tile + in_b + c0) * a.rows + in_unit;
            n_pages = c1 - c0 + 1;
        }
        core0 = ((int64_t)b * per_tile + in_b) * a.csplits * a.rows + in_unit;
        n = n_pages + a.csplits;
        return true;
    };
    auto lm = [&](int i) {   // (normaliser, reference) of a set
        return *(i < n_pages ? a.parts_lm + page0 + (int64_t)i * a.rows : a.cparts_lm + core0 + (int64_t)(i - n_pages) * a.rows);
    };
    const bool to_join = score || (hq0 < s.hq && find_sets(hq0));
    grid_dependency_wait();   // the partial rows (and everything before them) are there from here on
    if (!to_join) return;
    // a warp's reference and normaliser over all sets, in an order that the number of sets alone decides
    auto totals = [&](float& m, float& l) {
        m = -CUDART_INF_F;
#pragma unroll 4
        for (int i = lane; i < n; i += 32) m = fmaxf(m, lm(i).y);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float ref = m == -CUDART_INF_F ? 0.f : m;
        l = 0.f;
#pragma unroll 4
        for (int i = lane; i < n; i += 32) {
            const float2 v = lm(i);
            l = fmaf(ex2(v.y - ref), v.x, l);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    };
    const int64_t step = (int64_t)a.rows * dv;
    if (!score && !cols) {
        float m, l;
        totals(m, l);
        const float ref = m == -CUDART_INF_F ? 0.f : m;
        const int64_t row = (int64_t)b * s.hq + hq0;
        const bool empty = nothing(m, l);
        for (int col = lane * 4; col < dv; col += 128) {
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            const float* rows_p = a.parts + page0 * dv + col;
            const float* rows_c = a.cparts + core0 * dv + col;
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
                const float f = ex2(lm(i).y - ref);
                const float4 v = *reinterpret_cast<const float4*>(i < n_pages ? rows_p + i * step
                                                                              : rows_c + (i - n_pages) * step);
                o.x = fmaf(f, v.x, o.x), o.y = fmaf(f, v.y, o.y), o.z = fmaf(f, v.z, o.z), o.w = fmaf(f, v.w, o.w);
            }
            float* to = a.out + row * dv + col;
            to[0] = empty ? 0.f : o.x / l, to[1] = empty ? 0.f : o.y / l;
            to[2] = empty ? 0.f : o.z / l, to[3] = empty ? 0.f : o.w / l;
        }
        if (lane == 0 && a.lse) a.lse[row] = log_sum(m, l);
        return;
    }
    if (!score) {
        // the maximum over all sets
        float m = -CUDART_INF_F;
        for (int i = threadIdx.x; i < n; i += kJoinThreads) m = fmaxf(m, lm(i).y);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) red[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, red[w]);
        const float ref = m == -CUDART_INF_F ? 0.f : m;
        const int quads = cols / 4, groups = kJoinThreads / quads, q = threadIdx.x % quads, sg = threadIdx.x / quads;
        const int col = col0 + q * 4;
        const bool in = col < dv && sg < groups;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f;
        for (int i0 = 0; i0 < n; i0 += kJoinSets) {
            const int held = min(kJoinSets, n - i0);
            __syncthreads();
            for (int i = threadIdx.x; i < held; i += kJoinThreads) {
                const float2 v = lm(i0 + i);
                const float f = ex2(v.y - ref);
                weight[i] = f;
                l = fmaf(f, v.x, l);
            }
            __syncthreads();
            if (in) {
                const float* rows_p = a.parts + page0 * dv + col;
                const float* rows_c = a.cparts + core0 * dv + col;
#pragma unroll 4
                for (int i = sg; i < held; i += groups) {
                    const int j = i0 + i;
                    const float4 v = *reinterpret_cast<const float4*>(j < n_pages ? rows_p + j * step
                                                                                  : rows_c + (j - n_pages) * step);
                    const float f = weight[i];
                    o.x = fmaf(f, v.x, o.x), o.y = fmaf(f, v.y, o.y), o.z = fmaf(f, v.z, o.z), o.w = fmaf(f, v.w, o.w);
                }
            }
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
        __syncthreads();
        if (lane == 0) red[warp] = l;
        sums[threadIdx.x] = o;
        __syncthreads();
        l = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) l += red[w];
        for (int half = groups; half > 1;) {   // the groups' sums, in a fixed tree
            const int low = (half + 1) / 2;
            if (sg < low && sg + low < half) {
                const float4 v = sums[threadIdx.x + low * quads];
                float4& t = sums[threadIdx.x];
                t.x += v.x, t.y += v.y, t.z += v.z, t.w += v.w;
            }
            half = low;
            __syncthreads();
        }
        const int64_t row = (int64_t)b * s.hq + hq0;
        const bool empty = nothing(m, l);
        if (threadIdx.x < cols && col0 + threadIdx.x < dv)
            a.out[row * dv + col0 + threadIdx.x] = empty ? 0.f : reinterpret_cast<const float*>(sums)[threadIdx.x] / l;
        if (threadIdx.x == 0 && col0 == 0 && a.lse) a.lse[row] = log_sum(m, l);
        return;
    }
    // the stretches of kScoreKeys positions that this block takes, every chunks-th of them
    for (; key0 < len; key0 += chunks * kScoreKeys) {
        float acc[kScoreKeys / kJoinThreads];
#pragma unroll
        for (int i = 0; i < kScoreKeys / kJoinThreads; ++i) acc[i] = 0.f;
        for (int r0 = 0; r0 < s.group; r0 += kScoreRows) {
            const int rows = min(kScoreRows, s.group - r0);
            if (key0 == key_first || s.group > kScoreRows) {
                __syncthreads();
                for (int r = warp; r < rows; r += kJoinWarps) {
                    find_sets(hq0 + r0 + r);
                    float m, l;
                    totals(m, l);
                    if (lane == 0) {
                        refs[r][0] = m == -CUDART_INF_F ? 0.f : m;
                        refs[r][1] = nothing(m, l) ? 0.f : 1.f / l;   // no weight anywhere: 0 for every key
                    }
                }
                __syncthreads();
            }
#pragma unroll 4
            for (int r = 0; r < rows; ++r) {
                const float* x = a.logits + ((int64_t)b * s.hq + hq0 + r0 + r) * s.cap;
                const float ref = refs[r][0], inv = refs[r][1];
#pragma unroll
                for (int i = 0; i < kScoreKeys / kJoinThreads; ++i) {
                    const int key = key0 + i * kJoinThreads + threadIdx.x;
                    if (key < len) acc[i] = fmaf(ex2(x[key] - ref), inv, acc[i]);
                }
            }
        }
        float* out = a.scores + ((int64_t)b * s.hkv + hq0 / s.group) * s.cap;
#pragma unroll
        for (int i = 0; i < kScoreKeys / kJoinThreads; ++i) {
            const int key = key0 + i * kJoinThreads + threadIdx.x;
            if (key < len) out[key] += acc[i];
        }
    }
}

// Blocks of a kernel that the current device holds at once with `smem` bytes
// each.  The answer (and the kernel's shared-memory limit, set before it is
// asked for) is kept per kernel, device and size: the calls cost more than a
// short attention's kernels do.
wc_status resident_blocks(const void* kern, int threads, int smem, int* out) {
    struct Entry { const void* kern; int dev, smem, blocks; };
    constexpr int kEntries = 256;
    static Entry table[kEntries];
    static std::atomic<int> used{0};
    static std::mutex lock;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return WC_ERR_CUDA;
    auto find = [&](int n) {
        for (int i = 0; i < n; ++i)
            if (table[i].kern == kern && table[i].dev == dev && table[i].smem == smem) return table[i].blocks;
        return 0;
    };
    if ((*out = find(used.load(std::memory_order_acquire))) > 0) return WC_OK;
    std::lock_guard<std::mutex> hold(lock);
    const int n = used.load(std::memory_order_relaxed);
    if ((*out = find(n)) > 0) return WC_OK;
    int nsm = 0, per_sm = 0, limit = 0;
    if (cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&limit, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess)
        return WC_ERR_CUDA;
    // the device's whole limit, so that entries of other sizes stay valid
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, limit - (int)fa.sharedSizeBytes) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem) != cudaSuccess || per_sm < 1)
        return WC_ERR_CUDA;
    *out = nsm * per_sm;
    if (n < kEntries) {
        table[n] = Entry{kern, dev, smem, *out};
        used.store(n + 1, std::memory_order_release);
    }
    return WC_OK;
}

using Kernel = void (*)(AttendArgs);

// Steps of a warp up to which a table counts as short, where the units are
// fewer than two an SM and where they are more.  Measured (with scores; one
// launch against two): 8 heads of 256 tokens, bf16 7.7 us against 9.3, of 512
// (8 steps) 12.0 against 9.6; 512 heads of up to 256 tokens 17.7 us against 22.3,
// of 512 27.5 against 28.0, of 1024 (16 steps) 49 against 42; fp32, half as many
// keys a step, alike by steps.
constexpr int kShortSteps = 6, kShortStepsMany = 8;

// Launches the coreset's kernel where there is one, the pages' (as many blocks
// as the GPU holds at once, or one per tile where there are fewer), and the join.
wc_status run(AttendArgs a, Kernel pages, Kernel short_pages, int warps, int smem, int tile, Kernel core, int core_smem,
              cudaStream_t st) {
    int room = 0, core_room = 0;
    const int64_t all_units = (int64_t)a.s.B * a.s.hkv * a.row_tiles;
    // Short tables without a coreset: a block for a unit, one launch and no partial rows.
    const int steps = (a.s.cap + tile * warps - 1) / (tile * warps);
    if (steps <= (all_units >= 2 * 148 ? kShortStepsMany : kShortSteps) && !a.csplits && !(a.scores && a.row_tiles > 1) && all_units <= INT32_MAX) {
        if (resident_blocks(reinterpret_cast<const void*>(short_pages), warps * 32, smem, &room) != WC_OK ||
            !launch(short_pages, all_units, warps * 32, smem, st, a))
            return WC_ERR_CUDA;
        return WC_OK;
    }
    const int64_t units = all_units, most = units * unit_places(a.s.cap, tile);
    const int64_t rows = (int64_t)a.s.B * a.s.hq, pairs = (int64_t)a.s.B * a.s.hkv;
    // score blocks of one (sequence, kv head): a stretch each, at most about 4096 blocks in all
    const int64_t chunks = min((int64_t)(a.s.cap + kScoreKeys - 1) / kScoreKeys, (4096 + pairs - 1) / pairs);
    // Where the rows are at most the blocks that the GPU holds at once, a block for as few columns (32 and up) of
    // a row as that allows (32 rows of 150 sets each: 3 us against 8 for a warp a row); where they are more, a
    // warp for a row (1024 rows of 5 sets: 7 us against 9).
    const int64_t most_blocks = 4 * 148;
    int cols = rows <= most_blocks ? 32 : 0;
    while (cols && cols < a.s.dv && rows * ((a.s.dv + cols - 1) / cols) > most_blocks) cols *= 2;
    const int64_t join = (cols ? rows * ((a.s.dv + cols - 1) / cols) : (int64_t)a.s.B * ((a.s.hq + kJoinWarps - 1) / kJoinWarps)) +
                         (a.scores ? chunks * pairs : 0);
    // (places are counted in 32 bits, also where they are rounded up to a multiple of the warps)
    if (most + max_warps(a.s) > INT32_MAX || join > INT32_MAX || units * a.csplits > INT32_MAX) return WC_ERR_UNSUPPORTED;
    if (resident_blocks(reinterpret_cast<const void*>(pages), warps * 32, smem, &room) != WC_OK) return WC_ERR_CUDA;
    if (a.csplits) {
        if (resident_blocks(reinterpret_cast<const void*>(core), kCoresetWarps * 32, core_smem, &core_room) != WC_OK ||
            !launch(core, units * a.csplits, kCoresetWarps * 32, core_smem, st, a))
            return WC_ERR_CUDA;
    }
    a.blocks = (int)min((most + warps - 1) / warps, (int64_t)min(room, max_warps(a.s) / warps));
    if (!launch(pages, a.blocks, warps * 32, smem, st, a) ||
        !launch(cache_join_kernel, join, kJoinThreads, 0, st, a, tile, a.blocks * warps, cols, (int)chunks))
        return WC_ERR_CUDA;
    return WC_OK;
}

template <int DP, int RG>
wc_status run_simt(const AttendArgs& a, cudaStream_t st) {
    return run(a, cache_attend_simt_kernel<DP, RG, false>, cache_attend_simt_kernel<DP, RG, true>, kSimtWarps, SimtSmem<DP, RG>::total, kSimtKeys,
               cache_coreset_kernel<float, RG, 8, DP>, CoresetSmem<float, 8, RG, DP>(a.s.d, a.s.dv).total, st);
}

template <int DP>
wc_status by_rows(const AttendArgs& a, cudaStream_t st) {
    switch (a.rows) {
        case 1: return run_simt<DP, 1>(a, st);
        case 2: return run_simt<DP, 2>(a, st);
        case 4: return run_simt<DP, 4>(a, st);
        default: return run_simt<DP, 8>(a, st);
    }
}

template <int DP, int SETS>
wc_status run_mma(const AttendArgs& a, cudaStream_t st) {
    constexpr int rows = SETS == 1 ? 4 : SETS == 2 ? 8 : 16;
    return run(a, cache_attend_mma_kernel<DP, SETS, false>, cache_attend_mma_kernel<DP, SETS, true>, kMmaWarps<DP>, kMmaWarps<DP> * MmaRing<DP>::kBytes, kMmaKeys,
               cache_coreset_kernel<__nv_bfloat16, rows, 8, DP>,
               CoresetSmem<__nv_bfloat16, 8, rows, DP>(a.s.d, a.s.dv).total, st);
}

template <int DP>
wc_status by_sets(const AttendArgs& a, cudaStream_t st) {
    return a.rows == 4 ? run_mma<DP, 1>(a, st) : a.rows == 8 ? run_mma<DP, 2>(a, st) : run_mma<DP, 3>(a, st);
}

}  // namespace

wc_status launch_attend(const AttendArgs& a, cudaStream_t st) {
    const int w = max(a.s.d, a.s.dv);
    if (a.s.dtype == WC_BF16)
        return w <= 64 ? by_sets<64>(a, st) : w <= 128 ? by_sets<128>(a, st) : by_sets<256>(a, st);
    return w <= 64 ? by_rows<64>(a, st) : w <= 128 ? by_rows<128>(a, st) : by_rows<256>(a, st);
}

}  // namespace cache
}  // namespace wc
