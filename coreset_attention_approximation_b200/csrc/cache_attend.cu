// cache_attend.cu — attention of one new token per sequence over a paged
// cache, optionally together with a weighted coreset:
//   L = sum_i a_i + sum_s a'_s W[s, dv],   a = exp(beta <q, k>)
//   out = (sum_i a_i v_i + sum_s a'_s W[s, :dv]) / L
// One pass over the keys and values with a running maximum per query row (in
// log2 units, so one multiplication by beta log2(e) is folded into the query):
// a partial result is (O, l, m) with O = sum 2^(x - m) v, l = sum 2^(x - m).
// The key tiles of the whole batch are divided evenly over the blocks
// (wc_cache.cuh), whatever the lengths, and a second kernel joins a unit's
// partial rows in order of the blocks.
#include "wc_cache.cuh"

namespace wc {
namespace cache {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

// Where a warp's 16 or 8 keys lie: lane j < NT holds key j's byte offsets.
struct KeyPlace {
    int64_t k, v;
    bool valid;
};

// Shared memory of one block of the CUDA-core kernel, in bytes.
template <int NT, int RG>
struct SimtSmem {
    int k_row, v_row;      // bytes of a staged row; k rows padded to an odd number of 16-byte units
    int stage, warp;       // bytes of one stage and of one warp's stages
    int q, p, merge, total;
    __host__ __device__ SimtSmem(int d, int dv, int esize) {
        k_row = d * esize;
        if ((k_row / 16) % 2 == 0) k_row += 16;
        v_row = dv * esize;
        stage = NT * (k_row + v_row);
        warp = 2 * stage;
        q = kWarps * warp;
        p = q + RG * d * 4;
        merge = p + kWarps * NT * RG * 4;
        total = merge + kWarps * RG * (dv + 2) * 4;
    }
};

template <typename T> __device__ __forceinline__ void load_chunk(const char* p, float* x);
template <> __device__ __forceinline__ void load_chunk<float>(const char* p, float* x) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
template <> __device__ __forceinline__ void load_chunk<__nv_bfloat16>(const char* p, float* x) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
// Four consecutive values as floats.
__device__ __forceinline__ void load_four(const char* row, int chunk, float x[4], float) {
    load_chunk<float>(row + chunk * 16, x);
}
__device__ __forceinline__ void load_four(const char* row, int chunk, float x[4], __nv_bfloat16) {
    const uint2 v = *reinterpret_cast<const uint2*>(row + chunk * 8);
    x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xffff0000u);
}

// The running state of one warp: its keys' sums for RG query rows.
template <int RG, int NVI>
struct Running {
    float m[RG], l[RG], o[RG][NVI * 4];   // l: this lane's share; o: this lane's columns and key group
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int g = 0; g < RG; ++g) {
            m[g] = -CUDART_INF_F;
            l[g] = 0.f;
#pragma unroll
            for (int i = 0; i < NVI * 4; ++i) o[g][i] = 0.f;
        }
    }
};

// Logits of NT staged keys against RG query rows: lane = (key, part of d).
// Every lane ends with its key's whole sums.
template <typename T, int RG, int NT>
__device__ __forceinline__ void tile_logits(const char* krows, int k_row, const float* q, int d, float s[RG]) {
    constexpr int kPer = 16 / sizeof(T);
    const int lane = threadIdx.x & 31, key = lane % NT, part = lane / NT;
    const char* row = krows + key * k_row;
#pragma unroll
    for (int g = 0; g < RG; ++g) s[g] = 0.f;
    for (int c = part; c < d / kPer; c += 32 / NT) {
        float x[kPer];
        load_chunk<T>(row + c * 16, x);
#pragma unroll
        for (int g = 0; g < RG; ++g) {
#pragma unroll
            for (int i = 0; i < kPer; i += 4) {
                const float4 y = *reinterpret_cast<const float4*>(q + g * d + c * kPer + i);
                s[g] = fmaf(x[i], y.x, s[g]);
                s[g] = fmaf(x[i + 1], y.y, s[g]);
                s[g] = fmaf(x[i + 2], y.z, s[g]);
                s[g] = fmaf(x[i + 3], y.w, s[g]);
            }
        }
    }
#pragma unroll
    for (int o = NT; o < 32; o <<= 1)
#pragma unroll
        for (int g = 0; g < RG; ++g) s[g] += __shfl_xor_sync(0xffffffffu, s[g], o);
}

// New maxima from a tile's logits (-inf where masked); rescales the state and
// leaves the tile's weights in p (shared, [NT][RG]).
template <int RG, int NT, int NVI>
__device__ __forceinline__ void tile_weights(Running<RG, NVI>& st, const float s[RG], float* p) {
    const int lane = threadIdx.x & 31, key = lane % NT, part = lane / NT;
#pragma unroll
    for (int g = 0; g < RG; ++g) {
        float top = s[g];
#pragma unroll
        for (int o = 1; o < NT; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (top > st.m[g]) {
            const float f = ex2(st.m[g] - top);   // 0 where nothing was summed yet
            st.m[g] = top;
            st.l[g] *= f;
#pragma unroll
            for (int i = 0; i < NVI * 4; ++i) st.o[g][i] *= f;
        }
        // nothing but masked keys so far: the reference is 0, every weight 2^-inf = 0
        const float w = ex2(s[g] - (st.m[g] == -CUDART_INF_F ? 0.f : st.m[g]));
        if (part == 0) {
            st.l[g] += w;
            p[key * RG + g] = w;
        }
    }
}

// Sums a warp's state over its lanes and leaves it in shared memory:
// [RG][dv + 2] with m and l behind the columns.
template <int RG, int NVI>
__device__ __forceinline__ void leave_state(Running<RG, NVI>& st, float* to, int dv, int groups) {
    const int lane = threadIdx.x & 31, cols = 32 / groups;
#pragma unroll
    for (int g = 0; g < RG; ++g) {
        float l = st.l[g];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        for (int o = cols; o < 32; o <<= 1)
#pragma unroll
            for (int i = 0; i < NVI * 4; ++i) st.o[g][i] += __shfl_xor_sync(0xffffffffu, st.o[g][i], o);
        float* row = to + g * (dv + 2);
        if (lane < cols) {
#pragma unroll
            for (int i = 0; i < NVI; ++i) {
                const int c = lane + i * cols;
                if (c < dv / 4)
#pragma unroll
                    for (int e = 0; e < 4; ++e) row[c * 4 + e] = st.o[g][i * 4 + e];
            }
        }
        if (lane == 0) {
            row[dv] = st.m[g];
            row[dv + 1] = l;
        }
    }
}

// No key was summed (every one masked, or none there).  A NaN among the logits
// leaves l NaN and is no such row.
__device__ __forceinline__ bool nothing(float m, float l) { return m == -CUDART_INF_F && l == 0.f; }

// log of the normaliser l 2^m.
__device__ __forceinline__ float log_sum(float m, float l) {
    return nothing(m, l) ? m : (float)(((double)m + log2((double)l)) * 0.69314718055994530942);
}

// Joins the block's warps (shared, [warps][RG][dv + 2]) and writes the rows:
// as partial rows (O, l, m) at `part`, or finished to out / lse.
template <int RG>
__device__ __forceinline__ void join_warps(const AttendArgs& a, const float* merge, float* part, int64_t row0,
                                           int rows) {
    const int dv = a.s.dv, ld = dv + 2;
    for (int g = 0; g < rows; ++g) {
        const float* r = merge + g * ld;
        float m = -CUDART_INF_F;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, r[w * RG * ld + dv]);
        const float ref = m == -CUDART_INF_F ? 0.f : m;
        float f[kWarps], l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            f[w] = ex2(r[w * RG * ld + dv] - ref);
            l += f[w] * r[w * RG * ld + dv + 1];
        }
        for (int c = threadIdx.x; c < dv; c += kThreads) {
            float o = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) o = fmaf(f[w], r[w * RG * ld + c], o);
            if (part) part[(int64_t)g * c1_row(dv) + c] = o;
            else a.out[(row0 + g) * dv + c] = nothing(m, l) ? 0.f : o / l;
        }
        if (threadIdx.x == 0) {
            if (part) {
                part[(int64_t)g * c1_row(dv) + dv] = l;
                part[(int64_t)g * c1_row(dv) + dv + 1] = m;
            } else if (a.lse) {
                a.lse[row0 + g] = log_sum(m, l);
            }
        }
    }
}

// Query rows of one unit into shared memory as fp32, scaled to log2 units;
// rows past the group are zero.
template <typename T, int RG>
__device__ __forceinline__ void load_queries(const AttendArgs& a, int b, int g0, int rows, float* q) {
    const T* src = static_cast<const T*>(a.Q) + b * a.q_batch + (int64_t)g0 * a.q_head;
    for (int i = threadIdx.x; i < RG * a.s.d; i += kThreads) {
        const int g = i / a.s.d, c = i - g * a.s.d;
        q[i] = g < rows ? to_f32(src[g * a.q_head + c]) * a.qscale : 0.f;
    }
}

// One block of the coreset's share: rows [first, last) of unit (b, h)'s
// coreset against RG query rows.  W is fp32 with a row of dv + 1 values, so its
// rows are read in place, 4 bytes a lane; the row's last value is its weight
// in the normaliser.
template <typename T, int RG, int NT>
__device__ void coreset_block(const AttendArgs& a, int index, char* smem) {
    const View& s = a.s;
    const SimtSmem<NT, RG> L(s.d, s.dv, sizeof(T));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* q = reinterpret_cast<float*>(smem + L.q);
    float* p = reinterpret_cast<float*>(smem + L.p) + warp * NT * RG;
    float* merge = reinterpret_cast<float*>(smem + L.merge);
    char* krows = smem + warp * L.warp;
    const int split = index % a.csplits, unit = index / a.csplits;
    const int rt = unit % a.row_tiles, h = unit / a.row_tiles % s.hkv, b = unit / a.row_tiles / s.hkv;
    const int rows = min(a.rows, s.group - rt * a.rows);
    int n = a.rank ? __ldg(a.rank + b * s.hkv + h) : a.r;
    if (n < 0 || n > a.r) {
        record_status(a.status, WC_ERR_BOUNDS);
        n = n < 0 ? 0 : a.r;
    }
    const int first = split * a.csplit_len, last = min(first + a.csplit_len, n);
    load_queries<T, RG>(a, b, h * s.group + rt * a.rows, rows, q);
    __syncthreads();
    constexpr int kMaxCols = 8;   // dv <= 256: at most 8 columns a lane
    float m[RG], l[RG], o[RG][kMaxCols];
#pragma unroll
    for (int g = 0; g < RG; ++g) {
        m[g] = -CUDART_INF_F;
        l[g] = 0.f;
#pragma unroll
        for (int i = 0; i < kMaxCols; ++i) o[g][i] = 0.f;
    }
    const int64_t base = ((int64_t)b * s.hkv + h) * a.r;
    const int ck = s.d * (int)sizeof(T) / 16;
    for (int at = first + warp * NT; at < last; at += kWarps * NT) {
        __syncwarp();
        for (int i = lane; i < NT * ck; i += 32) {
            const int row = i / ck, c = i - row * ck;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (at + row < last)
                v = __ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(a.Ks) +
                                                         (base + at + row) * s.d * (int64_t)sizeof(T)) + c);
            *reinterpret_cast<uint4*>(krows + row * L.k_row + c * 16) = v;
        }
        __syncwarp();
        float x[RG];
        tile_logits<T, RG, NT>(krows, L.k_row, q, s.d, x);
        const int key = lane % NT;
#pragma unroll
        for (int g = 0; g < RG; ++g) {
            float v = at + key < last ? x[g] : -CUDART_INF_F, top = v;
#pragma unroll
            for (int e = 1; e < NT; e <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, e));
            if (top > m[g]) {
                const float f = ex2(m[g] - top);
                m[g] = top;
                l[g] *= f;
#pragma unroll
                for (int i = 0; i < kMaxCols; ++i) o[g][i] *= f;
            }
            const float w = ex2(v - (m[g] == -CUDART_INF_F ? 0.f : m[g]));
            if (lane < NT) p[key * RG + g] = w;
        }
        __syncwarp();
        const int live = min(NT, last - at);
        for (int j = 0; j < live; ++j) {
            const float* w = a.W + (base + at + j) * (s.dv + 1);
            float y[kMaxCols];
#pragma unroll
            for (int i = 0; i < kMaxCols; ++i) y[i] = lane + 32 * i < s.dv ? __ldg(w + lane + 32 * i) : 0.f;
            const float z = __ldg(w + s.dv);
#pragma unroll
            for (int g = 0; g < RG; ++g) {
                const float e = p[j * RG + g];
                l[g] = fmaf(e, z, l[g]);
#pragma unroll
                for (int i = 0; i < kMaxCols; ++i) o[g][i] = fmaf(e, y[i], o[g][i]);
            }
        }
    }
    const int ld = s.dv + 2;
#pragma unroll
    for (int g = 0; g < RG; ++g) {
        float* row = merge + (warp * RG + g) * ld;
#pragma unroll
        for (int i = 0; i < kMaxCols; ++i)
            if (lane + 32 * i < s.dv) row[lane + 32 * i] = o[g][i];
        if (lane == 0) {
            row[s.dv] = m[g];
            row[s.dv + 1] = l[g];
        }
    }
    __syncthreads();
    join_warps<RG>(a, merge, a.cparts + (int64_t)index * a.rows * c1_row(s.dv), 0, rows);
}

// The pages' share on CUDA cores, any type and width.  Each warp takes NT keys
// of every 4 NT-key tile through its own two stages of shared memory (filled
// by cp.async, so warps never wait for one another inside a unit); a lane
// holds one key's logits for the RG query rows, then four value columns.
template <typename T, int RG, int NT, int NVI>
__global__ void __launch_bounds__(kThreads) cache_attend_simt_kernel(const AttendArgs a) {
    extern __shared__ __align__(16) char smem[];
    __shared__ int64_t place_sh[4 + kWarps];
    const View& s = a.s;
    const int blocks = a.blocks;
    if ((int)blockIdx.x >= blocks) {
        coreset_block<T, RG, NT>(a, blockIdx.x - blocks, smem);
        return;
    }
    constexpr int kTile = kWarps * NT;
    const SimtSmem<NT, RG> L(s.d, s.dv, sizeof(T));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* q = reinterpret_cast<float*>(smem + L.q);
    float* p = reinterpret_cast<float*>(smem + L.p) + warp * NT * RG;
    float* merge = reinterpret_cast<float*>(smem + L.merge);
    char* stages = smem + warp * L.warp;
    const int per_tile = s.hkv * a.row_tiles;
    const int c = blockIdx.x;
    const Place at = find_place<kThreads>(s, a.lens, kTile, per_tile, c, blocks, -1, a.status, place_sh);
    if (c >= at.blocks) return;
    int64_t t = block_first(at.total, c, at.blocks);
    const int64_t t_last = block_first(at.total, c + 1, at.blocks);
    int b = at.b;
    int len = checked_len(a.lens, b, s.cap, a.status);
    int tiles = (len + kTile - 1) / kTile;
    int in_b = (int)((t - at.before) / tiles);          // unit within the sequence: h * row_tiles + rt
    int k0 = (int)((t - at.before) % tiles);
    const int ck = s.d * (int)sizeof(T) / 16, cv = s.dv * (int)sizeof(T) / 16;
    const int vchunks = s.dv / 4;
    const int groups = vchunks <= 8 ? 4 : vchunks <= 16 ? 2 : 1;   // key groups when few columns fill a warp
    const int cols = 32 / groups;
    while (t < t_last) {
        const int k1 = (int)min((int64_t)tiles, k0 + (t_last - t));
        const int h = in_b / a.row_tiles, rt = in_b % a.row_tiles;
        const int rows = min(a.rows, s.group - rt * a.rows), g0 = h * s.group + rt * a.rows;
        load_queries<T, RG>(a, b, g0, rows, q);
        __syncthreads();
        Running<RG, NVI> st;
        st.clear();
        const char* kh = a.kp + h * s.k_head;
        const char* vh = a.vp + h * s.v_head;
        // lane j < NT: where key j of tile i is
        auto locate = [&](int i) {
            KeyPlace w{0, 0, false};
            const int key = i * kTile + warp * NT + lane;
            if (lane < NT && i < k1 && key < len) {
                const int tp = key / s.page, slot = key - tp * s.page;
                const int pg = checked_page(s, a.s.table, b, tp, a.status);
                if (pg >= 0) {
                    w.k = pg * s.k_page + slot * s.k_token;
                    w.v = pg * s.v_page + slot * s.v_token;
                    w.valid = true;
                }
            }
            return w;
        };
        auto load = [&](int stage, const KeyPlace& w) {
            const uint32_t kd = (uint32_t)__cvta_generic_to_shared(stages + stage * L.stage);
            const uint32_t vd = kd + NT * L.k_row;
            for (int i = lane, n = (NT * ck + 31) / 32; n > 0; --n, i += 32) {
                const int row = i / ck, ch = i - row * ck;
                const int64_t off = __shfl_sync(0xffffffffu, w.k, row & (NT - 1));
                const bool ok = __shfl_sync(0xffffffffu, (int)w.valid, row & (NT - 1)) != 0;
                if (row < NT) cp_async16(kd + row * L.k_row + ch * 16, kh + off + ch * 16, ok);
            }
            for (int i = lane, n = (NT * cv + 31) / 32; n > 0; --n, i += 32) {
                const int row = i / cv, ch = i - row * cv;
                const int64_t off = __shfl_sync(0xffffffffu, w.v, row & (NT - 1));
                const bool ok = __shfl_sync(0xffffffffu, (int)w.valid, row & (NT - 1)) != 0;
                if (row < NT) cp_async16(vd + row * L.v_row + ch * 16, vh + off + ch * 16, ok);
            }
        };
        KeyPlace next = locate(k0);
        uint32_t mask = __ballot_sync(0xffffffffu, next.valid);
        load(0, next);
        cp_async_commit();
        for (int i = k0; i < k1; ++i) {
            const int stage = (i - k0) & 1;
            const uint32_t live = mask;
            next = locate(i + 1);
            mask = __ballot_sync(0xffffffffu, next.valid);
            if (i + 1 < k1) load(stage ^ 1, next);
            cp_async_commit();
            cp_async_wait<1>();
            __syncwarp();
            const char* krows = stages + stage * L.stage;
            const char* vrows = krows + NT * L.k_row;
            float x[RG];
            tile_logits<T, RG, NT>(krows, L.k_row, q, s.d, x);
            const int key = lane % NT;
            const bool ok = (live >> key) & 1;
#pragma unroll
            for (int g = 0; g < RG; ++g) x[g] = ok ? x[g] : -CUDART_INF_F;
            if (a.logits && lane < NT) {
                const int pos = i * kTile + warp * NT + key;
                if (pos < len)
                    for (int g = 0; g < rows; ++g)
                        a.logits[((int64_t)b * s.hq + g0 + g) * s.cap + pos] = x[g];
            }
            tile_weights<RG, NT, NVI>(st, x, p);
            __syncwarp();
            for (int j = lane / cols; j < NT; j += groups) {
                float w[RG];
#pragma unroll
                for (int g = 0; g < RG; ++g) w[g] = p[j * RG + g];
#pragma unroll
                for (int n = 0; n < NVI; ++n) {
                    const int ch = lane % cols + n * cols;
                    if (ch < vchunks) {
                        float y[4];
                        load_four(vrows + j * L.v_row, ch, y, T());
#pragma unroll
                        for (int g = 0; g < RG; ++g)
#pragma unroll
                            for (int e = 0; e < 4; ++e) st.o[g][n * 4 + e] = fmaf(w[g], y[e], st.o[g][n * 4 + e]);
                    }
                }
            }
            __syncwarp();
        }
        cp_async_wait<0>();
        leave_state<RG, NVI>(st, merge + warp * RG * (s.dv + 2), s.dv, groups);
        __syncthreads();
        const bool whole = k0 == 0 && k1 == tiles && !a.csplits && !a.logits;
        const int64_t unit = (int64_t)b * per_tile + in_b;
        join_warps<RG>(a, merge, whole ? nullptr : a.parts + (unit + c) * a.rows * c1_row(s.dv),
                       (int64_t)b * s.hq + g0, rows);
        __syncthreads();
        t += k1 - k0;
        k0 = 0;
        if (t < t_last && ++in_b == per_tile) {
            in_b = 0;
            do {
                len = checked_len(a.lens, ++b, s.cap, a.status);
            } while (len == 0);
            tiles = (len + kTile - 1) / kTile;
        }
    }
}

// Joins the partial rows of every query row, and adds the step's weights to
// the scores.  Blocks [0, B hq) take a query row each; with scores, the others
// take kScoreKeys positions of one (sequence, kv head) each.
constexpr int kJoinThreads = 128;
constexpr int kScoreKeys = 1024;

struct Parts {
    const float* p; int n; int64_t step;   // sets of the pages' share, one per block
    const float* c; int nc; int64_t cstep; // sets of the coreset's share
};

__global__ void __launch_bounds__(kJoinThreads) cache_join_kernel(const AttendArgs a, int tile) {
    __shared__ int64_t place_sh[4 + kJoinThreads / 32];
    __shared__ float red[kJoinThreads / 32][2];
    const View& s = a.s;
    const int per_tile = s.hkv * a.row_tiles, dv = s.dv, ld = c1_row(dv);
    const bool score = (int)blockIdx.x >= s.B * s.hq;
    const int chunks = (s.cap + kScoreKeys - 1) / kScoreKeys;
    int b, hq0, n_rows, key0 = 0;
    if (!score) {
        b = blockIdx.x / s.hq;
        hq0 = blockIdx.x % s.hq;
        n_rows = 1;
    } else {
        const int i = blockIdx.x - s.B * s.hq;
        b = i / chunks / s.hkv;
        hq0 = i / chunks % s.hkv * s.group;
        key0 = i % chunks * kScoreKeys;
        n_rows = s.group;
    }
    const int len = checked_len(a.lens, b, s.cap, a.status);
    if (score && key0 >= len) return;
    const Place at = find_place<kJoinThreads>(s, a.lens, tile, per_tile, 0, a.blocks, b, a.status, place_sh);
    const int tiles = (len + tile - 1) / tile;
    float acc[kScoreKeys / kJoinThreads];
#pragma unroll
    for (int i = 0; i < kScoreKeys / kJoinThreads; ++i) acc[i] = 0.f;
    for (int r = 0; r < n_rows; ++r) {
        const int g = (hq0 + r) % s.group, in_b = (hq0 + r) / s.group * a.row_tiles + g / a.rows;
        const int in_unit = g % a.rows;
        Parts ps{nullptr, 0, (int64_t)a.rows * ld, nullptr, 0, (int64_t)a.rows * ld};
        if (tiles > 0) {
            const int64_t t0 = at.before + (int64_t)in_b * tiles;
            const int c0 = block_of(t0, at.total, at.blocks), c1 = block_of(t0 + tiles - 1, at.total, at.blocks);
            if (c0 == c1 && !a.csplits && !a.logits) return;   // finished by the block itself
            ps.p = a.parts + ((int64_t)b * per_tile + in_b + c0) * ps.step + in_unit * ld;
            ps.n = c1 - c0 + 1;
        }
        if (a.csplits) {
            ps.c = a.cparts + ((int64_t)b * per_tile + in_b) * a.csplits * ps.cstep + in_unit * ld;
            ps.nc = a.csplits;
        }
        const int n = ps.n + ps.nc;
        auto set = [&](int i) { return i < ps.n ? ps.p + i * ps.step : ps.c + (i - ps.n) * ps.cstep; };
        // the maximum and the normaliser over all sets (fixed order: by set within a thread, then by thread)
        float m = -CUDART_INF_F;
        for (int i = threadIdx.x; i < n; i += kJoinThreads) m = fmaxf(m, set(i)[dv + 1]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5][0] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kJoinThreads / 32; ++w) m = fmaxf(m, red[w][0]);
        const float ref = m == -CUDART_INF_F ? 0.f : m;
        float l = 0.f;
        for (int i = threadIdx.x; i < n; i += kJoinThreads) l += ex2(set(i)[dv + 1] - ref) * set(i)[dv];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5][1] = l;
        __syncthreads();
        l = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinThreads / 32; ++w) l += red[w][1];
        __syncthreads();
        const bool empty = nothing(m, l);
        if (!score) {
            const int64_t row = (int64_t)b * s.hq + hq0;
            for (int c = threadIdx.x; c < dv; c += kJoinThreads) {
                float o = 0.f;
                for (int i = 0; i < n; ++i) o = fmaf(ex2(set(i)[dv + 1] - ref), set(i)[c], o);
                a.out[row * dv + c] = empty ? 0.f : o / l;
            }
            if (threadIdx.x == 0 && a.lse)
                a.lse[row] = log_sum(m, l);
        } else if (!empty) {
            const float* x = a.logits + ((int64_t)b * s.hq + hq0 + r) * s.cap;
            const float inv = 1.f / l;
#pragma unroll
            for (int i = 0; i < kScoreKeys / kJoinThreads; ++i) {
                const int key = key0 + i * kJoinThreads + threadIdx.x;
                if (key < len) acc[i] = fmaf(ex2(x[key] - ref), inv, acc[i]);
            }
        }
    }
    if (score) {
        float* out = a.scores + ((int64_t)b * s.hkv + hq0 / s.group) * s.cap;
#pragma unroll
        for (int i = 0; i < kScoreKeys / kJoinThreads; ++i) {
            const int key = key0 + i * kJoinThreads + threadIdx.x;
            if (key < len) out[key] += acc[i];
        }
    }
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return n;
}

template <typename T, int RG, int NT, int NVI>
wc_status run_simt(AttendArgs a, cudaStream_t st) {
    auto kern = cache_attend_simt_kernel<T, RG, NT, NVI>;
    const SimtSmem<NT, RG> L(a.s.d, a.s.dv, sizeof(T));
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L.total) != cudaSuccess)
        return WC_ERR_CUDA;
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kThreads, L.total) != cudaSuccess)
        return WC_ERR_CUDA;
    const int nsm = sm_count();
    if (nsm < 1 || per_sm < 1) return WC_ERR_CUDA;
    constexpr int tile = kWarps * NT;
    const int64_t most = (int64_t)a.s.B * a.s.hkv * a.row_tiles * ((a.s.cap + tile - 1) / tile);
    a.blocks = (int)min(most, (int64_t)min(nsm * per_sm, kMaxBlocks));
    const int64_t grid = a.blocks + (int64_t)a.csplits * a.s.B * a.s.hkv * a.row_tiles;
    if (grid > INT32_MAX) return WC_ERR_UNSUPPORTED;
    kern<<<(unsigned)grid, kThreads, L.total, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return WC_ERR_CUDA;
    const int64_t chunks = (a.s.cap + kScoreKeys - 1) / kScoreKeys;
    const int64_t join = (int64_t)a.s.B * a.s.hq + (a.scores ? chunks * a.s.B * a.s.hkv : 0);
    if (join > INT32_MAX) return WC_ERR_UNSUPPORTED;
    cache_join_kernel<<<(unsigned)join, kJoinThreads, 0, st>>>(a, tile);
    return cudaGetLastError() == cudaSuccess ? WC_OK : WC_ERR_CUDA;
}

template <typename T, int RG, int NT>
wc_status by_width(const AttendArgs& a, cudaStream_t st) {
    return a.s.dv <= 128 ? run_simt<T, RG, NT, 1>(a, st) : run_simt<T, RG, NT, 2>(a, st);
}

template <typename T, int RG>
wc_status by_keys(const AttendArgs& a, cudaStream_t st) {
    // 16 keys a warp while two stages of them fit shared memory beside the rest (rows of up to 1024 bytes)
    return (a.s.d + a.s.dv) * (int)sizeof(T) <= 1024 ? by_width<T, RG, 16>(a, st) : by_width<T, RG, 8>(a, st);
}

template <typename T>
wc_status by_rows(const AttendArgs& a, cudaStream_t st) {
    switch (a.rows) {
        case 1: return by_keys<T, 1>(a, st);
        case 2: return by_keys<T, 2>(a, st);
        case 4: return by_keys<T, 4>(a, st);
        default: return by_keys<T, 8>(a, st);
    }
}

}  // namespace

wc_status launch_attend(const AttendArgs& a, cudaStream_t st) {
    return a.s.dtype == WC_BF16 ? by_rows<__nv_bfloat16>(a, st) : by_rows<float>(a, st);
}

}  // namespace cache
}  // namespace wc
