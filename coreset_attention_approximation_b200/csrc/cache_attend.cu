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
#include <atomic>
#include <mutex>

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

// Shared memory of one coreset block, in bytes: two stages a warp of NT keys
// and their rows of W (as they lie in memory, dv + 1 values each).  The warps'
// sums go where the stages were.
template <int NT, int RG>
struct CoresetSmem {
    int k_row, w_row, w, stage, q, p, total;
    __host__ __device__ CoresetSmem(int d, int dv, int esize) {
        k_row = d * esize;
        if ((k_row / 16) % 2 == 0) k_row += 16;
        w_row = (dv + 1) * 4;
        w = NT * k_row;
        stage = (w + NT * w_row + 15) / 16 * 16;
        const int stages = kWarps * 2 * stage, merge = kWarps * RG * (dv + 2) * 4;
        q = ((stages > merge ? stages : merge) + 15) / 16 * 16;
        p = q + RG * d * 4;
        total = p + kWarps * NT * RG * 4;
    }
};

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// One block of the coreset's share: rows [first, last) of unit (b, h)'s
// coreset against RG query rows, NT at a time for each warp.  W is fp32 with
// rows of dv + 1 values (no 16-byte alignment), so a step's rows, which lie
// side by side, come in by 4-byte asynchronous copies while the step before is
// summed; a lane holds columns lane, lane + 32, ... and the row's last value is
// its weight in the normaliser.  Sums in fp32 on CUDA cores: W's values cancel
// one another, and there are few rows.
template <typename T, int RG, int NT, int COLS>
__device__ void coreset_block(const AttendArgs& a, int index, char* smem) {
    const View& s = a.s;
    const CoresetSmem<NT, RG> L(s.d, s.dv, sizeof(T));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* q = reinterpret_cast<float*>(smem + L.q);
    float* p = reinterpret_cast<float*>(smem + L.p) + warp * NT * RG;
    char* stages = smem + warp * 2 * L.stage;
    const int split = index % a.csplits, unit = index / a.csplits;
    const int rt = unit % a.row_tiles, h = unit / a.row_tiles % s.hkv, b = unit / a.row_tiles / s.hkv;
    const int rows = min(a.rows, s.group - rt * a.rows);
    int n = a.rank ? __ldg(a.rank + b * s.hkv + h) : a.r;
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
            int row = lane / ck, c = lane - row * ck;
            for (int i = lane; i < NT * ck; i += 32) {
                cp_async16(kd + row * L.k_row + c * 16, k + (row < live ? i : 0) * 16, row < live);
                for (c += 32; c >= ck; c -= ck) ++row;
            }
            const float* w = a.W + (base + at) * (s.dv + 1);
            for (int i = lane; i < live * (s.dv + 1); i += 32) cp_async4(wd + i * 4, w + i);
        }
        cp_async_commit();
    };
    int at = first + warp * NT;
    load(0, at);
    load_queries<T, RG>(a, b, h * s.group + rt * a.rows, rows, q);
    __syncthreads();
    float m[RG], l[RG], o[RG][COLS];
#pragma unroll
    for (int g = 0; g < RG; ++g) {
        m[g] = -CUDART_INF_F;
        l[g] = 0.f;
#pragma unroll
        for (int i = 0; i < COLS; ++i) o[g][i] = 0.f;
    }
    for (int stage = 0; at < last; at += kWarps * NT, stage ^= 1) {
        load(stage ^ 1, at + kWarps * NT);
        cp_async_wait<1>();
        __syncwarp();
        const char* krows = stages + stage * L.stage;
        const float* wrows = reinterpret_cast<const float*>(krows + L.w);
        float x[RG];
        tile_logits<T, RG, NT>(krows, L.k_row, q, s.d, x);
        const int key = lane % NT, live = min(NT, last - at);
#pragma unroll
        for (int g = 0; g < RG; ++g) {
            const float v = key < live ? x[g] : -CUDART_INF_F;
            float top = v;
#pragma unroll
            for (int e = 1; e < NT; e <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, e));
            if (top > m[g]) {
                const float f = ex2(m[g] - top);
                m[g] = top;
                l[g] *= f;
#pragma unroll
                for (int i = 0; i < COLS; ++i) o[g][i] *= f;
            }
            const float w = ex2(v - (m[g] == -CUDART_INF_F ? 0.f : m[g]));
            if (lane < NT) p[key * RG + g] = w;
        }
        __syncwarp();
#pragma unroll 2
        for (int j = 0; j < live; ++j) {
            const float* w = wrows + j * (s.dv + 1);
            float y[COLS], e[RG];
#pragma unroll
            for (int i = 0; i < COLS; ++i) y[i] = lane + 32 * i < s.dv ? w[lane + 32 * i] : 0.f;
            const float z = w[s.dv];
#pragma unroll
            for (int g = 0; g < RG; ++g) e[g] = p[j * RG + g];
#pragma unroll
            for (int g = 0; g < RG; ++g) {
                l[g] = fmaf(e[g], z, l[g]);
#pragma unroll
                for (int i = 0; i < COLS; ++i) o[g][i] = fmaf(e[g], y[i], o[g][i]);
            }
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
        for (int i = 0; i < COLS; ++i)
            if (lane + 32 * i < s.dv) row[lane + 32 * i] = o[g][i];
        if (lane == 0) {
            row[s.dv] = m[g];
            row[s.dv + 1] = l[g];
        }
    }
    __syncthreads();
    join_warps<RG>(a, merge, a.cparts + (int64_t)index * a.rows * c1_row(s.dv), 0, rows);
}

// fp32 pages, on CUDA cores (their products keep 24 bits).  Each warp takes NT keys
// of every 4 NT-key tile through its own two stages of shared memory (filled
// by cp.async, so warps never wait for one another inside a unit); a lane
// holds one key's logits for the RG query rows, then four value columns.
template <int RG, int NT, int NVI>
__global__ void __launch_bounds__(kThreads) cache_attend_simt_kernel(const AttendArgs a) {
    using T = float;
    extern __shared__ __align__(128) char smem[];
    __shared__ int64_t place_sh[4 + kWarps];
    grid_dependents_launch();
    const View& s = a.s;
    const int blocks = a.blocks;
    if ((int)blockIdx.x >= blocks) {
        coreset_block<T, RG, NT, NVI * 4>(a, blockIdx.x - blocks, smem);
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
                const int pg = checked_page(s, s.table, b, tp, a.status);
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
                        load_chunk<float>(vrows + j * L.v_row + ch * 16, y);
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
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%10,%10,%10,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// c += a b.
__device__ __forceinline__ void mma16816(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// The three bf16 terms of a pair of weights, x = t0 + t1 + t2 up to 2^-24 x:
// one term alone (half a step, 2^-9 relative) would be the largest error of the
// whole attention, whose output is fp32.
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t t[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        t[i] = pack_bf16(x, y);
        x -= __uint_as_float(t[i] << 16);
        y -= __uint_as_float(t[i] & 0xffff0000u);
    }
}

// (x, y) += (u, v) as one packed fp32 addition.
__device__ __forceinline__ void add2(float& x, float& y, float u, float v) {
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tadd.rn.f32x2 a, a, b;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(u), "f"(v));
}

constexpr int kMmaKeys = 16;     // keys of one warp's step
constexpr int kMmaStages = 3;
template <int DP> constexpr int kCoresetKeys = DP > 128 ? 8 : 16;   // (two stages of wider rows leave too little room)

// bf16 pages on tensor cores (mma.sync: a group's 1 to 16 query rows fill one
// 16-row tile at most, and the pass is bound by the bytes of the keys and
// values, so the wider tcgen05 tiles would only hold more padding).  A warp
// takes 16 keys of every 64-key tile through its own ring of three stages;
// 128-byte groups of a row are XOR-swizzled by the row so that ldmatrix reads
// without bank conflicts.  DP: d and dv rounded up to 64, 128 or 256 (columns
// past the width are zeros).
// SETS: how the weights' three terms meet the 16 rows of the value product.
//   1  up to 4 query rows, each four times in the tile (r, r + 4, r + 8, r + 12):
//      the copies carry the terms, so one product adds all three
//   2  up to 8 rows, each twice: two products
//   3  up to 16 rows: three products
template <int DP, int SETS>
__global__ void __launch_bounds__(kThreads) cache_attend_mma_kernel(const AttendArgs a) {
    using bf16 = __nv_bfloat16;
    constexpr int kRows = SETS == 1 ? 4 : SETS == 2 ? 8 : 16;
    constexpr int kChunks = DP / 8;                        // 16-byte pieces of a row
    constexpr int kRowBytes = DP * 2;
    constexpr int kStage = 2 * kMmaKeys * kRowBytes;       // keys, then values
    constexpr int kTile = kWarps * kMmaKeys;
    constexpr int kPerLoad = 32 / kChunks > 0 ? 32 / kChunks : 1;   // rows of one warp-wide load
    constexpr int kLoads = kMmaKeys * kChunks / 32;
    extern __shared__ __align__(128) char smem[];
    __shared__ int64_t place_sh[4 + kWarps];
    grid_dependents_launch();
    const View& s = a.s;
    const int blocks = a.blocks;
    if ((int)blockIdx.x >= blocks) {
        coreset_block<bf16, kRows, kCoresetKeys<DP>, DP / 32>(a, blockIdx.x - blocks, smem);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = lane >> 2, pair = lane & 3;           // fragment row and column pair
    char* stages = smem + warp * kMmaStages * kStage;
    const uint32_t stages_u = (uint32_t)__cvta_generic_to_shared(stages);
    const int per_tile = s.hkv * a.row_tiles;
    const int c = blockIdx.x;
    const Place at = find_place<kThreads>(s, a.lens, kTile, per_tile, c, blocks, -1, a.status, place_sh);
    if (c >= at.blocks) return;
    int64_t t = block_first(at.total, c, at.blocks);
    const int64_t t_last = block_first(at.total, c + 1, at.blocks);
    int b = at.b;
    int len = checked_len(a.lens, b, s.cap, a.status);
    int tiles = (len + kTile - 1) / kTile;
    int in_b = (int)((t - at.before) / tiles);
    int k0 = (int)((t - at.before) % tiles);
    const int ck = s.d / 8, cv = s.dv / 8;
    const bool whole_pages = s.page % kMmaKeys == 0;       // 16 keys of a step then share a page
    while (t < t_last) {
        const int k1 = (int)min((int64_t)tiles, k0 + (t_last - t));
        const int h = in_b / a.row_tiles, rt = in_b % a.row_tiles;
        const int rows = min(a.rows, s.group - rt * a.rows), g0 = h * s.group + rt * a.rows;
        const char* kh = a.kp + h * s.k_head;
        const char* vh = a.vp + h * s.v_head;
        float o[DP / 8][4];
#pragma unroll
        for (int n = 0; n < DP / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
        constexpr int kMine = SETS == 3 ? 2 : 1;           // rows of this lane
        float m[kMine], l[kMine];
#pragma unroll
        for (int i = 0; i < kMine; ++i) m[i] = -CUDART_INF_F, l[i] = 0.f;

        // lane j < 16: where key j of tile i is, and how many keys there are
        auto locate = [&](int i) {
            KeyPlace w{0, 0, false};
            const int key = i * kTile + warp * kMmaKeys + (whole_pages ? 0 : lane & 15);
            if (i < k1 && key < len) {
                const int tp = key / s.page, slot = key - tp * s.page;
                const int pg = checked_page(s, s.table, b, tp, a.status);
                if (pg >= 0) {
                    w.k = pg * s.k_page + slot * s.k_token;
                    w.v = pg * s.v_page + slot * s.v_token;
                    w.valid = true;
                }
            }
            return w;
        };
        auto live_keys = [&](int i, const KeyPlace& w) {
            const int n = len - (i * kTile + warp * kMmaKeys);
            if (i >= k1 || n <= 0) return 0u;
            if (!whole_pages) return __ballot_sync(0xffffffffu, w.valid) & 0xffffu;
            return w.valid ? (n >= kMmaKeys ? 0xffffu : (1u << n) - 1) : 0u;
        };
        auto load = [&](int stage, const KeyPlace& w, uint32_t live) {
            const uint32_t kd = stages_u + stage * kStage, vd = kd + kMmaKeys * kRowBytes;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int row = kChunks >= 32 ? i * 32 / kChunks : i * kPerLoad + lane / kChunks;
                const int ch = lane % kChunks;
                int64_t ko = w.k, vo = w.v;
                if (whole_pages) {
                    ko += row * s.k_token;
                    vo += row * s.v_token;
                } else {
                    ko = __shfl_sync(0xffffffffu, w.k, row);
                    vo = __shfl_sync(0xffffffffu, w.v, row);
                }
                const bool ok = (live >> row) & 1;
                const uint32_t to = row * kRowBytes + (ch ^ (row & 7)) * 16;
                const bool kok = ok && ch < ck, vok = ok && ch < cv;
                cp_async16(kd + to, kok ? kh + ko + ch * 16 : a.kp, kok);
                cp_async16(vd + to, vok ? vh + vo + ch * 16 : a.vp, vok);
            }
        };
        uint32_t live[kMmaStages];
        KeyPlace next;
#pragma unroll
        for (int p = 0; p < kMmaStages - 1; ++p) {
            next = locate(k0 + p);
            live[p] = live_keys(k0 + p, next);
            if (k0 + p < k1) load(p, next, live[p]);
            cp_async_commit();
        }
        next = locate(k0 + kMmaStages - 1);
        // Query fragments, as they are (the logits are scaled in fp32): rows
        // quad and, where the rows are not copies, quad + 8.
        uint32_t q[DP / 16][SETS == 3 ? 4 : 2];
        {
            const bf16* src = static_cast<const bf16*>(a.Q) + b * a.q_batch + (int64_t)g0 * a.q_head;
            auto two = [&](int row, int col) {
                uint32_t v = 0;
                if (row < rows && col < s.d) {
                    const bf16* p = src + row * a.q_head + col;
                    if (a.q_pairs) v = *reinterpret_cast<const uint32_t*>(p);
                    else v = (uint32_t)__bfloat16_as_ushort(p[0]) | (uint32_t)__bfloat16_as_ushort(p[1]) << 16;
                }
                return v;
            };
            const int r0 = quad % kRows;
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) {
                const int col = k * 16 + pair * 2;
                if (SETS == 3) {
                    q[k][0] = two(quad, col); q[k][1] = two(quad + 8, col);
                    q[k][SETS == 3 ? 2 : 0] = two(quad, col + 8); q[k][SETS == 3 ? 3 : 1] = two(quad + 8, col + 8);
                } else {
                    q[k][0] = two(r0, col);
                    q[k][1] = two(r0, col + 8);
                }
            }
        }
        int stage = 0;
        for (int i = k0; i < k1; ++i) {
            cp_async_wait<kMmaStages - 2>();
            __syncwarp();
            const uint32_t kd = stages_u + stage * kStage, vd = kd + kMmaKeys * kRowBytes;
            const uint32_t mask = live[0];
            {   // the stage read in the last step is free: load three tiles ahead
                const int ahead = i + kMmaStages - 1, to = stage == 0 ? kMmaStages - 1 : stage - 1;
                const uint32_t lv = live_keys(ahead, next);
                if (ahead < k1) load(to, next, lv);
                cp_async_commit();
                next = locate(ahead + 1);
#pragma unroll
                for (int p = 0; p < kMmaStages - 2; ++p) live[p] = live[p + 1];
                live[kMmaStages - 2] = lv;
            }
            // logits: keys 0..7 in x[0], 8..15 in x[1]
            float x[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
            {
                const int row = (lane & 7) + ((lane >> 4) << 3);
                const uint32_t base = kd + row * kRowBytes;
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    uint32_t f[4];
                    ldmatrix4(f, base + (((2 * k + ((lane >> 3) & 1)) ^ (row & 7)) << 4));
                    if (SETS == 3) {
                        mma16816(x[0], q[k][0], q[k][1], q[k][SETS == 3 ? 2 : 0], q[k][SETS == 3 ? 3 : 1], f[0], f[1]);
                        mma16816(x[1], q[k][0], q[k][1], q[k][SETS == 3 ? 2 : 0], q[k][SETS == 3 ? 3 : 1], f[2], f[3]);
                    } else {
                        mma16816(x[0], q[k][0], q[k][0], q[k][1], q[k][1], f[0], f[1]);
                        mma16816(x[1], q[k][0], q[k][0], q[k][1], q[k][1], f[2], f[3]);
                    }
                }
            }
            uint32_t w[kMine][2][3];                       // weights' terms: [row][key octet][term]
#pragma unroll
            for (int r = 0; r < kMine; ++r) {
                float y[4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        y[2 * n + e] = (mask >> (n * 8 + pair * 2 + e)) & 1 ? x[n][2 * r + e] * a.qscale
                                                                            : -CUDART_INF_F;
                if (a.logits) {
                    const int g = quad + 8 * r;
                    if (g < rows) {
                        const int pos = i * kTile + warp * kMmaKeys;
                        float* to = a.logits + ((int64_t)b * s.hq + g0 + g) * s.cap + pos;
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int key = n * 8 + pair * 2 + e;
                                if (pos + key < len) to[key] = y[2 * n + e];
                            }
                    }
                }
                float top = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // The reference follows the maximum only when it has grown by more than 2^8, which
                // spares most steps the rescaling; weights up to 2^8 lose nothing in fp32.
                const bool grow = top > m[r] + 8.f;
                if (__any_sync(0xffffffffu, grow)) {
                    const float f = grow ? ex2(m[r] - top) : 1.f;
                    if (grow) m[r] = top;
                    l[r] *= f;
                    if (SETS == 3) {
#pragma unroll
                        for (int n = 0; n < DP / 8; ++n) o[n][2 * r] *= f, o[n][2 * r + 1] *= f;
                    } else {
#pragma unroll
                        for (int n = 0; n < DP / 8; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[n][e] *= f;
                    }
                }
                const float ref = m[r] == -CUDART_INF_F ? 0.f : m[r];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = ex2(y[e] - ref);
                l[r] += (y[0] + y[1]) + (y[2] + y[3]);
                split_bf16(y[0], y[1], w[r][0]);
                split_bf16(y[2], y[3], w[r][1]);
            }
            // values
            {
                const int row = lane & 15;
                const uint32_t base = vd + row * kRowBytes;
                uint32_t p0 = 0, p1 = 0, p2 = 0, p3 = 0;
                if (SETS == 1) {   // rows 0-3: term 0, 8-11: term 1, 4-7: term 2, 12-15: nothing
                    const bool up = quad < 4;
                    p0 = up ? w[0][0][0] : w[0][0][2]; p1 = up ? w[0][0][1] : 0u;
                    p2 = up ? w[0][1][0] : w[0][1][2]; p3 = up ? w[0][1][1] : 0u;
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
                        // (4.3e-6 of the output at 131072 keys, 0.9e-6 so).
                        float z[4];
                        const uint32_t b0 = f[2 * u], b1 = f[2 * u + 1];
                        if (SETS == 1) {
                            mma16816_new(z, p0, p1, p2, p3, b0, b1);
                        } else if (SETS == 2) {
                            mma16816_new(z, w[0][0][0], w[0][0][1], w[0][1][0], w[0][1][1], b0, b1);
                            mma16816(z, w[0][0][2], 0u, w[0][1][2], 0u, b0, b1);
                        } else {
                            mma16816_new(z, w[0][0][0], w[kMine - 1][0][0], w[0][1][0], w[kMine - 1][1][0], b0, b1);
                            mma16816(z, w[0][0][1], w[kMine - 1][0][1], w[0][1][1], w[kMine - 1][1][1], b0, b1);
                            mma16816(z, w[0][0][2], w[kMine - 1][0][2], w[0][1][2], w[kMine - 1][1][2], b0, b1);
                        }
                        add2(o[2 * n + u][0], o[2 * n + u][1], z[0], z[1]);
                        add2(o[2 * n + u][2], o[2 * n + u][3], z[2], z[3]);
                    }
                }
            }
            stage = stage + 1 == kMmaStages ? 0 : stage + 1;
            __syncwarp();
        }
        cp_async_wait<0>();
        __syncthreads();
        // the warps' sums into the stages, which are idle now: [warp][kRows][dv + 2]
        float* merge = reinterpret_cast<float*>(smem);
        const int ld = s.dv + 2;
#pragma unroll
        for (int r = 0; r < kMine; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            const int g = quad + 8 * r;
            float* row = merge + (warp * kRows + (g < kRows ? g : 0)) * ld;
#pragma unroll
            for (int n = 0; n < DP / 8; ++n) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = o[n][2 * r + e];
                    if (SETS != 3) v += o[n][2 + e];
                    if (SETS == 1) v += __shfl_xor_sync(0xffffffffu, v, 16);
                    const int col = n * 8 + pair * 2 + e;
                    if (g < kRows && col < s.dv) row[col] = v;
                }
            }
            if (g < kRows && pair == 0) {
                row[s.dv] = m[r];
                row[s.dv + 1] = l[r];
            }
        }
        __syncthreads();
        const bool whole = k0 == 0 && k1 == tiles && !a.csplits && !a.logits;
        const int64_t unit = (int64_t)b * per_tile + in_b;
        join_warps<kRows>(a, merge, whole ? nullptr : a.parts + (unit + c) * a.rows * c1_row(s.dv),
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
// the scores.  Blocks [0, B hq) take a query row each: a warp takes every
// fourth set, a lane four columns.  With scores, the others take kScoreKeys
// positions of one (sequence, kv head) each: the rows' references and
// normalisers first (a warp a row), then the logits that the pages' kernel
// left, 2^(x - m) / L summed over the group's rows.
constexpr int kJoinThreads = 128;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kScoreKeys = 1024;
constexpr int kScoreRows = 64;    // rows whose references are held at a time

__global__ void __launch_bounds__(kJoinThreads) cache_join_kernel(const AttendArgs a, int tile) {
    __shared__ int64_t place_sh[4 + kJoinWarps];
    __shared__ float sums[kJoinWarps][256];
    __shared__ float refs[kScoreRows][2];
    const View& s = a.s;
    const int per_tile = s.hkv * a.row_tiles, dv = s.dv, ld = c1_row(dv);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool score = (int)blockIdx.x >= s.B * s.hq;
    const int chunks = (s.cap + kScoreKeys - 1) / kScoreKeys;
    int b, hq0, key0 = 0;
    if (!score) {
        b = blockIdx.x / s.hq;
        hq0 = blockIdx.x % s.hq;
    } else {
        const int i = blockIdx.x - s.B * s.hq;
        b = i / chunks / s.hkv;
        hq0 = i / chunks % s.hkv * s.group;
        key0 = i % chunks * kScoreKeys;
    }
    const int len = checked_len(a.lens, b, s.cap, a.status);
    if (score && key0 >= len) return;
    grid_dependency_wait();   // the partial rows (and everything before them) are there from here on
    const Place at = find_place<kJoinThreads>(s, a.lens, tile, per_tile, 0, a.blocks, b, a.status, place_sh);
    const int tiles = (len + tile - 1) / tile;
    // sets of partial rows of query row hq: first of the pages' (one per block), then of the coreset's
    const float *pages = nullptr, *core = nullptr;
    int n_pages = 0, n = 0;
    const int64_t step = (int64_t)a.rows * ld;
    auto find_sets = [&](int hq) {
        const int g = hq % s.group, in_b = hq / s.group * a.row_tiles + g / a.rows, in_unit = g % a.rows;
        n_pages = 0;
        if (tiles > 0) {
            const int64_t t0 = at.before + (int64_t)in_b * tiles;
            const int c0 = block_of(t0, at.total, at.blocks), c1 = block_of(t0 + tiles - 1, at.total, at.blocks);
            if (c0 == c1 && !a.csplits && !a.logits) return false;   // finished by the block itself
            pages = a.parts + ((int64_t)b * per_tile + in_b + c0) * step + in_unit * ld;
            n_pages = c1 - c0 + 1;
        }
        if (a.csplits) core = a.cparts + ((int64_t)b * per_tile + in_b) * a.csplits * step + in_unit * ld;
        n = n_pages + a.csplits;
        return true;
    };
    auto set = [&](int i) { return i < n_pages ? pages + i * step : core + (i - n_pages) * step; };
    // a warp's reference and normaliser over all sets, in an order that the number of sets alone decides
    auto total = [&](float& m, float& l) {
        m = -CUDART_INF_F;
        for (int i = lane; i < n; i += 32) m = fmaxf(m, set(i)[dv + 1]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float ref = m == -CUDART_INF_F ? 0.f : m;
        l = 0.f;
        for (int i = lane; i < n; i += 32) l = fmaf(ex2(set(i)[dv + 1] - ref), set(i)[dv], l);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    };
    if (!score) {
        if (!find_sets(hq0)) return;
        float m, l;
        total(m, l);
        const float ref = m == -CUDART_INF_F ? 0.f : m;
        float o[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[k][e] = 0.f;
#pragma unroll 4
        for (int i = warp; i < n; i += kJoinWarps) {
            const float* p = set(i);
            const float f = ex2(p[dv + 1] - ref);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (k * 128 + lane * 4 < dv) {
                    const float4 v = *reinterpret_cast<const float4*>(p + k * 128 + lane * 4);
                    o[k][0] = fmaf(f, v.x, o[k][0]);
                    o[k][1] = fmaf(f, v.y, o[k][1]);
                    o[k][2] = fmaf(f, v.z, o[k][2]);
                    o[k][3] = fmaf(f, v.w, o[k][3]);
                }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (k * 128 + lane * 4 < dv)
                *reinterpret_cast<float4*>(&sums[warp][k * 128 + lane * 4]) = make_float4(o[k][0], o[k][1], o[k][2], o[k][3]);
        __syncthreads();
        const int64_t row = (int64_t)b * s.hq + hq0;
        const bool empty = nothing(m, l);
        for (int c = threadIdx.x; c < dv; c += kJoinThreads) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kJoinWarps; ++w) v += sums[w][c];
            a.out[row * dv + c] = empty ? 0.f : v / l;
        }
        if (threadIdx.x == 0 && a.lse) a.lse[row] = log_sum(m, l);
        return;
    }
    float acc[kScoreKeys / kJoinThreads];
#pragma unroll
    for (int i = 0; i < kScoreKeys / kJoinThreads; ++i) acc[i] = 0.f;
    for (int r0 = 0; r0 < s.group; r0 += kScoreRows) {
        const int rows = min(kScoreRows, s.group - r0);
        __syncthreads();
        for (int r = warp; r < rows; r += kJoinWarps) {
            find_sets(hq0 + r0 + r);
            float m, l;
            total(m, l);
            if (lane == 0) {
                refs[r][0] = m == -CUDART_INF_F ? 0.f : m;
                refs[r][1] = nothing(m, l) ? 0.f : 1.f / l;   // no weight anywhere: 0 for every key
            }
        }
        __syncthreads();
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

// Blocks of a kernel that the current device holds at once with `smem` bytes
// each.  The answer (and the kernel's shared-memory limit, set before it is
// asked for) is kept per kernel, device and size: the calls cost more than a
// short attention's kernels do.
wc_status resident_blocks(const void* kern, int smem, int* out) {
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
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kThreads, smem) != cudaSuccess || per_sm < 1)
        return WC_ERR_CUDA;
    *out = nsm * per_sm;
    if (n < kEntries) {
        table[n] = Entry{kern, dev, smem, *out};
        used.store(n + 1, std::memory_order_release);
    }
    return WC_OK;
}

// Launches one of the page kernels (its grid: as many blocks as the GPU holds
// at once, or one per tile where there are fewer) and the join.
wc_status run(AttendArgs a, void (*kern)(const AttendArgs), int smem, int tile, cudaStream_t st) {
    int room = 0;
    if (resident_blocks(reinterpret_cast<const void*>(kern), smem, &room) != WC_OK) return WC_ERR_CUDA;
    const int64_t most = (int64_t)a.s.B * a.s.hkv * a.row_tiles * ((a.s.cap + tile - 1) / tile);
    a.blocks = (int)min(most, (int64_t)min(room, kMaxBlocks));
    const int64_t grid = a.blocks + (int64_t)a.csplits * a.s.B * a.s.hkv * a.row_tiles;
    if (grid > INT32_MAX) return WC_ERR_UNSUPPORTED;
    kern<<<(unsigned)grid, kThreads, smem, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return WC_ERR_CUDA;
    const int64_t chunks = (a.s.cap + kScoreKeys - 1) / kScoreKeys;
    const int64_t join = (int64_t)a.s.B * a.s.hq + (a.scores ? chunks * a.s.B * a.s.hkv : 0);
    if (join > INT32_MAX) return WC_ERR_UNSUPPORTED;
    // the join's blocks may start while the last page blocks run; they wait before they read partial rows
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)join);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cache_join_kernel, a, tile) == cudaSuccess ? WC_OK : WC_ERR_CUDA;
}

template <int RG, int NT>
wc_status run_simt(const AttendArgs& a, cudaStream_t st) {
    int smem = SimtSmem<NT, RG>(a.s.d, a.s.dv, 4).total;
    if (a.csplits) smem = max(smem, CoresetSmem<NT, RG>(a.s.d, a.s.dv, 4).total);
    return a.s.dv <= 128 ? run(a, cache_attend_simt_kernel<RG, NT, 1>, smem, kWarps * NT, st)
                         : run(a, cache_attend_simt_kernel<RG, NT, 2>, smem, kWarps * NT, st);
}

template <int RG>
wc_status by_keys(const AttendArgs& a, cudaStream_t st) {
    // 16 keys a warp while two stages of them fit shared memory beside the rest (rows of up to 1024 bytes)
    return (a.s.d + a.s.dv) * 4 <= 1024 ? run_simt<RG, 16>(a, st) : run_simt<RG, 8>(a, st);
}

template <int DP, int SETS>
wc_status run_mma(const AttendArgs& a, cudaStream_t st) {
    constexpr int rows = SETS == 1 ? 4 : SETS == 2 ? 8 : 16;
    int smem = kWarps * kMmaStages * 2 * kMmaKeys * DP * 2;
    if (a.csplits) smem = max(smem, CoresetSmem<kCoresetKeys<DP>, rows>(a.s.d, a.s.dv, 2).total);
    return run(a, cache_attend_mma_kernel<DP, SETS>, smem, kWarps * kMmaKeys, st);
}

template <int DP>
wc_status by_sets(const AttendArgs& a, cudaStream_t st) {
    return a.rows == 4 ? run_mma<DP, 1>(a, st) : a.rows == 8 ? run_mma<DP, 2>(a, st) : run_mma<DP, 3>(a, st);
}

}  // namespace

wc_status launch_attend(const AttendArgs& a, cudaStream_t st) {
    if (a.s.dtype == WC_BF16) {
        const int w = max(a.s.d, a.s.dv);
        return w <= 64 ? by_sets<64>(a, st) : w <= 128 ? by_sets<128>(a, st) : by_sets<256>(a, st);
    }
    switch (a.rows) {
        case 1: return by_keys<1>(a, st);
        case 2: return by_keys<2>(a, st);
        case 4: return by_keys<4>(a, st);
        default: return by_keys<8>(a, st);
    }
}

}  // namespace cache
}  // namespace wc
