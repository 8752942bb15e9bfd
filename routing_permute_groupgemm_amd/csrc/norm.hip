// Layer norm of the tokens in front of the router and the experts, with the
// residual stream's addition, and its backward pass.
//
//   s = x + add,  y = (s - mean) * rstd * weight + bias     (rms: mean = 0, no bias needed)
// Backward, with xh = (s - mean) * rstd and g = dy * weight:
//   dx = rstd * (g - avg(g) - xh * avg(g * xh)) + d_sum     (rms: without avg(g))
//   dw = sum over tokens of dy * xh,  db = sum over tokens of dy
//
// A row is held in registers by a group of G threads (a wave, or a workgroup),
// 8 neighbouring columns a thread and chunk, so every array passes once: the
// bound is HBM.  The mean is taken first and the spread from the differences, so
// an offset that is large against the spread costs no digits; a second sum of
// the differences corrects the mean's own rounding.
//
// In the backward a thread keeps the sums of dy * xh and dy of its columns over
// all rows its group takes; the groups' sums become one partial row per
// workgroup, and column_sums adds those in a fixed order: no atomics, equal bits
// from run to run.
#include "columns.hpp"

using moe_host::misaligned;

namespace moe {

// The 8 columns of one chunk, as stored: 16 bytes of bf16 or 32 of fp32.
template <typename X>
struct Chunk;
template <>
struct Chunk<uint16_t> {
    u32x4 v;
    __device__ __forceinline__ void load(const uint16_t* p) { v = *(const u32x4*)p; }
    __device__ __forceinline__ void store(uint16_t* p) const { *(u32x4*)p = v; }
    __device__ __forceinline__ void zero() { v = u32x4{0u, 0u, 0u, 0u}; }
    __device__ __forceinline__ float get(int i) const { return i & 1 ? bf_hi(v[i >> 1]) : bf_lo(v[i >> 1]); }
    __device__ __forceinline__ void set(const float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = pack_bf2x(f[2 * i], f[2 * i + 1]);
    }
};
template <>
struct Chunk<float> {
    f32x4 v[2];
    __device__ __forceinline__ void load(const float* p) {
        v[0] = *(const f32x4*)p;
        v[1] = *(const f32x4*)(p + 4);
    }
    __device__ __forceinline__ void store(float* p) const {
        *(f32x4*)p = v[0];
        *(f32x4*)(p + 4) = v[1];
    }
    __device__ __forceinline__ void zero() { v[0] = v[1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f}; }
    __device__ __forceinline__ float get(int i) const { return v[i >> 2][i & 3]; }
    __device__ __forceinline__ void set(const float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i >> 2][i & 3] = f[i];
    }
};

// Sums of N values over the G threads of a row's group, the same bits in each of
// them: a butterfly over a wave's lanes, then the waves' sums in wave order.
// `red` holds two buffers that calls use in turn, so one barrier a call is enough.
template <int G, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float (*red)[G / 64][N], int& turn) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], o, 64);
    if constexpr (G > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) red[turn][wave][i] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = red[turn][0][i];
            for (int w = 1; w < G / 64; ++w) v[i] += red[turn][w][i];
        }
        turn ^= 1;
    }
}

constexpr int wg_threads(int G) { return G < 256 ? 256 : G; }

template <typename X, int G, int V, bool RMS>
__global__ __launch_bounds__(wg_threads(G)) void norm_kernel(const X* x, const uint16_t* __restrict__ add,
                                                             int64_t T, int H, const float* __restrict__ weight,
                                                             const float* __restrict__ bias, float eps, X* sum,
                                                             uint16_t* __restrict__ y, float* __restrict__ mean,
                                                             float* __restrict__ rstd) {
    constexpr int kRows = wg_threads(G) / G;  // rows of a workgroup
    __shared__ float red[2][G / 64][2];
    int turn = 0;
    const int tid = threadIdx.x % G;
    const float cols = (float)H;
    for (int64_t t = (int64_t)blockIdx.x * kRows + threadIdx.x / G; t < T; t += (int64_t)gridDim.x * kRows) {
        Chunk<X> c[V];
        float v[V][8];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int n = (j * G + tid) * 8;
            if (n < H) c[j].load(x + t * H + n);
            else c[j].zero();
        }
        if (add) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int n = (j * G + tid) * 8;
                if (n >= H) continue;
                Chunk<uint16_t> a;
                a.load(add + t * H + n);
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = c[j].get(i) + a.get(i);
                c[j].set(f);  // the sum as it is stored: what the backward reads
            }
        }
        if (sum) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int n = (j * G + tid) * 8;
                if (n < H) c[j].store(sum + t * H + n);
            }
        }
        float m0 = 0.0f;
        if constexpr (!RMS) {
            float s[1] = {0.0f};
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) s[0] += c[j].get(i);
            group_sum<G, 1>(s, (float(*)[G / 64][1])red, turn);
            m0 = s[0] / cols;
        }
        float q[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const bool in = (j * G + tid) * 8 < H;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[j][i] = in ? c[j].get(i) - m0 : 0.0f;
                q[0] += v[j][i] * v[j][i];
                q[1] += v[j][i];
            }
        }
        float d = 0.0f;
        if constexpr (RMS) {
            float s[1] = {q[0]};
            group_sum<G, 1>(s, (float(*)[G / 64][1])red, turn);
            q[0] = s[0] / cols;
        } else {
            group_sum<G, 2>(q, red, turn);
            d = q[1] / cols;
            q[0] = q[0] / cols - d * d;
            if (q[0] < 0.0f) q[0] = 0.0f;  // a NaN stays
        }
        const float r = 1.0f / sqrtf(q[0] + eps);
        if (tid == 0) {
            if (!RMS && mean) mean[t] = m0 + d;
            if (rstd) rstd[t] = r;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int n = (j * G + tid) * 8;
            if (n >= H) continue;
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = (v[j][i] - d) * r;
            if (weight) {
                Chunk<float> w;
                w.load(weight + n);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] *= w.get(i);
            }
            if (bias) {
                Chunk<float> b;
                b.load(bias + n);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] += b.get(i);
            }
            Chunk<uint16_t> o;
            o.set(f);
            o.store(y + t * H + n);
        }
    }
}

// part: [gridDim.x][2 * H] (the partial sums of dw, then of db), or NULL.
template <typename X, int G, int V, bool RMS>
__global__ __launch_bounds__(wg_threads(G)) void norm_backward_kernel(
    const uint16_t* __restrict__ dy, const X* __restrict__ s, int64_t T, int H, const float* __restrict__ weight,
    const float* __restrict__ mean, const float* __restrict__ rstd, const X* d_sum, X* dx, float* __restrict__ part) {
    constexpr int kRows = wg_threads(G) / G;
    __shared__ float red[2][G / 64][2];
    __shared__ __attribute__((aligned(16))) float merge[kRows > 1 ? kRows - 1 : 1][kRows > 1 ? G * 8 : 4];
    int turn = 0;
    const int tid = threadIdx.x % G, group = threadIdx.x / G;
    const float cols = (float)H;
    float w[V][8], dw[V][8], db[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int n = (j * G + tid) * 8;
        Chunk<float> c;
        if (weight && n < H) c.load(weight + n);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[j][i] = weight && n < H ? c.get(i) : 1.0f;
            dw[j][i] = db[j][i] = 0.0f;
        }
    }
    for (int64_t t = (int64_t)blockIdx.x * kRows + group; t < T; t += (int64_t)gridDim.x * kRows) {
        Chunk<uint16_t> cd[V];
        Chunk<X> cs[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int n = (j * G + tid) * 8;
            if (n < H) {
                cd[j].load(dy + t * H + n);
                cs[j].load(s + t * H + n);
            }
        }
        const float m = RMS ? 0.0f : mean[t], r = rstd[t];
        float q[2] = {0.0f, 0.0f};
        float g[V][8], xh[V][8];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const bool in = (j * G + tid) * 8 < H;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = in ? cd[j].get(i) : 0.0f;
                xh[j][i] = in ? (cs[j].get(i) - m) * r : 0.0f;
                g[j][i] = v * w[j][i];
                dw[j][i] += v * xh[j][i];
                db[j][i] += v;
                q[0] += g[j][i] * xh[j][i];
                q[1] += g[j][i];
            }
        }
        if constexpr (RMS) {
            float a[1] = {q[0]};
            group_sum<G, 1>(a, (float(*)[G / 64][1])red, turn);
            q[0] = a[0];
            q[1] = 0.0f;
        } else {
            group_sum<G, 2>(q, red, turn);
        }
        const float c2 = q[0] / cols, c1 = q[1] / cols;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int n = (j * G + tid) * 8;
            if (n >= H) continue;
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = r * (g[j][i] - c1 - xh[j][i] * c2);
            if (d_sum) {
                Chunk<X> a;
                a.load(d_sum + t * H + n);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] += a.get(i);
            }
            Chunk<X> o;
            o.set(f);
            o.store(dx + t * H + n);
        }
    }
    if (!part) return;
    // the groups' sums in group order, then one partial row
#pragma unroll
    for (int which = 0; which < (RMS ? 1 : 2); ++which)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int n = (j * G + tid) * 8;
            float(&a)[8] = which ? db[j] : dw[j];
            if constexpr (kRows > 1) {
                __syncthreads();
                if (group > 0) {
                    *(f32x4*)(&merge[group - 1][tid * 4]) = f32x4{a[0], a[1], a[2], a[3]};
                    *(f32x4*)(&merge[group - 1][G * 4 + tid * 4]) = f32x4{a[4], a[5], a[6], a[7]};
                }
                __syncthreads();
                if (group == 0)
#pragma unroll
                    for (int o = 0; o < kRows - 1; ++o) {
                        const f32x4 lo = *(const f32x4*)(&merge[o][tid * 4]);
                        const f32x4 hi = *(const f32x4*)(&merge[o][G * 4 + tid * 4]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            a[i] += lo[i];
                            a[4 + i] += hi[i];
                        }
                    }
            }
            if (group == 0 && n < H) {
                float* p = part + (int64_t)blockIdx.x * 2 * H + (which ? H : 0) + n;
                *(f32x4*)p = f32x4{a[0], a[1], a[2], a[3]};
                *(f32x4*)(p + 4) = f32x4{a[4], a[5], a[6], a[7]};
            }
        }
}

// 64 columns (16 lanes x 4) by 16 strands of the rows; the strands' sums meet in LDS
// and are added in strand order.
__global__ __launch_bounds__(256) void column_sums_kernel(const float* __restrict__ part, int rows, int64_t stride, int n,
                                                          float* __restrict__ out0, float* __restrict__ out1) {
    __shared__ f32x4 s_sum[16][16];
    const int lane = threadIdx.x & 15, strand = threadIdx.x >> 4;
    int c = (int)blockIdx.x * 64 + lane * 4;
    float* out = out0;
    if (c >= n || !out0) {
        if (out0) c -= n;
        out = out1;
    }
    const int64_t at = out == out1 && out1 ? (int64_t)n + c : c;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int p = strand; p < rows; p += 16) acc += *(const f32x4*)(part + p * stride + at);
    s_sum[strand][lane] = acc;
    __syncthreads();
    if (strand == 0) {
#pragma unroll
        for (int i = 1; i < 16; ++i) acc += s_sum[i][lane];
        *(f32x4*)(out + c) = acc;
    }
}

// Threads of a row and chunks of a thread.
struct NormPlan {
    int G, V;
};
static NormPlan norm_plan(int64_t T, int H) {
    const int chunks = H / 8;
    int G = chunks <= 256 ? 64 : chunks <= 1024 ? 256 : 1024;
    // few rows: as many threads a row as it has chunks, since only a row's own latency counts
    if (T <= moe_host::num_cus()) G = chunks <= 64 ? 64 : chunks <= 256 ? 256 : 1024;
    const int v = (chunks + G - 1) / G;
    return {G, v <= 1 ? 1 : v <= 2 ? 2 : 4};
}

constexpr int kNormMaxH = 16384;

static int norm_grid(int64_t T, int G, int per_cu) {
    const int rows = wg_threads(G) / G;
    return (int)std::min<int64_t>((T + rows - 1) / rows, (int64_t)moe_host::num_cus() * per_cu);
}

// Workgroups of the backward, and so partial rows.
static int norm_backward_grid(int64_t T, int G) { return norm_grid(T, G, G == 1024 ? 1 : 2); }

#define MOE_NORM_CASES(X, RMS)                                  \
    if (p.G == 64 && p.V == 1) MOE_NORM_LAUNCH(X, 64, 1, RMS);  \
    else if (p.G == 64 && p.V == 2) MOE_NORM_LAUNCH(X, 64, 2, RMS);  \
    else if (p.G == 64) MOE_NORM_LAUNCH(X, 64, 4, RMS);         \
    else if (p.G == 256 && p.V == 1) MOE_NORM_LAUNCH(X, 256, 1, RMS); \
    else if (p.G == 256 && p.V == 2) MOE_NORM_LAUNCH(X, 256, 2, RMS); \
    else if (p.G == 256) MOE_NORM_LAUNCH(X, 256, 4, RMS);       \
    else if (p.V == 1) MOE_NORM_LAUNCH(X, 1024, 1, RMS);        \
    else MOE_NORM_LAUNCH(X, 1024, 2, RMS);

static int check_norm(int T, int H) {
    if (T < 0 || H <= 0 || H > kNormMaxH) return MOE_EINVAL;
    if (H % 64) return MOE_ESHAPE;
    return MOE_OK;
}

}  // namespace moe

namespace moe_host {

int column_sums(const float* part, int rows, int64_t stride, int n, float* out0, float* out1, hipStream_t s) {
    const int sets = (out0 ? 1 : 0) + (out1 ? 1 : 0);
    if (sets == 0 || n == 0) return MOE_OK;
    moe::column_sums_kernel<<<sets * (n / 64), 256, 0, s>>>(part, rows, stride, n, out0, out1);
    return launch_status();
}

}  // namespace moe_host

extern "C" int moe_layer_norm(const void* x, int x_f32, const moe_bf16* add, int T, int H, const float* weight,
                              const float* bias, float eps, int rms, void* sum, moe_bf16* y, float* mean, float* rstd,
                              moe_stream stream) {
    using namespace moe;
    const int st = check_norm(T, H);
    if (st != MOE_OK) return st;
    if ((x_f32 & ~1) || (rms & ~1) || !(eps >= 0.0f)) return MOE_EINVAL;
    if (T == 0) return MOE_OK;
    if (!x || !y) return MOE_EINVAL;
    if (misaligned(x) || misaligned(add) || misaligned(weight) || misaligned(bias) || misaligned(sum) || misaligned(y) ||
        misaligned(mean) || misaligned(rstd))
        return MOE_EALIGN;
    hipStream_t s = (hipStream_t)stream;
    const NormPlan p = norm_plan(T, H);
    const int grid = norm_grid(T, p.G, p.G == 1024 ? 2 : 8);
#define MOE_NORM_LAUNCH(X, G, V, RMS)                                                                             \
    norm_kernel<X, G, V, RMS><<<grid, wg_threads(G), 0, s>>>((const X*)x, add, T, H, weight, bias, eps, (X*)sum, y, \
                                                             mean, rstd)
    if (x_f32) {
        if (rms) { MOE_NORM_CASES(float, true) }
        else { MOE_NORM_CASES(float, false) }
    } else {
        if (rms) { MOE_NORM_CASES(uint16_t, true) }
        else { MOE_NORM_CASES(uint16_t, false) }
    }
#undef MOE_NORM_LAUNCH
    return moe_host::launch_status();
}

extern "C" size_t moe_layer_norm_backward_workspace_size(int T, int H) {
    using namespace moe;
    if (check_norm(T, H) != MOE_OK || T == 0) return 0;
    return (size_t)norm_backward_grid(T, norm_plan(T, H).G) * 2 * H * 4;
}

extern "C" int moe_layer_norm_backward(const moe_bf16* dy, const void* s, int x_f32, int T, int H, const float* weight,
                                       const float* mean, const float* rstd, int rms, const void* d_sum, void* dx,
                                       float* dw, float* db, void* ws, size_t ws_bytes, moe_stream stream) {
    using namespace moe;
    const int st = check_norm(T, H);
    if (st != MOE_OK) return st;
    if ((x_f32 & ~1) || (rms & ~1) || (rms && db)) return MOE_EINVAL;
    if (T > 0 && (!dy || !s || !rstd || !dx || (!rms && !mean))) return MOE_EINVAL;
    if (misaligned(dy) || misaligned(s) || misaligned(weight) || misaligned(mean) || misaligned(rstd) ||
        misaligned(d_sum) || misaligned(dx) || misaligned(dw) || misaligned(db) || misaligned(ws))
        return MOE_EALIGN;
    hipStream_t q = (hipStream_t)stream;
    if (T == 0) return moe_host::column_sums(nullptr, 0, 0, H, dw, db, q);
    const bool sums = dw || db;
    if (sums && (!ws || ws_bytes < moe_layer_norm_backward_workspace_size(T, H))) return MOE_EWORKSPACE;
    const NormPlan p = norm_plan(T, H);
    const int grid = norm_backward_grid(T, p.G);
    float* part = sums ? (float*)ws : nullptr;
#define MOE_NORM_LAUNCH(X, G, V, RMS)                                                                             \
    norm_backward_kernel<X, G, V, RMS><<<grid, wg_threads(G), 0, q>>>(dy, (const X*)s, T, H, weight, mean, rstd,   \
                                                                      (const X*)d_sum, (X*)dx, part)
    if (x_f32) {
        if (rms) { MOE_NORM_CASES(float, true) }
        else { MOE_NORM_CASES(float, false) }
    } else {
        if (rms) { MOE_NORM_CASES(uint16_t, true) }
        else { MOE_NORM_CASES(uint16_t, false) }
    }
#undef MOE_NORM_LAUNCH
    const int rc = moe_host::launch_status();
    if (rc != MOE_OK || !sums) return rc;
    return moe_host::column_sums(part, grid, 2 * (int64_t)H, H, dw, db, q);
}
