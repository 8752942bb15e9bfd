// Layer norm of the tokens in front of the router and the experts, with the
// residual stream's addition, and its backward pass.
//
//   s = x + add,  y = (s - mean) * rstd * weight + bias     (rms: mean = 0, no bias needed)
// Backward, with xh = (s - mean) * rstd and g = dy * weight:
//   dx = rstd * (g - avg(g) - xh * avg(g * xh)) + d_sum     (rms: without avg(g))
//   dw = sum over tokens of dy * xh,  db = sum over tokens of dy
//
// A row is held in registers by a group of G threads (a wave, or several), so
// every array passes once: the bound is HBM.  The mean is taken first and the spread from the differences, so
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

// C neighbouring columns of a thread: 16 bytes of the residual stream's type (8 bf16 or 4 fp32), and as many of a bf16
// array beside it.  NT: the access carries the non-temporal hint.
template <typename V, bool NT>
__device__ __forceinline__ V load_vec(const void* p) {
    return NT ? __builtin_nontemporal_load((const V*)p) : *(const V*)p;
}
template <bool NT, typename V>
__device__ __forceinline__ void store_vec(void* p, V v) {
    if (NT) __builtin_nontemporal_store(v, (V*)p);
    else *(V*)p = v;
}
template <typename X, int C>
struct Piece;
template <int C>
struct Piece<uint16_t, C> {
    typedef __attribute__((ext_vector_type(C / 2))) uint32_t vec;
    vec v;
    template <bool NT>
    __device__ __forceinline__ void load(const uint16_t* p) { v = load_vec<vec, NT>(p); }
    template <bool NT>
    __device__ __forceinline__ void store(uint16_t* p) const { store_vec<NT>(p, v); }
    __device__ __forceinline__ float get(int i) const { return i & 1 ? bf_hi(v[i >> 1]) : bf_lo(v[i >> 1]); }
    __device__ __forceinline__ void set(const float (&f)[C]) {
#pragma unroll
        for (int i = 0; i < C / 2; ++i) v[i] = pack_bf2x(f[2 * i], f[2 * i + 1]);
    }
};
template <int C>
struct Piece<float, C> {
    f32x4 v[C / 4];
    template <bool NT>
    __device__ __forceinline__ void load(const float* p) {
#pragma unroll
        for (int i = 0; i < C / 4; ++i) v[i] = load_vec<f32x4, NT>(p + 4 * i);
    }
    template <bool NT>
    __device__ __forceinline__ void store(float* p) const {
#pragma unroll
        for (int i = 0; i < C / 4; ++i) store_vec<NT>(p + 4 * i, v[i]);
    }
    __device__ __forceinline__ float get(int i) const { return v[i >> 2][i & 3]; }
    __device__ __forceinline__ void set(const float (&f)[C]) {
#pragma unroll
        for (int i = 0; i < C; ++i) v[i >> 2][i & 3] = f[i];
    }
};
template <typename X>
constexpr int kPieceCols = 16 / (int)sizeof(X);

// Sum over the 64 lanes, the same bits in each: exchanges within 4, 8 and 16 lanes by DPP, then between rows of 16
// and halves by lane swaps (no LDS round trip).
__device__ __forceinline__ float wave_sum(float v) {
    auto add_dpp = [&](auto ctrl) {
        v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), ctrl(), 0xf, 0xf, true));
    };
    add_dpp([]() constexpr { return 0xB1; });   // quad [1,0,3,2]
    add_dpp([]() constexpr { return 0x4E; });   // quad [2,3,0,1]
    add_dpp([]() constexpr { return 0x141; });  // row_half_mirror
    add_dpp([]() constexpr { return 0x140; });  // row_mirror
    const uint32_t u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const uint32_t x = __float_as_uint(v);
    const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Sums of N values over the G threads of a row's group, the same bits in each of
// them: over a wave's lanes, then the waves' sums in wave order.
// `red` holds two buffers that calls use in turn, so one barrier a call is enough.
template <int G, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float (*red)[G / 64][N], int& turn) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if constexpr (G > 64) {
        const int wave = (threadIdx.x % G) >> 6;  // of the group
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

// Threads of a workgroup: four rows of a wave each, or one row.
constexpr int wg_threads(int G) { return G == 64 ? 256 : G; }

template <typename X, int G, int V, bool RMS, bool NT>
__global__ __launch_bounds__(wg_threads(G)) void norm_kernel(const X* x, const uint16_t* __restrict__ add, int64_t T,
                                                             int H, const float* __restrict__ weight,
                                                             const float* __restrict__ bias, float eps, X* sum,
                                                             uint16_t* __restrict__ y, float* __restrict__ mean,
                                                             float* __restrict__ rstd) {
    constexpr int C = kPieceCols<X>, P = V * 8 / C;
    constexpr int kRows = wg_threads(G) / G;  // rows of a workgroup
    __shared__ float red[2][G / 64][2];
    int turn = 0;
    const int tid = threadIdx.x % G;
    const float cols = (float)H;
    for (int64_t t = (int64_t)blockIdx.x * kRows + threadIdx.x / G; t < T; t += (int64_t)gridDim.x * kRows) {
        Piece<X, C> c[P];
        Piece<uint16_t, C> a[P];
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const int n = (j * G + tid) * C;
            if (n < H) {
                c[j].template load<NT>(x + t * H + n);
                if (add) a[j].template load<NT>(add + t * H + n);
            }
        }
        float v[P][C];
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const int n = (j * G + tid) * C;
            if (add) {
                float f[C];
#pragma unroll
                for (int i = 0; i < C; ++i) f[i] = c[j].get(i) + a[j].get(i);
                c[j].set(f);  // the sum as it is stored: what the backward reads
            }
            if (sum && n < H) c[j].template store<NT>(sum + t * H + n);
        }
        float m0 = 0.0f;
        if constexpr (!RMS) {
            float s[1] = {0.0f};
#pragma unroll
            for (int j = 0; j < P; ++j)
#pragma unroll
                for (int i = 0; i < C; ++i) s[0] += (j * G + tid) * C < H ? c[j].get(i) : 0.0f;
            group_sum<G, 1>(s, (float(*)[G / 64][1])red, turn);
            m0 = s[0] / cols;
        }
        float q[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const bool in = (j * G + tid) * C < H;
#pragma unroll
            for (int i = 0; i < C; ++i) {
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
        for (int j = 0; j < P; ++j) {
            const int n = (j * G + tid) * C;
            if (n >= H) continue;
            float f[C];
#pragma unroll
            for (int i = 0; i < C; ++i) f[i] = (v[j][i] - d) * r;
            if (weight) {
                Piece<float, C> w;
                w.template load<false>(weight + n);
#pragma unroll
                for (int i = 0; i < C; ++i) f[i] *= w.get(i);
            }
            if (bias) {
                Piece<float, C> b;
                b.template load<false>(bias + n);
#pragma unroll
                for (int i = 0; i < C; ++i) f[i] += b.get(i);
            }
            Piece<uint16_t, C> o;
            o.set(f);
            o.template store<NT>(y + t * H + n);
        }
    }
}

// Threads of the backward's workgroups: its rows' sums are merged before they leave, so the more rows a workgroup has,
// the fewer partial rows are written and read again.
constexpr int back_threads(int G) { return G < 512 ? 512 : G; }

// Workgroup b leaves its sums of dw at dw_out + b * stride and those of db at db_out + b * stride (either NULL: not
// wanted): partial rows, or the results themselves where there is one workgroup.
template <typename X, int G, int V, bool RMS, bool NT>
__global__ __launch_bounds__(back_threads(G)) void norm_backward_kernel(
    const uint16_t* __restrict__ dy, const X* __restrict__ s, int64_t T, int H, const float* __restrict__ weight,
    const float* __restrict__ mean, const float* __restrict__ rstd, const X* d_sum, X* dx, float* __restrict__ dw_out,
    float* __restrict__ db_out, int64_t stride) {
    constexpr int C = kPieceCols<X>, P = V * 8 / C;
    constexpr int kRows = back_threads(G) / G;
    __shared__ float red[kRows][2][G / 64][2];
    __shared__ __attribute__((aligned(16))) f32x4 merge[kRows > 1 ? kRows - 1 : 1][kRows > 1 ? G : 1];
    int turn = 0;
    const int tid = threadIdx.x % G, group = threadIdx.x / G;
    const float cols = (float)H;
    // with one chunk a thread the weights stay in registers; two leave no room for them (1024 threads have 128 each)
    constexpr bool kKeep = V == 1;
    float w[P][C], dw[P][C], db[P][C];
    auto weights = [&]() {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const int n = (j * G + tid) * C;
            Piece<float, C> c;
            if (weight && n < H) c.template load<false>(weight + n);
#pragma unroll
            for (int i = 0; i < C; ++i) w[j][i] = n >= H ? 0.0f : weight ? c.get(i) : 1.0f;
        }
    };
    if (kKeep) weights();
#pragma unroll
    for (int j = 0; j < P; ++j)
#pragma unroll
        for (int i = 0; i < C; ++i) dw[j][i] = db[j][i] = 0.0f;
    // every group of the workgroup makes as many rounds (the sums' barriers), past the last row with nothing
    for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < T; t0 += (int64_t)gridDim.x * kRows) {
        const int64_t t = t0 + group;
        const bool row = t < T;
        Piece<uint16_t, C> cd[P];
        Piece<X, C> cs[P], add[P];
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const int n = (j * G + tid) * C;
            if (row && n < H) {
                cd[j].template load<NT>(dy + t * H + n);
                cs[j].template load<NT>(s + t * H + n);
                if (d_sum) add[j].template load<NT>(d_sum + t * H + n);
            }
        }
        const float m = RMS || !row ? 0.0f : mean[t], r = row ? rstd[t] : 0.0f;
        if (!kKeep) weights();
        float q[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const bool in = row && (j * G + tid) * C < H;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const float v = in ? cd[j].get(i) : 0.0f, xh = in ? (cs[j].get(i) - m) * r : 0.0f;
                dw[j][i] += v * xh;
                db[j][i] += v;
                q[0] += v * w[j][i] * xh;
                q[1] += v * w[j][i];
            }
        }
        if constexpr (RMS) {
            float a[1] = {q[0]};
            group_sum<G, 1>(a, (float(*)[G / 64][1])red[group], turn);
            q[0] = a[0];
            q[1] = 0.0f;
        } else {
            group_sum<G, 2>(q, red[group], turn);
        }
        const float c2 = q[0] / cols, c1 = q[1] / cols;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const int n = (j * G + tid) * C;
            if (!row || n >= H) continue;
            float f[C];
#pragma unroll
            for (int i = 0; i < C; ++i) {
                f[i] = r * (cd[j].get(i) * w[j][i] - c1 - (cs[j].get(i) - m) * r * c2);
                if (d_sum) f[i] += add[j].get(i);
            }
            Piece<X, C> o;
            o.set(f);
            o.template store<NT>(dx + t * H + n);
        }
    }
    // the groups' sums in group order
#pragma unroll
    for (int which = 0; which < (RMS ? 1 : 2); ++which) {
        float* out = which ? db_out : dw_out;
        if (!out) continue;
#pragma unroll
        for (int j = 0; j < P; ++j)
#pragma unroll
            for (int h = 0; h < C / 4; ++h) {
                const int n = (j * G + tid) * C + 4 * h;
                float(&from)[C] = which ? db[j] : dw[j];
                f32x4 a = {from[4 * h], from[4 * h + 1], from[4 * h + 2], from[4 * h + 3]};
                if constexpr (kRows > 1) {
                    __syncthreads();
                    if (group > 0) merge[group - 1][tid] = a;
                    __syncthreads();
                    if (group == 0)
#pragma unroll
                        for (int o = 0; o < kRows - 1; ++o) a += merge[o][tid];
                }
                if (group == 0 && n < H) *(f32x4*)(out + (int64_t)blockIdx.x * stride + n) = a;
            }
    }
}

__global__ __launch_bounds__(256) void column_sums_kernel(const float* __restrict__ part, int rows, int64_t stride, int n,
                                                          float* __restrict__ out0, float* __restrict__ out1) {
    // the blocks of out0's columns, then those of out1's
    const bool second = !out0 || (int)blockIdx.x * 16 >= n;
    const int c = (int)blockIdx.x * 16 - (second && out0 ? n : 0);
    sum_columns(part + (second ? n : 0) + c, rows, stride, (second ? out1 : out0) + c);
}

// Threads of a row and chunks of 8 columns of a thread (G threads hold 8*G*V columns), and the hint, from the sizes.
// Measured (us; rows x columns, bf16 with the addition, rms, if nothing else is said):
//   forward: up to 4 chunks a thread, so that a row's sums cross few waves; few rows: as many threads a row as it has
//     chunks, since only a row's own latency counts (1 x 7168: 2.6).
//   backward: one chunk, whose columns' sums leave registers for many waves: 16384 x 2048 51 against 62 with four chunks
//     and a wave a row; rows of more than 8192 columns take two.
//   backward's workgroups: 512 threads, one or two a CU, so that there are few partial rows: with 128-thread workgroups
//     (2048 partial rows) 16384 x 2048 61.
//   the hint, for passes of 128 MB and more: 131072 x 7168 forward 1484 against 1633 and backward 1368 against 1492 (of
//     the kernels of the time); 1000 x 7168 (57 MB) backward 20 without, 25 with it.
struct NormPlan {
    int G, V;
};
static NormPlan norm_plan(int64_t T, int H, bool back) {
    const int chunks = H / 8;
    const int most = back || T <= moe_host::num_cus() ? 1 : 4;
    int G = 64;
    while (G < 1024 && chunks > G * most) G *= 2;
    const int v = (chunks + G - 1) / G;
    return {G, v <= 1 ? 1 : v <= 2 ? 2 : 4};
}

constexpr int kNormMaxH = 16384;

// Workgroups of a pass that gives a CU this many threads.
static int norm_grid(int64_t T, int G, int wg, int threads) {
    const int rows = wg / G;
    return (int)std::min<int64_t>((T + rows - 1) / rows, (int64_t)moe_host::num_cus() * (threads / wg));
}

// Workgroups of the backward, and so partial rows.
// Up to four rows a group (two of the widest) one workgroup takes them all, which spares the launch that adds the partial
// rows: 2 x 2112 takes 3.3 us so, 4 x 2112 4.9, 5 x 2112 in two launches 5.0.
static int norm_backward_grid(int64_t T, NormPlan p) {
    if (T <= (p.G == 1024 ? 2 : 4) * (back_threads(p.G) / p.G)) return 1;
    return norm_grid(T, p.G, back_threads(p.G), 1024);
}

// Whether a pass that moves this many bytes passes the caches by.
static bool norm_stream(int64_t bytes) { return bytes >= (128ll << 20); }

// The plans that norm_plan gives, by pass.
#define MOE_NORM_CASE(X, G, V, RMS) \
    case G * 8 + V: MOE_NORM_LAUNCH(X, G, V, RMS); break;
#define MOE_NORM_FORWARD(X, RMS)                                                                         \
    switch (p.G * 8 + p.V) {                                                                             \
        MOE_NORM_CASE(X, 64, 1, RMS) MOE_NORM_CASE(X, 64, 2, RMS) MOE_NORM_CASE(X, 64, 4, RMS)           \
        MOE_NORM_CASE(X, 128, 1, RMS) MOE_NORM_CASE(X, 128, 4, RMS) MOE_NORM_CASE(X, 256, 1, RMS)        \
        MOE_NORM_CASE(X, 256, 4, RMS) MOE_NORM_CASE(X, 512, 1, RMS) MOE_NORM_CASE(X, 512, 4, RMS)        \
        MOE_NORM_CASE(X, 1024, 1, RMS) MOE_NORM_CASE(X, 1024, 2, RMS)                                    \
        default: return MOE_EINVAL;                                                                      \
    }
#define MOE_NORM_BACKWARD(X, RMS)                                                                        \
    switch (p.G * 8 + p.V) {                                                                             \
        MOE_NORM_CASE(X, 64, 1, RMS) MOE_NORM_CASE(X, 128, 1, RMS) MOE_NORM_CASE(X, 256, 1, RMS)         \
        MOE_NORM_CASE(X, 512, 1, RMS) MOE_NORM_CASE(X, 1024, 1, RMS) MOE_NORM_CASE(X, 1024, 2, RMS)      \
        default: return MOE_EINVAL;                                                                      \
    }

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
    moe::column_sums_kernel<<<sets * (n / 16), 256, 0, s>>>(part, rows, stride, n, out0, out1);
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
    const NormPlan p = norm_plan(T, H, false);
    const int grid = norm_grid(T, p.G, wg_threads(p.G), 2048);
    const int size = x_f32 ? 4 : 2;
    const bool nt = norm_stream((int64_t)T * H * (size + 2 + (add ? 2 : 0) + (sum ? size : 0)));
#define MOE_NORM_LAUNCH(X, G, V, RMS)                                                                              \
    if (nt)                                                                                                        \
        norm_kernel<X, G, V, RMS, true><<<grid, wg_threads(G), 0, s>>>((const X*)x, add, T, H, weight, bias, eps,  \
                                                                       (X*)sum, y, mean, rstd);                    \
    else                                                                                                           \
        norm_kernel<X, G, V, RMS, false><<<grid, wg_threads(G), 0, s>>>((const X*)x, add, T, H, weight, bias, eps, \
                                                                        (X*)sum, y, mean, rstd)
    if (x_f32) {
        if (rms) { MOE_NORM_FORWARD(float, true) }
        else { MOE_NORM_FORWARD(float, false) }
    } else {
        if (rms) { MOE_NORM_FORWARD(uint16_t, true) }
        else { MOE_NORM_FORWARD(uint16_t, false) }
    }
#undef MOE_NORM_LAUNCH
    return moe_host::launch_status();
}

extern "C" size_t moe_layer_norm_backward_workspace_size(int T, int H) {
    using namespace moe;
    if (check_norm(T, H) != MOE_OK || T == 0) return 0;
    const int grid = norm_backward_grid(T, norm_plan(T, H, true));
    return grid > 1 ? (size_t)grid * 2 * H * 4 : 0;
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
    const NormPlan p = norm_plan(T, H, true);
    const int grid = norm_backward_grid(T, p);
    const bool sums = grid > 1 && (dw || db);
    if (sums && (!ws || ws_bytes < moe_layer_norm_backward_workspace_size(T, H))) return MOE_EWORKSPACE;
    float* part = (float*)ws;
    float *dw_out = sums && dw ? part : dw, *db_out = sums && db ? part + H : db;
    const int64_t stride = sums ? 2 * (int64_t)H : 0;
    const int size = x_f32 ? 4 : 2;
    const bool nt = norm_stream((int64_t)T * H * (2 + 2 * size + (d_sum ? size : 0)));
#define MOE_NORM_LAUNCH(X, G, V, RMS)                                                                          \
    if (nt)                                                                                                    \
        norm_backward_kernel<X, G, V, RMS, true><<<grid, back_threads(G), 0, q>>>(                             \
            dy, (const X*)s, T, H, weight, mean, rstd, (const X*)d_sum, (X*)dx, dw_out, db_out, stride);                         \
    else                                                                                                       \
        norm_backward_kernel<X, G, V, RMS, false><<<grid, back_threads(G), 0, q>>>(                            \
            dy, (const X*)s, T, H, weight, mean, rstd, (const X*)d_sum, (X*)dx, dw_out, db_out, stride)
    if (x_f32) {
        if (rms) { MOE_NORM_BACKWARD(float, true) }
        else { MOE_NORM_BACKWARD(float, false) }
    } else {
        if (rms) { MOE_NORM_BACKWARD(uint16_t, true) }
        else { MOE_NORM_BACKWARD(uint16_t, false) }
    }
#undef MOE_NORM_LAUNCH
    const int rc = moe_host::launch_status();
    if (rc != MOE_OK || !sums) return rc;
    return moe_host::column_sums(part, grid, 2 * (int64_t)H, H, dw, db, q);
}
