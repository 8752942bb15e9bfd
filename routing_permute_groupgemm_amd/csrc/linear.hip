// Dense product with bias, activation and residual in its epilogue, and its
// backward: the products of a block that do not go by expert (a shared expert's
// down product onto the routed experts' output, a dense feed-forward layer).
//
//   z = x . w + bias (fp32),  y = bf16(act(z) + residual),  optionally bf16(z) for the backward
//   dz = bf16(dy * act'(z)),  dx = bf16(dz . w^T),  dw = x^T . dz (fp32),  db = sum over rows of dy * act'(z) (fp32)
//
// Forward, by the number of rows:
//   few rows (at most kFewRows)  the weights' bytes are the time: linear_rows streams them (rows_stream.hpp), the
//     contraction in chunks over the workgroups where the columns alone are too few;
//   more rows  the GroupGEMM's kernel on one dense group with EPI_LINEAR, or, where its tiles would leave most of the
//     chip idle, 128 x 128 tiles over chunks of the contraction.
// Chunks leave fp32 partial sums, which linear_finish adds in chunk order before it does what the epilogue does.
// The backward's products are the GroupGEMM's as well; linear_slope forms dz and the partial column sums of db in
// one pass.
#include "columns.hpp"
#include "gemm_kernel.hpp"
#include "rows_stream.hpp"

using moe_host::misaligned;

namespace moe {

constexpr int kFewRows = 64;
constexpr int kRowsCols = 128;  // columns of a linear_rows workgroup

struct LinearParams {
    const uint16_t* x;
    const uint16_t* w;
    const float* bias;
    const uint16_t* res;
    uint16_t* z;
    uint16_t* y;
    float* part;  // [chunks][T][N], or NULL: one chunk
    int T, Kd, N, act;
    int steps;    // contraction steps of 32 in a chunk
};

// Columns n .. n+3 of row t from their sum.
__device__ __forceinline__ void finish4(const LinearParams& p, int64_t t, int n, f32x4 f) {
    const int64_t at = t * p.N + n;
    if (p.bias) f += *(const f32x4*)(p.bias + n);
    if (p.z) *(u32x2*)(p.z + at) = u32x2{pack_bf2x(f[0], f[1]), pack_bf2x(f[2], f[3])};
    activate(f, p.act);
    if (p.res) f += widen4(*(const u32x2*)(p.res + at));
    *(u32x2*)(p.y + at) = u32x2{pack_bf2x(f[0], f[1]), pack_bf2x(f[2], f[3])};
}

template <int MT, int S, int W>
__global__ __launch_bounds__(64 * W) void linear_rows(LinearParams p) {
    __shared__ __attribute__((aligned(16))) WaveSums<1, 8, W> sums;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slabs = (p.N + kRowsCols - 1) / kRowsCols;
    const int chunk = (int)blockIdx.x / slabs, col0 = ((int)blockIdx.x % slabs) * kRowsCols;
    uint32_t x_at[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) x_at[m] = (uint32_t)min(16 * m + (lane & 15), p.T - 1) * (uint32_t)(p.Kd * 2);
    const uint16_t* const w[1] = {p.w};
    RowStream<1, 8, MT, S, false> r;
    // columns past the last are read as the last ones; their sums are not stored
    r.run(w, p.N, min(col0 + 8 * (lane & 15), p.N - 8), p.x, x_at, p.T, chunk * p.steps + wave, W,
          min((chunk + 1) * p.steps, p.Kd / 32));
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (16 * m >= p.T) break;
        if (m > 0) __syncthreads();
        sums.put(r, m, wave, lane);
        __syncthreads();
        for (int i = tid; i < 512; i += 64 * W) {
            const int row = 16 * m + (i >> 5), c = (i & 31) * 4;
            if (row >= p.T || col0 + c >= p.N) continue;
            const f32x4 f = sums.get(i >> 5, c);
            if (p.part) *(f32x4*)(p.part + ((int64_t)chunk * p.T + row) * p.N + col0 + c) = f;
            else finish4(p, row, col0 + c, f);
        }
    }
}

__global__ __launch_bounds__(256) void linear_finish(LinearParams p, int chunks) {
    const int64_t n4 = (int64_t)p.T * p.N / 4, stride = n4;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (int64_t)gridDim.x * 256) {
        const f32x4* at = (const f32x4*)p.part + i;
        f32x4 f = *at;
        for (int c = 1; c < chunks; ++c) f += at[c * stride];
        const int64_t t = i * 4 / p.N;
        finish4(p, t, (int)(i * 4 - t * p.N), f);
    }
}

// dz = bf16(dy * act'(z)) (dz NULL: not written) and partial column sums of the unrounded products: a workgroup takes
// 512 columns (64 threads of 8) of the rows blockIdx.y * 4 + r, + 4 * gridDim.y, ...; its four strands of rows meet in
// LDS.
__global__ __launch_bounds__(256) void linear_slope(const uint16_t* dy, const uint16_t* __restrict__ z,
                                                    int64_t T, int N, int act, uint16_t* dz, float* __restrict__ part) {
    __shared__ __attribute__((aligned(16))) float merge[3][512];
    const int lane = threadIdx.x & 63, strand = threadIdx.x >> 6;
    const int n = (int)blockIdx.x * 512 + lane * 8;
    float sum[8] = {};
    if (n < N) {
        for (int64_t t = (int64_t)blockIdx.y * 4 + strand; t < T; t += 4 * (int64_t)gridDim.y) {
            const u32x4 d = *(const u32x4*)(dy + t * N + n);
            u32x4 v = {};
            if (act != MOE_ACT_NONE) v = *(const u32x4*)(z + t * N + n);
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[i] = i & 1 ? bf_hi(d[i >> 1]) : bf_lo(d[i >> 1]);
                if (act != MOE_ACT_NONE) f[i] *= slope(i & 1 ? bf_hi(v[i >> 1]) : bf_lo(v[i >> 1]), act);
                sum[i] += f[i];
            }
            if (dz)
                *(u32x4*)(dz + t * N + n) = u32x4{pack_bf2x(f[0], f[1]), pack_bf2x(f[2], f[3]), pack_bf2x(f[4], f[5]),
                                                  pack_bf2x(f[6], f[7])};
        }
    }
    if (!part) return;
    if (strand > 0) {
        *(f32x4*)&merge[strand - 1][lane * 8] = f32x4{sum[0], sum[1], sum[2], sum[3]};
        *(f32x4*)&merge[strand - 1][lane * 8 + 4] = f32x4{sum[4], sum[5], sum[6], sum[7]};
    }
    __syncthreads();
    if (strand == 0 && n < N) {
#pragma unroll
        for (int o = 0; o < 3; ++o)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] += merge[o][lane * 8 + i];
        float* p = part + (int64_t)blockIdx.y * N + n;
        *(f32x4*)p = f32x4{sum[0], sum[1], sum[2], sum[3]};
        *(f32x4*)(p + 4) = f32x4{sum[4], sum[5], sum[6], sum[7]};
    }
}

enum : int { FORM_ROWS = 0, FORM_SMALL = 1, FORM_BIG = 2 };

struct LinearPlan {
    int form, chunks, steps;      // forward
    int slope_rows;               // row blocks of linear_slope, and so partial rows of db
    int dw_chunks, dw_rows;       // weight gradient: row chunks
    size_t forward_bytes, db_bytes, backward_bytes;
};

static LinearPlan linear_plan(int T, int Kd, int N) {
    LinearPlan r{};
    const int64_t cus = moe_host::num_cus();
    const int kt = Kd / 32;
    r.chunks = 1;
    r.steps = kt;
    const int64_t big = (int64_t)((T + 255) / 256) * ((N + 255) / 256);
    if (T <= kFewRows) {
        r.form = FORM_ROWS;
        const int64_t slabs = (N + kRowsCols - 1) / kRowsCols;
        const int64_t want = std::max<int64_t>(1, std::min<int64_t>(cus / slabs, kt / 8));
        r.steps = (int)((kt + want - 1) / want);
        r.chunks = (kt + r.steps - 1) / r.steps;
    } else if (big >= cus) {
        r.form = FORM_BIG;
    } else {
        r.form = FORM_SMALL;
        split_steps((int64_t)((T + 127) / 128) * ((N + 127) / 128), kt, &r.chunks, &r.steps);
    }
    r.forward_bytes = r.chunks > 1 ? (size_t)r.chunks * T * N * 4 : 0;
    const int64_t blocks = (N + 511) / 512;
    r.slope_rows = (int)std::max<int64_t>(1, std::min<int64_t>(((int64_t)T + 15) / 16, 4 * cus / blocks));
    r.db_bytes = round256((size_t)r.slope_rows * N * 4);
    int steps;
    split_steps((int64_t)((Kd + 255) / 256) * ((N + 255) / 256), ((int64_t)T + 31) / 32, &r.dw_chunks, &steps);
    r.dw_rows = steps * 32;
    r.dw_chunks = std::max(1, (int)(((int64_t)T + r.dw_rows - 1) / r.dw_rows));
    r.backward_bytes = r.db_bytes + (r.dw_chunks > 1 ? (size_t)r.dw_chunks * Kd * N * 4 : 0);
    return r;
}

static int linear_check(int T, int Kd, int N, int act) {
    if (T < 0 || T > (1 << 30) || Kd <= 0 || N <= 0 || act < MOE_ACT_NONE || act > MOE_ACT_GELU) return MOE_EINVAL;
    if (Kd % 64 || N % 64) return MOE_ESHAPE;
    // 256 rows of an operand and the weights stay below 2 GiB (32-bit load offsets)
    if (Kd > (1 << 21) || N > (1 << 21) || (int64_t)256 * std::max(Kd, N) * 2 >= (1ll << 31) ||
        (int64_t)Kd * N * 2 >= (1ll << 31))
        return MOE_EINVAL;
    return MOE_OK;
}

template <int MT, int S>
static int launch_linear_rows(const LinearParams& p, int chunks, hipStream_t s) {
    constexpr int W = 4;
    const int grid = (p.N + kRowsCols - 1) / kRowsCols * chunks;
    linear_rows<MT, S, W><<<grid, 64 * W, 0, s>>>(p);
    return moe_host::launch_status();
}

static int linear_gemm(const LinearParams& l, const LinearPlan& r, hipStream_t s) {
    GemmParams p{};
    p.a = l.x;
    p.lda = l.Kd;
    p.w0 = l.w;
    p.ldw = l.N;
    p.dense_rows = l.T;
    p.row_chunk = l.T;
    p.e_local = 1;
    p.cap = l.T;
    p.N = l.N;
    p.Kd = l.Kd;
    p.ldc = l.N;
    if (r.chunks > 1) {
        p.cf = l.part;
        p.ksplit = r.chunks;
        p.kchunk = r.steps * 32;
        p.part_stride = (int64_t)l.T * l.N;
        return launch_rows_f32_small(p, s);
    }
    p.c = l.y;
    p.c2 = l.z;
    p.bias = l.bias;
    p.res = l.res;
    p.act = l.act;
    if (r.form == FORM_SMALL) return launch_cfg<128, 128, 32, 2, 2, LAY_MN, EPI_LINEAR, SCHED_ROWS, kLdsBudget>(p, s);
    return launch_cfg<256, 256, 32, 2, 2, LAY_MN, EPI_LINEAR, SCHED_ROWS, kLdsBudget>(p, s);
}

}  // namespace moe

extern "C" size_t moe_linear_workspace_size(int T, int Kd, int N) {
    using namespace moe;
    if (linear_check(T, Kd, N, MOE_ACT_NONE) != MOE_OK || T == 0) return 0;
    return linear_plan(T, Kd, N).forward_bytes;
}

extern "C" int moe_linear(const moe_bf16* x, int T, int Kd, const moe_bf16* w, int N, const float* bias, int act,
                          const moe_bf16* residual, moe_bf16* z, moe_bf16* y, void* ws, size_t ws_bytes,
                          moe_stream stream) {
    using namespace moe;
    const int st = linear_check(T, Kd, N, act);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    if (!x || !w || !y) return MOE_EINVAL;
    if (misaligned(x) || misaligned(w) || misaligned(bias) || misaligned(residual) || misaligned(z) || misaligned(y) ||
        misaligned(ws))
        return MOE_EALIGN;
    const LinearPlan r = linear_plan(T, Kd, N);
    if (r.chunks > 1 && (!ws || ws_bytes < r.forward_bytes)) return MOE_EWORKSPACE;
    hipStream_t s = (hipStream_t)stream;
    LinearParams p{x, w, bias, residual, z, y, r.chunks > 1 ? (float*)ws : nullptr, T, Kd, N, act, r.steps};
    int rc;
    if (r.form != FORM_ROWS) rc = linear_gemm(p, r, s);
    else if (T <= 16) rc = launch_linear_rows<1, 3>(p, r.chunks, s);
    else if (T <= 32) rc = launch_linear_rows<2, 2>(p, r.chunks, s);
    else rc = launch_linear_rows<4, 2>(p, r.chunks, s);
    if (rc != MOE_OK || r.chunks == 1) return rc;
    const int64_t blocks = std::min<int64_t>(((int64_t)T * N / 4 + 255) / 256, (int64_t)moe_host::num_cus() * 8);
    linear_finish<<<(int)blocks, 256, 0, s>>>(p, r.chunks);
    return moe_host::launch_status();
}

extern "C" size_t moe_linear_backward_workspace_size(int T, int Kd, int N) {
    using namespace moe;
    if (linear_check(T, Kd, N, MOE_ACT_NONE) != MOE_OK) return 0;
    return linear_plan(T, Kd, N).backward_bytes;
}

extern "C" int moe_linear_backward(const moe_bf16* dy, const moe_bf16* x, int T, int Kd, const moe_bf16* w, int N, int act,
                                   const moe_bf16* z, moe_bf16* dz, moe_bf16* dx, float* dw, float* db, void* ws,
                                   size_t ws_bytes, moe_stream stream) {
    using namespace moe;
    const int st = linear_check(T, Kd, N, act);
    if (st != MOE_OK) return st;
    const bool none = act == MOE_ACT_NONE;
    if (T > 0 && (!dy || (dw && !x) || (dx && !w) || (!none && (!z || !dz)))) return MOE_EINVAL;
    if (misaligned(dy) || misaligned(x) || misaligned(w) || misaligned(z) || misaligned(dz) || misaligned(dx) ||
        misaligned(dw) || misaligned(db) || misaligned(ws))
        return MOE_EALIGN;
    const LinearPlan r = linear_plan(T, Kd, N);
    const bool split = r.dw_chunks > 1;
    const size_t need = dw && split ? r.backward_bytes : db ? r.db_bytes : 0;
    if (need && (!ws || ws_bytes < need)) return MOE_EWORKSPACE;
    hipStream_t s = (hipStream_t)stream;
    float* db_part = (float*)ws;
    float* dw_part = (float*)((char*)ws + r.db_bytes);
    int rc;
    if (T > 0 && (db || !none)) {
        linear_slope<<<dim3((N + 511) / 512, r.slope_rows), 256, 0, s>>>(dy, z, T, N, act, none ? nullptr : dz,
                                                                        db ? db_part : nullptr);
        rc = moe_host::launch_status();
        if (rc != MOE_OK) return rc;
    }
    if (db) {
        rc = moe_host::column_sums(db_part, T > 0 ? r.slope_rows : 0, N, N, db, nullptr, s);
        if (rc != MOE_OK) return rc;
    }
    const uint16_t* d = none ? dy : dz;
    if (dx && T > 0) {  // w [Kd][N] is the [N][Kd] weight of this product, contraction contiguous
        GemmParams p{};
        p.a = d;
        p.lda = N;
        p.w0 = w;
        p.ldw = N;
        p.dense_rows = T;
        p.row_chunk = T;
        p.e_local = 1;
        p.cap = T;
        p.N = Kd;
        p.Kd = N;
        p.c = dx;
        p.ldc = Kd;
        rc = launch_rows_kc(p, EPI_BF16, s);
        if (rc != MOE_OK) return rc;
    }
    if (!dw) return MOE_OK;
    GemmParams q{};
    q.a = x;
    q.lda = Kd;
    q.b = d;
    q.ldb = N;
    q.dense_rows = T;
    q.row_chunk = r.dw_rows;
    q.e_local = r.dw_chunks;
    q.cap = T;
    q.M = Kd;
    q.N = N;
    q.cf = split ? dw_part : dw;
    q.n_split = N;
    rc = launch_wgrad(q, s);
    if (rc != MOE_OK || !split) return rc;
    return moe_host::sum_partials(dw_part, r.dw_chunks, (int64_t)Kd * N, (int64_t)Kd * N, nullptr, N, dw, s);
}
