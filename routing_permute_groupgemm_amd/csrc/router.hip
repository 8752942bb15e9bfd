// Elementwise passes of the router projection and its backward.
//
// UniEP paper, "MoE workflow": the router network gives every token a score
// per expert.  Here that is logits = x . W_r (+ a per-expert bias) on the
// GroupGEMM kernel as one dense group; when the contraction is split into
// chunks for parallelism, each chunk leaves an fp32 partial and the pass
// below adds the partials in chunk order, so the result does not depend on
// scheduling.  The backward takes the score gradient in bf16 (as every other
// activation gradient of the path), which the second pass rounds.  The bias's
// gradient is the column sums of the unrounded score gradient.
#include "columns.hpp"

using moe_host::misaligned;

namespace moe {

// out[i] = part[0][i] + part[1][i] + ... (chunk order) + bias[i % period]
__global__ __launch_bounds__(256) void sum_partials_kernel(const f32x4* __restrict__ part, int S, int64_t n4,
                                                           int64_t stride4, const float* __restrict__ bias,
                                                           int period, f32x4* __restrict__ out) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (int64_t)gridDim.x * 256) {
        f32x4 acc = __builtin_nontemporal_load(part + i);
        for (int s = 1; s < S; ++s) acc += __builtin_nontemporal_load(part + s * stride4 + i);
        if (bias) acc += *(const f32x4*)(bias + (i * 4) % period);
        out[i] = acc;
    }
}

// 8 fp32 -> 8 bf16 (nearest even) per thread and step
__global__ __launch_bounds__(256) void cast_bf16_kernel(const f32x4* __restrict__ in, int64_t n8,
                                                        u32x4* __restrict__ out) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += (int64_t)gridDim.x * 256) {
        const f32x4 a = __builtin_nontemporal_load(in + 2 * i);
        const f32x4 b = __builtin_nontemporal_load(in + 2 * i + 1);
        out[i] = u32x4{pack_bf2(a[0], a[1]), pack_bf2(a[2], a[3]), pack_bf2(b[0], b[1]), pack_bf2(b[2], b[3])};
    }
}

// Column sums of d [T][E], a row of E at out for each blockIdx.y: a workgroup takes 256 columns (64 threads of 4) of
// blocks of 16 rows, a strand of 64 threads four rows of each, which are asked for together; the four strands' sums meet
// in LDS, in order.  Bound by d's bytes: 131072 x 256 takes 26.8 us with the join of its 1024 partial rows (5.0 TB/s).
__global__ __launch_bounds__(256) void bias_rows_kernel(const float* __restrict__ d, int64_t T, int E,
                                                        float* __restrict__ out) {
    constexpr int R = 4;
    __shared__ f32x4 merge[3][64];
    const int lane = threadIdx.x & 63, strand = threadIdx.x >> 6;
    const int n = (int)blockIdx.x * 256 + lane * 4;
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    if (n < E) {
        for (int64_t t0 = (int64_t)blockIdx.y * 4 * R + strand * R; t0 < T; t0 += 4 * R * (int64_t)gridDim.y) {
            f32x4 v[R];
#pragma unroll
            for (int r = 0; r < R; ++r)
                v[r] = t0 + r < T ? *(const f32x4*)(d + (t0 + r) * E + n) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int r = 0; r < R; ++r) sum += v[r];
        }
    }
    if (strand > 0) merge[strand - 1][lane] = sum;
    __syncthreads();
    if (strand == 0 && n < E) {
#pragma unroll
        for (int o = 0; o < 3; ++o) sum += merge[o][lane];
        *(f32x4*)(out + (int64_t)blockIdx.y * E + n) = sum;
    }
}

// Row blocks of bias_rows_kernel, and so partial rows: up to four workgroups a CU.  One block's sums are the gradient
// itself, so up to 32 rows, two turns of a workgroup, are left to one.
static int bias_rows(int T, int E) {
    const int64_t blocks = (E + 255) / 256;
    if (T <= 32) return 1;
    return (int)std::max<int64_t>(1, std::min<int64_t>(((int64_t)T + 15) / 16, 4 * moe_host::num_cus() / blocks));
}

static int bias_check(int T, int E) {
    if (T < 0 || E <= 0 || E > 4096) return MOE_EINVAL;
    return E % 64 ? MOE_ESHAPE : MOE_OK;
}

}  // namespace moe

namespace moe_host {

static int grid_for(int64_t items) {
    const int64_t blocks = (items + 255) / 256;
    return (int)std::min<int64_t>(blocks, (int64_t)num_cus() * 8);
}

int sum_partials(const float* part, int S, int64_t n, int64_t stride, const float* bias, int period, float* out,
                 hipStream_t s) {
    const int64_t n4 = n / 4;
    if (n4 == 0) return MOE_OK;
    moe::sum_partials_kernel<<<grid_for(n4), 256, 0, s>>>((const moe::f32x4*)part, S, n4, stride / 4, bias, period,
                                                          (moe::f32x4*)out);
    return launch_status();
}

int cast_f32_bf16(const float* in, int64_t n, uint16_t* out, hipStream_t s) {
    const int64_t n8 = n / 8;
    if (n8 == 0) return MOE_OK;
    moe::cast_bf16_kernel<<<grid_for(n8), 256, 0, s>>>((const moe::f32x4*)in, n8, (moe::u32x4*)out);
    return launch_status();
}

}  // namespace moe_host

extern "C" size_t moe_router_bias_backward_workspace_size(int T, int E) {
    using namespace moe;
    if (bias_check(T, E) != MOE_OK) return 0;
    const int rows = bias_rows(T, E);
    return rows > 1 ? (size_t)rows * E * 4 : 0;
}

extern "C" int moe_router_bias_backward(const float* dlogits, int T, int E, float* dbias, void* ws, size_t ws_bytes,
                                        moe_stream stream) {
    using namespace moe;
    const int st = bias_check(T, E);
    if (st != MOE_OK) return st;
    if (!dbias || (T > 0 && !dlogits)) return MOE_EINVAL;
    if (misaligned(dlogits) || misaligned(dbias) || misaligned(ws)) return MOE_EALIGN;
    const int rows = bias_rows(T, E);
    if (rows > 1 && (!ws || ws_bytes < moe_router_bias_backward_workspace_size(T, E))) return MOE_EWORKSPACE;
    hipStream_t s = (hipStream_t)stream;
    bias_rows_kernel<<<dim3((E + 255) / 256, rows), 256, 0, s>>>(dlogits, T, E, rows > 1 ? (float*)ws : dbias);
    const int rc = moe_host::launch_status();
    if (rc != MOE_OK || rows == 1) return rc;
    return moe_host::column_sums((const float*)ws, rows, E, E, dbias, nullptr, s);
}
