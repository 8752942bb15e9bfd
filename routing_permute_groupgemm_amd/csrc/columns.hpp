// Column sums over many rows in two steps: a pass leaves one fp32 partial row per
// workgroup, and column_sums adds the partial rows in a fixed order.
#pragma once

#include "moe_common.hpp"

namespace moe {

// 16 columns by a workgroup of 256 threads, 4 lanes x 4 columns by 64 strands of the rows; the strands' sums meet in LDS,
// sixteen threads add four neighbouring strands each and one adds the sixteen, in order.
__device__ __forceinline__ void sum_columns(const float* __restrict__ part, int rows, int64_t stride,
                                            float* __restrict__ out) {
    __shared__ f32x4 s_sum[64][4];
    const int lane = threadIdx.x & 3, strand = threadIdx.x >> 2;
    const float* at = part + 4 * lane;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int p = strand; p < rows; p += 64) acc += *(const f32x4*)(at + p * stride);
    s_sum[strand][lane] = acc;
    __syncthreads();
    if (strand < 16) {
        acc = s_sum[4 * strand][lane];
#pragma unroll
        for (int i = 1; i < 4; ++i) acc += s_sum[4 * strand + i][lane];
    }
    __syncthreads();
    if (strand < 16) s_sum[strand][lane] = acc;
    __syncthreads();
    if (strand == 0) {
#pragma unroll
        for (int i = 1; i < 16; ++i) acc += s_sum[i][lane];
        *(f32x4*)(out + 4 * lane) = acc;
    }
}

}  // namespace moe

namespace moe_host {

// out0[c] = sum over p of part[p][c] for c < n, and out1[c] = sum over p of part[p][n + c] (either may be NULL).
// part fp32 [rows][stride]; n a multiple of 64.  rows = 0 writes zeros.
int column_sums(const float* part, int rows, int64_t stride, int n, float* out0, float* out1, hipStream_t s);

}  // namespace moe_host
