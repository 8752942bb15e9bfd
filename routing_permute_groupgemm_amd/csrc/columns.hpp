// Column sums over many rows in two steps: a pass leaves one fp32 partial row per
// workgroup, and column_sums adds the partial rows in a fixed order.
#pragma once

#include "moe_common.hpp"

namespace moe_host {

// out0[c] = sum over p of part[p][c] for c < n, and out1[c] = sum over p of part[p][n + c] (either may be NULL).
// part fp32 [rows][stride]; n a multiple of 64.  rows = 0 writes zeros.
int column_sums(const float* part, int rows, int64_t stride, int n, float* out0, float* out1, hipStream_t s);

}  // namespace moe_host
