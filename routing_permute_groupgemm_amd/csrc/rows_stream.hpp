// Products of a few rows with a bf16 weight matrix [Kd][N], N contiguous, by one
// wave: the weights pass once through registers, and every access to them is a
// whole piece of a matrix row.
//
// A wave owns 16*CW neighbouring columns.  Lane l loads columns CW*(l%16) .. +CW-1
// of the contraction rows 32*kt + 8*(l/16) + i, i = 0..7: 16 lanes cover 32*CW
// bytes of a row.  The matrix instruction wants 8 contraction values of one column
// in a lane, which is what the 8 loads hold of each of the lane's CW columns, so
// two byte permutations a register pair column i of the loads up, nothing crosses
// lanes and no LDS is needed: "column tile" t of v_mfma_f32_16x16x32_bf16 is the
// columns CW*c + t, c = 0..15.  The rows are the second operand (16 a tile, lane l:
// 8 contraction values of row l%16), so lane l ends with row l%16, and its register
// r of column tile t is column CW*(4*(l/16) + r) + t: CW neighbouring columns over
// the tiles.
//
// Rows past the last one are read as the last one again; their sums are not used.
#pragma once

#include "moe_common.hpp"

namespace moe {

template <int CW>
struct ColumnPiece;
template <>
struct ColumnPiece<4> {
    typedef u32x2 type;
};
template <>
struct ColumnPiece<8> {
    typedef u32x4 type;
};

// MATS matrices of one shape, MT tiles of 16 rows, S stages (a stage: 32
// contraction values) of which S - 1 are in flight.  NTL: the weights carry the
// non-temporal hint.  PAIR: a row is the sum of two bf16 rows (its rounded values and
// what the rounding left), the second `rest` bytes behind the first; the weights'
// operands serve both.
template <int MATS, int CW, int MT, int S, bool NTL, bool PAIR = false>
struct RowStream {
    static constexpr int kParts = PAIR ? 2 : 1;
    typedef typename ColumnPiece<CW>::type piece;
    struct Stage {
        piece w[MATS][8];
        u32x4 x[kParts][MT];
    };
    f32x4 acc[MATS][CW][MT];

    // w[q]: the matrices (the same in every lane); col: this lane's first column;
    // x_at[m]: byte offset in x of row 16*m + l%16 (or of any valid row); rows: how many there are.
    // Contraction steps first, first + step, ... below end, 32 values each.
    __device__ __forceinline__ void run(const uint16_t* const (&w)[MATS], int ld, int col, const uint16_t* x,
                                        const uint32_t (&x_at)[MT], int rows, int first, int step, int end,
                                        uint32_t rest = 0) {
        const int g = (threadIdx.x & 63) >> 4;
        const uint32_t w_at = ((uint32_t)(8 * g) * (uint32_t)ld + (uint32_t)col) * 2u;
        Stage st[S];
#pragma unroll
        for (int q = 0; q < MATS; ++q)
#pragma unroll
            for (int t = 0; t < CW; ++t)
#pragma unroll
                for (int m = 0; m < MT; ++m) acc[q][t][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        auto load = [&](Stage& s, int kt) {
#pragma unroll
            for (int q = 0; q < MATS; ++q)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const char* row = (const char*)(w[q] + (int64_t)(kt * 32 + i) * ld);
                    const piece* p = (const piece*)(row + w_at);
                    s.w[q][i] = NTL ? __builtin_nontemporal_load(p) : *p;
                }
#pragma unroll
            for (int h = 0; h < kParts; ++h)
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    if (m == 0 || 16 * m < rows)
                        s.x[h][m] = *(const u32x4*)((const char*)x + x_at[m] + ((uint32_t)(kt * 64 + 16 * g) + h * rest));
        };
        auto multiply = [&](const Stage& s) {
#pragma unroll
            for (int q = 0; q < MATS; ++q)
#pragma unroll
                for (int t = 0; t < CW; ++t) {
                    u32x4 v;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[i] = __builtin_amdgcn_perm(s.w[q][2 * i + 1][t >> 1], s.w[q][2 * i][t >> 1],
                                                     t & 1 ? 0x07060302u : 0x05040100u);
#pragma unroll
                    for (int h = 0; h < kParts; ++h)
#pragma unroll
                        for (int m = 0; m < MT; ++m)
                            if (m == 0 || 16 * m < rows)
                                acc[q][t][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                    __builtin_bit_cast(bf16x8, v), __builtin_bit_cast(bf16x8, s.x[h][m]), acc[q][t][m], 0, 0,
                                    0);
                }
        };
#pragma unroll
        for (int u = 0; u < S - 1; ++u)
            if (first + u * step < end) load(st[u], first + u * step);
        for (int kt = first; kt < end; kt += S * step) {
#pragma unroll
            for (int u = 0; u < S; ++u) {
                const int at = kt + u * step;
                if (at >= end) break;
                if (at + (S - 1) * step < end) load(st[(u + S - 1) % S], at + (S - 1) * step);
                multiply(st[u]);
            }
        }
    }
};

// The W waves' sums of one row tile, in LDS: [W][16 rows][MATS * 16 * CW columns], rows padded by 4.
template <int MATS, int CW, int W>
struct WaveSums {
    static constexpr int kCols = MATS * 16 * CW;
    static constexpr int kPitch = kCols + 4;
    float v[W][16][kPitch];

    template <int MT, int S, bool NTL, bool PAIR>
    __device__ __forceinline__ void put(const RowStream<MATS, CW, MT, S, NTL, PAIR>& r, int m, int wave, int lane) {
        const int row = lane & 15, g = lane >> 4;
#pragma unroll
        for (int q = 0; q < MATS; ++q)
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int t = 0; t < CW; t += 4)
                    *(f32x4*)&v[wave][row][q * 16 * CW + CW * (4 * g + c) + t] =
                        f32x4{r.acc[q][t][m][c], r.acc[q][t + 1][m][c], r.acc[q][t + 2][m][c], r.acc[q][t + 3][m][c]};
    }
    // 4 columns of a row, the waves W0 .. W1-1 added in order
    template <int W0 = 0, int W1 = W>
    __device__ __forceinline__ f32x4 get(int row, int col) const {
        f32x4 s = *(const f32x4*)&v[W0][row][col];
#pragma unroll
        for (int w = W0 + 1; w < W1; ++w) s += *(const f32x4*)&v[w][row][col];
        return s;
    }
};

}  // namespace moe
