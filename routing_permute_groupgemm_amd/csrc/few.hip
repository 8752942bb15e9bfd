// A whole layer for a few tokens in two kernels: what a decode step on bf16
// weights runs instead of the routing, the permutation, two GroupGEMMs and the
// combine.
//
//   out[t] = bf16(residual[t] + sum over k ascending of gate[t,k] * y[t,k])
//   y[t,k] = h . Wd_j,   h = silu(x_t . Wg_j) * (x_t . Wu_j),   j = the k-th expert of token t, if it is local
// h is kept as two bf16 values, itself rounded and what that left (16 bits in all), so that the output's rounding is the
// only one that counts.  The down product reads so few rows that the second costs nothing beside the weights (H = 4096, F =
// 1536, 128 experts, 64 tokens 827 us without and 836 with it, 16 tokens 532 and 534), but for experts with dozens of rows
// (8 experts, 64 rows each: 144 and 155).
// Almost every byte is a weight of an expert that has a token (6*H*F bytes each), read once for every 16 rows that the
// expert has (32 or 64 where they have as many on average): the time is that of streaming them.
//
//   few_up    every workgroup routes the T tokens itself (T <= 64, so an expert's
//             tokens are a 64-bit mask and a token's row among them a popcount), then
//             takes blocks of columns of gate and up of the experts that have
//             tokens.  Its waves take the contraction's steps in turn; their sums
//             meet in LDS, in wave order.  Workgroup 0 also writes the choices, the
//             gates and the plan that the second kernel reads, and clears its counters.
//   few_down  a workgroup takes 128 columns of an expert's down product, fp32 rows in
//             the workspace; the last of a column block's workgroups to finish
//             forms the tokens' gated sums there, so no third launch is needed.
//             Which one that is does not change what is added in which order.
// A token's bits do not depend on the other tokens of the call, nor on how many there are.
#include <math.h>

#include "route_select.hpp"
#include "rows_stream.hpp"

using moe_host::misaligned;

namespace moe {

constexpr int kFewT = 64;
constexpr int kFewGroups = 512;
constexpr int kFewDownCols = 128;
constexpr int few_up_cols(bool wide) { return wide ? 128 : 64; }

// An expert with tokens: its rows row0 .. row0+rows-1 of the expert-grouped order.
struct FewExpert {
    int j, row0, rows, pad;
};

struct FewParams {
    const float* logits;
    const uint16_t* x;
    int T, E, K, e_begin, e_local;
    const uint16_t *w_gate, *w_up, *w_down;
    int H, F;
    const uint16_t* residual;
    int32_t* topk_idx;
    float* gates;
    uint16_t* out;
    // workspace
    int* n_active;
    int* arrived;       // [column blocks of the down product]
    FewExpert* active;  // [min(e_local, T*K)]
    int* pos;           // [T*K]: the pair's row, or -1
    uint16_t* h;        // [2][rows][F]: rounded to bf16, and the rests
    uint32_t h_rest;    // bytes from the one to the other
    float* y;           // [rows][H]
};

template <int EPL>
__device__ __forceinline__ void choose(const float* row, int E, int K, int lane, int& idx, float& score, float& s_max) {
    uint32_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = i * 64 + lane;
        key[i] = e < E ? score_key(row[e]) : 0u;
    }
    select_rounds<EPL>(key, K, lane, idx, score, s_max);
}

struct FewPlan {
    unsigned long long mask[kFewGroups];  // tokens of a local expert
    uint16_t expert[kFewGroups];          // the experts that have tokens, ascending
    uint16_t row0[kFewGroups];            // their first rows
    uint16_t start[kFewGroups];           // a local expert's first row
    int16_t local[kFewT * 16];            // a pair's local expert, or -1
    uint8_t token[kFewT * 16];            // a row's token
    int n_active;
};

// Routing of all tokens by this workgroup of W waves, into `s`; the workgroup `write` also writes the call's outputs
// and the plan.
template <int W>
__device__ __forceinline__ void route_few(const FewParams& p, FewPlan& s, bool write) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    for (int j = tid; j < p.e_local; j += 64 * W) s.mask[j] = 0ull;
    __syncthreads();
    for (int t = wave; t < p.T; t += W) {
        const float* row = p.logits + (int64_t)t * p.E;
        int idx = 0;
        float score = 0.0f, s_max = 0.0f;
        if (p.E <= 64) choose<1>(row, p.E, p.K, lane, idx, score, s_max);
        else if (p.E <= 128) choose<2>(row, p.E, p.K, lane, idx, score, s_max);
        else if (p.E <= 256) choose<4>(row, p.E, p.K, lane, idx, score, s_max);
        else choose<8>(row, p.E, p.K, lane, idx, score, s_max);
        if (write) {
            const float ex = lane < p.K ? expf(score - s_max) : 0.0f;
            float z = 0.0f;
            for (int k = 0; k < p.K; ++k) z += __shfl(ex, k, 64);
            if (lane < p.K) {
                p.topk_idx[t * p.K + lane] = idx;
                p.gates[t * p.K + lane] = ex / z;
            }
        }
        if (lane < p.K) {
            const int j = idx - p.e_begin;
            const bool in = j >= 0 && j < p.e_local;
            s.local[t * p.K + lane] = in ? (int16_t)j : (int16_t)-1;
            if (in) atomicOr(&s.mask[j], 1ull << t);
        }
    }
    __syncthreads();
    if (wave == 0) {  // lane l: experts 8l .. 8l+7
        int rows = 0, used = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = lane * 8 + i;
            const int n = j < p.e_local ? __popcll(s.mask[j]) : 0;
            rows += n;
            used += n > 0;
        }
        int r = rows, u = used;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int a = __shfl_up(r, o, 64), b = __shfl_up(u, o, 64);
            if (lane >= o) {
                r += a;
                u += b;
            }
        }
        if (lane == 63) s.n_active = u;
        r -= rows;
        u -= used;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = lane * 8 + i;
            const int n = j < p.e_local ? __popcll(s.mask[j]) : 0;
            if (j < p.e_local) s.start[j] = (uint16_t)r;
            if (n > 0) {
                s.expert[u] = (uint16_t)j;
                s.row0[u] = (uint16_t)r;
                if (write) p.active[u] = FewExpert{j, r, n, 0};
                ++u;
                r += n;
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < p.T * p.K; i += 64 * W) {
        const int j = s.local[i], t = i / p.K;
        int row = -1;
        if (j >= 0) {
            row = s.start[j] + __popcll(s.mask[j] & ((1ull << t) - 1ull));
            s.token[row] = (uint8_t)t;
        }
        if (write) p.pos[i] = row;
    }
    if (write) {
        if (tid == 0) *p.n_active = s.n_active;
        for (int i = tid; i < (p.H + kFewDownCols - 1) / kFewDownCols; i += 64 * W) p.arrived[i] = 0;
    }
    __syncthreads();
}

// Workgroup b runs on XCD b % 8, and each XCD takes a contiguous run of the column blocks (neighbouring blocks of an
// expert read neighbouring pieces of the same matrix rows, and the same tokens): 475 against 492 us for 64 tokens on 32
// of 256 experts.  (The down kernel did not gain from it.)
__device__ __forceinline__ int xcd_order(int b, int run) { return (b & 7) * run + (b >> 3); }

// A wave of a narrow block has 64 columns of both matrices and every W-th step of the contraction; of a wide one, 128
// columns of one matrix (the first half of the waves gate, the second up) and every W/2-th step.
template <int MT, int S, int W, bool WIDE, bool NTL>
__global__ __launch_bounds__(64 * W) void few_up(FewParams p) {
    __shared__ FewPlan plan;
    constexpr int MATS = WIDE ? 1 : 2, CW = WIDE ? 8 : 4, KW = WIDE ? W / 2 : W;
    constexpr int kCols = few_up_cols(WIDE), kQuads = kCols / 4;
    __shared__ __attribute__((aligned(16))) WaveSums<MATS, CW, W> sums;
    route_few<W>(p, plan, blockIdx.x == 0);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slabs = (p.F + kCols - 1) / kCols;
    const int total = plan.n_active * slabs, run = (total + 7) / 8;
    for (int b = blockIdx.x; b < 8 * run; b += gridDim.x) {
        const int id = xcd_order(b, run);
        if (id >= total) continue;
        const int a = id / slabs, col0 = (id - a * slabs) * kCols;
        const int j = __builtin_amdgcn_readfirstlane((int)plan.expert[a]);
        const int64_t at = (int64_t)j * p.H * p.F;
        const uint16_t* w[MATS];
        w[0] = (WIDE && wave >= KW ? p.w_up : p.w_gate) + at;
        if constexpr (!WIDE) w[1] = p.w_up + at;
        const int end = __builtin_amdgcn_readfirstlane((int)plan.row0[a] + __popcll(plan.mask[j]));
        for (int row0 = __builtin_amdgcn_readfirstlane((int)plan.row0[a]); row0 < end; row0 += 16 * MT) {
            const int rows = min(16 * MT, end - row0);
            uint32_t x_at[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m)
                x_at[m] = (uint32_t)plan.token[row0 + min(16 * m + (lane & 15), rows - 1)] * (uint32_t)(p.H * 2);
            RowStream<MATS, CW, MT, S, NTL> r;
            // columns past the last are read as the last ones; their sums are not stored
            r.run(w, p.F, min(col0 + CW * (lane & 15), p.F - CW), p.x, x_at, rows, wave % KW, KW, p.H / 32);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (16 * m >= rows) break;
                __syncthreads();  // the sums of the block before are read
                sums.put(r, m, wave, lane);
                __syncthreads();
                for (int i = tid; i < 16 * kQuads; i += 64 * W) {
                    const int row = i / kQuads, c = (i % kQuads) * 4;
                    if (16 * m + row >= rows || col0 + c >= p.F) continue;
                    f32x4 g, u;
                    if constexpr (WIDE) {
                        g = sums.template get<0, KW>(row, c);
                        u = sums.template get<KW, W>(row, c);
                    } else {
                        g = sums.get(row, c);
                        u = sums.get(row, 64 + c);
                    }
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = silu_f(g[e]) * u[e];
                    const u32x2 hi = {pack_bf2x(v[0], v[1]), pack_bf2x(v[2], v[3])};
                    const float top[4] = {bf_lo(hi[0]), bf_hi(hi[0]), bf_lo(hi[1]), bf_hi(hi[1])};
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = fabsf(top[e]) < __builtin_inff() ? v[e] - top[e] : 0.0f;
                    uint16_t* to = p.h + (int64_t)(row0 + 16 * m + row) * p.F + col0 + c;
                    *(u32x2*)to = hi;
                    *(u32x2*)((char*)to + p.h_rest) = u32x2{pack_bf2x(v[0], v[1]), pack_bf2x(v[2], v[3])};
                }
            }
        }
    }
}

// fp32 rows that workgroups on other XCDs read within the same launch: accesses of the whole GPU's scope, which an
// XCD's own L2 does not keep back.  Fences over it would write back and drop all of that L2 instead: with one a
// workgroup the down kernel took 292 us for 23 tokens
// (H = 2048, F = 768, 128 experts, top 8), with one that a single thread issues 127, and 64 without.
__device__ __forceinline__ void store_shared(float* p, f32x4 v) {
    const u32x4 u = __builtin_bit_cast(u32x4, v);
    unsigned long long* q = (unsigned long long*)p;
    __hip_atomic_store(q, (unsigned long long)u[1] << 32 | u[0], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(q + 1, (unsigned long long)u[3] << 32 | u[2], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f32x4 load_shared(const float* p) {
    unsigned long long* q = (unsigned long long*)p;
    const unsigned long long a = __hip_atomic_load(q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const unsigned long long b = __hip_atomic_load(q + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return __builtin_bit_cast(f32x4, u32x4{(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)});
}

// The gated sums of columns col0 .. col0+127 of every token.
template <int W>
__device__ __forceinline__ void combine_few(const FewParams& p, int col0) {
    const int cols = min(kFewDownCols, p.H - col0) / 4;
    for (int i = threadIdx.x; i < p.T * (kFewDownCols / 4); i += 64 * W) {
        const int t = i / (kFewDownCols / 4), c = i % (kFewDownCols / 4);
        if (c >= cols) continue;
        const int n = col0 + 4 * c;
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int k = 0; k < p.K; ++k) {
            const int r = p.pos[t * p.K + k];
            if (r >= 0) acc += p.gates[t * p.K + k] * load_shared(p.y + (int64_t)r * p.H + n);
        }
        if (p.residual) {
            const u32x2 v = *(const u32x2*)(p.residual + (int64_t)t * p.H + n);
            acc += f32x4{bf_lo(v[0]), bf_hi(v[0]), bf_lo(v[1]), bf_hi(v[1])};
        }
        *(u32x2*)(p.out + (int64_t)t * p.H + n) = u32x2{pack_bf2x(acc[0], acc[1]), pack_bf2x(acc[2], acc[3])};
    }
}

// A pass over the rows of expert e and the columns col0 .. col0+127 of its down product, into p.y; PAIR: both values of h.
// Of a pass without the second, the sums that the pass with both left finite stay.  Whether a sum was not finite -> far.
template <int MT, int S, int W, bool NTL, bool PAIR>
__device__ __forceinline__ void down_rows(const FewParams& p, const FewExpert& e, int col0, WaveSums<1, 8, W>& sums,
                                          bool& far) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = __builtin_amdgcn_readfirstlane(e.j);
    const int end = __builtin_amdgcn_readfirstlane(e.row0 + e.rows);
    const uint16_t* const w[1] = {p.w_down + (int64_t)j * p.F * p.H};
    for (int row0 = __builtin_amdgcn_readfirstlane(e.row0); row0 < end; row0 += 16 * MT) {
        const int rows = min(16 * MT, end - row0);
        uint32_t x_at[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m)
            x_at[m] = (uint32_t)(row0 + min(16 * m + (lane & 15), rows - 1)) * (uint32_t)(p.F * 2);
        RowStream<1, 8, MT, S, NTL, PAIR> r;
        // columns past the last are read as the last ones; their sums are not stored
        r.run(w, p.H, min(col0 + 8 * (lane & 15), p.H - 8), p.h, x_at, rows, wave, W, p.F / 32, p.h_rest);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if (16 * m >= rows) break;
            __syncthreads();  // the sums of the block before are read
            sums.put(r, m, wave, lane);
            __syncthreads();
            for (int i = tid; i < 512; i += 64 * W) {
                const int row = i >> 5, c = (i & 31) * 4;
                if (16 * m + row >= rows || col0 + c >= p.H) continue;
                float* at = p.y + (int64_t)(row0 + 16 * m + row) * p.H + col0 + c;
                f32x4 v = sums.get(row, c);
                if constexpr (PAIR) {
                    far |= !(fabsf(v[0]) + fabsf(v[1]) + fabsf(v[2]) + fabsf(v[3]) < __builtin_inff());
                } else {
                    const f32x4 u = load_shared(at);
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = fabsf(u[k]) < __builtin_inff() ? u[k] : v[k];
                }
                store_shared(at, v);
            }
        }
    }
}

template <int MT, int S, int W, bool NTL>
__global__ __launch_bounds__(64 * W) void few_down(FewParams p) {
    __shared__ __attribute__((aligned(16))) WaveSums<1, 8, W> sums;
    __shared__ int s_last, s_far;
    const int tid = threadIdx.x;
    const int slabs = (p.H + kFewDownCols - 1) / kFewDownCols;
    const int n_active = *p.n_active;
    const int a = (int)blockIdx.x / slabs, slab = (int)blockIdx.x - a * slabs, col0 = slab * kFewDownCols;
    if (a >= n_active) {
        // no pair is local: the sums are empty
        if (n_active == 0 && a == 0) combine_few<W>(p, col0);
        return;
    }
    if (tid == 0) s_far = 0;  // an expert has a row, and its pass a barrier before the flag is set
    const FewExpert e = p.active[a];
    bool far = false;
    down_rows<MT, S, W, NTL, true>(p, e, col0, sums, far);
    if (far) s_far = 1;
    // The last of the column block's workgroups to count itself finds every other's rows in memory: a wave's stores
    // have arrived there when its count of outstanding ones is 0, all waves have when the barrier is passed, and only
    // then does the workgroup count itself.  The last one's loads are issued after it has the full count.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    // An infinite weight times a rest that is 0 or of the other sign is a NaN where the product with h is an infinity:
    // sums that are not finite are taken again from the rounded values alone.  Looking for them costs what a barrier's flag
    // does (64 tokens on the sizes B and C below: 237 us without and 240 with it, 446 to 451 and 446 to 453).
    if (s_far) {
        down_rows<MT, S, W, NTL, false>(p, e, col0, sums, far);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
    }
    if (tid == 0) s_last = __hip_atomic_fetch_add(p.arrived + slab, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == n_active - 1;
    __syncthreads();
    if (s_last) combine_few<W>(p, col0);
}

struct FewSizes {
    size_t arrived, active, pos, h, y, total;
};
static size_t up256(size_t b) { return (b + 255) / 256 * 256; }

static FewSizes few_sizes(int T, int K, int e_local, int H, int F) {
    const size_t rows = (size_t)T * std::min(K, e_local);
    FewSizes s{};
    s.arrived = 256;
    s.active = s.arrived + up256((size_t)(H + kFewDownCols - 1) / kFewDownCols * 4);
    s.pos = s.active + up256(std::min<size_t>(e_local, rows) * sizeof(FewExpert));
    s.h = s.pos + up256((size_t)T * K * 4);
    s.y = s.h + up256(rows * F * 4);
    s.total = s.y + up256(rows * H * 4);
    return s;
}

static int few_check(int T, int E, int K, int e_local, int H, int F) {
    if (T < 0 || T > kFewT || E < 1 || E > 512 || K < 1 || K > 16 || e_local < 0 || e_local > kFewGroups || H <= 0 ||
        F <= 0)
        return MOE_EINVAL;
    if (K > E || H % 64 || F % 64) return MOE_ESHAPE;
    if ((int64_t)H * F * 2 >= (1ll << 31) || H > 65536 || F > 65536) return MOE_EINVAL;
    return MOE_OK;
}

// The weights that the tokens can touch would fill half of the last-level cache (256 MB) or more.
static bool few_stream(const FewParams& p) {
    return (int64_t)std::min(p.e_local, p.T * p.K) * 6 * p.H * p.F >= (128ll << 20);
}

template <int MT, int S, int W, bool WIDE>
static int launch_few_up(const FewParams& p, int per_cu, hipStream_t s) {
    const int cols = few_up_cols(WIDE), experts = std::min(p.e_local, p.T * p.K);
    const unsigned grid = (unsigned)std::max<int64_t>(
        1, std::min<int64_t>((int64_t)experts * ((p.F + cols - 1) / cols), per_cu * moe_host::num_cus()));
    if (few_stream(p)) few_up<MT, S, W, WIDE, true><<<grid, 64 * W, 0, s>>>(p);
    else few_up<MT, S, W, WIDE, false><<<grid, 64 * W, 0, s>>>(p);
    return moe_host::launch_status();
}

template <int MT, int S, int W>
static int launch_few_down(const FewParams& p, hipStream_t s) {
    const int experts = std::max(1, std::min(p.e_local, p.T * p.K));
    const unsigned grid = (unsigned)experts * ((p.H + kFewDownCols - 1) / kFewDownCols);
    if (few_stream(p)) few_down<MT, S, W, true><<<grid, 64 * W, 0, s>>>(p);
    else few_down<MT, S, W, false><<<grid, 64 * W, 0, s>>>(p);
    return moe_host::launch_status();
}

// Row tiles a pass over an expert's weights (MT), stages (S) and the width of gate and up's blocks, from the sizes; the
// numbers are us a call.  A: H = 4096, F = 1536, 128 experts, B: H = 2048, F = 768, 128 experts, C: H = 7168, F = 2048, 32 of
// 256 experts, top 8 each; D: A with 8 experts, all of them chosen.
//   waves Four share a contraction in every form (a wide block's eight are four a matrix), so that a token's sums, added in
//         wave order, do not depend on how many others there are.  Eight would be 6 to 12% faster where the rows' loads count
//         (D, 16 tokens: 78 against 83; D, top 2, 64 tokens: 86 against 96), and slower elsewhere (B, 64: 268 against 244).
//   MT    one tile of 16 rows: an expert with more takes another pass over its weights, which is rare while T*K/E, the
//         rows that it has on average, are few (C, 64 tokens: 457, and 589 with four tiles, whose sums cost the registers
//         of loads in flight; A with 16 experts, top 4, 24 tokens: 119, and 132 with two).  From 8 on two (the same, 64
//         tokens: 171, over 198 with four; 48 tokens: 159, 176 with one), from 32 on four (D, 64 tokens: 154, 278 with
//         one).
//   width A wide block reads pieces of 256 bytes of a matrix row, a narrow one of 128, but there are half as many.  With one
//         a CU and up to a CU's worth they gain (A, 2 tokens: 115 against 135; C, 8: 147 against 162), and where there are
//         so many that an uneven end does not count (A, 64 tokens: 821 against 875; B, 64: 240 against 260; C, 64: 457
//         against 481), not with few (A, one token: 90 against 68), nor with a few more than CUs (A, 4 tokens: 211 against
//         199).  How many experts will have a token is taken from a uniform router.
//   narrow: S = 3 with at most one workgroup a CU (A, one token: 67.8, and 70.6 with 2) and for T > 32, else 2 (A, 4 tokens
//         200 against 205).
//   wide: two workgroups a CU and S = 2 (A, 16 tokens: 534, and 540 in the other form), from T > 32 one, which routes
//         once, and S = 4 (C, 64 tokens: 457, and 468).
static int launch_few(const FewParams& p, hipStream_t s) {
    const int rows = p.T * p.K / p.E, cus = moe_host::num_cus();
    int rc;
    if (rows >= 32 && p.T > 32) {
        rc = launch_few_up<4, 2, 4, false>(p, 4, s);
        return rc != MOE_OK ? rc : launch_few_down<4, 2, 4>(p, s);
    }
    if (rows >= 8 && p.T > 16) {
        rc = launch_few_up<2, 2, 4, false>(p, 4, s);
        return rc != MOE_OK ? rc : launch_few_down<2, 2, 4>(p, s);
    }
    const double active = p.e_local * (1.0 - pow(1.0 - (double)p.K / p.E, p.T));
    const double blocks = active * ((p.F + 127) / 128);
    const bool wide = rows < 8 && ((blocks >= 0.4 * cus && blocks <= 1.03 * cus) || blocks >= 1.7 * cus);
    if (wide) rc = p.T > 32 ? launch_few_up<1, 4, 8, true>(p, 1, s) : launch_few_up<1, 2, 8, true>(p, 2, s);
    else if (rows >= 8 || p.T > 32 || std::min(p.e_local, p.T * p.K) * (p.F / 64) <= cus)
        rc = launch_few_up<1, 3, 4, false>(p, 3, s);
    else rc = launch_few_up<1, 2, 4, false>(p, 4, s);
    return rc != MOE_OK ? rc : launch_few_down<1, 3, 4>(p, s);
}

}  // namespace moe

extern "C" size_t moe_layer_few_workspace_size(int T, int K, int e_local, int H, int F) {
    using namespace moe;
    if (few_check(T, 512, K, e_local, H, F) != MOE_OK || T == 0) return 0;
    return few_sizes(T, K, e_local, H, F).total;
}

extern "C" int moe_layer_few(const float* logits, const moe_bf16* x, int T, int E, int K, int e_begin, int e_local,
                             const moe_bf16* w_gate, const moe_bf16* w_up, const moe_bf16* w_down, int H, int F,
                             const moe_bf16* residual, int32_t* topk_idx, float* gates, moe_bf16* out, void* ws,
                             size_t ws_bytes, moe_stream stream) {
    using namespace moe;
    const int rc = few_check(T, E, K, e_local, H, F);
    if (rc != MOE_OK) return rc;
    if (e_begin < 0 || e_begin > E - e_local) return MOE_EINVAL;
    if (T == 0) return MOE_OK;
    if (!logits || !topk_idx || !gates || !out) return MOE_EINVAL;
    if (e_local > 0 && (!x || !w_gate || !w_up || !w_down)) return MOE_EINVAL;
    if (misaligned(logits) || misaligned(x) || misaligned(w_gate) || misaligned(w_up) || misaligned(w_down) ||
        misaligned(residual) || misaligned(topk_idx) || misaligned(gates) || misaligned(out) || misaligned(ws))
        return MOE_EALIGN;
    const FewSizes z = few_sizes(T, K, e_local, H, F);
    if (!ws || ws_bytes < z.total) return MOE_EWORKSPACE;
    char* b = (char*)ws;
    FewParams p{};
    p.logits = logits;
    p.x = x;
    p.T = T;
    p.E = E;
    p.K = K;
    p.e_begin = e_begin;
    p.e_local = e_local;
    p.w_gate = w_gate;
    p.w_up = w_up;
    p.w_down = w_down;
    p.H = H;
    p.F = F;
    p.residual = residual;
    p.topk_idx = topk_idx;
    p.gates = gates;
    p.out = out;
    p.n_active = (int*)b;
    p.arrived = (int*)(b + z.arrived);
    p.active = (FewExpert*)(b + z.active);
    p.pos = (int*)(b + z.pos);
    p.h = (uint16_t*)(b + z.h);
    p.h_rest = (uint32_t)(T * std::min(K, e_local) * F * 2);
    p.y = (float*)(b + z.y);
    return launch_few(p, (hipStream_t)stream);
}
