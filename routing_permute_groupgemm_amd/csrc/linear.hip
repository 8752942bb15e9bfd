// Dense product with bias, activation and residual in its epilogue, and its
// backward: the products of a block that do not go by expert (a shared expert's
// down product onto the routed experts' output, a dense feed-forward layer).
//
//   z = x . w + bias (fp32),  y = bf16(act(z) + residual),  optionally bf16(z) for the backward
//   dz = bf16(dy * act'(z)),  dx = bf16(dz . w^T),  dw = x^T . dz (fp32),  db = sum over rows of dy * act'(z) (fp32)
//
// Forward, by the sizes (linear_plan):
//   few rows   the weights' bytes are the time: linear_rows streams them (rows_stream.hpp), the contraction in chunks
//              over the workgroups where the columns alone are too few;
//   more rows  the GroupGEMM's kernel on one dense group with EPI_LINEAR, in tiles of 256 x 256, 128 x 256 or 128 x 128, or
//              128 x 128 tiles over chunks of the contraction where the tiles alone would leave most of the chip idle.
// Chunks leave fp32 partial sums, which linear_finish adds in chunk order before it does what the epilogue does.
// The backward's products are the GroupGEMM's as well; linear_slope forms dz and the partial column sums of db in
// one pass.
#include "columns.hpp"
#include "linear_tiles.hpp"
#include "rows_stream.hpp"

using moe_host::misaligned;

namespace moe {

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

// Blocks of 16*MT rows (blockIdx.y), 16*CW columns and contraction chunks.
template <int CW, int MT, int S, int W>
__global__ __launch_bounds__(64 * W) void linear_rows(LinearParams p) {
    constexpr int kCols = 16 * CW, kQuads = kCols / 4;
    __shared__ __attribute__((aligned(16))) WaveSums<1, CW, W> sums;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slabs = (p.N + kCols - 1) / kCols;
    const int chunk = (int)blockIdx.x / slabs, col0 = ((int)blockIdx.x % slabs) * kCols;
    const int row0 = (int)blockIdx.y * 16 * MT, rows = min(16 * MT, p.T - row0);
    uint32_t x_at[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) x_at[m] = (uint32_t)min(16 * m + (lane & 15), rows - 1) * (uint32_t)(p.Kd * 2);
    const uint16_t* const w[1] = {p.w};
    RowStream<1, CW, MT, S, false> r;
    // columns past the last are read as the last ones; their sums are not stored
    r.run(w, p.N, min(col0 + CW * (lane & 15), p.N - CW), p.x + (int64_t)row0 * p.Kd, x_at, rows, chunk * p.steps + wave,
          W, min((chunk + 1) * p.steps, p.Kd / 32));
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (16 * m >= rows) break;
        if (m > 0) __syncthreads();
        sums.put(r, m, wave, lane);
        __syncthreads();
        for (int i = tid; i < 16 * kQuads; i += 64 * W) {
            const int row = 16 * m + i / kQuads, c = (i % kQuads) * 4;
            if (row >= rows || col0 + c >= p.N) continue;
            const f32x4 f = sums.get(i / kQuads, c);
            if (p.part) *(f32x4*)(p.part + ((int64_t)chunk * p.T + row0 + row) * p.N + col0 + c) = f;
            else finish4(p, row0 + row, col0 + c, f);
        }
    }
}

__global__ __launch_bounds__(256) void linear_finish(LinearParams p, int chunks) {
    const int64_t n4 = (int64_t)p.T * p.N / 4, stride = n4;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (int64_t)gridDim.x * 256) {
        const f32x4* at = (const f32x4*)p.part + i;
        f32x4 f = *at;
#pragma unroll 4
        for (int c = 1; c < chunks; ++c) f += at[c * stride];
        const int64_t t = i * 4 / p.N;
        finish4(p, t, (int)(i * 4 - t * p.N), f);
    }
}

// dz = bf16(dy * act'(z)) (dz NULL: not written) and column sums of the unrounded products (part NULL: not wanted; a row
// of N for each blockIdx.y): a workgroup takes 512 columns (64 threads of 8) of blocks of 16 rows, a strand of 64 threads
// four rows of each, which are asked for together; the four strands' sums meet in LDS.  dz may be dy: a thread's rows are
// read before they are written.  Bound by its bytes (131072 x 7168 without an activation, one array read: 283 us; with
// ReLU, three arrays moved: 738), with GELU its arithmetic takes part (815).
template <bool NT>
__global__ __launch_bounds__(256) void linear_slope(const uint16_t* dy, const uint16_t* __restrict__ z, int64_t T, int N,
                                                    int act, uint16_t* dz, float* __restrict__ part) {
    constexpr int R = 4;
    __shared__ __attribute__((aligned(16))) float merge[3][512];
    const int lane = threadIdx.x & 63, strand = threadIdx.x >> 6;
    const int n = (int)blockIdx.x * 512 + lane * 8;
    float sum[8] = {};
    if (n < N) {
        for (int64_t t0 = (int64_t)blockIdx.y * 4 * R + strand * R; t0 < T; t0 += 4 * R * (int64_t)gridDim.y) {
            u32x4 d[R], v[R] = {};
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int64_t at = min(t0 + r, T - 1) * N + n;
                d[r] = NT ? __builtin_nontemporal_load((const u32x4*)(dy + at)) : *(const u32x4*)(dy + at);
                if (act != MOE_ACT_NONE)
                    v[r] = NT ? __builtin_nontemporal_load((const u32x4*)(z + at)) : *(const u32x4*)(z + at);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (t0 + r >= T) break;
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    f[i] = i & 1 ? bf_hi(d[r][i >> 1]) : bf_lo(d[r][i >> 1]);
                    if (act != MOE_ACT_NONE) f[i] *= slope(i & 1 ? bf_hi(v[r][i >> 1]) : bf_lo(v[r][i >> 1]), act);
                    sum[i] += f[i];
                }
                if (dz)
                    *(u32x4*)(dz + (t0 + r) * N + n) = u32x4{pack_bf2x(f[0], f[1]), pack_bf2x(f[2], f[3]),
                                                             pack_bf2x(f[4], f[5]), pack_bf2x(f[6], f[7])};
            }
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

// The partial rows of db (16 columns a workgroup, the first of them) and the chunks of dw, each in order, in one launch:
// 4001 x 2048 x 768 takes 60.0 us backward so, 61.1 with a launch for each.
__global__ __launch_bounds__(256) void linear_join(const float* __restrict__ db_part, int rows, int N, float* __restrict__ db,
                                                   const f32x4* __restrict__ dw_part, int chunks, int64_t n4,
                                                   f32x4* __restrict__ dw) {
    const int first = N / 16;
    if ((int)blockIdx.x < first) {
        sum_columns(db_part + 16 * blockIdx.x, rows, N, db + 16 * blockIdx.x);
        return;
    }
    const int64_t step = (int64_t)(gridDim.x - first) * 256;
    for (int64_t i = (int64_t)(blockIdx.x - first) * 256 + threadIdx.x; i < n4; i += step) {
        f32x4 acc = __builtin_nontemporal_load(dw_part + i);
        for (int c = 1; c < chunks; ++c) acc += __builtin_nontemporal_load(dw_part + c * n4 + i);
        dw[i] = acc;
    }
}

// What a product on the GroupGEMM kernel takes, in us, fitted to what it was measured to take on the MI355X.  Of 80
// products of 257 to 65536 rows by 256 to 8192 columns and contraction values, timed in every tile and number of chunks,
// what these choose was the fastest or within 5% of it for 73, within 10% for 76, and lost up to 19% for the others
// (512 x 4096 x 4096 40.7, in four chunks 34.3).  A step is 32 contraction values, `step` and `fixed` a step's and a
// tile's share.
// Tiles that have a CU to themselves (all but the 128 x 128 ones of four waves, of which a CU takes two):
static double tiles_us(int64_t n, int64_t steps, double step, double fixed) {
    const int64_t cus = moe_host::num_cus();
    return (double)((n + cus - 1) / cus) * (step * (double)steps + fixed);
}
static double shared_us(int64_t n, int64_t steps, double alone, double shared) {
    const int64_t cus = moe_host::num_cus();
    return n <= cus ? alone * (double)steps + 4.0
                    : (double)((n + 2 * cus - 1) / (2 * cus)) * (shared * (double)steps + 8.0);
}
// Partial sums of chunks (fp32), written and read, and the launch that adds them.
static double partials_us(int64_t chunks, int64_t values, double launch) {
    return chunks > 1 ? launch + (double)(chunks * values) * 8.0 / 7e6 : 0.0;
}

static int64_t tiles_of(int64_t rows, int64_t cols, int bm, int bn) {
    return ((rows + bm - 1) / bm) * ((cols + bn - 1) / bn);
}

enum : int { FORM_ROWS = 0, FORM_SMALL = TILES_SMALL, FORM_MID = TILES_MID, FORM_BIG = TILES_BIG, FORM_CHUNKS = 4 };
constexpr int kFewRows = 256;

struct LinearPlan {
    int form, chunks, steps;      // forward
    bool wide;                    // FORM_ROWS: 128 columns a workgroup, not 64
    int slope_rows;               // row blocks of linear_slope, and so partial rows of db
    bool dw_small;                // weight gradient: 128 x 128 tiles, not 256 x 256
    int dw_chunks, dw_rows;       // and its row chunks
    size_t forward_bytes, db_bytes, backward_bytes;
};

// Few rows, measured (us, one product): blocks of 64 columns and up to 64 rows, in chunks that fill the GPU once, of at
// least 8 steps.  1 x 7168 x 2048 (rows, contraction, columns): 9.6 with 8 chunks, 19 without; but a chunk's sums pass
// through memory, so products of few rows and a short contraction are not cut (1 x 2048 x 7168: 8.2, and 8.9 in two), nor
// those that fill most of the GPU (128 x 2048 x 7168: 17.3, and 22.7 in two).  128 columns, whose workgroups read the rows
// half as often, where the columns are many: 64 x 7168 x 7168 31 against 38; 128 x 4096 x 1536 15.6 against 13.7.
// 256 x 4096 x 1536 takes 18 in rows and 22 in tiles, 512 x 4096 x 1536 24 in tiles and more in rows; smaller products of
// more than 256 rows would still be faster in rows (512 x 2048 x 2048 16 against 24, 1000 x 2048 x 768 16 against 20).
static void plan_rows(LinearPlan& r, int T, int kt, int N) {
    const int64_t cus = moe_host::num_cus();
    r.form = FORM_ROWS;
    r.wide = T > 32 && N >= 4096;
    const int cols = r.wide ? 128 : 64;
    // the backward of no rows asks for a plan too
    const int64_t blocks = (int64_t)((N + cols - 1) / cols) * std::max(1, (T + 63) / 64);
    int64_t want = 1;
    if (!(T <= 16 && kt <= 64) && 5 * blocks < 4 * cus)
        want = std::max<int64_t>(1, std::min<int64_t>(cus / blocks, kt / 8));
    r.steps = (int)((kt + want - 1) / want);
    r.chunks = (kt + r.steps - 1) / r.steps;
}

static LinearPlan linear_plan(int T, int Kd, int N) {
    LinearPlan r{};
    const int64_t cus = moe_host::num_cus();
    const int kt = Kd / 32;
    if (T <= kFewRows) {
        plan_rows(r, T, kt, N);
    } else {
        r.form = FORM_BIG;
        r.chunks = 1;
        r.steps = kt;
        double best = tiles_us(tiles_of(T, N, 256, 256), kt, 0.8, 10.0);
        auto take = [&](int form, int chunks, int steps, double us) {
            if (us >= best) return;
            best = us;
            r.form = form;
            r.chunks = chunks;
            r.steps = steps;
        };
        take(FORM_MID, 1, kt, tiles_us(tiles_of(T, N, 128, 256), kt, 0.5, 9.0));
        const int64_t small = tiles_of(T, N, 128, 128);
        if (small <= cus) take(FORM_SMALL, 1, kt, tiles_us(small, kt, 0.27, 8.0));
        for (int c : {2, 3, 4, 6, 8, 12, 16}) {  // (with 5 or 10, workgroups on 240 of 256 CUs ran 10% slower than on 192)
            if (kt / c < 8) break;
            const int steps = (kt + c - 1) / c, chunks = (kt + steps - 1) / steps;
            take(FORM_CHUNKS, chunks, steps, shared_us(small * chunks, steps, 0.37, 0.56) + partials_us(chunks, (int64_t)T * N, 6.0));
        }
    }
    r.forward_bytes = r.chunks > 1 ? (size_t)r.chunks * T * N * 4 : 0;
    // up to 32 rows one row block, whose column sums are db itself: no partial rows and no launch that adds them (30 x 192
    // 5.6 us, 65 x 1536 in two launches 6.1, 64 x 1536 in one 9.8)
    const int64_t blocks = (N + 511) / 512;
    r.slope_rows = T <= 32 ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>(((int64_t)T + 15) / 16, 4 * cus / blocks));
    r.db_bytes = r.slope_rows > 1 ? round256((size_t)r.slope_rows * N * 4) : 0;
    // the weight gradient: the rows are the contraction
    const int64_t rt = std::max<int64_t>(1, ((int64_t)T + 31) / 32), out = (int64_t)Kd * N;
    int steps;
    split_steps(tiles_of(Kd, N, 256, 256), rt, &r.dw_chunks, &steps);
    double dw_best = tiles_us(tiles_of(Kd, N, 256, 256) * r.dw_chunks, steps, 0.8, 11.0) + partials_us(r.dw_chunks, out, 2.0);
    for (int c = 1; c <= 32 && (c == 1 || rt / c >= 8); ++c) {
        const int st = (int)((rt + c - 1) / c), chunks = (int)((rt + st - 1) / st);
        const double t = shared_us(tiles_of(Kd, N, 128, 128) * chunks, st, 0.45, 0.62) + partials_us(chunks, out, 2.0);
        if (t < dw_best) {
            dw_best = t;
            r.dw_small = true;
            r.dw_chunks = chunks;
            steps = st;
        }
    }
    r.dw_rows = steps * 32;
    r.backward_bytes = r.db_bytes + (r.dw_chunks > 1 ? (size_t)r.dw_chunks * Kd * N * 4 : 0);
    return r;
}

static int linear_check(int T, int Kd, int N, int act) {
    if (T < 0 || T > (1 << 30) || Kd <= 0 || N <= 0 || act < MOE_ACT_NONE || act > MOE_ACT_GELU) return MOE_EINVAL;
    if (Kd % 64 || N % 64) return MOE_ESHAPE;
    // 256 rows of an operand and the weights stay below 2 GiB (32-bit load offsets), the tiles below 2^31
    if (Kd > (1 << 21) || N > (1 << 21) || (int64_t)256 * std::max(Kd, N) * 2 >= (1ll << 31) ||
        (int64_t)Kd * N * 2 >= (1ll << 31) || (int64_t)T * std::max(Kd, N) >= (1ll << 40))
        return MOE_EINVAL;
    return MOE_OK;
}

template <int CW, int MT, int S, int W>
static int launch_linear_rows(const LinearParams& p, int chunks, hipStream_t s) {
    const dim3 grid((p.N + 16 * CW - 1) / (16 * CW) * chunks, (p.T + 16 * MT - 1) / (16 * MT));
    linear_rows<CW, MT, S, W><<<grid, 64 * W, 0, s>>>(p);
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
    switch (l.act) {
        case MOE_ACT_RELU: return launch_linear_relu(p, r.form, s);
        case MOE_ACT_SILU: return launch_linear_silu(p, r.form, s);
        case MOE_ACT_GELU: return launch_linear_gelu(p, r.form, s);
        default: return launch_linear_none(p, r.form, s);
    }
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
    else if (r.wide) rc = launch_linear_rows<8, 4, 2, 4>(p, r.chunks, s);
    else if (T <= 16) rc = launch_linear_rows<4, 1, 3, 8>(p, r.chunks, s);
    else if (T <= 32) rc = launch_linear_rows<4, 2, 2, 8>(p, r.chunks, s);
    else rc = launch_linear_rows<4, 4, 2, 8>(p, r.chunks, s);
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
    const bool rows = db && T > 0 && r.slope_rows > 1;  // partial rows of db
    const size_t need = dw && split ? r.backward_bytes : rows ? r.db_bytes : 0;
    if (need && (!ws || ws_bytes < need)) return MOE_EWORKSPACE;
    hipStream_t s = (hipStream_t)stream;
    float* db_part = (float*)ws;
    float* dw_part = (float*)((char*)ws + r.db_bytes);
    int rc;
    if (T > 0 && (db || !none)) {
        const dim3 grid((N + 511) / 512, r.slope_rows);
        // arrays that fill half of the last-level cache (256 MB) pass it by
        const bool nt = (int64_t)T * N * (none ? 2 : 4) >= (128ll << 20);
        if (nt) linear_slope<true><<<grid, 256, 0, s>>>(dy, z, T, N, act, none ? nullptr : dz, rows ? db_part : db);
        else linear_slope<false><<<grid, 256, 0, s>>>(dy, z, T, N, act, none ? nullptr : dz, rows ? db_part : db);
        rc = moe_host::launch_status();
        if (rc != MOE_OK) return rc;
    }
    if ((rows && !(dw && split)) || (db && T == 0)) {
        rc = moe_host::column_sums(db_part, rows ? r.slope_rows : 0, N, N, db, nullptr, s);
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
        const int64_t n = tiles_of(T, Kd, 128, 128), cus = moe_host::num_cus();
        const bool small = (n <= cus ? tiles_us(n, N / 32, 0.27, 8.0) : shared_us(n, N / 32, 0.0, 0.56)) <
                           tiles_us(tiles_of(T, Kd, 256, 256), N / 32, 0.82, 12.0);
        rc = small ? launch_rows_kc_small(p, n <= cus, s) : launch_rows_kc(p, EPI_BF16, s);
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
    rc = r.dw_small ? launch_wgrad_small(q, s) : launch_wgrad(q, s);
    if (rc != MOE_OK || !split) return rc;
    if (rows) {
        const int64_t n4 = (int64_t)Kd * N / 4;
        const int64_t blocks = N / 16 + std::min<int64_t>((n4 + 255) / 256, (int64_t)moe_host::num_cus() * 8);
        linear_join<<<(int)blocks, 256, 0, s>>>(db_part, r.slope_rows, N, db, (const f32x4*)dw_part, r.dw_chunks, n4,
                                               (f32x4*)dw);
        return moe_host::launch_status();
    }
    return moe_host::sum_partials(dw_part, r.dw_chunks, (int64_t)Kd * N, (int64_t)Kd * N, nullptr, N, dw, s);
}
