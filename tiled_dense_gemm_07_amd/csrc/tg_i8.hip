// Entry points of the 8-bit integer path: quantisation, product, and both in
// one call.  Arguments are checked before any HIP call; the kernel is chosen
// by sizes and alignment.
#include <hip/hip_runtime.h>

#include <stdio.h>

#include "tg_host.h"
#include "tg_kernel_i8.h"
#include "tg_kernel_i8_gemv.h"
#include "tg_kernel_quant.h"

namespace {

using tg::ceil_div;
using tg::kMaxDim;
using tg::overlap;
using tg::span;
using tg::span1;

// Kernel for rows of K elements: a row to one wave, or to a workgroup of four,
// eight or sixteen, the fewest threads whose registers hold it (bf16, 8192
// rows: K = 1024 5.3 us with two chunks a lane of one wave, 8.6 with one chunk a
// thread of four; K = 4096 16.8 with two of four waves, 17.7 with one of eight;
// K = 8192 30.7 with two of eight, 34.2 with one of sixteen).  ODD: 16-bit rows
// of an odd length.
template <int DT, bool ODD>
const void* quant_kernel(int64_t K, int* threads, int* rows)
{
    *threads = 256;
    *rows = K <= 2048 ? 4 : 1;
    if (K <= 512)
        return (const void*)&tg::quant_i8_kernel<DT, 256, 64, 1, ODD>;
    if (K <= 1024)
        return (const void*)&tg::quant_i8_kernel<DT, 256, 64, 2, ODD>;
    if (K <= 2048)
        return (const void*)&tg::quant_i8_kernel<DT, 256, 64, 4, ODD>;
    if (K <= 4096)
        return (const void*)&tg::quant_i8_kernel<DT, 256, 256, 2, ODD>;
    *threads = 512;
    if (K <= 8192)
        return (const void*)&tg::quant_i8_kernel<DT, 512, 512, 2, ODD>;
    *threads = 1024;
    if (K <= 32768)
        return (const void*)&tg::quant_i8_kernel<DT, 1024, 1024, 4, ODD>;
    return (const void*)&tg::quant_i8_kernel<DT, 1024, 1024, 0, ODD>;
}

tg_status launch_quant(const tg::QuantParams& p, int dtype, hipStream_t stream)
{
    int threads, rows;
    const bool odd = p.K % 2 != 0;
    const void* k;
    if (dtype == TG_F32)
        k = quant_kernel<tg::DT_F32, false>(p.K, &threads, &rows);
    else if (dtype == TG_F16)
        k = odd ? quant_kernel<tg::DT_F16, true>(p.K, &threads, &rows)
                : quant_kernel<tg::DT_F16, false>(p.K, &threads, &rows);
    else
        k = odd ? quant_kernel<tg::DT_BF16, true>(p.K, &threads, &rows)
                : quant_kernel<tg::DT_BF16, false>(p.K, &threads, &rows);
    tg::QuantParams q = p;
    int64_t grid = ceil_div(p.M, rows);
    q.first = (tg::u32)grid;
    if (p.N > 0) {
        q.rows = 4 * threads / (p.kq / 16);
        q.rows = q.rows < 1 ? 1 : q.rows;
        grid += ceil_div(p.N, q.rows);
    }
    return tg::launch_kernel(k, grid, 1, threads, &q, stream, "quant_i8");
}

constexpr int64_t kMaxStride = kMaxDim / 256;  // of A and W: a tile's offsets fit 31 bits

tg_status check_dims(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > tg::kMaxI8K)
        return TG_ERR_BAD_SHAPE;
    return TG_OK;
}

// The LDS-DMA kernels, and what one costs on this card in microseconds with
// its weights from HBM: t0 + strips of 128 k times `one` when every workgroup
// has a compute unit to itself, else times `full` for each round of 256 per_cu
// workgroups.  Fitted to 150 shapes (M 17 to 8192, N and K 1000 to 8192, odd
// ones among them): within 10 to 15% on average, and the choice by it 4% on
// average above the fastest kernel of the set (33% at most, on 5 us calls).
struct I8Tile {
    const char* name;
    const void* kernel[3];  // by C's type
    int bm, bn, threads, per_cu;
    float t0, one, full;
};

#define TG_I8_TILE(BM, BN, BK, WGM, WGN, NS, OCC, PER_CU, T0, ONE, FULL)                   \
    {                                                                                      \
        "i8_" #BM "x" #BN "x" #BK "_w" #WGM "x" #WGN "_s" #NS "_dma",                      \
            {(const void*)&tg::i8_dma_kernel<tg::DT_F32, BM, BN, BK, WGM, WGN, NS, OCC>,   \
             (const void*)&tg::i8_dma_kernel<tg::DT_F16, BM, BN, BK, WGM, WGN, NS, OCC>,   \
             (const void*)&tg::i8_dma_kernel<tg::DT_BF16, BM, BN, BK, WGM, WGN, NS, OCC>}, \
            BM, BN, WGM* WGN * 64, PER_CU, T0, ONE, FULL                                   \
    }
// Kernels for any layout.  Fitted to 156 shapes of odd K (M 17 to 4096): the
// choice is 0.2% on average above the fastest of the three (15% at most).
#define TG_I8_ANY(BM, BN, PD, T0, ROUND)                                       \
    {                                                                          \
        "i8_any_" #BM "x" #BN,                                                 \
            {(const void*)&tg::i8_any_kernel<tg::DT_F32, BM, BN, PD>,          \
             (const void*)&tg::i8_any_kernel<tg::DT_F16, BM, BN, PD>,          \
             (const void*)&tg::i8_any_kernel<tg::DT_BF16, BM, BN, PD>},        \
            BM, BN, 256, 1, T0, ROUND, ROUND                                   \
    }
const I8Tile kAny[] = {
    TG_I8_ANY(64, 64, 2, 3.97f, 0.490f),
    TG_I8_ANY(64, 128, 1, 5.11f, 0.687f),
    TG_I8_ANY(128, 128, 1, 6.84f, 0.970f),
};

const I8Tile kTiles[] = {
    TG_I8_TILE(32, 64, 256, 1, 2, 4, 1, 1, 3.68f, 0.182f, 0.261f),
    TG_I8_TILE(64, 64, 128, 2, 2, 5, 2, 2, 3.26f, 0.230f, 0.498f),
    TG_I8_TILE(128, 64, 128, 4, 2, 6, 2, 1, 4.27f, 0.273f, 0.893f),
    TG_I8_TILE(128, 128, 128, 2, 4, 4, 2, 1, 3.86f, 0.427f, 0.694f),
    TG_I8_TILE(128, 128, 128, 2, 2, 2, 2, 2, 3.53f, 0.738f, 1.144f),
    TG_I8_TILE(256, 256, 128, 2, 4, 2, 2, 1, 6.00f, 1.250f, 1.820f),
};

float tile_cost(const I8Tile& t, int64_t M, int64_t N, int64_t K)
{
    const int64_t tiles = ceil_div(M, t.bm) * ceil_div(N, t.bn);
    return t.t0 + (float)ceil_div(K, 128) *
                      (tiles <= 256 ? t.one : t.full * (float)ceil_div(tiles, 256 * t.per_cu));
}

// Rows of W (1), or of A or both (2), that do not start at dwords.
int shift_i8(const void* A, int64_t lda, const void* W, int64_t ldw)
{
    const auto off = [](const void* p, int64_t ld) {
        return (((uintptr_t)p | (uint64_t)ld) & 3) != 0;
    };
    return off(A, lda) ? 2 : (off(W, ldw) ? 1 : 0);
}

// The streaming kernel: 16 tokens to a workgroup while every workgroup has a CU
// to itself, else 32, and its cost, likewise: a CU's workgroups share its path to
// L2 and HBM, so rounds of 256 workgroups add up.  Fitted to 84 shapes of 17 to
// 128 tokens, N and K from 1000 to 14336, and 99 with odd K.  Shifting A as well
// leaves registers for one workgroup of 32 tokens on a CU, which gains nothing
// (32 x 4096 x 4095: 14.0 us and 15.5 with 16; 32 x 5120 x 5119: 31.0 and 26.3).
struct I8Stream {
    int tokens;
    float cost;
};

I8Stream stream_i8(int64_t M, int64_t N, int64_t K, int shift)
{
    static const float kPerK[3][2] = {{7.3e-4f, 1.16e-3f}, {1.2e-3f, 1.75e-3f}, {1.5e-3f, 0.0f}};
    const int64_t rows = ceil_div(N, 16);
    const int64_t r16 = ceil_div(ceil_div(M, 16) * rows, 256);
    if (M <= 16 || r16 <= 1 || shift == 2)
        return {16, 3.0f + kPerK[shift][0] * (float)(K * r16)};
    return {32, 2.8f + kPerK[shift][1] * (float)(K * ceil_div(ceil_div(M, 32) * rows, 256))};
}

struct I8Pick {
    const I8Tile* tile;  // NULL: the streaming kernel
    int tokens;          // its workgroup's
    float cost;
    int64_t m1, n1;  // of the first launch; a second one takes what is left of M or N
};

// Up to 16 tokens: the streaming kernel (M = 1, 8192 x 8192: 14.6 us, and 18.4
// for the best tile kernel; M = 16: 17.3 and 19.0).  Up to 128: whichever costs
// less (M = 32, 4096 x 4096: 8.5 us and 11.2; M = 32, 8192 x 8192: 24.6 and
// 19.9; over the 84 shapes the choice is 0.8% slower than the best of all, 13%
// at most).  Above: the cheapest tile.
// Rows that do not start at 16-byte boundaries, or K % 16 != 0, leave the
// streaming kernel, which takes any address (M = 32, 4096 x 4095, levels of
// linear_i8: 11.4 us, and 24.8 with tiles; 64 x 8192 x 8191: 57.5 and 47), and
// the tiles for any layout (256 x 4096 x 4095: 23.2 us with 64 x 64, 30.4 with 64
// x 128; 512 x 4096 x 4095: 34.8 and 29.0; 4096 x 4096 x 4095: 127 with 128 x
// 128, 174 with 64 x 128).
// Where the last round of 256 x 256 tiles is less than half full, the rounds before
// it and, in a second launch, whatever is best for the rows or columns left, if
// that costs a tenth less (4096 x 4224 x 4096: 68 us, 90 in one launch; 4096 x
// 4097 x 1024: 31 and 38; 6000 x 6000 x 2000: 90 and 99).  Not for the smaller
// tiles, whose last workgroups find the paths to L2 free (1088 x 4096 x 4096 with
// 128 x 128: 30 us, 27.5 in one launch).
I8Pick pick_i8(int64_t M, int64_t N, int64_t K, bool aligned, int shift, bool one_launch = false)
{
    const I8Stream s = stream_i8(M, N, K, shift);
    I8Pick p{nullptr, s.tokens, s.cost, M, N};
    if (M <= 16)
        return p;
    if (M > 128)
        p.cost = 1e30f;
    const auto take = [&](const I8Tile& t, float cost, int64_t m1, int64_t n1) {
        if (cost < p.cost)
            p = {&t, 0, cost, m1, n1};
    };
    const auto consider = [&](const I8Tile& t) {
        take(t, tile_cost(t, M, N, K), M, N);
        const int64_t tm = ceil_div(M, t.bm), tn = ceil_div(N, t.bn), round = 256 * t.per_cu;
        const int64_t left = tm * tn % round, whole = tm * tn - left;
        if (one_launch || t.bm < 256 || whole == 0 || left == 0 || 2 * left >= round)
            return;
        const int64_t n1 = whole / tm * t.bn, m1 = whole / tn * t.bm;
        if (n1 > 0)
            take(t, 1.1f * (tile_cost(t, M, n1, K) +
                            pick_i8(M, N - n1, K, aligned, shift, true).cost), M, n1);
        if (m1 > 0)
            take(t, 1.1f * (tile_cost(t, m1, N, K) +
                            pick_i8(M - m1, N, K, aligned, shift, true).cost), m1, N);
    };
    if (aligned)
        for (const I8Tile& t : kTiles)
            consider(t);
    else
        for (const I8Tile& t : kAny)
            consider(t);
    return p;
}

// Rows that the LDS-DMA copies can take: whole 16-byte chunks at 16-byte
// boundaries.
bool dma_rows(const void* p, int64_t ld) { return ((uintptr_t)p & 15) == 0 && ld % 16 == 0; }

tg_status launch_pick(tg::I8Params p, const I8Pick& k, int shift, hipStream_t stream)
{
    if (!k.tile) {
        static const void* const kernels[3][2] = {
            {(const void*)&tg::i8_gemv_kernel<1, 8, 0>, (const void*)&tg::i8_gemv_kernel<2, 8, 0>},
            {(const void*)&tg::i8_gemv_kernel<1, 8, 1>, (const void*)&tg::i8_gemv_kernel<2, 8, 1>},
            {(const void*)&tg::i8_gemv_kernel<1, 8, 2>, nullptr}};
        const int mt = k.tokens / 16;
        return tg::launch_kernel(kernels[shift][mt - 1], ceil_div(p.N, 16), ceil_div(p.M, k.tokens),
                                 512, &p, stream, "i8_gemv", 8 * mt * 1024);
    }
    // Tile order: patches of 4 tile rows, as the 16-bit kernels' largest tiles.
    const int es = tg::dtype_size(p.dt_out);
    p.group_m = tg::swizzle_override() > 0 ? tg::swizzle_override() : 4;
    p.tiles_m = (int)ceil_div(p.M, k.tile->bm);
    p.tiles_n = (int)ceil_div(p.N, k.tile->bn);
    p.c_vec = ((uintptr_t)p.C & 15) == 0 && p.ldc * es % 16 == 0 && p.N * es % 16 == 0 &&
              32 * p.ldc * es <= kMaxDim;
    return tg::launch_kernel(k.tile->kernel[p.dt_out], (int64_t)p.tiles_m * p.tiles_n, 1,
                             k.tile->threads, &p, stream, k.tile->name);
}

tg_status launch_i8(tg::I8Params p, hipStream_t stream)
{
    p.stamps = tg::clock_stamps();
    const bool aligned = p.K > 0 && p.K % 16 == 0 && dma_rows(p.A, p.lda) && dma_rows(p.W, p.ldw);
    const int shift = shift_i8(p.A, p.lda, p.W, p.ldw);
    const I8Pick k = pick_i8(p.M, p.N, p.K, aligned, shift);
    tg::I8Params rest = p;
    p.M = (int)k.m1;
    p.N = (int)k.n1;
    if (tg_status st = launch_pick(p, k, shift, stream))
        return st;
    if (rest.M == p.M && rest.N == p.N)
        return TG_OK;
    const int64_t m = rest.M == p.M ? 0 : p.M, n = rest.N == p.N ? 0 : p.N;
    rest.M -= (int)m;
    rest.N -= (int)n;
    rest.A += m * p.lda;
    rest.sa += m;
    rest.W += n * p.ldw;
    rest.sw += n;
    rest.bias = p.bias ? p.bias + n : nullptr;
    rest.C = (char*)p.C + (m * p.ldc + n) * tg::dtype_size(p.dt_out);
    rest.stamps = nullptr;  // the record is the first launch's
    return launch_pick(rest, pick_i8(rest.M, rest.N, rest.K, aligned, shift, true), shift, stream);
}

// tg_linear_i8 with K % 16 != 0: whether W's rows are copied to 16-byte
// boundaries, for the LDS-DMA tiles, by the launch that quantises.  Measured
// with the copy and without, both launches: 256 x 1024 x 4095 15.8 us and 20.3,
// 1000 x 4096 x 4095 29.1 and 40.1, 4096 x 4096 x 4095 73.0 and 118, 64 x 4096 x
// 4095 18.3 and 18.9, 256 x 8192 x 1023 15.3 and 13.4; by this rule 0.4% above
// the better of the two on average over 86 shapes (7% at most).
bool pack_linear(int64_t M, int64_t N, int64_t K)
{
    if (K % 16 == 0 || K < 16 || M <= 16)
        return false;
    const float copy = 1.5f + (float)N * (float)K / 3e6f;
    return pick_i8(M, N, ceil_div(K, 16) * 16, true, 0).cost + copy <
           pick_i8(M, N, K, false, 1).cost;
}

// tg_linear_i8 in one launch: up to 8 tokens (a wave or more to a row), whose
// quantisation in every workgroup takes less than a launch of its own would.
// Measured with both launches and with one, N = 1024 to 8192: 8 x 1024 5.7 us
// and 3.9, 8 x 2048 6.2 and 5.4, 4 x 4096 7.6 and 7.3, 8 x 4096 7.8 and 9.7, 2
// x 8192 16.5 and 16.5, 4 x 8192 16.7 and 19.9; rows count as their power of
// two.
bool fused_linear(int64_t M, int64_t K)
{
    const int64_t rows = M <= 1 ? 1 : (M <= 2 ? 2 : (M <= 4 ? 4 : 8));
    return M <= 8 && K > 0 && rows * K <= 16384;
}

tg_status launch_fused(const tg::I8Params& p, int dtype, const void* X, int64_t ldx,
                       hipStream_t stream)
{
    tg::I8LinearParams l{p, {X, ldx}};
    l.p.stamps = tg::clock_stamps();
    static const void* const kernels[2][3] = {
        {(const void*)&tg::i8_linear_gemv_kernel<tg::DT_F32, 8, 0>,
         (const void*)&tg::i8_linear_gemv_kernel<tg::DT_F16, 8, 0>,
         (const void*)&tg::i8_linear_gemv_kernel<tg::DT_BF16, 8, 0>},
        {(const void*)&tg::i8_linear_gemv_kernel<tg::DT_F32, 8, 1>,
         (const void*)&tg::i8_linear_gemv_kernel<tg::DT_F16, 8, 1>,
         (const void*)&tg::i8_linear_gemv_kernel<tg::DT_BF16, 8, 1>}};
    const void* k = kernels[shift_i8(nullptr, 0, p.W, p.ldw)][dtype];
    const unsigned levels =
        (unsigned)(p.M * tg::I8Gemv<tg::DT_BF16, 1, 8, 0, true>::level_row(p.K));
    return tg::launch_kernel(k, ceil_div(p.N, 16), 1, 512, &l, stream, "i8_linear_gemv",
                             levels > 8192 ? levels : 8192);
}

}  // namespace

namespace tg {

void describe_i8(int64_t M, int64_t N, int64_t K, char* buf, size_t len)
{
    const bool aligned = K > 0 && K % 16 == 0;
    const int shift = shift_i8(nullptr, K, nullptr, K);
    const auto one = [&](const I8Pick& k, int64_t m, int64_t n, char* to, size_t room) {
        return k.tile ? snprintf(to, room, "%s grid=%lld threads=%d", k.tile->name,
                                 (long long)(ceil_div(m, k.tile->bm) * ceil_div(n, k.tile->bn)),
                                 k.tile->threads)
                      : snprintf(to, room, "i8_gemv_%d grid=%lldx%lld threads=512", k.tokens,
                                 (long long)ceil_div(n, 16), (long long)ceil_div(m, k.tokens));
    };
    const I8Pick k = pick_i8(M, N, K, aligned, shift);
    int at = one(k, k.m1, k.n1, buf, len);
    if (k.m1 == M && k.n1 == N)
        return;
    const int64_t m = k.m1 == M ? M : M - k.m1, n = k.n1 == N ? N : N - k.n1;
    if (at >= 0 && (size_t)at < len)
        at += snprintf(buf + at, len - at, " + ");
    if (at >= 0 && (size_t)at < len)
        one(pick_i8(m, n, K, aligned, shift, true), m, n, buf + at, len - at);
}

}  // namespace tg

extern "C" {

tg_status tg_quant_i8(int64_t M, int64_t K, tg_dtype dtype, const void* X, int64_t ldx, int8_t* Q,
                      int64_t ldq, float* s, tg_stream_t stream)
{
    if (!tg::dtype_ok(dtype))
        return TG_ERR_BAD_DTYPE;
    if (M < 0 || K < 0 || M > kMaxDim || K > kMaxDim / 4 || ldx < K || ldq < K)
        return TG_ERR_BAD_SHAPE;
    if (M == 0)
        return TG_OK;
    if (!s || (K > 0 && (!X || !Q)))
        return TG_ERR_NULL_POINTER;
    const auto x = span(X, M, K, ldx, tg::dtype_size(dtype)), q = span(Q, M, K, ldq, 1),
               ss = span1(s, M, 4);
    if (overlap(x, q) || overlap(x, ss) || overlap(q, ss))
        return TG_ERR_ALIAS;
    tg::QuantParams p{};
    p.X = X;
    p.Q = Q;
    p.s = s;
    p.M = (int)M;
    p.K = p.kq = (int)K;
    p.ldx = ldx;
    p.ldq = ldq;
    return launch_quant(p, dtype, (hipStream_t)stream);
}

tg_status tg_gemm_i8(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda,
                     const float* sa, const int8_t* W, int64_t ldw, const float* sw,
                     const float* bias, tg_dtype dtype, void* C, int64_t ldc, tg_epilogue epi,
                     tg_stream_t stream)
{
    if (!tg::dtype_ok(dtype))
        return TG_ERR_BAD_DTYPE;
    if (epi != TG_EPI_NONE && epi != TG_EPI_RELU)
        return TG_ERR_BAD_EPILOGUE;
    if (tg_status st = check_dims(M, N, K))
        return st;
    if (lda < K || ldw < K || ldc < N || lda > kMaxStride || ldw > kMaxStride)
        return TG_ERR_BAD_SHAPE;
    if (M == 0 || N == 0)
        return TG_OK;
    if (!C || !sa || !sw || (K > 0 && (!A || !W)))
        return TG_ERR_NULL_POINTER;
    const auto c = span(C, M, N, ldc, tg::dtype_size(dtype));
    if (overlap(c, span(A, M, K, lda, 1)) || overlap(c, span(W, N, K, ldw, 1)) ||
        overlap(c, span1(sa, M, 4)) || overlap(c, span1(sw, N, 4)) ||
        overlap(c, span1(bias, N, 4)))
        return TG_ERR_ALIAS;
    tg::I8Params p{};
    p.A = A;
    p.W = W;
    p.sa = sa;
    p.sw = sw;
    p.bias = bias;
    p.C = C;
    p.dt_out = dtype;
    p.M = (int)M;
    p.N = (int)N;
    p.K = (int)K;
    p.lda = lda;
    p.ldw = ldw;
    p.ldc = ldc;
    p.relu = epi == TG_EPI_RELU;
    return launch_i8(p, (hipStream_t)stream);
}

tg_status tg_linear_i8_workspace_size(int64_t M, int64_t N, int64_t K, tg_dtype dtype,
                                      size_t* bytes)
{
    if (!bytes)
        return TG_ERR_NULL_POINTER;
    if (!tg::dtype_ok(dtype))
        return TG_ERR_BAD_DTYPE;
    if (tg_status st = check_dims(M, N, K))
        return st;
    // scales, then rows of levels (and of W) padded to whole 16-byte chunks
    *bytes = M == 0 || N == 0 || fused_linear(M, K)
                 ? 0
                 : (size_t)(ceil_div(4 * M, 256) * 256 +
                            (M + (pack_linear(M, N, K) ? N : 0)) * ceil_div(K, 16) * 16);
    return TG_OK;
}

tg_status tg_linear_i8(int64_t M, int64_t N, int64_t K, tg_dtype dtype, const void* X, int64_t ldx,
                       const int8_t* W, int64_t ldw, const float* sw, const float* bias, void* C,
                       int64_t ldc, tg_epilogue epi, void* workspace, size_t workspace_bytes,
                       tg_stream_t stream)
{
    if (!tg::dtype_ok(dtype))
        return TG_ERR_BAD_DTYPE;
    if (epi != TG_EPI_NONE && epi != TG_EPI_RELU)
        return TG_ERR_BAD_EPILOGUE;
    size_t need = 0;
    if (tg_status st = tg_linear_i8_workspace_size(M, N, K, dtype, &need))
        return st;
    if (ldx < K || ldw < K || ldc < N || ldw > kMaxStride)
        return TG_ERR_BAD_SHAPE;
    if (M == 0 || N == 0)
        return TG_OK;
    if (!C || !sw || (K > 0 && (!X || !W)))
        return TG_ERR_NULL_POINTER;
    if (need > 0 && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 15)))
        return TG_ERR_WORKSPACE;
    const int es = tg::dtype_size(dtype);
    const auto c = span(C, M, N, ldc, es), x = span(X, M, K, ldx, es), w = span(W, N, K, ldw, 1),
               s = span1(sw, N, 4), bs = span1(bias, N, 4),
               ws = span1(workspace, (int64_t)need, 1);
    if (overlap(c, x) || overlap(c, w) || overlap(c, s) || overlap(c, bs) || overlap(ws, c) ||
        overlap(ws, x) || overlap(ws, w) || overlap(ws, s) || overlap(ws, bs))
        return TG_ERR_ALIAS;
    tg::I8Params p{};
    p.W = W;
    p.sw = sw;
    p.bias = bias;
    p.C = C;
    p.dt_out = dtype;
    p.M = (int)M;
    p.N = (int)N;
    p.K = (int)K;
    p.ldw = ldw;
    p.ldc = ldc;
    p.relu = epi == TG_EPI_RELU;
    if (fused_linear(M, K))
        return launch_fused(p, dtype, X, ldx, (hipStream_t)stream);
    const int64_t ldq = ceil_div(K, 16) * 16;
    float* sa = (float*)workspace;
    int8_t* A = (int8_t*)workspace + ceil_div(4 * M, 256) * 256;
    tg::QuantParams q{};
    q.X = X;
    q.Q = A;
    q.s = sa;
    q.M = (int)M;
    q.K = (int)K;
    q.ldx = ldx;
    q.ldq = ldq;
    q.kq = (int)ldq;
    if (pack_linear(M, N, K)) {
        q.W = W;
        q.Wq = A + M * ldq;
        q.ldw = ldw;
        q.N = (int)N;
        p.W = q.Wq;
        p.ldw = ldq;
        p.K = (int)ldq;  // zeros past K in both
    }
    if (tg_status st = launch_quant(q, dtype, (hipStream_t)stream))
        return st;
    p.A = A;
    p.sa = sa;
    p.lda = ldq;
    return launch_i8(p, (hipStream_t)stream);
}

}  // extern "C"
