// Entry points of the 8-bit integer path: quantisation, product, and both in
// one call.  Arguments are checked before any HIP call; the kernel is chosen
// by sizes and alignment.
#include <hip/hip_runtime.h>

#include "tg_host.h"
#include "tg_kernel_i8.h"
#include "tg_kernel_quant.h"

namespace {

using tg::ceil_div;
using tg::kMaxDim;
using tg::overlap;
using tg::span;
using tg::span1;

// Kernel for rows of K elements: one wave for a row, four waves, or sixteen,
// with 1, 2 or 4 chunks of 8 elements for each thread.
template <int DT>
const void* quant_kernel(int64_t K, int* threads, int* rows)
{
    *threads = 256;
    *rows = K <= 2048 ? 4 : 1;
    if (K <= 512)
        return (const void*)&tg::quant_i8_kernel<DT, 256, 64, 1>;
    if (K <= 2048)
        return (const void*)&tg::quant_i8_kernel<DT, 256, 64, 4>;
    if (K <= 4096)
        return (const void*)&tg::quant_i8_kernel<DT, 256, 256, 2>;
    if (K <= 8192)
        return (const void*)&tg::quant_i8_kernel<DT, 256, 256, 4>;
    *threads = 1024;
    if (K <= 32768)
        return (const void*)&tg::quant_i8_kernel<DT, 1024, 1024, 4>;
    return (const void*)&tg::quant_i8_kernel<DT, 1024, 1024, 0>;
}

tg_status launch_quant(const tg::QuantParams& p, int dtype, hipStream_t stream)
{
    int threads, rows;
    const void* k = dtype == TG_F32   ? quant_kernel<tg::DT_F32>(p.K, &threads, &rows)
                    : dtype == TG_F16 ? quant_kernel<tg::DT_F16>(p.K, &threads, &rows)
                                      : quant_kernel<tg::DT_BF16>(p.K, &threads, &rows);
    tg::QuantParams q = p;
    return tg::launch_kernel(k, ceil_div(p.M, rows), 1, threads, &q, stream, "quant_i8");
}

constexpr int64_t kMaxK = 131071;  // 128 * 128 * K stays below 2^31

tg_status check_dims(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxK)
        return TG_ERR_BAD_SHAPE;
    return TG_OK;
}

tg_status launch_i8(tg::I8Params p, hipStream_t stream)
{
    p.stamps = tg::clock_stamps();
    p.group_m = tg::swizzle_override() > 0 ? tg::swizzle_override() : 8;
    p.tiles_m = (int)ceil_div(p.M, tg::I8Any::BM);
    p.tiles_n = (int)ceil_div(p.N, tg::I8Any::BN);
    return tg::launch_kernel((const void*)&tg::i8_any_kernel, (int64_t)p.tiles_m * p.tiles_n, 1,
                             256, &p, stream, "i8_any");
}

}  // namespace

extern "C" {

tg_status tg_quant_i8(int64_t M, int64_t K, tg_dtype dtype, const void* X, int64_t ldx, int8_t* Q,
                      int64_t ldq, float* s, tg_stream_t stream)
{
    if (!tg::dtype_ok(dtype))
        return TG_ERR_BAD_DTYPE;
    if (M < 0 || K < 0 || M > kMaxDim || K > kMaxDim / 2 || ldx < K || ldq < K)
        return TG_ERR_BAD_SHAPE;
    if (M == 0)
        return TG_OK;
    if (!s || (K > 0 && (!X || !Q)))
        return TG_ERR_NULL_POINTER;
    const auto x = span(X, M, K, ldx, tg::dtype_size(dtype)), q = span(Q, M, K, ldq, 1),
               ss = span1(s, M, 4);
    if (overlap(x, q) || overlap(x, ss) || overlap(q, ss))
        return TG_ERR_ALIAS;
    tg::QuantParams p{X, Q, s, M, (int)K, ldx, ldq, (int)K};
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
    if (lda < K || ldw < K || ldc < N)
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
    // scales, then rows of levels padded to whole 16-byte chunks
    *bytes = M == 0 || N == 0 ? 0
                              : (size_t)(ceil_div(4 * M, 256) * 256 + M * ceil_div(K, 16) * 16);
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
    if (ldx < K || ldw < K || ldc < N)
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
    const int64_t ldq = ceil_div(K, 16) * 16;
    float* sa = (float*)workspace;
    int8_t* A = (int8_t*)workspace + ceil_div(4 * M, 256) * 256;
    tg::QuantParams q{X, A, sa, M, (int)K, ldx, ldq, (int)ldq};
    if (tg_status st = launch_quant(q, dtype, (hipStream_t)stream))
        return st;
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
    p.lda = ldq;
    p.ldw = ldw;
    p.ldc = ldc;
    p.relu = epi == TG_EPI_RELU;
    return launch_i8(p, (hipStream_t)stream);
}

}  // extern "C"
