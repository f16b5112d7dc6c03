// Entry points of the microscaled linear path: quantisation to blocks and back,
// the linear layer with its activations quantised within the call, and its
// gradients.  Arguments are checked before any HIP call; the kernel is chosen by
// sizes and alignment.
#include <hip/hip_runtime.h>

#include "tg_host.h"
#include "tg_kernel_mx_linear.h"
#include "tg_kernel_mx_quant.h"
#include "tg_mx_kernels.h"

namespace {

using tg::ceil_div;
using tg::kMaxDim;
using tg::mx_padded;
using tg::overlap;
using tg::Span;
using tg::span;
using tg::span1;

constexpr int64_t kMaxN = (1 << 27) - 16;   // workgroups of 16 columns, 512 threads
constexpr int64_t kMaxLen = kMaxDim / 256;  // of a summed axis: a tile's offsets fit 31 bits

bool fmt_ok(int f) { return f == TG_MX_E2M1 || f == TG_MX_E4M3; }
int64_t code_bytes(int fmt, int64_t n) { return fmt == TG_MX_E4M3 ? n : n / 2; }
bool misaligned(const void* codes, const void* scales)
{
    return ((uintptr_t)codes & 15) != 0 || ((uintptr_t)scales & 3) != 0;
}

// Calls f with type and format as compile-time constants.
template <class F>
auto by_type(int dt, int fmt, const F& f)
{
    using std::integral_constant;
    using E2 = integral_constant<int, tg::MX_E2M1>;
    using E4 = integral_constant<int, tg::MX_E4M3>;
    const bool e4 = fmt == TG_MX_E4M3;
    if (dt == TG_F32)
        return e4 ? f(integral_constant<int, tg::DT_F32>{}, E4{})
                  : f(integral_constant<int, tg::DT_F32>{}, E2{});
    if (dt == TG_F16)
        return e4 ? f(integral_constant<int, tg::DT_F16>{}, E4{})
                  : f(integral_constant<int, tg::DT_F16>{}, E2{});
    return e4 ? f(integral_constant<int, tg::DT_BF16>{}, E4{})
              : f(integral_constant<int, tg::DT_BF16>{}, E2{});
}

// --------------------------------------------------------------------------
// Quantisation.
// --------------------------------------------------------------------------
// Units of eight elements of a thread, in flight together: two of 16 bits from 8 Mi
// elements on, else one (4096 x 4096 bf16 8.7 us, 9.3 with one; 1000 x 4096 4.2 and
// 4.0; 8192 x 8192 fp32 56.1 and 53.8; four are slower still but for large bf16).
int units_of(int dt, int64_t elements) { return dt != TG_F32 && elements >= (8 << 20) ? 2 : 1; }

tg::u32 unit_magic(int64_t Kp, int units)
{
    const uint64_t per = (uint64_t)Kp / 8;
    return per == 0 || per >= 256u * units
               ? 0
               : (tg::u32)((((uint64_t)1 << 32) + per - 1) / per);
}

const void* columns_kernel(int dt, int fmt, bool rows, bool cols, bool sums)
{
    return by_type(dt, fmt, [&](auto D, auto F) -> const void* {
        constexpr int DT = decltype(D)::value, FMT = decltype(F)::value;
        if (!cols)
            return rows ? (const void*)&tg::mx_columns_kernel<DT, FMT, true, false, true>
                        : (const void*)&tg::mx_columns_kernel<DT, FMT, false, false, true>;
        if (sums)
            return rows ? (const void*)&tg::mx_columns_kernel<DT, FMT, true, true, true>
                        : (const void*)&tg::mx_columns_kernel<DT, FMT, false, true, true>;
        return rows ? (const void*)&tg::mx_columns_kernel<DT, FMT, true, true, false>
                    : (const void*)&tg::mx_columns_kernel<DT, FMT, false, true, false>;
    });
}

// Blocks along the rows (Q), the columns (Qt), or both in one launch; sums: the
// columns' sums over each 128 rows.
tg::MxQuantParams quant_params(int64_t M, int64_t K, const void* X, int64_t ldx, uint8_t* Q,
                               uint8_t* S, uint8_t* Qt, uint8_t* St, float* sums)
{
    tg::MxQuantParams p{};
    p.X = X;
    p.ldx = ldx;
    p.M = (int)M;
    p.K = (int)K;
    p.Kp = (int)mx_padded(K);
    p.Mp = (int)mx_padded(M);
    p.Q = Q;
    p.S = S;
    p.Qt = Qt;
    p.St = St;
    p.sums = sums;
    p.tiles_m = (int)ceil_div(p.Mp, 256);
    p.tiles_n = (int)ceil_div(K, 128);
    return p;
}

tg_status launch_quant(tg::MxQuantParams p, int dt, int fmt, hipStream_t stream)
{
    if (!p.Qt && !p.sums) {
        const int64_t all = (int64_t)p.M * (p.Kp / 8);
        const int u = units_of(dt, 8 * all);
        const void* k = by_type(dt, fmt, [u](auto D, auto F) {
            constexpr int DT = decltype(D)::value, FMT = decltype(F)::value;
            if constexpr (DT != tg::DT_F32)
                if (u == 2)
                    return (const void*)&tg::mx_rows_kernel<DT, FMT, 2>;
            return (const void*)&tg::mx_rows_kernel<DT, FMT, 1>;
        });
        p.magic = unit_magic(p.Kp, u);
        return tg::launch_kernel(k, ceil_div(all, 256 * u), 1, 256, &p, stream, "mx_rows");
    }
    return tg::launch_kernel(columns_kernel(dt, fmt, p.Q != nullptr, p.Qt != nullptr,
                                            p.sums != nullptr),
                             (p.Q ? 2 : 1) * (int64_t)p.tiles_m * p.tiles_n, 1, 256, &p, stream,
                             "mx_columns");
}

// Columns of up to two matrices of one type to E2M1 (those with Qt), and the sums
// (those with an output).
tg_status launch_rest(const tg::MxQuantParams& a, const tg::MxQuantParams& b,
                      const tg::MxSumParams& sums, int dt, hipStream_t stream)
{
    const auto groups = [](const tg::MxQuantParams& q) {
        return q.Qt ? (int64_t)q.tiles_m * q.tiles_n : 0;
    };
    const int64_t e0 = groups(a), e1 = e0 + groups(b),
                  all = e1 + (sums.out ? ceil_div(sums.K, 256) : 0);
    if (all == 0)
        return TG_OK;
    if (all > kMaxDim)
        return TG_ERR_BAD_SHAPE;
    tg::MxRestParams p{{a, b}, sums, {(int)e0, (int)e1}};
    const void* k = dt == TG_F32   ? (const void*)&tg::mx_rest_kernel<tg::DT_F32>
                    : dt == TG_F16 ? (const void*)&tg::mx_rest_kernel<tg::DT_F16>
                                   : (const void*)&tg::mx_rest_kernel<tg::DT_BF16>;
    return tg::launch_kernel(k, all, 1, 256, &p, stream, "mx_rest");
}

// --------------------------------------------------------------------------
// Product of two matrices of blocks.
// --------------------------------------------------------------------------
using tg::MxKernel;

float kernel_cost(const MxKernel& k, int64_t M, int64_t N, int64_t K)
{
    const int64_t groups = ceil_div(M, k.bm) * ceil_div(N, k.bn);
    const float strips = (float)(K / 128);
    return k.t0 + (groups <= 256 ? strips * k.one
                                 : (float)ceil_div(groups, 256) * (k.round + strips * k.full));
}

// The cheapest; up to 16 tokens among the streaming kernels (1 x 14336 x 4096 in E4M3
// 10.2 us, 15.5 with 64 x 64 tiles), above 256 among the tiles.
const MxKernel* pick_kernel(int64_t M, int64_t N, int64_t K, int fmt)
{
    const MxKernel* best = nullptr;
    float cost = 0.0f;
    const tg::MxKernels all =
        fmt == TG_MX_E4M3 ? tg::mx_kernels_e4m3() : tg::mx_kernels_e2m1();
    for (const MxKernel* k = all.begin; k != all.end; ++k) {
        if (K % k->strip != 0 || (k->lds ? M > 256 : M <= 16))
            continue;
        const float c = kernel_cost(*k, M, N, K);
        if (!best || c < cost) {
            best = k;
            cost = c;
        }
    }
    return best;
}

struct Product {
    int64_t M, N, K;  // K padded
    int fmt, dt;
    const uint8_t *A, *As, *W, *Ws;
    const float* bias;
    void* C;
    int64_t ldc;
    bool relu;
};

tg::MxLinearParams product_params(const Product& q)
{
    tg::MxLinearParams p{};
    p.g.A = q.A;
    p.g.As = q.As;
    p.g.B = q.W;
    p.g.Bs = q.Ws;
    p.g.C = q.C;
    p.g.M = (int)q.M;
    p.g.N = (int)q.N;
    p.g.K = (int)q.K;
    p.g.relu = q.relu;
    p.g.stamps = tg::clock_stamps();
    p.bias = q.bias;
    p.ldc = q.ldc;
    return p;
}

tg_status launch_product(const Product& q, hipStream_t stream)
{
    tg::MxLinearParams p = product_params(q);
    const MxKernel* k = pick_kernel(q.M, q.N, q.K, q.fmt);
    const int64_t tm = ceil_div(q.M, k->bm), tn = ceil_div(q.N, k->bn);
    if (k->lds) {
        tg::MxStreamParams s{p, q.dt, nullptr, 0, 0};
        return tg::launch_kernel(k->kernel[0], tn, tm, k->threads, &s, stream, k->name, k->lds);
    }
    const int es = tg::dtype_size(q.dt);
    p.g.group_m = tg::swizzle_override() > 0 ? tg::swizzle_override() : 4;
    p.g.tiles_m = (int)tm;
    p.g.tiles_n = (int)tn;
    p.g.c_vec = ((uintptr_t)q.C & 15) == 0 && q.ldc * es % 16 == 0 && q.N * es % 16 == 0 &&
                32 * q.ldc * es <= kMaxDim;
    return tg::launch_kernel(k->kernel[q.dt], tm * tn, 1, k->threads, &p, stream, k->name);
}

tg_status launch_fill(int64_t M, int64_t N, int dt, const float* bias, void* C, int64_t ldc,
                      bool relu, hipStream_t stream)
{
    if (M == 0 || N == 0)
        return TG_OK;
    tg::MxFillParams p{bias, C, ldc, (int)M, (int)N, dt, relu};
    const int64_t groups = ceil_div(M * N, 256);
    return tg::launch_kernel((const void*)&tg::mx_fill_kernel, groups < (1 << 20) ? groups : 1 << 20,
                             1, 256, &p, stream, "mx_fill");
}

// --------------------------------------------------------------------------
// The linear layer.
// --------------------------------------------------------------------------
// In one launch: a few tokens, whose quantisation in every workgroup takes less
// than a launch of its own would.  Measured with both launches and with one: 1 x 1024
// x 1024 4.2 us and 2.9, 8 x 4096 x 1024 4.7 and 3.4, 8 x 2048 x 2048 5.2 and 4.0, 4 x
// 8192 x 8192 15.0 and 13.6, 8 x 4096 x 4096 7.3 and 7.0, 6 x 1024 x 8192 8.1 and 9.3;
// with more than two workgroups to a compute unit half as much: 4 x 14336 x 4096 12.5
// and 11.8, 6 x 14336 x 4096 12.3 and 13.7.
bool fused_linear(int64_t M, int64_t N, int64_t K)
{
    return M <= 16 && K > 0 && M * K <= (N <= 8192 ? 32768 : 16384);
}

size_t linear_bytes(int64_t M, int64_t N, int64_t K, int fmt)
{
    if (M == 0 || N == 0 || K == 0 || fused_linear(M, N, K))
        return 0;
    const int64_t Kp = mx_padded(K);
    return (size_t)(ceil_div(M * (Kp / 32), 256) * 256 + M * code_bytes(fmt, Kp));
}

tg_status check_linear(int64_t M, int64_t N, int64_t K, int dtype, int fmt)
{
    if (!tg::dtype_ok(dtype) || !fmt_ok(fmt))
        return TG_ERR_BAD_DTYPE;
    if (M < 0 || N < 0 || K < 0 || M > kMaxDim / 4 || N > kMaxN || K > kMaxLen - 128)
        return TG_ERR_BAD_SHAPE;
    return TG_OK;
}

// How a backward call lays out its workspace, in bytes from its start; parts
// that are not needed are empty.
struct GradPlan {
    int64_t Mp, Np;
    bool dx, dw, db;
    int64_t dy, dys, dyt, dyts, wt, wts, xt, xts, sums, bytes;
};

GradPlan grad_plan(const tg_linear_mx_grad_args& a)
{
    GradPlan g{};
    g.Mp = mx_padded(a.M);
    g.Np = mx_padded(a.N);
    const bool any = a.M > 0 && a.N > 0;
    g.dx = a.dX && any && a.K > 0;
    g.dw = a.dW && any && a.K > 0;
    g.db = a.dbias && any;
    const auto take = [&](bool need, int64_t n) {
        const int64_t at = g.bytes;
        g.bytes += need ? ceil_div(n, 256) * 256 : 0;
        return at;
    };
    g.dy = take(g.dx, a.M * code_bytes(a.fmt, g.Np));
    g.dys = take(g.dx, a.M * (g.Np / 32));
    g.dyt = take(g.dw, a.N * code_bytes(a.fmt, g.Mp));
    g.dyts = take(g.dw, a.N * (g.Mp / 32));
    g.wt = take(g.dx, a.K * (g.Np / 2));
    g.wts = take(g.dx, a.K * (g.Np / 32));
    g.xt = take(g.dw, a.K * (g.Mp / 2));
    g.xts = take(g.dw, a.K * (g.Mp / 32));
    g.sums = take(g.db, g.Mp / 128 * a.N * 4);
    return g;
}

tg_status check_grad(const tg_linear_mx_grad_args* a)
{
    if (!a)
        return TG_ERR_NULL_POINTER;
    if (!tg::dtype_ok(a->dtype) || !tg::dtype_ok(a->wtype) || !fmt_ok(a->fmt) ||
        (a->wtype != a->dtype && a->wtype != TG_F32))
        return TG_ERR_BAD_DTYPE;
    const int64_t most = kMaxLen - 128;
    if (a->M < 0 || a->N < 0 || a->K < 0 || a->M > most || a->N > most || a->K > most)
        return TG_ERR_BAD_SHAPE;
    const auto bad = [](const void* p, int64_t ld, int64_t n) { return p && ld < n; };
    if (bad(a->dY, a->lddy, a->N) || bad(a->X, a->ldx, a->K) || bad(a->W, a->ldw, a->K) ||
        bad(a->dX, a->lddx, a->K) || bad(a->dW, a->lddw, a->K))
        return TG_ERR_BAD_SHAPE;
    return TG_OK;
}

}  // namespace

extern "C" {

tg_status tg_quant_mx(int64_t M, int64_t K, tg_dtype dtype, const void* X, int64_t ldx,
                      tg_mx_format fmt, uint8_t* Q, uint8_t* S, uint8_t* Qt, uint8_t* St,
                      tg_stream_t stream)
{
    if (!tg::dtype_ok(dtype) || !fmt_ok(fmt))
        return TG_ERR_BAD_DTYPE;
    if (M < 0 || K < 0 || M > kMaxDim / 4 || K > kMaxDim / 4 || ldx < K)
        return TG_ERR_BAD_SHAPE;
    if (M == 0 || K == 0)
        return TG_OK;
    if (!X || (!Q && !Qt) || !Q != !S || !Qt != !St)
        return TG_ERR_NULL_POINTER;
    if (misaligned(Q, S) || misaligned(Qt, St))
        return TG_ERR_NO_CONFIG;
    const int64_t Kp = mx_padded(K), Mp = mx_padded(M);
    const Span x = span(X, M, K, ldx, tg::dtype_size(dtype));
    const Span out[] = {span1(Q, M * code_bytes(fmt, Kp), 1), span1(S, M * (Kp / 32), 1),
                        span1(Qt, K * code_bytes(fmt, Mp), 1), span1(St, K * (Mp / 32), 1)};
    for (int o = 0; o < 4; ++o) {
        if (overlap(out[o], x))
            return TG_ERR_ALIAS;
        for (int i = 0; i < o; ++i)
            if (overlap(out[o], out[i]))
                return TG_ERR_ALIAS;
    }
    return launch_quant(quant_params(M, K, X, ldx, Q, S, Qt, St, nullptr), dtype, fmt,
                        (hipStream_t)stream);
}

tg_status tg_dequant_mx(int64_t M, int64_t K, tg_mx_format fmt, const uint8_t* Q, const uint8_t* S,
                        tg_dtype dtype, void* X, int64_t ldx, tg_stream_t stream)
{
    if (!tg::dtype_ok(dtype) || !fmt_ok(fmt))
        return TG_ERR_BAD_DTYPE;
    if (M < 0 || K < 0 || M > kMaxDim / 4 || K > kMaxDim / 4 || ldx < K)
        return TG_ERR_BAD_SHAPE;
    if (M == 0 || K == 0)
        return TG_OK;
    if (!X || !Q || !S)
        return TG_ERR_NULL_POINTER;
    if (misaligned(Q, S))
        return TG_ERR_NO_CONFIG;
    const int64_t Kp = mx_padded(K);
    const Span x = span(X, M, K, ldx, tg::dtype_size(dtype));
    if (overlap(x, span1(Q, M * code_bytes(fmt, Kp), 1)) || overlap(x, span1(S, M * (Kp / 32), 1)))
        return TG_ERR_ALIAS;
    const int64_t all = M * (Kp / 8);
    const int u = units_of(dtype, 8 * all);
    tg::MxDequantParams p{Q, S, X, ldx, (int)M, (int)K, (int)Kp, unit_magic(Kp, u)};
    const void* k = by_type(dtype, fmt, [u](auto D, auto F) {
        constexpr int DT = decltype(D)::value, FMT = decltype(F)::value;
        if constexpr (DT != tg::DT_F32)
            if (u == 2)
                return (const void*)&tg::mx_dequant_kernel<DT, FMT, 2>;
        return (const void*)&tg::mx_dequant_kernel<DT, FMT, 1>;
    });
    return tg::launch_kernel(k, ceil_div(all, 256 * u), 1, 256, &p, (hipStream_t)stream,
                             "mx_dequant");
}

tg_status tg_linear_mx_workspace_size(int64_t M, int64_t N, int64_t K, tg_dtype dtype,
                                      tg_mx_format fmt, size_t* bytes)
{
    if (!bytes)
        return TG_ERR_NULL_POINTER;
    if (tg_status s = check_linear(M, N, K, dtype, fmt))
        return s;
    *bytes = linear_bytes(M, N, K, fmt);
    return TG_OK;
}

tg_status tg_linear_mx(int64_t M, int64_t N, int64_t K, tg_dtype dtype, const void* X, int64_t ldx,
                       tg_mx_format fmt, const uint8_t* Wq, const uint8_t* Ws, const float* bias,
                       void* C, int64_t ldc, tg_epilogue epi, void* workspace,
                       size_t workspace_bytes, tg_stream_t stream)
{
    if (tg_status s = check_linear(M, N, K, dtype, fmt))
        return s;
    if (epi != TG_EPI_NONE && epi != TG_EPI_RELU)
        return TG_ERR_BAD_EPILOGUE;
    if (ldx < K || ldc < N)
        return TG_ERR_BAD_SHAPE;
    if (M == 0 || N == 0)
        return TG_OK;
    if (!C || (K > 0 && (!X || !Wq || !Ws)))
        return TG_ERR_NULL_POINTER;
    const int64_t Kp = mx_padded(K);
    if (K > 0 && misaligned(Wq, Ws))
        return TG_ERR_NO_CONFIG;
    const size_t need = linear_bytes(M, N, K, fmt);
    if (need > 0 && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 15)))
        return TG_ERR_WORKSPACE;
    const int es = tg::dtype_size(dtype);
    const Span in[] = {span(X, M, K, ldx, es), span1(Wq, N * (Kp / 2), 1),
                       span1(Ws, N * (Kp / 32), 1), span1(bias, N, 4)};
    const Span c = span(C, M, N, ldc, es), ws = span1(workspace, (int64_t)need, 1);
    for (const Span& i : in)
        if (overlap(c, i) || overlap(ws, i))
            return TG_ERR_ALIAS;
    if (overlap(c, ws))
        return TG_ERR_ALIAS;
    const hipStream_t hs = (hipStream_t)stream;
    const bool relu = epi == TG_EPI_RELU;
    if (K == 0)
        return launch_fill(M, N, dtype, bias, C, ldc, relu, hs);
    Product q{M, N, Kp, fmt, dtype, nullptr, nullptr, Wq, Ws, bias, C, ldc, relu};
    if (fused_linear(M, N, K)) {
        tg::MxStreamParams s{product_params(q), (int)dtype, X, ldx, (int)K};
        int lds = 0;
        const void* k = by_type(dtype, fmt, [&](auto D, auto F) {
            constexpr int DT = decltype(D)::value, FMT = decltype(F)::value;
            lds = tg::MxStream<DT, FMT, 1, 1, 2, 8, true>::lds_bytes((int)M, (int)Kp);
            return (const void*)&tg::mx_stream_kernel<DT, FMT, 1, 1, 2, 8, true>;
        });
        return tg::launch_kernel(k, ceil_div(N, 16), 1, 512, &s, hs, "mx_linear_stream",
                                 (unsigned)lds);
    }
    uint8_t* As = (uint8_t*)workspace;
    uint8_t* A = As + ceil_div(M * (Kp / 32), 256) * 256;
    if (tg_status s = launch_quant(quant_params(M, K, X, ldx, A, As, nullptr, nullptr, nullptr),
                                   dtype, fmt, hs))
        return s;
    q.A = A;
    q.As = As;
    return launch_product(q, hs);
}

tg_status tg_linear_mx_backward_workspace_size(const tg_linear_mx_grad_args* a, size_t* bytes)
{
    if (!bytes)
        return TG_ERR_NULL_POINTER;
    if (tg_status s = check_grad(a))
        return s;
    *bytes = (size_t)grad_plan(*a).bytes;
    return TG_OK;
}

tg_status tg_linear_mx_backward(const tg_linear_mx_grad_args* a, void* workspace,
                                size_t workspace_bytes, tg_stream_t stream)
{
    if (tg_status s = check_grad(a))
        return s;
    const int64_t M = a->M, N = a->N, K = a->K;
    const bool out = (a->dX && M > 0 && K > 0) || (a->dW && N > 0 && K > 0) || (a->dbias && N > 0);
    // nothing to write: outputs that are empty may be NULL
    if (!a->dX && !a->dW && !a->dbias && M > 0 && N > 0 && K > 0)
        return TG_ERR_NULL_POINTER;
    if (!out)
        return TG_OK;
    const GradPlan g = grad_plan(*a);
    if (((g.dx || g.dw || g.db) && !a->dY) || (g.dx && !a->W) || (g.dw && !a->X))
        return TG_ERR_NULL_POINTER;
    if (g.bytes > 0 &&
        (!workspace || workspace_bytes < (size_t)g.bytes || ((uintptr_t)workspace & 15)))
        return TG_ERR_WORKSPACE;
    const int es = tg::dtype_size(a->dtype), wes = tg::dtype_size(a->wtype);
    const Span in[] = {span(a->dY, M, N, a->lddy, es), span(a->X, M, K, a->ldx, es),
                       span(a->W, N, K, a->ldw, wes)};
    const Span outs[] = {span(a->dX, M, K, a->lddx, es), span(a->dW, N, K, a->lddw, wes),
                         span1(a->dbias, N, 4), span1(workspace, g.bytes, 1)};
    for (int o = 0; o < 4; ++o) {
        for (const Span& i : in)
            if (overlap(outs[o], i))
                return TG_ERR_ALIAS;
        for (int i = 0; i < o; ++i)
            if (overlap(outs[o], outs[i]))
                return TG_ERR_ALIAS;
    }
    const hipStream_t hs = (hipStream_t)stream;
    uint8_t* ws = (uint8_t*)workspace;
    if (g.dx || g.dw || g.db) {
        const auto at = [ws](bool wanted, int64_t o) { return wanted ? ws + o : nullptr; };
        if (tg_status s = launch_quant(
                quant_params(M, N, a->dY, a->lddy, at(g.dx, g.dy), at(g.dx, g.dys),
                             at(g.dw, g.dyt), at(g.dw, g.dyts), (float*)at(g.db, g.sums)),
                a->dtype, a->fmt, hs))
            return s;
        const tg::MxQuantParams w = quant_params(N, K, a->W, a->ldw, nullptr, nullptr,
                                                 at(g.dx, g.wt), at(g.dx, g.wts), nullptr),
                                x = quant_params(M, K, a->X, a->ldx, nullptr, nullptr,
                                                 at(g.dw, g.xt), at(g.dw, g.xts), nullptr);
        const tg::MxSumParams sums{(const float*)(ws + g.sums), g.db ? a->dbias : nullptr,
                                   (int)(g.Mp / 128), (int)N};
        const bool one = a->wtype == a->dtype;
        if (tg_status s = launch_rest(one ? w : tg::MxQuantParams{}, x, sums, a->dtype, hs))
            return s;
        if (!one)
            if (tg_status s = launch_rest(w, {}, {}, a->wtype, hs))
                return s;
    }
    if (g.dx) {
        const Product q{M,          K,          g.Np,        a->fmt,  a->dtype, ws + g.dy,
                        ws + g.dys, ws + g.wt,  ws + g.wts,  nullptr, a->dX,    a->lddx,
                        false};
        if (tg_status s = launch_product(q, hs))
            return s;
    } else if (a->dX) {
        if (tg_status s = launch_fill(M, K, a->dtype, nullptr, a->dX, a->lddx, false, hs))
            return s;
    }
    if (g.dw) {
        const Product q{N,           K,          g.Mp,        a->fmt,  a->wtype, ws + g.dyt,
                        ws + g.dyts, ws + g.xt,  ws + g.xts,  nullptr, a->dW,    a->lddw,
                        false};
        if (tg_status s = launch_product(q, hs))
            return s;
    } else if (a->dW) {
        if (tg_status s = launch_fill(N, K, a->wtype, nullptr, a->dW, a->lddw, false, hs))
            return s;
    }
    return a->dbias && !g.db ? launch_fill(1, N, TG_F32, nullptr, a->dbias, N, false, hs) : TG_OK;
}

}  // extern "C"
