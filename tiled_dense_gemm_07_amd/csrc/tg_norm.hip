// Entry points of the norms between blocks and their gradients.  Arguments are
// checked before any HIP call; the kernel is chosen by the row length.
#include <hip/hip_runtime.h>

#include "tg_host.h"
#include "tg_kernel_norm.h"

namespace {

using tg::ceil_div;
using tg::overlap;
using tg::Span;
using tg::span;
using tg::span1;

constexpr int64_t kMaxD = 32768;    // 1024 threads of 32 elements
constexpr int64_t kMaxT = 1 << 30;  // sums of two row numbers fit 31 bits

bool types_ok(int xt, int bt)
{
    return tg::dtype_ok(xt) && tg::dtype_ok(bt) && (xt == bt || xt == TG_F32);
}

// Calls f with the two types as compile-time constants.
template <class F>
auto by_types(int xt, int bt, const F& f)
{
    using std::integral_constant;
    if (xt == TG_BF16)
        return f(integral_constant<int, tg::DT_BF16>{}, integral_constant<int, tg::DT_BF16>{});
    if (xt == TG_F16)
        return f(integral_constant<int, tg::DT_F16>{}, integral_constant<int, tg::DT_F16>{});
    if (bt == TG_BF16)
        return f(integral_constant<int, tg::DT_F32>{}, integral_constant<int, tg::DT_BF16>{});
    if (bt == TG_F16)
        return f(integral_constant<int, tg::DT_F32>{}, integral_constant<int, tg::DT_F16>{});
    return f(integral_constant<int, tg::DT_F32>{}, integral_constant<int, tg::DT_F32>{});
}

struct Pick {
    const void* kernel;
    int threads;  // of a workgroup
    int rows;     // of a workgroup
};

// A row to one wave, or to a workgroup of four, eight or sixteen.  Measured
// (bf16, h and 8-bit h, 8192 rows; 4096 of D = 8192): D = 1024 11.4 and 12.2 us
// with two chunks a lane of one wave, 14.8 and 18.1 with one chunk a thread of
// four; D = 2048 20.9 and 21.2 with four of one wave, 21.0 and 22.0 with one of
// four (2.9 and 2.6 us for one row); D = 4096 39.5 and 37.0 with two of four,
// 39.2 and 40.0 with one of eight; D = 8192 39.7 and 38.1 with two of eight, 40.6
// and 43.2 with one of sixteen.
// ODD: rows with an odd number of elements, some of them of 16 bits.
template <int XT, int BT, bool ODD>
Pick pick_forward_of(int64_t D)
{
    if (D <= 512)
        return {(const void*)&tg::block_norm_kernel<XT, BT, 256, 64, 1, ODD>, 256, 4};
    if (D <= 1024)
        return {(const void*)&tg::block_norm_kernel<XT, BT, 256, 64, 2, ODD>, 256, 4};
    if (D <= 2048)
        return {(const void*)&tg::block_norm_kernel<XT, BT, 256, 256, 1, ODD>, 256, 1};
    if (D <= 4096)
        return {(const void*)&tg::block_norm_kernel<XT, BT, 256, 256, 2, ODD>, 256, 1};
    if (D <= 8192)
        return {(const void*)&tg::block_norm_kernel<XT, BT, 512, 512, 2, ODD>, 512, 1};
    if (D <= 16384)
        return {(const void*)&tg::block_norm_kernel<XT, BT, 1024, 1024, 2, ODD>, 1024, 1};
    return {(const void*)&tg::block_norm_kernel<XT, BT, 1024, 1024, 4, ODD>, 1024, 1};
}

Pick pick_forward(int64_t D, int xt, int bt)
{
    return by_types(xt, bt, [&](auto X, auto B) -> Pick {
        constexpr int XT = decltype(X)::value, BT = decltype(B)::value;
        if constexpr (BT == tg::DT_F32)
            return pick_forward_of<XT, BT, false>(D);
        else
            return D % 2 ? pick_forward_of<XT, BT, true>(D) : pick_forward_of<XT, BT, false>(D);
    });
}

// One workgroup to a compute unit: 1024 threads (128 registers each) in teams,
// or 512 where both types are fp32, whose rows take twice the registers.  From D
// = 8193 on (both fp32: 4097) the registers do not hold a thread's sums and row,
// and some are spilled (tg_kernel_norm.h has the times).
template <int XT, int BT, bool ODD>
Pick pick_backward_of(int64_t D)
{
    constexpr int NT = XT == tg::DT_F32 && BT == tg::DT_F32 ? 512 : 1024;
    constexpr int W = NT / 256;  // waves to a SIMD
    if (D <= 512)
        return {(const void*)&tg::block_norm_grad_kernel<XT, BT, NT, 64, 1, W, ODD>, NT, 1};
    if (D <= 1024)
        return {(const void*)&tg::block_norm_grad_kernel<XT, BT, NT, 128, 1, W, ODD>, NT, 1};
    if (D <= 2048)
        return {(const void*)&tg::block_norm_grad_kernel<XT, BT, NT, 256, 1, W, ODD>, NT, 1};
    if (D <= 4096)
        return {(const void*)&tg::block_norm_grad_kernel<XT, BT, NT, 512, 1, W, ODD>, NT, 1};
    if (D <= 8192)
        return {(const void*)&tg::block_norm_grad_kernel<XT, BT, 1024, 1024, 1, 4, ODD>, 1024, 1};
    if (D <= 16384)
        return {(const void*)&tg::block_norm_grad_kernel<XT, BT, 1024, 1024, 2, 4, ODD>, 1024, 1};
    return {(const void*)&tg::block_norm_grad_kernel<XT, BT, 1024, 1024, 4, 4, ODD>, 1024, 1};
}

Pick pick_backward(int64_t D, int xt, int bt)
{
    return by_types(xt, bt, [&](auto X, auto B) -> Pick {
        constexpr int XT = decltype(X)::value, BT = decltype(B)::value;
        if constexpr (BT == tg::DT_F32)
            return pick_backward_of<XT, BT, false>(D);
        else
            return D % 2 ? pick_backward_of<XT, BT, true>(D) : pick_backward_of<XT, BT, false>(D);
    });
}

bool bad_size(int64_t T, int64_t D) { return T < 0 || D < 0 || T > kMaxT || D > kMaxD; }
bool bad_stride(const void* p, int64_t ld, int64_t D) { return p && ld < D; }

// How the gradient kernel's workgroups share the rows, and the workspace.
struct GradPlan {
    int64_t groups;  // rows of gate (1 without a gate)
    int64_t gate_rows;
    int64_t rows;   // rows of a workgroup
    int64_t parts;  // workgroups of a group; 0: whole groups, each to a team
    int64_t P;      // workgroups
    int64_t Dp;
    bool pre, y;    // partial sums kept: of dw_pre; of dw_post and shared gates
    size_t bytes;
};

GradPlan grad_plan(const tg_block_norm_grad_args& a)
{
    GradPlan g{};
    // One workgroup to a compute unit, and at least a row for each of its
    // teams and two in all: with fewer, the partial sums would cost more than
    // the rows.
    const int64_t teams =
        a.D <= 512 ? 16 : (a.D <= 1024 ? 8 : (a.D <= 2048 ? 4 : (a.D <= 4096 ? 2 : 1)));
    int64_t want = ceil_div(a.T, 256);
    want = want < teams ? teams : want;
    want = want < 2 ? 2 : want;
    g.gate_rows = a.gate ? (a.gate_rows < a.T ? a.gate_rows : a.T) : a.T;
    g.groups = ceil_div(a.T, g.gate_rows);
    // Parts of groups, rows to the teams in turn; or whole groups, at least
    // one for each team.  The rows that a team takes one after the other, for
    // each round of 256 workgroups, decide; where a workgroup has one group, its
    // partial sums count as two rows more, and the sums of each 128 groups as
    // one.  (Whole groups also where the sums of a group each would be more than
    // a grid's y dimension.)  Backward of 8192 x 512 with gates of 16 tokens: 16
    // us and 8 for the column sums by parts; whole groups left one team of 16 at
    // work.
    const int64_t parts = ceil_div(g.gate_rows, want);
    const int64_t part_rows = ceil_div(g.gate_rows, parts);
    const int64_t inter =
        ceil_div(g.groups * parts, 256) * (ceil_div(part_rows, teams) + 2) + g.groups / 128;
    const int64_t least = want > teams * g.gate_rows ? want : teams * g.gate_rows;
    const int64_t in_wg = ceil_div(least, g.gate_rows);  // groups
    const int64_t whole =
        ceil_div(g.groups, 256 * in_wg) * (g.gate_rows * ceil_div(in_wg, teams));
    if (a.gate && (whole < inter || g.groups > 32768)) {
        g.parts = 0;
        g.rows = in_wg * g.gate_rows;
        g.P = ceil_div(g.groups, in_wg);
    } else {
        g.parts = parts;
        g.rows = part_rows;
        g.P = g.groups * parts;
    }
    g.Dp = ceil_div(a.D, 8) * 8;
    g.pre = a.dw_pre != nullptr;
    g.y = a.dw_post != nullptr || (a.dgate != nullptr && g.parts > 0);
    g.bytes = (size_t)(g.P * g.Dp * 4) * ((g.pre ? 1 : 0) + (g.y ? 1 : 0));
    return g;
}

// Sizes, types and the operands that go together.
tg_status check_grad(const tg_block_norm_grad_args* a)
{
    if (!a)
        return TG_ERR_NULL_POINTER;
    if (!types_ok(a->xtype, a->btype))
        return TG_ERR_BAD_DTYPE;
    if (bad_size(a->T, a->D) || (a->gate && a->gate_rows < 1))
        return TG_ERR_BAD_SHAPE;
    if (bad_stride(a->x_new, a->ldx_new, a->D) || bad_stride(a->y, a->ldy, a->D) ||
        bad_stride(a->dx_new, a->lddx_new, a->D) || bad_stride(a->dh, a->lddh, a->D) ||
        bad_stride(a->dx, a->lddx, a->D) || bad_stride(a->dy, a->lddy, a->D))
        return TG_ERR_BAD_SHAPE;
    return TG_OK;
}

}  // namespace

extern "C" {

tg_status tg_block_norm(const tg_block_norm_args* a, tg_stream_t stream)
{
    if (!a)
        return TG_ERR_NULL_POINTER;
    if (!types_ok(a->xtype, a->btype))
        return TG_ERR_BAD_DTYPE;
    const int64_t T = a->T, D = a->D;
    if (bad_size(T, D) || (a->gate && a->gate_rows < 1))
        return TG_ERR_BAD_SHAPE;
    if (bad_stride(a->x, a->ldx, D) || bad_stride(a->y, a->ldy, D) ||
        bad_stride(a->x_out, a->ldx_out, D) || bad_stride(a->h, a->ldh, D) ||
        bad_stride(a->hq, a->ldhq, D))
        return TG_ERR_BAD_SHAPE;
    if (T == 0 || D == 0)
        return TG_OK;
    if (!a->x || (a->y && !a->x_out) || (!a->x_out && !a->h && !a->hq) || (!a->hq != !a->hs))
        return TG_ERR_NULL_POINTER;
    if ((!a->y && (a->x_out || a->gate || a->w_post || a->r_post)) ||
        (!a->post_norm && (a->w_post || a->r_post)) || (!a->h && !a->hq && (a->r_pre || a->w_pre)))
        return TG_ERR_BAD_LAYOUT;
    const int xs = tg::dtype_size(a->xtype), bs = tg::dtype_size(a->btype);
    const int64_t gr = a->gate ? (a->gate_rows < T ? a->gate_rows : T) : T;
    const Span in[] = {span(a->x, T, D, a->ldx, xs), span(a->y, T, D, a->ldy, bs),
                       span1(a->gate, ceil_div(T, gr) * D, bs), span1(a->w_post, D, bs),
                       span1(a->w_pre, D, bs)};
    const Span out[] = {span(a->x_out, T, D, a->ldx_out, xs), span(a->h, T, D, a->ldh, bs),
                        span(a->hq, T, D, a->ldhq, 1),        span1(a->hs, T, 4),
                        span1(a->r_post, T, 4),               span1(a->r_pre, T, 4)};
    const bool in_place = a->x_out == a->x && a->ldx_out == a->ldx;
    for (int o = 0; o < 6; ++o) {
        for (int i = 0; i < 5; ++i)
            if (overlap(out[o], in[i]) && !(o == 0 && i == 0 && in_place))
                return TG_ERR_ALIAS;
        for (int q = 0; q < o; ++q)
            if (overlap(out[o], out[q]))
                return TG_ERR_ALIAS;
    }
    tg::NormParams p{};
    p.x = a->x;
    p.y = a->y;
    p.gate = a->gate;
    p.w_post = a->w_post;
    p.w_pre = a->w_pre;
    p.x_out = a->x_out;
    p.h = a->h;
    p.hq = a->hq;
    p.hs = a->hs;
    p.r_post = a->r_post;
    p.r_pre = a->r_pre;
    p.T = (int)T;
    p.ldx = a->ldx;
    p.ldy = a->ldy;
    p.ldxo = a->ldx_out;
    p.ldh = a->ldh;
    p.ldhq = a->ldhq;
    p.gate_rows = (int)gr;
    p.D = (int)D;
    p.post = a->post_norm != 0;
    p.alpha = a->alpha;
    p.eps = a->eps;
    const Pick k = pick_forward(D, a->xtype, a->btype);
    return tg::launch_kernel(k.kernel, ceil_div(T, k.rows), 1, k.threads, &p, (hipStream_t)stream,
                             "block_norm");
}

tg_status tg_block_norm_backward_workspace_size(const tg_block_norm_grad_args* a, size_t* bytes)
{
    if (!bytes)
        return TG_ERR_NULL_POINTER;
    if (tg_status s = check_grad(a))
        return s;
    *bytes = a->T == 0 || a->D == 0 ? 0 : grad_plan(*a).bytes;
    return TG_OK;
}

tg_status tg_block_norm_backward(const tg_block_norm_grad_args* a, void* workspace,
                                 size_t workspace_bytes, tg_stream_t stream)
{
    if (tg_status s = check_grad(a))
        return s;
    const int64_t T = a->T, D = a->D;
    if (T == 0 || D == 0)
        return TG_OK;
    if ((!a->dx_new && !a->dh) || (a->dh && (!a->x_new || !a->r_pre)) ||
        (a->y && a->post_norm && !a->r_post) ||
        (!a->dx && !a->dy && !a->dgate && !a->dw_post && !a->dw_pre))
        return TG_ERR_NULL_POINTER;
    if ((!a->y && (a->gate || a->w_post || a->dy || a->dgate || a->dw_post)) ||
        (!a->post_norm && a->w_post) || (a->dgate && !a->gate) || (a->dw_post && !a->w_post) ||
        (a->dw_pre && (!a->w_pre || !a->dh)))
        return TG_ERR_BAD_LAYOUT;
    const GradPlan g = grad_plan(*a);
    if (g.bytes > 0 &&
        (!workspace || workspace_bytes < g.bytes || ((uintptr_t)workspace & 15)))
        return TG_ERR_WORKSPACE;
    const int xs = tg::dtype_size(a->xtype), bs = tg::dtype_size(a->btype);
    const Span in[] = {span(a->x_new, T, D, a->ldx_new, xs), span(a->y, T, D, a->ldy, bs),
                       span1(a->gate, g.groups * D, bs),     span1(a->w_post, D, bs),
                       span1(a->w_pre, D, bs),               span1(a->r_post, T, 4),
                       span1(a->r_pre, T, 4),                span(a->dx_new, T, D, a->lddx_new, xs),
                       span(a->dh, T, D, a->lddh, bs)};
    const Span out[] = {span(a->dx, T, D, a->lddx, xs), span(a->dy, T, D, a->lddy, bs),
                        span1(a->dgate, g.groups * D, 4), span1(a->dw_post, D, 4),
                        span1(a->dw_pre, D, 4), span1(workspace, (int64_t)g.bytes, 1)};
    for (int o = 0; o < 6; ++o) {
        for (const Span& i : in)
            if (overlap(out[o], i))
                return TG_ERR_ALIAS;
        for (int q = 0; q < o; ++q)
            if (overlap(out[o], out[q]))
                return TG_ERR_ALIAS;
    }
    tg::NormGradParams p{};
    p.x_new = a->x_new;
    p.y = a->y;
    p.gate = a->gate;
    p.w_post = a->w_post;
    p.w_pre = a->w_pre;
    p.dx_new = a->dx_new;
    p.dh = a->dh;
    p.r_post = a->r_post;
    p.r_pre = a->r_pre;
    p.dx = a->dx;
    p.dy = a->dy;
    p.dgate = a->dgate;
    float* at = (float*)workspace;
    if (g.pre) {
        p.part_pre = at;
        at += g.P * g.Dp;
    }
    if (g.y)
        p.part_y = at;
    p.T = (int)T;
    p.ldx = a->ldx_new;
    p.ldy = a->ldy;
    p.lddxn = a->lddx_new;
    p.lddh = a->lddh;
    p.lddx = a->lddx;
    p.lddy = a->lddy;
    p.gate_rows = (int)g.gate_rows;
    p.rows = (int)g.rows;
    p.parts = (int)g.parts;
    p.D = (int)D;
    p.Dp = (int)g.Dp;
    p.post = a->y && a->post_norm;
    p.alpha = a->y ? a->alpha : 1.0f;  // without y, x' is x
    const Pick k = pick_backward(D, a->xtype, a->btype);
    if (tg_status s = tg::launch_kernel(k.kernel, g.P, 1, k.threads, &p, (hipStream_t)stream,
                                        "block_norm_grad"))
        return s;
    if (g.bytes == 0)
        return TG_OK;
    const bool by_group = a->dgate && g.parts > 0;
    tg::ColumnParams c{p.part_pre, p.part_y, a->dw_pre, a->dw_post, a->dgate, a->w_post,
                       a->gate,    g.P,      (int)g.parts, (int)D,  (int)g.Dp};
    const void* kc = by_types(TG_F32, a->btype, [](auto, auto B) {
        return (const void*)&tg::block_norm_columns_kernel<decltype(B)::value>;
    });
    return tg::launch_kernel(kc, ceil_div(g.Dp, 32), 2 + (by_group ? g.groups : 0), 256, &c,
                             (hipStream_t)stream, "block_norm_columns");
}

}  // extern "C"
