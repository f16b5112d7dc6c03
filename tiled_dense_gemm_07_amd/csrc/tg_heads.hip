// Entry points of the head norms with rotation and their gradients.  Arguments
// are checked before any HIP call; the kernel is chosen by the head's length and
// how it is rotated.
#include <hip/hip_runtime.h>

#include "tg_host.h"
#include "tg_kernel_heads.h"

namespace {

using tg::ceil_div;
using tg::overlap;
using tg::Span;
using tg::span;
using tg::span1;

constexpr int64_t kMaxHeadD = 1024;
constexpr int64_t kMaxT = 1 << 30;
constexpr int64_t kMaxHeads = 1 << 16;
constexpr int64_t kMaxWaves = 1 << 25;  // of the forward kernel: 2^31 threads

struct Pick {
    const void* kernel;
    int per_wave;  // heads of a unit
};

template <int DT, int V, int G, int NC, bool INTER, bool RAGGED>
Pick pick_of(bool grad)
{
    return {grad ? (const void*)&tg::heads_grad_kernel<DT, V, G, NC, INTER, RAGGED>
                 : (const void*)&tg::heads_kernel<DT, V, G, NC, INTER, RAGGED>,
            64 / G};
}

// far: one head to a unit.
template <int DT, bool INTER, bool RAGGED>
Pick pick_wide(int64_t chunks, bool grad, bool far)
{
    constexpr int V = 4;
    if constexpr (RAGGED && !INTER)
        if (chunks > 128)  // 1023 values, 6 of them turned
            return pick_of<DT, V, 64, 3, INTER, RAGGED>(grad);
    if (chunks > 64)
        return pick_of<DT, V, 64, 2, INTER, RAGGED>(grad);
    if (far || chunks > 32)
        return pick_of<DT, V, 64, 1, INTER, RAGGED>(grad);
    if (chunks <= 4)
        return pick_of<DT, V, 4, 1, INTER, RAGGED>(grad);
    if (chunks <= 8)
        return pick_of<DT, V, 8, 1, INTER, RAGGED>(grad);
    if (chunks <= 16)
        return pick_of<DT, V, 16, 1, INTER, RAGGED>(grad);
    return pick_of<DT, V, 32, 1, INTER, RAGGED>(grad);
}

// Four values to a load (eight of 16 bits, 8192 tokens of 40 heads of 128: forward
// 30.0 us either way, backward 50.2 and 45.1 with four, whose registers hold another
// wave to a SIMD).  Sizes that they do not divide cost shifts and selects (backward
// of 1537 tokens of 15 heads of 99 in fp32 11.2 us; 13.0 with one value at a time);
// heads of fewer than four values, or tables of fewer in all, take one at a time.
template <int DT>
Pick pick_type(int64_t D, int64_t R, int64_t P, bool inter, bool grad, bool far)
{
    constexpr int V = 4;
    if (D < V || (R > 0 && P * (R / 2) < V)) {
        const int64_t pairs = (D + 1) / 2;
        return pairs <= 64    ? pick_of<DT, 1, 64, 1, false, false>(grad)
               : pairs <= 128 ? pick_of<DT, 1, 64, 2, false, false>(grad)
               : pairs <= 256 ? pick_of<DT, 1, 64, 4, false, false>(grad)
                              : pick_of<DT, 1, 64, 8, false, false>(grad);
    }
    if (D % (2 * V) == 0 && R % (2 * V) == 0)
        return inter ? pick_wide<DT, true, false>(D / (2 * V), grad, far)
                     : pick_wide<DT, false, false>(D / (2 * V), grad, far);
    if (inter)
        return pick_wide<DT, true, true>(ceil_div(D, 2 * V), grad, far);
    return pick_wide<DT, false, true>(ceil_div(R / 2, V) + ceil_div((D - R + 1) / 2, V), grad, far);
}

// apart: the largest stride of heads; a unit's heads are within 32 bits of bytes, or
// one head is a unit.
Pick pick(int dt, int64_t D, int64_t R, int64_t P, bool inter, bool grad, int64_t apart)
{
    const auto of = [&](bool far) {
        if (dt == TG_F32)
            return pick_type<tg::DT_F32>(D, R, P, inter, grad, far);
        if (dt == TG_F16)
            return pick_type<tg::DT_F16>(D, R, P, inter, grad, far);
        return pick_type<tg::DT_BF16>(D, R, P, inter, grad, far);
    };
    const Pick k = of(false);
    const int64_t most = ((int64_t)1 << 32) / tg::dtype_size(dt) - kMaxHeadD;
    return (k.per_wave - 1) * apart > most ? of(true) : k;
}

int64_t larger(int64_t a, int64_t b) { return a > b ? a : b; }

// Byte range of T tokens of H heads of D values.  Tokens that hold their heads
// are the rows of a strided matrix, and so are heads that hold their tokens;
// other strides (of inputs only: values read more than once) count as the whole
// range.
Span heads_span(const void* p, int64_t T, int64_t H, int64_t D, int64_t st, int64_t sh, int es)
{
    const int64_t in_token = (H - 1) * sh + D, in_head = (T - 1) * st + D;
    if (T <= 1 || st >= in_token)
        return span(p, T, H > 0 ? in_token : 0, st, es);
    if (H <= 1 || sh >= in_head)
        return span(p, H, in_head, sh, es);
    return span1(p, H > 0 ? (T - 1) * st + in_token : 0, es);
}

// Heads of T tokens at given strides, and the range that heads_span has for them.
struct Heads {
    Span s;
    const char* p;
    int64_t H, st, sh;
};
Heads heads_at(const void* p, int64_t T, int64_t H, int64_t D, int64_t st, int64_t sh, int es)
{
    return {heads_span(p, T, H, D, st, sh, es), (const char*)p, H, st, sh};
}

// Whether two sets of heads have a value in common.  Ranges that overlap are looked at
// by heads where both have the same strides (heads of queries and keys in turn): head i
// of a and head j of b are o apart, j - i being what counts, and of the tokens the two
// that bring them nearest.
bool overlap(const Heads& a, const Heads& b, int64_t T, int64_t D, int es)
{
    if (!overlap(a.s, b.s))
        return false;
    const int64_t st = T <= 1 ? 0 : a.st, sh = a.H > 1 ? a.sh : b.sh;
    if ((T > 1 && a.st != b.st) || (a.H > 1 && b.H > 1 && a.sh != b.sh))
        return true;
    const int64_t width = D * es, step = st * es;
    for (int64_t h = 1 - a.H; h < b.H; ++h) {
        const int64_t o = (int64_t)((uintptr_t)b.p - (uintptr_t)a.p) + h * sh * es;
        int64_t t = step > 0 ? -o / step : 0;  // rounded towards zero: it or a neighbour
        for (int64_t n = t - 1; n <= t + 1; ++n) {
            const int64_t c = n < 1 - T ? 1 - T : (n > T - 1 ? T - 1 : n), off = o + c * step;
            if (off < width && off > -width)
                return true;
        }
    }
    return false;
}

// Strides are not negative, and offsets stay far below 63 bits.
bool bad_in(const void* p, int64_t T, int64_t H, int64_t st, int64_t sh)
{
    const double most = (double)((int64_t)1 << 48);
    return p && (st < 0 || sh < 0 || (double)T * (double)st > most || (double)H * (double)sh > most);
}
// Outputs: no two heads may overlap.
bool bad_out(const void* p, int64_t T, int64_t H, int64_t D, int64_t st, int64_t sh)
{
    if (!p || H == 0)
        return false;
    if (bad_in(p, T, H, st, sh) || (H > 1 && sh < D) || (T > 1 && st < D))
        return true;
    return T > 1 && H > 1 && st < (H - 1) * sh + D && sh < (T - 1) * st + D;
}

struct Common {
    int64_t T, Hq, Hk, D, R, P;
    int dtype;
    const void *q, *k, *w_q, *w_k, *cos, *sin, *positions;
    int64_t q_t, q_h, k_t, k_h;
};

template <class Args>
Common common(const Args& a)
{
    return {a.T,   a.Hq,  a.Hk,  a.D,   a.R,         a.P,   a.dtype, a.q,  a.k,
            a.w_q, a.w_k, a.cos, a.sin, a.positions, a.q_t, a.q_h,   a.k_t, a.k_h};
}

tg_status check_sizes(const Common& a)
{
    if (!tg::dtype_ok(a.dtype))
        return TG_ERR_BAD_DTYPE;
    if (a.T < 0 || a.T > kMaxT || a.Hq < 0 || a.Hk < 0 || a.Hq > kMaxHeads || a.Hk > kMaxHeads ||
        a.D < 1 || a.D > kMaxHeadD || a.R < 0 || a.R > a.D || a.R % 2 != 0 || a.P < 0 ||
        a.P > tg::kMaxDim || bad_in(a.q, a.T, a.Hq, a.q_t, a.q_h) ||
        bad_in(a.k, a.T, a.Hk, a.k_t, a.k_h))
        return TG_ERR_BAD_SHAPE;
    // token t at position t needs a table of T rows
    if (a.R > 0 && a.T > 0 && (a.P < 1 || (!a.positions && a.P < a.T)))
        return TG_ERR_BAD_SHAPE;
    return TG_OK;
}

tg_status check_inputs(const Common& a)
{
    if ((a.Hq > 0 && !a.q) || (a.Hk > 0 && !a.k) || (a.R > 0 && (!a.cos || !a.sin)))
        return TG_ERR_NULL_POINTER;
    return TG_OK;
}

struct Inputs {
    Heads heads[2];
    Span s[5];
};
Inputs input_spans(const Common& a)
{
    const int es = tg::dtype_size(a.dtype);
    return {{heads_at(a.q, a.T, a.Hq, a.D, a.q_t, a.q_h, es),
             heads_at(a.k, a.T, a.Hk, a.D, a.k_t, a.k_h, es)},
            {span1(a.w_q, a.D, es), span1(a.w_k, a.D, es), span1(a.cos, a.P * (a.R / 2), 4),
             span1(a.sin, a.P * (a.R / 2), 4), span1(a.positions, a.T, 8)}};
}

tg::HeadsParams params(const Common& a, float eps, int interleaved, int per_wave)
{
    tg::HeadsParams p{};
    const auto side = [&](tg::HeadSide& s, const void* x, const void* w, int64_t xt, int64_t xh,
                          int64_t H) {
        s.x = x;
        s.w = w;
        s.xt = xt;
        s.xh = xh;
        s.H = (int)H;
        s.units = (int)ceil_div(H, per_wave);
    };
    side(p.s[0], a.q, a.w_q, a.q_t, a.q_h, a.Hq);
    side(p.s[1], a.k, a.w_k, a.k_t, a.k_h, a.Hk);
    p.cos = (const float*)a.cos;
    p.sin = (const float*)a.sin;
    p.pos = (const int64_t*)a.positions;
    p.T = (int)a.T;
    p.D = (int)a.D;
    p.R = (int)a.R;
    p.P = (int)a.P;
    p.interleaved = interleaved != 0;
    p.eps = eps;
    p.inv_d = 1.0f / (float)a.D;
    return p;
}

// How a backward call shares the units: workgroups of a side.
// Workgroups at once on the card: two to a compute unit.
constexpr int64_t kGradGroups = 512;
struct GradPlan {
    Pick k;
    int64_t blocks[2];
    size_t bytes;
};

GradPlan grad_plan(const tg_head_norm_rope_grad_args& a)
{
    GradPlan g{};
    g.k = pick(a.dtype, a.D, a.R, a.P, a.interleaved != 0, true,
               larger(larger(larger(a.q_h, a.k_h), larger(a.dq_out_h, a.dk_out_h)),
                      larger(a.dq_h, a.dk_h)));
    const int64_t uq = a.T * ceil_div(a.Hq, g.k.per_wave), uk = a.T * ceil_div(a.Hk, g.k.per_wave);
    // All workgroups resident at once, shared out by the sides' units; a wave has at
    // least one unit.  (8192 tokens of 40 heads of 128 in bf16: 45 us; one workgroup
    // more, which runs alone after the others, 63; 1024 workgroups 48.)
    const int64_t all = uq + uk, W = tg::kHeadsGradWaves;
    const int64_t most = all < kGradGroups * W ? ceil_div(all, W) : kGradGroups;
    if (all > 0) {
        g.blocks[1] = uk > 0 ? (most * uk + all / 2) / all : 0;
        g.blocks[1] = uk > 0 && g.blocks[1] < 1 ? 1 : g.blocks[1];
        g.blocks[0] = uq > 0 ? most - g.blocks[1] : 0;
        g.blocks[0] = uq > 0 && g.blocks[0] < 1 ? 1 : g.blocks[0];
    }
    g.bytes = (size_t)((a.dw_q ? g.blocks[0] : 0) + (a.dw_k ? g.blocks[1] : 0)) * a.D * 4;
    return g;
}

}  // namespace

extern "C" {

tg_status tg_head_norm_rope(const tg_head_norm_rope_args* a, tg_stream_t stream)
{
    if (!a)
        return TG_ERR_NULL_POINTER;
    const Common c = common(*a);
    if (tg_status s = check_sizes(c))
        return s;
    if (bad_out(a->q_out, a->T, a->Hq, a->D, a->q_out_t, a->q_out_h) ||
        bad_out(a->k_out, a->T, a->Hk, a->D, a->k_out_t, a->k_out_h))
        return TG_ERR_BAD_SHAPE;
    if (a->T == 0 || a->Hq + a->Hk == 0)
        return TG_OK;
    if (tg_status s = check_inputs(c))
        return s;
    if ((a->Hq > 0 && !a->q_out) || (a->Hk > 0 && !a->k_out))
        return TG_ERR_NULL_POINTER;
    const int es = tg::dtype_size(a->dtype);
    const Inputs in = input_spans(c);
    const Heads out[] = {heads_at(a->q_out, a->T, a->Hq, a->D, a->q_out_t, a->q_out_h, es),
                         heads_at(a->k_out, a->T, a->Hk, a->D, a->k_out_t, a->k_out_h, es)};
    const bool same[] = {a->q_out == a->q && a->q_out_t == a->q_t && a->q_out_h == a->q_h,
                         a->k_out == a->k && a->k_out_t == a->k_t && a->k_out_h == a->k_h};
    for (int o = 0; o < 2; ++o) {
        for (int i = 0; i < 2; ++i)
            if (!(i == o && same[o]) && overlap(out[o], in.heads[i], a->T, a->D, es))
                return TG_ERR_ALIAS;
        for (const Span& i : in.s)
            if (overlap(out[o].s, i))
                return TG_ERR_ALIAS;
    }
    if (overlap(out[0], out[1], a->T, a->D, es))
        return TG_ERR_ALIAS;
    const Pick k = pick(a->dtype, a->D, a->R, a->P, a->interleaved != 0, false,
                        larger(larger(a->q_h, a->k_h), larger(a->q_out_h, a->k_out_h)));
    tg::HeadsParams p = params(c, a->eps, a->interleaved, k.per_wave);
    p.s[0].out = a->q_out;
    p.s[0].ot = a->q_out_t;
    p.s[0].oh = a->q_out_h;
    p.s[1].out = a->k_out;
    p.s[1].ot = a->k_out_t;
    p.s[1].oh = a->k_out_h;
    const int64_t units = p.s[0].units + p.s[1].units, total = units * a->T;
    int64_t per = total / 16384;
    per = per < 1 ? 1 : (per > units ? units : per);
    per = larger(per, ceil_div(total, kMaxWaves));
    p.per = (int)per;
    return tg::launch_kernel(k.kernel, ceil_div(total, 4 * per), 1, 256, &p, (hipStream_t)stream,
                             "heads");
}

tg_status tg_head_norm_rope_backward_workspace_size(const tg_head_norm_rope_grad_args* a,
                                                    size_t* bytes)
{
    if (!bytes || !a)
        return TG_ERR_NULL_POINTER;
    if (tg_status s = check_sizes(common(*a)))
        return s;
    *bytes = grad_plan(*a).bytes;
    return TG_OK;
}

tg_status tg_head_norm_rope_backward(const tg_head_norm_rope_grad_args* a, void* workspace,
                                     size_t workspace_bytes, tg_stream_t stream)
{
    if (!a)
        return TG_ERR_NULL_POINTER;
    const Common c = common(*a);
    if (tg_status s = check_sizes(c))
        return s;
    if (bad_in(a->dq_out, a->T, a->Hq, a->dq_out_t, a->dq_out_h) ||
        bad_in(a->dk_out, a->T, a->Hk, a->dk_out_t, a->dk_out_h) ||
        bad_out(a->dq, a->T, a->Hq, a->D, a->dq_t, a->dq_h) ||
        bad_out(a->dk, a->T, a->Hk, a->D, a->dk_t, a->dk_h))
        return TG_ERR_BAD_SHAPE;
    if ((a->dw_q && !a->w_q) || (a->dw_k && !a->w_k))
        return TG_ERR_BAD_LAYOUT;
    const hipStream_t hs = (hipStream_t)stream;
    const bool work = a->T > 0 && a->Hq + a->Hk > 0;
    if (!work && !a->dw_q && !a->dw_k)
        return TG_OK;
    const GradPlan g = grad_plan(*a);
    if (work) {
        if (tg_status s = check_inputs(c))
            return s;
        if ((a->Hq > 0 && (!a->dq_out || !a->dq)) || (a->Hk > 0 && (!a->dk_out || !a->dk)))
            return TG_ERR_NULL_POINTER;
        if (g.bytes > 0 && (!workspace || workspace_bytes < g.bytes || ((uintptr_t)workspace & 15)))
            return TG_ERR_WORKSPACE;
    }
    const int es = tg::dtype_size(a->dtype);
    const Inputs in = input_spans(c);
    // heads: those out, then those in
    const Heads heads[] = {heads_at(a->dq, a->T, a->Hq, a->D, a->dq_t, a->dq_h, es),
                           heads_at(a->dk, a->T, a->Hk, a->D, a->dk_t, a->dk_h, es),
                           in.heads[0], in.heads[1],
                           heads_at(a->dq_out, a->T, a->Hq, a->D, a->dq_out_t, a->dq_out_h, es),
                           heads_at(a->dk_out, a->T, a->Hk, a->D, a->dk_out_t, a->dk_out_h, es)};
    const Span more[] = {span1(a->dw_q, a->D, 4), span1(a->dw_k, a->D, 4),
                         span1(workspace, (int64_t)g.bytes, 1)};
    for (int o = 0; o < 2; ++o) {
        for (int i = o + 1; i < 6; ++i)
            if (overlap(heads[o], heads[i], a->T, a->D, es))
                return TG_ERR_ALIAS;
        for (const Span& i : in.s)
            if (overlap(heads[o].s, i))
                return TG_ERR_ALIAS;
    }
    for (int o = 0; o < 3; ++o) {
        for (const Heads& i : heads)
            if (overlap(more[o], i.s))
                return TG_ERR_ALIAS;
        for (const Span& i : in.s)
            if (overlap(more[o], i))
                return TG_ERR_ALIAS;
        for (int i = 0; i < o; ++i)
            if (overlap(more[o], more[i]))
                return TG_ERR_ALIAS;
    }
    float* at = (float*)workspace;
    tg::HeadSums sums{};
    sums.D = (int)a->D;
    sums.out[0] = a->dw_q;
    sums.out[1] = a->dw_k;
    if (work) {
        tg::HeadsParams p = params(c, a->eps, a->interleaved, g.k.per_wave);
        const auto side = [&](int i, const void* d, int64_t dt, int64_t dh, void* o, int64_t ot,
                              int64_t oh, const float* dw) {
            tg::HeadSide& s = p.s[i];
            s.d = d;
            s.dt = dt;
            s.dh = dh;
            s.out = o;
            s.ot = ot;
            s.oh = oh;
            s.blocks = (int)g.blocks[i];
            if (dw) {
                s.part = at;
                sums.part[i] = at;
                sums.blocks[i] = s.blocks;
                at += g.blocks[i] * a->D;
            }
        };
        side(0, a->dq_out, a->dq_out_t, a->dq_out_h, a->dq, a->dq_t, a->dq_h, a->dw_q);
        side(1, a->dk_out, a->dk_out_t, a->dk_out_h, a->dk, a->dk_t, a->dk_h, a->dw_k);
        if (tg_status s = tg::launch_kernel(g.k.kernel, g.blocks[0] + g.blocks[1], 1,
                                            64 * tg::kHeadsGradWaves, &p, hs, "heads_grad"))
            return s;
    }
    if (!a->dw_q && !a->dw_k)
        return TG_OK;
    return tg::launch_kernel((const void*)&tg::heads_sums_kernel, ceil_div(a->D, 8), 2, 256, &sums,
                             hs, "heads_sums");
}

}  // extern "C"
