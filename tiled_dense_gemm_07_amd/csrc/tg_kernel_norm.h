// What stands between two blocks of a transformer, in one pass over memory
// (tg_block_norm) and its gradients (tg_block_norm_backward):
//   n = y r1, r1 = (mean y^2 + eps)^(-1/2)      (no post norm: n = y)
//   x' = alpha x + g n w_post                    rounded to the residual's type
//   h = x' r2 w_pre, r2 = (mean x'^2 + eps)^(-1/2)
// A team of TPR threads holds a row in registers (8 NC TPR elements at most).
// Sums, norms and every intermediate value are fp32; x' is rounded to its
// stored type before h is computed from it, so that h, and the gradients
// taken from the stored x', belong to the x' the caller holds.
// 8-bit h has the exact levels of x' r2 w_pre: r2 cancels in them, so they are
// taken from x' w_pre (bf16: 16 bits, which fp32 divides exactly; else 64 bits next
// to a tie, tg_rows.h).  Against levels of h in fp32: bf16 8192 x 4096 and 4096 x
// 8192 the same time, fp32 x' with bf16 4096 x 8192 68.3 and 69.3 us, 2048 x 16384
// 85 and 92 (one workgroup to a unit, whose arithmetic no other one's loads hide).
// Bound by memory: bf16 8192 x 4096 with h 44.6 us in a trace (268 MB, 6.0 TB/s,
// part of it from the last-level cache; a large copy reaches 5.2); one row of
// 4096 2.7 us, which is launch, two reductions and latency.
#pragma once

#include "tg_rows.h"

namespace tg {

struct NormParams {
    const void *x, *y, *gate, *w_post, *w_pre;
    void *x_out, *h;
    int8_t* hq;
    float *hs, *r_post, *r_pre;
    int64_t ldx, ldy, ldxo, ldh, ldhq;
    int T, gate_rows, D;
    int post;
    float alpha, eps;
};

template <int XT, int BT, int NT, int TPR, int NC, bool ODD>
__global__ __attribute__((amdgpu_flat_work_group_size(NT, NT))) void block_norm_kernel(NormParams p)
{
    __shared__ u32 slots[3][16];
    __shared__ float rest[16];
    const int t = threadIdx.x % TPR;
    const int row = (int)blockIdx.x * (NT / TPR) +
                    __builtin_amdgcn_readfirstlane((int)(threadIdx.x / TPR));
    if (row >= p.T)
        return;  // whole waves; rows share a workgroup only when TPR is one wave
    const float inv_d = 1.0f / (float)p.D;
    const auto at = [&](int c) { return 8 * (t + c * TPR); };
    const Row<BT, ODD> w1(p.w_post, 0, 0, p.D), w2(p.w_pre, 0, 0, p.D);
    const Row<XT, ODD> x(p.x, row, p.ldx, p.D);
    Raw8<XT> rx[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c)
        x.load(rx[c], at(c));
    if (p.y) {
        const Row<BT, ODD> y(p.y, row, p.ldy, p.D);
        const Row<BT, ODD> gate(
            p.gate, __builtin_amdgcn_readfirstlane(p.gate ? row / p.gate_rows : 0), p.D, p.D);
        const Row<XT, ODD> xo(p.x_out, row, p.ldxo, p.D);
        Raw8<BT> ry[NC], rw[NC], rg[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c)
            y.load(ry[c], at(c));
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            w1.load(rw[c], at(c));
            gate.load(rg[c], at(c));
        }
        float r1 = 1.0f;
        if (p.post) {
            float s[1] = {0.0f};
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float v = get8<BT>(ry[c], i);
                    s[0] = __builtin_fmaf(v, v, s[0]);
                }
            row_sum<TPR, 1>(s, slots[0]);
            r1 = __builtin_amdgcn_rsqf(s[0] * inv_d + p.eps);
            if (p.r_post && t == 0)
                p.r_post[row] = r1;
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float z[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                z[i] = get8<BT>(ry[c], i) * r1;
            if (p.w_post) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    z[i] *= get8<BT>(rw[c], i);
            }
            if (p.gate) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    z[i] *= get8<BT>(rg[c], i);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                z[i] = __builtin_fmaf(p.alpha, get8<XT>(rx[c], i), z[i]);
            put8<XT>(rx[c], z);
            xo.store(rx[c], at(c));
        }
    }
    if (!p.h && !p.hq)
        return;
    Raw8<BT> rw[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c)
        w2.load(rw[c], at(c));
    float s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = get8<XT>(rx[c], i);
            s[0] = __builtin_fmaf(v, v, s[0]);
        }
    row_sum<TPR, 1>(s, slots[1]);
    const float r2 = __builtin_amdgcn_rsqf(s[0] * inv_d + p.eps);
    if (p.r_pre && t == 0)
        p.r_pre[row] = r2;
    if (p.h) {
        const Row<BT, ODD> out(p.h, row, p.ldh, p.D);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[i] = get8<XT>(rx[c], i) * r2;
            if (p.w_pre) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    h[i] *= get8<BT>(rw[c], i);
            }
            Raw8<BT> r;
            put8<BT>(r, h);
            out.store(r, at(c));
        }
    }
    if (p.hq) {
        // h = u f, f (1 to 2) being what r2 has beyond a power of two: the levels
        // are those of u = (x' pow) w, which r2 and its roundings have no part in
        const u32 rb = __builtin_bit_cast(u32, r2);
        const float pow = __builtin_bit_cast(float, rb & 0x7F800000u);
        const float f = __builtin_bit_cast(float, (rb & 0x007FFFFFu) | 0x3F800000u);
        const auto xp = [&](int c, int i) { return get8<XT>(rx[c], i) * pow; };
        const auto w = [&](int c, int i) { return p.w_pre ? get8<BT>(rw[c], i) : 1.0f; };
        const auto v = [&](int c, int i) { return xp(c, i) * w(c, i); };  // u in fp32
        const auto bits = [](float x) { return __builtin_bit_cast(u32, x) & 0x7FFFFFFFu; };
        // the largest |v|, of all and of each chunk (zeros past the end; NaN
        // there, with r2 infinite or NaN, only in a row without a norm)
        u32 m[1] = {0}, top[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            top[c] = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                top[c] = MaxOp::of(top[c], bits(v(c, i)));
            m[0] = MaxOp::of(top[c], m[0]);
        }
        const auto store = [&](float scale, const auto& levels) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                int q[8];
                levels(c, q);
                store_levels(p.hq + row * p.ldhq, at(c), p.D - at(c), q);
            }
            if (t == 0)
                p.hs[row] = scale;
        };
        if constexpr (XT == DT_BF16) {  // u has 16 bits
            row_all<MaxOp, TPR, 1>(m, slots[2]);
            RowLevels L;
            L.of_amax(m[0], f);
            store(L.scale, [&](int c, int (&q)[8]) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    q[i] = L.level(v(c, i));
            });
        } else {
            const auto unpack_again = [&] {
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    repack<XT>(rx[c]);
                    repack<BT>(rw[c]);
                }
            };
            unpack_again();
            float e = 0.0f;
            if constexpr (XT == DT_F16) {  // u has 22 bits, 127 u too many
                row_all<MaxOp, TPR, 1>(m, slots[2]);
            } else {
                // the largest |u| is among those that round to the largest |v|
                m[0] = wave_all<MaxOp>(m[0]);
                e = -__builtin_inff();
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    if (top[c] == m[0]) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (bits(v(c, i)) == m[0])
                                e = fmaxf(e, __builtin_fmaf(fabsf(xp(c, i)), fabsf(w(c, i)),
                                                            -fabsf(v(c, i))));
                    }
                e = __builtin_bit_cast(float, wave_all<MaxFloatOp>(__builtin_bit_cast(u32, e)));
                if constexpr (TPR > 64) {
                    if ((threadIdx.x & 63) == 0) {
                        slots[2][t >> 6] = m[0];
                        rest[t >> 6] = e;
                    }
                    __syncthreads();
#pragma unroll
                    for (int j = 0; j < TPR / 64; ++j)
                        m[0] = MaxOp::of(m[0], slots[2][j]);
                    e = -__builtin_inff();
#pragma unroll
                    for (int j = 0; j < TPR / 64; ++j)
                        e = slots[2][j] == m[0] ? fmaxf(e, rest[j]) : e;
                }
            }
            unpack_again();
            WideLevels L;
            L.of_amax(m[0], e, f);
            if (L.ok)
                store(L.scale, [&](int c, int (&q)[8]) {
                    L.levels([&](int i) { return xp(c, i); }, [&](int i) { return w(c, i); }, q);
                });
            else
                store(L.scale, [](int, int (&q)[8]) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        q[i] = 0;
                });
        }
    }
}

// --------------------------------------------------------------------------
// Gradients.  With p = dh w_pre, u = x' r2, e = dx' + r2 p, q = g w_post n:
//   d  = e - r2 c2 u,              c2 = mean(p u)       (the gradient at x')
//   dx = alpha d
//   dy = r1 (d g w_post - n c1),   c1 = mean(d q) = mean(e q) - r2 c2 mean(u q)
//   dw_pre = sum dh u,  dgate = w_post sum_group d n,  dw_post = sum d g n
// The three means of a row are taken together, so a row needs one reduction.
// A workgroup of NT threads holds NT / TPR teams, each with a row in flight
// and the next one's loads issued before this one's arithmetic.  It takes
// consecutive rows: whole groups of rows that share a gate row (parts == 0; a
// group to a team), or one of the `parts` of a group (its rows to the teams in
// turn).
// Column sums stay in registers over those rows (NC = 1: all but the fp32 / fp32
// kernel of 1024 threads, which spills 30), are added over the teams in LDS, and
// leave one partial row of each in the workspace, which block_norm_columns_kernel
// adds in a fixed order.
// Bound by memory: bf16 8192 x 4096 with 2048-token gates 83 us (403 MB and 8 MB
// of partial sums, 5.0 TB/s) and 5.5 us for the columns.  512 workgroups of half
// the threads took as long and left twice the partial sums (12.7 us for the
// columns).  The unpacked values of a row are not kept over its reduction but
// unpacked again (repack): kept, they spill.
// NC = 2 and 4 (D > 8192) hold 24 NC column sums a lane beside their row, in 128
// registers: 89 to 237 and 436 to 722 of them are spilled, and the row loop goes
// through scratch memory.  2048 x 16384: bf16 134 to 143 us (2.8 to 3.0 TB/s), fp32
// with bf16 210 to 220, fp32 474 to 486; 1024 x 32768: 447 to 468, 612 to 632 and 950
// to 975 (0.8 to 1 TB/s).  The sums would have to go to LDS, or a row to two
// workgroups.
// --------------------------------------------------------------------------
struct NormGradParams {
    const void *x_new, *y, *gate, *w_post, *w_pre, *dx_new, *dh;
    const float *r_post, *r_pre;
    void *dx, *dy;
    float* dgate;
    // [P][Dp] or NULL: sums of dh u; and of d n for each part of a group, or
    // of d g n where a workgroup takes whole groups (and writes dgate itself)
    float *part_pre, *part_y;
    int64_t ldx, ldy, lddxn, lddh, lddx, lddy;
    int T, gate_rows;
    int rows;   // rows of a workgroup
    int parts;  // workgroups of a group; 0: whole groups to a workgroup
    int D, Dp;
    int post;
    float alpha;
};

template <int XT, int BT, int NC>
struct GradRow {
    Raw8<XT> x[NC], d[NC];
    Raw8<BT> y[NC], h[NC];
    Raw8<BT> g[NC];  // the row's gate, if it opens a group
    float r1, r2;
};

template <int XT, int BT, int TPR, int NC, bool ODD>
__device__ __forceinline__ void load_grad_row(GradRow<XT, BT, NC>& R, const NormGradParams& p,
                                              int row, int t, int gate_row)
{
    // x' is read with dh only; a matrix that is not there reads as zeros
    const Row<XT, ODD> x(p.dh ? p.x_new : nullptr, row, p.ldx, p.D), d(p.dx_new, row, p.lddxn, p.D);
    const Row<BT, ODD> y(p.y, row, p.ldy, p.D), h(p.dh, row, p.lddh, p.D);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int at = 8 * (t + c * TPR);
        x.load(R.x[c], at);
        h.load(R.h[c], at);
        d.load(R.d[c], at);
        y.load(R.y[c], at);
    }
    if (gate_row >= 0) {
        const Row<BT, ODD> gate(p.gate, gate_row, p.D, p.D);
#pragma unroll
        for (int c = 0; c < NC; ++c)
            gate.load(R.g[c], 8 * (t + c * TPR));
    }
    R.r1 = p.post ? p.r_post[row] : 1.0f;
    R.r2 = p.dh ? p.r_pre[row] : 0.0f;
}

template <int XT, int BT, int NT, int TPR, int NC, int WPE, bool ODD>
__global__ __attribute__((amdgpu_flat_work_group_size(NT, NT), amdgpu_waves_per_eu(WPE, WPE))) void
block_norm_grad_kernel(NormGradParams p)
{
    constexpr int TEAMS = NT / TPR;
    __shared__ u32 slots[2][TEAMS][48];
    __shared__ float sums[TEAMS > 1 ? NT * 8 : 1];
    const int t = threadIdx.x % TPR;
    const int team = __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
    const float inv_d = 1.0f / (float)p.D;
    const bool whole = p.parts == 0;
    // Row numbers fit 32 bits.  The divisions are done on the vector ALU:
    // their results are read back as scalars, so that row addresses are.
    const int b = (int)blockIdx.x;
    const int per = whole ? p.gate_rows : 1;  // rows a team takes together
    int group = __builtin_amdgcn_readfirstlane(whole ? 0 : b / p.parts);
    int r0, r1;
    if (whole) {
        r0 = b * p.rows;
        r1 = r0 + p.rows;
        group = __builtin_amdgcn_readfirstlane(r0 / per) + team;
    } else {
        const int base = group * p.gate_rows;
        r0 = base + (b - group * p.parts) * p.rows;
        r1 = r0 + p.rows < base + p.gate_rows ? r0 + p.rows : base + p.gate_rows;
    }
    r1 = r1 < p.T ? r1 : p.T;

    // The team's rows: of a part, every TEAMS-th; of whole groups, the rows of
    // every TEAMS-th group in turn.  All teams take `count` steps, so that
    // they meet at the barriers; a step past r1 has no row.
    const int n = r1 > r0 ? r1 - r0 : 0;
    const int count =
        __builtin_amdgcn_readfirstlane(((n + per - 1) / per + TEAMS - 1) / TEAMS) * per;
    int row = r0 + team * per;
    int in_group = 0;  // row's place in its group (whole)

    float a_pre[NC][8], a_post[NC][8], a_g[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            a_pre[c][i] = a_post[c][i] = a_g[c][i] = 0.0f;

    // weights of this thread's columns (ones where there are none)
    const float one[8] = {1, 1, 1, 1, 1, 1, 1, 1};
    Raw8<BT> w1[NC], w2[NC], g[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int at = 8 * (t + c * TPR);
        put8<BT>(w1[c], one);
        put8<BT>(w2[c], one);
        put8<BT>(g[c], one);
        if (p.w_post)
            Row<BT, ODD>(p.w_post, 0, 0, p.D).load(w1[c], at);
        if (p.w_pre)
            Row<BT, ODD>(p.w_pre, 0, 0, p.D).load(w2[c], at);
    }
    if (!whole && p.gate && n > 0) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
            Row<BT, ODD>(p.gate, group, p.D, p.D).load(g[c], 8 * (t + c * TPR));
    }

    GradRow<XT, BT, NC> R;
    // The next row's loads in flight during this one's arithmetic, where 128
    // registers hold two rows; spilled ones cost far more than the overlap
    // gives (4096 x 8192 fp32 383 us so, 186 with one row at a time).  With NC > 1
    // not even one row fits (see above).
    constexpr bool AHEAD = NC == 1 && (TPR < 1024 || (XT != DT_F32 && !ODD));
    const bool own_gate = whole && p.gate;  // each group's gate with its first row
    if (AHEAD && row < r1)
        load_grad_row<XT, BT, TPR, NC, ODD>(R, p, row, t, own_gate ? group : -1);
    for (int i = 0; i < count; ++i) {
        const bool valid = row < r1;
        GradRow<XT, BT, NC> Q;
        if constexpr (AHEAD)
            Q = R;
        else  // a step past the end reads its last row again
            load_grad_row<XT, BT, TPR, NC, ODD>(Q, p, valid ? row : r1 - 1, t,
                                                own_gate && valid && in_group == 0 ? group : -1);
        if (own_gate && in_group == 0) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
                g[c] = Q.g[c];
        }
        const bool last = in_group + 1 == per;  // of its group, where that is whole
        const int next = last ? row + 1 + (TEAMS - 1) * per : row + 1;
        if (AHEAD && i + 1 < count && next < r1)
            load_grad_row<XT, BT, TPR, NC, ODD>(R, p, next, t,
                                                own_gate && last ? group + TEAMS : -1);
        float s[3] = {0.0f, 0.0f, 0.0f};
        if (valid) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float pp = get8<BT>(Q.h[c], k) * get8<BT>(w2[c], k);
                    const float u = get8<XT>(Q.x[c], k) * Q.r2;
                    const float e = __builtin_fmaf(Q.r2, pp, get8<XT>(Q.d[c], k));
                    const float q =
                        get8<BT>(g[c], k) * get8<BT>(w1[c], k) * (get8<BT>(Q.y[c], k) * Q.r1);
                    s[0] = __builtin_fmaf(pp, u, s[0]);
                    s[1] = __builtin_fmaf(e, q, s[1]);
                    s[2] = __builtin_fmaf(u, q, s[2]);
                }
        }
        row_sum<TPR, 3>(s, slots[i & 1][team]);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            repack<XT>(Q.x[c]);
            repack<XT>(Q.d[c]);
            repack<BT>(Q.y[c]);
            repack<BT>(Q.h[c]);
            repack<BT>(w1[c]);
            repack<BT>(w2[c]);
            repack<BT>(g[c]);
        }
        const int at_row = row, at_group = group;
        row = next;
        in_group = last ? 0 : in_group + 1;
        group = whole && last ? group + TEAMS : group;
        if (!valid)
            continue;
        const float k2 = Q.r2 * s[0] * inv_d;
        const float c1 = p.post ? (s[1] - k2 * s[2]) * inv_d : 0.0f;
        const Row<XT, ODD> rdx(p.dx, at_row, p.lddx, p.D);
        const Row<BT, ODD> rdy(p.dy, at_row, p.lddy, p.D);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int at = 8 * (t + c * TPR);
            float dx[8], dy[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float dh = get8<BT>(Q.h[c], k);
                const float u = get8<XT>(Q.x[c], k) * Q.r2;
                const float e =
                    __builtin_fmaf(Q.r2, dh * get8<BT>(w2[c], k), get8<XT>(Q.d[c], k));
                const float d = __builtin_fmaf(-k2, u, e);
                const float nn = get8<BT>(Q.y[c], k) * Q.r1;
                a_pre[c][k] = __builtin_fmaf(dh, u, a_pre[c][k]);
                a_g[c][k] = __builtin_fmaf(d, nn, a_g[c][k]);
                dx[k] = p.alpha * d;
                dy[k] = Q.r1 * __builtin_fmaf(d, get8<BT>(g[c], k) * get8<BT>(w1[c], k), -nn * c1);
            }
            Raw8<XT> ox;
            put8<XT>(ox, dx);
            rdx.store(ox, at);
            Raw8<BT> oy;
            put8<BT>(oy, dy);
            rdy.store(oy, at);
        }
        // the end of a group that this team holds whole
        if (whole && (last || at_row + 1 == r1)) {
            const Row<DT_F32, ODD> out(p.dgate, at_group, p.D, p.D);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    a_post[c][k] = __builtin_fmaf(get8<BT>(g[c], k), a_g[c][k], a_post[c][k]);
                    v[k] = get8<BT>(w1[c], k) * a_g[c][k];
                    a_g[c][k] = 0.0f;
                }
                Raw8<DT_F32> r;
                put8<DT_F32>(r, v);
                out.store(r, 8 * (t + c * TPR));
            }
        }
    }

    // partial column sums (Dp is D rounded up to whole chunks), over the
    // teams in order
    const auto leave = [&](float* to, float (&v)[NC][8]) {
        if (!to)
            return;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int at = 8 * (t + c * TPR);
            if constexpr (TEAMS > 1) {
                __syncthreads();
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    sums[k * NT + threadIdx.x] = v[c][k];
                __syncthreads();
                if (team == 0) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        for (int j = 1; j < TEAMS; ++j)
                            v[c][k] += sums[k * NT + j * TPR + t];
                }
            }
            if (team == 0 && at < p.Dp) {
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    *(f32x4*)(to + (int64_t)b * p.Dp + at + 4 * k) =
                        f32x4{v[c][4 * k], v[c][4 * k + 1], v[c][4 * k + 2], v[c][4 * k + 3]};
            }
        }
    };
    leave(p.part_pre, a_pre);
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            a_g[c][k] = whole ? a_post[c][k] : a_g[c][k];
    leave(p.part_y, a_g);
}

// Sums of the partial rows: blockIdx.y 0 takes dw_pre, 1 takes dw_post (the
// sums of d n of a part times its group's gate), 2 + j the gate row j (its
// `parts` rows, times w_post).
struct ColumnParams {
    const float *part_pre, *part_y;
    float *dw_pre, *dw_post, *dgate;
    const void *w_post, *gate;
    int64_t P;
    int parts, D, Dp;
};

template <int BT>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256))) void
block_norm_columns_kernel(ColumnParams p)
{
    constexpr int CL = 8, RL = 32;  // threads along columns (4 each) and rows
    __shared__ f32x4 red[RL][CL];
    const int which = blockIdx.y;
    const float* from = which == 0 ? p.part_pre : p.part_y;
    float* to = which == 0 ? p.dw_pre : (which == 1 ? p.dw_post : p.dgate);
    if (!from || !to)
        return;
    const int64_t group = which < 2 ? 0 : which - 2;
    const int64_t first = which < 2 ? 0 : group * p.parts;
    const int64_t rows = which < 2 ? p.P : p.parts;
    const bool weigh = which == 1 && p.parts > 0 && p.gate;
    const int cl = threadIdx.x % CL, rl = threadIdx.x / CL;
    const int at = 4 * (blockIdx.x * CL + cl);
    f32x4 s = {0, 0, 0, 0};
    if (at < p.Dp && weigh) {
        // past the end of a gate row its last element again: no branch, and
        // those sums are not stored
#pragma unroll 4
        for (int r = rl; r < (int)rows; r += RL) {
            const f32x4 v = *(const f32x4*)(from + (int64_t)r * p.Dp + at);
            const char* gate = elem_ptr<BT>(p.gate, (int64_t)(r / p.parts) * p.D);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int col = at + i < p.D ? at + i : p.D - 1;
                Raw8<BT> g;
                if constexpr (BT == DT_F32)
                    g.v[0][0] = ((const u32*)gate)[col];
                else
                    g.v[0][0] = ((const uint16_t*)gate)[col];
                s[i] = __builtin_fmaf(get8<BT>(g, 0), v[i], s[i]);
            }
        }
    } else if (at < p.Dp) {
#pragma unroll 4
        for (int64_t r = rl; r < rows; r += RL)
            s += *(const f32x4*)(from + (first + r) * p.Dp + at);
    }
    red[rl][cl] = s;
    __syncthreads();
    if (rl == 0 && at < p.Dp) {
#pragma unroll
        for (int j = 1; j < RL; ++j)
            s += red[j][cl];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (at + i < p.D) {
                float v = s[i];
                if (which >= 2 && p.w_post) {
                    Raw8<BT> w;
                    load8<BT>(w, p.w_post, at + i, 1);
                    v *= get8<BT>(w, 0);
                }
                to[group * p.D + at + i] = v;
            }
    }
}

}  // namespace tg
