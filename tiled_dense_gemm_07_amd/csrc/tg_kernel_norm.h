// What stands between two blocks of a transformer, in one pass over memory
// (tg_block_norm) and its gradients (tg_block_norm_backward):
//   n = y r1, r1 = (mean y^2 + eps)^(-1/2)      (no post norm: n = y)
//   x' = alpha x + g n w_post                    rounded to the residual's type
//   h = x' r2 w_pre, r2 = (mean x'^2 + eps)^(-1/2)
// A team of TPR threads holds a row in registers (8 NC TPR elements at most).
// Sums, norms and every intermediate value are fp32; x' is rounded to its
// stored type before h is computed from it, so that h, and the gradients
// taken from the stored x', belong to the x' the caller holds.
#pragma once

#include "tg_rows.h"

namespace tg {

struct NormParams {
    const void *x, *y, *gate, *w_post, *w_pre;
    void *x_out, *h;
    int8_t* hq;
    float *hs, *r_post, *r_pre;
    int64_t T, ldx, ldy, ldxo, ldh, ldhq, gate_rows;
    int D;
    int post;
    float alpha, eps;
};

template <int XT, int BT, int NT, int TPR, int NC>
__global__ __attribute__((amdgpu_flat_work_group_size(NT, NT))) void block_norm_kernel(NormParams p)
{
    __shared__ u32 slots[3][16];
    const int t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * (NT / TPR) + threadIdx.x / TPR;
    if (row >= p.T)
        return;  // whole waves; rows share a workgroup only when TPR is one wave
    const char* x = elem_ptr<XT>(p.x, row * p.ldx);
    const float inv_d = 1.0f / (float)p.D;
    Raw8<XT> rx[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int at = 8 * (t + c * TPR);
        load8<XT>(rx[c], x, at, p.D - at);
    }
    if (p.y) {
        const char* y = elem_ptr<BT>(p.y, row * p.ldy);
        Raw8<BT> ry[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int at = 8 * (t + c * TPR);
            load8<BT>(ry[c], y, at, p.D - at);
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
        const char* gate =
            p.gate ? elem_ptr<BT>(p.gate, row / p.gate_rows * (int64_t)p.D) : nullptr;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int at = 8 * (t + c * TPR);
            const int left = p.D - at;
            float z[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                z[i] = get8<BT>(ry[c], i) * r1;
            if (p.w_post) {
                Raw8<BT> w;
                load8<BT>(w, p.w_post, at, left);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    z[i] *= get8<BT>(w, i);
            }
            if (gate) {
                Raw8<BT> g;
                load8<BT>(g, gate, at, left);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    z[i] *= get8<BT>(g, i);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                z[i] = __builtin_fmaf(p.alpha, get8<XT>(rx[c], i), z[i]);
            put8<XT>(rx[c], z);
            if (p.x_out)
                store8<XT>(const_cast<char*>(elem_ptr<XT>(p.x_out, row * p.ldxo)), at, left, rx[c]);
        }
    }
    if (!p.h && !p.hq)
        return;
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
    float h[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int at = 8 * (t + c * TPR);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            h[c][i] = get8<XT>(rx[c], i) * r2;
        if (p.w_pre) {
            Raw8<BT> w;
            load8<BT>(w, p.w_pre, at, p.D - at);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[c][i] *= get8<BT>(w, i);
        }
    }
    if (p.h) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int at = 8 * (t + c * TPR);
            Raw8<BT> r;
            put8<BT>(r, h[c]);
            store8<BT>(const_cast<char*>(elem_ptr<BT>(p.h, row * p.ldh)), at, p.D - at, r);
        }
    }
    if (p.hq) {
        u32 m[1] = {0};
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const u32 b = __builtin_bit_cast(u32, h[c][i]) & 0x7FFFFFFFu;
                if (8 * (t + c * TPR) + i < p.D)
                    m[0] = b > m[0] ? b : m[0];
            }
        row_all<MaxOp, TPR, 1>(m, slots[2]);
        RowLevels L;
        L.of_amax(m[0]);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            int q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                q[i] = L.level(h[c][i]);
            const int at = 8 * (t + c * TPR);
            store_levels(p.hq + row * p.ldhq, at, p.D - at, q);
        }
        if (t == 0)
            p.hs[row] = L.scale;
    }
}

// --------------------------------------------------------------------------
// Gradients.  With p = dh w_pre, u = x' r2, e = dx' + r2 p, q = g w_post n:
//   d  = e - r2 c2 u,              c2 = mean(p u)       (the gradient at x')
//   dx = alpha d
//   dy = r1 (d g w_post - n c1),   c1 = mean(d q) = mean(e q) - r2 c2 mean(u q)
//   dw_pre = sum dh u,  dgate = w_post sum_group d n,  dw_post = sum d g n
// The three means of a row are taken together, so a row needs one reduction.
// A workgroup takes consecutive rows: whole groups of rows that share a gate
// row, or a part of one group; it keeps the column sums in registers and
// leaves one partial row of each in the workspace, which
// block_norm_columns_kernel adds in a fixed order.
// --------------------------------------------------------------------------
struct NormGradParams {
    const void *x_new, *y, *gate, *w_post, *w_pre, *dx_new, *dh;
    const float *r_post, *r_pre;
    void *dx, *dy;
    float *dgate, *dw_post, *dw_pre;
    float *part_pre, *part_post, *part_gate;  // [P][Dp], or NULL
    int64_t T, ldx, ldy, lddxn, lddh, lddx, lddy, gate_rows;
    int64_t rows;  // rows for each workgroup (parts == 1), or of each part of a group
    int parts;     // parts of each group (1: whole groups)
    int D, Dp;
    int post;
    float alpha;
};

template <int XT, int BT, int TPR, int NC>
__global__ __attribute__((amdgpu_flat_work_group_size(TPR, TPR))) void
block_norm_grad_kernel(NormGradParams p)
{
    __shared__ u32 slots[2][48];
    const int t = threadIdx.x;
    const float inv_d = 1.0f / (float)p.D;
    const int64_t b = blockIdx.x;
    int64_t r0, r1;
    if (p.parts == 1) {
        r0 = b * p.rows;
        r1 = r0 + p.rows;
    } else {
        const int64_t base = b / p.parts * p.gate_rows;
        r0 = base + b % p.parts * p.rows;
        r1 = r0 + p.rows < base + p.gate_rows ? r0 + p.rows : base + p.gate_rows;
    }
    r1 = r1 < p.T ? r1 : p.T;

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
            load8<BT>(w1[c], p.w_post, at, p.D - at);
        if (p.w_pre)
            load8<BT>(w2[c], p.w_pre, at, p.D - at);
    }

    int64_t group = -1, group_end = r0;
    const auto flush = [&]() {  // end of the rows of one gate row in this workgroup
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int at = 8 * (t + c * TPR);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float s = a_g[c][i];
                a_post[c][i] = __builtin_fmaf(get8<BT>(g[c], i), s, a_post[c][i]);
                if (p.dgate && p.parts == 1 && at + i < p.D)
                    p.dgate[group * p.D + at + i] = get8<BT>(w1[c], i) * s;
                if (p.parts == 1)
                    a_g[c][i] = 0.0f;
            }
        }
    };

    for (int64_t row = r0; row < r1; ++row) {
        if (row >= group_end) {
            if (group >= 0)
                flush();
            group = p.gate ? row / p.gate_rows : 0;
            group_end = p.gate ? (group + 1) * p.gate_rows : p.T;
            if (p.gate) {
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const int at = 8 * (t + c * TPR);
                    load8<BT>(g[c], elem_ptr<BT>(p.gate, group * (int64_t)p.D), at, p.D - at);
                }
            }
        }
        Raw8<XT> rx[NC], rd[NC];
        Raw8<BT> ry[NC], rh[NC];
        const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int at = 8 * (t + c * TPR);
            const int left = p.D - at;
            if (p.dx_new)
                load8<XT>(rd[c], elem_ptr<XT>(p.dx_new, row * p.lddxn), at, left);
            else
                put8<XT>(rd[c], zero);
            if (p.dh) {
                load8<XT>(rx[c], elem_ptr<XT>(p.x_new, row * p.ldx), at, left);
                load8<BT>(rh[c], elem_ptr<BT>(p.dh, row * p.lddh), at, left);
            } else {
                put8<XT>(rx[c], zero);
                put8<BT>(rh[c], zero);
            }
            if (p.y)
                load8<BT>(ry[c], elem_ptr<BT>(p.y, row * p.ldy), at, left);
            else
                put8<BT>(ry[c], zero);
        }
        const float rr1 = p.post ? p.r_post[row] : 1.0f;
        const float rr2 = p.dh ? p.r_pre[row] : 0.0f;
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float pp = get8<BT>(rh[c], i) * get8<BT>(w2[c], i);
                const float u = get8<XT>(rx[c], i) * rr2;
                const float e = __builtin_fmaf(rr2, pp, get8<XT>(rd[c], i));
                const float q =
                    get8<BT>(g[c], i) * get8<BT>(w1[c], i) * (get8<BT>(ry[c], i) * rr1);
                s[0] = __builtin_fmaf(pp, u, s[0]);
                s[1] = __builtin_fmaf(e, q, s[1]);
                s[2] = __builtin_fmaf(u, q, s[2]);
            }
        row_sum<TPR, 3>(s, slots[row & 1]);
        const float k2 = rr2 * s[0] * inv_d;
        const float c1 = p.post ? (s[1] - k2 * s[2]) * inv_d : 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int at = 8 * (t + c * TPR);
            float dx[8], dy[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float dh = get8<BT>(rh[c], i);
                const float u = get8<XT>(rx[c], i) * rr2;
                const float e =
                    __builtin_fmaf(rr2, dh * get8<BT>(w2[c], i), get8<XT>(rd[c], i));
                const float d = __builtin_fmaf(-k2, u, e);
                const float n = get8<BT>(ry[c], i) * rr1;
                a_pre[c][i] = __builtin_fmaf(dh, u, a_pre[c][i]);
                a_g[c][i] = __builtin_fmaf(d, n, a_g[c][i]);
                dx[i] = p.alpha * d;
                dy[i] = rr1 * __builtin_fmaf(d, get8<BT>(g[c], i) * get8<BT>(w1[c], i), -n * c1);
            }
            if (p.dx) {
                Raw8<XT> r;
                put8<XT>(r, dx);
                store8<XT>(const_cast<char*>(elem_ptr<XT>(p.dx, row * p.lddx)), at, p.D - at, r);
            }
            if (p.dy) {
                Raw8<BT> r;
                put8<BT>(r, dy);
                store8<BT>(const_cast<char*>(elem_ptr<BT>(p.dy, row * p.lddy)), at, p.D - at, r);
            }
        }
    }
    if (group >= 0)
        flush();
    // partial column sums (Dp is D rounded up to whole chunks)
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int at = 8 * (t + c * TPR);
        if (at >= p.Dp)
            continue;
        const int64_t o = b * p.Dp + at;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const auto put = [&](float* to, const float (&v)[8]) {
                if (to)
                    *(f32x4*)(to + o + 4 * i) =
                        f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
            };
            put(p.part_pre, a_pre[c]);
            put(p.part_post, a_post[c]);
            put(p.part_gate, a_g[c]);
        }
    }
}

// Sums of the partial rows: blockIdx.y 0 and 1 take dw_pre and dw_post (P
// rows each), 2 + j the gate row j (its `parts` rows, times w_post).
struct ColumnParams {
    const float *part_pre, *part_post, *part_gate;
    float *dw_pre, *dw_post, *dgate;
    const void* w_post;
    int64_t P;
    int parts, D, Dp;
};

template <int BT>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256))) void
block_norm_columns_kernel(ColumnParams p)
{
    constexpr int CL = 16, RL = 16;  // threads along columns (4 each) and rows
    __shared__ f32x4 red[RL][CL];
    const int which = blockIdx.y;
    const float* from = which == 0 ? p.part_pre : (which == 1 ? p.part_post : p.part_gate);
    float* to = which == 0 ? p.dw_pre : (which == 1 ? p.dw_post : p.dgate);
    if (!from || !to)
        return;
    const int64_t group = which < 2 ? 0 : which - 2;
    const int64_t first = which < 2 ? 0 : group * p.parts;
    const int64_t rows = which < 2 ? p.P : p.parts;
    const int cl = threadIdx.x % CL, rl = threadIdx.x / CL;
    const int at = 4 * (blockIdx.x * CL + cl);
    f32x4 s = {0, 0, 0, 0};
    if (at < p.Dp)
        for (int64_t r = rl; r < rows; r += RL)
            s += *(const f32x4*)(from + (first + r) * p.Dp + at);
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
