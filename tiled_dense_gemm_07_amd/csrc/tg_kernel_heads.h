// Norms of query and key heads with the rotation to the token's position
// (tg_head_norm_rope), and their gradients.  For a head x of D values
//   n = x r, r = 1 / sqrt(mean(x^2) + eps),  y = n w,
//   out = y with pair i of its first R values turned by the token's angle i:
//     (a cos - b sin, a sin + b cos).
// Backward, dy being d(out) turned back:
//   dw = sum over tokens and heads of dy n,   p = dy w,   dx = r (p - n mean(p n)).
//
// Bound by memory: every value is read and written once.  A group of G lanes
// holds a head; lane j has pairs j V .. j V + V - 1 (and, where a head has more,
// those G V further): the V values of 16 bytes that are their first members and
// the V that are their second, so that a turn crosses no lanes (members half
// of R apart; neighbours are 2 V consecutive values).  Values past R form such
// pairs, too, half of what is left apart, and are not turned.  Where sizes do
// not divide so, V is 1.
// A unit is one token and 64 / G heads of one kind, to a wave; a wave takes
// consecutive units, so that a token's cosines and sines are loaded once and its
// position is uniform.
#pragma once

#include "tg_rows.h"

namespace tg {

struct HeadSide {
    const void* x;   // heads in: values of token t, head h at t xt + h xh
    const void* w;   // [D] or NULL
    const void* d;   // backward: gradients in
    void* out;       // forward: heads out; backward: gradients out
    float* part;     // backward: [blocks][D] partial sums of dw, or NULL
    int64_t xt, xh, dt, dh, ot, oh;
    int H;
    int units;       // of a token: ceil(H / (64 / G))
    int blocks;      // backward: workgroups of this side
};

struct HeadsParams {
    HeadSide s[2];  // queries, keys
    const float *cos, *sin;  // [P][R / 2]
    const int64_t* pos;      // [T] or NULL: token t is at position t
    int T, D, R, P;
    int interleaved;
    int per;  // units of a wave
    float eps;
};

// V values as stored, 16 bytes or one value.
template <int DT, int V>
struct HeadRaw {
    static constexpr int ES = DT == DT_F32 ? 4 : 2;
    static constexpr bool WIDE = V > 1;
    u32x4 v;  // WIDE, else v[0]

    __device__ __forceinline__ void load(const char* p, bool there)
    {
        struct __attribute__((packed, aligned(ES))) Any {
            u32x4 v;
        };
        v = u32x4{0, 0, 0, 0};
        if (!there)
            return;
        if constexpr (WIDE)
            v = ((const Any*)p)->v;
        else if constexpr (DT == DT_F32)
            v[0] = *(const u32*)p;
        else
            v[0] = *(const uint16_t*)p;
    }
    __device__ __forceinline__ void store(char* p) const
    {
        struct __attribute__((packed, aligned(ES))) Any {
            u32x4 v;
        };
        if constexpr (WIDE)
            ((Any*)p)->v = v;
        else if constexpr (DT == DT_F32)
            *(u32*)p = v[0];
        else
            *(uint16_t*)p = (uint16_t)v[0];
    }
    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (DT == DT_F32) {
            const u32 w = v[i];
            return __builtin_bit_cast(float, w);
        }
        const u32 w = v[i >> 1];
        if constexpr (DT == DT_BF16)
            return __builtin_bit_cast(float, (i & 1) ? (w & 0xFFFF0000u) : (w << 16));
        return (float)__builtin_bit_cast(_Float16, (uint16_t)((i & 1) ? (w >> 16) : w));
    }
    // Rounds once to the type (nearest even).
    __device__ __forceinline__ void put(const float* f)
    {
        if constexpr (DT == DT_F32) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[i] = __builtin_bit_cast(u32, f[i]);
        } else if constexpr (WIDE) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = pack2(f[2 * i], f[2 * i + 1], DT);
        } else {
            v[0] = cvt1(f[0], DT);
        }
    }
};

// Sum over the G lanes of a group, to each of them, in a fixed order.
template <int G>
__device__ __forceinline__ float group_sum(float f)
{
    u32 v = __builtin_bit_cast(u32, f);
    if constexpr (G >= 2)
        v = SumOp::of(v, dpp<0xB1>(v));
    if constexpr (G >= 4)
        v = SumOp::of(v, dpp<0x4E>(v));
    if constexpr (G >= 8)
        v = SumOp::of(v, dpp<0x141>(v));
    if constexpr (G >= 16)
        v = SumOp::of(v, dpp<0x140>(v));
    if constexpr (G >= 32) {
        const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = SumOp::of(s[0], s[1]);
    }
    if constexpr (G >= 64) {
        const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = SumOp::of(s[0], s[1]);
    }
    return __builtin_bit_cast(float, v);
}

// What a lane holds of a head of D values.
template <int DT, int V, int G, int NC, bool INTER>
struct HeadLane {
    using Raw = HeadRaw<DT, V>;
    static constexpr int ES = DT == DT_F32 ? 4 : 2;
    struct Values {
        Raw a[NC], b[NC];
    };
    struct Turn {
        float c[NC][V], s[NC][V];
    };
    int oa[NC], ob[NC];  // places of the first and the second members; past D: none
    int i0[NC];          // first pair
    int D, R;

    __device__ __forceinline__ HeadLane(const HeadsParams& p, int j) : D(p.D), R(p.R)
    {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int i = (j + c * G) * V;
            i0[c] = i;
            if (V == 1 ? p.interleaved != 0 : INTER) {
                oa[c] = 2 * i;
                ob[c] = 2 * i + V;
            } else if (i < R / 2) {
                oa[c] = i;
                ob[c] = i + R / 2;
            } else {
                const int half = (D - R + 1) / 2;
                const int t = i - R / 2;
                oa[c] = t < half ? R + t : D;
                ob[c] = R + half + t;
            }
        }
    }
    __device__ __forceinline__ void load(Values& v, const void* base, int64_t at, bool there) const
    {
        const char* p = (const char*)base + at * ES;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            v.a[c].load(p + oa[c] * ES, there && oa[c] < D);
            v.b[c].load(p + ob[c] * ES, there && ob[c] < D);
        }
    }
    __device__ __forceinline__ void store(void* base, int64_t at, const float (&f)[NC][2 * V]) const
    {
        char* p = (char*)base + at * ES;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            Raw r;
            if (oa[c] < D) {
                r.put(&f[c][0]);
                r.store(p + oa[c] * ES);
            }
            if (ob[c] < D) {
                r.put(&f[c][V]);
                r.store(p + ob[c] * ES);
            }
        }
    }
    // Values in the order of the lane's registers: pair i is (i, V + i), or
    // (2 i, 2 i + 1) where members are neighbours.
    static __device__ __forceinline__ void unpack(const Values& v, float (&f)[NC][2 * V])
    {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                f[c][i] = v.a[c].get(i);
                f[c][V + i] = v.b[c].get(i);
            }
    }
    static constexpr __device__ __forceinline__ int first(int i) { return INTER && V > 1 ? 2 * i : i; }
    static constexpr __device__ __forceinline__ int second(int i)
    {
        return INTER && V > 1 ? 2 * i + 1 : V + i;
    }
    // The token's cosines and sines; NaN for a position that the tables lack.
    __device__ __forceinline__ void turn(Turn& t, const HeadsParams& p, int token) const
    {
        const int64_t pos = p.pos ? p.pos[token] : token;
        const bool in = pos >= 0 && pos < p.P;
        const int64_t row = (in ? pos : 0) * (R / 2);
        struct __attribute__((packed, aligned(4))) Any {
            f32x4 v;
        };
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const bool turned = i0[c] < R / 2;
            const float *pc = p.cos + row + i0[c], *ps = p.sin + row + i0[c];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                t.c[c][i] = 1.0f;
                t.s[c][i] = 0.0f;
            }
            if (!turned)
                continue;
            if constexpr (V > 1) {
#pragma unroll
                for (int i = 0; i < V; i += 4) {
                    const f32x4 vc = ((const Any*)(pc + i))->v, vs = ((const Any*)(ps + i))->v;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        t.c[c][i + e] = in ? vc[e] : __builtin_nanf("");
                        t.s[c][i + e] = in ? vs[e] : __builtin_nanf("");
                    }
                }
            } else {
                t.c[c][0] = in ? *pc : __builtin_nanf("");
                t.s[c][0] = in ? *ps : __builtin_nanf("");
            }
        }
    }
};

__device__ __forceinline__ float head_root(float sum, int D, float eps)
{
    return 1.0f / sqrtf(sum / (float)D + eps);
}

template <int DT, int V, int G, int NC, bool INTER>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256))) void heads_kernel(HeadsParams p)
{
    using Lane = HeadLane<DT, V, G, NC, INTER>;
    constexpr int NG = 64 / G;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const Lane L(p, lane % G);
    const int units = p.s[0].units + p.s[1].units;
    const int64_t total = (int64_t)p.T * units;
    const int64_t u0 = ((int64_t)blockIdx.x * 4 + w) * p.per;
    if (u0 >= total)
        return;
    int token = (int)(u0 / units), at = (int)(u0 - (int64_t)token * units);
    const int64_t left = total - u0;
    const int n = left < p.per ? (int)left : p.per;
    typename Lane::Turn t;
    typename Lane::Values wv;
    int have = -1, side = -1;
    for (int i = 0; i < n; ++i) {
        const int sd = at >= p.s[0].units;
        const HeadSide& s = p.s[sd];
        const int h = (at - (sd ? p.s[0].units : 0)) * NG + lane / G;
        const bool there = h < s.H;
        typename Lane::Values xv;
        L.load(xv, s.x, token * s.xt + h * s.xh, there);
        if (have != token) {
            L.turn(t, p, token);
            have = token;
        }
        if (side != sd) {
            if (s.w)
                L.load(wv, s.w, 0, true);
            side = sd;
        }
        float x[NC][2 * V], wf[NC][2 * V];
        Lane::unpack(xv, x);
        Lane::unpack(wv, wf);
        float ss = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < 2 * V; ++e)
                ss += x[c][e] * x[c][e];
        const float r = head_root(group_sum<G>(ss), p.D, p.eps);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
#pragma unroll
            for (int e = 0; e < 2 * V; ++e)
                x[c][e] = s.w ? x[c][e] * r * wf[c][e] : x[c][e] * r;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float a = x[c][Lane::first(e)], b = x[c][Lane::second(e)];
                x[c][Lane::first(e)] = a * t.c[c][e] - b * t.s[c][e];
                x[c][Lane::second(e)] = a * t.s[c][e] + b * t.c[c][e];
            }
        }
        if (there)
            L.store(s.out, token * s.ot + h * s.oh, x);
        if (++at == units) {
            at = 0;
            ++token;
        }
    }
}

// Backward.  A workgroup takes the units of one side; its waves' sums of dw are
// added over the wave's heads, then over the waves, and written to its row of
// partial sums, which heads_sums_kernel adds in order.
constexpr int kHeadsGradWaves = 8;

template <int DT, int V, int G, int NC, bool INTER>
__global__ __attribute__((amdgpu_flat_work_group_size(64 * kHeadsGradWaves,
                                                      64 * kHeadsGradWaves))) void
heads_grad_kernel(HeadsParams p)
{
    constexpr int NW = kHeadsGradWaves;
    using Lane = HeadLane<DT, V, G, NC, INTER>;
    constexpr int NG = 64 / G;
    __shared__ float red[NW][NC * 2 * V * G];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int sd = (int)blockIdx.x >= p.s[0].blocks;
    const HeadSide& s = p.s[sd];
    const int block = (int)blockIdx.x - (sd ? p.s[0].blocks : 0);
    const Lane L(p, lane % G);
    const int64_t total = (int64_t)p.T * s.units;
    const int64_t u0 = ((int64_t)block * NW + w) * p.per;
    const int64_t left = total - u0;
    const int n = left <= 0 ? 0 : (left < p.per ? (int)left : p.per);
    int token = (int)(u0 / s.units), at = (int)(u0 - (int64_t)token * s.units);
    float acc[NC][2 * V];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 2 * V; ++e)
            acc[c][e] = 0.0f;
    typename Lane::Turn t;
    typename Lane::Values wv;
    if (s.w)
        L.load(wv, s.w, 0, true);
    int have = -1;
    for (int i = 0; i < n; ++i) {
        const int h = at * NG + lane / G;
        const bool there = h < s.H;
        typename Lane::Values xv, dv;
        L.load(xv, s.x, token * s.xt + h * s.xh, there);
        L.load(dv, s.d, token * s.dt + h * s.dh, there);
        if (have != token) {
            L.turn(t, p, token);
            have = token;
        }
        float x[NC][2 * V], d[NC][2 * V], wf[NC][2 * V];
        Lane::unpack(xv, x);
        Lane::unpack(dv, d);
        Lane::unpack(wv, wf);
        float ss = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < 2 * V; ++e)
                ss += x[c][e] * x[c][e];
        const float r = head_root(group_sum<G>(ss), p.D, p.eps);
        float dot = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float a = d[c][Lane::first(e)], b = d[c][Lane::second(e)];
                d[c][Lane::first(e)] = a * t.c[c][e] + b * t.s[c][e];
                d[c][Lane::second(e)] = b * t.c[c][e] - a * t.s[c][e];
            }
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) {
                x[c][e] *= r;
                acc[c][e] += there ? d[c][e] * x[c][e] : 0.0f;
                d[c][e] = s.w ? d[c][e] * wf[c][e] : d[c][e];
                dot += d[c][e] * x[c][e];
            }
        }
        const float m = group_sum<G>(dot) / (float)p.D;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < 2 * V; ++e)
                d[c][e] = r * (d[c][e] - x[c][e] * m);
        if (there)
            L.store(s.out, token * s.ot + h * s.oh, d);
        if (++at == s.units) {
            at = 0;
            ++token;
        }
    }
    if (!s.part)
        return;  // the whole workgroup
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) {
#pragma unroll
            for (int o = G; o < 64; o *= 2)
                acc[c][e] += __shfl_xor(acc[c][e], o);
            if (lane < G)
                red[w][(c * 2 * V + e) * G + lane] = acc[c][e];
        }
    __syncthreads();
    // value o of the head is in the lane and register that hold it; each thread
    // adds one, over the waves
    for (int i = threadIdx.x; i < NC * 2 * V * G; i += 64 * NW) {
        const int j = i % G, r = i / G;
        const Lane l(p, j);
        int o = p.D;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < 2 * V; ++e)
                if (r == c * 2 * V + e) {
                    const int base = e < V ? l.oa[c] : l.ob[c];
                    o = base < p.D ? base + e % V : p.D;
                }
        if (o < p.D) {
            float s8 = red[0][i];
#pragma unroll
            for (int v = 1; v < NW; ++v)
                s8 += red[v][i];
            s.part[(int64_t)block * p.D + o] = s8;
        }
    }
}

struct HeadSums {
    const float* part[2];
    float* out[2];
    int blocks[2];
    int D;
};

// dw of one side (blockIdx.y), 8 values to a workgroup: 32 rows of partial sums at
// a time, four of them in flight, then the 32 sums, in order.
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256))) void
heads_sums_kernel(HeadSums p)
{
    __shared__ float red[32][8];
    const int side = (int)blockIdx.y;
    const int c = threadIdx.x & 7, t = threadIdx.x >> 3;
    const int k = (int)blockIdx.x * 8 + c;
    const bool there = p.out[side] && k < p.D;
    const int n = there ? p.blocks[side] : 0;
    const float* part = p.part[side] + k;
    float s = 0.0f;
    for (int b0 = t; b0 < n; b0 += 128) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = b0 + 32 * i < n ? part[(int64_t)(b0 + 32 * i) * p.D] : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s += v[i];
    }
    red[t][c] = s;
    __syncthreads();
    if (t == 0 && there) {
#pragma unroll
        for (int i = 1; i < 32; ++i)
            s += red[i][c];
        p.out[side][k] = s;
    }
}

}  // namespace tg
