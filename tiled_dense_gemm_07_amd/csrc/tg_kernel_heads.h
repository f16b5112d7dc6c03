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
// those G V further): the V values that are their first members and the V that are
// their second, so that a turn crosses no lanes (members half of R apart;
// neighbours are 2 V consecutive values).  Values past R form such pairs, too, half
// of what is left apart, and are not turned.  RAGGED: sizes that V does not divide; the
// last chunk of a run has fewer pairs, and a chunk that would end past the head is
// loaded that much lower and shifted.
// A unit is one token and 64 / G heads of one kind, to a wave, so that a token's
// position is uniform and what addresses it scalar.
// Measured (bf16, 8192 tokens of 32 + 8 heads of 128, slices of one buffer): forward
// 30 us (5.6 TB/s, what a large copy reaches), backward 45 us and 4.6 for the sums of
// dw (5.6 TB/s); one token 2.5 us, which is launch and latency.
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
    float eps, inv_d;  // inv_d: 1 / D
};

// V values as stored (one, or whole words).
template <int DT, int V>
struct HeadRaw {
    static constexpr int ES = DT == DT_F32 ? 4 : 2;
    static constexpr bool WIDE = V > 1;
    static constexpr int NW = WIDE ? V * ES / 4 : 1;
    typedef __attribute__((ext_vector_type(NW))) u32 Words;
    struct __attribute__((packed, aligned(ES))) Any {
        Words v;
    };
    u32 v[NW];

    __device__ __forceinline__ void load(const char* p)
    {
        Words w;
        if constexpr (WIDE || DT == DT_F32)
            w = ((const Any*)p)->v;
        else
            w = (Words)(u32) * (const uint16_t*)p;
#pragma unroll
        for (int i = 0; i < NW; ++i)
            v[i] = w[i];
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < NW; ++i)
            v[i] = 0;
    }
    __device__ __forceinline__ void store(char* p) const
    {
        if constexpr (WIDE || DT == DT_F32) {
            Words w;
#pragma unroll
            for (int i = 0; i < NW; ++i)
                w[i] = v[i];
            ((Any*)p)->v = w;
        } else {
            *(uint16_t*)p = (uint16_t)v[0];
        }
    }
    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (DT == DT_F32)
            return __builtin_bit_cast(float, v[i]);
        const u32 w = v[i >> 1];
        if constexpr (DT == DT_BF16)
            return __builtin_bit_cast(float, (i & 1) ? (w & 0xFFFF0000u) : (w << 16));
        return (float)__builtin_bit_cast(_Float16, (uint16_t)((i & 1) ? (w >> 16) : w));
    }
    // Rounds once to the type (nearest even).
    __device__ __forceinline__ void put(const float (&f)[V])
    {
        if constexpr (DT == DT_F32) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[i] = __builtin_bit_cast(u32, f[i]);
        } else if constexpr (WIDE) {
#pragma unroll
            for (int i = 0; i < NW; ++i)
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
template <int DT, int V, int G, int NC, bool INTER, bool RAGGED>
struct HeadLane {
    using Raw = HeadRaw<DT, V>;
    static constexpr int ES = DT == DT_F32 ? 4 : 2;
    static constexpr int NG = 64 / G;
    struct Values {
        Raw a[NC], b[NC];
    };
    struct Turn {
        float c[NC][V], s[NC][V];
    };
    int oa[NC], ob[NC];  // places of the first and the second members
    int na[NC], nb[NC];  // how many there are: V or 0, RAGGED any
    int i0[NC];          // first pair
    int D, R;
    int g;  // which of the unit's heads

    __device__ __forceinline__ HeadLane(const HeadsParams& p, int lane)
        : D(p.D), R(p.R), g(lane / G)
    {
        // chunks of pairs that are turned, then of those that are not (halves)
        const int turned = (R / 2 + V - 1) / V, half = (D - R + 1) / 2;
        const auto count = [](int n) { return n < 0 ? 0 : (n < V ? n : V); };
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int j = lane % G + c * G;
            i0[c] = j * V;
            if (V == 1 ? p.interleaved != 0 : INTER) {
                oa[c] = 2 * V * j;
                ob[c] = 2 * V * j + V;
                na[c] = count(D - oa[c]);
                nb[c] = count(D - ob[c]);
            } else if (j < turned) {
                oa[c] = V * j;
                ob[c] = V * j + R / 2;
                na[c] = nb[c] = count(R / 2 - V * j);
            } else {
                const int t = V * (j - turned);
                oa[c] = R + t;
                ob[c] = R + half + t;
                na[c] = count(half - t);
                nb[c] = count(D - R - half - t);
                i0[c] = R / 2 + t;
            }
        }
    }
    // The first of a unit's heads: `at` is the unit's place in its token.
    static __device__ __forceinline__ char* first_head(const void* base, int64_t st, int64_t sh,
                                                       int token, int at)
    {
        return (char*)base + (token * st + (int64_t)(at * NG) * sh) * ES;
    }
    // Bytes from there to the lane's head; the host sees to it that they fit.
    static __device__ __forceinline__ u32 head_offset(int64_t sh, int head)
    {
        return (u32)head * (u32)sh * (u32)ES;
    }
    // Where the chunk at o of n values is loaded from; n == 0: the head's first values,
    // which have no part in anything.
    __device__ __forceinline__ int from(int o, int n) const
    {
        if (n == 0)
            return 0;
        return RAGGED && o > D - V ? D - V : o;
    }
    // No load stands in a branch, so that all of them are in flight together.
    __device__ __forceinline__ void load(Values& v, const char* p, u32 off) const
    {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            v.a[c].load(p + (off + (u32)(from(oa[c], na[c]) * ES)));
            v.b[c].load(p + (off + (u32)(from(ob[c], nb[c]) * ES)));
        }
    }
    __device__ __forceinline__ void store(char* p, u32 off, const float (&f)[NC][2 * V]) const
    {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            store_chunk<0>(p + (off + (u32)(oa[c] * ES)), f[c], na[c]);
            store_chunk<V>(p + (off + (u32)(ob[c] * ES)), f[c], nb[c]);
        }
    }
    // Values AT .. of f: n of them.
    template <int AT>
    static __device__ __forceinline__ void store_chunk(char* to, const float (&f)[2 * V], int n)
    {
        if (n == V) {
            Raw r;
            float v[V];
#pragma unroll
            for (int e = 0; e < V; ++e)
                v[e] = f[AT + e];
            r.put(v);
            r.store(to);
        } else if constexpr (RAGGED) {
#pragma unroll
            for (int e = 0; e < V - 1; ++e)
                if (e < n) {
                    HeadRaw<DT, 1> r;
                    const float v[1] = {f[AT + e]};
                    r.put(v);
                    r.store(to + e * ES);
                }
        }
    }
    // Values in the order of the lane's registers: pair i is (i, V + i), or
    // (2 i, 2 i + 1) where members are neighbours.  RAGGED: shifted down to their
    // places, zeros where there are none.
    __device__ __forceinline__ void unpack(const Values& v, float (&f)[NC][2 * V]) const
    {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                f[c][i] = v.a[c].get(i);
                f[c][V + i] = v.b[c].get(i);
            }
            if constexpr (RAGGED) {
                shift<0>(f[c], na[c] ? oa[c] - from(oa[c], na[c]) : 0, na[c]);
                shift<V>(f[c], nb[c] ? ob[c] - from(ob[c], nb[c]) : 0, nb[c]);
            }
        }
    }
    // Values AT .. AT + V - 1 of f moved down by `by`, zeros from n on (V is 4).
    template <int AT, int N>
    static __device__ __forceinline__ void shift(float (&f)[N], int by, int n)
    {
        static_assert(!RAGGED || V == 4, "two steps of a shift");
        const bool one = by & 1, two = by & 2;
        float v[V];  // by value: a choice between elements of f would keep it in memory
#pragma unroll
        for (int e = 0; e < V; ++e)
            v[e] = f[AT + e];
#pragma unroll
        for (int e = 0; e + 1 < V; ++e) {
            const float lo = v[e], hi = v[e + 1];
            v[e] = one ? hi : lo;
        }
#pragma unroll
        for (int e = 0; e + 2 < V; ++e) {
            const float lo = v[e], hi = v[e + 2];
            v[e] = two ? hi : lo;
        }
#pragma unroll
        for (int e = 0; e < V; ++e)
            f[AT + e] = e < n ? v[e] : 0.0f;
    }
    static constexpr __device__ __forceinline__ int first(int i) { return INTER && V > 1 ? 2 * i : i; }
    static constexpr __device__ __forceinline__ int second(int i)
    {
        return INTER && V > 1 ? 2 * i + 1 : V + i;
    }
    // Sum over the head of x y.
    __device__ __forceinline__ float dot(const float (&x)[NC][2 * V],
                                         const float (&y)[NC][2 * V]) const
    {
        float t = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float ta = 0.0f, tb = 0.0f;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                ta = __builtin_fmaf(x[c][e], y[c][e], ta);
                tb = __builtin_fmaf(x[c][V + e], y[c][V + e], tb);
            }
            // not RAGGED: V > 1 both are there or neither, and what was read in
            // their place counts for nothing
            if constexpr (RAGGED)
                t += ta + tb;
            else if constexpr (V > 1)
                t += na[c] ? ta + tb : 0.0f;
            else
                t += (na[c] ? ta : 0.0f) + (nb[c] ? tb : 0.0f);
        }
        return group_sum<G>(t);
    }
    // 1 / sqrt(mean of x^2 + eps): the instruction is good to a step, but takes
    // subnormal numbers for zero.
    __device__ __forceinline__ float root(const float (&x)[NC][2 * V], const HeadsParams& p) const
    {
        const float v = dot(x, x) * p.inv_d + p.eps;
        const bool tiny = v < 0x1p-96f;
        return __builtin_amdgcn_rsqf(tiny ? v * 0x1p96f : v) * (tiny ? 0x1p48f : 1.0f);
    }
    // The weights, ones where there are none.
    __device__ __forceinline__ void weights(float (&w)[NC][2 * V], const void* base) const
    {
        if (base) {
            Values v;
            load(v, (const char*)base, 0);
            unpack(v, w);
            return;
        }
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < 2 * V; ++e)
                w[c][e] = 1.0f;
    }
    // The token's position: read-only to the kernel, hence by the scalar path, whose
    // waits are apart from those of vector loads and stores.
    static __device__ __forceinline__ int64_t position(const HeadsParams& p, int token)
    {
        typedef const __attribute__((address_space(4))) int64_t Const;
        return p.pos ? ((Const*)(uintptr_t)p.pos)[token] : token;
    }
    // Its cosines and sines as loaded, and as they are used: NaN for a position that
    // the tables lack, RAGGED no turn for what stands past a run's end in its last chunk.
    __device__ __forceinline__ void load(Turn& t, const HeadsParams& p, int64_t pos) const
    {
        if (R == 0)
            return;
        const int64_t row = (pos >= 0 && pos < p.P ? pos : 0) * (R / 2);
        const char *pc = (const char*)(p.cos + row), *ps = (const char*)(p.sin + row);
        typedef __attribute__((ext_vector_type(V))) float Vec;
        struct __attribute__((packed, aligned(4))) Any {
            Vec v;
        };
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            // RAGGED: on into the next row, but not past the tables
            const int off = ((i0[c] < R / 2 ? i0[c] : 0) - lower(p, row, c)) * 4;
            const Vec vc = ((const Any*)(pc + off))->v, vs = ((const Any*)(ps + off))->v;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                t.c[c][i] = vc[i];
                t.s[c][i] = vs[i];
            }
        }
    }
    // By how much lower the chunk's cosines are loaded so as to end with the table.
    __device__ __forceinline__ int lower(const HeadsParams& p, int64_t row, int c) const
    {
        if (!RAGGED)
            return 0;
        const int64_t end = row + (i0[c] < R / 2 ? i0[c] : 0) + V - (int64_t)p.P * (R / 2);
        return end > 0 ? (int)end : 0;
    }
    __device__ __forceinline__ void settle(Turn& t, const HeadsParams& p, int64_t pos) const
    {
        const bool in = pos >= 0 && pos < p.P;
        if (!RAGGED && in)
            return;
        const int n = R / 2;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if constexpr (RAGGED) {
                const int by = lower(p, (in ? pos : 0) * n, c);
                shift<0>(t.c[c], by, V);
                shift<0>(t.s[c], by, V);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const bool turned = (RAGGED ? i0[c] + i : i0[c]) < n;
                t.c[c][i] = turned ? (in ? t.c[c][i] : __builtin_nanf("")) : 1.0f;
                t.s[c][i] = turned ? (in ? t.s[c][i] : __builtin_nanf("")) : 0.0f;
            }
        }
    }
    // Turned to the token's position, or back.  Values past R stay as they are: times
    // one and zero an infinity or NaN would spread to the other of its pair.  Chunks are
    // turned whole or not at all but where neighbours are pairs and R ends in one.
    template <bool BACK>
    __device__ __forceinline__ void turn(float (&x)[NC][2 * V], const Turn& t) const
    {
        constexpr bool PART = RAGGED && INTER;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (!PART && i0[c] >= R / 2)
                continue;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float a = x[c][first(e)], b = x[c][second(e)];
                const float k = t.c[c][e], n = BACK ? -t.s[c][e] : t.s[c][e];
                const bool on = !PART || i0[c] + e < R / 2;
                x[c][first(e)] = on ? a * k - b * n : a;
                x[c][second(e)] = on ? a * n + b * k : b;
            }
        }
    }
};

template <int DT, int V, int G, int NC, bool INTER, bool RAGGED>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256))) void heads_kernel(HeadsParams p)
{
    using Lane = HeadLane<DT, V, G, NC, INTER, RAGGED>;
    constexpr int NG = 64 / G;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const Lane L(p, threadIdx.x & 63);
    const int units = p.s[0].units + p.s[1].units;
    const int64_t total = (int64_t)p.T * units;
    const int64_t u0 = ((int64_t)blockIdx.x * 4 + w) * p.per;
    if (u0 >= total)
        return;
    int token = (int)(u0 / units), at = (int)(u0 - (int64_t)token * units);
    const int64_t left = total - u0;
    const int n = left < p.per ? (int)left : p.per;
    typename Lane::Turn t;
    float wf[NC][2 * V];
    int have = -1, side = -1;
    for (int i = 0; i < n; ++i) {
        const int sd = at >= p.s[0].units;
        const HeadSide& s = p.s[sd];
        const int a = at - (sd ? p.s[0].units : 0);
        const bool there = a * NG + L.g < s.H;
        typename Lane::Values xv;
        L.load(xv, Lane::first_head(s.x, s.xt, s.xh, token, a),
               Lane::head_offset(s.xh, there ? L.g : 0));
        if (have != token) {
            const int64_t pos = Lane::position(p, token);
            L.load(t, p, pos);
            L.settle(t, p, pos);
            have = token;
        }
        if (side != sd) {
            L.weights(wf, s.w);
            side = sd;
        }
        float x[NC][2 * V];
        L.unpack(xv, x);
        const float r = L.root(x, p);
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < 2 * V; ++e)
                x[c][e] = x[c][e] * r * wf[c][e];
        L.template turn<false>(x, t);
        if (there)
            L.store(Lane::first_head(s.out, s.ot, s.oh, token, a), Lane::head_offset(s.oh, L.g), x);
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

template <int DT, int V, int G, int NC, bool INTER, bool RAGGED>
__global__ __attribute__((amdgpu_flat_work_group_size(64 * kHeadsGradWaves,
                                                      64 * kHeadsGradWaves))) void
heads_grad_kernel(HeadsParams p)
{
    constexpr int NW = kHeadsGradWaves;
    using Lane = HeadLane<DT, V, G, NC, INTER, RAGGED>;
    constexpr int NG = 64 / G;
    __shared__ float red[NW][NC * 2 * V * G];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int sd = (int)blockIdx.x >= p.s[0].blocks;
    const HeadSide& s = p.s[sd];
    const int block = (int)blockIdx.x - (sd ? p.s[0].blocks : 0);
    const Lane L(p, lane);
    float acc[NC][2 * V], wf[NC][2 * V];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 2 * V; ++e)
            acc[c][e] = 0.0f;
    L.weights(wf, s.w);
    // A unit's loads are issued a unit ahead, all together and before the stores of
    // the one at hand: vector loads and stores are waited for in the order in which
    // they were issued.  Its position is read two units ahead.
    struct Unit {
        typename Lane::Values x, d;
        typename Lane::Turn t;
        int64_t pos;
        int token, at;
    };
    const auto fetch = [&](Unit& n) {
        const int g = n.at * NG + L.g < s.H ? L.g : 0;
        L.load(n.x, Lane::first_head(s.x, s.xt, s.xh, n.token, n.at), Lane::head_offset(s.xh, g));
        L.load(n.d, Lane::first_head(s.d, s.dt, s.dh, n.token, n.at), Lane::head_offset(s.dh, g));
        L.load(n.t, p, n.pos);
    };
    // Unit u of this side is unit u % units of token u / units; a step adds
    // (step_t, step_a) to the two.
    const int step = s.blocks * NW, step_t = step / s.units, step_a = step - step_t * s.units;
    int token = (block * NW + w) / s.units, at = (block * NW + w) - token * s.units;
    const auto next = [&](Unit& n) {
        n.token = token < p.T ? token : p.T - 1;
        n.at = token < p.T ? at : 0;
        n.pos = Lane::position(p, n.token);
        at += step_a;
        token += step_t;
        if (at >= s.units) {
            at -= s.units;
            ++token;
        }
    };
    int count = 0;  // the wave's units
    {
        const int64_t total = (int64_t)p.T * s.units, u0 = block * NW + w;
        count = u0 < total ? (int)((total - u0 + step - 1) / step) : 0;
    }
    Unit n1, n2;
    if (count > 0) {
        next(n1);
        fetch(n1);
        next(n2);
    }
    for (int i = 0; i < count; ++i) {
        Unit n = n1;
        n1 = n2;
        if (i + 1 < count)
            fetch(n1);
        next(n2);
        L.settle(n.t, p, n.pos);
        const bool there = n.at * NG + L.g < s.H;
        if (n.at * NG + NG > s.H && !there) {
            // a head that is not there (another one was read): no part in dw
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                n.d.a[c].clear();
                n.d.b[c].clear();
            }
        }
        float x[NC][2 * V], d[NC][2 * V];
        L.unpack(n.x, x);
        L.unpack(n.d, d);
        const float r = L.root(x, p);
        L.template turn<true>(d, n.t);
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) {
                x[c][e] *= r;
                acc[c][e] = __builtin_fmaf(d[c][e], x[c][e], acc[c][e]);
                d[c][e] *= wf[c][e];
            }
        const float m = L.dot(d, x) * p.inv_d;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < 2 * V; ++e)
                d[c][e] = r * __builtin_fmaf(-x[c][e], m, d[c][e]);
        if (there)
            L.store(Lane::first_head(s.out, s.ot, s.oh, n.token, n.at),
                    Lane::head_offset(s.oh, L.g), d);
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
        const int r = i / G;
        const Lane l(p, i % G);
        int o = p.D;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < 2 * V; ++e)
                if (r == c * 2 * V + e && e % V < (e < V ? l.na[c] : l.nb[c]))
                    o = (e < V ? l.oa[c] : l.ob[c]) + e % V;
        if (o < p.D) {
            float t = red[0][i];
#pragma unroll
            for (int v = 1; v < NW; ++v)
                t += red[v][i];
            s.part[(int64_t)block * p.D + o] = t;
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
// a time, sixteen of them in flight, then the 32 sums, in order.
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
    for (int b0 = t; b0 < n; b0 += 512) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int b = b0 + 32 * i;
            v[i] = part[(int64_t)(b < n ? b : t) * p.D];
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
            s += b0 + 32 * i < n ? v[i] : 0.0f;
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
