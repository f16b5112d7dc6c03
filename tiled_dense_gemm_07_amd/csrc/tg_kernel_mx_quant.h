// Quantisation to microscaled blocks (tg_quant_mx) and back (tg_dequant_mx).
//
// mx_rows_kernel: blocks along the rows.  A lane takes eight elements, four lanes
// a block.
//
// mx_columns_kernel: blocks along the columns, written as rows of the transpose,
// and on request those along the rows from the same read.  A lane holds a block
// of 32 rows by the columns of one 16-byte load (8 of 16 bits, 4 of 32) in
// registers, so that no value crosses lanes: its codes of a column are 16 or 32
// consecutive bytes of the transpose, and its columns of a row a part of that
// row's block, whose largest magnitude is found over 4 or 8 lanes.  A wave takes
// 128 rows (four lanes down) by 16 lanes across; the four waves of a workgroup
// two by two, so that its writes are whole cache lines.
#pragma once

#include "tg_mx.h"

namespace tg {

struct MxQuantParams {
    const void* X;
    int64_t ldx;
    int M, K;
    int Kp, Mp;        // rounded up to whole runs of 128
    uint8_t *Q, *S;    // along the rows
    uint8_t *Qt, *St;  // along the columns
    float* sums;       // [Mp / 128][K]: the columns' sums over each 128 rows
    u32 magic;         // ceil(2^32 / (Kp / 8)), for the row of a unit
};

template <int DT, int FMT, int U>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256))) void
mx_rows_kernel(MxQuantParams p)
{
    const u32 per = (u32)p.Kp / 8;  // units of a row
    const uint64_t first = (uint64_t)blockIdx.x * (256 * U);
    const uint64_t row0 = first / per;
    const u32 rem = (u32)(first - row0 * per);
    const uint64_t total = (uint64_t)p.M * per;
    Raw8<DT> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        // rows past row0: at most one where a row has as many units as the
        // workgroup, else a division by multiplication, exact for these sizes
        const u32 at = rem + threadIdx.x + 256 * u;
        const u32 d = per >= 256 * U ? (at >= per ? 1u : 0u) : __umulhi(at, p.magic);
        const uint64_t row = row0 + d;
        const int k = (int)(8 * (at - d * per));
        if (row < (uint64_t)p.M)
            load8<DT>(r[u], elem_ptr<DT>(p.X, (int64_t)row * p.ldx), k, p.K - k);
        else
            load8<DT>(r[u], p.X, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint64_t at = first + threadIdx.x + 256 * u;
        u32 m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = MaxOp::of(m, __builtin_bit_cast(u32, get8<DT>(r[u], i)) & 0x7FFFFFFFu);
        MxScale s;
        s.of_amax<FMT>(mx_block_max<4>(m));
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = s.ok ? get8<DT>(r[u], i) : 0.0f;
        if (at >= total)
            continue;
        if constexpr (FMT == MX_E2M1)
            ((u32*)p.Q)[at] = mx_codes4(v, s.p);
        else
            ((u32x2*)p.Q)[at] = u32x2{mx_codes8(v[0], v[1], v[2], v[3], s.p),
                                      mx_codes8(v[4], v[5], v[6], v[7], s.p)};
        if ((threadIdx.x & 3) == 0)
            p.S[at / 4] = (uint8_t)s.byte;
    }
}

// The columns of one 16-byte load.
template <int DT>
struct MxLane {
    static constexpr int V = DT == DT_F32 ? 4 : 8;
    u32x4 v;

    // left: columns that exist from `p` on
    __device__ __forceinline__ void load(const char* p, int left)
    {
        constexpr int ES = DT == DT_F32 ? 4 : 2;
        struct __attribute__((packed, aligned(ES))) Any {
            u32x4 v;
        };
        if (left >= V) {
            v = ((const Any*)p)->v;
            return;
        }
        v = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < left) {
                if constexpr (DT == DT_F32)
                    v[i] = ((const u32*)p)[i];
                else
                    v[i >> 1] |= (u32)((const uint16_t*)p)[i] << (16 * (i & 1));
            }
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
};

// Magnitudes as stored, two of 16 bits to a word: their order is that of their
// bit patterns, NaN above infinity.
template <int DT>
__device__ __forceinline__ u32 mx_max_word(u32 m, u32 w)
{
    if constexpr (DT == DT_F32)
        return MaxOp::of(m, w & 0x7FFFFFFFu);
    typedef __attribute__((ext_vector_type(2))) unsigned short u16x2;
    return __builtin_bit_cast(u32, __builtin_elementwise_max(
                                       __builtin_bit_cast(u16x2, m),
                                       __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu)));
}
// The fp32 bit pattern of magnitude i of such words.
template <int DT>
__device__ __forceinline__ u32 mx_bits(const u32x4& m, int i)
{
    MxLane<DT> l;
    l.v = m;
    return __builtin_bit_cast(u32, l.get(i));
}

template <int DT, int FMT, bool ROWS, bool COLS, bool SUMS>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256))) void
mx_columns_kernel(MxQuantParams p)
{
    using Lane = MxLane<DT>;
    constexpr int V = Lane::V, CL = 16, TC = CL * V;  // a wave's columns
    constexpr int ES = DT == DT_F32 ? 4 : 2;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int tiles = (p.K + 2 * TC - 1) / (2 * TC);  // workgroups across
    const int wg = (int)blockIdx.x;
    const int mt = wg / tiles;
    const int m0 = mt * 256 + (w >> 1) * 128;
    const int c0 = (wg - mt * tiles) * 2 * TC + (w & 1) * TC;
    if (m0 >= p.Mp || c0 >= p.Kp)
        return;  // whole waves, and no barrier follows
    const int cl = lane & (CL - 1), b = lane / CL;
    const int c = c0 + cl * V, m = m0 + 32 * b;
    Lane x[32];
    if (m0 + 128 <= p.M && c0 + TC <= p.K) {
        const char* at = (const char*)p.X + ((int64_t)m * p.ldx + c) * ES;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            x[i].load(at + (int64_t)i * p.ldx * ES, V);
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            x[i].load((const char*)p.X + ((int64_t)(m + i) * p.ldx + c) * ES,
                      m + i < p.M ? p.K - c : 0);
    }
    if constexpr (SUMS) {
        float s[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            s[j] = 0.0f;
#pragma unroll
            for (int i = 0; i < 32; ++i)
                s[j] += x[i].get(j);
            s[j] += __shfl_xor(s[j], 16);
            s[j] += __shfl_xor(s[j], 32);
        }
        if (b == 0) {
            float* to = p.sums + (int64_t)(m0 / 128) * p.K + c;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (c + j < p.K)
                    to[j] = s[j];
        }
    }
    if constexpr (COLS) {
        u32x4 top = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 32; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                top[j] = mx_max_word<DT>(top[j], x[i].v[j]);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            MxScale s;
            s.of_amax<FMT>(mx_bits<DT>(top, j));
            const int64_t at = (int64_t)(c + j) * p.Mp + m;
            u32x4 q[FMT == MX_E2M1 ? 1 : 2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = s.ok ? x[8 * i + e].get(j) : 0.0f;
                if constexpr (FMT == MX_E2M1) {
                    q[0][i] = mx_codes4(v, s.p);
                } else {
                    q[i >> 1][(i & 1) * 2] = mx_codes8(v[0], v[1], v[2], v[3], s.p);
                    q[i >> 1][(i & 1) * 2 + 1] = mx_codes8(v[4], v[5], v[6], v[7], s.p);
                }
            }
            if (c + j < p.K) {
                u32x4* to = (u32x4*)(p.Qt + mx_bytes<FMT>(at));
                to[0] = q[0];
                if constexpr (FMT == MX_E4M3)
                    to[1] = q[1];
                p.St[at / 32] = (uint8_t)s.byte;
            }
        }
    }
    if constexpr (ROWS) {
        const int rows = p.M - m;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            u32 t = 0;
#pragma unroll
            for (int j = 0; j < V; ++j)
                t = MaxOp::of(t, __builtin_bit_cast(u32, x[i].get(j)) & 0x7FFFFFFFu);
            MxScale s;
            s.of_amax<FMT>(mx_block_max<32 / V>(t));
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = s.ok && j < V ? x[i].get(j < V ? j : 0) : 0.0f;
            if (i >= rows)
                continue;
            const int64_t at = (int64_t)(m + i) * p.Kp + c;
            uint8_t* to = p.Q + mx_bytes<FMT>(at);
            if constexpr (FMT == MX_E2M1) {
                if constexpr (V == 8)
                    *(u32*)to = mx_codes4(v, s.p);
                else
                    *(uint16_t*)to = (uint16_t)mx_codes4(v, s.p);
            } else {
                if constexpr (V == 8)
                    *(u32x2*)to = u32x2{mx_codes8(v[0], v[1], v[2], v[3], s.p),
                                        mx_codes8(v[4], v[5], v[6], v[7], s.p)};
                else
                    *(u32*)to = mx_codes8(v[0], v[1], v[2], v[3], s.p);
            }
            if ((cl & (32 / V - 1)) == 0)
                p.S[at / 32] = (uint8_t)s.byte;
        }
    }
}

// Sums of the columns' partial sums, in order.
struct MxSumParams {
    const float* part;  // [parts][K]
    float* out;         // [K]
    int parts, K;
};

__global__ __attribute__((amdgpu_flat_work_group_size(256, 256))) void
mx_sums_kernel(MxSumParams p)
{
    const int k = (int)(blockIdx.x * 256 + threadIdx.x);
    if (k >= p.K)
        return;
    float s = 0.0f;
    for (int i = 0; i < p.parts; ++i)
        s += p.part[(int64_t)i * p.K + k];
    p.out[k] = s;
}

struct MxDequantParams {
    const uint8_t *Q, *S;
    void* X;
    int64_t ldx;
    int M, K, Kp;
    u32 magic;
};

// A lane takes eight elements; elements past K are not written.  Elements times
// their power of two are exact in fp32 down to its smallest subnormal, and
// rounded once to X's type.
template <int DT, int FMT, int U>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256))) void
mx_dequant_kernel(MxDequantParams p)
{
    const u32 per = (u32)p.Kp / 8;
    const uint64_t first = (uint64_t)blockIdx.x * (256 * U);
    const uint64_t row0 = first / per;
    const u32 rem = (u32)(first - row0 * per);
    const uint64_t total = (uint64_t)p.M * per;
    u32x2 q[U];
    u32 sb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        uint64_t at = first + threadIdx.x + 256 * u;
        at = at < total ? at : total - 1;
        if constexpr (FMT == MX_E2M1)
            q[u] = u32x2{((const u32*)p.Q)[at], 0u};
        else
            q[u] = ((const u32x2*)p.Q)[at];
        sb[u] = p.S[at / 4];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const u32 at = rem + threadIdx.x + 256 * u;
        const u32 d = per >= 256 * U ? (at >= per ? 1u : 0u) : __umulhi(at, p.magic);
        const uint64_t row = row0 + d;
        const int k = (int)(8 * (at - d * per));
        const float s = __builtin_bit_cast(
            float, sb[u] == 255 ? 0x7FC00000u : (sb[u] > 0 ? sb[u] << 23 : 0x00400000u));
        float v[8];
        if constexpr (FMT == MX_E2M1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // twice the magnitude, 0 to 12, from a word of nibbles
                const u32 c = q[u][0] >> (4 * i);
                const float m = (float)((0xC8643210u >> ((c & 7) * 4)) & 15u) * 0.5f;
                v[i] = ((c & 8) ? -m : m) * s;
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[u][h], false);
                const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[u][h], true);
                v[4 * h] = a[0] * s;
                v[4 * h + 1] = a[1] * s;
                v[4 * h + 2] = b[0] * s;
                v[4 * h + 3] = b[1] * s;
            }
        }
        if (row >= (uint64_t)p.M || k >= p.K)
            continue;
        Raw8<DT> r;
        put8<DT>(r, v);
        store8<DT>((void*)elem_ptr<DT>(p.X, (int64_t)row * p.ldx), k, p.K - k, r);
    }
}

}  // namespace tg
