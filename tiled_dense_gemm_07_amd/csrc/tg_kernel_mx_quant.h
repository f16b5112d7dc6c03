// Quantisation to microscaled blocks (tg_quant_mx) and back (tg_dequant_mx).
//
// All are bound by memory from some 4096 x 4096 on, below by launch and the latency
// of a wave's loads, conversions and stores.  Times: bf16 to E2M1, inputs in turn.
//
// mx_rows_kernel: blocks along the rows.  A lane takes eight elements, four lanes
// a block.  8192 x 8192 29 to 33 us (5.2 to 5.9 TB/s; 24 where the last-level cache
// still holds the input), 1000 x 4096 3.6, 16 x 8192 2.6; back (mx_dequant_kernel) 25
// to 30 us, 4.0 and 2.4.
//
// mx_columns_kernel: blocks along the columns, written as rows of the transpose,
// in tiles of 256 rows by 128 columns.  A lane holds 32 rows of four columns in
// registers, so that no value crosses lanes: its codes of a column are 16 or 32
// consecutive bytes of the transpose.  A wave takes 128 rows (four lanes down) by 64
// columns (16 lanes across); the four waves of a workgroup two by two.  Neighbouring
// workgroups stay on one XCD, whose L2 joins their parts of cache lines.  8192 x 8192
// 37 us (4.6 TB/s), 2048 x 4096 6.7, 512 x 512 4.2.  Blocks along both: every other
// workgroup takes the rows of the tile whose columns the one beside it takes, from the
// same L2 (one workgroup for both, each value loaded once: 512 x 512 7.1 us and 5.0,
// 2048 x 4096 10.5 and 9.4, 8192 x 8192 54.6 and 56.6).
#pragma once

#include "tg_mx.h"
#include "tg_sched.h"

namespace tg {

struct MxQuantParams {
    const void* X;
    int64_t ldx;
    int M, K;
    int Kp, Mp;        // rounded up to whole runs of 128
    uint8_t *Q, *S;    // along the rows
    uint8_t *Qt, *St;  // along the columns
    float* sums;       // [Mp / 128][K]: the columns' sums over each 128 rows
    int tiles_m, tiles_n;  // workgroups down and across (columns kernel)
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
        u32 byte;
        const u32x2 w = mx_codes<DT, FMT>(r[u], byte);
        if (at >= total)
            continue;
        if constexpr (FMT == MX_E2M1)
            ((u32*)p.Q)[at] = w[0];
        else
            ((u32x2*)p.Q)[at] = w;
        if ((threadIdx.x & 3) == 0)
            p.S[at / 4] = (uint8_t)byte;
    }
}

// Four consecutive elements of a row.
template <int DT>
struct MxLane {
    static constexpr int NW = DT == DT_F32 ? 4 : 2;  // words
    static constexpr int ES = DT == DT_F32 ? 4 : 2;
    u32 v[NW];

    __device__ __forceinline__ void load(const char* p)
    {
        typedef __attribute__((ext_vector_type(NW))) u32 Vec;
        struct __attribute__((packed, aligned(ES))) Any {
            Vec v;
        };
        const Vec w = ((const Any*)p)->v;
#pragma unroll
        for (int i = 0; i < NW; ++i)
            v[i] = w[i];
    }
    // Drops the first s elements (0 to 4), zeros from above.
    __device__ __forceinline__ void drop(int s)
    {
        if constexpr (DT == DT_F32) {
            const bool one = s & 1, two = s & 2;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = one ? (i < 3 ? v[i < 3 ? i + 1 : 3] : 0u) : v[i];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = s >= 4 ? 0u : (two ? (i < 2 ? v[i < 2 ? i + 2 : 3] : 0u) : v[i]);
        } else {
            const uint64_t w = s >= 4 ? 0 : ((uint64_t)v[1] << 32 | v[0]) >> (16 * (s & 3));
            v[0] = (u32)w;
            v[1] = (u32)(w >> 32);
        }
    }
    // Of a row of fewer than four elements.
    __device__ __forceinline__ void load_few(const char* p, int left)
    {
#pragma unroll
        for (int i = 0; i < NW; ++i)
            v[i] = 0;
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < left) {
                if constexpr (DT == DT_F32)
                    v[i] = ((const u32*)p)[i];
                else
                    v[i >> 1] |= (u32)((const uint16_t*)p)[i] << (16 * (i & 1));
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
};

// Keeps the compiler from holding the rows' unpacked values across this point.
template <int DT>
__device__ __forceinline__ void mx_repack(MxLane<DT> (&x)[32])
{
    if constexpr (DT != DT_F32) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            asm volatile("" : "+v"(x[i].v[0]), "+v"(x[i].v[1]));
    }
    __builtin_amdgcn_sched_barrier(0);
}

// Codes of element j of eight rows x[0 .. 7], to a dword (E2M1) or two.
template <int DT, int FMT>
__device__ __forceinline__ u32x2 mx_column_codes(const MxLane<DT>* x, int j, const MxScale& s)
{
    u32x2 w;
    if constexpr (FMT == MX_E2M1 && DT != DT_F32) {
        // pairs of rows as the instruction takes them
        const u32 sel = (j & 1) ? 0x07060302u : 0x05040100u;
        const auto pair = [&](int i) {
            return __builtin_amdgcn_perm(x[i + 1].v[j >> 1], x[i].v[j >> 1], sel);
        };
        w = u32x2{mx_codes4_16<DT>(pair(0), pair(2), pair(4), pair(6), s.p), 0u};
    } else {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = x[e].get(j);
        if constexpr (FMT == MX_E2M1)
            w = u32x2{mx_codes4(v, s.p), 0u};
        else
            w = u32x2{mx_codes8(v[0], v[1], v[2], v[3], s.p),
                      mx_codes8(v[4], v[5], v[6], v[7], s.p)};
    }
    return s.ok ? w : u32x2{0u, 0u};
}

// The rows of one tile of 256 rows by 128 columns, eight elements to a lane.
template <int DT, int FMT>
__device__ __forceinline__ void mx_tile_rows(const MxQuantParams& p, int m0, int c0)
{
    using Lane = MxLane<DT>;
    constexpr int ES = Lane::ES, U = 16;  // units of a thread
    const int c = c0 + ((int)threadIdx.x & 15) * 8;
    const int m = m0 + ((int)threadIdx.x >> 4);
    Raw8<DT> r[U];
    if (m0 + 256 <= p.M && c0 + 128 <= p.K) {
        const char* at = (const char*)p.X + ((int64_t)m * p.ldx + c) * ES;
#pragma unroll
        for (int u = 0; u < U; ++u)
            load8<DT>(r[u], at + (int64_t)(16 * u) * p.ldx * ES, 0, 8);
    } else {
        // across an edge, in two halves, as mx_columns does
        Lane h[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = m + 16 * u;
            const char* at = (const char*)p.X + (int64_t)(row < p.M ? row : p.M - 1) * p.ldx * ES;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int k = c + 4 * i, over = k - (p.K - 4);
                if (p.K >= 4)
                    h[u][i].load(at + (int64_t)(over > 0 ? p.K - 4 : k) * ES);
                else
                    h[u][i].load_few(at, k == 0 ? p.K : 0);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int over = p.K >= 4 ? c + 4 * i - (p.K - 4) : 0;
                h[u][i].drop(m + 16 * u < p.M ? (over < 0 ? 0 : (over < 4 ? over : 4)) : 4);
#pragma unroll
                for (int w = 0; w < Lane::NW; ++w) {
                    if constexpr (DT == DT_F32)
                        r[u].v[i][w] = h[u][i].v[w];
                    else
                        r[u].v[0][2 * i + w] = h[u][i].v[w];
                }
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        u32 byte;
        const u32x2 w = mx_codes<DT, FMT>(r[u], byte);
        const int row = m + 16 * u;
        if (row >= p.M)
            continue;
        const int64_t at = ((int64_t)row * p.Kp + c) / 8;
        if constexpr (FMT == MX_E2M1)
            ((u32*)p.Q)[at] = w[0];
        else
            ((u32x2*)p.Q)[at] = w;
        if ((threadIdx.x & 3) == 0)
            p.S[at / 4] = (uint8_t)byte;
    }
}

// The columns of one tile of 256 rows by 128 columns.
template <int DT, int FMT, bool COLS, bool SUMS>
__device__ __forceinline__ void mx_tile_columns(const MxQuantParams& p, int tile_m, int tile_c)
{
    using Lane = MxLane<DT>;
    constexpr int V = 4, CL = 16, TC = CL * V;  // a wave's columns
    constexpr int ES = Lane::ES;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int m0 = tile_m + (w >> 1) * 128;
    const int c0 = tile_c + (w & 1) * TC;
    if (m0 >= p.Mp || c0 >= p.Kp)
        return;  // whole waves, and no barrier follows
    const int cl = lane & (CL - 1), b = lane / CL;
    const int c = c0 + cl * V, m = m0 + 32 * b;
    Lane x[32];
    if (m0 + 128 <= p.M && c0 + TC <= p.K) {
        const char* at = (const char*)p.X + ((int64_t)m * p.ldx + c) * ES;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            x[i].load(at + (int64_t)i * p.ldx * ES);
    } else if (p.K >= V) {
        // across an edge: the row's last four elements shifted down, the last
        // row again for rows that are not there
        const int over = c - (p.K - V);
        const char* at = (const char*)p.X + (int64_t)(over > 0 ? p.K - V : c) * ES;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            x[i].load(at + (int64_t)(m + i < p.M ? m + i : p.M - 1) * p.ldx * ES);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            x[i].drop(m + i < p.M ? (over < 0 ? 0 : (over < V ? over : V)) : V);
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            x[i].load_few((const char*)p.X + (int64_t)(m + i) * p.ldx * ES,
                          m + i < p.M && c == 0 ? p.K : 0);
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
        mx_repack(x);
    }
    if constexpr (COLS) {
        u32 top[Lane::NW];
#pragma unroll
        for (int j = 0; j < Lane::NW; ++j) {
            top[j] = 0;
#pragma unroll
            for (int i = 0; i < 32; ++i)
                top[j] = mx_max_word<DT>(top[j], x[i].v[j]);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            MxScale s;
            s.of_amax<FMT>(mx_bits<DT>(top[DT == DT_F32 ? j : j >> 1], j & 1));
            u32x4 q[FMT == MX_E2M1 ? 1 : 2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const u32x2 k = mx_column_codes<DT, FMT>(x + 8 * i, j, s);
                if constexpr (FMT == MX_E2M1) {
                    q[0][i] = k[0];
                } else {
                    q[i >> 1][(i & 1) * 2] = k[0];
                    q[i >> 1][(i & 1) * 2 + 1] = k[1];
                }
            }
            if (c + j < p.K) {
                const int64_t at = (int64_t)(c + j) * p.Mp + m;
                u32x4* to = (u32x4*)(p.Qt + mx_bytes<FMT>(at));
                to[0] = q[0];
                if constexpr (FMT == MX_E4M3)
                    to[1] = q[1];
                p.St[at / 32] = (uint8_t)s.byte;
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

template <int DT, int FMT, bool ROWS, bool COLS, bool SUMS>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256))) void
mx_columns_kernel(MxQuantParams p)
{
    // ROWS: every other workgroup takes a tile's rows, the one beside it, on the same
    // XCD, its columns
    const TileCoord tc = tile_of((int)blockIdx.x, p.tiles_m, ROWS ? 2 * p.tiles_n : p.tiles_n, 1);
    const int m0 = tc.m * 256, c0 = (ROWS ? tc.n >> 1 : tc.n) * 128;
    if (ROWS && (tc.n & 1))
        mx_tile_rows<DT, FMT>(p, m0, c0);
    else
        mx_tile_columns<DT, FMT, COLS, SUMS>(p, m0, c0);
}

// Sums of the columns' partial sums, in order, 256 to a workgroup.
struct MxSumParams {
    const float* part;  // [parts][K]
    float* out;         // [K]
    int parts, K;
};

__device__ __forceinline__ void mx_sums(const MxSumParams& p, int block)
{
    const int k = block * 256 + (int)threadIdx.x;
    if (k >= p.K)
        return;
    float s = 0.0f;
    const float* at = p.part + k;
    int i = 0;
    for (; i + 8 <= p.parts; i += 8) {  // eight loads in flight, added in order
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = at[(int64_t)(i + j) * p.K];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s += v[j];
    }
    for (; i < p.parts; ++i)
        s += at[(int64_t)i * p.K];
    p.out[k] = s;
}

// The rest of a backward pass' quantisation in one launch: the columns of two
// matrices to E2M1 (workgroups up to end[0] and up to end[1]), and the sums of the
// columns of a third that an earlier launch left in parts.
struct MxRestParams {
    MxQuantParams q[2];
    MxSumParams sums;
    int end[2];
};

template <int DT>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256))) void
mx_rest_kernel(MxRestParams p)
{
    const int b = (int)blockIdx.x;
    if (b >= p.end[1]) {
        mx_sums(p.sums, b - p.end[1]);
        return;
    }
    const MxQuantParams& q = b < p.end[0] ? p.q[0] : p.q[1];
    const TileCoord tc = tile_of(b < p.end[0] ? b : b - p.end[0], q.tiles_m, q.tiles_n, 1);
    mx_tile_columns<DT, MX_E2M1, true, false>(q, tc.m * 256, tc.n * 128);
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
            const auto two = [&](auto v2, int i) {
                v[i] = v2[0] * s;
                v[i + 1] = v2[1] * s;
            };
            two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u][0], 1.0f, 0), 0);
            two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u][0], 1.0f, 1), 2);
            two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u][0], 1.0f, 2), 4);
            two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u][0], 1.0f, 3), 6);
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

// C = epilogue(bias) where K is 0.
struct MxFillParams {
    const float* bias;
    void* C;
    int64_t ldc;
    int M, N, dt, relu;
};

__global__ __attribute__((amdgpu_flat_work_group_size(256, 256))) void
mx_fill_kernel(MxFillParams p)
{
    const int64_t all = (int64_t)p.M * p.N;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all;
         i += (int64_t)gridDim.x * 256) {
        const int64_t m = i / p.N, n = i - m * p.N;
        const float v = mx_result(0.0f, p.bias ? p.bias[n] : 0.0f, p.relu);
        if (p.dt == DT_F32)
            ((float*)p.C)[m * p.ldc + n] = v;
        else
            ((uint16_t*)p.C)[m * p.ldc + n] = cvt1(v, p.dt);
    }
}

}  // namespace tg
