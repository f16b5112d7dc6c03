// Row operators (quantisation, norms): a team of threads holds one row in
// registers, eight consecutive elements to a chunk, chunk c of thread t being
// elements 8 (t + c * TPR) ...  Rows start at any element: the hardware takes
// 16-byte accesses at any address.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tg_kernel.h"

namespace tg {

// Eight elements as stored.
template <int DT>
struct Raw8 {
    u32x4 v[DT == DT_F32 ? 2 : 1];
};

template <int DT>
__device__ __forceinline__ const char* elem_ptr(const void* p, int64_t at)
{
    return (const char*)p + at * (DT == DT_F32 ? 4 : 2);
}

template <int DT>
__device__ __forceinline__ void load8(Raw8<DT>& r, const void* row, int at, int left)
{
    if constexpr (DT == DT_F32) {
        struct __attribute__((packed, aligned(4))) V {
            u32x4 v;
        };
        const float* p = (const float*)row + at;
        if (left >= 8) {
            r.v[0] = ((const V*)p)[0].v;
            r.v[1] = ((const V*)p)[1].v;
        } else {
            r.v[0] = r.v[1] = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left)
                    r.v[i >> 2][i & 3] = __builtin_bit_cast(u32, p[i]);
        }
    } else {
        struct __attribute__((packed, aligned(2))) V {
            u32x4 v;
        };
        const uint16_t* p = (const uint16_t*)row + at;
        if (left >= 8) {
            r.v[0] = ((const V*)p)->v;
        } else {
            r.v[0] = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left)
                    r.v[0][i >> 1] |= (u32)p[i] << (16 * (i & 1));
        }
    }
}

template <int DT>
__device__ __forceinline__ float get8(const Raw8<DT>& r, int i)
{
    if constexpr (DT == DT_F32) {
        const u32 w = r.v[i >> 2][i & 3];  // by value: a bit cast of the vector
        return __builtin_bit_cast(float, w);  // element itself reads element 0
    }
    const u32 w = r.v[0][i >> 1];
    if constexpr (DT == DT_BF16)
        return __builtin_bit_cast(float, (i & 1) ? (w & 0xFFFF0000u) : (w << 16));
    return (float)__builtin_bit_cast(_Float16, (uint16_t)((i & 1) ? (w >> 16) : w));
}

// Keeps the compiler from holding the unpacked values of r across this point:
// they are unpacked again after it, which takes an instruction each and no
// registers.
template <int DT>
__device__ __forceinline__ void repack(Raw8<DT>& r)
{
    asm volatile("" : "+v"(r.v[0]));
    if constexpr (DT == DT_F32)
        asm volatile("" : "+v"(r.v[1]));
}

// Rounds once to the type (nearest even).
template <int DT>
__device__ __forceinline__ void put8(Raw8<DT>& r, const float (&v)[8])
{
    if constexpr (DT == DT_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            r.v[i >> 2][i & 3] = __builtin_bit_cast(u32, v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r.v[0][i] = pack2(v[2 * i], v[2 * i + 1], DT);
    }
}

template <int DT>
__device__ __forceinline__ void store8(void* row, int at, int left, const Raw8<DT>& r)
{
    if constexpr (DT == DT_F32) {
        struct __attribute__((packed, aligned(4))) V {
            u32x4 v;
        };
        float* p = (float*)row + at;
        if (left >= 8) {
            ((V*)p)[0].v = r.v[0];
            ((V*)p)[1].v = r.v[1];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left)
                    p[i] = get8<DT_F32>(r, i);
        }
    } else {
        struct __attribute__((packed, aligned(2))) V {
            u32x4 v;
        };
        uint16_t* p = (uint16_t*)row + at;
        if (left >= 8) {
            ((V*)p)->v = r.v[0];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left)
                    p[i] = (uint16_t)(r.v[0][i >> 1] >> (16 * (i & 1)));
        }
    }
}

// One row of a matrix, through a buffer resource of the row: the lane's place is
// one register for all rows and all matrices, chunks may start at any address,
// and the hardware's range check, which looks at each dword of an access by
// itself, gives zeros past the end of the row, or from a matrix that is not
// there (NULL), and drops stores there.  ODD: rows with an odd number of
// elements, whose last 16-bit element ends inside a dword and fails that check:
// it is moved by an access of its own, in the lane that holds it.  No access
// stands in a branch, so that all of a row's loads are in flight together.
// The row number has to be uniform over the wave.
template <int DT, bool ODD>
struct Row {
    static constexpr int ES = DT == DT_F32 ? 4 : 2;
    static constexpr bool LAST = ODD && DT != DT_F32;
    int n;
    __amdgpu_buffer_rsrc_t rs;

    __device__ __forceinline__ Row(const void* base, int64_t row, int64_t ld, int cols)
    {
        n = base ? cols : 0;
        rs = make_rsrc((const char*)base + row * ld * ES, (u32)(n * ES));
    }
    // Offset of the last element in the lane whose chunk (at `at`) holds it,
    // out of range in the others; it is the low half of dword last_dword().
    __device__ __forceinline__ u32 last_offset(int at) const
    {
        return (u32)(n - 1 - at) < 8u ? (u32)(n - 1) * 2u : kOob;
    }
    __device__ __forceinline__ int last_dword() const { return ((n - 1) & 7) >> 1; }

    __device__ __forceinline__ void load(Raw8<DT>& r, int at) const
    {
        const u32 off = (u32)at * (u32)ES;
        r.v[0] = buf_load16(rs, off);
        if constexpr (DT == DT_F32)
            r.v[1] = buf_load16(rs, off + 16u);
        if constexpr (LAST) {
            const u32 e = buf_load2(rs, last_offset(at));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                r.v[0][i] |= i == last_dword() ? e : 0u;
        }
    }
    __device__ __forceinline__ void store(const Raw8<DT>& r, int at) const
    {
        const int off = at * ES;
        __builtin_amdgcn_raw_buffer_store_b128(r.v[0], rs, off, 0, 0);
        if constexpr (DT == DT_F32)
            __builtin_amdgcn_raw_buffer_store_b128(r.v[1], rs, off + 16, 0, 0);
        if constexpr (LAST) {
            u32 w = r.v[0][0];
#pragma unroll
            for (int i = 1; i < 4; ++i)
                w = i == last_dword() ? r.v[0][i] : w;
            __builtin_amdgcn_raw_buffer_store_b16((uint16_t)w, rs, (int)last_offset(at), 0, 0);
        }
    }
};

// --------------------------------------------------------------------------
// Reductions over the TPR threads that hold a row.  Every thread gets the
// result; the order of the additions is fixed.
// --------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ u32 dpp(u32 v)
{
    return (u32)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}

struct SumOp {
    static __device__ __forceinline__ u32 of(u32 a, u32 b)
    {
        return __builtin_bit_cast(u32, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
    }
};
struct MaxOp {  // of bit patterns: for magnitudes, NaN > Inf > finite
    static __device__ __forceinline__ u32 of(u32 a, u32 b) { return a > b ? a : b; }
};

struct MaxFloatOp {
    static __device__ __forceinline__ u32 of(u32 a, u32 b)
    {
        return __builtin_bit_cast(
            u32, fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)));
    }
};

template <class Op>
__device__ __forceinline__ u32 wave_all(u32 v)
{
    v = Op::of(v, dpp<0xB1>(v));   // quad_perm 1 0 3 2
    v = Op::of(v, dpp<0x4E>(v));   // quad_perm 2 3 0 1
    v = Op::of(v, dpp<0x141>(v));  // row_half_mirror
    v = Op::of(v, dpp<0x140>(v));  // row_mirror
    const auto s16 = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = Op::of(s16[0], s16[1]);
    const auto s32 = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return Op::of(s32[0], s32[1]);
}

// N values reduced together over TPR threads (whole waves).  `slot`: LDS of
// N * 16 words that no reduction in flight uses; reductions that alternate
// between two slots need no barrier between them.
template <class Op, int TPR, int N>
__device__ __forceinline__ void row_all(u32 (&v)[N], u32* slot)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = wave_all<Op>(v[i]);
    if constexpr (TPR > 64) {
        constexpr int NW = TPR / 64;
        const int w = (threadIdx.x % TPR) >> 6;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                slot[i * 16 + w] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            u32 s = slot[i * 16];
#pragma unroll
            for (int j = 1; j < NW; ++j)
                s = Op::of(s, slot[i * 16 + j]);
            v[i] = s;
        }
    }
}

template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], u32* slot)
{
    u32 b[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        b[i] = __builtin_bit_cast(u32, v[i]);
    row_all<SumOp, TPR, N>(b, slot);
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = __builtin_bit_cast(float, b[i]);
}

// --------------------------------------------------------------------------
// Quantisation of a row to 8-bit levels: q = 127 v / a with ties to even, a =
// the row's largest magnitude (at least 127 * 2^-126, so that the scale
// a / 127 is never subnormal).  A row with an infinity or NaN gets the scale
// NaN and zero levels: a product taken from it is NaN (zero after a ReLU).
// --------------------------------------------------------------------------
struct RowLevels {
    float scale;  // a / 127, rounded
    float c;      // 127, or 127 * 2^-32 where 127 a would overflow
    float a, ra;  // a (times the same power of two), and its reciprocal
    bool ok;

    // bits: of the largest |v|; f: a factor of the whole row (1 to 2) that v lacks
    __device__ __forceinline__ void of_amax(u32 bits, float f = 1.0f)
    {
        constexpr float least = 127.0f * 0x1p-126f;
        float m = __builtin_bit_cast(float, bits);
        ok = m * f < __builtin_inff();
        m = ok ? m : 1.0f;
        scale = ok ? fmaxf(m * f, least) / 127.0f : __builtin_nanf("");
        m = m * f < least ? least / f : m;
        const bool big = m > 0x1p100f;
        c = big ? 127.0f * 0x1p-32f : 127.0f;
        a = big ? m * 0x1p-32f : m;
        ra = 1.0f / a;
    }

    // One Newton step corrects the quotient to its rounded value.  For v of 16
    // significant bits or fewer (a product of two bf16 values has 16), 127 v is exact
    // and a quotient that is no tie lies a whole step of fp32 or more from one (with
    // steps of v and a of 2^i and 2^j, 254 v and (2 k + 1) a differ by one at least):
    // the level is the exact one.
    __device__ __forceinline__ int level(float v) const
    {
        const float x = v * c;
        const float q0 = x * ra;
        const float q = __builtin_fmaf(__builtin_fmaf(-q0, a, x), ra, q0);
        return ok ? (int)__builtin_rintf(q) : 0;
    }

    // The same for fp32 inputs in 64 bits, where 127 v is exact and a
    // quotient that is no tie lies more than 2^-32 from one.
    __device__ __forceinline__ int level64(float v) const
    {
        const double x = 127.0 * (double)v, d = (double)(a * (c == 127.0f ? 1.0f : 0x1p32f));
        const double r = (double)ra * (c == 127.0f ? 1.0 : 0x1p-32);
        double q = x * r;                                   // to about 2^-23
        q = __builtin_fma(__builtin_fma(-q, d, x), r, q);   // to about 2^-46
        q = __builtin_fma(__builtin_fma(-q, d, x), r, q);   // rounded
        return ok ? (int)__builtin_rint(q) : 0;
    }
};

// The same for u = x w of more bits, v = u rounded to fp32; f as above.  The fp32
// quotient of v is within 127 * 4 roundings, less than 2^-14, of the exact one and
// decides all levels but those that near to a tie, one of 8192.  Those are
// taken in 64 bits: 127 u is exact (but for a product of two fp32 values, 55
// bits), a quotient that is no tie lies more than 2^-48 (relative) from one, and
// the corrected one within 2^-52 of the exact one.
struct WideLevels {
    float scale, c;  // c: 127 / a
    double a;        // max|u|, or what stands for it where the scale is the least
    bool ok;

    // bits: of the largest |v|; e: what the largest |u| has beyond it
    __device__ __forceinline__ void of_amax(u32 bits, float e, float f)
    {
        constexpr float least = 127.0f * 0x1p-126f;
        float m = __builtin_bit_cast(float, bits);
        ok = m * f < __builtin_inff();
        m = ok ? m : 1.0f;
        scale = ok ? fmaxf(m * f, least) / 127.0f : __builtin_nanf("");
        a = m * f < least ? (double)(least / f) : (double)m + (double)e;
        c = 127.0f / (float)a;
    }
    // Levels of eight elements x(i), w(i) of a row that is ok.
    template <class X, class W>
    __device__ __forceinline__ void levels(const X& x, const W& w, int (&q)[8]) const
    {
        float off = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = x(i) * w(i) * c, n = __builtin_rintf(v);
            off = fmaxf(off, fabsf(v - n));
            q[i] = (int)n;
        }
        if (off > 0.5f - 0x1p-14f) {
            const double ra = 1.0 / a;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const double u = 127.0 * ((double)x(i) * (double)w(i)), y = u * ra;
                q[i] = (int)__builtin_rint(__builtin_fma(__builtin_fma(-y, a, u), ra, y));
            }
        }
    }
};

// Eight levels to bytes.
__device__ __forceinline__ void store_levels(int8_t* row, int at, int left, const int (&q)[8])
{
    struct __attribute__((packed, aligned(1))) V {
        u32x2 v;
    };
    if (left >= 8) {
        u32x2 b;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            b[i] = (u32)(q[4 * i] & 255) | (u32)(q[4 * i + 1] & 255) << 8 |
                   (u32)(q[4 * i + 2] & 255) << 16 | (u32)q[4 * i + 3] << 24;
        ((V*)(row + at))->v = b;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left)
                row[at + i] = (int8_t)q[i];
    }
}

}  // namespace tg
