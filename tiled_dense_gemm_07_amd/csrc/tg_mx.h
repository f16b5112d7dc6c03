// Microscaled blocks (OCP MX v1.0): 32 consecutive elements share one power of
// two.  For a block with the largest magnitude a,
//   P = 2^(floor(log2 a) - emax), at least 2^-127   (emax: 2 for E2M1, 8 for E4M3),
//   element = x / P rounded to the format, ties to even, at most its largest,
// so that a lands in the format's highest octave.  The scale byte is P's
// exponent + 127.  A block that holds an infinity or NaN gets the scale byte
// 255 (NaN) and zero elements, a block of zeros the byte 0.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tg_kernel_mx.h"
#include "tg_rows.h"

namespace tg {

// Rows of codes are whole runs of 128 elements, zeros past the end.
__host__ __device__ __forceinline__ int64_t mx_padded(int64_t K) { return (K + 127) / 128 * 128; }
// Bytes of n elements.
template <int FMT>
__host__ __device__ __forceinline__ constexpr int64_t mx_bytes(int64_t n)
{
    return FMT == MX_E2M1 ? n / 2 : n;
}

// A block's scale from the bit pattern of its largest magnitude in fp32.
struct MxScale {
    u32 byte;
    float p;   // P
    bool ok;

    template <int FMT>
    __device__ __forceinline__ void of_amax(u32 bits)
    {
        constexpr u32 emax = FMT == MX_E2M1 ? 2 : 8;
        const u32 e = bits >> 23;  // floor(log2 a) + 127; 0 for subnormal a, whose byte is 0
        ok = e != 255;
        byte = e > emax ? e - emax : 0;
        p = __builtin_bit_cast(float, byte > 0 ? byte << 23 : 0x00400000u);  // 2^-127 is subnormal
        byte = ok ? byte : 255;
    }
};

// Eight (E2M1) or four (E4M3) values to a dword of codes, the first one lowest.
// The instruction divides by P and rounds in one step, ties to even (checked
// over all 16-bit values, ties and their neighbours); it gives E2M1's largest
// magnitude for larger ones, but NaN in E4M3, hence the clamp.
__device__ __forceinline__ u32 mx_codes4(const float (&v)[8], float p)
{
    u32 w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], p, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], p, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], p, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], p, 3);
}
__device__ __forceinline__ u32 mx_codes8(float a, float b, float c, float d, float p)
{
    typedef __attribute__((ext_vector_type(2))) short s16x2;
    const float top = 448.0f * p;
    const auto in = [top](float x) { return __builtin_amdgcn_fmed3f(x, -top, top); };
    s16x2 r = {0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, in(a), in(b), p, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, in(c), in(d), p, true);
    return __builtin_bit_cast(u32, r);
}

// Largest magnitude over the quad (4 lanes) or half row (8 lanes) of a lane.
template <int LANES>
__device__ __forceinline__ u32 mx_block_max(u32 m)
{
    m = MaxOp::of(m, dpp<0xB1>(m));
    m = MaxOp::of(m, dpp<0x4E>(m));
    if constexpr (LANES == 8)
        m = MaxOp::of(m, dpp<0x141>(m));
    return m;
}

}  // namespace tg
