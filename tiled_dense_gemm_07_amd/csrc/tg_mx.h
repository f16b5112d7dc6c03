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
// The same of words of two 16-bit values.
template <int DT>
__device__ __forceinline__ u32 mx_codes4_16(u32 a, u32 b, u32 c, u32 d, float p)
{
    if constexpr (DT == DT_BF16) {
        const auto v = [](u32 x) { return __builtin_bit_cast(bf16x2, x); };
        u32 w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(0u, v(a), p, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, v(b), p, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, v(c), p, 2);
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, v(d), p, 3);
    } else {
        typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;
        const auto v = [](u32 x) { return __builtin_bit_cast(f16x2, x); };
        u32 w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(0u, v(a), p, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, v(b), p, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, v(c), p, 2);
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, v(d), p, 3);
    }
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

// Largest magnitude over the quad (4 lanes) of a lane.
__device__ __forceinline__ u32 mx_block_max(u32 m)
{
    m = MaxOp::of(m, dpp<0xB1>(m));
    return MaxOp::of(m, dpp<0x4E>(m));
}

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
// The fp32 bit pattern of a magnitude of such a word (the upper one: hi).
template <int DT>
__device__ __forceinline__ u32 mx_bits(u32 w, bool hi)
{
    if constexpr (DT == DT_F32)
        return w;
    if constexpr (DT == DT_BF16)
        return hi ? w & 0xFFFF0000u : w << 16;
    return __builtin_bit_cast(
        u32, (float)__builtin_bit_cast(_Float16, (uint16_t)(hi ? w >> 16 : w)));
}

// Eight elements of a row, a quarter of a block (the other lanes of the quad hold
// the rest), to a dword of codes (E4M3: two), and the block's scale byte.
template <int DT, int FMT>
__device__ __forceinline__ u32x2 mx_codes(const Raw8<DT>& r, u32& byte)
{
    u32 m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m = mx_max_word<DT>(m, r.v[0][i]);
        if constexpr (DT == DT_F32)
            m = mx_max_word<DT>(m, r.v[1][i]);
    }
    if constexpr (DT != DT_F32)
        m = MaxOp::of(mx_bits<DT>(m, false), mx_bits<DT>(m, true));
    MxScale s;
    s.of_amax<FMT>(mx_block_max(m));
    byte = s.byte;
    u32x2 w;
    if constexpr (FMT == MX_E2M1 && DT != DT_F32) {
        w = u32x2{mx_codes4_16<DT>(r.v[0][0], r.v[0][1], r.v[0][2], r.v[0][3], s.p), 0u};
    } else {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = get8<DT>(r, i);
        if constexpr (FMT == MX_E2M1)
            w = u32x2{mx_codes4(v, s.p), 0u};
        else
            w = u32x2{mx_codes8(v[0], v[1], v[2], v[3], s.p),
                      mx_codes8(v[4], v[5], v[6], v[7], s.p)};
    }
    return s.ok ? w : u32x2{0u, 0u};
}

// A sum of products to the layer's result.
__device__ __forceinline__ float mx_result(float v, float bias, int relu)
{
    v += bias;
    return (relu && !(v > 0.0f)) ? 0.0f : v;
}

}  // namespace tg
