// What the 8-bit integer kernels and their host entry points share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tg_kernel.h"

namespace tg {

typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(16))) int i32x16;

// C = epilogue((A W^T) sa sw + bias), see tg_gemm_i8.
struct I8Params {
    const int8_t* A;    // [M][lda]
    const int8_t* W;    // [N][ldw]
    const float* sa;    // [M]
    const float* sw;    // [N]
    const float* bias;  // [N] or NULL
    void* C;            // [M][ldc] of type dt_out
    int dt_out;
    int M, N, K;
    int64_t lda, ldw, ldc;  // in elements
    int tiles_m, tiles_n;
    int relu;
    int c_vec;                   // C rows take 4-element vector stores
    int group_m;                 // swizzle group (tile rows), as in tg_sched.h
    unsigned long long* stamps;  // optional clock record, as in GemmParams
};

// 16 bytes of a row from any byte address, or the `left` (< 16, or <= 0)
// bytes that the row still has and zeros after them.  The hardware takes
// 16-byte global loads from any byte address.
__device__ __forceinline__ u32x4 load16_any(const int8_t* p, int left)
{
    struct __attribute__((packed, aligned(1))) Any {
        u32x4 v;
    };
    if (left >= 16)
        return ((const Any*)p)->v;
    u32x4 v = {0, 0, 0, 0};
    for (int i = 0; i < left; ++i)
        v[i >> 2] |= (u32)(uint8_t)p[i] << (8 * (i & 3));
    return v;
}

// One result of the product: the exact integer sum, scaled in fp32.
__device__ __forceinline__ float i8_result(int acc, float sa, float sw, float bias, int relu)
{
    const float v = __builtin_fmaf((float)acc * sa, sw, bias);
    return (relu && !(v > 0.0f)) ? 0.0f : v;
}

__device__ __forceinline__ void store_out(void* C, int dt, int64_t at, float v)
{
    if (dt == DT_F32)
        ((float*)C)[at] = v;
    else
        ((uint16_t*)C)[at] = cvt1(v, dt);
}

}  // namespace tg
