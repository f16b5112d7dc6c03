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

// v shifted down by s bytes (0 .. 16), zeros from above.
__device__ __forceinline__ u32x4 shift_bytes(u32x4 v, int s)
{
    uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
    lo = s & 8 ? hi : lo;
    hi = s & 8 ? 0 : hi;
    const int b = (s & 7) * 8;
    lo = b ? lo >> b | hi << (64 - b) : lo;
    hi = hi >> b;
    const bool none = s >= 16;
    return u32x4{none ? 0u : (u32)lo, none ? 0u : (u32)(lo >> 32), none ? 0u : (u32)hi,
                 none ? 0u : (u32)(hi >> 32)};
}

// 16 bytes of a row of K at k, from any address (the hardware takes 16-byte
// loads at any byte), zeros past K.  A chunk across the end is the row's last
// 16 bytes shifted down, so that it, too, is one load and no branch.
struct RowEnd {
    u32x4 v;  // as loaded
    int s;

    __device__ __forceinline__ void load(const int8_t* row, int k, int K)
    {
        struct __attribute__((packed, aligned(1))) Any {
            u32x4 v;
        };
        if (K >= 16) {
            const int over = k - (K - 16);
            s = over < 0 ? 0 : (over < 16 ? over : 16);
            v = ((const Any*)(row + (over < 0 ? k : K - 16)))->v;
            return;
        }
        s = 0;
        v = u32x4{0, 0, 0, 0};
        for (int i = 0; k + i < K; ++i)
            v[i >> 2] |= (u32)(uint8_t)row[k + i] << (8 * (i & 3));
    }
    __device__ __forceinline__ u32x4 bytes() const { return shift_bytes(v, s); }
};

__device__ __forceinline__ u32x4 load16_row(const int8_t* row, int k, int K)
{
    RowEnd e;
    e.load(row, k, K);
    return e.bytes();
}

// A row, and 16-byte chunks of it from whole dwords: the hardware takes 16-byte
// loads at any byte, but those that are not at a dword take four times as long.
// SHIFT: the chunk at k is in the 5 dwords from the one that holds byte k on;
// 4 where the row starts at a dword, and the fifth is the fourth again.  Every
// dword read holds a byte of the chunk, so it lies in the row's memory pages.
template <bool SHIFT>
struct Row16 {
    const int8_t* p;  // SHIFT: down to the dword that holds the first byte
    u32 s;            // bytes from there to the row
    int x;            // offset of the fifth dword

    struct Chunk {
        u32x4 v;
        u32 x;
    };

    __device__ __forceinline__ void at(const int8_t* row)
    {
        s = SHIFT ? (u32)(uintptr_t)row & 3 : 0;
        x = s ? 16 : 12;
        p = row - s;
    }
    __device__ __forceinline__ const int8_t* row() const { return p + s; }
    // of a whole chunk (k + 16 <= K), as it was loaded
    __device__ __forceinline__ Chunk load(int k) const
    {
        struct __attribute__((packed, aligned(SHIFT ? 4 : 1))) Any {
            u32x4 v;
        };
        Chunk c;
        c.v = ((const Any*)(p + k))->v;
        c.x = SHIFT ? *(const u32*)(p + k + x) : 0;
        return c;
    }
    // across or past the row's end: zeros past K, nothing to shift
    __device__ __forceinline__ Chunk load_end(int k, int K) const
    {
        return Chunk{load16_row(row(), k, K), 0};
    }
    static __device__ __forceinline__ u32x4 bytes(const Chunk& c, u32 s)
    {
        if constexpr (!SHIFT)
            return c.v;
        return u32x4{__builtin_amdgcn_alignbyte(c.v[1], c.v[0], s),
                     __builtin_amdgcn_alignbyte(c.v[2], c.v[1], s),
                     __builtin_amdgcn_alignbyte(c.v[3], c.v[2], s),
                     __builtin_amdgcn_alignbyte(c.x, c.v[3], s)};
    }
};

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
