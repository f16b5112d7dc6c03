// 8-bit integer matrix product with a scale for each token and channel:
//   C[m][n] = epilogue(sa[m] sw[n] sum_k A[m][k] W[n][k] + bias[n]),
// A and W in 8 bits with k contiguous, the sum exact in 32-bit integers
// (v_mfma_i32_*_i8), scales, bias and ReLU in fp32, one rounding to C's type.
// Integer sums do not depend on their order, so every kernel here gives the
// same bits.
//
// i8_any_kernel: any sizes, strides and addresses.  128 x 128 x 64 tiles, four
// waves of 64 x 64; strips go through registers with 16-byte loads from any
// byte address (row tails byte by byte) into a two-stage LDS ring.
#pragma once

#include "tg_i8.h"
#include "tg_kernel_dma.h"

namespace tg {

// Results of one wave's FM x FN blocks of 32 x 32 straight from the
// accumulators: lane l holds row l % 32 and, for element 4 q + e, column
// 8 q + 4 (l / 32) + e of its block.
template <int FM, int FN>
__device__ __forceinline__ void i8_store_direct(const i32x16 (&acc)[FM][FN], const I8Params& p,
                                                int mw0, int nw0, int lane)
{
    const int lr = lane & 31;
    const int g = lane >> 5;
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
        const int m = mw0 + fm * 32 + lr;
        if (m >= p.M)
            continue;
        const float sa = p.sa[m];
#pragma unroll
        for (int fn = 0; fn < FN; ++fn) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int n = nw0 + fn * 32 + 8 * q + 4 * g;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (n + e < p.N)
                        store_out(p.C, p.dt_out, (int64_t)m * p.ldc + n + e,
                                  i8_result(acc[fm][fn][4 * q + e], sa, p.sw[n + e],
                                            p.bias ? p.bias[n + e] : 0.0f, p.relu));
                }
            }
        }
    }
}

struct I8Any {
    static constexpr int BM = 128, BN = 128, BK = 64;
    static constexpr int STAGE = (BM + BN) * BK;

    static __device__ __forceinline__ void run(const I8Params& p)
    {
        __shared__ __attribute__((aligned(16))) char smem[2 * STAGE];
        lds_char* sm = (lds_char*)smem;
        const int tid = threadIdx.x;
        const int lane = tid & 63;
        const int w = tid >> 6;
        const TileCoord tc = tile_of(blockIdx.x, p.tiles_m, p.tiles_n, p.group_m);
        const int m0 = tc.m * BM, n0 = tc.n * BN;
        const int wm0 = (w >> 1) * 64, wn0 = (w & 1) * 64;

        // thread t moves chunk t % 4 of rows t / 4 and t / 4 + 64 of each
        // operand; rows past the end read the last row (their results are
        // not stored)
        const int c = tid & 3;
        const int8_t* a[2];
        const int8_t* b[2];
        u32 st[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = (tid >> 2) + 64 * j;
            const int am = m0 + r < p.M ? m0 + r : p.M - 1;
            const int bn = n0 + r < p.N ? n0 + r : p.N - 1;
            a[j] = p.A + (int64_t)am * p.lda;
            b[j] = p.W + (int64_t)bn * p.ldw;
            st[j] = r * BK + ((c ^ swz_a(r)) << 4);
        }
        u32x4 ra[2], rb[2];
        const auto load = [&](int k0) {
            const int k = k0 + 16 * c;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                ra[j] = load16_any(a[j] + k, p.K - k);
                rb[j] = load16_any(b[j] + k, p.K - k);
            }
        };
        const auto store = [&](int s) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                *(lds_u32x4*)(sm + s * STAGE + st[j]) = ra[j];
                *(lds_u32x4*)(sm + s * STAGE + BM * BK + st[j]) = rb[j];
            }
        };
        i32x16 acc[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    acc[i][j][r] = 0;

        const int KT = (p.K + BK - 1) / BK;
        if (KT > 0) {
            load(0);
            store(0);
        }
        for (int t = 0; t < KT; ++t) {
            if (t + 1 < KT)
                load((t + 1) * BK);
            // strip t is in stage t & 1, and every wave is done with strip
            // t - 1, whose stage strip t + 1 takes below
            __syncthreads();
            const lds_char* s0 = sm + (t & 1) * STAGE;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                i32x4 fa[2], fb[2];
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const int rm = wm0 + 32 * f + (lane & 31);
                    const int rn = wn0 + 32 * f + (lane & 31);
                    const int ch = 2 * s + (lane >> 5);
                    fa[f] = __builtin_bit_cast(
                        i32x4, *(const lds_u32x4*)(s0 + rm * BK + ((ch ^ swz_a(rm)) << 4)));
                    fb[f] = __builtin_bit_cast(
                        i32x4,
                        *(const lds_u32x4*)(s0 + BM * BK + rn * BK + ((ch ^ swz_a(rn)) << 4)));
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[j], fa[i], acc[i][j],
                                                                         0, 0, 0);
            }
            if (t + 1 < KT)
                store((t + 1) & 1);
        }
        i8_store_direct<2, 2>(acc, p, m0 + wm0, n0 + wn0, lane);
    }
};

__global__ __attribute__((amdgpu_flat_work_group_size(256, 256))) void i8_any_kernel(I8Params p)
{
    I8Any::run(p);
}

}  // namespace tg
