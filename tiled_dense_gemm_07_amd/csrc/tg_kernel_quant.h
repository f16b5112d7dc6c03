// Quantisation of activations to 8 bits, one scale for each row (tg_quant_i8).
// One pass over memory: a team of TPR threads holds a row of up to 8 NC TPR
// elements in registers between the search for its largest magnitude and the
// conversion.  Longer rows (NC = 0) are read twice.  Bound by memory: bf16 8192
// x 8192 30.7 us (201 MB, 6.5 TB/s, part of it from the last-level cache; three
// inputs in turn 36, 5.6 TB/s), 16 x 8192 2.7 us, which is launch and latency.  The
// correction of the quotient (three operations an element) hides under the loads,
// and so do the 64-bit levels of fp32 inputs: three inputs in turn 8192 x 8192 61.8
// us, 8192 x 4096 31.2, 8192 x 1024 8.6 (5.4, 5.4 and 4.9 TB/s).
// tg_linear_i8 may have the same launch copy W's rows to 16-byte boundaries, in
// workgroups after those of the activations: 4096 x 4095 6 to 7 us more.
#pragma once

#include "tg_rows.h"

namespace tg {

struct QuantParams {
    const void* X;
    int8_t* Q;
    float* s;
    int M, K;
    int64_t ldx, ldq;
    int kq;  // columns of Q to write: past K, zeros
    // Rows of 8-bit weights that the workgroups from `first` on copy, `rows`
    // each, to rows of kq bytes, zeros past K (none: first is the grid).
    const int8_t* W;
    int8_t* Wq;
    int64_t ldw;
    int N, rows;
    u32 first;
};

// Copies rows of W from any address to 16-byte boundaries, a chunk to a thread,
// four of them in flight (K >= 16).
template <int NT>
__device__ __forceinline__ void pack_rows(const QuantParams& p, int block)
{
    struct __attribute__((packed, aligned(1))) Any {
        u32x4 v;
    };
    constexpr int U = 4;
    const int n0 = block * p.rows;
    const int8_t* W = p.W + (int64_t)n0 * p.ldw;
    u32x4* to = (u32x4*)(p.Wq + (int64_t)n0 * p.kq);
    const int per = p.kq / 16;
    const int rows = p.N - n0 < p.rows ? p.N - n0 : p.rows;
    const int total = rows * per;
    for (int i0 = threadIdx.x; i0 < total; i0 += U * NT) {
        u32x4 v[U];
        int s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * NT < total ? i0 + u * NT : total - 1;
            const int n = i / per, k = 16 * (i - n * per);
            const int over = k - (p.K - 16);  // a chunk across the end, as load16_row
            s[u] = over < 0 ? 0 : over;
            v[u] = ((const Any*)(W + n * p.ldw + (over < 0 ? k : p.K - 16)))->v;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * NT < total)
                to[i0 + u * NT] = shift_bytes(v[u], s[u]);
    }
}

template <int DT>
__device__ __forceinline__ void quant_chunk(const Raw8<DT>& r, const RowLevels& L, int8_t* row,
                                            int at, int left)
{
    int q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (DT == DT_F32)
            q[i] = L.level64(get8<DT>(r, i));
        else
            q[i] = L.level(get8<DT>(r, i));
    }
    store_levels(row, at, left, q);
}

template <int DT>
__device__ __forceinline__ u32 chunk_amax(const Raw8<DT>& r, u32 m)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const u32 b = __builtin_bit_cast(u32, get8<DT>(r, i)) & 0x7FFFFFFFu;
        m = b > m ? b : m;
    }
    return m;
}

// NT threads, NT / TPR rows per workgroup.
template <int DT, int NT, int TPR, int NC, bool ODD>
__global__ __attribute__((amdgpu_flat_work_group_size(NT, NT))) void quant_i8_kernel(QuantParams p)
{
    __shared__ u32 slot[16];
    if (blockIdx.x >= p.first) {
        pack_rows<NT>(p, (int)(blockIdx.x - p.first));
        return;
    }
    const int t = threadIdx.x % TPR;
    const u32 row =
        blockIdx.x * (NT / TPR) + (u32)__builtin_amdgcn_readfirstlane((int)(threadIdx.x / TPR));
    if (row >= (u32)p.M)
        return;  // whole waves; rows share a workgroup only when TPR is one wave
    const Row<DT, ODD> x(p.X, row, p.ldx, p.K);
    int8_t* q = p.Q + row * p.ldq;
    u32 m[1] = {0};
    RowLevels L;
    if constexpr (NC > 0) {
        Raw8<DT> r[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int at = 8 * (t + c * TPR);
            x.load(r[c], at);
        }
#pragma unroll
        for (int c = 0; c < NC; ++c)
            m[0] = chunk_amax<DT>(r[c], m[0]);
        row_all<MaxOp, TPR, 1>(m, slot);
        L.of_amax(m[0]);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int at = 8 * (t + c * TPR);
            quant_chunk<DT>(r[c], L, q, at, p.kq - at);
        }
    } else {
        for (int at = 8 * t; at < p.K; at += 8 * TPR) {
            Raw8<DT> r;
            x.load(r, at);
            m[0] = chunk_amax<DT>(r, m[0]);
        }
        row_all<MaxOp, TPR, 1>(m, slot);
        L.of_amax(m[0]);
        for (int at = 8 * t; at < p.kq; at += 8 * TPR) {
            Raw8<DT> r;
            x.load(r, at);
            quant_chunk<DT>(r, L, q, at, p.kq - at);
        }
    }
    if (t == 0)
        p.s[row] = L.scale;
}

}  // namespace tg
