// 8-bit integer product for few tokens (decoding): the time is that of
// streaming W once, so W goes from memory straight into the operand registers
// of v_mfma_i32_16x16x64_i8, with no LDS on its way.
//  * A workgroup owns 16 rows of W and 16 MT rows of A, and all of k; its NW
//    waves take runs of 256 k in turn.  In a run, lane (r = l % 16,
//    g = l / 16) loads 16 bytes of row r at k = 64 c + 16 g, c = 0 .. 3: an
//    instruction takes 64 contiguous bytes of 16 rows, and the run whole cache
//    lines.  A and W take the same k in the same lanes, so the order inside a
//    step does not matter.
//  * The loads of a wave's next run are issued before the MFMAs of this one.
//  * The waves' integer sums are added in LDS.
//  * Rows past M or N read the last row again; their results are not stored.
//    Zeros past the end of a row in its last, partial run.  Any addresses and
//    strides: rows that do not start at dwords are read in whole dwords and
//    shifted (SHIFT; W from HBM, 8192 x 8191, one token: 18.7 us, 33.9 with
//    16-byte loads at any byte; 16 tokens: 27.9 and 59.4; where the rows do
//    start at dwords it costs up to a quarter more).
//  * FUSED (tg_linear_i8): A is given in 16 or 32 bits.  Every workgroup
//    quantises the M rows itself, into LDS, while the loads of its first run
//    of W are in flight: one launch instead of two, for as few rows as that
//    takes no longer than those loads.
// Measured with W from HBM: one token 8192 x 8192 14.6 us (4.6 TB/s of the 5.2
// that a large copy reaches), 4096 x 4096 6.4 us; 16 tokens 8192 x 8192 17.3-17.8
// us: every workgroup reads all of A, as many bytes as its own rows of W.  More
// tokens: 16 to a workgroup while every workgroup has a CU of its own (32 tokens,
// 2048 x 8192: 9.7 us, 13.2 with 32), else 32 (17 tokens, 4096 x 4096: 7.3 us,
// 9.3 with 16).  Eight waves; 4 or 16 waves and 32 rows to a workgroup measured
// within 6% or slower.
#pragma once

#include "tg_i8.h"
#include "tg_rows.h"

namespace tg {

// What the fused form reads in place of A and sa.
struct I8Source {
    const void* X;  // [M][ldx]
    int64_t ldx;
};

template <int DTX, int MT, int NW, int SHIFT, bool FUSED>
struct I8Gemv {
    static constexpr int RUN = 256;
    static constexpr int TOKENS = 16 * MT;
    // levels: rows of K rounded up to a run, 16 bytes apart from a multiple
    // of the bank line so that the 16 rows of a fragment read spread
    static __host__ __device__ __forceinline__ int level_row(int K)
    {
        return (K + RUN - 1) / RUN * RUN + 16;
    }

    // SHIFT: rows that do not start at dwords, of W (1), of W or A (2)
    using RowW = Row16<(SHIFT >= 1)>;
    using RowA = Row16<(SHIFT >= 2)>;

    struct Run {
        typename RowW::Chunk w[4];
        typename RowA::Chunk a[FUSED ? 1 : MT][4];
    };

    static __device__ __forceinline__ void load(Run& R, const RowW& w, const RowA (&a)[MT],
                                                int k0, int K, int g, bool whole)
    {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int k = k0 + 64 * c + 16 * g;
            R.w[c] = whole ? w.load(k) : w.load_end(k, K);
            if constexpr (!FUSED) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    R.a[m][c] = whole ? a[m].load(k) : a[m].load_end(k, K);
            }
        }
    }

    static __device__ __forceinline__ void multiply(i32x4 (&acc)[MT], const Run& R, const RowW& w,
                                                    const RowA (&a)[MT], const char* levels, int k0,
                                                    int g, bool whole)
    {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const u32x4 vw = RowW::bytes(R.w[c], whole ? w.s : 0);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                u32x4 va;
                if constexpr (FUSED)
                    va = *(const u32x4*)(levels + k0 + 64 * c + 16 * g);
                else
                    va = RowA::bytes(R.a[m][c], whole ? a[m].s : 0);
                acc[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                    __builtin_bit_cast(i32x4, vw), __builtin_bit_cast(i32x4, va), acc[m], 0, 0, 0);
            }
        }
    }

    // Quantises the M <= NW rows of X into `levels` (rows of `ld` bytes, zeros
    // past K), their scales into sc.  NW / R waves to a row, R the power of two
    // that is at least M.
    static __device__ __forceinline__ void quantise(const I8Params& p, const I8Source& x,
                                                    char* levels, float* sc, u32* amax, int ld)
    {
        int R = 1;
        while (R < p.M)
            R *= 2;
        const int per = NW * 64 / R;  // threads of a row
        const int row = threadIdx.x / per, t = threadIdx.x % per;
        const bool mine = row < p.M;
        const char* src = elem_ptr<DTX>(x.X, (mine ? row : 0) * x.ldx);
        Raw8<DTX> r0;  // the thread's first chunk stays in registers
        load8<DTX>(r0, src, 8 * t, mine ? p.K - 8 * t : 0);
        u32 m = 0;
        const auto top = [&](const Raw8<DTX>& r) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const u32 b = __builtin_bit_cast(u32, get8<DTX>(r, i)) & 0x7FFFFFFFu;
                m = b > m ? b : m;
            }
        };
        top(r0);
        if (mine)
            for (int at = 8 * (t + per); at < p.K; at += 8 * per) {
                Raw8<DTX> r;
                load8<DTX>(r, src, at, p.K - at);
                top(r);
            }
        m = wave_all<MaxOp>(m);
        if ((threadIdx.x & 63) == 0 && mine)
            atomicMax(&amax[row], m);
        __syncthreads();
        if (!mine)
            return;
        RowLevels L;
        L.of_amax(amax[row]);
        if (t == 0)
            sc[row] = L.scale;
        const auto put = [&](const Raw8<DTX>& r, int at) {
            int q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if constexpr (DTX == DT_F32)
                    q[i] = L.level64(get8<DTX>(r, i));
                else
                    q[i] = L.level(get8<DTX>(r, i));
            }
            store_levels((int8_t*)levels + row * ld, at, 8, q);
        };
        const int kr = ld - 16;  // K rounded up to a run
        if (8 * t < kr)
            put(r0, 8 * t);
        for (int at = 8 * (t + per); at < kr; at += 8 * per) {
            Raw8<DTX> r;
            load8<DTX>(r, src, at, p.K - at);
            put(r, at);
        }
    }

    static __device__ __forceinline__ void run(const I8Params& p, const I8Source& x)
    {
        extern __shared__ __attribute__((aligned(16))) char gemv_lds[];
        __shared__ float sc[16];
        __shared__ u32 amax[16];
        const int tid = threadIdx.x;
        const int lane = tid & 63;
        const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int m0 = (int)blockIdx.y * TOKENS, n0 = (int)blockIdx.x * 16;
        const int ln = lane & 15, g = lane >> 4;
        RowW wr;
        RowA ar[MT];
        wr.at(p.W + (int64_t)(n0 + ln < p.N ? n0 + ln : p.N - 1) * p.ldw);
        const char* levels = nullptr;
        if constexpr (FUSED) {
            levels = gemv_lds + (ln < p.M ? ln : p.M - 1) * level_row(p.K);
        } else {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int t = m0 + 16 * m + ln;
                ar[m].at(p.A + (int64_t)(t < p.M ? t : p.M - 1) * p.lda);
            }
        }
        i32x4 acc[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m)
            acc[m] = i32x4{0, 0, 0, 0};

        // whole runs w, w + NW, ...; the partial one, if any, is run `whole`
        const int whole = p.K / RUN;
        Run R;
        int r = w;
        if (r < whole)
            load(R, wr, ar, r * RUN, p.K, g, true);
        if constexpr (FUSED) {
            if (tid < 16)
                amax[tid] = 0;
            __syncthreads();
            quantise(p, x, gemv_lds, sc, amax, level_row(p.K));
            __syncthreads();
        }
        while (r < whole) {
            const int next = r + NW;
            Run S = R;
            if (next < whole)
                load(R, wr, ar, next * RUN, p.K, g, true);
            __builtin_amdgcn_sched_barrier(0);
            multiply(acc, S, wr, ar, levels, r * RUN, g, true);
            r = next;
        }
        if (p.K % RUN != 0 && w == whole % NW) {
            load(R, wr, ar, whole * RUN, p.K, g, false);
            multiply(acc, R, wr, ar, levels, whole * RUN, g, false);
        }

        int* red = (int*)gemv_lds;
        if constexpr (FUSED)
            __syncthreads();  // the levels' last reads
#pragma unroll
        for (int m = 0; m < MT; ++m)
            *(i32x4*)&red[(w * MT + m) * 256 + lane * 4] = acc[m];
        __syncthreads();
        // lane l of a block holds token l % 16, rows 4 (l / 16) + 0 .. 3 of W
        for (int o = tid; o < MT * 256; o += NW * 64) {
            int s = 0;
#pragma unroll
            for (int v = 0; v < NW; ++v)
                s += red[v * MT * 256 + o];
            const int l = (o >> 2) & 63;
            const int m = m0 + 16 * (o >> 8) + (l & 15);
            const int n = n0 + 4 * (l >> 4) + (o & 3);
            if (m < p.M && n < p.N)
                store_out(p.C, p.dt_out, (int64_t)m * p.ldc + n,
                          i8_result(s, FUSED ? sc[m & 15] : p.sa[m], p.sw[n],
                                    p.bias ? p.bias[n] : 0.0f, p.relu));
        }
    }
};

template <int MT, int NW, int SHIFT>
__global__ __attribute__((amdgpu_flat_work_group_size(NW * 64, NW * 64))) void
i8_gemv_kernel(I8Params p)
{
    GemmParams rec{};
    rec.stamps = p.stamps;
    const ClockStamp clk = stamp_begin(rec);
    I8Gemv<DT_F32, MT, NW, SHIFT, false>::run(p, I8Source{});
    stamp_end(rec, clk);
}

struct I8LinearParams {
    I8Params p;
    I8Source x;
};

template <int DTX, int NW, int SHIFT>
__global__ __attribute__((amdgpu_flat_work_group_size(NW * 64, NW * 64))) void
i8_linear_gemv_kernel(I8LinearParams l)
{
    GemmParams rec{};
    rec.stamps = l.p.stamps;
    const ClockStamp clk = stamp_begin(rec);
    I8Gemv<DTX, 1, NW, SHIFT, true>::run(l.p, l.x);
    stamp_end(rec, clk);
}

}  // namespace tg
