// 8-bit integer matrix product with a scale for each token and channel:
//   C[m][n] = epilogue(sa[m] sw[n] sum_k A[m][k] W[n][k] + bias[n]),
// A and W in 8 bits with k contiguous, the sum exact in 32-bit integers
// (v_mfma_i32_*_i8), scales, bias and ReLU in fp32, one rounding to C's type.
// Integer sums do not depend on their order, so every kernel here gives the
// same bits.
//
// i8_dma_kernel: K % 16 == 0 and rows that start at 16-byte boundaries.  The
// 16-bit LDS-DMA kernel's scheme (tg_kernel_dma.h) on 8-bit data: an operand
// row of BK bytes to a strip is handled as BK / 2 words, so copies, LDS layout,
// swizzles and fragment addresses are those of its k-contiguous operands, and
// a fragment (16 bytes of one row for each lane) is the operand of
// v_mfma_i32_32x32x32_i8, which does twice the 16-bit instruction's work.
// Measured: 8192^3 bf16 out 444-466 us (2.4-2.5 POP/s; back to back on the same
// data 410, at 1.57 GHz, power-limited, and 81% of the matrix rate at that clock;
// 308 us and 2.28 GHz with zeros), 4096^3 56-60 us.  256 x 8192 x 8192: 24.5 us;
// its copies alone take 18.5 us from L2 and the last-level cache and 28 us from
// HBM, through LDS or registers alike, so what bounds grids of small tiles is the
// unit's path to L2 (62 GB/s of 85).  Not kept: the sums of k split over wave
// groups (same time: LDS reads are not the bound), and a dword of each row touched
// ahead to bring its line into L2 (a third slower: the lines touched count, not
// the bytes).
//
// i8_any_kernel: any sizes, strides and addresses (LDS-DMA copies want aligned
// ones).  Strips of 128 bytes of k go through registers: 16-byte loads at any
// byte, PD strips ahead, into a two-stage LDS ring.  Measured (W from HBM): 1000
// x 1001 x 1003 8.0 us with 64 x 64 tiles, 512 x 4096 x 4095 29 us with 64 x 128,
// 4096 x 4096 x 4095 127 us with 128 x 128.  Bound by the unit's path to L2: 128
// bytes of a row that starts anywhere lie in two lines, so 11 bytes reach a
// unit's registers in a cycle where the aligned copies above bring 22 (the same
// with rows at dwords, 4092 for 4095: 10 to 20% less time).  Not kept: strips of
// 256 bytes, three lines for two (256 x 4096 x 4095 21.4 us for 23.2, but 1000 x
// 1001 x 1003 9.4: half the workgroups fit); whole dwords and a shift, as the
// streaming kernel does (no gain here: the lines count); 256 x 128 tiles, four
// strips ahead (within 5%).
#pragma once

#include "tg_i8.h"
#include "tg_kernel_dma.h"

namespace tg {

// Results of one wave's FM x FN blocks through its own LDS region `st` (32
// rows of FN * 32 results), 32 rows at a time: scaled, rounded, written as
// 16-byte chunks (chunk c of row r at c ^ (r % CH)), read back whole and
// stored 16 bytes to a lane, so that a store instruction writes runs of whole
// rows.  The reads of one 32-row stripe are issued before the writes of the
// next, and a wave's LDS accesses complete in order.  The stores write through
// (kStoreThrough) as the other kernels' do (8192^3 415 us, 556 with each lane
// storing its own 4 x 4 results) (c_vec: whole aligned chunks, and 32
// rows within 31 bits of offset); other C rows take unaligned stores, and the
// chunk across column N single ones.
template <int DT, int FM, int FN>
__device__ __forceinline__ void i8_store_staged(const i32x16 (&acc)[FM][FN], const I8Params& p,
                                                int mw0, int nw0, int lane, lds_char* st)
{
    constexpr int ES = DT == DT_F32 ? 4 : 2;
    constexpr int EPC = 16 / ES;
    constexpr int ROWB = FN * 32 * ES;
    constexpr int CH = ROWB / 16;
    constexpr int RPI = 64 / CH;  // rows of a store instruction
    static_assert((CH & (CH - 1)) == 0 && CH >= 4 && CH <= 64, "rows of 64 to 1024 bytes");
    const int lr = lane & 31, g = lane >> 5;
    // scales and bias of this lane's columns: 8 q + 4 g + 0..3 of each block
    f32x4 sw[FN][4], bs[FN][4];
#pragma unroll
    for (int fn = 0; fn < FN; ++fn)
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int n = nw0 + fn * 32 + 8 * q + 4 * g + e;
                const int nc = n < p.N ? n : p.N - 1;
                sw[fn][q][e] = p.sw[nc];
                bs[fn][q][e] = p.bias ? p.bias[nc] : 0.0f;
            }
    const int c = lane % CH;
    const int n = nw0 + EPC * c;
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
        const int mr = mw0 + fm * 32 + lr;
        const float sa = p.sa[mr < p.M ? mr : p.M - 1];
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = i8_result(acc[fm][fn][4 * q + e], sa, sw[fn][q][e], bs[fn][q][e],
                                     p.relu);
                if constexpr (DT == DT_F32) {
                    const int ch = 8 * fn + 2 * q + g;
                    *(lds_u32x4*)(st + lr * ROWB + ((ch ^ (lr & (CH - 1))) << 4)) =
                        __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]});
                } else {
                    const int ch = 4 * fn + q;
                    *(lds_u32x2*)(st + lr * ROWB + ((ch ^ (lr & (CH - 1))) << 4) + 8 * g) =
                        u32x2{pack2(v[0], v[1], DT), pack2(v[2], v[3], DT)};
                }
            }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // own region: no barrier needed
        const auto rs =
            make_rsrc((char*)p.C + ((int64_t)(mw0 + fm * 32) * p.ldc + nw0) * ES, 0x7FFFFFFFu);
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += RPI) {
            const int r = r0 + lane / CH;
            const int m = mw0 + fm * 32 + r;
            const u32x4 v = *(const lds_u32x4*)(st + r * ROWB + ((c ^ (r & (CH - 1))) << 4));
            if (m >= p.M || n >= p.N)
                continue;
            if (p.c_vec) {
                __builtin_amdgcn_raw_buffer_store_b128(
                    v, rs, (int)((u32)(r * (int)p.ldc + EPC * c) * (u32)ES), 0, kStoreThrough);
                continue;
            }
            char* to = (char*)p.C + ((int64_t)m * p.ldc + n) * ES;
            if (n + EPC <= p.N) {
                struct __attribute__((packed, aligned(ES))) Any {
                    u32x4 v;
                };
                ((Any*)to)->v = v;
            } else {
#pragma unroll
                for (int e = 0; e < EPC; ++e)
                    if (n + e < p.N) {
                        const u32 w = v[e * ES / 4];
                        if constexpr (DT == DT_F32)
                            ((u32*)to)[e] = w;
                        else
                            ((uint16_t*)to)[e] = (uint16_t)(w >> (16 * (e & 1)));
                    }
            }
        }
    }
}

// BM x BN tiles, four waves in a 2 x 2 grid.  Each step reads a strip's fragments
// from one LDS stage, multiplies, writes the next strip into the other, which
// every wave has read by the barrier of the step before, and issues the loads of
// the strip PD steps on.  The row's end, if it is not a whole strip, is loaded
// first and multiplied last, so that no load in the loop needs a branch.
template <int DT, int BM, int BN, int PD>
struct I8Any {
    static constexpr int BK = 128;
    static constexpr int WTM = BM / 2, WTN = BN / 2;
    static constexpr int FM = WTM / 32, FN = WTN / 32;
    static constexpr int JA = BM / 32, JB = BN / 32;  // chunks of a thread and strip
    static constexpr int JN = JA > JB ? JA : JB;
    static constexpr int STAGE = (BM + BN) * BK;
    using Row = Row16<false>;

    struct Strip {
        typename Row::Chunk a[JA], b[JB];
    };
    struct Rows {
        Row a[JA], b[JB];
    };

    static __device__ __forceinline__ void load(Strip& s, const Rows& r, int k)
    {
#pragma unroll
        for (int j = 0; j < JA; ++j)
            s.a[j] = r.a[j].load(k);
#pragma unroll
        for (int j = 0; j < JB; ++j)
            s.b[j] = r.b[j].load(k);
    }

    static __device__ __forceinline__ void write(const Strip& s, const Rows& r, lds_char* stage,
                                                 const u32 (&st)[JN])
    {
#pragma unroll
        for (int j = 0; j < JA; ++j)
            *(lds_u32x4*)(stage + st[j]) = Row::bytes(s.a[j], r.a[j].s);
#pragma unroll
        for (int j = 0; j < JB; ++j)
            *(lds_u32x4*)(stage + BM * BK + st[j]) = Row::bytes(s.b[j], r.b[j].s);
    }

    static __device__ __forceinline__ void multiply(i32x16 (&acc)[FM][FN], const lds_char* stage,
                                                    int lane, int wm0, int wn0)
    {
        i32x4 fa[BK / 32][FM], fb[BK / 32][FN];
#pragma unroll
        for (int s = 0; s < BK / 32; ++s) {
            const int ch = 2 * s + (lane >> 5);
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                const int r = wm0 + 32 * f + (lane & 31);
                fa[s][f] = __builtin_bit_cast(
                    i32x4, *(const lds_u32x4*)(stage + r * BK + ((ch ^ swz8(r)) << 4)));
            }
#pragma unroll
            for (int f = 0; f < FN; ++f) {
                const int r = wn0 + 32 * f + (lane & 31);
                fb[s][f] = __builtin_bit_cast(
                    i32x4, *(const lds_u32x4*)(stage + BM * BK + r * BK + ((ch ^ swz8(r)) << 4)));
            }
        }
        if constexpr (FM * FN <= 2)  // all reads before the first MFMA waits for one
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < BK / 32; ++s)
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int k = 0; k < FN; ++k)
                    acc[i][k] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[s][k], fa[s][i],
                                                                     acc[i][k], 0, 0, 0);
    }

    // the LDS writes and reads of all waves, but not the loads in flight
    static __device__ __forceinline__ void publish()
    {
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }

    static __device__ __forceinline__ void run(const I8Params& p)
    {
        __shared__ __attribute__((aligned(1024))) char smem[2 * STAGE];
        lds_char* sm = (lds_char*)smem;
        const int tid = threadIdx.x;
        const int lane = tid & 63;
        const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
        const TileCoord tc = tile_of(blockIdx.x, p.tiles_m, p.tiles_n, p.group_m);
        const int m0 = tc.m * BM, n0 = tc.n * BN;
        const int wm0 = (w >> 1) * WTM, wn0 = (w & 1) * WTN;

        // thread t moves chunk t % 8 of rows t / 8 + 32 j; rows past the end
        // read the last row again (their results are not stored)
        const int c = tid & 7;
        Rows rows;
        u32 st[JN];
#pragma unroll
        for (int j = 0; j < JN; ++j) {
            const int r = (tid >> 3) + 32 * j;
            st[j] = r * BK + ((c ^ swz8(r)) << 4);
            if (j < JA)
                rows.a[j].at(p.A + (int64_t)(m0 + r < p.M ? m0 + r : p.M - 1) * p.lda);
            if (j < JB)
                rows.b[j].at(p.W + (int64_t)(n0 + r < p.N ? n0 + r : p.N - 1) * p.ldw);
        }
        i32x16 acc[FM][FN];
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    acc[i][j][r] = 0;

        const int KW = p.K / BK;  // whole strips
        const int KT = (p.K + BK - 1) / BK;
        RowEnd ea[JA], eb[JB];
        if (KT > KW) {
#pragma unroll
            for (int j = 0; j < JA; ++j)
                ea[j].load(rows.a[j].row(), KW * BK + 16 * c, p.K);
#pragma unroll
            for (int j = 0; j < JB; ++j)
                eb[j].load(rows.b[j].row(), KW * BK + 16 * c, p.K);
        }
        const auto write_end = [&](lds_char* stage) {
#pragma unroll
            for (int j = 0; j < JA; ++j)
                *(lds_u32x4*)(stage + st[j]) = ea[j].bytes();
#pragma unroll
            for (int j = 0; j < JB; ++j)
                *(lds_u32x4*)(stage + BM * BK + st[j]) = eb[j].bytes();
        };
        if (KW > 0) {
            // loads past the last whole strip read it again
            const auto at = [&](int t) { return (t < KW ? t : KW - 1) * BK + 16 * c; };
            Strip S[PD];
#pragma unroll
            for (int j = 0; j < PD; ++j)
                load(S[j], rows, at(j));
            write(S[0], rows, sm, st);
            load(S[0], rows, at(PD));
            publish();
            for (int t0 = 0; t0 < KT; t0 += PD) {
#pragma unroll
                for (int j = 0; j < PD; ++j) {
                    const int t = t0 + j;
                    if (t >= KT)
                        break;  // uniform
                    multiply(acc, sm + (t & 1) * STAGE, lane, wm0, wn0);
                    if (t + 1 < KW)
                        write(S[(j + 1) % PD], rows, sm + ((t + 1) & 1) * STAGE, st);
                    else
                        write_end(sm + ((t + 1) & 1) * STAGE);
                    load(S[(j + 1) % PD], rows, at(t + 1 + PD));
                    publish();
                }
            }
        } else if (KT > 0) {
            write_end(sm);
            publish();
            multiply(acc, sm, lane, wm0, wn0);
        }
        __syncthreads();  // the last strip's reads, before the results take their place
        constexpr int ES = DT == DT_F32 ? 4 : 2;
        static_assert(4 * 32 * WTN * ES <= 2 * STAGE, "a 32-row stripe for each wave");
        i8_store_staged<DT, FM, FN>(acc, p, m0 + wm0, n0 + wn0, lane, sm + w * (32 * WTN * ES));
    }
};

template <int DT, int BM, int BN, int PD>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(2))) void
i8_any_kernel(I8Params p)
{
    GemmParams rec{};
    rec.stamps = p.stamps;
    const ClockStamp clk = stamp_begin(rec);
    I8Any<DT, BM, BN, PD>::run(p);
    stamp_end(rec, clk);
}

// BM x BN tiles, strips of BK bytes of k, NS LDS stages, WGM x WGN waves.
// NS >= 3: one barrier for each strip, after its first MFMA: it publishes strip
// t + 1 and frees strip t - 1's stage, into which strip t + NS - 1 is copied
// over the whole strip.  NS == 2: the barrier stands at the last slab, when
// strip t's fragments are all in registers; strip t + 2 is copied into its
// stage from there on, over that slab and the next strip's first.  Fragments
// are read ahead of the MFMAs that take them, and the copies of the waves are
// staggered over the slots between MFMAs.
template <int DT, int BM, int BN, int BK, int WGM, int WGN, int NS>
struct I8Dma {
    static constexpr int NW = WGM * WGN;
    static constexpr int WTM = BM / WGM, WTN = BN / WGN;
    static constexpr int FM = WTM / 32, FN = WTN / 32;
    using OA = DmaOperand<true, BM, WTM, FM, NW, BK / 2>;
    using OB = DmaOperand<true, BN, WTN, FN, NW, BK / 2>;
    static constexpr int SL = BK / 32;  // MFMA slabs of a strip
    static constexpr int A_REGION = NS * OA::STAGE;
    static constexpr int LDS_BYTES = NS * (OA::STAGE + OB::STAGE);
    static constexpr int NM = FM * FN;
    static constexpr int NREAD = OA::NRD + OB::NRD;
    static constexpr int NCOPY = OA::J + OB::J;
    static constexpr int VM_AHEAD = NS >= 3 ? (NS - 3) * NCOPY : 0;
    static constexpr int STEPS = NM > NREAD ? NM : NREAD;
    static constexpr int SLOTS = SL * STEPS;
    static constexpr int CSLOTS = NS == 2 ? 2 * STEPS : SLOTS;
    // Fragment sets, each slab reading the one PFD = RF - 1 slabs ahead: two,
    // or four for waves of one or two MFMA blocks, whose MFMAs of one slab
    // would not cover the latency of an LDS read (three or more stages: with
    // two, no slab before the last may read the next strip).
    static constexpr int RF = (NS >= 3 && SL >= 4 && NM <= 2) ? 4 : 2;
    static constexpr int PFD = RF - 1;
    static_assert(WTM % 32 == 0 && WTN % 32 == 0, "wave tiles of whole 32x32 blocks");
    static_assert(NW <= 8 && NS >= 2 && NS <= 6, "up to eight waves, two to six stages");
    static_assert(LDS_BYTES <= 160 * 1024, "LDS budget");
    static_assert(SL >= 1 && (NS * SL) % RF == 0 && PFD <= SL && (NS > 2 || SL >= 2),
                  "the fragment sets wrap with the ring");

    static constexpr int cpos(int d, int W) { return ((d * NW + W) * CSLOTS) / (NCOPY * NW); }

    struct Frag {
        typename OA::Frag a;
        typename OB::Frag b;
    };
    struct Lane {
        typename OA::Lane a;
        typename OB::Lane b;
    };
    struct Strip {
        u32 so;    // byte offset of the strip in a row
        int krem;  // words left of k
    };

    static __device__ __forceinline__ Strip strip_of(int kw, int t)
    {
        return Strip{(u32)t * BK, kw - t * (BK / 2)};
    }

    template <int ST>
    static __device__ __forceinline__ void issue_copy(const Lane& L, const Strip& s, int d, int w,
                                                      u32 smem0)
    {
        if (d < OA::J)
            OA::template copy<ST>(L.a, typename OA::Strip{L.a.band, s.so}, s.krem, d, w, smem0);
        else
            OB::template copy<ST>(L.b, typename OB::Strip{L.b.band, s.so}, s.krem, d - OA::J, w,
                                  smem0 + A_REGION);
    }

    template <int ST>
    static __device__ __forceinline__ void issue_copies(const Lane& L, const Strip& s, int w,
                                                        u32 smem0)
    {
#pragma unroll
        for (int d = 0; d < NCOPY; ++d)
            issue_copy<ST>(L, s, d, w, smem0);
    }

    template <int ST, int S>
    static __device__ __forceinline__ void read_one(Frag& F, const Lane& L, lds_char* sm, int i)
    {
        if (i < OA::NRD)
            OA::template read<ST, S>(F.a, L.a, sm, i);
        else
            OB::template read<ST, S>(F.b, L.b, sm, i - OA::NRD);
    }

    static __device__ __forceinline__ void mfma_one(i32x16 (&acc)[FM][FN], const Frag& F, int i)
    {
        const int fm = i / FN, fn = i % FN;
        acc[fm][fn] = __builtin_amdgcn_mfma_i32_32x32x32_i8(
            __builtin_bit_cast(i32x4, F.b.v[fn]), __builtin_bit_cast(i32x4, F.a.v[fm]),
            acc[fm][fn], 0, 0, 0);
    }

    // Slot SLOT of strip t (stage ST) of wave W, then the following slots.
    template <int ST, int W, int SLOT>
    static __device__ __forceinline__ void slots(i32x16 (&acc)[FM][FN], Frag (&F)[RF],
                                                 const Lane& L, lds_char* sm, int kw, int t,
                                                 u32 smem0)
    {
        constexpr int NXT = (ST + 1) % NS;
        constexpr int S = SLOT / STEPS, I = SLOT % STEPS;
        if constexpr (I < NM) {
            mfma_one(acc, F[(ST * SL + S) % RF], I);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (NS == 2 && S == SL - 1 && I == 0) {
            wait_all_barrier();
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (NS >= 3 && SLOT == 0) {
            wait_copies_barrier<VM_AHEAD>();
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (I < NREAD) {
            constexpr int T = S + PFD;
            constexpr int SET = (ST * SL + T) % RF;
            if constexpr (T < SL)
                read_one<ST, T>(F[SET], L, sm, I);
            else
                read_one<NXT, T - SL>(F[SET], L, sm, I);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (NS >= 3) {
#pragma unroll
            for (int d = 0; d < NCOPY; ++d) {
                if (cpos(d, W) == SLOT) {
                    issue_copy<(ST + NS - 1) % NS>(L, strip_of(kw, t + NS - 1), d, W, smem0);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        } else {
            constexpr int LAST = (SL - 1) * STEPS;
#pragma unroll
            for (int d = 0; d < NCOPY; ++d) {
                if (cpos(d, W) < STEPS && LAST + cpos(d, W) == SLOT) {
                    issue_copy<ST>(L, strip_of(kw, t + 2), d, W, smem0);
                    __builtin_amdgcn_sched_barrier(0);
                } else if (cpos(d, W) >= STEPS && cpos(d, W) - STEPS == SLOT) {
                    issue_copy<NXT>(L, strip_of(kw, t + 1), d, W, smem0);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        if constexpr (SLOT + 1 < SLOTS)
            slots<ST, W, SLOT + 1>(acc, F, L, sm, kw, t, smem0);
    }

    // Strips 0 .. KT - 1, rounded up to whole rounds of the ring: strips past
    // the end copy zeros.
    template <int W>
    static __device__ __forceinline__ void main_loop(i32x16 (&acc)[FM][FN], Frag (&F)[RF],
                                                     const Lane& L, lds_char* sm, int kw, int KT,
                                                     u32 smem0)
    {
        for (int t = 0; t < KT; t += NS) {
            slots<0, W, 0>(acc, F, L, sm, kw, t, smem0);
            slots<1, W, 0>(acc, F, L, sm, kw, t + 1, smem0);
            if constexpr (NS > 2)
                slots<2 % NS, W, 0>(acc, F, L, sm, kw, t + 2, smem0);
            if constexpr (NS > 3)
                slots<3 % NS, W, 0>(acc, F, L, sm, kw, t + 3, smem0);
            if constexpr (NS > 4)
                slots<4 % NS, W, 0>(acc, F, L, sm, kw, t + 4, smem0);
            if constexpr (NS > 5)
                slots<5 % NS, W, 0>(acc, F, L, sm, kw, t + 5, smem0);
        }
    }

    template <int W>
    static __device__ __forceinline__ void loop_of(int w, i32x16 (&acc)[FM][FN], Frag (&F)[RF],
                                                   const Lane& L, lds_char* sm, int kw, int KT,
                                                   u32 smem0)
    {
        if constexpr (W + 1 < NW) {
            if (w != W)
                return loop_of<W + 1>(w, acc, F, L, sm, kw, KT, smem0);
        }
        main_loop<W>(acc, F, L, sm, kw, KT, smem0);
    }

    static __device__ __forceinline__ void run(const I8Params& p)
    {
        __shared__ __attribute__((aligned(1024))) char smem[LDS_BYTES];
        lds_char* sm = (lds_char*)smem;
        const u32 smem0 = lds_offset(smem);
        const int lane = threadIdx.x & 63;
        const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int wm = w / WGN, wn = w % WGN;
        const TileCoord tc = tile_of(blockIdx.x, p.tiles_m, p.tiles_n, p.group_m);
        const int m0 = tc.m * BM, n0 = tc.n * BN;
        const int kw = p.K / 2;  // K in 16-bit words
        const int KT = (p.K + BK - 1) / BK;

        Lane L;
        OA::setup(L.a, m0, p.M, (int)(p.lda / 2), w, lane, wm * WTM, 0, p.A, kw);
        OB::setup(L.b, n0, p.N, (int)(p.ldw / 2), w, lane, wn * WTN, A_REGION, p.W, kw);

        i32x16 acc[FM][FN];
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    acc[i][j][r] = 0;

        issue_copies<0>(L, strip_of(kw, 0), w, smem0);
        if constexpr (NS == 2) {
            // the part of strip 1 that strip -1 would have copied
#pragma unroll
            for (int d = 0; d < NCOPY; ++d)
                if (((d * NW + w) * CSLOTS) / (NCOPY * NW) < STEPS)
                    issue_copy<1>(L, strip_of(kw, 1), d, w, smem0);
        }
        if constexpr (NS > 2)
            issue_copies<1>(L, strip_of(kw, 1), w, smem0);
        if constexpr (NS > 3)
            issue_copies<2 % NS>(L, strip_of(kw, 2), w, smem0);
        if constexpr (NS > 4)
            issue_copies<3 % NS>(L, strip_of(kw, 3), w, smem0);
        if constexpr (NS > 5)
            issue_copies<4 % NS>(L, strip_of(kw, 4), w, smem0);
        wait_copies_barrier<(NS == 2 ? 0 : NS - 2) * NCOPY>();
        Frag F[RF];
#pragma unroll
        for (int i = 0; i < NREAD; ++i)
            read_one<0, 0>(F[0], L, sm, i);
        if constexpr (PFD > 1) {
#pragma unroll
            for (int i = 0; i < NREAD; ++i)
                read_one<0, 1 % SL>(F[1], L, sm, i);
#pragma unroll
            for (int i = 0; i < NREAD; ++i)
                read_one<0, 2 % SL>(F[2], L, sm, i);
        }
        loop_of<0>(w, acc, F, L, sm, kw, KT, smem0);
        // every wave's reads are done, and its copies of strips past the end
        wait_all_barrier();
        constexpr int ES = DT == DT_F32 ? 4 : 2;
        static_assert(NW * 32 * WTN * ES <= LDS_BYTES, "a 32-row stripe for each wave");
        i8_store_staged<DT, FM, FN>(acc, p, m0 + wm * WTM, n0 + wn * WTN, lane,
                                    sm + w * (32 * WTN * ES));
    }
};

template <int DT, int BM, int BN, int BK, int WGM, int WGN, int NS, int OCC>
__global__ __attribute__((amdgpu_flat_work_group_size(WGM * WGN * 64, WGM * WGN * 64),
                          amdgpu_waves_per_eu(OCC, OCC))) void
i8_dma_kernel(I8Params p)
{
    GemmParams rec{};
    rec.stamps = p.stamps;
    const ClockStamp clk = stamp_begin(rec);
    I8Dma<DT, BM, BN, BK, WGM, WGN, NS>::run(p);
    stamp_end(rec, clk);
}

}  // namespace tg
