// Linear layer in microscaled blocks (tg_linear_mx, tg_linear_mx_backward):
//   C[m][n] = epilogue(sum_k a(m, k) w(n, k) + bias[n]),
// a in E2M1 or E4M3 and w in E2M1, each 32 k of a row with one power of two;
// fp32 accumulation, one rounding to C's type.
//
// mx_linear_kernel: the tiles and main loops of tg_kernel_mx.h and
// tg_kernel_mx2.h, with bias, any C type and any C rows in the epilogue.  bf16 out:
// 8192^3 264 to 288 us (E2M1, 3.8 to 4.2 PFLOP/s, 256 x 256 tiles; MFMAs 56% busy at
// the power-limited clock, the units' LDS behind them) and 445 us (E4M3, 2.5 PFLOP/s,
// 128 x 256 tiles), 2048 x 4096 x 4096 25 and 31 us (128 x 256), 1000 x 1001 x 1024
// 5.6 us (64 x 64; launch, and latency of eight steps of k).
//
// mx_stream_kernel: for few tokens the time is that of streaming W once, so W
// goes from memory straight into the operand registers of
// v_mfma_scale_f32_16x16x128_f8f6f4, with no LDS on its way.
//  * Lane layout of that instruction (measured with an in-bounds probe): lane l
//    supplies row l % 16 and, with g = l / 16, the scale byte of k-block g and, in
//    E2M1, that block's 16 bytes; in E4M3 its bytes 0 .. 15 are k = 16 g .. and
//    16 .. 31 are k = 64 + 16 g ..; it holds results of column l % 16 (second
//    operand), rows 4 g + 0 .. 3.
//  * A workgroup owns 16 NT rows of W and 16 MT tokens, and all of k; its NW waves
//    take runs of 128 ST k in turn.  An instruction loads 64 bytes of 16 rows; with
//    ST 4 one more loads the 16 scale bytes that each row has in the run (a dword for
//    each 128 k touches as many cache lines as the codes: 16 x 8192 x 8192 E4M3 17.2
//    us, and 13.2).  32 or 64 rows share the reads of the activations, which every
//    workgroup takes whole, where there are workgroups enough (128 x 4096 x 4096 E4M3
//    13.3 us with 64 rows and 32 tokens, 18.0 with 32 rows, 27.2 with 16 and 16).
//  * The loads of a wave's next run are issued before the MFMAs of this one.
//  * E4M3 activations go in two halves (mx_halves), whose products are exact: 16 x
//    8192 x 8192 took 16.2 us in both launches with one instruction, now 16.9 (half of
//    it the second instruction, half the masks).  The comparisons above are of one.
//  * The waves' sums are added in LDS, in the waves' order.
//  * Rows past M or N read the last row again; their results are not stored.
//  * FUSED: the activations are given in 16 or 32 bits and every workgroup
//    quantises them itself, into LDS, while its first loads of W are in flight:
//    one launch instead of two.
// Bound by the stream of W and, on small ones, by launch and latency.  8192 x 8192 with
// W from HBM (36 MB): 16 tokens 12.3 us (2.9 TB/s; a large copy reaches 5.2), in E4M3
// 14.8, 32 tokens 14.6 and 19.3; FUSED one token 12.4, on 1024 x 1024 3.4 us.
#pragma once

#include "tg_kernel_mx2.h"
#include "tg_mx.h"

namespace tg {

struct MxLinearParams {
    GemmParams g;  // A, As, B (W), Bs, C, M, N, K (padded), tiles, relu, c_vec, group_m, stamps
    const float* bias;  // [N] or NULL
    int64_t ldc;
};

// Results of one wave's FM x FN blocks (lane l holds row l % 32 and, for element
// 4 q + e, column 8 q + 4 (l / 32) + e of a block) through its own LDS region
// `st` (32 rows of FN * 32 results), 32 rows at a time: rounded, written as
// 16-byte chunks (chunk c of row r at c ^ (r % CH)), read back and stored 16
// bytes to a lane, so that a store instruction writes runs of whole rows.  c_vec:
// whole aligned chunks and 32 rows within 31 bits of offset; other C rows take
// unaligned stores, and the chunk across column N single ones.
template <int DT, int FM, int FN>
__device__ __forceinline__ void mx_store_staged(const f32x16 (&acc)[FM][FN],
                                                const MxLinearParams& p, int mw0, int nw0,
                                                int lane, lds_char* st)
{
    constexpr int ES = DT == DT_F32 ? 4 : 2;
    constexpr int EPC = 16 / ES;
    constexpr int ROWB = FN * 32 * ES;
    constexpr int CH = ROWB / 16;
    constexpr int RPI = 64 / CH;  // rows of a store instruction
    static_assert((CH & (CH - 1)) == 0 && CH >= 4 && CH <= 64, "rows of 64 to 1024 bytes");
    const GemmParams& g = p.g;
    const int lr = lane & 31, h = lane >> 5;
    f32x4 bs[FN][4];
#pragma unroll
    for (int fn = 0; fn < FN; ++fn)
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int n = nw0 + fn * 32 + 8 * q + 4 * h + e;
                bs[fn][q][e] = p.bias ? p.bias[n < g.N ? n : g.N - 1] : 0.0f;
            }
    const int c = lane % CH;
    const int n = nw0 + EPC * c;
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = mx_result(acc[fm][fn][4 * q + e], bs[fn][q][e], g.relu);
                if constexpr (DT == DT_F32) {
                    const int ch = 8 * fn + 2 * q + h;
                    *(lds_u32x4*)(st + lr * ROWB + ((ch ^ (lr & (CH - 1))) << 4)) =
                        __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]});
                } else {
                    const int ch = 4 * fn + q;
                    *(lds_u32x2*)(st + lr * ROWB + ((ch ^ (lr & (CH - 1))) << 4) + 8 * h) =
                        u32x2{pack2(v[0], v[1], DT), pack2(v[2], v[3], DT)};
                }
            }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // own region: no barrier needed
        const auto rs =
            make_rsrc((char*)g.C + ((int64_t)(mw0 + fm * 32) * p.ldc + nw0) * ES, 0x7FFFFFFFu);
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += RPI) {
            const int r = r0 + lane / CH;
            const int m = mw0 + fm * 32 + r;
            const u32x4 v = *(const lds_u32x4*)(st + r * ROWB + ((c ^ (r & (CH - 1))) << 4));
            if (m >= g.M || n >= g.N)
                continue;
            if (g.c_vec) {
                __builtin_amdgcn_raw_buffer_store_b128(
                    v, rs, (int)((u32)(r * (int)p.ldc + EPC * c) * (u32)ES), 0, kStoreThrough);
                continue;
            }
            char* to = (char*)g.C + ((int64_t)m * p.ldc + n) * ES;
            if (n + EPC <= g.N) {
                struct __attribute__((packed, aligned(ES))) Any {
                    u32x4 v;
                };
                ((Any*)to)->v = v;
            } else {
#pragma unroll
                for (int e = 0; e < EPC; ++e)
                    if (n + e < g.N) {
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

// G: DmaMx or DmaMx2 of a tile.
template <class G, int DT>
__device__ __forceinline__ void mx_linear_run(const MxLinearParams& p, int group_m)
{
    constexpr int NW = G::NW, WTM = G::WTM, WTN = G::WTN, FM = G::FM, FN = G::FN;
    constexpr int WGN = G::BNT / WTN;
    constexpr int ES = DT == DT_F32 ? 4 : 2;
    static_assert(NW * 32 * WTN * ES <= G::LDS_BYTES, "32 staged rows to a wave");
    __shared__ __attribute__((aligned(1024))) char smem[G::LDS_BYTES];
    lds_char* sm = (lds_char*)smem;
    const u32 smem0 = lds_offset(smem);
    const GemmParams& g = p.g;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int wm = w / WGN, wn = w % WGN;
    const TileCoord tc = tile_of(blockIdx.x, g.tiles_m, g.tiles_n, group_of(g, group_m));
    const int m0 = tc.m * G::BMT, n0 = tc.n * G::BNT;
    const int KT = (g.K + G::BK - 1) / G::BK;
    typename G::Lane L;
    G::setup(L, g, m0, n0, w, lane, wm, wn);
    f32x16 acc[FM][FN];
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                acc[fm][fn][r] = 0.0f;
    switch (w) {
    case 0:
        G::template main_loop<0>(acc, L, sm, g, m0, n0, KT, smem0);
        break;
    case 1:
        G::template main_loop<1>(acc, L, sm, g, m0, n0, KT, smem0);
        break;
    case 2:
        G::template main_loop<2>(acc, L, sm, g, m0, n0, KT, smem0);
        break;
    case 3:
        G::template main_loop<3>(acc, L, sm, g, m0, n0, KT, smem0);
        break;
    case 4:
        G::template main_loop<4 % NW>(acc, L, sm, g, m0, n0, KT, smem0);
        break;
    case 5:
        G::template main_loop<5 % NW>(acc, L, sm, g, m0, n0, KT, smem0);
        break;
    case 6:
        G::template main_loop<6 % NW>(acc, L, sm, g, m0, n0, KT, smem0);
        break;
    default:
        G::template main_loop<7 % NW>(acc, L, sm, g, m0, n0, KT, smem0);
        break;
    }
    wait_all_barrier();  // every wave's copies landed and reads done
    mx_store_staged<DT, FM, FN>(acc, p, m0 + wm * WTM, n0 + wn * WTN, lane,
                                sm + w * (32 * WTN * ES));
}

// The 256-k strips of tg_kernel_mx2.h for any K that is a whole number of 128: after
// its groups of four strips come up to three single ones, and the first two steps of
// a last one.  What the copies of that one bring from past a row's end (the next
// row, zeros past the last) is not multiplied.
template <int AFMT, int BM, int BN, int WGM, int WGN, bool WHOLE>
struct DmaMx2Any : DmaMx2<AFMT, BM, BN, WGM, WGN, 4, WHOLE> {
    using Base = DmaMx2<AFMT, BM, BN, WGM, WGN, 4, WHOLE>;
    using typename Base::Frag;
    using typename Base::Lane;
    using typename Base::Res;
    using typename Base::Scales;
    using typename Base::StripOff;
    static constexpr int FM = Base::FM, FN = Base::FN, NM = Base::NM, NRD = Base::NRD;

    // Steps 0 and 1 of the strip in stage ST, whose step 0 is in F[0].
    template <int ST, int CUR>
    static __device__ __forceinline__ void half(f32x16 (&acc)[FM][FN], Frag (&F)[2],
                                                const Scales (&SC)[2], const Lane& L, lds_char* sm)
    {
#pragma unroll
        for (int i = 0; i < NRD; ++i)
            Base::template read_one<ST, 1>(F[1], L, sm, i);
#pragma unroll
        for (int i = 0; i < NM; ++i)
            Base::template mfma_one<0>(acc, F[0], SC[CUR], L, i);
#pragma unroll
        for (int i = 0; i < NM; ++i)
            Base::template mfma_one<1>(acc, F[1], SC[CUR], L, i);
    }

    template <int W>
    static __device__ __forceinline__ void main_loop(f32x16 (&acc)[FM][FN], const Lane& L,
                                                     lds_char* sm, const GemmParams& p, int m0,
                                                     int n0, int, u32 smem0)
    {
        const Res res = Base::band_res(p, m0, n0);
#pragma unroll
        for (int d = 0; d < Base::JS; ++d)
            Base::template issue_chunk<W>(L, res, p, 0, d, smem0);
        {
            const StripOff o0 = Base::strip_off(p, 0), o1 = Base::strip_off(p, 1);
#pragma unroll
            for (int d = 0; d < Base::NCOPY; ++d) {
                Base::template issue_copy<0, W>(L, res, o0, d, smem0);
                if (Base::cpos(d, W) < Base::STEPS)
                    Base::template issue_copy<1, W>(L, res, o1, d, smem0);
            }
        }
        wait_all_barrier();
        Frag F[2];
        Scales SC[2];
        Base::template read_scales<0>(SC[0], L, sm, 0);
#pragma unroll
        for (int i = 0; i < NRD; ++i)
            Base::template read_one<0, 0>(F[0], L, sm, i);
        const int whole = p.K / 256;
        const bool rest = p.K % 256 != 0;
        int t = 0;
        for (; t + 4 <= whole; t += 4) {
            Base::template strip<0, 0, W>(acc, F, SC, L, res, sm, p, t, smem0);
            Base::template strip<1, 1, W>(acc, F, SC, L, res, sm, p, t + 1, smem0);
            Base::template strip<0, 2, W>(acc, F, SC, L, res, sm, p, t + 2, smem0);
            Base::template strip<1, 3, W>(acc, F, SC, L, res, sm, p, t + 3, smem0);
        }
        if (t < whole) {
            Base::template strip<0, 0, W>(acc, F, SC, L, res, sm, p, t, smem0);
            if (t + 1 < whole) {
                Base::template strip<1, 1, W>(acc, F, SC, L, res, sm, p, t + 1, smem0);
                if (t + 2 < whole) {
                    Base::template strip<0, 2, W>(acc, F, SC, L, res, sm, p, t + 2, smem0);
                    if (rest)
                        half<1, 1>(acc, F, SC, L, sm);
                } else if (rest) {
                    half<0, 0>(acc, F, SC, L, sm);
                }
            } else if (rest) {
                half<1, 1>(acc, F, SC, L, sm);
            }
        } else if (rest) {
            half<0, 0>(acc, F, SC, L, sm);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
};

// A tile's kernel.  KIND 0: strips of 128 k; 1: of 256, K a whole number of 1024; 2:
// of 256, any K.
enum { MX_S128 = 0, MX_S256_1024 = 1, MX_S256 = 2 };
// E4M3 products exact (two instructions for one).  fp32 C shows what is cut off of them
// otherwise; in 16 bits it is far less than C's last step, and the tiles are bound by
// those instructions: 8192^3 bf16 460 us, and 869 with both; 2048 x 4096 x 4096 39 and 60 (fp32 C 45 and
// 68).
constexpr bool mx_whole(int dt, int afmt) { return afmt == MX_E4M3 && dt == DT_F32; }
template <int KIND, int DT, int AFMT, int BM, int BN, int WGM, int WGN, int NS>
struct MxTileOf;
template <int DT, int AFMT, int BM, int BN, int WGM, int WGN, int NS>
struct MxTileOf<MX_S128, DT, AFMT, BM, BN, WGM, WGN, NS>
    : DmaMx<AFMT, BM, BN, WGM, WGN, NS, 4, false, mx_whole(DT, AFMT)> {
    static constexpr int BMT = BM, BNT = BN;
    static constexpr int OCC = MxOcc<AFMT, BM, BN, WGM * WGN>::value;
};
template <int DT, int AFMT, int BM, int BN, int WGM, int WGN, int NS>
struct MxTileOf<MX_S256_1024, DT, AFMT, BM, BN, WGM, WGN, NS>
    : DmaMx2<AFMT, BM, BN, WGM, WGN, 4, mx_whole(DT, AFMT)> {
    static constexpr int BMT = BM, BNT = BN;
    static constexpr int OCC = WGM * WGN > 4 ? 2 : 1;
};
template <int DT, int AFMT, int BM, int BN, int WGM, int WGN, int NS>
struct MxTileOf<MX_S256, DT, AFMT, BM, BN, WGM, WGN, NS>
    : DmaMx2Any<AFMT, BM, BN, WGM, WGN, mx_whole(DT, AFMT)> {
    static constexpr int BMT = BM, BNT = BN;
    static constexpr int OCC = WGM * WGN > 4 ? 2 : 1;
};

template <int KIND, int DT, int AFMT, int BM, int BN, int WGM, int WGN, int NS>
__global__ __attribute__((
    amdgpu_flat_work_group_size(WGM * WGN * 64, WGM * WGN * 64),
    amdgpu_waves_per_eu(MxTileOf<KIND, DT, AFMT, BM, BN, WGM, WGN, NS>::OCC,
                        MxTileOf<KIND, DT, AFMT, BM, BN, WGM, WGN, NS>::OCC))) void
mx_linear_kernel(MxLinearParams p)
{
    const ClockStamp clk = stamp_begin(p.g);
    mx_linear_run<MxTileOf<KIND, DT, AFMT, BM, BN, WGM, WGN, NS>, DT>(p, 4);
    stamp_end(p.g, clk);
}

// --------------------------------------------------------------------------
// Few tokens.
// --------------------------------------------------------------------------
struct MxStreamParams {
    MxLinearParams l;
    int dt_out;
    const void* X;  // FUSED: activations [M][ldx], Kx columns
    int64_t ldx;
    int Kx;
};

// NT groups of 16 rows of W and MT of 16 tokens to a workgroup; runs of ST steps of
// 128 k (ST 4: a row's scale bytes of a run are one 16-byte load).
template <int DTX, int AFMT, int NT, int MT, int ST, int NW, bool FUSED>
struct MxStream {
    static constexpr bool A8 = AFMT == MX_E4M3;
    // Sums of the two halves: apart where a wave has one group of rows, whose second
    // instruction would wait for its first (one token, 8192 x 8192: 10.8 us, together 11.1);
    // together otherwise (16 tokens 16.9 us, apart 17.1).
    static constexpr int NH = A8 && FUSED ? 2 : 1;
    static constexpr int RUN = 128 * ST;
    static constexpr int TOKENS = 16 * MT, ROWS = 16 * NT;

    // FUSED: LDS bytes of a token's codes, 16 apart from a multiple of the bank
    // line so that the rows of a fragment read spread, and of its scales.
    static __host__ __device__ __forceinline__ int code_row(int Kp)
    {
        return (int)mx_bytes<AFMT>(Kp) + 16;
    }
    static __host__ __device__ __forceinline__ int lds_bytes(int M, int Kp)
    {
        const int a = FUSED ? M * (code_row(Kp) + Kp / 32) : 0, r = NW * NT * MT * 1024;
        return a > r ? a : r;
    }

    struct Run {
        u32x4 w[NT][ST];
        u32 ws[NT][ST];
        u32x4 a[FUSED ? 1 : MT][ST][A8 ? 2 : 1];
        u32 as[FUSED ? 1 : MT][ST];
    };
    struct Rows {
        const uint8_t *w[NT], *ws[NT];
        const uint8_t *a[MT], *as[MT];
    };

    static __device__ __forceinline__ void load_scales(u32 (&s)[ST], const uint8_t* p, bool whole)
    {
        if constexpr (ST == 4) {
            if (whole) {
                struct __attribute__((packed, aligned(4))) Any {
                    u32x4 v;
                };
                const u32x4 v = ((const Any*)p)->v;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[i] = v[i];
                return;
            }
        }
#pragma unroll
        for (int i = 0; i < ST; ++i)
            s[i] = whole || i == 0 ? ((const u32*)p)[i] : 0;
    }
    // A whole run at k0, or its first step.
    static __device__ __forceinline__ void load(Run& R, const Rows& at, int k0, bool whole, int g)
    {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int s = 0; s < ST; ++s)
                if (whole || s == 0)
                    R.w[n][s] = *(const u32x4*)(at.w[n] + k0 / 2 + 64 * s + 16 * g);
            load_scales(R.ws[n], at.ws[n] + k0 / 32, whole);
        }
        if constexpr (!FUSED) {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int s = 0; s < ST; ++s)
                    if (whole || s == 0) {
                        const uint8_t* a = at.a[m] + mx_bytes<AFMT>(k0 + 128 * s) + 16 * g;
                        R.a[m][s][0] = *(const u32x4*)a;
                        if constexpr (A8)
                            R.a[m][s][1] = *(const u32x4*)(a + 64);
                    }
                load_scales(R.as[m], at.as[m] + k0 / 32, whole);
            }
        }
    }

    static __device__ __forceinline__ void multiply(f32x4 (&acc)[NT][MT][NH], const Run& R,
                                                    const uint8_t* codes, const uint8_t* scales,
                                                    int k0, bool whole, int g)
    {
#pragma unroll
        for (int s = 0; s < ST; ++s) {
            if (!whole && s > 0)
                break;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                u32x4 lo, hi;
                u32 as;
                if constexpr (FUSED) {
                    const uint8_t* a = codes + mx_bytes<AFMT>(k0 + 128 * s) + 16 * g;
                    lo = *(const u32x4*)a;
                    hi = A8 ? *(const u32x4*)(a + (A8 ? 64 : 0)) : u32x4{0, 0, 0, 0};
                    as = *(const u32*)(scales + k0 / 32 + 4 * s);
                } else {
                    lo = R.a[m][s][0];
                    hi = A8 ? R.a[m][s][A8 ? 1 : 0] : u32x4{0, 0, 0, 0};
                    as = R.as[m][s];
                }
                const i32x8 aop = {(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
                                   (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
                const MxHalves half = A8 ? mx_halves(aop) : MxHalves{aop, aop};
                // first one half of all rows, then the other
#pragma unroll
                for (int h = 0; h < (A8 ? 2 : 1); ++h)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const u32x4 w = R.w[n][s];
                        const i32x8 wop = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
                        acc[n][m][h % NH] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            wop, h ? half.small : half.large, acc[n][m][h % NH], MX_E2M1, AFMT, 0,
                            (int)(R.ws[n][s] >> (8 * g)), 0, (int)(as >> (8 * g)));
                    }
            }
        }
    }

    // The M tokens' blocks into LDS: rows of code_row(Kp) bytes, then the scales.
    static __device__ __forceinline__ void quantise(const MxStreamParams& p, uint8_t* codes,
                                                    uint8_t* scales)
    {
        // eight elements to a thread, four times at once; whole quads: per % 16 == 0
        constexpr int NT_ = NW * 64, U = 4;
        const int Kp = p.l.g.K, per = Kp / 8, row_b = code_row(Kp), total = p.l.g.M * per;
        for (int u0 = threadIdx.x; u0 < total; u0 += U * NT_) {
            Raw8<DTX> r[U];
            int row[U], k[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int u = u0 + i * NT_;
                row[i] = u / per;
                k[i] = 8 * (u - row[i] * per);
                if (u < total)
                    load8<DTX>(r[i], elem_ptr<DTX>(p.X, row[i] * p.ldx), k[i], p.Kx - k[i]);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (u0 + i * NT_ >= total)
                    break;
                u32 byte;
                const u32x2 w = mx_codes<DTX, AFMT>(r[i], byte);
                uint8_t* to = codes + row[i] * row_b + mx_bytes<AFMT>(k[i]);
                if constexpr (A8)
                    *(u32x2*)to = w;
                else
                    *(u32*)to = w[0];
                if ((k[i] & 31) == 0)
                    scales[row[i] * (Kp / 32) + k[i] / 32] = (uint8_t)byte;
            }
        }
    }

    static __device__ __forceinline__ void run(const MxStreamParams& p)
    {
        extern __shared__ __attribute__((aligned(16))) uint8_t mx_lds[];
        const GemmParams& gp = p.l.g;
        const int tid = threadIdx.x;
        const int lane = tid & 63;
        const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int m0 = (int)blockIdx.y * TOKENS, n0 = (int)blockIdx.x * ROWS;
        const int ln = lane & 15, g = lane >> 4;
        const int K = gp.K;
        Rows at;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int r = n0 + 16 * i + ln;
            const int64_t n = r < gp.N ? r : gp.N - 1;
            at.w[i] = (const uint8_t*)gp.B + n * (K / 2);
            at.ws[i] = (const uint8_t*)gp.Bs + n * (K / 32);
        }
        const uint8_t *codes = nullptr, *scales = nullptr;
        if constexpr (FUSED) {
            const int m = ln < gp.M ? ln : gp.M - 1;
            codes = mx_lds + m * code_row(K);
            scales = mx_lds + gp.M * code_row(K) + m * (K / 32);
        } else {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int t = m0 + 16 * i + ln;
                const int64_t m = t < gp.M ? t : gp.M - 1;
                at.a[i] = (const uint8_t*)gp.A + m * mx_bytes<AFMT>(K);
                at.as[i] = (const uint8_t*)gp.As + m * (K / 32);
            }
        }
        f32x4 acc[NT][MT][NH];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < NH; ++h)
                    acc[n][m][h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        // whole runs w, w + NW, ...; the steps of a partial one go to the waves after
        const int whole = K / RUN, rest = K % RUN / 128;
        Run R;
        int r = w;
        if (r < whole)
            load(R, at, r * RUN, true, g);
        if constexpr (FUSED) {
            quantise(p, mx_lds, mx_lds + gp.M * code_row(K));
            __syncthreads();
        }
        while (r < whole) {
            const int next = r + NW;
            Run S = R;
            if (next < whole)
                load(R, at, next * RUN, true, g);
            __builtin_amdgcn_sched_barrier(0);
            multiply(acc, S, codes, scales, r * RUN, true, g);
            r = next;
        }
        if constexpr (ST > 1) {
            const int step = (w - whole % NW + NW) % NW;
            if (step < rest) {
                load(R, at, whole * RUN + 128 * step, false, g);
                multiply(acc, R, codes, scales, whole * RUN + 128 * step, false, g);
            }
        }
        float* red = (float*)mx_lds;
        if constexpr (FUSED)
            __syncthreads();  // the codes' last reads
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                *(f32x4*)&red[((w * NT + n) * MT + m) * 256 + lane * 4] =
                    NH == 2 ? acc[n][m][0] + acc[n][m][NH - 1] : acc[n][m][0];
        __syncthreads();
        // element e of lane l: token l % 16, row 4 (l / 16) + e of its block; threads
        // go along the rows
        for (int o = tid; o < NT * MT * 256; o += NW * 64) {
            const int nr = o % ROWS, mr = o / ROWS;
            const int at_r = ((nr >> 4) * MT + (mr >> 4)) * 256 +
                             (((nr & 15) >> 2) * 16 + (mr & 15)) * 4 + (nr & 3);
            float s = 0.0f;
#pragma unroll
            for (int v = 0; v < NW; ++v)
                s += red[v * NT * MT * 256 + at_r];
            const int m = m0 + mr, n = n0 + nr;
            if (m < gp.M && n < gp.N) {
                const float v = mx_result(s, p.l.bias ? p.l.bias[n] : 0.0f, gp.relu);
                const int64_t c = (int64_t)m * p.l.ldc + n;
                if (p.dt_out == DT_F32)
                    ((float*)gp.C)[c] = v;
                else
                    ((uint16_t*)gp.C)[c] = cvt1(v, p.dt_out);
            }
        }
    }
};

template <int DTX, int AFMT, int NT, int MT, int ST, int NW, bool FUSED>
__global__ __attribute__((amdgpu_flat_work_group_size(NW * 64, NW * 64))) void
mx_stream_kernel(MxStreamParams p)
{
    const ClockStamp clk = stamp_begin(p.l.g);
    MxStream<DTX, AFMT, NT, MT, ST, NW, FUSED>::run(p);
    stamp_end(p.l.g, clk);
}

}  // namespace tg
