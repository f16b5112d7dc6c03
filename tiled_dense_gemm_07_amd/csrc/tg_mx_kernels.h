// Kernels of the product in microscaled blocks, and what they cost: one table for
// each format of the activations, each in a source file of its own.
#pragma once

#include <stdint.h>

namespace tg {

// One of the product's kernels, and what it costs on this card in microseconds: t0 +
// strips of 128 k times `one` while its workgroups are at most 256, else for each
// round of 256 workgroups `round` + strips times `full`.  The tiles' rows were fitted to
// 270 to 330 shapes of each format (M 1 to 8192, N 128 to 14336, K 128 to 8192, odd ones
// among them), within 8 to 13% on average; the streams' rows afterwards to shapes of up
// to 256 tokens alone, E4M3 with one instruction (two take some 4% more) and a 16-bit
// C.  The choice by both was then 2.8% (E2M1) and 3.1% (E4M3) on average above the
// fastest of all that were measured: 30% at most on calls of a few microseconds, but 60%
// on 64 tokens by weights of 25 MB in E4M3, since the cost does not know HBM from the
// cache.
struct MxKernel {
    const char* name;
    const void* kernel[3];  // by C's type
    int bm, bn, threads;
    int strip;      // K has to be a multiple of it
    unsigned lds;   // bytes, streaming kernels (0: a tile)
    float t0, one, round, full;
};

struct MxKernels {
    const MxKernel* begin;
    const MxKernel* end;
};
MxKernels mx_kernels_e2m1();
MxKernels mx_kernels_e4m3();

#define TG_MX_TILE(KIND, AFMT, BM, BN, WGM, WGN, NS, STRIP, T0, ONE, ROUND, FULL)                  \
    {                                                                                              \
        "mx_linear_" #AFMT "_" #BM "x" #BN "_w" #WGM "x" #WGN "_s" #NS "_" #KIND,                  \
            {(const void*)&tg::mx_linear_kernel<tg::KIND, tg::DT_F32, tg::AFMT, BM, BN, WGM, WGN,  \
                                                NS>,                                               \
             (const void*)&tg::mx_linear_kernel<tg::KIND, tg::DT_F16, tg::AFMT, BM, BN, WGM, WGN,  \
                                                NS>,                                               \
             (const void*)&tg::mx_linear_kernel<tg::KIND, tg::DT_BF16, tg::AFMT, BM, BN, WGM, WGN, \
                                                NS>},                                              \
            BM, BN, WGM* WGN * 64, STRIP, 0, T0, ONE, ROUND, FULL                                  \
    }
#define TG_MX_STREAM(AFMT, NT, MT, ST, NW, T0, ONE, ROUND, FULL)                                  \
    {                                                                                             \
        "mx_stream_" #AFMT "_n" #NT "_m" #MT "_st" #ST "_w" #NW,                                  \
            {(const void*)&tg::mx_stream_kernel<tg::DT_F32, tg::AFMT, NT, MT, ST, NW, false>,     \
             (const void*)&tg::mx_stream_kernel<tg::DT_F32, tg::AFMT, NT, MT, ST, NW, false>,     \
             (const void*)&tg::mx_stream_kernel<tg::DT_F32, tg::AFMT, NT, MT, ST, NW, false>},    \
            16 * MT, 16 * NT, NW * 64, 128, NW* NT* MT * 1024, T0, ONE, ROUND, FULL               \
    }

}  // namespace tg
