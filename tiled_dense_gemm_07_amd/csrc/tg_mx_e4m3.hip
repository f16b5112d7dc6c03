// Product in microscaled blocks with E4M3 activations: its kernels and their costs.
// (256 x 256 tiles on eight waves need more registers than there are: 8192^3 481 us,
// 445 with 128 x 256; 2048 x 8192 x 8192 120 and 111.)
#include "tg_kernel_mx_linear.h"
#include "tg_mx_kernels.h"

namespace tg {

static const MxKernel kKernels[] = {
    TG_MX_STREAM(MX_E4M3, 1, 1, 4, 4, 2.08f, 0.0816f, 0.13f, 0.0874f),
    TG_MX_STREAM(MX_E4M3, 1, 1, 4, 8, 2.17f, 0.0746f, 0.35f, 0.0956f),
    TG_MX_STREAM(MX_E4M3, 2, 1, 4, 4, 2.28f, 0.1171f, 0.36f, 0.1204f),
    TG_MX_STREAM(MX_E4M3, 2, 2, 4, 4, 2.55f, 0.1625f, 1.07f, 0.1962f),
    TG_MX_STREAM(MX_E4M3, 4, 2, 4, 4, 3.08f, 0.2382f, 1.52f, 0.2812f),
    TG_MX_TILE(MX_S128, MX_E4M3, 64, 64, 2, 2, 4, 128, 3.31f, 0.2197f, 1.68f, 0.2535f),
    TG_MX_TILE(MX_S256, MX_E4M3, 128, 128, 2, 4, 2, 128, 4.05f, 0.4018f, 2.55f, 0.4553f),
    TG_MX_TILE(MX_S256, MX_E4M3, 128, 256, 2, 4, 2, 128, 5.56f, 0.6108f, 3.59f, 0.67f),
};

MxKernels mx_kernels_e4m3()
{
    return {kKernels, kKernels + sizeof(kKernels) / sizeof(kKernels[0])};
}

}  // namespace tg
