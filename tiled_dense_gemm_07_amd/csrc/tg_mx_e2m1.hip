// Product in microscaled blocks with E2M1 activations: its kernels and their costs.
#include "tg_kernel_mx_linear.h"
#include "tg_mx_kernels.h"

namespace tg {

static const MxKernel kKernels[] = {
    TG_MX_STREAM(MX_E2M1, 1, 1, 4, 4, 1, 2.08f, 0.0565f, 0.08f, 0.0611f),
    TG_MX_STREAM(MX_E2M1, 1, 1, 4, 8, 1, 2.09f, 0.0521f, 0.23f, 0.0611f),
    TG_MX_STREAM(MX_E2M1, 2, 1, 4, 4, 2, 2.2f, 0.0929f, 0.44f, 0.1914f),
    TG_MX_STREAM(MX_E2M1, 2, 2, 2, 8, 1, 2.39f, 0.1114f, 1.05f, 0.149f),
    TG_MX_TILE(MX_S128, MX_E2M1, 64, 64, 2, 2, 4, 128, 3.05f, 0.1963f, 0.6f, 0.2093f),
    TG_MX_TILE(MX_S256, MX_E2M1, 64, 64, 2, 2, 2, 128, 3.12f, 0.2207f, 1.66f, 0.2292f),
    TG_MX_TILE(MX_S256, MX_E2M1, 128, 128, 2, 4, 2, 128, 3.76f, 0.319f, 2.47f, 0.3431f),
    TG_MX_TILE(MX_S256, MX_E2M1, 256, 128, 2, 4, 2, 128, 5.11f, 0.4695f, 3.21f, 0.5066f),
    TG_MX_TILE(MX_S256, MX_E2M1, 128, 256, 2, 4, 2, 128, 5.22f, 0.4618f, 3.32f, 0.496f),
    TG_MX_TILE(MX_S128, MX_E2M1, 256, 256, 2, 4, 4, 128, 7.4f, 0.7563f, 4.16f, 0.9746f),
    TG_MX_TILE(MX_S256_1024, MX_E2M1, 256, 256, 2, 4, 2, 1024, 7.61f, 0.6678f, 2.7f, 0.8306f),
};

MxKernels mx_kernels_e2m1()
{
    return {kKernels, kKernels + sizeof(kKernels) / sizeof(kKernels[0])};
}

}  // namespace tg
