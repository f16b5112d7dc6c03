// Product in microscaled blocks with E2M1 activations: its kernels and their costs.
#include "tg_kernel_mx_linear.h"
#include "tg_mx_kernels.h"

namespace tg {

static const MxKernel kKernels[] = {
    TG_MX_STREAM(MX_E2M1, 1, 1, 4, 4, 2.09f, 0.0598f, 0.09f, 0.0621f),
    TG_MX_STREAM(MX_E2M1, 1, 1, 4, 8, 2.12f, 0.0566f, 0.24f, 0.0605f),
    TG_MX_STREAM(MX_E2M1, 2, 1, 4, 4, 2.25f, 0.0981f, 0.26f, 0.0955f),
    TG_MX_STREAM(MX_E2M1, 2, 2, 4, 4, 2.51f, 0.1226f, 0.45f, 0.1302f),
    TG_MX_STREAM(MX_E2M1, 4, 2, 4, 4, 3.07f, 0.187f, 1.57f, 0.2177f),
    TG_MX_TILE(MX_S128, MX_E2M1, 64, 64, 2, 2, 4, 128, 3.05f, 0.1963f, 0.6f, 0.2093f),
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
