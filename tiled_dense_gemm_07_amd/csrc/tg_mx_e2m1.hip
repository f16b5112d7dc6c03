// Product in microscaled blocks with E2M1 activations: its kernels and their costs.
#include "tg_kernel_mx_linear.h"
#include "tg_mx_kernels.h"

namespace tg {

static const MxKernel kKernels[] = {
    TG_MX_STREAM(MX_E2M1, 1, 1, 4, 4, 1, 2.08f, 0.0565f, 0.08f, 0.0611f),
    TG_MX_STREAM(MX_E2M1, 1, 1, 4, 8, 1, 2.09f, 0.0521f, 0.23f, 0.0611f),
    TG_MX_STREAM(MX_E2M1, 2, 1, 4, 4, 2, 2.2f, 0.0929f, 0.44f, 0.1914f),
    TG_MX_STREAM(MX_E2M1, 2, 2, 2, 8, 1, 2.39f, 0.1114f, 1.05f, 0.149f),
    TG_MX_TILE(MX_S128, MX_E2M1, 64, 64, 2, 2, 4, 128, 3.05f, 0.1963f, 0.6f, 0.2099f),
    TG_MX_TILE(MX_S256, MX_E2M1, 64, 64, 2, 2, 2, 128, 3.11f, 0.2209f, 1.69f, 0.2301f),
    TG_MX_TILE(MX_S256, MX_E2M1, 128, 128, 2, 4, 2, 128, 3.76f, 0.3195f, 2.5f, 0.3458f),
    TG_MX_TILE(MX_S256, MX_E2M1, 256, 128, 2, 2, 2, 128, 7.26f, 0.4521f, 4.43f, 0.5079f),
    TG_MX_TILE(MX_S128, MX_E2M1, 256, 256, 2, 4, 4, 128, 7.44f, 0.7601f, 5.0f, 0.9702f),
    TG_MX_TILE(MX_S256_1024, MX_E2M1, 256, 256, 2, 4, 2, 1024, 7.92f, 0.6661f, 4.35f, 0.7835f),
};

MxKernels mx_kernels_e2m1()
{
    return {kKernels, kKernels + sizeof(kKernels) / sizeof(kKernels[0])};
}

}  // namespace tg
