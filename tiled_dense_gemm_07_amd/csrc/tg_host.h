// Host-side pieces shared by the translation units that hold entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/tilegemm.h"

namespace tg {

constexpr int64_t kMaxDim = 0x7FFFFFFF;
constexpr int64_t kMaxI8K = 131071;  // 128 * 128 * K stays below 2^31

// Settings of tg_set_clock_stamps and tg_set_swizzle_override.
unsigned long long* clock_stamps();
int swizzle_override();

// Launches `kernel` with the parameter struct `params`; a forced failure
// (environment TG_FAULT=launch, for testing error reporting) and the
// runtime's own launch errors give TG_ERR_HIP.  `what` names the launch in
// the log (environment TG_LOG).
tg_status launch_kernel(const void* kernel, int64_t grid_x, int64_t grid_y, int threads,
                        void* params, hipStream_t stream, const char* what, unsigned lds = 0);

// Name and grid of the kernel a tg_gemm_i8 call with 16-byte aligned rows
// would launch (for tg_query_config).
void describe_i8(int64_t M, int64_t N, int64_t K, char* buf, size_t len);

// A strided matrix of `rows` rows of `cols` elements: its byte range, row
// length and row stride.  Two matrices of one stride may interleave (column
// slices of one buffer): they overlap only if their columns do.
struct Span {
    uintptr_t lo, hi;
    uintptr_t width, stride;
};
inline Span span(const void* p, int64_t rows, int64_t cols, int64_t ld, int esize)
{
    if (!p || rows <= 0 || cols <= 0)
        return {0, 0, 0, 0};
    const uintptr_t lo = (uintptr_t)p;
    return {lo, lo + (uintptr_t)(((rows - 1) * ld + cols) * esize), (uintptr_t)(cols * esize),
            (uintptr_t)(ld * esize)};
}
inline Span span1(const void* p, int64_t n, int esize) { return span(p, 1, n, n, esize); }
inline bool overlap(const Span& a, const Span& b)
{
    if (!(a.lo < b.hi && b.lo < a.hi))
        return false;
    if (a.stride == b.stride && a.stride > 0) {
        const Span &f = a.lo <= b.lo ? a : b, &s = a.lo <= b.lo ? b : a;
        const uintptr_t d = (s.lo - f.lo) % a.stride;  // s's columns start d bytes into f's rows
        return !(d >= f.width && d + s.width <= a.stride);
    }
    return true;
}

inline int dtype_size(int dt) { return dt == TG_F32 ? 4 : 2; }
inline bool dtype_ok(int dt) { return dt == TG_F32 || dt == TG_F16 || dt == TG_BF16; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace tg
