// fp4_linear.cu -- entry points of include/fp4.h for the product of a few
// rows of activations with an FP4 weight: argument checks and the launches.
#include <climits>
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "fp4.h"
#include "fp4_launch.cuh"
#include "fp4_linear.cuh"

namespace {

using namespace fp4_launch;
using fp4::kThreads;

} // namespace

extern "C" {

size_t fp4_linear_workspace_bytes(int64_t rows, int64_t K)
{
    if (rows < 0 || K < 0 || rows > INT_MAX || K > INT_MAX)
        return 0;
    return 16;
}

fp4_status fp4_linear(fp4_format fmt, const void *x, fp4_dtype dtype, int64_t rows, int64_t K, int64_t x_stride,
                      const uint8_t *packed, const uint8_t *scales_mma, const float *global_scale, int64_t N, void *y,
                      fp4_dtype out_dtype, void *workspace, size_t workspace_bytes, int32_t *status,
                      cudaStream_t stream)
{
    if ((fmt != FP4_NVFP4 && fmt != FP4_MXFP4) || !valid_dtype(dtype) || !valid_dtype(out_dtype) || rows < 0 ||
        K < 0 || N < 0 || !status)
        return FP4_ERR_INVALID_ARG;
    const int64_t group = fmt == FP4_NVFP4 ? 16 : 32;
    const int64_t in = dtype == FP4_BF16 ? 2 : 4, on = out_dtype == FP4_BF16 ? 2 : 4;
    if (rows > INT_MAX || K > INT_MAX - 1024 || N > INT_MAX - 1024)
        return FP4_ERR_SHAPE;
    const int64_t Kp = (K + group - 1) / group * group;
    if (Kp % 32)
        return FP4_ERR_SHAPE;
    if (rows == 0 || N == 0)
        return FP4_OK;
    if (x_stride < K || x_stride > INT64_MAX / 8 / rows)
        return FP4_ERR_SHAPE;
    if (!y)
        return FP4_ERR_INVALID_ARG;
    if (!aligned(y, on))
        return FP4_ERR_ALIGN;
    if (K == 0) { // an empty sum
        if (cudaMemsetAsync(y, 0, (size_t)(rows * N * on), stream) != cudaSuccess) {
            (void)cudaGetLastError();
            return FP4_ERR_CUDA;
        }
        return FP4_OK;
    }
    if (!x || !packed || !scales_mma || (fmt == FP4_NVFP4 && !global_scale))
        return FP4_ERR_INVALID_ARG;
    if (!aligned(x, in) || !aligned(packed, 16) || !aligned(scales_mma, 16) ||
        (fmt == FP4_NVFP4 && !aligned(global_scale, 4)))
        return FP4_ERR_ALIGN;
    if (!workspace || workspace_bytes < fp4_linear_workspace_bytes(rows, K))
        return FP4_ERR_WORKSPACE;
    if (!aligned(workspace, 16))
        return FP4_ERR_ALIGN;
    const dim3 grid((unsigned)((N + kThreads / 32 - 1) / (kThreads / 32)));
    auto run = [&](auto *xt, auto *yt, auto nv) {
        using T = std::remove_const_t<std::remove_pointer_t<decltype(xt)>>;
        using TOut = std::remove_pointer_t<decltype(yt)>;
        return launch_cfg(fp4::linear_kernel<T, TOut, decltype(nv)::value>, grid, kThreads, 0, stream, xt, (int)rows,
                          (int)K, x_stride, packed, scales_mma, global_scale, (int)N, (int)Kp, yt, status);
    };
    auto by_out = [&](auto *xt, auto nv) {
        return out_dtype == FP4_BF16 ? run(xt, static_cast<uint16_t *>(y), nv) : run(xt, static_cast<float *>(y), nv);
    };
    auto by_in = [&](auto nv) {
        return dtype == FP4_BF16 ? by_out(static_cast<const uint16_t *>(x), nv)
                                 : by_out(static_cast<const float *>(x), nv);
    };
    return fmt == FP4_NVFP4 ? by_in(std::true_type{}) : by_in(std::false_type{});
}

} // extern "C"
