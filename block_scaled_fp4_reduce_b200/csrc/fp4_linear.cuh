// fp4_linear.cuh -- y = x W^^T for a few rows of unquantised activations and
// an FP4 weight.
//
// One warp per output column n: its lanes stride over K, decode the codes
// of row n of the weight once per row of x and sum in fp32.
#pragma once

#include <cstdint>

#include "fp4_kernels.cuh"

namespace fp4 {

template <typename T> __device__ __forceinline__ float to_f32(T v)
{
    if constexpr (sizeof(T) == 2)
        return __uint_as_float((uint32_t)v << 16);
    else
        return v;
}

// Byte of the MMA scale layout that holds the scale of (row, block).
__device__ __forceinline__ int64_t mma_scale_at(int64_t row, int64_t block, int64_t tiles_per_band)
{
    const int64_t band = row >> 7, r = row & 127;
    return (band * tiles_per_band + (block >> 2)) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (block & 3);
}

template <typename T, typename TOut, bool kNv>
__global__ void __launch_bounds__(kThreads)
    linear_kernel(const T *x, int rows, int K, int64_t x_stride, const uint8_t *packed, const uint8_t *scales_mma,
                  const float *global_scale, int N, int Kp, TOut *y, int32_t *status)
{
    pdl_begin();
    constexpr int G = kNv ? 16 : 32;
    const int lane = (int)threadIdx.x & 31;
    const int64_t n = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (n >= N)
        return;
    const float g = kNv ? __ldcg(global_scale) : 1.0f;
    const int64_t tiles = (Kp / G + 3) / 4;
    bool bad = false;
    for (int m = 0; m < rows; ++m) {
        float s = 0.0f;
        for (int k = lane; k < K; k += 32) {
            const float xv = to_f32(__ldcg(x + m * x_stride + k));
            bad |= (__float_as_uint(xv) & 0x7FFFFFFFu) >= kNonFiniteBits;
            float lo, hi;
            f16x2_to_f32(e2m1x2_to_f16x2(__ldcg(packed + n * (Kp / 2) + k / 2)), lo, hi);
            const uint32_t sb = __ldcg(scales_mma + mma_scale_at(n, k / G, tiles));
            const float w = __fmul_rn((k & 1) ? hi : lo, kNv ? e4m3_to_f32(sb) : e8m0_to_f32(sb));
            s = fmaf(xv, __fmul_rn(w, g), s); // g with the weight: x p s alone may overflow
        }
        for (int d = 16; d; d >>= 1)
            s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        if (lane == 0)
            y[(int64_t)m * N + n] = to_out<TOut>(s);
    }
    if (bad)
        raise_status(status, kStatusNonFinite);
}

} // namespace fp4
