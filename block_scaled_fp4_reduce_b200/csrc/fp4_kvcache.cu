// fp4_kvcache.cu -- entry points of include/fp4.h for the paged FP4 cache:
// argument checks and the launches.
#include <climits>
#include <cstdint>

#include <cuda_runtime.h>

#include "fp4.h"
#include "fp4_kv_args.cuh"
#include "fp4_kvcache.cuh"
#include "fp4_launch.cuh"

namespace {

using namespace fp4_launch;
using fp4::kThreads;

// What fp4_kv_write and fp4_kv_read check alike: k, v are the tokens' side.
fp4_status check_rows(const fp4_kv_cache &c, const void *k, const void *v, fp4_dtype dtype, int64_t tokens,
                      int64_t k_stride, int64_t v_stride, const int64_t *slots)
{
    const int64_t row = (int64_t)c.heads * c.head_dim, size = dtype == FP4_BF16 ? 2 : 4;
    if (k_stride < row || v_stride < row || k_stride > INT64_MAX / 8 / tokens || v_stride > INT64_MAX / 8 / tokens)
        return FP4_ERR_SHAPE;
    if (!k || !v || !slots)
        return FP4_ERR_INVALID_ARG;
    if (!aligned(k, 32) || !aligned(v, 32) || k_stride * size % 32 || v_stride * size % 32 || !aligned(slots, 8))
        return FP4_ERR_ALIGN;
    return FP4_OK;
}

// Units of a row side by side in a CTA, and the grid over them: x walks the
// tokens (at most most_per_sm CTAs an SM, each thread keeping its unit), y the
// units beyond one CTA's.
template <typename K>
fp4_status kv_grid(K kernel, int64_t units, int64_t tokens, int most_per_sm, int &per, dim3 &grid)
{
    per = (int)(units < kThreads ? units : kThreads);
    const int64_t tiles = (units + per - 1) / per, per_cta = kThreads / per;
    const int64_t steps = (tokens + per_cta - 1) / per_cta;
    const int most = grid_for(kernel, INT_MAX, 1, kThreads, 0, most_per_sm);
    if (most <= 0)
        return FP4_ERR_CUDA;
    int64_t x = most / tiles > 1 ? most / tiles : 1;
    if (x > steps)
        x = steps;
    grid = dim3((unsigned)x, (unsigned)tiles);
    return FP4_OK;
}

template <typename T, bool kNv, bool kCeil>
fp4_status launch_write(const fp4_kv_cache &c, const void *k, const void *v, int64_t tokens, int64_t k_stride,
                        int64_t v_stride, const int64_t *slots, int32_t *status, cudaStream_t stream)
{
    auto kernel = fp4::kv_write_kernel<T, kNv, kCeil>;
    const fp4::KvCache d = fp4_kv::device_cache(c);
    int per;
    dim3 grid;
    const fp4_status st = kv_grid(kernel, (int64_t)2 * d.heads * d.blocks, tokens, 0, per, grid);
    if (st != FP4_OK)
        return st;
    return launch_cfg(kernel, grid, kThreads, 0, stream, d, static_cast<const T *>(k), static_cast<const T *>(v),
                      k_stride, v_stride, slots, tokens, per, status);
}

template <typename T, bool kNv>
fp4_status launch_read(const fp4_kv_cache &c, void *k, void *v, int64_t tokens, int64_t k_stride, int64_t v_stride,
                       const int64_t *slots, int32_t *status, cudaStream_t stream)
{
    auto kernel = fp4::kv_read_kernel<T, kNv>;
    const fp4::KvCache d = fp4_kv::device_cache(c);
    int per;
    dim3 grid;
    const fp4_status st = kv_grid(kernel, (int64_t)2 * d.heads * (c.head_dim / 16), tokens, fp4::kKvReadCtas, per, grid);
    if (st != FP4_OK)
        return st;
    return launch_cfg(kernel, grid, kThreads, 0, stream, d, static_cast<T *>(k), static_cast<T *>(v), k_stride,
                      v_stride, slots, tokens, per, status);
}

} // namespace

extern "C" {

fp4_status fp4_kv_write(const fp4_kv_cache *cache, const void *k, const void *v, fp4_dtype dtype, int64_t tokens,
                        int64_t k_stride, int64_t v_stride, const int64_t *slots, fp4_mx_rule rule, int32_t *status,
                        cudaStream_t stream)
{
    if (!valid_dtype(dtype) || tokens < 0 || !status || (rule != FP4_MX_FLOOR && rule != FP4_MX_CEIL))
        return FP4_ERR_INVALID_ARG;
    fp4_status st = fp4_kv::check_cache(cache);
    if (st != FP4_OK || tokens == 0)
        return st;
    if ((st = check_rows(*cache, k, v, dtype, tokens, k_stride, v_stride, slots)) != FP4_OK)
        return st;
    const bool bf = dtype == FP4_BF16;
#define FP4_KV_WRITE(T, NV, CEIL) \
    launch_write<T, NV, CEIL>(*cache, k, v, tokens, k_stride, v_stride, slots, status, stream)
    if (cache->format == FP4_NVFP4)
        return bf ? FP4_KV_WRITE(uint16_t, true, false) : FP4_KV_WRITE(float, true, false);
    if (rule == FP4_MX_CEIL)
        return bf ? FP4_KV_WRITE(uint16_t, false, true) : FP4_KV_WRITE(float, false, true);
    return bf ? FP4_KV_WRITE(uint16_t, false, false) : FP4_KV_WRITE(float, false, false);
#undef FP4_KV_WRITE
}

fp4_status fp4_kv_read(const fp4_kv_cache *cache, const int64_t *slots, int64_t tokens, void *k, void *v,
                       fp4_dtype out_dtype, int64_t k_stride, int64_t v_stride, int32_t *status, cudaStream_t stream)
{
    if (!valid_dtype(out_dtype) || tokens < 0 || !status)
        return FP4_ERR_INVALID_ARG;
    fp4_status st = fp4_kv::check_cache(cache);
    if (st != FP4_OK || tokens == 0)
        return st;
    if ((st = check_rows(*cache, k, v, out_dtype, tokens, k_stride, v_stride, slots)) != FP4_OK)
        return st;
    const bool bf = out_dtype == FP4_BF16;
#define FP4_KV_READ(T, NV) launch_read<T, NV>(*cache, k, v, tokens, k_stride, v_stride, slots, status, stream)
    if (cache->format == FP4_NVFP4)
        return bf ? FP4_KV_READ(uint16_t, true) : FP4_KV_READ(float, true);
    return bf ? FP4_KV_READ(uint16_t, false) : FP4_KV_READ(float, false);
#undef FP4_KV_READ
}

} // extern "C"
