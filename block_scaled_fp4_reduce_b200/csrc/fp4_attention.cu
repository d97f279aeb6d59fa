// fp4_attention.cu -- entry points of include/fp4.h for attention over the
// paged FP4 cache: argument checks and the launch.
#include <climits>
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "fp4.h"
#include "fp4_attention.cuh"
#include "fp4_kv_args.cuh"
#include "fp4_launch.cuh"

namespace {

using namespace fp4_launch;
using fp4::kThreads;

fp4_status check_attention(const fp4_kv_cache *cache, int64_t batch, int64_t q_tokens, int64_t q_heads,
                           int64_t table_width)
{
    const fp4_status st = fp4_kv::check_cache(cache);
    if (st != FP4_OK)
        return st;
    if (batch < 0 || q_tokens < 0 || q_heads < 1 || table_width < 0)
        return FP4_ERR_INVALID_ARG;
    const int64_t d = cache->head_dim;
    if ((d != 64 && d != 128 && d != 256) || q_heads % cache->heads || q_heads > (1 << 20) / d ||
        batch > INT_MAX || q_tokens > INT_MAX || table_width > (INT_MAX - 255) / cache->page_size ||
        (batch > 0 && q_tokens > INT_MAX / q_heads / batch))
        return FP4_ERR_SHAPE;
    return FP4_OK;
}

} // namespace

extern "C" {

size_t fp4_kv_attention_workspace_bytes(const fp4_kv_cache *cache, int64_t batch, int64_t q_tokens, int64_t q_heads,
                                        int64_t table_width)
{
    if (check_attention(cache, batch, q_tokens, q_heads, table_width) != FP4_OK)
        return 0;
    return 16;
}

fp4_status fp4_kv_attention(const fp4_kv_cache *cache, const void *q, fp4_dtype dtype, int64_t batch,
                            int64_t q_tokens, int64_t q_heads, int64_t q_stride, const int32_t *page_table,
                            int64_t table_width, const int32_t *seq_lens, float softmax_scale, int64_t window,
                            void *out, float *lse, void *workspace, size_t workspace_bytes, int32_t *status,
                            cudaStream_t stream)
{
    if (!valid_dtype(dtype) || !status || window < 0 || !std::isfinite(softmax_scale))
        return FP4_ERR_INVALID_ARG;
    fp4_status st = check_attention(cache, batch, q_tokens, q_heads, table_width);
    if (st != FP4_OK || batch == 0 || q_tokens == 0)
        return st;
    const int64_t size = dtype == FP4_BF16 ? 2 : 4;
    if (q_stride < q_heads * cache->head_dim || q_stride > INT64_MAX / 8 / (batch * q_tokens))
        return FP4_ERR_SHAPE;
    if (!q || !out || !seq_lens || (table_width > 0 && !page_table))
        return FP4_ERR_INVALID_ARG;
    if (!aligned(q, 16) || q_stride * size % 16 || !aligned(out, 16) || !aligned(seq_lens, 4) ||
        !aligned(page_table, 4) || !aligned(lse, 4))
        return FP4_ERR_ALIGN;
    if (!workspace || workspace_bytes < fp4_kv_attention_workspace_bytes(cache, batch, q_tokens, q_heads, table_width))
        return FP4_ERR_WORKSPACE;
    if (!aligned(workspace, 16))
        return FP4_ERR_ALIGN;
    fp4::AttnArgs a = {};
    a.c = fp4_kv::device_cache(*cache);
    a.q = q;
    a.batch = (int)batch;
    a.q_tokens = (int)q_tokens;
    a.q_heads = (int)q_heads;
    a.head_dim = cache->head_dim;
    a.q_stride = q_stride;
    a.page_table = page_table;
    a.table_width = table_width;
    a.window = window;
    a.seq_lens = seq_lens;
    a.scale = softmax_scale;
    a.out = out;
    a.lse = lse;
    a.status = status;
    const dim3 grid((unsigned)((batch * q_tokens * q_heads + kThreads / 32 - 1) / (kThreads / 32)));
    const bool bf = dtype == FP4_BF16, nv = cache->format == FP4_NVFP4;
    auto kernel = nv ? (bf ? fp4::kv_attention_kernel<uint16_t, true> : fp4::kv_attention_kernel<float, true>)
                     : (bf ? fp4::kv_attention_kernel<uint16_t, false> : fp4::kv_attention_kernel<float, false>);
    return launch_cfg(kernel, grid, kThreads, 0, stream, a);
}

} // extern "C"
