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

// How a call is split.  `capacity` bounds the tokens any row tile needs.
struct Plan {
    int nt, rows, row_tiles, splits, chunk;
    int64_t units;
    size_t partial, stats; // bytes
};

// The tokens are split so that the CTAs fill the GPU about twice over
// (kFill CTAs per SM), in whole rounds of the CTA's warps: a split below
// kMinChunk tokens has too few steps per warp to cover its start and end.
constexpr int kMostSms = 160; // of any Blackwell data-centre GPU
constexpr int kMinChunk = 256, kRound = fp4::kAttnWarps * fp4::kAttnStep, kFill = 8;

fp4_status make_plan(const fp4_kv_cache &c, bool bf16, int64_t batch, int64_t q_tokens, int64_t q_heads,
                     int64_t capacity, int64_t sms, Plan &p)
{
    const int64_t rows = q_tokens * (q_heads / c.heads);
    p.rows = (int)rows;
    p.nt = rows > 8 && bf16 && c.head_dim < 256 ? 2 : 1;
    const int64_t r = 8 * p.nt, tiles = (rows + r - 1) / r;
    p.row_tiles = (int)tiles;
    p.units = batch * c.heads * tiles;
    const int64_t want = sms * kFill / (p.units > 0 ? p.units : 1);
    int64_t chunk = want > 1 ? (capacity + want - 1) / want : capacity;
    chunk = (chunk + kRound - 1) / kRound * kRound;
    if (chunk < kMinChunk)
        chunk = kMinChunk;
    int64_t splits = (capacity + chunk - 1) / chunk;
    if (splits < 1)
        splits = 1;
    if (p.units > INT_MAX || p.units * splits > INT_MAX)
        return FP4_ERR_SHAPE;
    p.chunk = (int)chunk;
    p.splits = (int)splits;
    const size_t lines = splits > 1 ? (size_t)(p.units * splits * r) : 0;
    p.partial = lines * (size_t)c.head_dim * sizeof(float);
    p.stats = lines * sizeof(float4);
    return FP4_OK;
}

template <typename TQ, bool kNv, int D, int NT>
fp4_status launch_attention_t(const fp4::AttnArgs &a, int64_t blocks, cudaStream_t stream)
{
    constexpr int smem = fp4::attn_smem<kNv, D, NT>();
    auto kernel = fp4::kv_attention_kernel<TQ, kNv, D, NT>;
    if (!smem_attr(kernel, smem))
        return FP4_ERR_CUDA;
    fp4_status st = launch_cfg(kernel, dim3((unsigned)blocks), fp4::kAttnThreads, smem, stream, a);
    if (st != FP4_OK || a.splits == 1)
        return st;
    const int64_t lines = (int64_t)a.batch * a.c.heads * a.rows;
    return launch_cfg(fp4::kv_attention_merge_kernel<TQ, kNv, D, NT>,
                      dim3((unsigned)lines), fp4::kAttnThreads, 0, stream, a);
}

template <typename TQ, bool kNv>
fp4_status launch_attention(const fp4::AttnArgs &a, int dim, int nt, int64_t blocks, cudaStream_t stream)
{
    if (dim == 256)
        return launch_attention_t<TQ, kNv, 256, 1>(a, blocks, stream);
    if constexpr (sizeof(TQ) == 2)
        if (nt == 2)
            return dim == 64 ? launch_attention_t<TQ, kNv, 64, 2>(a, blocks, stream)
                             : launch_attention_t<TQ, kNv, 128, 2>(a, blocks, stream);
    return dim == 64 ? launch_attention_t<TQ, kNv, 64, 1>(a, blocks, stream)
                     : launch_attention_t<TQ, kNv, 128, 1>(a, blocks, stream);
}

} // namespace

extern "C" {

size_t fp4_kv_attention_workspace_bytes(const fp4_kv_cache *cache, int64_t batch, int64_t q_tokens, int64_t q_heads,
                                        int64_t table_width)
{
    if (check_attention(cache, batch, q_tokens, q_heads, table_width) != FP4_OK)
        return 0;
    // units * splits <= kMostSms * kFill wherever a call is split (make_plan),
    // in lines of at most 16 rows: one size for every call on the cache
    return (size_t)kMostSms * kFill * (cache->head_dim < 256 ? 16 : 8) * (cache->head_dim * sizeof(float) + sizeof(float4));
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
    int dev = 0;
    const int sms = sm_count(dev);
    if (sms <= 0)
        return FP4_ERR_CUDA;
    const bool bf = dtype == FP4_BF16, nv = cache->format == FP4_NVFP4;
    // a window bounds the tokens of a row tile: the window, the tile's new tokens, the rounding to 16
    int64_t capacity = table_width * cache->page_size;
    if (window > 0 && window < capacity - q_tokens - 15)
        capacity = window + q_tokens + 15;
    Plan p;
    if ((st = make_plan(*cache, bf, batch, q_tokens, q_heads, capacity, sms < kMostSms ? sms : kMostSms, p)) != FP4_OK)
        return st;
    fp4::AttnArgs a = {};
    a.c = fp4_kv::device_cache(*cache);
    a.q = q;
    a.batch = (int)batch;
    a.q_tokens = (int)q_tokens;
    a.q_heads = (int)q_heads;
    a.q_stride = q_stride;
    a.page_table = page_table;
    a.table_width = (int)table_width;
    a.capacity = table_width * cache->page_size;
    a.window = window;
    const uint64_t page16 = (uint64_t)cache->page_size / 16;
    a.page_magic = ~(uint64_t)0 / page16 + 1;
    a.seq_lens = seq_lens;
    a.scale = softmax_scale * 1.44269504088896341f; // scores in units of log2
    a.out = out;
    a.lse = lse;
    a.partial = static_cast<float *>(workspace);
    a.stats = reinterpret_cast<float4 *>(static_cast<char *>(workspace) + p.partial);
    a.status = status;
    a.group = (int)(q_heads / cache->heads);
    a.rows = p.rows;
    a.row_tiles = p.row_tiles;
    a.splits = p.splits;
    a.chunk = p.chunk;
    const int64_t blocks = p.units * p.splits;
    if (nv)
        return bf ? launch_attention<uint16_t, true>(a, cache->head_dim, p.nt, blocks, stream)
                  : launch_attention<float, true>(a, cache->head_dim, p.nt, blocks, stream);
    return bf ? launch_attention<uint16_t, false>(a, cache->head_dim, p.nt, blocks, stream)
              : launch_attention<float, false>(a, cache->head_dim, p.nt, blocks, stream);
}

} // extern "C"
