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
        batch > INT_MAX || q_tokens > INT_MAX || table_width > (1 << 30) / cache->page_size ||
        (batch > 0 && q_tokens > INT_MAX / q_heads / batch))
        return FP4_ERR_SHAPE;
    return FP4_OK;
}

// Row tiles of a call, and its workspace: two lines of outputs and statistics
// a CTA of the largest grid, then a counter for each unit.  The counters lie
// behind an area of one size for every call on a cache of this head_dim, so
// that no other call's outputs overwrite them.
struct Plan {
    int nt, rows, row_tiles;
    size_t stats, arrived, bytes; // offsets, and the whole
};

constexpr int kUnitsFill = 8;
constexpr int kMostSms = 160, kMostCtas = 5; // of any Blackwell data-centre GPU; per SM

fp4_status make_plan(const fp4_kv_cache &c, bool bf16, int64_t batch, int64_t q_tokens, int64_t q_heads, Plan &p)
{
    const int64_t rows = q_tokens * (q_heads / c.heads);
    p.rows = (int)rows;
    p.nt = rows > 8 && bf16 && c.head_dim < 256 ? 2 : 1;
    const int64_t r = 8 * p.nt, tiles = (rows + r - 1) / r;
    if (batch > 65535 || c.heads * tiles > 65535)
        return FP4_ERR_SHAPE; // the grid's y and z
    p.row_tiles = (int)tiles;
    const size_t lines = (size_t)2 * kMostSms * kMostCtas * (c.head_dim < 256 ? 16 : 8);
    p.stats = lines * (size_t)c.head_dim * sizeof(float);
    p.arrived = p.stats + lines * sizeof(float4);
    p.bytes = p.arrived + (size_t)(batch * c.heads * tiles) * sizeof(uint32_t);
    return FP4_OK;
}

template <typename TQ, bool kNv, int D, int NT>
fp4_status launch_attention_t(fp4::AttnArgs a, cudaStream_t stream)
{
    constexpr int smem = fp4::attn_smem<kNv, D, NT>(), ctas = fp4::kAttnCtas<TQ, D, NT>;
    static_assert(ctas <= kMostCtas, "workspace");
    auto kernel = fp4::kv_attention_kernel<TQ, kNv, D, NT>;
    int dev = 0;
    const int sms = sm_count(dev);
    if (sms <= 0 || !smem_attr(kernel, smem))
        return FP4_ERR_CUDA;
    // A CTA per unit where the table holds few tokens, or the units fill the GPU
    // several times over; otherwise the tokens are shared out.  Measured (8 heads x
    // 128, 4 query heads each, cold L2, one call between two events, us, of which these
    // take about 5, a CTA per unit | shared out): one sequence of 600 tokens 13.3 |
    // 18.4, 1024 16.4 | 18.4, 1280 18.4 | 18.4, 2048 22.5 | 18.5; 32 of 1024 20.4 |
    // 26.6, of 4096 47.1 | 47.1.  With many units a CTA each is faster while the
    // lengths are alike (256 sequences of 2000 tokens 123 | 133, of 0 to 2000 78 | 84),
    // but a single long sequence among short ones then takes as long as one CTA needs
    // for it (7 us a thousand tokens), so that the units have to be many before it is
    // chosen.
    const int64_t units = (int64_t)a.batch * a.c.heads * a.row_tiles, slots = (int64_t)(sms < kMostSms ? sms : kMostSms) * ctas;
    int64_t most = a.capacity;
    if (a.window > 0 && a.window < most - a.q_tokens - 15) // the window, the tile's new tokens, the rounding to 16
        most = a.window + a.q_tokens + 15;
    a.split = most > fp4::kAttnWhole * fp4::kAttnRound && units < kUnitsFill * slots &&
              units <= INT_MAX / (most / fp4::kAttnRound + 2 + fp4::kAttnStart); // all is numbered with 32 bits
    const dim3 grid = a.split ? dim3((unsigned)slots)
                              : dim3(1u, (unsigned)(a.c.heads * a.row_tiles), (unsigned)a.batch);
    return launch_cfg(kernel, grid, fp4::kAttnThreads, smem, stream, a);
}

template <typename TQ, bool kNv>
fp4_status launch_attention(const fp4::AttnArgs &a, int dim, int nt, cudaStream_t stream)
{
    if (dim == 256)
        return launch_attention_t<TQ, kNv, 256, 1>(a, stream);
    if constexpr (sizeof(TQ) == 2)
        if (nt == 2)
            return dim == 64 ? launch_attention_t<TQ, kNv, 64, 2>(a, stream)
                             : launch_attention_t<TQ, kNv, 128, 2>(a, stream);
    return dim == 64 ? launch_attention_t<TQ, kNv, 64, 1>(a, stream)
                     : launch_attention_t<TQ, kNv, 128, 1>(a, stream);
}

} // namespace

extern "C" {

size_t fp4_kv_attention_workspace_bytes(const fp4_kv_cache *cache, int64_t batch, int64_t q_tokens, int64_t q_heads,
                                        int64_t table_width)
{
    if (check_attention(cache, batch, q_tokens, q_heads, table_width) != FP4_OK)
        return 0;
    size_t most = 16;
    for (int bf = 0; bf < 2; ++bf) { // either type of q
        Plan p;
        if (make_plan(*cache, bf, batch, q_tokens, q_heads, p) != FP4_OK)
            return 0;
        most = p.bytes > most ? p.bytes : most;
    }
    return most;
}

fp4_status fp4_kv_attention(const fp4_kv_cache *cache, const void *q, fp4_dtype dtype, int64_t batch,
                            int64_t q_tokens, int64_t q_heads, int64_t q_stride, const int32_t *page_table,
                            int64_t table_width, const int32_t *seq_lens, float softmax_scale, int64_t window,
                            void *out, float *lse, void *workspace, size_t workspace_bytes, int32_t *status,
                            cudaStream_t stream)
{
    if (!valid_dtype(dtype) || !status || window < 0 || !std::isfinite(softmax_scale * 1.5f)) // log2(e) joins the scale
        return FP4_ERR_INVALID_ARG;
    fp4_status st = check_attention(cache, batch, q_tokens, q_heads, table_width);
    if (st != FP4_OK || batch == 0 || q_tokens == 0)
        return st;
    const int64_t size = dtype == FP4_BF16 ? 2 : 4;
    if (q_stride < q_heads * cache->head_dim || q_stride > INT64_MAX / 8 / (batch * q_tokens))
        return FP4_ERR_SHAPE;
    Plan p;
    if ((st = make_plan(*cache, dtype == FP4_BF16, batch, q_tokens, q_heads, p)) != FP4_OK)
        return st;
    if (!q || !out || !seq_lens || (table_width > 0 && !page_table))
        return FP4_ERR_INVALID_ARG;
    if (!aligned(q, 16) || q_stride * size % 16 || !aligned(out, 16) || !aligned(seq_lens, 4) ||
        !aligned(page_table, 4) || !aligned(lse, 4))
        return FP4_ERR_ALIGN;
    if (!workspace || workspace_bytes < fp4_kv_attention_workspace_bytes(cache, batch, q_tokens, q_heads, table_width))
        return FP4_ERR_WORKSPACE;
    if (!aligned(workspace, 16))
        return FP4_ERR_ALIGN;
    const bool bf = dtype == FP4_BF16, nv = cache->format == FP4_NVFP4;
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
    a.stats = reinterpret_cast<float4 *>(static_cast<char *>(workspace) + p.stats);
    a.status = status;
    a.group = (int)(q_heads / cache->heads);
    a.group_magic = ~(uint64_t)0 / (uint64_t)a.group + 1;
    a.rows = p.rows;
    a.row_tiles = p.row_tiles;
    a.arrived = reinterpret_cast<uint32_t *>(static_cast<char *>(workspace) + p.arrived);
    if (nv)
        return bf ? launch_attention<uint16_t, true>(a, cache->head_dim, p.nt, stream)
                  : launch_attention<float, true>(a, cache->head_dim, p.nt, stream);
    return bf ? launch_attention<uint16_t, false>(a, cache->head_dim, p.nt, stream)
              : launch_attention<float, false>(a, cache->head_dim, p.nt, stream);
}

} // extern "C"
