// fp4_attention.cuh -- attention of a few new tokens over the paged FP4 cache.
//
//   x_j = scale q . k^_j,  m = max_j x_j,  out = sum_j e^(x_j - m) v^_j / sum_j e^(x_j - m)
//
// One warp per query row (sequence, new token, query head): its lanes share
// the head's elements, the tokens run one after the other with the running
// maximum and sum of the softmax in registers, so the scores are never
// stored.
#pragma once

#include <cstdint>

#include "fp4_kvcache.cuh"

namespace fp4 {

struct AttnArgs {
    KvCache c;
    const void *q;
    int batch, q_tokens, q_heads, head_dim;
    int64_t q_stride;
    const int32_t *page_table;
    int64_t table_width, window;
    const int32_t *seq_lens;
    float scale;
    void *out;
    float *lse;
    int32_t *status;
};

template <typename T> __device__ __forceinline__ float to_f32(T v)
{
    if constexpr (sizeof(T) == 2)
        return __uint_as_float((uint32_t)v << 16);
    else
        return v;
}

// One element of a cached row: code, block scale, global scale.
template <bool kNv> __device__ __forceinline__ float kv_value(const KvCache &c, int sel, int64_t row, int d, float g)
{
    constexpr int G = kNv ? 16 : 32;
    const uint32_t byte = __ldcg(c.packed[sel] + row * (c.blocks * G / 2) + d / 2);
    float lo, hi;
    f16x2_to_f32(e2m1x2_to_f16x2(byte), lo, hi);
    const uint32_t s = __ldcg(c.scales[sel] + row * c.blocks + d / G);
    return __fmul_rn(__fmul_rn((d & 1) ? hi : lo, kNv ? e4m3_to_f32(s) : e8m0_to_f32(s)), g);
}

template <typename T, bool kNv> __global__ void __launch_bounds__(kThreads) kv_attention_kernel(const AttnArgs a)
{
    pdl_begin();
    constexpr int kMost = 256 / 32; // elements of a lane
    const int lane = (int)threadIdx.x & 31;
    const int64_t rows = (int64_t)a.batch * a.q_tokens * a.q_heads;
    const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (row >= rows)
        return;
    const int h = (int)(row % a.q_heads);
    const int64_t bi = row / a.q_heads;
    const int i = (int)(bi % a.q_tokens), b = (int)(bi / a.q_tokens);
    const int kvh = h / (a.q_heads / a.c.heads), per = a.head_dim / 32;
    const T *q = static_cast<const T *>(a.q) + bi * a.q_stride + (int64_t)h * a.head_dim;
    float qv[kMost], o[kMost];
    bool bad = false;
    for (int e = 0; e < kMost; ++e) {
        qv[e] = e < per ? to_f32(__ldcg(q + e * 32 + lane)) : 0.0f;
        bad |= (__float_as_uint(qv[e]) & 0x7FFFFFFFu) >= kNonFiniteBits;
        o[e] = 0.0f;
    }
    if (bad)
        raise_status(a.status, kStatusNonFinite);
    const float gk = kNv ? __ldcg(a.c.g[0] + kvh) : 1.0f, gv = kNv ? __ldcg(a.c.g[1] + kvh) : 1.0f;
    int64_t n = __ldcg(a.seq_lens + b);
    if (n < 0 || n > a.table_width * a.c.page) {
        raise_status(a.status, kStatusIndex);
        n = 0;
    }
    const int64_t p = n - a.q_tokens + i;
    int64_t first = a.window > 0 ? p - a.window + 1 : 0;
    first = first < 0 ? 0 : first;
    float m = -INFINITY, l = 0.0f;
    for (int64_t j = first; j <= p; ++j) {
        const int64_t page = __ldcg(a.page_table + b * a.table_width + j / a.c.page);
        if (page < 0 || page >= a.c.slots / a.c.page) {
            raise_status(a.status, kStatusIndex);
            continue;
        }
        const int64_t at = kv_row(a.c, page * a.c.page + j % a.c.page, kvh);
        float x = 0.0f;
        for (int e = 0; e < kMost; ++e)
            if (e < per)
                x = fmaf(qv[e], kv_value<kNv>(a.c, 0, at, e * 32 + lane, gk), x);
        for (int s = 16; s; s >>= 1)
            x += __shfl_xor_sync(0xFFFFFFFFu, x, s);
        x *= a.scale;
        const float mn = fmaxf(m, x), alpha = expf(m - mn), w = expf(x - mn);
        l = fmaf(l, alpha, w);
        for (int e = 0; e < kMost; ++e)
            if (e < per)
                o[e] = fmaf(o[e], alpha, w * kv_value<kNv>(a.c, 1, at, e * 32 + lane, gv));
        m = mn;
    }
    T *out = static_cast<T *>(a.out) + row * a.head_dim;
    for (int e = 0; e < kMost; ++e)
        if (e < per)
            out[e * 32 + lane] = to_out<T>(l > 0.0f ? o[e] / l : 0.0f);
    if (a.lse && lane == 0)
        a.lse[row] = l > 0.0f ? m + logf(l) : -INFINITY;
}

} // namespace fp4
