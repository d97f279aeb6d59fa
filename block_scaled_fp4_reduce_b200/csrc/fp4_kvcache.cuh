// fp4_kvcache.cuh -- keys and values quantised as they are written into a
// paged FP4 cache, and read back.
//
// A cache page holds its tokens head by head: [heads, page_size, D/2] codes
// and [heads, page_size, D/G] scale bytes, so that the tokens of one head,
// which attention reads together, are contiguous.  Per block of G elements
// the codec is the quantisers' (fp4_kernels.cuh): NVFP4 under the head's
// global scale, MXFP4 by either scale rule; reading back is fp4_dequantize's
// arithmetic.  Both directions are one pass over the data.
//
// Measured, 65536 tokens x 8 heads x 128, bf16, keys and values (344 MB, 52.6 us
// at the copy rate), GPU time (calls back to back in a graph): reading back 58 us,
// writing MXFP4 58 us, HBM both; writing NVFP4 92 us, bound by its instructions
// (issue slots 68 % used; 260 warp instructions for 32 blocks, where the row
// quantiser takes 151 for the same arithmetic: what is round it, slots, places
// and a block chosen by the thread, is the difference).  64 tokens take 3.4 us to
// write and 2.1 to read.  One or three tokens in flight a thread, and three CTAs
// an SM in place of four, are within 5 %.
#pragma once

#include <cstdint>
#include <type_traits>

#include "fp4_kernels.cuh"

namespace fp4 {

// The cache as the kernels take it; `sel` 0 = keys, 1 = values.
struct KvCache {
    uint8_t *packed[2], *scales[2];
    const float *g[2];
    int64_t slots;       // num_pages * page_size
    uint64_t page_magic; // 2^64 / page, rounded up: slots lie below 2^40
    int heads, blocks, page; // blocks of a token's head: head_dim / G
    bool narrow;             // a slot's units of 16 elements can be numbered with 31 bits, and
    uint32_t magic32;        // slot / 16 divided by page / 16 (2^32 over it, rounded up; 0 for 1) in 32
};

// Where a head's block (or 16-code unit) of a slot lies, in units:
//   (page heads + head) page_size units + (slot - page page_size) units + block
//   = slot units + page skip + first.
struct KvPlace {
    int64_t first, skip;
};

__device__ __forceinline__ KvPlace kv_place(const KvCache &c, int units, int head, int block)
{
    return {(int64_t)head * c.page * units + block, (int64_t)(c.heads - 1) * c.page * units};
}

__device__ __forceinline__ int64_t kv_at(const KvCache &c, const KvPlace &p, int units, int64_t slot)
{
    if (c.narrow) {
        const uint32_t n = (uint32_t)slot, page = c.magic32 ? __umulhi(n >> 4, c.magic32) : n >> 4;
        return (int64_t)(n * (uint32_t)units + page * (uint32_t)p.skip + (uint32_t)p.first);
    }
    const int64_t page = (int64_t)__umul64hi((uint64_t)slot, c.page_magic);
    return slot * units + page * p.skip + p.first;
}

// The share of one thread: a unit is one block of one head of the keys or
// of the values, and a thread keeps one unit for all its tokens, so that
// what depends on the head (the double reciprocal of 6 g above all) is
// formed once.  `per` units side by side in a CTA, kThreads / per tokens;
// blockIdx.y walks units beyond kThreads.
struct KvUnit {
    int sel, head, block;
    int64_t first; // its first token
    int step;      // tokens between its tokens
    bool any;
};

__device__ __forceinline__ KvUnit kv_unit(const KvCache &c, int units_of_row, int per)
{
    KvUnit u;
    const int lane = (int)threadIdx.x % per, tok = (int)threadIdx.x / per;
    const int per_cta = kThreads / per;
    const int i = (int)blockIdx.y * per + lane; // keys' units, then the values'
    const int one = c.heads * units_of_row;
    u.any = tok < per_cta && i < 2 * one;
    u.sel = i >= one;
    const int j = i - (u.sel ? one : 0);
    u.head = j / units_of_row;
    u.block = j - u.head * units_of_row;
    u.first = (int64_t)blockIdx.x * per_cta + tok;
    u.step = (int)gridDim.x * per_cta;
    return u;
}

// ---------------------------------------------------------------------------
// Write.  One thread per block (32-byte loads, one packed store, one scale
// byte), kKvWriteTokens tokens in flight.  The loop is the CTA's, so that its
// warps stay whole for the NVFP4 bf16 path, whose half-blocks next to a
// rounding border are divided by the whole warp (nv_quantize_warp).
// ---------------------------------------------------------------------------
constexpr int kKvWriteTokens = 2;

template <typename T, bool kNv, bool kCeil>
__global__ void __launch_bounds__(kThreads, kNv && sizeof(T) == 2 ? 4 : 1)
    kv_write_kernel(const KvCache c, const T *__restrict__ k, const T *__restrict__ v, int64_t k_stride,
                    int64_t v_stride, const int64_t *__restrict__ slots, int64_t tokens, int per, int32_t *status)
{
    constexpr int G = kNv ? 16 : 32, U = kKvWriteTokens;
    constexpr bool kShared = kNv && sizeof(T) == 2;
    struct None {};
    using Queue = std::conditional_t<kShared, NvExactQueue<U>, None>;
    __shared__ Queue queue[kShared ? kThreads / 32 : 1];
    pdl_begin();
    KvUnit u = kv_unit(c, c.blocks, per);
    NvScaleConsts sc = {};
    if constexpr (kNv) {
        float g = u.any ? __ldcg((u.sel ? c.g[1] : c.g[0]) + u.head) : 1.0f;
        // 448 g has to be finite, and a subnormal g has no usable reciprocal
        if (!(g >= 0x1p-126f && g <= 3.4028234663852886e38f / 2688.0f)) {
            raise_status(status, kStatusRange);
            u.any = false;
            g = 1.0f;
        }
        sc = nv_scale_consts(g);
    }
    const T *x = (u.sel ? v : k) + (int64_t)(u.head * c.blocks + u.block) * G;
    const int64_t stride = u.sel ? v_stride : k_stride;
    const KvPlace place = kv_place(c, c.blocks, u.head, u.block);
    // (not indexed by u.sel: that would copy the arguments to local memory)
    uint8_t *const packed = u.sel ? c.packed[1] : c.packed[0], *const scales = u.sel ? c.scales[1] : c.scales[0];
    int32_t err = 0;
    const int64_t tok = u.first - (int64_t)blockIdx.x * (kThreads / per); // the thread's place among the CTA's tokens
    for (int64_t t = u.first; t - tok < tokens; t += (int64_t)U * u.step) {
        Blk<T, G> blk[U];
        int64_t at[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t ti = t + (int64_t)i * u.step;
            at[i] = u.any && ti < tokens ? __ldcg(slots + ti) : -1;
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (at[i] >= c.slots) {
                err = kStatusIndex;
                at[i] = -1;
            }
            if (at[i] >= 0) {
                load_blk(x + (t + (int64_t)i * u.step) * stride, 0, blk[i]);
            } else {
#pragma unroll
                for (int j = 0; j < Blk<T, G>::kWords; ++j)
                    blk[i].w[j] = 0u;
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (at[i] >= 0)
                at[i] = kv_at(c, place, c.blocks, at[i]);
        if constexpr (kShared) {
            uint2 pk[U];
            uint32_t code[U];
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (absmax_bits(blk[i]) >= kNonFiniteBits)
                    err = kStatusNonFinite;
            nv_quantize_warp<U>(blk, sc, queue[threadIdx.x >> 5], pk, code);
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (at[i] >= 0) {
                    reinterpret_cast<uint2 *>(packed)[at[i]] = pk[i];
                    scales[at[i]] = (uint8_t)code[i];
                }
        } else {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (at[i] < 0)
                    continue;
                if constexpr (kNv) {
                    if (absmax_bits(blk[i]) >= kNonFiniteBits)
                        err = kStatusNonFinite;
                    nv_quantize_block(blk[i], sc, reinterpret_cast<uint2 *>(packed) + at[i], scales + at[i]);
                } else {
                    bool bad = false;
                    mx_quantize_block<kCeil>(blk[i], reinterpret_cast<uint4 *>(packed) + at[i], scales + at[i], bad);
                    if (bad)
                        err = kStatusNonFinite;
                }
            }
        }
    }
    if (err)
        raise_status(status, err);
}

// ---------------------------------------------------------------------------
// Read back.  One thread per 16 codes (8 packed bytes, one scale byte, 16
// outputs), as the dequantiser; kKvTokens tokens in flight,
// kKvReadCtas CTAs per SM.
// ---------------------------------------------------------------------------
constexpr int kKvTokens = 2, kKvReadCtas = 8;

template <typename T, bool kNv>
__global__ void __launch_bounds__(kThreads)
    kv_read_kernel(const KvCache c, T *__restrict__ k, T *__restrict__ v, int64_t k_stride, int64_t v_stride,
                   const int64_t *__restrict__ slots, int64_t tokens, int per, int32_t *status)
{
    pdl_begin();
    const int units = kNv ? c.blocks : 2 * c.blocks; // 16-code units of a row
    const KvUnit u = kv_unit(c, units, per);
    if (!u.any)
        return;
    const float g = kNv ? __ldcg((u.sel ? c.g[1] : c.g[0]) + u.head) : 1.0f;
    const uint64_t g2 = pack2(g, g);
    const KvPlace place = kv_place(c, units, u.head, u.block);
    T *y = (u.sel ? v : k) + (int64_t)(u.head * units + u.block) * 16;
    const int64_t stride = u.sel ? v_stride : k_stride;
    const uint2 *const packed = reinterpret_cast<const uint2 *>(u.sel ? c.packed[1] : c.packed[0]);
    const uint8_t *const scales = u.sel ? c.scales[1] : c.scales[0];
    bool bad = false;
    auto slot_of = [&](int64_t ti) -> int64_t { return ti < tokens ? __ldcg(slots + ti) : -1; };
    int64_t next[kKvTokens]; // slots are read a round ahead
#pragma unroll
    for (int i = 0; i < kKvTokens; ++i)
        next[i] = slot_of(u.first + (int64_t)i * u.step);
    for (int64_t t = u.first; t < tokens; t += (int64_t)kKvTokens * u.step) {
        uint2 pk[kKvTokens];
        uint32_t sbyte[kKvTokens];
#pragma unroll
        for (int i = 0; i < kKvTokens; ++i) {
            pk[i] = make_uint2(0u, 0u); // zeros where there is nothing to read
            sbyte[i] = kNv ? 0u : 127u;
            if (next[i] >= c.slots) {
                bad = true;
            } else if (next[i] >= 0) {
                const int64_t at = kv_at(c, place, units, next[i]);
                pk[i] = __ldcg(packed + at);
                sbyte[i] = __ldcg(scales + (kNv ? at : at >> 1));
            }
        }
#pragma unroll
        for (int i = 0; i < kKvTokens; ++i)
            next[i] = slot_of(t + (int64_t)(kKvTokens + i) * u.step);
#pragma unroll
        for (int i = 0; i < kKvTokens; ++i) {
            const int64_t ti = t + (int64_t)i * u.step;
            if (ti < tokens)
                dequant_unit<kNv>(pk[i], sbyte[i], g2, y + ti * stride);
        }
    }
    if (bad)
        raise_status(status, kStatusIndex);
}

} // namespace fp4
