// fp4_attention.cuh -- attention of a few new tokens over the paged FP4 cache.
//
//   x_j = scale q . k^_j,  m = max_j x_j,  out = sum_j e^(x_j - m) v^_j / sum_j e^(x_j - m)
//
// The query rows that read one KV head (new tokens x query heads of the
// group) form a tile of 8 NT rows.  A CTA takes one (sequence, KV head, row
// tile), or an even share of the tokens of all of them (attn_share); its
// kAttnWarps warps take steps of 32 tokens in turn, each warp on its own -- own
// ring of staged steps (cp.async, kStages deep), own running maximum, sum and
// output -- and meet once, at the end.
// One pass over the cache; scores live in registers.
//
// Tensor cores (mma.sync m16n8k16, fp16 in, fp32 out): the cached side is the
// M operand, so 16 tokens (or 16 elements of the head) meet 8 query rows per
// instruction and a group of 1 to 8 query heads wastes no rows.
//   scores   S^T [token, row] = K^ Q^T.  Lane (g, t) = (lane / 4, lane % 4)
//            reads tokens g and g + 8 of a 16-token tile, elements t D/4 ..
//            (t + 1) D/4 of each: contiguous codes, decoded to fp16 pairs and
//            scaled by the block's scale (code x E4M3 scale is exact in fp16).
//            Which element is which k index is free as long as Q's operand
//            agrees, so nothing is shuffled.
//   output   O^T [element, row] += V^T P^T.  Lane (g, t) reads elements g D/8
//            .. (g + 1) D/8 of tokens 2t, 2t + 1, 2t + 8, 2t + 9; the codes of
//            two tokens are interleaved nibble by nibble before they are
//            decoded, which gives the (token, token + 1) pairs of the operand
//            directly.  P comes out of the score tiles transposed by
//            movmatrix.
// Query rows enter as fp16 after a power of two that brings the row's maximum
// to 2^14 (exact for bf16 but for elements 2^-38 below the maximum); fp32
// rows as two fp16 terms.  Softmax weights enter as fp16 scaled by 2^11 over
// a reference that the running maximum passes by at most 2^4, so that weights
// down to 2^-25 of the largest keep all their bits and the rest down to 2^-36
// some; fp32 calls add a second term.  For bf16 one is enough: a weight is off by
// 2^-11 at most, an eighth of the result's own rounding, and the error against
// 64-bit arithmetic stays the rounding's (0.0016 of the result with one term or
// fp32 weights); a second term costs 2 x 131071 tokens 71.8 -> 81.5 us, 32 ragged
// sequences to 8192 43.9 -> 49.9.
//
// MXFP4: a block scale 2^e does not fit fp16.  Inside a token the scales are
// taken relative to the token's largest, 2^(e - E) (0 below 2^-24); 2^E of a
// key multiplies the finished score in fp32 (attn_factor), 2^E of a value joins
// the softmax weight: the weights' own reference is m' = max_j (x_j + E_j),
// beside the softmax's m, so that no value, however large or small, pushes
// another's weight out of fp16's range.
//
// What bounds it: instructions, and the waits between them.  A step of 32 tokens
// (D = 128, 8 rows) takes 588 warp instructions, 2.3 per element and lane: 256
// E2M1 conversions and products with the block scale, 64 to interleave nibbles,
// 32 MMAs, the loads, the softmax, one dependent chain in each warp; the SMs
// issue on 60 % of their cycles, with four CTAs of 128 registers a thread each.
// Measured, GPU time (calls back to back in a graph, three sets of inputs in
// turn, larger than L2): 2 sequences of 131071 tokens, 8 heads x 128, 8 query
// heads each, 71 us, 302 MB at 4.2 TB/s (0.65 of the copy rate); 32 of 4096
// tokens, 4 query heads each, 40 us, 151 MB at 3.8 TB/s.  Short calls are latency:
// the lengths, the page table and the first codes depend on one another (4 us),
// and joining pieces takes another 3.
// Not faster: CTAs of eight warps (2 x 131071 5 % less time, ragged batches 12 %
// more), and warps of an SM kept in step by barriers.
#pragma once

#include <cstdint>

#include "fp4_async.cuh"
#include "fp4_kvcache.cuh"
#include "fp4_mma.cuh"

namespace fp4 {

struct AttnArgs {
    KvCache c;
    const void *q;
    int batch, q_tokens, q_heads;
    int group, rows, row_tiles; // rows = q_tokens * group
    int split;                  // 0: a CTA per unit; 1: the tokens are shared out evenly (attn_share)
    uint64_t group_magic;       // 2^64 / group, rounded up
    int64_t q_stride;
    const int32_t *page_table;
    int table_width;
    int64_t capacity, window; // table_width * page
    uint64_t page_magic;      // 2^64 / (page / 16), rounded up
    const int32_t *seq_lens;
    float scale; // softmax scale * log2(e)
    void *out;
    float *lse;
    float *partial;  // [2 CTAs][8 NT][D] outputs of a piece of a unit, unnormalised
    float4 *stats;   // [2 CTAs][8 NT] m, l, m'
    uint32_t *arrived; // [unit] pieces of it that are done; zero between calls
    int32_t *status;
};

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kAttnStep = 32;       // tokens of a warp's step
constexpr int kAttnRound = kAttnWarps * kAttnStep; // of a step of all warps
constexpr int kAttnMinShare = 2;    // rounds of a CTA's share, at least
constexpr int kAttnStart = 2;       // what a unit's start and end count as, in rounds
constexpr int kAttnWhole = 8;       // rounds up to which a unit is left to one CTA
// Weights enter the tensor cores times 2^kAttnBias, and pass the reference
// by at most 2^kAttnSlack: 2^15 is the largest power of two in fp16.
constexpr float kAttnBias = 11.0f, kAttnSlack = 4.0f;
constexpr float kAttnNone = 1e30f;  // minus this: the reference before the first score
constexpr float kLn2 = 0.693147180559945309f;

// CTAs that share an SM.
template <typename TQ, int D, int NT>
constexpr int kAttnCtas = sizeof(TQ) == 4 ? (D == 256 ? 2 : D == 128 ? 3 : 4) : D == 256 ? 3 : D == 64 ? (NT == 2 ? 4 : 5) : (NT == 2 ? 3 : 4);

template <int D> constexpr int kAttnStages = D == 64 ? 4 : D == 128 ? 3 : 2;

// Bytes of one staged step: codes and scale bytes of 32 tokens' keys and values.
template <bool kNv, int D> constexpr int kAttnStageBytes = 2 * kAttnStep * (D / 2 + D / (kNv ? 16 : 32));

template <bool kNv, int D, int NT> constexpr int attn_smem()
{
    const int ring = kAttnWarps * kAttnStages<D> * kAttnStageBytes<kNv, D>;
    const int merge = kAttnWarps * 8 * NT * (D + 4) * 4;
    return ring > merge ? ring : merge;
}

// N 32-bit words, whole vectors (the address aligned to them).
template <typename T, int N> __device__ __forceinline__ void load_words(const T *p, uint32_t (&w)[N])
{
    if constexpr (N == 1) {
        w[0] = __ldcg(reinterpret_cast<const uint32_t *>(p));
    } else if constexpr (N == 2) {
        const uint2 v = __ldcg(reinterpret_cast<const uint2 *>(p));
        w[0] = v.x;
        w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 v = __ldcg(reinterpret_cast<const uint4 *>(p) + i / 4);
            w[i] = v.x;
            w[i + 1] = v.y;
            w[i + 2] = v.z;
            w[i + 3] = v.w;
        }
    }
}

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Largest of the four bytes of v.
__device__ __forceinline__ uint32_t max_byte(uint32_t v)
{
    const uint32_t a = max(v & 0xFFu, (v >> 8) & 0xFFu), b = max((v >> 16) & 0xFFu, v >> 24);
    return max(a, b);
}

// Positions that a row tile needs: tokens [lo, hi] (none where hi < lo), staged
// from `base` (lo rounded down to 16) in rounds of kAttnRound tokens.
struct AttnSpan {
    int n, lo, hi, base;
};

__device__ __forceinline__ AttnSpan attn_span(const AttnArgs &a, int n, int first_token, int last_token)
{
    AttnSpan s;
    s.n = n < 0 || n > a.capacity ? 0 : n; // (reported by the caller)
    s.hi = s.n - a.q_tokens + last_token;  // may be negative: nothing to see
    const int p = s.n - a.q_tokens + first_token;
    s.lo = a.window > 0 && p >= a.window ? p - (int)a.window + 1 : 0;
    s.base = s.lo & ~15;
    return s;
}

// Rounds of a unit, one at least (a unit that sees nothing is written too).
__device__ __forceinline__ int attn_rounds(const AttnSpan &s)
{
    return s.hi < s.lo ? 1 : (s.hi - s.base) / kAttnRound + 1;
}

// New token of row r of a KV head's rows.
__device__ __forceinline__ int attn_token(const AttnArgs &a, int r)
{
    return a.q_tokens == 1 ? 0 : a.group == 1 ? r : (int)__umul64hi((uint64_t)(uint32_t)r, a.group_magic);
}

// What turns a row's summed output into its result: g / l, or for MXFP4
// 2^(m' - m) / l.  In two factors: the power alone may leave fp32's range, and
// g / l its normal numbers where g itself does not.
// (Sums and weights both carry 2^kAttnBias.)
struct AttnScale {
    float f, f2;
};

template <bool kNv> __device__ __forceinline__ AttnScale attn_scale(float gv, float m, float mw, float l)
{
    AttnScale s = {0.0f, 1.0f};
    if (l > 0.0f) {
        if constexpr (kNv) {
            s.f = 1.0f / l;
            s.f2 = gv;
        } else {
            const float half = rintf(0.5f * (mw - m));
            s.f = ex2(half) / l;
            s.f2 = ex2((mw - m) - half);
        }
    }
    return s;
}

// The factor of a row's scores, scale g 2^e (g 1 for MXFP4).  In 64 bits: scale g
// alone may leave fp32's normal numbers.  MXFP4 multiplies the token's 2^E as well,
// and with halves of the factor on both sides of it no product leaves fp32's range
// that the score itself does not (a sum of 2^24 times E = 118 would, whatever the
// factor behind it).
struct AttnFactor {
    float f, f2;
};

template <bool kNv> __device__ __forceinline__ AttnFactor attn_factor(float scale, float g, int e)
{
    const double f = (double)scale * g * __hiloint2double((1023 + e) << 20, 0); // exact
    if constexpr (kNv)
        return {(float)f, 1.0f};
    const int half = (((__double2hiint(f) >> 20) & 0x7FF) - 1023) >> 1;     // (of zero: 2^-512 below, zero as well)
    return {(float)(f * __hiloint2double((1023 - half) << 20, 0)), (float)__hiloint2double((1023 + half) << 20, 0)};
}

__device__ __forceinline__ float attn_lse(float m, float l)
{
    return l == 0.0f ? -INFINITY : (m + (log2f(l) - kAttnBias)) * kLn2; // (NaN of a NaN)
}

// Place of a row's result among the rows of out and lse.
__device__ __forceinline__ int64_t attn_place(const AttnArgs &a, int b, int kvh, int row)
{
    const int i = attn_token(a, row);
    return ((int64_t)b * a.q_tokens + i) * a.q_heads + kvh * a.group + row - i * a.group;
}

// Four elements of a row's result.
template <typename TQ> __device__ __forceinline__ void attn_write(TQ *dst, float4 v, AttnScale f)
{
    const float y[4] = {v.x * f.f * f.f2, v.y * f.f * f.f2, v.z * f.f * f.f2, v.w * f.f * f.f2};
    if constexpr (sizeof(TQ) == 2) {
        uint2 w;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(y[1]), "f"(y[0]));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(y[3]), "f"(y[2]));
        *reinterpret_cast<uint2 *>(dst) = w;
    } else {
        *reinterpret_cast<float4 *>(dst) = make_float4(y[0], y[1], y[2], y[3]);
    }
}

// ---------------------------------------------------------------------------
// How the tokens are shared out.  A unit is one sequence, row tile and KV head;
// its work is its rounds, and kAttnStart more for its start and end.  With the
// units in that order (heads innermost) and all of this numbered through, CTA i
// takes the numbers [i s, (i + 1) s), s = the total over the CTAs that fit on
// the GPU: every CTA has the same work whatever the lengths are, in one wave
// (short sequences beside long ones: 256 sequences of 0 to 2000 tokens, 8 heads
// x 128, 4 query heads each, one call between two events: 131 us where starts
// count for nothing, 84 so; 3 and 4 rounds for a start are no better than 2).
// The lengths are on the device, so every CTA forms the numbering for itself, a
// scan over the sequences.  A CTA whose numbers cross units takes them one
// after the other; a unit that crosses CTAs leaves pieces, which the CTA that
// finishes the last of them joins.
// ---------------------------------------------------------------------------
template <int R> __device__ __forceinline__ uint32_t attn_sequence_rounds(const AttnArgs &a, int len)
{
    uint32_t sum = 0;
    for (int rt = 0; rt < a.row_tiles; ++rt) {
        const int row0 = rt * R, rows = min(R, a.rows - row0);
        sum += (uint32_t)attn_rounds(attn_span(a, len, attn_token(a, row0), attn_token(a, row0 + rows - 1))) + kAttnStart;
    }
    return sum * (uint32_t)a.c.heads;
}

// Inclusive scan of one value a thread over the CTA's kAttnThreads threads;
// `total` receives the sum.
__device__ __forceinline__ uint32_t attn_scan(uint32_t v, uint32_t *s_warp, uint32_t &total)
{
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (lane >= d)
            v += o;
    }
    __syncthreads();
    if (lane == 31)
        s_warp[warp] = v;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
        if (w < warp)
            v += s_warp[w];
        total += s_warp[w];
    }
    return v;
}

// This CTA's share: the sequence its first number lies in, that number within
// the sequence, how many there are from there on, and the CTAs' common share;
// false if there are none.  (The host sees to it that the numbers stay below
// 2^31.)
struct AttnShare {
    int b, len; // len: of sequence b
    uint32_t at, left, each, done; // done: numbers this CTA has behind it
};

template <int R> __device__ __forceinline__ bool attn_share(const AttnArgs &a, AttnShare &out)
{
    __shared__ uint32_t s_warp[kAttnWarps], s_at;
    __shared__ int s_b;
    const int tid = (int)threadIdx.x;
    uint32_t all = 0, mine = 0, upto = 0, total;
    if (a.batch <= 32) { // every warp finds it for itself
        const int lane = tid & 31;
        int len = 0;
        if (lane < a.batch) {
            len = __ldcg(a.seq_lens + lane);
            if ((len < 0 || len > a.capacity) && blockIdx.x == 0)
                raise_status(a.status, kStatusIndex);
            mine = attn_sequence_rounds<R>(a, len);
        }
        upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
            if (lane >= d)
                upto += o;
        }
        all = __shfl_sync(0xFFFFFFFFu, upto, 31);
        const uint32_t each = max((all + gridDim.x - 1) / gridDim.x, (uint32_t)kAttnMinShare);
        const uint32_t first = each * blockIdx.x;
        if (first >= all)
            return false;
        out.b = __ffs(__ballot_sync(0xFFFFFFFFu, first < upto)) - 1;
        out.at = first - __shfl_sync(0xFFFFFFFFu, upto - mine, out.b);
        out.len = __shfl_sync(0xFFFFFFFFu, len, out.b);
        out.left = min(each, all - first);
        out.each = each;
        out.done = 0;
        return true;
    }
    for (int b0 = 0; b0 < a.batch; b0 += kAttnThreads) {
        mine = 0;
        if (b0 + tid < a.batch) {
            const int len = __ldcg(a.seq_lens + b0 + tid);
            if ((len < 0 || len > a.capacity) && blockIdx.x == 0)
                raise_status(a.status, kStatusIndex);
            mine = attn_sequence_rounds<R>(a, len);
        }
        upto = attn_scan(mine, s_warp, total);
        all += total;
    }
    const uint32_t each = max((all + gridDim.x - 1) / gridDim.x, (uint32_t)kAttnMinShare);
    const uint32_t first = each * blockIdx.x; // below 2^32: each <= all / grid + kAttnMinShare
    if (first >= all)
        return false;
    uint32_t before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kAttnThreads) {
        if (a.batch > kAttnThreads) { // otherwise the one scan above holds
            mine = b0 + tid < a.batch ? attn_sequence_rounds<R>(a, __ldcg(a.seq_lens + b0 + tid)) : 0;
            upto = attn_scan(mine, s_warp, total);
        }
        if (first >= before + upto - mine && first < before + upto) {
            s_b = b0 + tid;
            s_at = first - (before + upto - mine);
        }
        before += total;
        if (first < before)
            break;
    }
    __syncthreads();
    out.b = s_b;
    out.len = __ldcg(a.seq_lens + s_b);
    out.at = s_at;
    out.left = min(each, all - first);
    out.each = each;
    out.done = 0;
    return true;
}

// ---------------------------------------------------------------------------
// The pieces of a unit, merged by the CTA that finishes the last of them:
// pieces first .. first + count - 1 are CTAs, the second of whose two lines is
// the first CTA's (its rounds end with the unit's beginning).  The sum runs in
// the order of the pieces, whoever forms it.
// ---------------------------------------------------------------------------
constexpr int kAttnMerge = 128; // pieces whose factors are held at a time

// What a row's elements are multiplied by, and where they go.
struct AttnRow {
    float w[kAttnWarps]; // the warps' results
    AttnScale f;
    int64_t at;
};

template <typename TQ, bool kNv, int D, int R>
__device__ __noinline__ void attn_merge(const float *partial, const float4 *stats, TQ *out, float *lse, uint8_t *smem,
                                        AttnRow *s_row, float gv, int rows, int first, int count)
{ // (a call of its own: inlined, its registers spill in the main loop)
    float(*const factor)[kAttnMerge] = reinterpret_cast<float(*)[kAttnMerge]>(smem); // [row][piece]
    float *const top = reinterpret_cast<float *>(smem + R * kAttnMerge * 4);         // [row] m'
    const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
    auto line = [&](int s, int r) -> int64_t { return (int64_t)(2 * (first + s) + (s == 0)) * R + r; };
    // A thread's share: kItems times four elements.  The outputs of kAhead
    // pieces are asked for at a time, the first of them together with the
    // statistics; rows past the tile's are read and dropped.
    constexpr int kItems = R * D / 4 / kAttnThreads, kAhead = kItems <= 2 ? 8 : 4;
    float4 p[kAhead][kItems], v[kItems];
    auto ask = [&](int s) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                const int idx = (int)threadIdx.x + i * kAttnThreads, r = idx / (D / 4), d = idx % (D / 4) * 4;
                p[k][i] = __ldcg(reinterpret_cast<const float4 *>(partial + line(min(s + k, count - 1), r) * D + d));
            }
    };
    // A warp takes rows warp, warp + 4, ...; a lane holds one piece's statistics
    // of each (pieces beyond 32 are read again where they are needed).
    constexpr int kMine = R / kAttnWarps;
    float4 own[kMine];
    float mm[kMine], mx[kMine], ll[kMine];
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        own[j] = make_float4(-kAttnNone, 0.0f, -kAttnNone, 0.0f);
        if (warp + j * kAttnWarps < rows && lane < count)
            own[j] = __ldcg(stats + line(lane, warp + j * kAttnWarps));
    }
    ask(0);
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        mm[j] = own[j].x;
        mx[j] = own[j].z;
        if (warp + j * kAttnWarps < rows)
            for (int s = lane + 32; s < count; s += 32) {
                const float4 st = __ldcg(stats + line(s, warp + j * kAttnWarps));
                mm[j] = fmaxf(mm[j], st.x);
                mx[j] = fmaxf(mx[j], st.z);
            }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1)
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            mm[j] = fmaxf(mm[j], __shfl_xor_sync(0xFFFFFFFFu, mm[j], d));
            mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xFFFFFFFFu, mx[j], d));
        }
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        ll[j] = own[j].y * ex2(own[j].x - mm[j]);
        if (warp + j * kAttnWarps < rows)
            for (int s = lane + 32; s < count; s += 32) {
                const float4 st = __ldcg(stats + line(s, warp + j * kAttnWarps));
                ll[j] = fmaf(st.y, ex2(st.x - mm[j]), ll[j]);
            }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1)
#pragma unroll
        for (int j = 0; j < kMine; ++j)
            ll[j] += __shfl_xor_sync(0xFFFFFFFFu, ll[j], d);
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        const int r = warp + j * kAttnWarps;
        factor[r][lane] = ex2(own[j].z - mx[j]);
        if (r < rows) {
            for (int s = lane + 32; s < min(count, kAttnMerge); s += 32)
                factor[r][s] = ex2(__ldcg(stats + line(s, r)).z - mx[j]);
            if (lane == 0) {
                top[r] = mx[j];
                s_row[r].f = attn_scale<kNv>(gv, mm[j], mx[j], ll[j]);
                if (lse)
                    lse[s_row[r].at] = attn_lse(mm[j], ll[j]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i)
        v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s0 = 0; s0 < count; s0 += kAttnMerge) {
        const int n = min(kAttnMerge, count - s0);
        __syncthreads();
        if (s0 > 0) {
            for (int r = warp; r < rows; r += kAttnWarps)
                for (int s = lane; s < n; s += 32)
                    factor[r][s] = ex2(__ldcg(stats + line(s0 + s, r)).z - top[r]);
            __syncthreads();
        }
        for (int s = 0; s < n; s += kAhead) {
            if (s0 + s > 0)
                ask(s0 + s);
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (s + k < n)
#pragma unroll
                    for (int i = 0; i < kItems; ++i) {
                        const float f = factor[((int)threadIdx.x + i * kAttnThreads) / (D / 4)][s + k];
                        v[i].x = fmaf(p[k][i].x, f, v[i].x);
                        v[i].y = fmaf(p[k][i].y, f, v[i].y);
                        v[i].z = fmaf(p[k][i].z, f, v[i].z);
                        v[i].w = fmaf(p[k][i].w, f, v[i].w);
                    }
        }
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int idx = (int)threadIdx.x + i * kAttnThreads, r = idx / (D / 4), d = idx % (D / 4) * 4;
        if (r < rows)
            attn_write(out + s_row[r].at * D + d, v[i], s_row[r].f);
    }
}

// ---------------------------------------------------------------------------
// TQ: uint16_t (bf16) or float.
// ---------------------------------------------------------------------------
template <typename TQ, bool kNv, int D, int NT>
__global__ void __launch_bounds__(kAttnThreads, kAttnCtas<TQ, D, NT>) kv_attention_kernel(const AttnArgs a)
{
    constexpr int kParts = sizeof(TQ) == 4 ? 2 : 1; // fp16 terms of a query element and of a weight
    constexpr int G = kNv ? 16 : 32, NB = D / G;    // scale bytes of a token
    constexpr int kStages = kAttnStages<D>, kStage = kAttnStageBytes<kNv, D>;
    constexpr int kCodes = kAttnStep * D / 2, kScales = kAttnStep * NB;
    constexpr int KS = D / 16; // k steps of the scores = 16-element tiles of the output
    constexpr int R = 8 * NT;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_exp[R]; // exponent of the power of two taken out of the row

    const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    pdl_begin();
    AttnShare share = {(int)blockIdx.z, 0, 0, 1, 0, 0};
    if (a.split && !attn_share<R>(a, share))
        return;
    const int64_t pages = a.c.slots / a.c.page;
    do { // one unit, or a piece of one
        const int b = share.b;
        int kvh = (int)blockIdx.y, rt = 0, len;
        if (a.split) {
            len = share.len;
        } else {
            if (a.row_tiles > 1) {
                kvh = (int)blockIdx.y / a.row_tiles;
                rt = (int)blockIdx.y - kvh * a.row_tiles;
            }
            len = 0; // read below, after the query rows are asked for
        }
        int from = 0, to = 0, all_rounds = 0; // rounds of the unit
        int number = 0, numbers = 0;          // where the share meets the unit's numbers, and how many it takes
        if (a.split) {
            uint32_t at = share.at, unit;
            for (;; ++rt) {
                const AttnSpan s = attn_span(a, len, attn_token(a, rt * R), attn_token(a, min(rt * R + R, a.rows) - 1));
                all_rounds = attn_rounds(s);
                unit = (uint32_t)(all_rounds + kAttnStart);
                if (at < unit * a.c.heads)
                    break;
                at -= unit * a.c.heads;
            }
            kvh = (int)(at / unit);
            number = (int)(at - kvh * unit);
            numbers = (int)min(unit - number, share.left);
            from = max(number - kAttnStart, 0);
            to = number + numbers - kAttnStart;
            if (to <= 0) // the share ends before the unit's first round
                return;
        }
        const int row0 = rt * R, rows = min(R, a.rows - row0);
        const int i0 = attn_token(a, row0); // new token of the first row
        // What the start needs from memory is asked for at once: the length, the
        // query rows (a warp takes rows warp, warp + 4, ...; a lane D / 32
        // neighbouring elements) and, below, the page table.
        if (!a.split)
            len = __ldcg(a.seq_lens + b);
        constexpr int kQRows = R / kAttnWarps, kPerLane = D / 32;
        uint32_t qraw[kQRows][kPerLane * (int)sizeof(TQ) / 4];
#pragma unroll
        for (int j = 0; j < kQRows; ++j) {
            const int r = warp + j * kAttnWarps;
            if (r < rows) {
                const int i = attn_token(a, row0 + r), h = kvh * a.group + (row0 + r) - i * a.group;
                load_words(static_cast<const TQ *>(a.q) + ((int64_t)b * a.q_tokens + i) * a.q_stride + (int64_t)h * D +
                               lane * kPerLane,
                           qraw[j]);
            } else {
#pragma unroll
                for (uint32_t &w : qraw[j])
                    w = 0u;
            }
        }
        const float gk = kNv ? __ldcg(a.c.g[0] + kvh) : 1.0f, gv = kNv ? __ldcg(a.c.g[1] + kvh) : 1.0f;
        if (!a.split && (len < 0 || len > a.capacity))
            raise_status(a.status, kStatusIndex);
        const AttnSpan sp = attn_span(a, len, i0, attn_token(a, row0 + rows - 1));
        if (!a.split)
            to = all_rounds = attn_rounds(sp);

        // this warp's steps: token tok0 + 32 (warp + 4 s), below `end`
        const int tok0 = sp.base + from * kAttnRound;
        const int end = sp.hi < sp.lo ? tok0 : min(sp.hi + 1, sp.base + to * kAttnRound);
        const int steps_all = (end - tok0 + kAttnStep - 1) / kAttnStep;
        const int steps = steps_all > warp ? (steps_all - warp + kAttnWarps - 1) / kAttnWarps : 0;
        uint8_t *const ring = smem + warp * kStages * kStage;
        const int32_t *const table = a.page_table + (int64_t)b * a.table_width;
        const int page16 = a.c.page >> 4;

        // Row (in tokens of this head) of the cache that holds the 16-token
        // granule `gr` of the sequence, -1 when no token of it is needed.
        auto granule_row = [&](int gr) -> int64_t {
            if (gr * 16 >= end)
                return -1;
            const int pi = page16 == 1 ? gr : (int)__umul64hi((uint64_t)(uint32_t)gr, a.page_magic);
            const int e = __ldcg(table + pi);
            if (e < 0 || e >= pages) {
                raise_status(a.status, kStatusIndex);
                return -1;
            }
            return ((int64_t)e * a.c.heads + kvh) * a.c.page + (int64_t)(gr - pi * page16) * 16;
        };
        // Each lane looks up one granule of the warp's next 16 steps (lane 2 s + h:
        // granule h of step s); a step's copies take theirs by shuffle.
        constexpr int kGrStep = 2 * kAttnWarps; // granules between a warp's steps
        const int gr0 = (tok0 >> 4) + 2 * warp;
        auto look_up = [&](int s16) -> int64_t {
            return granule_row(gr0 + (s16 * 16 + (lane >> 1)) * kGrStep + (lane & 1));
        };
        // Copies of one step into a stage.  Chunks of 16 bytes: codes D / 32 per
        // token, swizzled so that both operands' reads are free of bank
        // conflicts; scale bytes of the 32 keys, then of the 32 values.  A step
        // inside one page is contiguous in each array (every page of a multiple
        // of 32 tokens without a window); otherwise its two granules go apart.
        constexpr int kPer = D / 32; // chunks of a token
        const uint8_t *const kp = a.c.packed[0] + lane * 16, *const vp = a.c.packed[1] + lane * 16;
        // swizzles, the same for every 8 tokens on: XORed into the chunk's index
        const uint32_t lane_tok = (uint32_t)lane / kPer;
        const uint32_t kdst = (uint32_t)lane ^ (D == 256 ? lane_tok & 1 : 0u);
        const uint32_t vdst = (uint32_t)lane ^ (D == 64 ? (lane_tok >> 2 & 1) * 2 : (lane_tok >> 1 & 3) * 2);
        int64_t ahead = look_up(0);
        auto copy_codes = [&](uint32_t dst, int64_t row, int first, int count) { // pieces of 32 chunks
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (i < first || i >= first + count)
                    continue;
                // 32 chunks are 32 / kPer tokens: 4 for D = 256, whose swizzle alternates with the piece
                const uint32_t flip = D == 256 ? (uint32_t)(i & 1) * 4 : 0u;
                cp_async16(dst + (kdst + 32 * i) * 16, kp + row * (D / 2) + (i - first) * 512);
                cp_async16(dst + kCodes + ((vdst ^ flip) + 32 * i) * 16, vp + row * (D / 2) + (i - first) * 512);
            }
        };
        auto issue = [&](int s, uint32_t dst) {
            if (s > 0 && (s & 15) == 0)
                ahead = look_up(s >> 4);
            const int64_t row0 = __shfl_sync(0xFFFFFFFFu, ahead, 2 * (s & 15));
            const int64_t row1 = __shfl_sync(0xFFFFFFFFu, ahead, 2 * (s & 15) + 1);
            if (row0 >= 0 && row1 == row0 + 16) {
                copy_codes(dst, row0, 0, kPer);
#pragma unroll
                for (int i = 0; i < 4 * NB; i += 32)
                    if (4 * NB % 32 == 0 || i + lane < 4 * NB) {
                        const int c = i + lane; // 2 NB chunks of the keys', then of the values'
                        const uint8_t *src = c < 2 * NB ? a.c.scales[0] + c * 16 : a.c.scales[1] + (c - 2 * NB) * 16;
                        cp_async16(dst + 2 * kCodes + c * 16, src + row0 * NB);
                    }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int64_t row = h ? row1 : row0;
                    if (row < 0)
                        continue;
                    copy_codes(dst, row, h * (kPer / 2), kPer / 2);
                    if (lane < 2 * NB) {
                        const int c = lane < NB ? lane : lane - NB, v = lane >= NB;
                        cp_async16(dst + 2 * kCodes + v * kScales + h * 16 * NB + c * 16, a.c.scales[v] + row * NB + c * 16);
                    }
                }
            }
        };

        const uint32_t ring_at = smem_addr(ring);
        // fill the ring before anything else: the copies run under the query's preparation
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) {
            if (s < steps)
                issue(s, ring_at + s * kStage);
            cp_async_commit();
        }

        // Query rows to fp16, staged in the last stage of each warp's ring, which
        // the copies above left free.
        constexpr int kQRow = D + 8;
        static_assert(kParts * kQRows * kQRow * 2 <= kStage, "the staged query rows");
        auto q_at = [&](int p, int r) -> uint16_t * {
            uint8_t *const st = smem + ((r % kAttnWarps) * kStages + kStages - 1) * kStage;
            return reinterpret_cast<uint16_t *>(st) + (p * kQRows + r / kAttnWarps) * kQRow;
        };
#pragma unroll
        for (int j = 0; j < kQRows; ++j) {
            const int r = warp + j * kAttnWarps;
            float v[kPerLane];
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < kPerLane; ++e) {
                if constexpr (sizeof(TQ) == 2)
                    v[e] = __uint_as_float(e & 1 ? qraw[j][e / 2] & 0xFFFF0000u : qraw[j][e / 2] << 16);
                else
                    v[e] = __uint_as_float(qraw[j][e]);
                top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
            }
            top = __reduce_max_sync(0xFFFFFFFFu, top);
            if (top >= kNonFiniteBits && lane == 0)
                raise_status(a.status, kStatusNonFinite);
            // times 2^(14 - floor(log2 max)); rows below 2^-112 count as if their maximum were that
            int ex = max((int)(top >> 23), 15) - 127; // floor(log2 max)
            if (top >= kNonFiniteBits)
                ex = 14;
            const float up = __uint_as_float((uint32_t)(127 + (14 - ex)) << 23);
#pragma unroll
            for (int e = 0; e < kPerLane; e += 2) {
                const float x0 = v[e] * up, x1 = v[e + 1] * up;
                const uint32_t hi = pack_f16x2(x0, x1);
                *reinterpret_cast<uint32_t *>(q_at(0, r) + lane * kPerLane + e) = hi;
                if constexpr (kParts == 2) {
                    float b0, b1;
                    f16x2_to_f32(hi, b0, b1);
                    *reinterpret_cast<uint32_t *>(q_at(1, r) + lane * kPerLane + e) =
                        pack_f16x2((x0 - b0) * 2048.0f, (x1 - b1) * 2048.0f);
                }
            }
            if (lane == 0)
                s_exp[r] = ex - 14;
        }
        __syncthreads();
        // Q's operand: lane (g, t) holds row g, elements t D/4 + 4 s .. + 3 of k step s
        uint32_t qb[kParts][NT][KS][2];
        AttnFactor rowc[NT][2]; // of the scores of rows 2t, 2t + 1, in units of log2 (NVFP4: one)
        int last[NT][2], first[NT][2]; // their visible positions
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int p = 0; p < kParts; ++p)
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(q_at(p, n * 8 + g) + t * (D / 4) + 4 * s);
                    qb[p][n][s][0] = w.x;
                    qb[p][n][s][1] = w.y;
                }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = n * 8 + 2 * t + e;
                rowc[n][e] = attn_factor<kNv>(a.scale, gk, s_exp[r]);
                last[n][e] = r < rows ? sp.n - a.q_tokens + attn_token(a, row0 + r) : -1;
                first[n][e] = a.window > 0 ? last[n][e] - (int)min(a.window, (int64_t)0x40000000) + 1 : 0;
            }
        }

        float o[NT][KS][4], m[NT][2], mw[NT][2], l[NT][2]; // mw: the weights' reference (MXFP4; m for NVFP4)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[n][i][e] = 0.0f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[n][e] = mw[n][e] = -kAttnNone;
                l[n][e] = 0.0f;
            }
        }

        __syncthreads(); // the staged rows are read: their stages may be filled

        // every row of the tile sees all of [all_lo, all_hi]
        const int all_lo = a.window > 0 ? max(0, sp.hi - (int)min(a.window, (int64_t)0x40000000) + 1) : 0;
        const int all_hi = sp.n - a.q_tokens + i0;

        uint32_t v_at[2]; // the lane's codes of the values of tokens 2t and 2t + 1
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t r = (uint32_t)(2 * t + c);
            if constexpr (D == 64)
                v_at[c] = ((r * 2 + (g >> 2)) ^ ((r >> 2 & 1) * 2)) * 16 + (g & 3) * 4;
            else if constexpr (D == 128)
                v_at[c] = ((r * 4 + (g >> 1)) ^ ((r >> 1 & 3) * 2)) * 16 + (g & 1) * 8;
            else
                v_at[c] = ((r * 8 + g) ^ ((r >> 1 & 3) * 2)) * 16;
        }
        uint32_t rd = 0, wr = (kStages - 1) * kStage; // the stage to read, and the one to fill
        for (int s = 0; s < steps; ++s) {
            cp_async_wait<kStages - 2>();
            __syncwarp();
            if (s + kStages - 1 < steps)
                issue(s + kStages - 1, ring_at + wr);
            cp_async_commit();
            uint8_t *const st = ring + rd;
            wr = rd;
            rd = rd == (kStages - 1) * kStage ? 0 : rd + kStage;
            uint8_t *const ks = st + 2 * kCodes, *const vs = ks + kScales;
            const int tok = tok0 + kAttnStep * (warp + kAttnWarps * s);
            const bool edge = tok < all_lo || tok + kAttnStep - 1 > all_hi;
            if (edge) { // scale bytes of tokens that no row sees may be anything: zero them
                if (tok + lane < sp.lo || tok + lane > sp.hi) {
#pragma unroll
                    for (int i = 0; i < NB; i += 2) {
                        *reinterpret_cast<uint16_t *>(ks + lane * NB + i) = 0;
                        *reinterpret_cast<uint16_t *>(vs + lane * NB + i) = 0;
                    }
                }
                __syncwarp();
            }

            // ---- scores: two tiles of 16 tokens ----
            float x[NT][2][4];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                float acc[kParts][NT][4];
#pragma unroll
                for (int p = 0; p < kParts; ++p)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[p][n][e] = 0.0f;
                float tokf[2]; // MXFP4: 2^E of tokens g, g + 8
                constexpr int W = D / 32; // 32-bit words of a lane's codes of a token
                uint32_t w[2][W], sc[2][D / 64]; // NVFP4: the blocks' scales in pairs; MXFP4: each 16 elements' scale twice
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int r = mt * 16 + u * 8 + g;
                    if constexpr (D == 64) {
                        const uint2 v = *reinterpret_cast<const uint2 *>(st + r * 32 + t * 8);
                        w[u][0] = v.x;
                        w[u][1] = v.y;
                    } else {
#pragma unroll
                        for (int c = 0; c < W / 4; ++c) {
                            const int ch = D == 256 ? (2 * t + c) ^ (r & 1) : t;
                            const uint4 v = *reinterpret_cast<const uint4 *>(st + r * (D / 2) + ch * 16);
                            w[u][4 * c] = v.x;
                            w[u][4 * c + 1] = v.y;
                            w[u][4 * c + 2] = v.z;
                            w[u][4 * c + 3] = v.w;
                        }
                    }
                    if constexpr (kNv) {
                        if constexpr (D == 64) {
                            sc[u][0] = e4m3x2_to_f16x2(ks[r * NB + t]); // its low half
                        } else {
#pragma unroll
                            for (int c = 0; c < D / 128; ++c) {
                                const uint32_t f = e4m3x2_to_f16x2(
                                    *reinterpret_cast<const uint16_t *>(ks + r * NB + t * (D / 64) + 2 * c));
                                sc[u][c] = f; // the scales of two blocks
                            }
                        }
                        tokf[u] = 1.0f;
                    } else {
                        uint32_t lo4, top;
                        if constexpr (D == 64) {
                            lo4 = *reinterpret_cast<const uint16_t *>(ks + r * NB);
                            top = max(lo4 & 0xFFu, lo4 >> 8);
                            const int mine = (int)((lo4 >> (8 * (t >> 1))) & 0xFFu);
                            sc[u][0] = f16_exp2_neg((int)top - mine) * 0x10001u;
                        } else if constexpr (D == 128) {
                            lo4 = *reinterpret_cast<const uint32_t *>(ks + r * NB);
                            top = max_byte(lo4);
                            sc[u][0] = sc[u][1] = f16_exp2_neg((int)top - (int)((lo4 >> (8 * t)) & 0xFFu)) * 0x10001u;
                        } else {
                            const uint2 both = *reinterpret_cast<const uint2 *>(ks + r * NB);
                            top = max(max_byte(both.x), max_byte(both.y));
                            const uint32_t mine = ((t & 2) ? both.y : both.x) >> (16 * (t & 1));
                            sc[u][0] = sc[u][1] = f16_exp2_neg((int)top - (int)(mine & 0xFFu)) * 0x10001u;
                            sc[u][2] = sc[u][3] = f16_exp2_neg((int)top - (int)((mine >> 8) & 0xFFu)) * 0x10001u;
                        }
                        tokf[u] = e8m0_to_f32(top);
                    }
                }
#pragma unroll
                for (int wd = 0; wd < W; ++wd) { // two k steps a word: elements 8 wd .. 8 wd + 7
                    uint32_t f[2][4];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        e2m1_word(w[u][wd], f[u]);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            f[u][j] = kNv ? f16x2_mul_half(f[u][j], sc[u][wd / 4], wd & 2) : f16x2_mul(f[u][j], sc[u][wd / 2]);
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int p = 0; p < kParts; ++p)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma_f16(acc[p][n], f[0][2 * k], f[1][2 * k], f[0][2 * k + 1], f[1][2 * k + 1],
                                        qb[p][n][2 * wd + k][0], qb[p][n][2 * wd + k][1]);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v = acc[0][n][e];
                        if constexpr (kParts == 2)
                            v = fmaf(acc[1][n][e], 0x1p-11f, v);
                        v *= rowc[n][e & 1].f;
                        if constexpr (!kNv)
                            v = v * tokf[e >> 1] * rowc[n][e & 1].f2;
                        x[n][mt][e] = v;
                    }
            }
            if (edge) {
                // A NaN among a token's value scales would reach the rows that do not
                // see the token as well, 0 times NaN: it is taken out of the values
                // and put into the scores of the rows that do.  (MXFP4: 2^E of a value
                // joins the weight, so a weight of 0 stays one.)
                uint32_t nan = 0;
                if (kNv && a.q_tokens > 1) { // (rows of one new token see the same)
                    bool mine = false;
#pragma unroll
                    for (int i = 0; i < NB; i += 4) // a byte with seven bits set
                        mine |= __vcmpeq4(*reinterpret_cast<const uint32_t *>(vs + lane * NB + i) & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0u;
                    nan = __ballot_sync(0xFFFFFFFFu, mine);
                    if (nan) {
                        if (mine)
#pragma unroll
                            for (int i = 0; i < NB; i += 4)
                                *reinterpret_cast<uint32_t *>(vs + lane * NB + i) = 0u;
                        __syncwarp();
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int k = mt * 16 + (e >> 1) * 8 + g, j = tok + k;
                            if (j > last[n][e & 1] || j < first[n][e & 1])
                                x[n][mt][e] = -INFINITY;
                            else if (nan >> k & 1u)
                                x[n][mt][e] = NAN;
                        }
            }

            // ---- softmax of the step ----
            float ev[2][2]; // MXFP4: E of the values of token 16 mt + 8 u + g
            if constexpr (!kNv) {
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint8_t *p = vs + (mt * 16 + u * 8 + g) * NB;
                        uint32_t top;
                        if constexpr (D == 64)
                            top = max((uint32_t)p[0], (uint32_t)p[1]);
                        else if constexpr (D == 128)
                            top = max_byte(*reinterpret_cast<const uint32_t *>(p));
                        else
                            top = max(max_byte(*reinterpret_cast<const uint32_t *>(p)),
                                      max_byte(*reinterpret_cast<const uint32_t *>(p + 4)));
                        ev[mt][u] = (float)((int)top - 127);
                    }
            }
            // The reference of a row's weights follows its maximum only when a
            // score passes it by more than kAttnSlack: most steps then need no
            // exchange between lanes and no rescaling.
            bool passed = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float top = fmaxf(fmaxf(x[n][0][e], x[n][0][e + 2]), fmaxf(x[n][1][e], x[n][1][e + 2]));
                    passed |= top > m[n][e] + kAttnSlack;
                    if constexpr (!kNv) {
                        const float tw = fmaxf(fmaxf(x[n][0][e] + ev[0][0], x[n][0][e + 2] + ev[0][1]),
                                               fmaxf(x[n][1][e] + ev[1][0], x[n][1][e + 2] + ev[1][1]));
                        passed |= tw > mw[n][e] + kAttnSlack;
                    }
                }
            if (__any_sync(0xFFFFFFFFu, passed)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = fmaxf(fmaxf(x[n][0][e], x[n][0][e + 2]), fmaxf(x[n][1][e], x[n][1][e + 2]));
                        float tw = top;
                        if constexpr (!kNv)
                            tw = fmaxf(fmaxf(x[n][0][e] + ev[0][0], x[n][0][e + 2] + ev[0][1]),
                                       fmaxf(x[n][1][e] + ev[1][0], x[n][1][e + 2] + ev[1][1]));
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) {
                            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                            if constexpr (!kNv)
                                tw = fmaxf(tw, __shfl_xor_sync(0xFFFFFFFFu, tw, d));
                        }
                        if constexpr (kNv)
                            tw = top;
                        // (a row that has seen nothing yet has the reference -kAttnNone, below any score)
                        const float mn = fmaxf(m[n][e], top), mwn = fmaxf(mw[n][e], tw);
                        l[n][e] *= ex2(m[n][e] - mn);
                        const float alpha = ex2(mw[n][e] - mwn);
                        m[n][e] = mn;
                        mw[n][e] = mwn;
#pragma unroll
                        for (int i = 0; i < KS; ++i) {
                            o[n][i][e] *= alpha;
                            o[n][i][e + 2] *= alpha;
                        }
                    }
            }
            // weights of rows 2t, 2t + 1 for token g of each 8: transposed, they are the operand of row g
            uint32_t pb[kParts][NT][2][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float p[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float xx = x[n][mt][2 * u + e];
                            if constexpr (kNv) {
                                p[e] = ex2(xx - (m[n][e] - kAttnBias));
                                l[n][e] += p[e];
                            } else {
                                l[n][e] += ex2(xx - (m[n][e] - kAttnBias));
                                p[e] = ex2(xx + ev[mt][u] - (mw[n][e] - kAttnBias));
                            }
                        }
                        const uint32_t hi = pack_f16x2(p[0], p[1]);
                        pb[0][n][mt][u] = transpose8x8(hi);
                        if constexpr (kParts == 2) {
                            float b0, b1;
                            f16x2_to_f32(hi, b0, b1);
                            pb[1][n][mt][u] = transpose8x8(pack_f16x2(p[0] - b0, p[1] - b1));
                        }
                    }

            // ---- output: two k steps of 16 tokens ----
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                constexpr int W = D / 64 ? D / 64 : 1; // words of a lane's codes of a token
                uint32_t w[4][W];                      // tokens 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint8_t *v = st + kCodes + v_at[c & 1] + (mt * 16 + (c >> 1) * 8) * (D / 2);
                    if constexpr (D == 64) {
                        w[c][0] = *reinterpret_cast<const uint32_t *>(v);
                    } else if constexpr (D == 128) {
                        const uint2 x2 = *reinterpret_cast<const uint2 *>(v);
                        w[c][0] = x2.x;
                        w[c][1] = x2.y;
                    } else {
                        const uint4 x4 = *reinterpret_cast<const uint4 *>(v);
                        w[c][0] = x4.x;
                        w[c][1] = x4.y;
                        w[c][2] = x4.z;
                        w[c][3] = x4.w;
                    }
                }
                // scale pairs (token, token + 1) of the lane's 16-element pieces
                constexpr int SB = D >= 256 ? 2 : 1;
                uint32_t sv[2][SB];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int r = mt * 16 + 2 * t + 8 * c;
                    const uint8_t *p0 = vs + r * NB, *p1 = p0 + NB;
                    if constexpr (kNv) {
#pragma unroll
                        for (int i = 0; i < SB; ++i) {
                            const int at = D == 64 ? g >> 1 : SB * g + i;
                            sv[c][i] = e4m3x2_to_f16x2((uint32_t)p0[at] | (uint32_t)p1[at] << 8);
                        }
                    } else {
                        uint32_t top0, top1;
                        if constexpr (D == 64) {
                            top0 = max((uint32_t)p0[0], (uint32_t)p0[1]);
                            top1 = max((uint32_t)p1[0], (uint32_t)p1[1]);
                        } else if constexpr (D == 128) {
                            top0 = max_byte(*reinterpret_cast<const uint32_t *>(p0));
                            top1 = max_byte(*reinterpret_cast<const uint32_t *>(p1));
                        } else {
                            top0 = max(max_byte(*reinterpret_cast<const uint32_t *>(p0)),
                                       max_byte(*reinterpret_cast<const uint32_t *>(p0 + 4)));
                            top1 = max(max_byte(*reinterpret_cast<const uint32_t *>(p1)),
                                       max_byte(*reinterpret_cast<const uint32_t *>(p1 + 4)));
                        }
                        const int at = D == 64 ? g >> 2 : D == 128 ? g >> 1 : g;
                        const uint32_t pair = f16_exp2_neg((int)top0 - (int)p0[at]) |
                                              f16_exp2_neg((int)top1 - (int)p1[at]) << 16;
#pragma unroll
                        for (int i = 0; i < SB; ++i)
                            sv[c][i] = pair;
                    }
                }
                // the lane's D / 8 elements: its first D / 16 are the low rows of
                // the output tiles, its last D / 16 the high ones.  D >= 128: a
                // word of the first half with the same word of the second; D = 64:
                // the one word is both halves.
#pragma unroll
                for (int wd = 0; wd < (W + 1) / 2; ++wd) {
                    uint32_t ev_[2][2][4], od_[2][2][4]; // [half][token pair][byte]: even and odd elements of the pairs
#pragma unroll
                    for (int h = 0; h < (W > 1 ? 2 : 1); ++h)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const uint32_t w0 = w[2 * c][h * (W / 2) + wd], w1 = w[2 * c + 1][h * (W / 2) + wd];
                            // a byte: (token's element, next token's element)
                            e2m1_word((w0 & 0x0F0F0F0Fu) | ((w1 << 4) & 0xF0F0F0F0u), ev_[h][c]);
                            e2m1_word(((w0 >> 4) & 0x0F0F0F0Fu) | (w1 & 0xF0F0F0F0u), od_[h][c]);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                ev_[h][c][j] = f16x2_mul(ev_[h][c][j], sv[c][h % SB]);
                                od_[h][c][j] = f16x2_mul(od_[h][c][j], sv[c][h % SB]);
                            }
                        }
                    // element 2 j (+ 1) of a half: byte j; D = 64: bytes 0, 1 are the first half, 2, 3 the second
                    constexpr int kBytes = W > 1 ? 4 : 2;
#pragma unroll
                    for (int j = 0; j < kBytes; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t fa[4];
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const int h1 = W > 1 ? 1 : 0, j1 = W > 1 ? j : j + 2;
                                fa[2 * c] = i ? od_[0][c][j] : ev_[0][c][j];
                                fa[2 * c + 1] = i ? od_[h1][c][j1] : ev_[h1][c][j1];
                            }
#pragma unroll
                            for (int p = 0; p < kParts; ++p)
#pragma unroll
                                for (int n = 0; n < NT; ++n)
                                    mma_f16(o[n][wd * 8 + 2 * j + i], fa[0], fa[1], fa[2], fa[3], pb[p][n][mt][0],
                                            pb[p][n][mt][1]);
                        }
                }
            }
        }
        cp_async_wait<0>();

        // ---- the warps' results, merged ----
        float *const so = reinterpret_cast<float *>(smem); // [warp][row][D + 4]
        __shared__ float4 s_stats[kAttnWarps][R];
        __shared__ AttnRow s_row[R];
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[n][e];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
                    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
                const int r = n * 8 + 2 * t + e;
                if (g == 0)
                    s_stats[warp][r] = make_float4(m[n][e], sum, mw[n][e], 0.0f);
                float *dst = so + ((warp * R) + r) * (D + 4) + g * (D / 8);
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    dst[i] = o[n][i][e];
                    dst[D / 16 + i] = o[n][i][e + 2];
                }
            }
        __syncthreads();
        const bool whole = to - from == all_rounds;
        const int piece = 2 * (int)blockIdx.x + (from == 0); // a CTA's first unit may have begun before it, its last may go on
        if (threadIdx.x < rows) {
            const int r = (int)threadIdx.x;
            float mm = -kAttnNone, mx = -kAttnNone, ll = 0.0f;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                mm = fmaxf(mm, s_stats[w][r].x);
                mx = fmaxf(mx, s_stats[w][r].z);
            }
            AttnRow row;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                const float4 s = s_stats[w][r];
                ll = fmaf(s.y, ex2(s.x - mm), ll); // (a warp that saw nothing has y = 0 and a reference of -kAttnNone)
                row.w[w] = s.y > 0.0f ? ex2(s.z - mx) : 0.0f;
            }
            row.f = attn_scale<kNv>(gv, mm, mx, ll);
            row.at = attn_place(a, b, kvh, row0 + r);
            s_row[r] = row;
            if (!whole)
                a.stats[(int64_t)piece * R + r] = make_float4(mm, ll, mx, 0.0f);
            else if (a.lse)
                a.lse[row.at] = attn_lse(mm, ll);
        }
        __syncthreads();
        for (int idx = (int)threadIdx.x; idx < rows * (D / 4); idx += kAttnThreads) {
            const int r = idx / (D / 4), d = (idx % (D / 4)) * 4;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                const float f = s_row[r].w[w];
                const float4 p = *reinterpret_cast<const float4 *>(so + (w * R + r) * (D + 4) + d);
                v.x = fmaf(p.x, f, v.x);
                v.y = fmaf(p.y, f, v.y);
                v.z = fmaf(p.z, f, v.z);
                v.w = fmaf(p.w, f, v.w);
            }
            if (whole)
                attn_write(static_cast<TQ *>(a.out) + s_row[r].at * D + d, v, s_row[r].f);
            else
                *reinterpret_cast<float4 *>(a.partial + ((int64_t)piece * R + r) * D + d) = v;
        }
        if (a.split) {
            if (!whole) {
                // the unit's first round among all numbers, and the CTAs that have pieces of it
                const uint32_t u0 = share.each * blockIdx.x + share.done - (uint32_t)number + kAttnStart;
                const uint32_t first = u0 / share.each, last_cta = (u0 + (uint32_t)all_rounds - 1) / share.each;
                __shared__ bool s_last;
                __syncthreads();
                if (threadIdx.x == 0) {
                    uint32_t *const n = a.arrived + ((int64_t)b * a.row_tiles + rt) * a.c.heads + kvh;
                    uint32_t before; // releases what this CTA wrote, acquires what the others did
                    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(n) : "memory");
                    s_last = before == last_cta - first;
                    if (s_last)
                        *n = 0u;
                }
                __syncthreads();
                if (s_last)
                    attn_merge<TQ, kNv, D, R>(a.partial, a.stats, static_cast<TQ *>(a.out), a.lse, smem, s_row, gv, rows,
                                              (int)first, (int)(last_cta - first) + 1);
            }
            share.left -= numbers;
            share.at += numbers;
            share.done += numbers;
            if (kvh == a.c.heads - 1 && rt == a.row_tiles - 1 && to == all_rounds) {
                share.at = 0;
                if (++share.b < a.batch)
                    share.len = __ldcg(a.seq_lens + share.b);
            }
            __syncthreads(); // the merged results are read: the rings may be filled again
        } else {
            share.left = 0;
        }
    } while (share.left > 0);
}

} // namespace fp4
