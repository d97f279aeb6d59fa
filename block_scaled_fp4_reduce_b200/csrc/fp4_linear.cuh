// fp4_linear.cuh -- y = x W^^T for a few rows of unquantised activations and
// an FP4 weight.
//
// Bound by reading the weight once (0.53 to 0.56 bytes an element).  The
// weight is the M operand of tcgen05.mma kind::f16 (128 weight rows, fp16 by
// fp16 into fp32), so that its codes are decoded once whatever the number of
// activation rows, which are the N operand.
//
//   linear_pack_kernel  activations -> fp16 rows after a power of two per row
//                       that brings the row's maximum to 2^14 (bf16 x: exact
//                       but for what lies 2^-38 below the maximum; fp32 x: two
//                       terms, 22 bits, in two rows)
//   linear_kernel       a cluster of `splits` CTAs per 128 weight rows and up
//                       to 160 columns (activation rows, or terms of them);
//                       each CTA takes a share of K in chunks of 128 elements
//                       through a ring filled by TMA; each row's partial sums
//                       are written to the CTA of the cluster that owns the
//                       row (distributed shared memory) and added there in the
//                       order of the CTAs
//
// Roles of a CTA: warps 0-3 and 4-7 are two groups of decoders that take
// chunks in turn.  A decoder thread is one weight row: it reads the row's 64
// bytes of codes, turns them into fp16 pairs, multiplies the block scales in
// and stores the row into tensor memory (tcgen05.st; lane = row, two elements
// a column), where the MMA takes its A operand from: the decoded weight never
// passes through shared memory.  Warp 8 issues the copies, warp 9 the MMAs.
// While the MMA reads one decoded chunk the groups write the next ones.
//
// Scales: an E2M1 code times an E4M3 scale is exact in fp16.  An E8M0 scale
// does not fit fp16: MXFP4 weights are decoded relative to the largest scale
// of their row in the CTA's share of K (found by a scan of the scale bytes
// before the first chunk), 2^(e - E), which is exact down to 2^-23; the row's
// 2^E multiplies the sum.
//
// What bounds it (GPU time, calls back to back in a graph, weights larger than L2
// together): a weight of 57344 x 14336, 462 MB, takes 109 us with one activation
// row, 155 with 64 (copies alone 82).  The ring keeps HBM busy
// while a CTA is in its loop; the starts and ends of its units, about as long as
// six chunks each, and the last round of the grid are the rest.  With 64 rows the
// activations that every band of 128 weight rows reads again from L2 are 1.8
// times the weight's bytes.  An MXFP4 weight of 14336 x 4096 takes 16.6 us with 16
// rows: launch, packing and the first copies 3 us, the sums' way through the
// cluster 3, and 10 for bytes that HBM could bring in 5 (112 bands in two CTAs
// each leave half the SMs with one CTA where two fit).
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda.h>

#include "fp4_async.cuh"
#include "fp4_kernels.cuh"
#include "fp4_mma.cuh"
#include "fp4_tmem.cuh"

namespace fp4 {

constexpr int kLinRows = 128;          // weight rows of a CTA
constexpr int kLinChunk = 128;         // elements of K per stage
constexpr int kLinDecoders = 8;        // warps
constexpr int kLinThreads = 32 * (kLinDecoders + 2);
constexpr int kLinCodes = kLinRows * kLinChunk / 2; // 8 KB
constexpr int kLinScales = 1024;       // two 512-byte scale tiles (NVFP4; MXFP4 has one)
constexpr int kLinMaxCols = 160; // two part areas (below) have to fit in the ring
constexpr int kLinMaxStages = 8;
constexpr int kLinMaxSplits = 8;

// Partial sums: a CTA's own 128 rows on their way out, [owner][column][row],
// which take the ring's place, and those of the rows that it owns as they come
// in, [CTA][column][row], which have memory of their own up to 32 columns and
// follow the others in the ring's place beyond that, at the cost of a barrier
// more (every CTA has to be done with its ring).
constexpr int kLinLandingCols = 32;
__host__ __device__ constexpr int lin_part_bytes(int cols) { return cols * 4 * (kLinRows + kLinMaxSplits); }
__host__ __device__ constexpr int lin_landing_bytes(int cols) { return cols <= kLinLandingCols ? lin_part_bytes(cols) : 0; }

// Where a CTA's share of the activations is small, the decoders lay it out
// themselves, in shared memory, while the first codes are on their way: no
// packing grid and no workspace.  The most rows, and rows x chunks of K.  Laid
// out by the decoders | packed, cold L2, one call between two events, us, bf16:
// 1 x 8192 x 4096 (8 chunks a CTA) 14.5 | 16.3, 1 x 14336 x 4096 (16) 18.4 |
// 18.4, 2 x 8192 x 4096 16.3 | 16.4, 2 x 14336 x 4096 20.4 | 19.5, 4 x 4096 x
// 4096 (4) 16.4 | 14.3, 8 x 4096 x 4096 20.4 | 15.3.
constexpr int kLinFusedRows = 2, kLinFusedShare = 16;

// Codes and scales of a chunk, with its activations where those come packed.
__host__ __device__ constexpr int lin_stage_bytes(int cols, bool fused)
{
    return kLinCodes + kLinScales + (fused ? 0 : cols * kLinChunk * 2);
}
// Tensor memory: accumulators, then three decoded chunks of 64 columns.  The
// tensor core cuts a sum off rather than rounding it, which over the 112 MMAs
// of a share of 1792 elements costs 1.6e-6 of the result; with fp32 results
// the MMAs of a chunk therefore take turns on up to four accumulators, as many
// as fit (4e-7 with four).
constexpr int kLinSharedCols = 64; // the largest tile with two CTAs on an SM
constexpr int kLinBuffers = 3;
__host__ __device__ constexpr int lin_tmem_cols(int cols) { return cols <= kLinSharedCols ? 256 : 512; }
__host__ __device__ constexpr int lin_accumulators(int cols, bool f32)
{
    const int fit = (lin_tmem_cols(cols) - 64 * kLinBuffers) / cols;
    return !f32 || fit < 2 ? 1 : fit < 4 ? 2 : 4; // a power of two: MMA k of a chunk takes k modulo it
}

template <typename T> __device__ __forceinline__ float to_f32(T v)
{
    if constexpr (sizeof(T) == 2)
        return __uint_as_float((uint32_t)v << 16);
    else
        return v;
}

// fp16 terms of eight activations times `up`.
template <int kParts>
__device__ __forceinline__ void lin_terms(const float (&v)[8], float up, uint32_t (&hi)[4], uint32_t (&lo)[4])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float a = v[2 * j] * up, b = v[2 * j + 1] * up;
        hi[j] = pack_f16x2(a, b);
        if constexpr (kParts == 2) {
            float ah, bh;
            f16x2_to_f32(hi[j], ah, bh);
            lo[j] = pack_f16x2((a - ah) * 2048.0f, (b - bh) * 2048.0f);
        }
    }
}

// Eight activations from k on, zeros from n on; vec: 16-byte aligned.
template <typename T> __device__ __forceinline__ void lin_load8(const T *src, int k, int n, bool vec, float (&v)[8])
{
    if (vec && k + 8 <= n) {
        if constexpr (sizeof(T) == 2) {
            const uint4 w = __ldcg(reinterpret_cast<const uint4 *>(src + k));
            const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = __uint_as_float(a[j] << 16);
                v[2 * j + 1] = __uint_as_float(a[j] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float4 w = __ldcg(reinterpret_cast<const float4 *>(src + k) + j);
                v[4 * j] = w.x;
                v[4 * j + 1] = w.y;
                v[4 * j + 2] = w.z;
                v[4 * j + 3] = w.w;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = k + j < n ? to_f32(__ldcg(src + k + j)) : 0.0f;
    }
}

// 2^ex <= max < 2^(ex + 1) of a row whose largest magnitude has the bits
// `top`; a row below 2^-112 counts as if its maximum were that, one with a
// NaN or Inf (reported) as if no power were taken out.
__device__ __forceinline__ int lin_exponent(uint32_t top)
{
    return top >= kNonFiniteBits ? 14 : max((int)(top >> 23), 15) - 127;
}

// ---------------------------------------------------------------------------
// One CTA per activation row (padding rows of the last tile among them: zeros)
// and share of K, which are those of the product's CTAs: the power of two taken
// out of a row is that of the share, so that nothing is exchanged between CTAs
// and the elements are read once.  xh: fp16 [tiles * cols][Kpad]; a tile holds
// `per` rows and, for fp32 x, their second terms in the rows `per` on.  xe
// [tiles][shares][cols]: the exponent of the power of two that each of them is
// to be multiplied by.
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kThreads)
    linear_pack_kernel(const T *__restrict__ x, int rows, int K, int64_t x_stride, int per, int Kpad, int share, int more,
                       uint16_t *xh, int32_t *xe, int32_t *status)
{
    pdl_begin();
    // the product may start: it waits for this grid before it reads what is written here
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kParts = sizeof(T) == 4 ? 2 : 1;
    const int row = (int)blockIdx.x, tile = row / per, split = (int)blockIdx.y, splits = (int)gridDim.y;
    const int k0 = (split * share + min(split, more)) * kLinChunk, len = (share + (split < more ? 1 : 0)) * kLinChunk;
    const T *src = x + (int64_t)row * x_stride + k0;
    const int n = row < rows ? K - k0 : 0; // elements there are, from k0 on
    const bool vec = (reinterpret_cast<uintptr_t>(src) & 15u) == 0;
    float keep[8]; // the thread's first eight; a share beyond 2048 elements is read again
    uint32_t top = 0;
    for (int u = (int)threadIdx.x; u < len / 8; u += kThreads) {
        float v[8];
        lin_load8(src, u * 8, n, vec, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
            if (u < kThreads)
                keep[j] = v[j];
        }
    }
    top = cta_max_u32(top);
    if (top >= kNonFiniteBits && threadIdx.x == 0)
        raise_status(status, kStatusNonFinite);
    const int ex = lin_exponent(top), at = row - tile * per;
    const float up = __uint_as_float((uint32_t)(127 + (14 - ex)) << 23);
    if (threadIdx.x < kParts)
        xe[(tile * splits + split) * per * kParts + at + (threadIdx.x ? per : 0)] = ex - 14 - (threadIdx.x ? 11 : 0);
    uint16_t *const dst = xh + ((int64_t)tile * per * kParts + at) * Kpad + k0, *const dst2 = dst + (int64_t)per * Kpad;
    for (int u = (int)threadIdx.x; u < len / 8; u += kThreads) {
        uint32_t hi[4], lo[4];
        if (u >= kThreads)
            lin_load8(src, u * 8, n, vec, keep);
        lin_terms<kParts>(keep, up, hi, lo);
        *reinterpret_cast<uint4 *>(dst + u * 8) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if constexpr (kParts == 2)
            *reinterpret_cast<uint4 *>(dst2 + u * 8) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
}

// 2^k, -149 <= k <= 127; beyond, 0 and infinity.
__device__ __forceinline__ float exp2_int(int k)
{
    if (k < -126)
        return k < -149 ? 0.0f : __uint_as_float(1u << (k + 149));
    return k > 127 ? INFINITY : __uint_as_float((uint32_t)(k + 127) << 23);
}

__device__ __forceinline__ void cluster_arrive()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait()
{
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct LinearArgs {
    const void *x; // fused: the activations themselves
    int64_t x_stride;
    int K;
    const uint8_t *scales; // MMA layout, `tiles` 512-byte tiles per 128-row band
    const int32_t *xe;
    const float *g;
    void *y;
    int rows, N, parts, cols; // cols: columns of a tile
    int chunks, tiles, stages;
    int splits;       // CTAs of a cluster (grid x); grid y: tiles of columns, z: bands of the weight
    int share, more;  // chunks of a CTA, one more for the first `more`
    int most_share;   // chunks that the fused layout's memory holds
    int own, own_inv;   // weight rows that a CTA owns, and 2^16 / own rounded up
    uint32_t own_magic; // 2^32 / own rounded up (own = 1 does not occur)
    int accs;           // accumulators
    int out_bf16;
    int32_t *status;
};

// The decoders' layout of a CTA's activations: every thread takes eights of
// the rows; columns without a row are zeros.  Each element goes where a
// 128-byte swizzled TMA copy of the packed row would have put it: per 64
// elements a tile of 128-byte rows, 16-byte pieces XORed with the row's index
// modulo 8.  The power of two taken out of a row is that of the CTA's share of
// it, so nothing is exchanged between CTAs.
template <typename T>
__device__ __forceinline__ void lin_lay_out(const LinearArgs &a, uint8_t *x_area, float2 *factor, uint32_t *tops,
                                            int c0, int n, int row0, int have, int groups, uint64_t *laid)
{
    constexpr int kParts = sizeof(T) == 4 ? 2 : 1, kAll = 32 * kLinDecoders;
    const int tid = (int)threadIdx.x, lane = tid & 31;
    const int k0 = c0 * kLinChunk, units = n * (kLinChunk / 8), end = a.K - k0;
    auto at = [&](int u, int c) { return x_area + (u >> 3) * (a.cols * 128) + c * 128 + (((u & 7) ^ (c & 7)) * 16); };
    for (int i = tid; i < n * a.cols * (kLinChunk * 2 / 16); i += kAll)
        reinterpret_cast<uint4 *>(x_area)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tid < have)
        tops[tid] = 0u;
    asm volatile("bar.sync 1, 256;" ::: "memory");
    for (int m = 0; m < have; ++m) {
        const T *src = static_cast<const T *>(a.x) + (int64_t)(row0 + m) * a.x_stride + k0;
        const bool vec = (reinterpret_cast<uintptr_t>(src) & 15u) == 0;
        uint32_t top = 0;
        for (int u = tid; u < units; u += kAll) {
            float v[8];
            lin_load8(src, u * 8, end, vec, v);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
        }
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        if (lane == 0)
            atomicMax(&tops[m], top);
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    for (int m = 0; m < have; ++m) {
        const T *src = static_cast<const T *>(a.x) + (int64_t)(row0 + m) * a.x_stride + k0;
        const bool vec = (reinterpret_cast<uintptr_t>(src) & 15u) == 0;
        const int ex = lin_exponent(tops[m]);
        const float up = __uint_as_float((uint32_t)(127 + (14 - ex)) << 23);
        for (int u = tid; u < units; u += kAll) {
            float v[8];
            uint32_t hi[4], lo[4];
            lin_load8(src, u * 8, end, vec, v);
            lin_terms<kParts>(v, up, hi, lo);
            *reinterpret_cast<uint4 *>(at(u, m)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if constexpr (kParts == 2)
                *reinterpret_cast<uint4 *>(at(u, groups + m)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        if (tid < kParts) {
            const int e = ex - 14 - 11 * tid, e2 = e >> 1;
            factor[tid * groups + m] = make_float2(exp2_int(e2), exp2_int(e - e2));
            if (tops[m] >= kNonFiniteBits)
                raise_status(a.status, kStatusNonFinite);
        }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); // the tensor core reads what was written
    __syncwarp();
    if (lane == 0)
        mbar_arrive(laid);
}

// T: the activations' type where the kernel lays them out itself, void where
// they come packed.
template <bool kNv, typename T>
__global__ void __launch_bounds__(kLinThreads, 2)
    linear_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                  const LinearArgs a)
{
    constexpr int kTiles = kNv ? 2 : 1; // scale tiles of a chunk
    constexpr bool kFused = !std::is_void_v<T>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[kLinMaxStages], empty[kLinMaxStages], ready[kLinBuffers], done, laid, landed;
    __shared__ uint32_t tmem_slot;
    __shared__ float2 s_factor[kLinMaxCols]; // the column's power of two, in two factors
    __shared__ uint32_t s_top[kLinFusedRows];
    __shared__ float s_g;
    __shared__ int consumed; // chunks whose copies the MMA warp has seen land
    uint8_t *const smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
    const int splits = a.splits, split = (int)blockIdx.x, mtile = (int)blockIdx.y, band = (int)blockIdx.z;
    const int c0 = split * a.share + min(split, a.more), n = a.share + (split < a.more ? 1 : 0);
    const int stages = a.stages, stage_bytes = lin_stage_bytes(a.cols, kFused);
    const uint32_t tmem_cols = (uint32_t)lin_tmem_cols(a.cols);

    uint8_t *const x_area = smem + stages * stage_bytes; // fused: [chunk][two tiles of 64 elements]
    // Copies.  Where a packing grid precedes this one, it runs only once
    // everything before it is done, and the weight is no work of its: the first
    // stages of the weight are asked for before that grid ends, the
    // activations after.
    auto weight = [&](int i, int s) {
        const int c = c0 + i;
        uint8_t *const st = smem + s * stage_bytes;
        const uint32_t scale_bytes = (uint32_t)min(kTiles, a.tiles - c * kTiles) * 512u;
        mbar_expect_tx(&full[s], (uint32_t)(stage_bytes - kLinScales) + scale_bytes);
        tma_load_2d(st, &map_w, c * (kLinChunk / 2), band * kLinRows, &full[s]);
        bulk_load(st + kLinCodes, a.scales + ((int64_t)band * a.tiles + (int64_t)c * kTiles) * 512, scale_bytes, &full[s]);
    };
    auto activations = [&](int i, int s) {
        if constexpr (kFused)
            return;
        const int c = c0 + i;
        uint8_t *const st = smem + s * stage_bytes + kLinCodes + kLinScales;
        tma_load_2d(st, &map_x, c * kLinChunk, mtile * a.cols, &full[s]);
        tma_load_2d(st + a.cols * kLinChunk, &map_x, c * kLinChunk + kLinChunk / 2, mtile * a.cols, &full[s]);
    };
    const int first = n < stages ? n : stages;
    const int groups = a.cols / a.parts, have = min(groups, a.rows - mtile * groups); // activation rows of the tile
    if constexpr (kFused)
        pdl_begin();
    if (warp == kLinDecoders && elect_one()) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < kLinBuffers; ++i)
            mbar_init(&ready[i], kLinDecoders / 2);
        mbar_init(&done, 1);
        mbar_init(&laid, kLinDecoders);
        mbar_init(&landed, 1);
        mbar_init_fence();
        consumed = 0;
        mbar_expect_tx(&landed, (uint32_t)(splits * a.cols * a.own * 4));
        weight(0, 0); // the others once the rest of the CTA may go on
    }
    __syncwarp();
    if (warp == kLinDecoders + 1)
        tmem_alloc(&tmem_slot, tmem_cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot, tmem_a = tmem + tmem_cols - 64 * kLinBuffers;
    cluster_arrive(); // this CTA runs, its barriers are there: the others may copy into its shared memory

    bool timed_out = false;
    int issued = 0;
    uint32_t top = 0; // MXFP4: the largest scale byte of the thread's row in this share
    if (warp == kLinDecoders) {
        // (positions in the ring are carried along: a division by the run-time
        // number of stages costs more than the rest of a step)
        if (elect_one())
            for (int i = 1; i < first; ++i)
                weight(i, i);
        __syncwarp();
        pdl_begin();
        if (elect_one())
            for (int i = 0; i < first; ++i)
                activations(i, i);
        __syncwarp();
        issued = first;
        uint32_t phase = 0;
        for (int i = first, s = 0; i < n; ++i) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[s], phase))) {
                timed_out = true;
                break;
            }
            if (elect_one()) {
                weight(i, s);
                activations(i, s);
            }
            __syncwarp();
            ++issued;
            if (++s == stages) {
                s = 0;
                phase ^= 1u;
            }
        }
    } else if (warp == kLinDecoders + 1) {
        // MMAs: eight of K = 16 per chunk, A from tensor memory.  elect.sync, not
        // a test of the lane: the compiler then knows that one thread issues and
        // keeps the descriptors in uniform registers (measured alone at N = 16:
        // 10 cycles per MMA against 46).
        if constexpr (!kFused) {
            pdl_begin();
            for (int i = lane; i < a.cols; i += 32) { // for the epilogue
                const int e = __ldcg(a.xe + (mtile * splits + split) * a.cols + i), e2 = e >> 1;
                s_factor[i] = make_float2(exp2_int(e2), exp2_int(e - e2));
            }
        }
        if (kNv && lane == 0)
            s_g = __ldcg(a.g);
        const uint32_t idesc = (1u << 4) | ((uint32_t)(a.cols / 8) << 17) | ((uint32_t)(kLinRows / 16) << 24);
        const uint64_t x0 = smem_desc_sw128(smem_addr(kFused ? x_area : smem + kLinCodes + kLinScales));
        // in descriptor units of 16 bytes
        const uint32_t half = (uint32_t)a.cols * kLinChunk / 16, step = kFused ? 2 * half : (uint32_t)stage_bytes / 16;
        if (kFused && !__all_sync(0xFFFFFFFFu, mbar_wait(&laid, 0)))
            timed_out = true;
        // One thread runs the loop: votes and re-elections between its steps cost
        // more than the steps.
        if (elect_one()) {
            int i = 0;
            for (uint32_t s = 0, b = 0, phase = 0, ready_phase = 0; i < n && !timed_out; ++i) {
                if (!mbar_wait_both(&ready[b], ready_phase, &full[s], phase)) {
                    timed_out = true;
                    break;
                }
                tc_fence_after();
                const uint64_t x = x0 + (uint64_t)((kFused ? (uint32_t)i : s) * step);
                const uint32_t w = tmem_a + 64 * b;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    tc_mma_f16_ts(tmem + (uint32_t)((k & (a.accs - 1)) * a.cols), w + (uint32_t)(8 * k),
                                  x + (uint64_t)((k >> 2) * half + (uint32_t)(k & 3) * 2), idesc, i > 0 || k >= a.accs);
                tc_commit(&empty[s]);
                if (++s == (uint32_t)stages) {
                    s = 0;
                    phase ^= 1u;
                }
                if (++b == kLinBuffers) {
                    b = 0;
                    ready_phase ^= 1u;
                }
            }
            consumed = i;
            tc_commit(&done);
        }
        timed_out = __any_sync(0xFFFFFFFFu, timed_out);
    } else {
        const int group = warp >> 2, quarter = warp & 3; // rows 32 quarter .. + 31: the tensor-memory lanes this warp reaches
        const int row = quarter * 32 + lane, word = lane * 16 + quarter * 4; // its scale word in a tile
        if constexpr (kFused)
            lin_lay_out<T>(a, x_area, s_factor, s_top, c0, n, mtile * groups, have, groups, &laid);
        if constexpr (!kNv) {
            const uint8_t *p = a.scales + ((int64_t)band * a.tiles + c0) * 512 + word;
            uint32_t m4 = 0;
            const int tiles = min(c0 + n, a.tiles) - c0;
#pragma unroll 8
            for (int i = 0; i < tiles; ++i)
                m4 = __vmaxu4(m4, __ldcg(reinterpret_cast<const uint32_t *>(p + (int64_t)i * 512)));
            top = max(max(m4 & 0xFFu, (m4 >> 8) & 0xFFu), max((m4 >> 16) & 0xFFu, m4 >> 24));
        }
        // positions of this chunk in the ring and among the buffers, and of the
        // chunk that the buffer held before
        int s = group, b = group, old = group;
        uint32_t phase = 0, old_phase = 0;
        for (int i = group; i < n; i += 2) {
            // (from chunk 3 on: and the MMA has read what the buffer held, chunk i - 3)
            const bool ok = i >= kLinBuffers ? mbar_wait_both(&full[s], phase, &empty[old], old_phase)
                                             : mbar_wait(&full[s], phase);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                timed_out = true;
                break;
            }
            const uint8_t *const st = smem + s * stage_bytes;
            const uint8_t *const codes = st + row * 64, *const sf = st + kLinCodes + word;
            const uint32_t dst = tmem_a + (uint32_t)(64 * b) + ((uint32_t)(quarter * 32) << 16);
            uint32_t s4[kTiles];
#pragma unroll
            for (int j = 0; j < kTiles; ++j)
                // (a weight's last chunk may have one tile alone; nothing is copied past it)
                s4[j] = j == 0 || (c0 + i) * kTiles + j < a.tiles ? *reinterpret_cast<const uint32_t *>(sf + j * 512) : 0u;
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < 2; ++h) { // 64 elements
                uint32_t f[32];
#pragma unroll
                for (int q = 0; q < 2; ++q) { // 32 elements: one 16-byte read
                    const int ch = 2 * h + q;
                    const uint4 v = *reinterpret_cast<const uint4 *>(codes + ((ch ^ (row >> 1 & 3)) * 16));
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    uint32_t sc[2];
                    if constexpr (kNv) { // blocks 2 ch, 2 ch + 1
                        const uint32_t p = e4m3x2_to_f16x2(s4[h] >> (16 * q));
                        sc[0] = __byte_perm(p, p, 0x1010);
                        sc[1] = __byte_perm(p, p, 0x3232);
                    } else {
                        sc[0] = sc[1] = f16_exp2_neg((int)top - (int)((s4[0] >> (8 * ch)) & 0xFFu)) * 0x10001u;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t d[4];
                        e2m1_word(w[j], d);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            f[16 * q + 4 * j + e] = f16x2_mul(d[e], sc[j >> 1]);
                    }
                }
                tc_store_32(dst + (uint32_t)(32 * h), f);
            }
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&ready[b]);
            if (i >= kLinBuffers)
                old += 2;
            else
                old = i + 2 - kLinBuffers; // chunk 0 or 1: the first that a buffer is taken from
            if (old >= stages) {
                old -= stages;
                old_phase ^= 1u;
            }
            s += 2;
            if (s >= stages) {
                s -= stages;
                phase ^= 1u;
            }
            b += 2;
            if (b >= kLinBuffers)
                b -= kLinBuffers;
        }
        if constexpr (!kFused)
            pdl_begin(); // what is read and written below follows the packing grid
    }

    // ---- the sums, times g or 2^E and the column's power of two, to the CTA that owns the row ----
    const bool ok = mbar_wait(&done, 0);
    if (!ok || timed_out)
        raise_status(a.status, kStatusTimeout);
    if (warp == kLinDecoders) // copies that nobody waited for (only after a timeout) land before the CTA ends
        for (int i = consumed; i < issued; ++i)
            (void)mbar_wait(&full[i % stages], (uint32_t)(i / stages) & 1u);
    float *const part = reinterpret_cast<float *>(smem);
    float *const land = reinterpret_cast<float *>(
        smem + (a.cols > kLinLandingCols ? lin_part_bytes(a.cols)
                                         : stages * stage_bytes + (kFused ? a.most_share * a.cols * kLinChunk * 2 : 0)));
    __syncthreads();
    if (warp < kLinDecoders) {
        tc_fence_after();
        const int quarter = warp & 3, row = quarter * 32 + lane;
        const int owner = (row * a.own_inv) >> 16; // row / own
        float *const to = part + owner * (a.cols - 1) * a.own + row; // [owner][column][row - owner * own]
        // The row's factor (g, or 2^E) between the two halves of the column's:
        // neither alone need keep a sum inside fp32's range that both together
        // leave there.
        const float r = kNv ? s_g : e8m0_to_f32(top);
        for (int c = (warp >> 2) * 8; c < a.cols; c += 16) {
            if (c >= have && (a.parts == 1 || c < groups || c >= groups + have))
                continue; // columns without a row
            float v[8];
            tc_load_8(tmem + (uint32_t)c + ((uint32_t)(quarter * 32) << 16), v);
            for (int q = 1; q < a.accs; ++q) {
                float more[8];
                tc_load_8(tmem + (uint32_t)(q * a.cols + c) + ((uint32_t)(quarter * 32) << 16), more);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] += more[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 f = s_factor[c + j];
                to[(c + j) * a.own] = v[j] * f.x * r * f.y;
            }
        }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); // the copies below read what was written
    tc_fence_before();
    __syncthreads();
    cluster_wait(); // every CTA of the cluster runs
    if (a.cols > kLinLandingCols) {
        cluster_arrive();
        cluster_wait(); // and is done with its ring
    }
    if (warp == kLinDecoders + 1)
        tmem_dealloc(tmem, tmem_cols);
    if (warp == 0 && lane < splits) { // each owner its rows (whole blocks: columns without a row hold anything)
        uint32_t dst, bar;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst) : "r"(smem_addr(land + split * a.cols * a.own)), "r"(lane));
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar) : "r"(smem_addr(&landed)), "r"(lane));
        asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                     "r"(smem_addr(part + lane * a.cols * a.own)), "r"(a.cols * a.own * 4), "r"(bar)
                     : "memory");
    }
    __syncwarp();

    // ---- the rows of this CTA, summed over the cluster in order ----
    if (!mbar_wait(&landed, 0))
        raise_status(a.status, kStatusTimeout);
    const int col0 = band * kLinRows + split * a.own;
    const int mine = min(min(a.own, kLinRows - split * a.own), a.N - col0);
    for (int i = (int)threadIdx.x; i < have * a.own; i += kLinThreads) {
        const int m = (int)__umulhi((uint32_t)i, a.own_magic), r = i - m * a.own; // i / own
        if (r >= mine)
            continue;
        float y = 0.0f;
        for (int p = 0; p < a.parts; ++p) {
            const float *const src = land + (p * groups + m) * a.own + r;
            float f[kLinMaxSplits];
#pragma unroll
            for (int s = 0; s < kLinMaxSplits; ++s)
                f[s] = s < splits ? src[s * a.cols * a.own] : 0.0f;
#pragma unroll
            for (int s = 0; s < kLinMaxSplits; ++s)
                y += f[s];
        }
        const int64_t o = (int64_t)(mtile * groups + m) * a.N + col0 + r;
        if (a.out_bf16)
            static_cast<uint16_t *>(a.y)[o] = to_out<uint16_t>(y);
        else
            static_cast<float *>(a.y)[o] = y;
    }
    // this CTA's shared memory is the source of copies until they have landed
    cluster_arrive();
    cluster_wait();
}

} // namespace fp4
