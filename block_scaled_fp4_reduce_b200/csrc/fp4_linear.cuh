// fp4_linear.cuh -- y = x W^^T for a few rows of unquantised activations and
// an FP4 weight.
//
// Bound by reading the weight once (0.53 to 0.56 bytes an element), so the
// weight is the M operand of the tensor cores: mma.sync m16n8k16 takes 16
// weight rows and 8 activation rows, the codes become fp16 in registers on
// their way from shared memory, and one decoded fragment serves every
// activation row.
//
//   linear_pack_kernel  activations -> fp16 after a power of two per row that
//                       brings its maximum to 2^14 (bf16 x: exact but for
//                       what lies 2^-38 below the maximum; fp32 x: two terms,
//                       22 bits), written in the order in which the MMA's B
//                       fragments are read
//   linear_kernel       a cluster of `splits` CTAs per 128 weight rows and 8
//                       kNt activation rows; each CTA takes a share of K in
//                       stages of 256 elements through a ring filled by TMA,
//                       the partial results meet over distributed shared
//                       memory, summed in the order of the CTAs
//
// Fragments (lane = 4 g + t): per 128 elements of K ("chunk"), lane (g, t)
// reads 32 codes of weight rows g and g + 8.  Which element is which k index
// of the MMA is free as long as both operands agree:
//   NVFP4  elements 32 t .. 32 t + 31, one 16-byte load, two blocks of 16; a
//          code times its E4M3 scale is exact in fp16, so the scale is
//          multiplied in before the MMA
//   MXFP4  elements 8 t .. 8 t + 7 of each of the four blocks of 32, so that
//          two MMAs cover one block: their sum is added in fp32 times one
//          factor, 2^e and the power of two of the activation row, so that
//          neither takes the sum out of fp32's range on its own
#pragma once

#include <cstdint>

#include <cuda.h>

#include "fp4_async.cuh"
#include "fp4_kernels.cuh"
#include "fp4_mma.cuh"

namespace fp4 {

constexpr int kLinRows = 128;               // weight rows of a CTA
constexpr int kLinStep = 256;               // elements of K per stage: two chunks of 128
constexpr int kLinWarps = 8;                // 4 groups of 32 rows x the stage's 2 chunks
constexpr int kLinThreads = 32 * (kLinWarps + 1); // + the producer
constexpr int kLinCodes = kLinRows * kLinStep / 2; // 16 KB: two boxes of 64 bytes x 128 rows
constexpr int kLinFrag = 2048;              // one chunk of 8 activation rows in fragment order
constexpr int kLinMaxSplits = 8;

template <bool kNv> constexpr int kLinScales = kNv ? 2048 : 1024; // scale tiles of a stage
template <bool kNv, int kNt> constexpr int kLinStage = kLinCodes + kLinScales<kNv> + 2 * kNt * kLinFrag;
// Two CTAs share an SM up to 16 activation rows (or terms of them), so that
// one's start and end run under the other's stream; beyond, the ring of one.
template <bool kNv, int kNt> constexpr int kLinStages = kNt <= 2 ? 4 : kNt == 4 ? 3 : 4;
template <bool kNv, int kNt> constexpr int kLinSmem = kLinStages<kNv, kNt> * kLinStage<kNv, kNt> + 1024;

// Address of the 16-byte unit `u` (8 elements) of a chunk of activation row g
// inside the chunk's 2 KB: [j][lane][8 halves].
template <bool kNv> __device__ __forceinline__ int lin_frag_at(int g, int u)
{
    const int t = kNv ? u >> 2 : u & 3, j = kNv ? u & 3 : u >> 2;
    return j * 512 + (4 * g + t) * 16;
}

template <typename T> __device__ __forceinline__ float to_f32(T v)
{
    if constexpr (sizeof(T) == 2)
        return __uint_as_float((uint32_t)v << 16);
    else
        return v;
}

// ---------------------------------------------------------------------------
// One CTA per activation row (rows past the last: zeros).  frags: [tile][chunk]
// [column group of 8][2 KB], fp32 rows as two terms, the second in the
// groups kNt / 2 on; xs: [tile][8 kNt] the power of two each column stands for.
// ---------------------------------------------------------------------------
template <typename T, bool kNv>
__global__ void __launch_bounds__(kThreads)
    linear_pack_kernel(const T *__restrict__ x, int rows, int K, int64_t x_stride, int nt, int chunks, uint8_t *frags,
                       float *xs, int32_t *status)
{
    pdl_begin();
    // the product may start: it waits for this grid before it reads what is written here
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kParts = sizeof(T) == 4 ? 2 : 1;
    const int row = (int)blockIdx.x;
    const int per = 8 * nt / kParts, tile = row / per, r = row - tile * per; // rows of a tile
    const T *src = x + (int64_t)row * x_stride;
    const int n = row < rows ? K : 0;
    const bool vec = (reinterpret_cast<uintptr_t>(src) & 15u) == 0;
    constexpr int kVec = 16 / (int)sizeof(T);
    uint32_t top = 0;
    const int nv = vec ? n / kVec : 0;
    for (int i = (int)threadIdx.x; i < nv; i += kThreads) {
        const uint4 w = __ldcg(reinterpret_cast<const uint4 *>(src) + i);
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(T) == 2)
                top = max(top, max((a[j] << 16) & 0x7FFF0000u, a[j] & 0x7FFF0000u));
            else
                top = max(top, a[j] & 0x7FFFFFFFu);
        }
    }
    for (int i = nv * kVec + (int)threadIdx.x; i < n; i += kThreads)
        top = max(top, __float_as_uint(to_f32(__ldcg(src + i))) & 0x7FFFFFFFu);
    top = cta_max_u32(top);
    const bool bad = top >= kNonFiniteBits;
    if (bad && threadIdx.x == 0)
        raise_status(status, kStatusNonFinite);
    // 2^ex <= max < 2^(ex + 1); a row below 2^-112 counts as if its maximum were that
    const int ex = bad ? 14 : max((int)(top >> 23), 15) - 127;
    const float up = __uint_as_float((uint32_t)(127 + (14 - ex)) << 23);
    const int groups = nt / kParts;
    if (threadIdx.x < kParts)
        xs[tile * 8 * nt + threadIdx.x * groups * 8 + r] =
            __uint_as_float((uint32_t)(127 + (ex - 14)) << 23) * (threadIdx.x ? 0x1p-11f : 1.0f);
    uint8_t *dst = frags + ((int64_t)tile * chunks * nt + (r >> 3)) * kLinFrag;
    for (int u = (int)threadIdx.x; u < chunks * 16; u += kThreads) { // units of 8 elements
        const int k = u * 8;
        float v[8];
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
        uint32_t hi[4], lo[4];
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
        uint8_t *p = dst + (int64_t)(u >> 4) * nt * kLinFrag + lin_frag_at<kNv>(r & 7, u & 15);
        *reinterpret_cast<uint4 *>(p) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if constexpr (kParts == 2)
            *reinterpret_cast<uint4 *>(p + groups * kLinFrag) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
}

__device__ __forceinline__ void cluster_sync()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct LinearArgs {
    const uint8_t *scales; // MMA layout, `tiles` 512-byte tiles per 128-row band
    const uint8_t *frags;
    const float *xs, *g;
    void *y;
    int rows, N, parts, stages, tiles, out_bf16;
    int splits, mtiles; // CTAs of a cluster, tiles of activation rows
    int32_t *status;
};

template <bool kNv, int kNt>
__global__ void __launch_bounds__(kLinThreads, kNt <= 4 ? 2 : 1)
    linear_kernel(const __grid_constant__ CUtensorMap map, const LinearArgs a)
{
    constexpr int kStages = kLinStages<kNv, kNt>, kStage = kLinStage<kNv, kNt>;
    constexpr int kTiles = kLinScales<kNv> / 512; // scale tiles of a stage
    constexpr int kCols = 8 * kNt;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[kStages], empty[kStages];
    uint8_t *const smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int unit = (int)blockIdx.x / a.splits, split = (int)blockIdx.x - unit * a.splits; // a cluster a unit
    const int band = unit / a.mtiles, mtile = unit - band * a.mtiles, splits = a.splits;
    const int s0 = (int)((int64_t)a.stages * split / splits), s1 = (int)((int64_t)a.stages * (split + 1) / splits);
    const int n_st = s1 - s0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kLinWarps);
        }
        mbar_init_fence();
    }
    // Scale bytes past the last tile are never copied: they must not be NaN.
    for (int i = (int)threadIdx.x; i < kStages * kLinScales<kNv> / 16; i += kLinThreads) {
        const int s = i / (kLinScales<kNv> / 16), at = i - s * (kLinScales<kNv> / 16);
        *reinterpret_cast<uint4 *>(smem + s * kStage + kLinCodes + at * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();

    float acc[2][kNt][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < kNt; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[i][n][e] = 0.0f;
    bool timed_out = false;

    if (warp == kLinWarps) {
        // Producer.  The weight is no work of the packing grid's, which runs
        // only once everything before it is done: its stages are asked for
        // before that grid ends, the activations after.
        auto weight = [&](int i) {
            const int s = i % kStages, k = s0 + i;
            uint8_t *const st = smem + s * kStage;
            const int tiles = min(kTiles, a.tiles - k * kTiles);
            mbar_expect_tx(&full[s], (uint32_t)(kLinCodes + tiles * 512 + 2 * kNt * kLinFrag));
            tma_load_2d(st, &map, k * 128, band * kLinRows, &full[s]);
            tma_load_2d(st + kLinCodes / 2, &map, k * 128 + 64, band * kLinRows, &full[s]);
            bulk_load(st + kLinCodes, a.scales + ((int64_t)band * a.tiles + (int64_t)k * kTiles) * 512,
                      (uint32_t)tiles * 512u, &full[s]);
        };
        auto activations = [&](int i) {
            const int s = i % kStages, k = s0 + i;
            bulk_load(smem + s * kStage + kLinCodes + kLinScales<kNv>,
                      a.frags + ((int64_t)mtile * a.stages + k) * (2 * kNt * kLinFrag), 2 * kNt * kLinFrag, &full[s]);
        };
        const int first = n_st < kStages ? n_st : kStages;
        if (lane == 0)
            for (int i = 0; i < first; ++i)
                weight(i);
        pdl_begin();
        if (lane == 0)
            for (int i = 0; i < first; ++i)
                activations(i);
        __syncwarp();
        int issued = first;
        for (int i = first; i < n_st; ++i) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[i % kStages], (uint32_t)(i / kStages - 1) & 1u))) {
                timed_out = true;
                break;
            }
            if (lane == 0) {
                weight(i);
                activations(i);
            }
            __syncwarp();
            ++issued;
        }
        // the last copies land before the shared memory has another use
        for (int i = issued - kStages > 0 ? issued - kStages : 0; i < issued; ++i)
            if (!mbar_wait(&full[i % kStages], (uint32_t)(i / kStages) & 1u))
                timed_out = true;
    } else {
        pdl_begin();
        const int wr = warp & 3, wk = warp >> 2; // rows 32 wr .. + 31, chunk wk of every stage
        float xs[kNt][2];
        if constexpr (!kNv) {
#pragma unroll
            for (int n = 0; n < kNt; ++n) {
                const float2 v = __ldcg(reinterpret_cast<const float2 *>(a.xs + mtile * kCols + n * 8 + 2 * t));
                xs[n][0] = v.x;
                xs[n][1] = v.y;
            }
        }
        for (int i = 0; i < n_st; ++i) {
            const int s = i % kStages;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[s], (uint32_t)(i / kStages) & 1u))) {
                timed_out = true;
                break;
            }
            const uint8_t *const st = smem + s * kStage;
            const uint8_t *const codes = st + wk * (kLinCodes / 2);
            const uint8_t *const sf = st + kLinCodes + wk * (kLinScales<kNv> / 2);
            const uint4 *const xf = reinterpret_cast<const uint4 *>(st + kLinCodes + kLinScales<kNv> + wk * kNt * kLinFrag) + lane;
            // row r of the band: codes at 64 r (16-byte chunks swizzled by
            // (r / 2) % 4), scale word at 16 (r % 32) + 4 (r / 32); the warp's
            // rows are 32 wr + 16 i + 8 u + g
            if constexpr (kNv) {
                uint32_t w[2][2][4], sc[2][2][2];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int r = 16 * m + 8 * u + g;
                        const uint4 v = *reinterpret_cast<const uint4 *>(codes + (wr * 32 + r) * 64 + ((t ^ (r >> 1 & 3)) * 16));
                        w[m][u][0] = v.x;
                        w[m][u][1] = v.y;
                        w[m][u][2] = v.z;
                        w[m][u][3] = v.w;
                        const uint32_t f = e4m3x2_to_f16x2(
                            *reinterpret_cast<const uint16_t *>(sf + (t >> 1) * 512 + r * 16 + wr * 4 + (t & 1) * 2));
                        sc[m][u][0] = __byte_perm(f, f, 0x1010);
                        sc[m][u][1] = __byte_perm(f, f, 0x3232);
                    }
#pragma unroll
                for (int j = 0; j < 4; ++j) { // 8 elements of each lane: two k steps
                    uint4 b[kNt];
#pragma unroll
                    for (int n = 0; n < kNt; ++n)
                        b[n] = xf[(n * kLinFrag + j * 512) / 16];
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        uint32_t f[2][4];
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            e2m1_word(w[m][u][j], f[u]);
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                f[u][q] = f16x2_mul(f[u][q], sc[m][u][j >> 1]);
                        }
#pragma unroll
                        for (int n = 0; n < kNt; ++n) {
                            mma_f16(acc[m][n], f[0][0], f[1][0], f[0][1], f[1][1], b[n].x, b[n].y);
                            mma_f16(acc[m][n], f[0][2], f[1][2], f[0][3], f[1][3], b[n].z, b[n].w);
                        }
                    }
                }
            } else {
                uint32_t se[2][2];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        se[m][u] = *reinterpret_cast<const uint32_t *>(sf + (16 * m + 8 * u + g) * 16 + wr * 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) { // block j of the chunk
                    uint4 b[kNt];
#pragma unroll
                    for (int n = 0; n < kNt; ++n)
                        b[n] = xf[(n * kLinFrag + j * 512) / 16];
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        uint32_t f[2][4];
                        float e[2];
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int r = 16 * m + 8 * u + g;
                            e2m1_word(*reinterpret_cast<const uint32_t *>(codes + (wr * 32 + r) * 64 +
                                                                          ((j ^ (r >> 1 & 3)) * 16) + 4 * t),
                                      f[u]);
                            e[u] = e8m0_to_f32((se[m][u] >> (8 * j)) & 0xFFu);
                        }
#pragma unroll
                        for (int n = 0; n < kNt; ++n) {
                            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            mma_f16(c, f[0][0], f[1][0], f[0][1], f[1][1], b[n].x, b[n].y);
                            mma_f16(c, f[0][2], f[1][2], f[0][3], f[1][3], b[n].z, b[n].w);
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                acc[m][n][q] = fmaf(c[q], xs[n][q & 1] * e[q >> 1], acc[m][n][q]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&empty[s]);
        }
    }
    if (timed_out)
        raise_status(a.status, kStatusTimeout);

    // ---- the two chunk halves, then the CTAs of the cluster ----
    float *const part = reinterpret_cast<float *>(smem); // [column][128 rows]
    __syncthreads();
    const int wr = warp & 3;
    auto at = [&](int m, int n, int q) { return (n * 8 + 2 * t + (q & 1)) * kLinRows + wr * 32 + 16 * m + 8 * (q >> 1) + g; };
    if (warp < kLinWarps && warp >= 4) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < kNt; ++n)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    part[at(m, n, q)] = acc[m][n][q];
    }
    __syncthreads();
    if (warp < 4) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < kNt; ++n)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    part[at(m, n, q)] += acc[m][n][q];
    }
    cluster_sync();
    const int per = kLinRows / splits, groups = kCols / a.parts; // weight rows of this CTA, activation rows of the tile
    const float gw = kNv ? __ldcg(a.g) : 1.0f;
    for (int i = (int)threadIdx.x; i < groups * per; i += kLinThreads) {
        const int m = i / per, r = split * per + (i - m * per);
        const int row = mtile * groups + m, col = band * kLinRows + r;
        if (row >= a.rows || col >= a.N)
            continue;
        auto column = [&](int c) { // summed over the cluster, in order
            const uint32_t src = smem_addr(part + c * kLinRows + r);
            float v = 0.0f;
            for (int s = 0; s < splits; ++s) {
                uint32_t remote;
                float f;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(src), "r"(s));
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(remote) : "memory");
                v += f;
            }
            return v;
        };
        // (in double: g and the row's power of two may take turns out of fp32's range)
        double y = column(m);
        if constexpr (kNv)
            y *= (double)__ldcg(a.xs + mtile * kCols + m);
        if (a.parts == 2) {
            double lo = column(groups + m);
            if constexpr (kNv)
                lo *= (double)__ldcg(a.xs + mtile * kCols + groups + m);
            y += lo;
        }
        const float out = kNv ? (float)(y * (double)gw) : (float)y;
        const int64_t o = (int64_t)row * a.N + col;
        if (a.out_bf16)
            static_cast<uint16_t *>(a.y)[o] = to_out<uint16_t>(out);
        else
            static_cast<float *>(a.y)[o] = out;
    }
    cluster_sync();
}

} // namespace fp4
