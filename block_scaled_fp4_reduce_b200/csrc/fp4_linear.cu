// fp4_linear.cu -- entry points of include/fp4.h for the product of a few
// rows of activations with an FP4 weight: argument checks and the launches.
#include <climits>
#include <cstdint>
#include <cstring>

#include <cuda.h>
#include <cuda_runtime.h>

#include "fp4.h"
#include "fp4_launch.cuh"
#include "fp4_linear.cuh"

namespace {

using namespace fp4_launch;
using fp4::kThreads;

// 2-D tensor map of the packed weight [N, Kp/2] bytes: boxes of 64 bytes x
// 128 rows, 64-byte swizzle.
fp4_status weight_map(const uint8_t *p, int64_t N, int64_t Kp, CUtensorMap *map)
{
    EncodeTiled enc = encode_tiled();
    if (!enc)
        return FP4_ERR_CUDA;
    const cuuint64_t dims[2] = {(cuuint64_t)(Kp / 2), (cuuint64_t)N};
    const cuuint64_t strides[1] = {(cuuint64_t)(Kp / 2)};
    const cuuint32_t box[2] = {64u, (cuuint32_t)fp4::kLinRows};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(p), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FP4_OK : FP4_ERR_CUDA;
}

// Column groups of 8 in a tile: enough for the rows (each `parts` columns),
// at most 8.
int tile_groups(int64_t rows, int parts)
{
    int nt = parts;
    while (nt < 8 && (int64_t)8 * nt < rows * parts)
        nt *= 2;
    return nt;
}

// Workspace of the laid-out activations: their fragments, then a power of
// two for each column.
struct Layout {
    int nt, stages;
    int64_t tiles; // of activation rows
    size_t frags, bytes;
};

Layout layout(int64_t rows, int64_t Kp, int parts)
{
    Layout l;
    l.nt = tile_groups(rows, parts);
    l.stages = (int)((Kp + fp4::kLinStep - 1) / fp4::kLinStep);
    l.tiles = (rows * parts + 8 * l.nt - 1) / (8 * l.nt);
    l.frags = (size_t)l.tiles * l.stages * 2 * l.nt * fp4::kLinFrag;
    l.bytes = l.frags + (size_t)l.tiles * 8 * l.nt * sizeof(float);
    return l;
}

// CTAs of a cluster: K is split until the grid fills the GPU twice over, as
// long as every CTA keeps two stages.
int pick_splits(int64_t tiles, int stages, int sms)
{
    int s = 1;
    while (s < fp4::kLinMaxSplits && tiles * s < 2 * sms && stages >= 4 * s)
        s *= 2;
    return s;
}

template <bool kNv, int kNt>
fp4_status launch_linear(const CUtensorMap &map, fp4::LinearArgs a, int64_t mtiles, int sms, cudaStream_t stream)
{
    auto kernel = fp4::linear_kernel<kNv, kNt>;
    constexpr int smem = fp4::kLinSmem<kNv, kNt>;
    if (!smem_attr(kernel, smem))
        return FP4_ERR_CUDA;
    const int64_t bands = (a.N + fp4::kLinRows - 1) / fp4::kLinRows;
    const int splits = pick_splits(bands * mtiles, a.stages, sms);
    cudaLaunchConfig_t cfg = {};
    if (bands * mtiles > INT_MAX / splits)
        return FP4_ERR_SHAPE;
    a.splits = splits;
    a.mtiles = (int)mtiles;
    cfg.gridDim = dim3((unsigned)(bands * mtiles * splits));
    cfg.blockDim = dim3(fp4::kLinThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)splits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kernel, map, a) != cudaSuccess) {
        (void)cudaGetLastError();
        return FP4_ERR_CUDA;
    }
    return FP4_OK;
}

template <typename T, bool kNv>
fp4_status run_linear(const T *x, int64_t rows, int64_t K, int64_t x_stride, const CUtensorMap &map, fp4::LinearArgs a,
                      const Layout &l, int sms, cudaStream_t stream)
{
    const int64_t packed_rows = l.tiles * 8 * l.nt / a.parts;
    fp4_status st = launch(fp4::linear_pack_kernel<T, kNv>, (int)packed_rows, stream, x, (int)rows, (int)K, x_stride,
                           l.nt, 2 * l.stages, const_cast<uint8_t *>(a.frags), const_cast<float *>(a.xs), a.status);
    if (st != FP4_OK)
        return st;
    switch (l.nt) {
    case 1: return launch_linear<kNv, 1>(map, a, l.tiles, sms, stream);
    case 2: return launch_linear<kNv, 2>(map, a, l.tiles, sms, stream);
    case 4: return launch_linear<kNv, 4>(map, a, l.tiles, sms, stream);
    default: return launch_linear<kNv, 8>(map, a, l.tiles, sms, stream);
    }
}

} // namespace

extern "C" {

size_t fp4_linear_workspace_bytes(int64_t rows, int64_t K)
{
    if (rows < 0 || K < 0 || rows > INT_MAX || K > INT_MAX - 1024)
        return 0;
    const size_t one = layout(rows, K, 1).bytes, two = layout(rows, K, 2).bytes; // either type of x
    return one > two ? one : two;
}

fp4_status fp4_linear(fp4_format fmt, const void *x, fp4_dtype dtype, int64_t rows, int64_t K, int64_t x_stride,
                      const uint8_t *packed, const uint8_t *scales_mma, const float *global_scale, int64_t N, void *y,
                      fp4_dtype out_dtype, void *workspace, size_t workspace_bytes, int32_t *status,
                      cudaStream_t stream)
{
    if ((fmt != FP4_NVFP4 && fmt != FP4_MXFP4) || !valid_dtype(dtype) || !valid_dtype(out_dtype) || rows < 0 ||
        K < 0 || N < 0 || !status)
        return FP4_ERR_INVALID_ARG;
    const int64_t group = fmt == FP4_NVFP4 ? 16 : 32;
    const int64_t in = dtype == FP4_BF16 ? 2 : 4, on = out_dtype == FP4_BF16 ? 2 : 4;
    if (rows > INT_MAX || K > INT_MAX - 1024 || N > INT_MAX - 1024)
        return FP4_ERR_SHAPE;
    const int64_t Kp = (K + group - 1) / group * group;
    if (Kp % 32)
        return FP4_ERR_SHAPE;
    if (rows == 0 || N == 0)
        return FP4_OK;
    if (x_stride < K || x_stride > INT64_MAX / 8 / rows)
        return FP4_ERR_SHAPE;
    if (!y)
        return FP4_ERR_INVALID_ARG;
    if (!aligned(y, on))
        return FP4_ERR_ALIGN;
    if (K == 0) { // an empty sum
        if (cudaMemsetAsync(y, 0, (size_t)(rows * N * on), stream) != cudaSuccess) {
            (void)cudaGetLastError();
            return FP4_ERR_CUDA;
        }
        return FP4_OK;
    }
    if (!x || !packed || !scales_mma || (fmt == FP4_NVFP4 && !global_scale))
        return FP4_ERR_INVALID_ARG;
    if (!aligned(x, in) || !aligned(packed, 16) || !aligned(scales_mma, 16) ||
        (fmt == FP4_NVFP4 && !aligned(global_scale, 4)))
        return FP4_ERR_ALIGN;
    if (!workspace || workspace_bytes < fp4_linear_workspace_bytes(rows, K))
        return FP4_ERR_WORKSPACE;
    if (!aligned(workspace, 16))
        return FP4_ERR_ALIGN;
    int dev = 0;
    const int sms = sm_count(dev);
    if (sms <= 0)
        return FP4_ERR_CUDA;
    const int parts = dtype == FP4_F32 ? 2 : 1;
    const Layout l = layout(rows, K, parts);
    CUtensorMap map;
    std::memset(&map, 0, sizeof(map));
    const fp4_status st = weight_map(packed, N, Kp, &map);
    if (st != FP4_OK)
        return st;
    fp4::LinearArgs a = {};
    a.scales = scales_mma;
    a.frags = static_cast<uint8_t *>(workspace);
    a.xs = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + l.frags);
    a.g = global_scale;
    a.y = y;
    a.rows = (int)rows;
    a.N = (int)N;
    a.parts = parts;
    a.stages = l.stages;
    a.tiles = (int)((Kp / group + 3) / 4);
    a.out_bf16 = out_dtype == FP4_BF16;
    a.status = status;
    const bool bf = dtype == FP4_BF16;
    const uint16_t *xb = static_cast<const uint16_t *>(x);
    const float *xf = static_cast<const float *>(x);
    if (fmt == FP4_NVFP4)
        return bf ? run_linear<uint16_t, true>(xb, rows, K, x_stride, map, a, l, sms, stream)
                  : run_linear<float, true>(xf, rows, K, x_stride, map, a, l, sms, stream);
    return bf ? run_linear<uint16_t, false>(xb, rows, K, x_stride, map, a, l, sms, stream)
              : run_linear<float, false>(xf, rows, K, x_stride, map, a, l, sms, stream);
}

} // extern "C"
