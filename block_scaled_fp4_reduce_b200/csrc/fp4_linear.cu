// fp4_linear.cu -- entry points of include/fp4.h for the product of a few
// rows of activations with an FP4 weight: argument checks and the launches.
#include <climits>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include <cuda.h>
#include <cuda_runtime.h>

#include "fp4.h"
#include "fp4_launch.cuh"
#include "fp4_linear.cuh"

namespace {

using namespace fp4_launch;

// 2-D tensor map of a row-major matrix: boxes of `box_cols` elements (64 or 128
// bytes, the swizzle's span) x `box_rows` rows; zeros outside.
fp4_status matrix_map(CUtensorMapDataType type, int size, const void *p, int64_t rows, int64_t cols, int box_cols,
                      int box_rows, CUtensorMapSwizzle swizzle, CUtensorMap *map)
{
    EncodeTiled enc = encode_tiled();
    if (!enc)
        return FP4_ERR_CUDA;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(cols * size)};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(map, type, 2, const_cast<void *>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FP4_OK : FP4_ERR_CUDA;
}

// Workspace: the activations as fp16 rows [tiles * cols][Kpad], then an
// exponent for each of them and share of K.
struct Layout {
    int cols, chunks; // columns of a tile (activation rows x parts, whole sixteens)
    int64_t tiles, Kpad;
    size_t xh, bytes;
};

Layout layout(int64_t rows, int64_t K, int parts)
{
    Layout l;
    const int64_t all = rows * parts, most = fp4::kLinMaxCols;
    l.tiles = (all + most - 1) / most;
    if (l.tiles < 1)
        l.tiles = 1;
    const int64_t per = (rows + l.tiles - 1) / l.tiles; // rows of a tile, spread evenly
    l.cols = (int)((per * parts + 15) / 16 * 16);
    l.chunks = (int)((K + fp4::kLinChunk - 1) / fp4::kLinChunk);
    l.Kpad = (int64_t)l.chunks * fp4::kLinChunk;
    l.xh = (size_t)(l.tiles * l.cols * l.Kpad) * 2;
    l.bytes = l.xh + (size_t)(l.tiles * l.cols) * fp4::kLinMaxSplits * sizeof(int32_t);
    return l;
}

// Stages of the ring: two CTAs share an SM up to kLinSharedCols columns,
// beyond that one CTA has the SM for itself.  fused: the chunks whose
// activations lie beside the ring, 0 where they come packed.
int pick_stages(int cols, int fused, size_t &smem)
{
    const int room = cols <= fp4::kLinSharedCols ? 112 * 1024 : 224 * 1024;
    const int fixed = 1024 + fp4::lin_landing_bytes(cols) + fused * cols * fp4::kLinChunk * 2;
    const int stage = fp4::lin_stage_bytes(cols, fused > 0);
    int s = (room - fixed) / stage;
    if (s > fp4::kLinMaxStages)
        s = fp4::kLinMaxStages;
    smem = (size_t)s * stage + fixed;
    return s;
}

// CTAs of a cluster.  A CTA's time is its chunks and about kLinFixed more for
// its start and end; what counts is that times the rounds the grid takes.  Of
// one to eight CTAs this picks the fastest or one within 4 % of it (cold L2,
// one call between two events, us; 1 x 57344 x 14336: 122, 112, 118, 118, 130,
// 140, 174, 172, picked 3 as 115 to 118; 16 x 8192 x 8192: 33.8, 27.7, 23.6,
// 21.5, 25.7, .., picked 4; 64 x 4096 x 14336: 66.5, 48.1, 33.8, 29.7, 29.7,
// 27.7, 25.6, 25.6, picked 8).
int pick_splits(int64_t tiles, int chunks, int64_t slots)
{
    constexpr int kLinFixed = 6;
    int best = 1;
    int64_t cost = INT64_MAX;
    for (int s = 1; s <= fp4::kLinMaxSplits && s <= chunks; ++s) {
        const int64_t c = (tiles * s + slots - 1) / slots * ((chunks + s - 1) / s + kLinFixed);
        if (c < cost) {
            cost = c;
            best = s;
        }
    }
    return best;
}

template <bool kNv, typename T>
fp4_status launch_linear(const CUtensorMap &map_w, const CUtensorMap &map_x, fp4::LinearArgs a, int64_t mtiles,
                         int64_t bands, cudaStream_t stream)
{
    auto kernel = fp4::linear_kernel<kNv, T>;
    if (!smem_attr(kernel, 224 * 1024))
        return FP4_ERR_CUDA;
    a.most_share = a.share + (a.more > 0);
    a.own = (fp4::kLinRows + a.splits - 1) / a.splits;
    a.own_inv = (65536 + a.own - 1) / a.own;
    a.own_magic = (uint32_t)((0x100000000ull + a.own - 1) / a.own);
    cudaLaunchConfig_t cfg = {};
    a.stages = pick_stages(a.cols, std::is_void_v<T> ? 0 : a.most_share, cfg.dynamicSmemBytes);
    cfg.gridDim = dim3((unsigned)a.splits, (unsigned)mtiles, (unsigned)bands);
    cfg.blockDim = dim3(fp4::kLinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.splits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kernel, map_w, map_x, a) != cudaSuccess) {
        (void)cudaGetLastError();
        return FP4_ERR_CUDA;
    }
    return FP4_OK;
}

} // namespace

extern "C" {

size_t fp4_linear_workspace_bytes(int64_t rows, int64_t K)
{
    if (rows < 0 || K < 0 || rows >= (1 << 23) || K > INT_MAX - 1024)
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
    const int parts = dtype == FP4_F32 ? 2 : 1;
    if (rows >= (1 << 23) || K > INT_MAX - 1024 || N > (int64_t)65535 * fp4::kLinRows || // the grid's z, and its y
        rows * parts > (int64_t)65535 * fp4::kLinMaxCols)
        return FP4_ERR_SHAPE;
    const int64_t bands = (N + fp4::kLinRows - 1) / fp4::kLinRows;
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
    const Layout l = layout(rows, K, parts);
    CUtensorMap map_w, map_x;
    std::memset(&map_w, 0, sizeof(map_w));
    std::memset(&map_x, 0, sizeof(map_x));
    fp4_status st = matrix_map(CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, packed, N, Kp / 2, fp4::kLinChunk / 2, fp4::kLinRows,
                               CU_TENSOR_MAP_SWIZZLE_64B, &map_w);
    if (st != FP4_OK)
        return st;
    fp4::LinearArgs a = {};
    a.x = x;
    a.x_stride = x_stride;
    a.K = (int)K;
    a.scales = scales_mma;
    a.g = global_scale;
    a.y = y;
    a.rows = (int)rows;
    a.N = (int)N;
    a.parts = parts;
    a.cols = l.cols;
    a.chunks = l.chunks;
    a.tiles = (int)((Kp / group + 3) / 4);
    a.out_bf16 = out_dtype == FP4_BF16;
    a.accs = fp4::lin_accumulators(l.cols, out_dtype == FP4_F32);
    a.status = status;
    a.splits = pick_splits(bands * l.tiles, a.chunks, (int64_t)sms * (a.cols <= fp4::kLinSharedCols ? 2 : 1));
    a.share = a.chunks / a.splits;
    a.more = a.chunks % a.splits;
    const bool bf = dtype == FP4_BF16, nv = fmt == FP4_NVFP4;
    const int share = (a.chunks + a.splits - 1) / a.splits;
    if (rows <= fp4::kLinFusedRows && rows * share <= fp4::kLinFusedShare) {
        if (nv)
            return bf ? launch_linear<true, uint16_t>(map_w, map_x, a, l.tiles, bands, stream)
                      : launch_linear<true, float>(map_w, map_x, a, l.tiles, bands, stream);
        return bf ? launch_linear<false, uint16_t>(map_w, map_x, a, l.tiles, bands, stream)
                  : launch_linear<false, float>(map_w, map_x, a, l.tiles, bands, stream);
    }
    uint16_t *const xh = static_cast<uint16_t *>(workspace);
    int32_t *const xe = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(workspace) + l.xh);
    a.xe = xe;
    st = matrix_map(CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, xh, l.tiles * l.cols, l.Kpad, fp4::kLinChunk / 2, l.cols,
                    CU_TENSOR_MAP_SWIZZLE_128B, &map_x);
    if (st != FP4_OK)
        return st;
    const int per = l.cols / parts, Kpad = (int)l.Kpad;
    const dim3 grid((unsigned)(l.tiles * per), (unsigned)a.splits);
    st = bf ? launch_cfg(fp4::linear_pack_kernel<uint16_t>, grid, fp4::kThreads, 0, stream,
                         static_cast<const uint16_t *>(x), (int)rows, (int)K, x_stride, per, Kpad, a.share, a.more, xh, xe,
                         status)
            : launch_cfg(fp4::linear_pack_kernel<float>, grid, fp4::kThreads, 0, stream, static_cast<const float *>(x),
                         (int)rows, (int)K, x_stride, per, Kpad, a.share, a.more, xh, xe, status);
    if (st != FP4_OK)
        return st;
    return nv ? launch_linear<true, void>(map_w, map_x, a, l.tiles, bands, stream)
              : launch_linear<false, void>(map_w, map_x, a, l.tiles, bands, stream);
}

} // extern "C"
