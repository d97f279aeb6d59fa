// fp4_kv_args.cuh -- the checks of an fp4_kv_cache that its entry points
// share, and the cache as their kernels take it.
#pragma once

#include <cstdint>

#include "fp4.h"
#include "fp4_kvcache.cuh"
#include "fp4_launch.cuh"

namespace fp4_kv {
namespace {

using fp4_launch::aligned;

inline fp4_status check_cache(const fp4_kv_cache *c)
{
    if (!c || (c->format != FP4_NVFP4 && c->format != FP4_MXFP4) || c->heads < 1 || c->head_dim < 1 ||
        c->page_size < 1 || c->num_pages < 1)
        return FP4_ERR_INVALID_ARG;
    if (c->page_size % 16 || c->head_dim % 32 || c->head_dim > 1024 || (int64_t)c->heads * c->head_dim > (1 << 20) ||
        c->num_pages > ((int64_t)1 << 40) / c->page_size)
        return FP4_ERR_SHAPE;
    if (!c->k_packed || !c->k_scales || !c->v_packed || !c->v_scales)
        return FP4_ERR_INVALID_ARG;
    if (c->format == FP4_NVFP4 && (!c->k_global_scale || !c->v_global_scale))
        return FP4_ERR_INVALID_ARG;
    if (!aligned(c->k_packed, 16) || !aligned(c->v_packed, 16) || !aligned(c->k_scales, 16) ||
        !aligned(c->v_scales, 16))
        return FP4_ERR_ALIGN;
    if (c->format == FP4_NVFP4 && (!aligned(c->k_global_scale, 4) || !aligned(c->v_global_scale, 4)))
        return FP4_ERR_ALIGN;
    return FP4_OK;
}

inline fp4::KvCache device_cache(const fp4_kv_cache &c)
{
    fp4::KvCache d = {};
    d.packed[0] = c.k_packed;
    d.packed[1] = c.v_packed;
    d.scales[0] = c.k_scales;
    d.scales[1] = c.v_scales;
    d.g[0] = c.k_global_scale;
    d.g[1] = c.v_global_scale;
    d.slots = c.num_pages * c.page_size;
    d.page_magic = ~(uint64_t)0 / (uint64_t)c.page_size + 1;
    d.heads = c.heads;
    d.blocks = c.head_dim / (c.format == FP4_NVFP4 ? 16 : 32);
    d.page = c.page_size;
    const int64_t granules = d.slots / 16, per = c.page_size / 16;
    d.narrow = d.slots < ((int64_t)1 << 31) / (c.heads * (c.head_dim / 16)) && granules < ((int64_t)1 << 32) / per;
    d.magic32 = per > 1 ? ~(uint32_t)0 / (uint32_t)per + 1 : 0;
    return d;
}

} // namespace
} // namespace fp4_kv
