// fp4_mma.cuh -- what the kernels that decode FP4 codes to fp16 for mma.sync
// share: the decoding, the pair arithmetic and the instruction itself.
#pragma once

#include <cstdint>

#include "fp4_codec.cuh"

namespace fp4 {

__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The pair a times one half of b (the high one if `high`).
__device__ __forceinline__ uint32_t f16x2_mul_half(uint32_t a, uint32_t b, bool high)
{
    uint32_t r;
    if (high)
        asm("{\n\t.reg .b16 l, h;\n\t.reg .b32 s;\n\tmov.b32 {l, h}, %2;\n\tmov.b32 s, {h, h};\n\tmul.rn.f16x2 %0, %1, s;\n\t}"
            : "=r"(r)
            : "r"(a), "r"(b));
    else
        asm("{\n\t.reg .b16 l, h;\n\t.reg .b32 s;\n\tmov.b32 {l, h}, %2;\n\tmov.b32 s, {l, l};\n\tmul.rn.f16x2 %0, %1, s;\n\t}"
            : "=r"(r)
            : "r"(a), "r"(b));
    return r;
}

// (lo, hi) -> f16x2, round to nearest even.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// The two E4M3 bytes in the low half of v as an f16 pair.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v)
{
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(v));
    return r;
}

// The eight codes of a word as f16 pairs (byte j of the word in h[j]).
__device__ __forceinline__ void e2m1_word(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n\t"
        ".reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t"
        "}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// 2^-d as f16 bits, d >= 0: normal to d = 14, subnormal to 24, then 0.
__device__ __forceinline__ uint32_t f16_exp2_neg(int d)
{
    return d <= 14 ? (uint32_t)(15 - d) << 10 : (d <= 24 ? 1u << (24 - d) : 0u);
}

} // namespace fp4
