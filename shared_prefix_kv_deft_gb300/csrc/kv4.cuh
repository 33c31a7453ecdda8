// kv4.cuh -- the 4-bit paged cache's format and its conversions.
//
// 16 consecutive elements of a token's head form a block with one scale s, an
// 8-bit float (4 exponent, 3 mantissa bits, largest 448); an element c is a
// 4-bit float (sign, 2 exponent bits, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3,
// 4, 6) and stands for c * s * g, with one fp32 g for K and one for V.  c has
// two significant bits and s four, so c * s has at most six: it is exact in
// fp16 (from 2^-10 to 2688) and in bf16.
//
// A page of one head is 9 * head_dim bytes: the elements, [16
// tokens][head_dim / 2] bytes with the even element in the low half, then
// the scales, [16 tokens][head_dim / 16].  Pages are multiples of 16 bytes
// long, so that one is one bulk copy.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "deft_internal.h"

namespace deft {
namespace kv4 {

constexpr int kBlock = 16;

template <int D>
struct Page {
    static constexpr int kRow = D / 2;                  // bytes of a token's elements
    static constexpr int kScaleRow = D / kBlock;        // ... of its scales
    static constexpr int kScales = kPageSize * kRow;    // where the scales begin
    static constexpr int kBytes = kScales + kPageSize * kScaleRow;
};
inline int64_t page_bytes(int32_t head_dim) { return (int64_t)kPageSize * (head_dim / 2 + head_dim / kBlock); }

// The four bytes of w, two elements each, as pairs of fp16 (exact).
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Two scale bytes (the low 16 bits) as a pair of fp16 (exact).
__device__ __forceinline__ uint32_t scales2(uint32_t two)
{
    uint32_t h;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(two));
    return h;
}

// One scale byte's value.
__device__ __forceinline__ float scale_value(uint32_t s)
{
    const uint32_t h = scales2(s);
    return __low2float(*reinterpret_cast<const __half2 *>(&h));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The larger magnitude, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A block's scale for its largest magnitude: amax / (6 g) to the nearest
// 8-bit float, at most 448 (NaN stays NaN).
__device__ __forceinline__ uint32_t scale_of(float amax, float six_g)
{
    uint16_t r;
    const float s = __fdiv_rn(amax, six_g);
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(s));
    return r & 0xffu;
}

// Eight elements as codes: x / sg (sg: the block's scale times g), rounded
// to the nearest, halfway to the even code, at most 6 in magnitude.  The
// codes are those of the correctly rounded quotient (tested for every bf16 x
// next to every border), by Markstein's division (IBM Journal of Research and
// Development 34, 1990): the product y0 = x * (1 / sg), its residual y0 * sg -
// x by one fused multiply-add, and one more that takes the residual over sg
// from y0.  A bf16 x over an 8-bit scale often lies exactly
// between two codes, where y0 alone is an ulp to either side.
__device__ __forceinline__ uint32_t pack8(const float (&x)[8], float amax, float sg)
{
    const float r = sg > 0.f ? __frcp_rn(sg) : 0.f;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = x[i];
    // Past the largest scale (or infinite): kept in range of the step below.
    if (sg > 0.f && amax > 8.f * sg) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = fminf(fmaxf(v[i], -8.f * sg), 8.f * sg);
    }
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float y[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float y0 = __fmul_rn(v[2 * i + k], r);
            y[k] = __fmaf_rn(-__fmaf_rn(y0, sg, -v[2 * i + k]), r, y0);   // (in signs that keep -0)
        }
        asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tmov.b32 %0, {t, 0, 0, 0};\n\t}"
            : "=r"(b[i])
            : "f"(y[1]), "f"(y[0]));
    }
    return b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24;
}

// ---- of the steps ----
// A weight is held as 2^kLift * 2^(s - m), m a maximum that is raised when a
// logit passes it by more than kUp (both in base 2).
constexpr float kUp = 4.f, kLift = 11.f;

__device__ __forceinline__ float nan() { return __int_as_float(0x7fffffff); }

__device__ __forceinline__ uint32_t f16x2(float lo, float hi)
{
    const __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ float pow2(int e)   // -126 <= e <= 127
{
    return __int_as_float((127 + e) << 23);
}

}  // namespace kv4
}  // namespace deft
