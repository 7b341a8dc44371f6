// ra_rows.cuh -- rows of dense tensors and of the paged cache, eight values to a
// lane: loads, stores, and the 8- and 4-bit codes with their powers of two.
#pragma once

#include <cuda_fp16.h>

#include "ra_paged.cuh"

namespace ra {

// Eight consecutive values in registers.
struct Eight {
    float x[8];
};

// The same as loaded: fewer registers while they wait.
template <typename T>
struct Raw {
    uint4 w[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw<T> load8(const T *p)
{
    Raw<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = reinterpret_cast<const uint4 *>(p)[i];
    return r;
}

__device__ __forceinline__ Eight widen(const Raw<__nv_bfloat16> &w)
{
    const uint32_t a[4] = {w.w[0].x, w.w[0].y, w.w[0].z, w.w[0].w};
    Eight r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.x[2 * i] = __uint_as_float(a[i] << 16);
        r.x[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
    return r;
}

__device__ __forceinline__ Eight widen(const Raw<float> &w)
{
    const uint32_t a[8] = {w.w[0].x, w.w[0].y, w.w[0].z, w.w[0].w, w.w[1].x, w.w[1].y, w.w[1].z, w.w[1].w};
    Eight r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.x[i] = __uint_as_float(a[i]);
    return r;
}

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const Eight &r)
{
    uint4 w;
    w.x = pack_bf16x2(r.x[0], r.x[1]);
    w.y = pack_bf16x2(r.x[2], r.x[3]);
    w.z = pack_bf16x2(r.x[4], r.x[5]);
    w.w = pack_bf16x2(r.x[6], r.x[7]);
    *reinterpret_cast<uint4 *>(p) = w;
}

__device__ __forceinline__ void store8(float *p, const Eight &r)
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(r.x[0], r.x[1], r.x[2], r.x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(r.x[4], r.x[5], r.x[6], r.x[7]);
}

// codes of four values, the first in the lowest byte
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// codes of eight values, the first in the lowest four bits
__device__ __forceinline__ uint32_t e2m1x8(const float *x)
{
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

// Eight e2m1 codes as four pairs of halves.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t *h)
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// The scale byte of a row from the bits of its largest magnitude: frexp's
// exponent less 9, or less 8 above 1.75 * 2^n; 255 when it is not finite.
__device__ __forceinline__ uint32_t row_exp(uint32_t amax_bits)
{
    if (amax_bits >= 0x7f800000u) return 255u;
    const int e = (int)(amax_bits >> 23) - 135 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)(max(e, -110) + 127);
}

// The same for a block of e2m1 codes, at most 6 = 1.5 * 2^2.
__device__ __forceinline__ uint32_t block_exp(uint32_t amax_bits)
{
    if (amax_bits >= 0x7f800000u) return 255u;
    const int e = (int)(amax_bits >> 23) - 129 + ((amax_bits & 0x7fffffu) > 0x400000u ? 1 : 0);
    return (uint32_t)(max(e, -110) + 127);
}

// 2^-(e - 127) of a stored scale byte e: its exponent field is 254 - e, in [7, 237]
__device__ __forceinline__ float exp_byte_inverse(uint32_t e) { return __uint_as_float((254u - e) << 23); }

} // namespace ra
