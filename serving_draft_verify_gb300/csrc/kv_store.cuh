// What a cache holds of a value, shared by the calls that write and read one: pieces of eight
// elements, 8 bits (e4m3), 4 bits (e2m1 with a scale for each block of 16).
//
// 4 bits.  A block of 16 adjacent elements of a head's row has one scale s (e4m3), the head one
// scale g (float32); element x is held as c in {0, 1/2, 1, 3/2, 2, 3, 4, 6} with a sign and stands for
// c s g:
//   s = e4m3(max |x| r), r = 1 / (6 g);   c = e2m1(x i), i = 1 / (s g),
// every operation in float32, rounded to nearest (reciprocals correctly rounded, halves to the even
// code), beyond the largest value the largest.  c = 0 where i is not finite (s = 0); a block with a
// NaN has s = NaN, so that it stays one.  c s has six significant bits and lies within 2^-10 and 2688: it
// is exact in f16.
//
// A page of one head: `page` rows of D / 2 bytes (element 2i in the low half of byte i), behind them
// `page` rows of the scales, each row's bytes rounded up to 4; the whole rounded up to 16 bytes.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace dspark {

struct Page4 {
    int code, scale, codes, whole;              // bytes: a row's codes, its scales, all codes, the whole page
};
__host__ __device__ inline Page4 page4_of(int page, int D) {
    Page4 g;
    g.code = D / 2;
    g.scale = (D / 16 + 3) / 4 * 4;
    g.codes = page * g.code;
    g.whole = (g.codes + page * g.scale + 15) / 16 * 16;
    return g;
}

// Eight floats as eight codes, the first in the lowest bits; eight codes as f16 pairs (exact).
__device__ __forceinline__ uint32_t e2m1x8(const float* x) {
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return w;
}
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t* h) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
// Two e4m3 bytes as two f16 (exact), four as four, and one as a float.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
    return r;
}
__device__ __forceinline__ void e4m3x4_f16(uint32_t four, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
}
__device__ __forceinline__ float f16lo(uint32_t w) {
    float f;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(w));
    return f;
}
__device__ __forceinline__ float f16hi(uint32_t w) {
    float f;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(f) : "r"(w));
    return f;
}
__device__ __forceinline__ float e4m3_float(uint32_t byte) { return f16lo(e4m3x2_f16x2(byte)); }

// The largest magnitude of eight, a NaN if there is one.
__device__ __forceinline__ float magnitude3(float x, float y, float z) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}
__device__ __forceinline__ float magnitude8(const float* x) {
    return magnitude3(magnitude3(x[0], x[1], x[2]), magnitude3(x[3], x[4], x[5]), magnitude3(x[6], x[7], 0.f));
}
// A block's scale from its largest magnitude; r = 1 / (6 g).
struct Scale4 {
    uint32_t byte;
    float inv;                                  // 0: the codes are 0; NaN where the block has one
};
__device__ __forceinline__ Scale4 scale4(float big, float g, float r) {
    Scale4 s;
    s.byte = big != big ? 0x7Fu : __nv_cvt_float_to_fp8(big * r, __NV_SATFINITE, __NV_E4M3);
    s.inv = __frcp_rn(e4m3_float(s.byte) * g);
    if (fabsf(s.inv) == __uint_as_float(0x7f800000u)) s.inv = 0.f;
    return s;
}
__device__ __forceinline__ uint32_t codes8(const float* x, float inv) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] * inv;
    const uint32_t w = e2m1x8(y);
    return inv != inv ? 0u : w;
}

template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
    uint4 w;
    __device__ void load(const void* p) { w = __ldg(static_cast<const uint4*>(p)); }
    __device__ void store(void* p) const { *static_cast<uint4*>(p) = w; }
    __device__ void floats(float* f) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16lo(u[i]);
            f[2 * i + 1] = bf16hi(u[i]);
        }
    }
};
template <>
struct Eight<float> {
    float4 a, b;
    __device__ void load(const void* p) {
        a = __ldg(static_cast<const float4*>(p));
        b = __ldg(static_cast<const float4*>(p) + 1);
    }
    __device__ void store(void* p) const {
        static_cast<float4*>(p)[0] = a;
        static_cast<float4*>(p)[1] = b;
    }
    __device__ void floats(float* f) const {
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
        f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
};

// How far to either side of x * (1 / s) a number that rounds to the bytes of x / s is looked for.  The
// two are within 2^-22 of each other; where s is a power of two they are the same, and 2^-30 is
// gone in the sum's rounding (but makes an infinite x differ, which then takes the quotient proper).
__device__ __forceinline__ float margin_of(float s) {
    const uint32_t u = __float_as_uint(s) & 0x7FFFFFFFu;
    return (u & 0x007FFFFFu) == 0 && u >= 0x00800000u && u < 0x7F800000u ? 0x1p-30f : 0x1p-21f;
}
// Two stored bytes of x / s.  The quotient proper costs nine instructions an element; where the numbers
// `margin` to either side of x * (1 / s) round to the same bytes so does the quotient (the rounding
// is monotonic).  One element in 100,000 does not end there where the quotients are spread evenly, but
// one in 16 where they keep bf16's few bits and are ties: 16384 rows at scale 1 took 33 us, without
// the margin 23; at 0.0125 (1 / 80) it is 28.
__device__ __forceinline__ uint32_t stored(float x, float y, float s, float inv, float margin) {
    const float a = x * inv, b = y * inv;
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(fmaf(a, -margin, a), fmaf(b, -margin, b)), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(fmaf(a, margin, a), fmaf(b, margin, b)), __NV_SATFINITE, __NV_E4M3);
    if (lo == hi && inv < 3e38f && inv > 1e-37f) return lo;
    return __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x, s), __fdiv_rn(y, s)), __NV_SATFINITE, __NV_E4M3);
}

}  // namespace dspark
