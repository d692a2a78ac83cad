// Device helpers of the 4-bit operands: E2M1 codes, E8M0 and E4M3 block scales, in
// the conversions that the hardware has for them.
#pragma once
#include "ll_device.cuh"
#include "rollout_internal.h"

namespace ll {

// The codes of eight values, the first in the lowest half byte.  To nearest, ties to the even
// code, 6 at most in magnitude.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}
// The values of eight codes.
__device__ __forceinline__ void e2m1_values(uint32_t codes, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

constexpr uint32_t kScaleNanMx = 0xffu, kScaleNanNv = 0x7fu;

// E4M3 of (lo, hi) in the low and high byte, to nearest even, 448 at most.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(byte)));
    return __half2float(__ushort_as_half(static_cast<uint16_t>(h & 0xffffu)));
}
// 2^(byte - 127); 255 is NaN.
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
    const uint32_t bits = byte == 0 ? 0x00400000u : byte == 255u ? 0x7fc00000u : byte << 23;
    return __uint_as_float(bits);
}

// The product of two matrices' scales as g * two, `two` a power of 2: 1 where the product lies
// within 2^-100 .. 2^100.  A sum of products is 0 or 2^-20 to 2^54 in size: times `two` and then g
// it is beyond FP32's range, or below it, only where the exact result is.
struct ScaleProduct {
    float g, two;
};
__device__ __forceinline__ ScaleProduct scale_product(float h, float w) {
    int eh, ew;
    const float m = frexpf(h, &eh) * frexpf(w, &ew);
    const int e = eh + ew, near = min(max(e, -100), 100);
    return {ldexpf(m, near), ldexpf(1.f, min(max(e - near, -126), 127))};
}

// Byte of block scale `b` of row r.
__device__ __forceinline__ int64_t scale_at(int64_t r, int64_t b, int64_t k_tiles) {
    return ((r / kFp4TileRows) * k_tiles + b / kFp4TileBlocks) * kFp4TileBytes + (r % 32) * 16 +
           (r % kFp4TileRows) / 32 * 4 + b % kFp4TileBlocks;
}

}  // namespace ll
