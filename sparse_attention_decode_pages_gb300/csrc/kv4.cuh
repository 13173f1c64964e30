// kv4.cuh -- the 4-bit paged cache's number format, shared by the kernels that
// write it (kv4.cu) and attend over it (attn4_decode.cu, attn4_verify.cu).
//
// A row of D channels is held in groups of 16: a scale s = e4m3(amax / (6 * 2^e))
// and sixteen e2m1 codes (sign, two exponent bits, one mantissa bit: 0, 0.5, 1,
// 1.5, 2, 3, 4, 6) of x / (s * 2^e).  code * s has at most 2 + 4 significant bits
// and lies between 2^-10 and 2688, so it is exact in fp16 and in bf16.
//
// Tile of one (physical page, KV head): [K | V], each ps * D / 2 bytes of codes
// (row-major, the even channel of a byte in its low bits) and ps * D / 16 scale
// bytes.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace spd {

__host__ __device__ constexpr int kv4_codes_bytes(int ps, int D) { return ps * D / 2; }
__host__ __device__ constexpr int kv4_half_bytes(int ps, int D) { return ps * D / 2 + ps * D / 16; }
__host__ __device__ constexpr int kv4_tile_bytes(int ps, int D) { return 2 * kv4_half_bytes(ps, D); }

// Two e2m1 codes (a byte, the low bits first) as an fp16 pair, exactly.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t* out) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
        : "r"(w));
}

// Two e4m3 bytes (the low one first) as an fp16 pair, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return h;
}

// v >= 0 rounded to the nearest e4m3 byte, saturating at 448.
__device__ __forceinline__ uint32_t to_e4m3(float v) {
    uint16_t h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(0.f), "f"(v));
    return h & 0xffu;
}

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    const uint32_t h = e4m3x2_to_f16(byte & 0xffu);
    return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}

// Eight floats as e2m1 codes, the first in the lowest bits: nearest, ties to the even code,
// saturating at 6.
__device__ __forceinline__ uint32_t to_e2m1x8(const float* y) {
    uint32_t codes;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(codes)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return codes;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// 2^e for an exponent of a normal float.
__host__ __device__ __forceinline__ float pow2f(int e) {
#ifdef __CUDA_ARCH__
    return __int_as_float((e + 127) << 23);
#else
    union {
        uint32_t u;
        float f;
    } v;
    v.u = (uint32_t)(e + 127) << 23;
    return v.f;
#endif
}

}  // namespace spd
