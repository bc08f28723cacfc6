// The FP4 latent cache's codec on the device: E2M1 codes (4 bits: 0, .5, 1, 1.5, 2, 3,
// 4, 6 and their negatives) with one E4M3 scale per token and 16-channel block, under
// one power of two for the whole cache (see dsa_quantize_latent_fp4 in dsa.h):
//
//   value[c] = 2^cache_exp * E4M3(scale[c / 16]) * E2M1(code[c])
//
// Shared by the cache encoder, the decode-time append and the attention kernels.
//
// A code times a scale has a 6-bit significand and lies in [2^-10, 2688] or is 0, so
// it is exact in f16 (and in bf16 under any cache_exp of the allowed range).
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace dsa {

constexpr int kF4Block = 16;     // channels under one scale
constexpr int kF4MaxExp = 64;    // |cache_exp| bound
constexpr float kF4ScaleMax = 448.f;

// 2^e for |e| <= 126.
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Two E4M3 bytes (low byte first) as packed f16, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((unsigned short)(two & 0xffffu)));
    return h2;
}

// Four bytes of E2M1 pairs (low nibble first) as four packed f16 pairs, exact.
__device__ __forceinline__ void e2m1x8_to_f16x8(uint32_t (&h)[4], uint32_t c) {
    asm("{\n.reg .b8 b0, b1, b2, b3;\n"
        "mov.b32 {b0, b1, b2, b3}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(c));
}
__device__ __forceinline__ uint32_t hmul2_u32(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Eight channels of one block: codes c times the scale pair s2 (the scale twice), f16.
__device__ __forceinline__ uint4 fp4_decode8(uint32_t c, uint32_t s2) {
    uint32_t h[4];
    e2m1x8_to_f16x8(h, c);
    return make_uint4(hmul2_u32(h[0], s2), hmul2_u32(h[1], s2), hmul2_u32(h[2], s2),
                      hmul2_u32(h[3], s2));
}

// One 16-channel block: bf16 values v (32 bytes) -> 8 bytes of codes and the scale byte.
//
// scale = E4M3 (nearest, ties to even, saturating) of amax * 2^-cache_exp / 6; codes =
// E2M1 (nearest, ties to even, saturating) of x * 2^-cache_exp / scale, sign kept. A
// zero scale gives codes 0; a block holding a NaN gets scale NaN (0x7F) and codes 0.
//
// The codes come from x times the rounded reciprocal of the scale, not from a division:
// the product is within 2^-22 of the quotient q, and rounding it to f16 first makes it
// the quotient's own f16 value wherever a code's rounding is decided. An E2M1 midpoint
// times the scale has at most 7 significant bits and x has 8, so q is either a midpoint
// exactly (then the f16 rounding restores it) or at least 2^-8 away from it (then an
// f16 rounding, 2^-11, does not cross it).
__device__ __forceinline__ uint2 fp4_encode16(const uint4 (&v)[2], int cache_exp, uint8_t* scale) {
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    uint32_t m2 = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m2 = __vmaxu2(m2, w[i] & 0x7fff7fffu);
    const uint32_t mb = max(m2 & 0xffffu, m2 >> 16);  // amax as bf16 bits; NaN above 0x7f80
    if (mb > 0x7f80u) {
        *scale = 0x7f;
        return make_uint2(0u, 0u);
    }
    const float down = pow2f(-cache_exp);
    const float want = __fdiv_rn(__uint_as_float(mb << 16) * down, 6.f);
    unsigned short sb;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(sb) : "f"(0.f), "f"(want));
    *scale = (uint8_t)sb;
    if ((sb & 0xff) == 0) return make_uint2(0u, 0u);
    const uint32_t s2 = e4m3x2_to_f16x2(sb);
    const float s = __half2float(__ushort_as_half((unsigned short)(s2 & 0xffffu)));
    const float k = __frcp_rn(s) * down;
    uint32_t out[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t r = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t u = w[4 * j + i];
            const __half2 h = __floats2half2_rn(bf16_lo(u) * k, bf16_hi(u) * k);
            const float2 q = __half22float2(h);
            uint32_t byte;
            asm("{\n.reg .b8 t;\ncvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\ncvt.u32.u8 %0, t;\n}\n"
                : "=r"(byte)
                : "f"(q.y), "f"(q.x));
            r |= byte << (8 * i);
        }
        out[j] = r;
    }
    return make_uint2(out[0], out[1]);
}

}  // namespace dsa
