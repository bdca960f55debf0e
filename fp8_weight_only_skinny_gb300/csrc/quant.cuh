// quant.cuh -- the rounding steps shared by everything that writes E2M1 / E4M3
// codes: the weight quantizers (quant.cu) and the key/value cache
// (kv4_append.cu).
#pragma once
#include <cstdint>
#include <cuda_fp16.h>

namespace sk {

// Two FP32 values -> two E4M3 codes, nearest-even, saturating; lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2_rn(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// Two FP32 values -> two E2M1 codes, nearest-even, saturating; lo in the low nibble.
__device__ __forceinline__ uint32_t e2m1x2_rn(float lo, float hi) {
    uint32_t d;
    asm("{ .reg .b8 t; cvt.rn.satfinite.e2m1x2.f32 t, %1, %2; cvt.u32.u8 %0, t; }" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// An E4M3 code -> its value (exact in FP16, then FP32).
__device__ __forceinline__ float e4m3_value(uint32_t code) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(uint16_t(code & 0xFFu)));
    return __half2float(__ushort_as_half(uint16_t(h2 & 0xFFFFu)));
}

// Codes of a quotient pair (x0 / d, x1 / d): each code is defined from the
// binary32 quotient rounded to nearest-even, q = RN(x / d).  The kernels form
// p = RN(x * r) with r = RN(1 / d), which is faster than the division and in
// all but a few cases rounds to the same code.  The two roundings each add a
// relative error of at most 2^-24, so |p - x / d| <= (2^-23 + 2^-48) |x / d|
// and q lies within 3 units in the last place of x / d's binade from p: within
// 6 steps of p's bit pattern (3, or up to twice that where p and q sit in
// neighbouring binades).  Every rounding boundary of the code format (a
// midpoint between neighbouring values) has a binary32 pattern whose low bits
// are zero: 19 bits for E4M3, subnormal midpoints included (MASK = 2^19 - 1),
// 21 for E2M1 (MASK = 2^21 - 1).  Rounding to a code is monotone in the
// magnitude, so p and q can get different codes only when a boundary lies
// between them, hence within 6 steps of p; p's code is taken unless p's pattern
// is within 8 steps of a multiple of MASK + 1, and the pair is divided then.
// A zero p (x = 0) is such a multiple and is divided too.
template <uint32_t MASK, typename Cvt>
__device__ __forceinline__ uint32_t quotient_codes(float x0, float x1, float d, float r, Cvt cvt) {
    const float p0 = __fmul_rn(x0, r), p1 = __fmul_rn(x1, r);
    const uint32_t b0 = __float_as_uint(p0), b1 = __float_as_uint(p1);
    if (((b0 + 8u) & MASK) < 16u || ((b1 + 8u) & MASK) < 16u) return cvt(__fdiv_rn(x0, d), __fdiv_rn(x1, d));
    return cvt(p0, p1);
}

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}

// One 16-element NVFP4 block (two 16-byte words of FP16) under the tensor scale
// G: its E4M3 scale code and its eight code bytes.
__device__ __forceinline__ uint32_t encode_block(const uint4 &v0, const uint4 &v1, float G, uint2 &cw) {
    float f[16];
    {
        float t[8];
        unpack8(v0, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = t[i];
        unpack8(v1, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[8 + i] = t[i];
    }
    float bmax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) bmax = fmaxf(bmax, fabsf(f[i]));
    const uint32_t sc = e4m3x2_rn(__fdiv_rn(__fdiv_rn(bmax, 6.f), G), 0.f) & 0xFFu;
    const float S = e4m3_value(sc);
    uint32_t out[2] = {0u, 0u};
    if (S == 0.f) {
        // The scale underflowed: every code is a zero carrying the input's sign.
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (__float_as_uint(f[i]) >> 31) out[i >> 3] |= 0x8u << (4 * (i & 7));
    } else {
        const float denom = __fmul_rn(S, G);
        const float rd = __frcp_rn(denom);
#pragma unroll
        for (int i = 0; i < 16; i += 2)
            out[i >> 3] |= quotient_codes<0x1FFFFFu>(f[i], f[i + 1], denom, rd, e2m1x2_rn) << (4 * (i & 7));
    }
    cw = make_uint2(out[0], out[1]);
    return sc;
}

}  // namespace sk
