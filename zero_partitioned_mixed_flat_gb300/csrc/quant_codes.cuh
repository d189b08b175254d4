// quant_codes.cuh -- the arithmetic of the 8-bit codes (device only), shared by
// the quantized gather (quant.cu) and the quantized norm output (norm.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace zk {
namespace {

// two floats -> two lp values in one packed conversion (each rounded to
// nearest, ties to even, as a separate conversion would)
template <bool BF16>
__device__ __forceinline__ uint32_t to_lp2_packed(float a, float b) {
    if constexpr (BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// byte k of w (a signed code) as an exact float without the conversion unit:
// w ^ 0x80808080 holds code + 128 in each byte; one byte permute places it in
// the low mantissa bits of 2^23, and subtracting 2^23 + 128 is exact.
__device__ __forceinline__ float code_to_float(uint32_t biased, int k) {
    const uint32_t bits = __byte_perm(biased, 0x4B000000u, 0x7540u + (uint32_t)k);
    return __fsub_rn(__uint_as_float(bits), 8388736.0f);
}

// The code of x: the nearest-even integer of the correctly rounded quotient
// x / scale, clamped to +-127, as a byte (the division, for the rare elements
// that the fast path below leaves to it).
__device__ __forceinline__ uint32_t code_by_division(float x, float scale) {
    if (!(scale > 0.0f)) return 0u;
    int c = __float2int_rn(__fdiv_rn(x, scale));
    c = c > 127 ? 127 : (c < -127 ? -127 : c);
    return (uint32_t)c & 0xffu;
}

// Adding 1.5 * 2^23 to a float q with |q| < 2^22 leaves the nearest-even
// integer k of q in the low mantissa bits (the adder rounds to nearest even,
// and 1.5 * 2^23 is even), so the low byte of the sum is k as a signed byte
// and subtracting the constant back gives k exactly.
constexpr float kRoundMagic = 12582912.0f;

// hardware reciprocal approximation (within one ulp of 1/x for normal x)
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// K codes of one thread's elements (K a multiple of 4), packed 4 per word
// (byte k = element k).
// Fast path, with p = x * rcp the exact product (rcp within one ulp of
// 1/scale, so p lies within 2^-23 |x/scale| <= 1.6e-5 of the exact quotient):
// one fused multiply-add rounds p to its nearest-even integer k (through the
// 1.5 * 2^23 addition) and another gives d = p - k rounded once.  When every
// |d| < 1/2 - 2^-13, the correctly rounded quotient RN(x / scale) (within
// 7.6e-6 of the exact one) is farther than 9e-5 from a half-integer and rounds
// to the same k (and |k| <= 127 needs no clamp).  Otherwise (rare: ties, a
// NaN element), and for a zero, subnormal-small, huge or non-finite scale,
// every element is divided.
template <int K>
__device__ __forceinline__ void quant_codes(const float v[K], float scale, uint32_t packed[K / 4]) {
    bool divide = !(scale >= 0x1p-100f && scale <= 0x1p+100f);
    if (!divide) {
        const float rcp = rcp_approx(scale);
        uint32_t t[K];
        bool near = false;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float r = __fmaf_rn(v[k], rcp, kRoundMagic);
            const float d = __fmaf_rn(v[k], rcp, -__fsub_rn(r, kRoundMagic));
            near |= !(fabsf(d) < 0.5f - 0x1p-13f);
            t[k] = __float_as_uint(r);
        }
#pragma unroll
        for (int w = 0; w < K / 4; ++w)
            packed[w] = __byte_perm(__byte_perm(t[4 * w], t[4 * w + 1], 0x0040u),
                                    __byte_perm(t[4 * w + 2], t[4 * w + 3], 0x0040u), 0x5410u);
        divide = near;
    }
    if (divide) {
#pragma unroll
        for (int w = 0; w < K / 4; ++w) packed[w] = 0u;
#pragma unroll
        for (int k = 0; k < K; ++k) packed[k >> 2] |= code_by_division(v[k], scale) << (8 * (k & 3));
    }
}

// scale = amax / 127 correctly rounded, without the division routine for the
// usual range: Markstein's correction step (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", IBM J. Res.
// Dev. 34(1), 1990): with y = RN(1/127) and q0 = RN(amax * y), the remainder
// r = amax - 127 q0 is exact in one fused multiply-add, and q1 = RN(q0 + r y)
// is the correctly rounded quotient.  The block maximum is always an lp value,
// and the test suite checks q1 against the IEEE division for every positive
// finite fp16 and bf16 value in [2^-90, 2^100]; outside that range (and for an
// infinite maximum) the division routine is used.
__device__ __forceinline__ float scale_of_amax(float amax) {
    if (!(amax >= 0x1p-90f && amax <= 0x1p+100f)) return __fdiv_rn(amax, 127.0f);
    constexpr float y = 1.0f / 127.0f;
    const float q0 = __fmul_rn(amax, y);
    const float r = __fmaf_rn(-q0, 127.0f, amax);
    return __fmaf_rn(r, y, q0);
}

// ---- fp8 (OCP E4M3) variant: a power-of-two block scale 2^e with
// e = floor(log2 amax) - 7 clamped to [-126, 120] (120 for an infinite amax),
// so amax / 2^e lies in [128, 256): code = E4M3(x * 2^-e), nearest even,
// finite overflow and infinities saturated to +-448.

// two floats -> two E4M3 codes, a in the low byte (one conversion instruction)
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// two E4M3 codes (low byte first) -> two exact floats
__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)two));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// the block scale exponent from amax's bits (amax >= 0, not NaN)
__device__ __forceinline__ int fp8_scale_exponent(float amax) {
    const int biased = (int)(__float_as_uint(amax) >> 23);
    int e = biased == 0 ? -126 : biased - 127 - 7;
    e = e < -126 ? -126 : e;
    return e > 120 ? 120 : e;
}

template <int K>
__device__ __forceinline__ void quant_codes_fp8(const float v[K], float amax, float &scale,
                                                uint32_t packed[K / 4]) {
    if (amax == 0.0f) {  // an all-zero block: scale 0 and codes 0 (also for -0)
        scale = 0.0f;
#pragma unroll
        for (int w = 0; w < K / 4; ++w) packed[w] = 0u;
        return;
    }
    const int e = fp8_scale_exponent(amax);
    scale = __uint_as_float((uint32_t)(e + 127) << 23);
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int w = 0; w < K / 4; ++w) {
        const uint32_t lo = to_e4m3x2(__fmul_rn(v[4 * w], inv), __fmul_rn(v[4 * w + 1], inv));
        const uint32_t hi = to_e4m3x2(__fmul_rn(v[4 * w + 2], inv), __fmul_rn(v[4 * w + 3], inv));
        packed[w] = lo | (hi << 16);
    }
}

template <bool BF16>
__device__ __forceinline__ void from_lp4(uint2 raw, float v[4]) {
    const uint32_t w[2] = {raw.x, raw.y};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if constexpr (BF16) {
            v[2 * k] = __uint_as_float(w[k] << 16);
            v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        } else {
            const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
            v[2 * k] = t.x;
            v[2 * k + 1] = t.y;
        }
    }
}

}  // namespace
}  // namespace zk
