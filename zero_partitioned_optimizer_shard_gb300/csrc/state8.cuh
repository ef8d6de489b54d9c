/*
 * state8.cuh -- the block-scaled 8-bit form of the optimizer states (include/zero.h, "8-bit
 * states"): codes, block exponents and the random bits of their rounding.
 *
 * A code c (7 bits of m, 8 of v) shifted left by 20 is a float with the code's exponent in
 * the low bits of the exponent field: 4 (m) or 5 (v) exponent bits over 3 mantissa bits,
 * and fp32's own subnormals serve as the code's (E = 0).  Multiplying by 2^112 (m) or 2^96
 * (v) puts the top exponent (15 or 31) at 1, multiplying by 2^(b-127) at the block's power
 * of two.  Both products are exact, so decoding rounds nothing.  Encoding runs backwards:
 * two multiplications by powers of two, then the 20 low bits are rounded away by adding r
 * in [0, 2^20) before the shift: r = 2^19 rounds to nearest, r uniform rounds up with a
 * probability equal to the fraction rounded away.  A carry out of the mantissa moves on to
 * the next exponent, as it should.  The second product may itself round in fp32's
 * subnormal range, 2^-20 of a code's spacing.
 *
 * The block's exponent b is that of its largest magnitude A with the mantissa rounded up
 * to 3 bits: A <= 1.875 * 2^(b-127), so rounding up never passes the largest code.
 */
#pragma once

#include "zero_internal.h"

namespace zero {
namespace {

constexpr uint32_t kMinExp = 27, kMaxExp = 253;  // 2^(b-127) and its reciprocal are normal
constexpr uint32_t kNearest = 1u << 19;
constexpr uint32_t kGolden = 0x9E3779B9u;
constexpr uint32_t kLcgMul = 1664525u, kLcgAdd = 1013904223u;

/* A bijection of 32-bit words that spreads every bit over the word: xor-shifts between
 * multiplications by odd constants (the leading fraction bits of sqrt 2 and sqrt 3). */
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t x)
{
    x ^= x >> 16;
    x *= 0x6A09E667u;
    x ^= x >> 15;
    x *= 0xBB67AE85u;
    return x ^ (x >> 16);
}

/* The key of step t's random bits. */
__host__ __device__ __forceinline__ uint32_t step_key(uint64_t seed, uint32_t t)
{
    return mix32(mix32((uint32_t)seed + t * kGolden) ^ (uint32_t)(seed >> 32));
}

/* The generator's k-th output is mul * s_0 + add. */
struct Jump {
    uint32_t mul, add;
};

__host__ __device__ constexpr Jump jump(int k)
{
    Jump j{1u, 0u};
    for (int i = 0; i < k; ++i) {
        j.mul *= kLcgMul;
        j.add = j.add * kLcgMul + kLcgAdd;
    }
    return j;
}

/* b for a block whose largest magnitude has these bits; NaN and infinity saturate. */
__device__ __forceinline__ uint32_t block_exponent(uint32_t top)
{
    const uint32_t b = (min(top, 0x7f800000u) + 0xfffffu) >> 23;
    return top == 0u ? 0u : min(max(b, kMinExp), kMaxExp);
}

/* 2^(b-127), 0 for b = 0; and its reciprocal (2^127 for b = 0, whose values are all 0). */
__device__ __forceinline__ float exp_scale(uint32_t b) { return __uint_as_float(b << 23); }
__device__ __forceinline__ float exp_unscale(uint32_t b) { return __uint_as_float((254u - b) << 23); }

__device__ __forceinline__ uint32_t encode_m(float x, float unscale, uint32_t r)
{
    const float y = __fmul_rn(__fmul_rn(fabsf(x), unscale), 0x1p-112f);
    return min((__float_as_uint(y) + r) >> 20, 127u) | (__float_as_uint(x) >> 24 & 0x80u);
}

__device__ __forceinline__ uint32_t encode_v(float x, float unscale, uint32_t r)
{
    const float y = __fmul_rn(__fmul_rn(fabsf(x), unscale), 0x1p-96f);
    // never 0 for x > 0: the update would divide by eps alone
    return max(min((__float_as_uint(y) + r) >> 20, 255u), x != 0.0f ? 1u : 0u);
}

/* One of a word's four codes as a float with the code's exponent in fp32's field: times
 * 2^112 (m) or 2^96 (v) and the block's 2^(b-127) it is the value. */
__device__ __forceinline__ float raw_m(uint32_t w, int byte)
{
    const int top = (int)__byte_perm(w, 0, byte << 12 | 0x444);  // the code in bits 31..24
    return __uint_as_float((uint32_t)(top >> 4) & 0x87f00000u);
}

__device__ __forceinline__ float raw_v(uint32_t w, int byte)
{
    return __uint_as_float(__byte_perm(w, 0, byte << 12 | 0x444) >> 4);
}

}  // namespace
}  // namespace zero
