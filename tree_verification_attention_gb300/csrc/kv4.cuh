// kv4.cuh - the 4-bit K/V record (include/tva.h, "4-bit cache"): layout, the rounding of
// 16 values to codes and a scale, and back.
//
// A record holds one cache row's K and V of one KV head:
//   [K codes d/2][V codes d/2][K scales d/16][V scales d/16][0 up to a multiple of 16].
// 16 bytes is the granule of a TMA copy, so a box of records can be fetched as it is.
// The little-endian code word i holds elements 8 i .. 8 i + 7: element 8 i + 2 j in bits
// 4 j .. 4 j + 3 and element 8 i + 2 j + 1 sixteen bits above it, so that one shift and
// one and-or put two neighbouring elements' codes into the halves of a 16-bit pair.
// A code n stands for (n - 8) * scale.  Scales are unsigned 5-bit-exponent, 3-bit-mantissa
// floats (bias 15, subnormals): a byte shifted left by 7 is the same value in fp16.  At
// most 3 + 4 significant bits meet in a product, so every value is exact in bf16 and fp16.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace tva {

// The largest scale byte: 1.25 * 2^11 = 2560, the largest for which 24 * scale (the offset
// that the fp16 form of kv4_pair subtracts) is finite in fp16.
constexpr int kKv4MaxScale = 210;

__host__ __device__ constexpr int kv4_record_bytes(int d) { return (9 * d / 8 + 15) / 16 * 16; }

// The scale byte of a block whose largest magnitude is `amax` (>= 0, infinity allowed):
// amax / 7 rounded to nearest, ties to the even byte, at most kKv4MaxScale.  amax * (1/7)
// is within 2 ulp of the quotient, so truncating it gives the byte below the quotient or,
// next to a byte, one less; comparing amax with 7 times the midpoint above that byte
// (8 significant bits: exact; the fused product's sign is exact) settles either case.
__device__ __forceinline__ int kv4_scale_byte(float amax) {
  const float t = amax * (1.0f / 7.0f);
  int base;
  float mid;
  if (t >= 6.103515625e-05f) {  // 2^-14: normal scales
    const uint32_t tb = __float_as_uint(t) >> 20;  // exponent and 3 mantissa bits
    base = (int)tb - 8 * (127 - 15);
    mid = __uint_as_float((tb << 20) | 0x80000u);
  } else {  // multiples of 2^-17
    base = (int)(t * 131072.0f);
    mid = ((float)base + 0.5f) * 7.62939453125e-06f;
  }
  const float r = fmaf(-7.0f, mid, amax);
  if (r > 0.0f || (r == 0.0f && (base & 1))) ++base;
  return base < kKv4MaxScale ? base : kKv4MaxScale;
}

__device__ __forceinline__ float kv4_scale_value(int byte) {
  return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}

// x / s to the nearest whole number (ties to even) within -7 .. 7, exact for every fp32 x:
// the rounded product with 1 / s is at most one off, and only next to a border, where the
// residual x - q s (exact there) says which side of the border x is on.  NaN gives 0, and
// so does every x at scale 0.
__device__ __forceinline__ int kv4_round(float x, float s, float inv) {
  if (s == 0.0f || x != x) return 0;
  float q = fminf(fmaxf(rintf(x * inv), -8.0f), 8.0f);
  const float r = fmaf(-q, s, x), h = 0.5f * s;
  if (fabsf(r) > h || (fabsf(r) == h && ((int)q & 1))) q += copysignf(1.0f, r);
  return (int)fminf(fmaxf(q, -7.0f), 7.0f);
}

// Position of element e (0 .. 7) of a code word.
__host__ __device__ constexpr int kv4_shift(int e) { return 4 * (e >> 1) + 16 * (e & 1); }

// ---- Codes to 16-bit values.
__device__ __forceinline__ uint32_t bf2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two scale bytes (bits 0 .. 7 and 16 .. 23) as a pair, and the pair that takes the codes'
// offset off.  Every step is exact: the scale has 4 significant bits; 136 = 8 x 17 times it
// at most 8 (17 x 15 = 255), 24 = 8 x 3 times it 6.
template <bool kBF16>
__device__ __forceinline__ void widen_scales(uint32_t b, uint32_t& s, uint32_t& c) {
  if constexpr (kBF16) {
    s = bf2_mul(b << 4, 0x77807780u);  // exponent bias 15 -> 127: times 2^112
    c = bf2_mul(s, 0xc308c308u);       // -136
  } else {
    s = b << 7;
    c = h2_mul(s, 0xce00ce00u);        // -24
  }
}
// The same for byte i of `scales` - a block's scale - in both halves.
template <bool kBF16>
__device__ __forceinline__ void widen_scale(uint32_t scales, int i, uint32_t& s, uint32_t& c) {
  widen_scales<kBF16>(__byte_perm(scales, 0u, 0x4040u + 0x0101u * i), s, c);
}

// One code word (8 values) to four pairs, in the order of the elements.
template <bool kBF16>
__device__ __forceinline__ uint4 widen8(uint32_t w, uint32_t s, uint32_t c) {
  uint4 o;
  if constexpr (kBF16) {  // 128 + n: a code in the low mantissa bits of 2^7
    o.x = bf2_fma((w & 0x000f000fu) | 0x43004300u, s, c);
    o.y = bf2_fma(((w >> 4) & 0x000f000fu) | 0x43004300u, s, c);
    o.z = bf2_fma(((w >> 8) & 0x000f000fu) | 0x43004300u, s, c);
    o.w = bf2_fma(((w >> 12) & 0x000f000fu) | 0x43004300u, s, c);
  } else {                // 16 + n: a code in the high mantissa bits of 2^4
    o.x = h2_fma(((w << 6) & 0x03c003c0u) | 0x4c004c00u, s, c);
    o.y = h2_fma(((w << 2) & 0x03c003c0u) | 0x4c004c00u, s, c);
    o.z = h2_fma(((w >> 2) & 0x03c003c0u) | 0x4c004c00u, s, c);
    o.w = h2_fma(((w >> 6) & 0x03c003c0u) | 0x4c004c00u, s, c);
  }
  return o;
}

}  // namespace tva
