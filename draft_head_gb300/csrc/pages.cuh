// A cache in pages (domino_paged_cache in domino.h) on the device: where a slot lies, and the
// quantised form of a head's vector: e4m3 codes with one power of two, 2^(byte - 127).
//
// A power of two costs at most one of e4m3's 16 binades against an fp32 scale and is exact to
// apply: code x scale fits bf16 (4 significant bits), so the attention kernels multiply in bf16
// and lose nothing.
#pragma once

#include <math.h>

#include "common.cuh"

namespace domino {

// Which cache a kernel is compiled for.
enum Cache { kWhole = 0, kPaged = 1, kPagedE4m3 = 2 };

constexpr int kLeastExp = -100, kMostExp = 120;  // of a scale
constexpr int kScaleNan = 255;                   // a vector that held an infinity or a NaN

// Page of slot s of request b, or -1 for one that is not there.
__device__ __forceinline__ int page_of(const PagesArgs& p, int b, int s) {
  int page;  // read where it is asked for: the compiler would move it to its use, behind other waits
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(page) : "l"(p.table + (int64_t)b * p.table_stride + (s >> p.shift)));
  return (unsigned)page < (unsigned)p.n_pages ? page : -1;
}
__device__ __forceinline__ int slot_in_page(const PagesArgs& p, int s) { return s & ((1 << p.shift) - 1); }
// A scale's place: [n_pages, heads, page size] bytes.
__device__ __forceinline__ int64_t scale_at(const PagesArgs& p, int heads, int page, int h, int s) {
  return (((int64_t)page * heads + h) << p.shift) + slot_in_page(p, s);
}

// The scale's byte for a vector whose largest magnitude has the bits `most`: the smallest exponent for which no element is above 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_byte(uint32_t most) {
  if (most >= 0x7f800000u) return kScaleNan;
  const int e = (int)(most >> 23) - 127 - 8 + ((most & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kLeastExp), kMostExp) + 127;
}
// What a vector is multiplied by before it is rounded to codes: 2^-e, and 0 for kScaleNan (whose codes are set to 0).
__device__ __forceinline__ float scale_inverse(int byte) {
  return byte == kScaleNan ? 0.0f : __uint_as_float((uint32_t)(254 - byte) << 23);
}
// Two values as codes, rounded to nearest even, `lo` in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four codes (low byte first) in fp32, without their scale. The fields of a code at fp32's places are its value times 2^-120,
// subnormal codes included. (The two codes that e4m3 gives to NaN are never written; here they are 480 and -480.)
__device__ __forceinline__ float4 codes_f32(uint32_t x) {
  auto one = [](uint32_t b) { return __uint_as_float(((b & 0x80u) << 24) | ((b & 0x7fu) << 20)) * 1.329227995784916e36f; };
  return make_float4(one(x), one(x >> 8), one(x >> 16), one(x >> 24));
}
// 2^e of a scale's byte, or NaN.
__device__ __forceinline__ float scale_f32(int byte) {
  return byte == kScaleNan ? __uint_as_float(0x7fffffffu) : __uint_as_float((uint32_t)byte << 23);
}

// Four codes, those of e4m3's NaN (which are never written, but may lie in slots that were not) as 448.
__device__ __forceinline__ uint32_t codes_that_are_numbers(uint32_t x) {
  return x & ~((((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7);
}
// Four codes (low byte first) as two fp16 pairs, without their scale: every code is a normal fp16 number or 0.
__device__ __forceinline__ uint2 codes_f16(uint32_t x) {
  uint2 r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
      : "=r"(r.x), "=r"(r.y)
      : "r"(x));
  return r;
}
// A row of queries in fp16, for products with codes: divided by a power of two that brings its largest magnitude, of these bits,
// to [16, 32), where fp16 holds bf16's 8 bits of every element above 2^-21 of the largest, and smaller ones to within 2^-29 of it. (Below
// 2^-122 it is 2^-126: fp16 then holds all that bf16 has there.)
__device__ __forceinline__ int query_exponent(uint32_t most) {
  return most >= 0x7f800000u ? 0 : min(max((int)(most >> 23) - 127 - 4, -126), 126);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// A bf16 pair times f in fp16. A finite element of a row with an infinity or a NaN stays finite.
__device__ __forceinline__ uint32_t query_f16(uint32_t x, float f) {
  float lo = __uint_as_float(x << 16) * f, hi = __uint_as_float(x & 0xffff0000u) * f;
  if (fabsf(lo) > 65504.0f && fabsf(lo) < INFINITY) lo = copysignf(65504.0f, lo);
  if (fabsf(hi) > 65504.0f && fabsf(hi) < INFINITY) hi = copysignf(65504.0f, hi);
  return pack_f16(lo, hi);
}

// A scale as the bf16 pairs by which codes at bf16's places, 2^-120 of their values, are multiplied: 2^(e + 120). From e = 8 on
// (vectors with elements above 57,344) that takes two factors.
struct Scale2 {
  uint32_t first, second;  // second 0: none
};
__device__ __forceinline__ Scale2 scale_bf16(int byte) {
  const int to = byte + 120;  // the factor's exponent field
  Scale2 s;
  const uint32_t one = byte == kScaleNan ? 0x7fffu : (uint32_t)min(to, 254) << 7;
  s.first = one | one << 16;
  const uint32_t two = byte == kScaleNan || to <= 254 ? 0u : (uint32_t)(to - 254 + 127) << 7;
  s.second = two | two << 16;
  return s;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Four codes as two bf16 pairs, times the first factor.
__device__ __forceinline__ uint2 codes_bf16(uint32_t x, uint32_t first) {
  const uint32_t a = __byte_perm(x, 0, 0x1404), b = __byte_perm(x, 0, 0x3424);  // a code in the high byte of each half
  return make_uint2(mul_bf16x2((a & 0x80008000u) | ((a >> 4) & 0x07f007f0u), first),
                    mul_bf16x2((b & 0x80008000u) | ((b >> 4) & 0x07f007f0u), first));
}
// Eight codes, scaled.
__device__ __forceinline__ uint4 codes8_bf16(uint2 x, const Scale2& s) {
  const uint2 a = codes_bf16(x.x, s.first), b = codes_bf16(x.y, s.first);
  if (s.second)
    return make_uint4(mul_bf16x2(a.x, s.second), mul_bf16x2(a.y, s.second), mul_bf16x2(b.x, s.second), mul_bf16x2(b.y, s.second));
  return make_uint4(a.x, a.y, b.x, b.y);
}

}  // namespace domino
