// The 8-bit paged KV cache: addressing and e4m3 conversions shared by the
// kernels that fill it (cache_fp8.cu), read it (decode_fp8.cu) and shorten it.
//
// Codes are e4m3 bytes [num_pages, page_size, kv_heads, D]; scales fp32
// [num_pages, page_size / block, kv_heads], block a power of two up to 128
// that divides page_size. With row = page * page_size + slot the code row of
// (token, head h) is row * kv_heads + h and, because blocks never straddle
// pages, its scale is (row / block) * kv_heads + h.
//
// Scales written here are powers of two: e4m3 is a floating format, so a power
// of two costs no precision against amax / 448 (only up to one binade of its
// 18-binade range), dividing by it is exact, and codes move from one scale to
// another unchanged unless they fall into the subnormals. Readers take any
// positive normal scale up to 2^127.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "jfa_internal.h"
#include "ptx.cuh"

namespace jfa {

// t / d for 0 <= t < 2^31 by a multiplication (Granlund and Montgomery,
// "Division by Invariant Integers using Multiplication", 1994): with
// 2^l >= d > 2^(l-1) and m = floor(2^32 (2^l - d) / d) + 1 the quotient is
// (mulhi(m, t) + t) >> l; t < 2^31 keeps the sum within 32 bits.
struct FastDiv {
  uint32_t d, mul, shift;
};
inline FastDiv make_fast_div(int32_t d) {
  FastDiv f;
  f.d = static_cast<uint32_t>(d);
  f.shift = 0;
  while ((uint64_t(1) << f.shift) < f.d) ++f.shift;
  f.mul = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << f.shift) - f.d)) / f.d + 1);
  return f;
}
__device__ __forceinline__ int fast_div(int t, const FastDiv& f) {
  return static_cast<int>((__umulhi(f.mul, static_cast<uint32_t>(t)) + static_cast<uint32_t>(t)) >> f.shift);
}

struct Fp8CacheView {
  uint8_t* kc;
  uint8_t* vc;
  float* ks;
  float* vs;
  int32_t hkv, num_pages, block_shift;
  FastDiv page;  // division by page_size
};

// Two e4m3 codes (low byte first) -> two fp16 values, exact (every e4m3 value
// is a normal fp16 number or zero; NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
  return r;
}
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  lo = e4m3x2_to_f16x2(static_cast<uint16_t>(codes & 0xFFFFu));
  hi = e4m3x2_to_f16x2(static_cast<uint16_t>(codes >> 16));
}

// Nearest e4m3 codes of two fp32 values of magnitude at most 448 (ties to
// even); a NaN becomes the NaN code.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The smallest power of two s >= 2^-126 with amax / s <= 448 = 1.75 * 2^8, for
// finite amax >= 0: amax / 2^8 = (1 + f) 2^e takes 2^e, one more if 1 + f > 1.75. (What
// is below 2^-126 there, where a division may round, takes 2^-126.)
__device__ __forceinline__ float e4m3_block_scale_from_256th(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(max(e, -126) + 127) << 23);
}
__device__ __forceinline__ float e4m3_block_scale(float amax) { return e4m3_block_scale_from_256th(amax * 0x1p-8f); }

// Any e4m3 NaN (0x7F or 0xFF) among four codes.
__device__ __forceinline__ bool e4m3_any_nan(uint32_t codes) {
  return (((codes & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
}

}  // namespace jfa
