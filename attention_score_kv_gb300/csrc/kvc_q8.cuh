// The 8-bit retained cache: its format, and the conversions of it.
//
// Rows are held in blocks of 16.  A row is D e4m3 codes, keys and values in
// arrays of their own, row after row; a block has one scale for its keys and one
// for its values, fp32 [block][2]:
//   scale = 2^k, k the least integer >= -100 with max|x| <= 448 * 2^k over the
//   block's rows;  code = x / scale, to nearest even.
// e4m3 has an exponent of its own, so a power of two loses no precision against
// max|x| / 448, and it makes three things exact: the quotient above, a value read
// back as bf16 (4 significant bits), and the new codes of a block whose scale
// grows (but for those that leave e4m3's normal numbers).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "kvc_internal.cuh"

namespace kvc {
namespace q8 {

constexpr int kRows = 16;                       // rows of a block
constexpr uint32_t kLeast = 27;                 // biased exponent of the smallest scale, 2^-100,
constexpr uint32_t kMost = 247;                 // and of the largest that finite values need
// Largest magnitude that is held, as bf16 bits: above 1.875 * 2^127 a value would
// round up to 2^128.
constexpr uint32_t kTop = 0x7f70u;

// Biased exponent of the scale for a largest magnitude (bf16 bits, <= kTop):
// 448 is 1.75 * 2^8, so the exponent of amax less 8, one more where its
// significand is above 1.75.
__device__ __forceinline__ uint32_t scale_exp(uint32_t amax) {
  const uint32_t e = (amax + 0x1fu) >> 7;
  return e < kLeast + 8 ? kLeast : e - 8;
}
__device__ __forceinline__ float pow2(uint32_t biased) { return __uint_as_float(biased << 23); }

// Four bf16 values (two words) times `inv` -> four codes.
__device__ __forceinline__ uint32_t codes_of(uint32_t a, uint32_t b, float inv) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n"
      : "=h"(lo)
      : "f"(__uint_as_float(a & 0xffff0000u) * inv), "f"(__uint_as_float(a << 16) * inv));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n"
      : "=h"(hi)
      : "f"(__uint_as_float(b & 0xffff0000u) * inv), "f"(__uint_as_float(b << 16) * inv));
  return (uint32_t)lo | (uint32_t)hi << 16;
}

// Four codes -> two half2, exact.
__device__ __forceinline__ void to_half2(uint32_t w, uint32_t (&h)[2]) {
  asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, u;\n}\n"
      : "=r"(h[0]), "=r"(h[1])
      : "r"(w));
}

}  // namespace q8
}  // namespace kvc
