// The 4-bit retained cache: its block format, and the conversions of it.
//
// Rows are held in blocks of 16.  A row's values are e2m1 codes (0, .5, 1, 1.5,
// 2, 3, 4, 6 and a sign) with one e4m3 scale per 16 of them: 4.5 bits a value.
// A code times its scale has at most 6 significant bits and is a multiple of
// 2^-10 up to 2688, so the product is exact in fp16 and in bf16.
//
// A block is 18*D bytes: 8D of key codes, 8D of value codes, D of key scales,
// D of value scales.  The order inside is that of the tensor-core fragments
// of the attention (mma m16n8k16, A operand), so that lane 4r + j of a warp
// reads its share of 16 rows with plain vector loads and uses it in place:
//  keys    A = K (16 rows x D).  [16 rows][4 quarters j][D/8 bytes]: byte b of
//          quarter j holds dims j*D/4 + b (low nibble) and j*D/4 + D/8 + b.
//          A lane's pairs of dims come from fixed scale groups, so one half2
//          of scales serves a row of a block.
//  values  A = V^T (D x 16 rows).  [half s][8 slices r][4 pairs j][D/8 bytes]:
//          byte b holds dim r*D/8 + b of rows 8s + 2j (low nibble) and
//          8s + 2j + 1: the rows are the contraction index there.
//  key scales    [8 rows r][4 j][row r, r + 8][D/64]
//  value scales  [D/16 groups][4 j][half s][rows 8s + 2j, 8s + 2j + 1]
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "kvc_internal.cuh"

namespace kvc {
namespace q4 {

constexpr int kRows = 16;                       // rows of a block
__host__ __device__ constexpr int block_bytes(int D) { return 18 * D; }
__host__ __device__ constexpr int k_codes(int) { return 0; }
__host__ __device__ constexpr int v_codes(int D) { return 8 * D; }
__host__ __device__ constexpr int k_scales(int D) { return 16 * D; }
__host__ __device__ constexpr int v_scales(int D) { return 17 * D; }

// Two e4m3 scales (low byte first) -> half2.
__device__ __forceinline__ uint32_t scales_to_half2(uint16_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(r) : "h"(two));
  return r;
}

// Four bytes of codes -> four half2 (byte i: low nibble in the low half).
__device__ __forceinline__ void codes_to_half2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The scale of a group: e4m3 of amax / 6, nearest even, at most 448.  `amax`
// is the bits of a bf16 magnitude.  inv gets the reciprocal of the scale's
// value, 0 for a zero scale.  The division is a true one, so that a quotient
// half way between two scales stays there.
__device__ __forceinline__ uint32_t scale_of(uint32_t amax, float* inv) {
  const float want = __fdiv_rn(__uint_as_float(amax << 16), 6.0f);
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(two) : "f"(0.0f), "f"(want));
  const uint32_t h = scales_to_half2(two);
  const float s = __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
  *inv = s > 0.0f ? __frcp_rn(s) : 0.0f;
  return two & 0xffu;
}

// Four pairs of values (packed in two words each: lo and hi, two pairs a word)
// -> four bytes of codes, inv the reciprocals of the pairs' two scales.
// x has 8 significant bits, the scale 4 and a border between codes 3, so x /
// scale either is a border exactly or stays a factor of 1 + 2^-9 away from it.
// x * inv is within 2^-23 of the quotient; rounding it to fp16's 11 significant
// bits puts it back on the border in the first case and crosses none in the
// second.  Magnitudes above 6 become 6.
__device__ __forceinline__ uint32_t code_bytes(const uint32_t* lo, const uint32_t* hi, float2 inv) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t l = lo[i >> 1], u = hi[i >> 1];
    const float2 x = make_float2(__uint_as_float((i & 1) ? l & 0xffff0000u : l << 16),
                                 __uint_as_float((i & 1) ? u & 0xffff0000u : u << 16));
    float2 t;
    asm("mul.rn.f32x2 %0, %1, %2;\n"
        : "=l"(reinterpret_cast<uint64_t&>(t))
        : "l"(reinterpret_cast<const uint64_t&>(x)), "l"(reinterpret_cast<const uint64_t&>(inv)));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(h[i]) : "f"(t.y), "f"(t.x));
  }
  uint32_t r;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f16x2 b0, %1;\n cvt.rn.satfinite.e2m1x2.f16x2 b1, %2;\n"
      " cvt.rn.satfinite.e2m1x2.f16x2 b2, %3;\n cvt.rn.satfinite.e2m1x2.f16x2 b3, %4;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n}\n"
      : "=r"(r)
      : "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]));
  return r;
}

// Bits of value i of packed bf16.
__device__ __forceinline__ uint32_t bf16_of(const uint32_t* w, int i) {
  return (i & 1) ? (w[i >> 1] >> 16) : (w[i >> 1] & 0xffffu);
}

}  // namespace q4

// Slots of the 4-bit cache, passed by value in the kernel argument block:
// head h owns rows off[h] .. off[h+1]-1 of its batch element's off[H_kv] rows
// (multiples of 16).
struct Q4Slots {
  int H_kv;
  int64_t off[kMaxHkv + 1];
};

}  // namespace kvc
