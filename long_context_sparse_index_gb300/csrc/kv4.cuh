// kv4.cuh -- keys and values in 4 bits: the format, and where its bytes lie.
//
// The 128 values of a key (or value) lie in 8 groups of 16.  A group has a scale
// of 8 bits, 5 of exponent and 3 of mantissa without a sign (the bits of an fp16
// number above its lowest seven: scale = fp16(bits << 7)), and a value a code of
// 4 bits, e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign).  It stands for
//   x = code * scale * 2^-4.
// Written: scale = the nearest to 2^4 max|x| / 6, at most 10240, and code = the
// nearest to 2^4 x / scale, ties to even in both; a group with an infinity or a
// NaN has the scale 0xFF, a NaN, and stands for 16 NaN.
//
// code * scale has at most six significant bits and lies between 2^-18 and
// 61440, so it is exact in fp16 (and x in bf16): a reader converts two codes at
// a time to fp16 (one instruction), multiplies by the scale without rounding,
// and leaves the 2^-4 to a factor that it has anyway.  The range of x, normal
// scales from max|x| = 2.3e-5 to 3840, needs no calibration; beyond 3840 values
// saturate.
//
// The 576 bytes of a pool of four tokens t lie together, so that a selected pool
// is one run of memory:
//   0    keys' codes    [t][64]            byte b: dimension 2b low, 2b + 1 high
//   256  values' codes  [group][t][8]      the same order within a group
//   512  keys' scales   [group / 2][t % 2][t / 2][group % 2]
//   544  values' scales [group][t]
// The orders are those of the attention's fragments: a lane reads 32 dimensions
// of a key, or 16 dimensions of two tokens' values, with one 16-byte load.
#pragma once

#include <cuda_fp16.h>
#include <cstdint>

namespace dsa {

constexpr int kPool4Bytes = 576;
constexpr int kPool4V = 256, kPool4KScale = 512, kPool4VScale = 544;
constexpr uint32_t kScaleMost = 0xE2u;  // 10240: six times it is 61440
constexpr uint32_t kScaleNan = 0xFFu;

__device__ __forceinline__ int k4_code_at(int t, int dim) { return t * 64 + dim / 2; }
__device__ __forceinline__ int v4_code_at(int t, int dim) { return kPool4V + dim / 16 * 32 + t * 8 + dim % 16 / 2; }
__device__ __forceinline__ int k4_scale_at(int t, int group) {
  return kPool4KScale + group / 2 * 8 + (t & 1) * 4 + t / 2 * 2 + (group & 1);
}
__device__ __forceinline__ int v4_scale_at(int t, int group) { return kPool4VScale + group * 4 + t; }

// The scale's bits for a group whose largest magnitude is `top` (finite).
__device__ __forceinline__ uint32_t scale4_of(float top) {
  const float m = __fdiv_rn(16.f * top, 6.f);
  if (m < 6.103515625e-5f)  // below 2^-14: steps of 2^-17 (8 of them are the smallest normal number's bits)
    return static_cast<uint32_t>(__float2int_rn(m * 131072.f));
  const uint32_t b = __float_as_uint(m);
  const uint32_t r = ((b + 0x7FFFFu + ((b >> 20) & 1u)) >> 20) - ((127u - 15u) << 3);
  return r < kScaleMost ? r : kScaleMost;
}
__device__ __forceinline__ float scale4(uint32_t bits) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(bits << 7)));
}

// Eight codes of x[0..7] for a scale: the word whose nibble e is x[e]'s.
__device__ __forceinline__ uint32_t codes4(const float (&x)[8], float scale) {
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    // (a group of scale 0 is nothing but zeros, or too small for the format)
    const float a = scale > 0.f ? __fdiv_rn(16.f * x[2 * e], scale) : 0.f;
    const float b = scale > 0.f ? __fdiv_rn(16.f * x[2 * e + 1], scale) : 0.f;
    uint32_t two;
    asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n cvt.u32.u8 %0, t;\n}" : "=r"(two) : "f"(b), "f"(a));
    w |= two << (8 * e);
  }
  return w;
}

// Codes of byte kB of a word as two fp16 numbers, the low nibble first.
template <int kB>
__device__ __forceinline__ uint32_t f16_of_codes(uint32_t w) {
  uint32_t d;
  if (kB == 0)
    asm("{\n .reg .b8 a, b, c, e;\n mov.b32 {a, b, c, e}, %1;\n cvt.rn.f16x2.e2m1x2 %0, a;\n}" : "=r"(d) : "r"(w));
  else if (kB == 1)
    asm("{\n .reg .b8 a, b, c, e;\n mov.b32 {a, b, c, e}, %1;\n cvt.rn.f16x2.e2m1x2 %0, b;\n}" : "=r"(d) : "r"(w));
  else if (kB == 2)
    asm("{\n .reg .b8 a, b, c, e;\n mov.b32 {a, b, c, e}, %1;\n cvt.rn.f16x2.e2m1x2 %0, c;\n}" : "=r"(d) : "r"(w));
  else
    asm("{\n .reg .b8 a, b, c, e;\n mov.b32 {a, b, c, e}, %1;\n cvt.rn.f16x2.e2m1x2 %0, e;\n}" : "=r"(d) : "r"(w));
  return d;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

}  // namespace dsa
