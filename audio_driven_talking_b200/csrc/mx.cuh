// mx.cuh - microscaled (block-scaled) 8- and 4-bit floating point: the number format's
// arithmetic, shared by the quantiser, the norm and the product's epilogue.
//
// A block is 32 consecutive values of a row with one power-of-two scale 2^e, stored as the
// byte e + 127 (e8m0). Elements are e4m3 (mxfp8, largest value 448) or e2m1 (mxfp4, largest
// value 6). e is the smallest integer, not below -127, with max|x| <= top * 2^e, so no value
// saturates; the element is x * 2^-e (exact in fp32) rounded to nearest, ties to even. A block
// that holds an infinity or a NaN gets the scale byte 255, e8m0's NaN, and zero elements: all
// its values read back as NaN, and so does every product with it.
//
// Scale bytes lie in tiles of 128 rows x 4 blocks, 512 bytes each, row tiles outermost: row r,
// block k at ((r / 128) * ceil(K / 128) + k / 4) * 512 + (r % 32) * 16 + ((r % 128) / 32) * 4 +
// k % 4, the order in which tcgen05.cp.32x128b.warpx4 spreads them over TMEM; what the last
// tiles hold beyond the tensor is 0. The product may read that padding, against zero elements.
#pragma once

#include "common.cuh"

namespace fh {

enum MxFormat { MX_FP8 = 0, MX_FP4 = 1 };

// byte offset of the 4-byte word with the scales of row r, blocks 4 kt .. 4 kt + 3
__host__ __device__ __forceinline__ size_t mx_scale_word(long r, long kt, long ktiles) {
  return ((size_t)(r >> 7) * ktiles + kt) * 512 + (size_t)((r & 31) * 16 + ((r >> 5) & 3) * 4);
}

// The scale byte of a block whose largest |x| has the bit pattern `amax` (an integer maximum of
// sign-less patterns orders infinities and NaN above every number). With amax = 1.f * 2^E,
// top = 1.75 * 2^8 (e4m3) or 1.5 * 2^2 (e2m1): e = E - 8 or E - 2, plus 1 where 1.f is above
// 1.75 or 1.5, which the addition carries into the exponent field. Subnormal amax: e = -127.
template <MxFormat F>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
  if (amax >= 0x7f800000u) return 255u;
  const int b = F == MX_FP8 ? (int)((amax + 0x1fffffu) >> 23) - 8 : (int)((amax + 0x3fffffu) >> 23) - 2;
  return b < 0 ? 0u : (uint32_t)b;
}

// 2^-e of a scale byte (at most 253), and 0 for the NaN byte, whose elements are then 0 once the
// block's infinities and NaN are replaced (mx_encode8)
__device__ __forceinline__ float mx_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// 2^e of a scale byte; 2^-127 is subnormal, 255 is NaN
__device__ __forceinline__ float mx_scale_value(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7fc00000u : byte == 0u ? 0x00400000u : byte << 23);
}

// two e4m3 codes (lo in the low byte)
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// eight e2m1 codes, v[0] in the low four bits
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Largest |v|, as a bit pattern: NaN (0x7fffffff) if any is, by three-way maxima
__device__ __forceinline__ float amax3(float m, float a, float b) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t mx_amax8(const float* v) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) m = amax3(m, v[i], v[i + 1]);
  return __float_as_uint(m);
}
__device__ __forceinline__ uint32_t mx_amax32(const float* v) {
  float m[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) m[j] = __uint_as_float(mx_amax8(v + 8 * j));
  return __float_as_uint(amax3(amax3(m[0], m[1], m[2]), m[3], 0.f));
}

// Two fp32 operations in one instruction
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 x, x, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 x, x, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

// Codes of eight values under a scale byte: 8 bytes (e4m3) or 4 bytes (e2m1, in .x).
template <MxFormat F>
__device__ __forceinline__ uint2 mx_encode8(const float* v, uint32_t byte) {
  if (byte == 255u) return make_uint2(0u, 0u);
  const float inv = mx_inv_scale(byte);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = v[i] * inv;
  if (F == MX_FP4) return make_uint2(cvt_e2m1x8(y), 0u);
  return make_uint2(cvt_e4m3x2(y[0], y[1]) | cvt_e4m3x2(y[2], y[3]) << 16,
                    cvt_e4m3x2(y[4], y[5]) | cvt_e4m3x2(y[6], y[7]) << 16);
}

// Values of two codes under a scale
__device__ __forceinline__ float2 mx_decode2_e4m3(uint32_t codes16, float scale) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes16));
  const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h));
  return make_float2(f.x * scale, f.y * scale);
}
__device__ __forceinline__ float2 mx_decode2_e2m1(uint32_t codes8, float scale) {
  uint32_t h;
  asm("{\n\t.reg .b8 b, z;\n\tmov.b16 {b, z}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
      : "=r"(h)
      : "h"((uint16_t)codes8));
  const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h));
  return make_float2(f.x * scale, f.y * scale);
}

}  // namespace fh
