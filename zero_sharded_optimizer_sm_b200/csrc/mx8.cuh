// Microscaled 8-bit (MX8) matrices, what a layer keeps of its activations for
// the backward pass: launch arguments, launchers and element arithmetic.
//
// An MX8 matrix keeps each row in blocks of 32 consecutive elements.  A block
// has one scale byte s, standing for 2^(s - 127) (255: not a number), and 32
// elements of 8 bits: sign, four exponent and three mantissa bits (E4M3, at
// most 448).  Quantising a block whose largest magnitude is m:
//   s = the smallest with m <= 448 * 2^(s - 127), not below 3 nor above 246;
//       255 when the block holds an infinity or a NaN
//   element = round(x * 2^(127 - s)) to nearest even, at most 448.
// The format's usual exponent, floor(log2 m) - 8, would cut magnitudes between
// 448 and 512 times the scale, an eighth of the largest at worst; a
// checkpoint's largest elements are the ones that a norm and a weight gradient
// hang on, so the scale is one step up there.  From s = 3 on the elements'
// step is at least 2^-133, bf16's smallest number, and up to s = 246 every
// value is below 2^128: what is read back is exact in bf16 and binary32.
#pragma once

#include "mx4.cuh"

namespace zsm {

// codes: a byte an element, 16-byte aligned rows of whole blocks.
using Mx8Matrix = MxMatrix;

struct Mx8QuantArgs {
  const void* src;  // rows x cols of `type`, ld elements between rows
  int type;
  int64_t rows, cols, ld;
  Mx8Matrix out;
};
struct Mx8DequantArgs {
  Mx8Matrix in;
  void* dst;
  int type;
  int64_t ld;
};

cudaError_t launch_mx8_quantize(const Mx8QuantArgs& a, int sm_count, cudaStream_t s);
cudaError_t launch_mx8_dequantize(const Mx8DequantArgs& a, int sm_count, cudaStream_t s);

#ifdef __CUDACC__
namespace mx {

constexpr uint32_t kMx8Low = 3, kMx8High = 246;

// The scale byte of a block from the largest magnitude's binary32 pattern:
// 448 is 1.75 * 2^8, so the exponent field less 8, and one more where the
// mantissa is over 1.75's.
__device__ __forceinline__ uint32_t scale_code8(uint32_t max_bits) {
  if (max_bits >= 0x7F800000u) return 255u;
  const uint32_t e = (max_bits + 0x1FFFFFu) >> 23;
  return min(max(e, kMx8Low + 8u) - 8u, kMx8High);
}

// Four scaled values to four elements (over 448: 448).
__device__ __forceinline__ uint32_t encode_e4m3(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 p, q;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 p, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 q, %4, %3;\n\t"
      "mov.b32 %0, {p, q};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Four elements' values (exact in binary16).
__device__ __forceinline__ void decode_e4m3(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 p, q;\n\t"
      "mov.b32 {p, q}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, p;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, q;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// The codes of eight values under a block's scale byte.
__device__ __forceinline__ uint2 encode8_mx8(const float (&v)[8], uint32_t s) {
  const float inv = inverse_scale(s);
  float u[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] = __fmul_rn(v[j], inv);
  const uint2 w = make_uint2(encode_e4m3(u[0], u[1], u[2], u[3]), encode_e4m3(u[4], u[5], u[6], u[7]));
  return s == 255u ? make_uint2(0u, 0u) : w;
}

// Eight elements' values.
__device__ __forceinline__ void values8_mx8(uint2 w, uint32_t s, float (&v)[8]) {
  uint32_t h[4];
  decode_e4m3(w.x, h[0], h[1]);
  decode_e4m3(w.y, h[2], h[3]);
  const float sc = scale_value(s);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 f = mul2(half2_float2(h[p]), make_float2(sc, sc));
    v[2 * p] = f.x, v[2 * p + 1] = f.y;
  }
}

// A value that is finite in MX8 stays so in binary16: its largest number
// instead of an infinity.  (An element is rounded up to 16 steps of an eighth,
// so binary16's own numbers from 63488 on become 65536.)
template <class T>
__device__ __forceinline__ void finite_in(float (&v)[8]) {
  if constexpr (T::kFinite > 0.0f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] > T::kFinite ? T::kFinite : v[j] < -T::kFinite ? -T::kFinite : v[j];
  }
}

}  // namespace mx
#endif

}  // namespace zsm
