// Microscaled 4-bit (MX4) matrices: launch arguments, launchers and the
// element arithmetic shared by the kernels of mx4.cu and mx4_gemm.cu.
//
// An MX4 matrix keeps each row in blocks of 32 consecutive elements.  A block
// has one scale byte s, standing for 2^(s - 127) (255: not a number), and 32
// elements of 4 bits (sign, two exponent bits, one mantissa bit), each one of
// +-{0, .5, 1, 1.5, 2, 3, 4, 6}; element 2i is the low half of byte i, element
// 2i + 1 the high half.  Quantising a block whose largest magnitude is m:
//   s = max(floor(log2 m) - 2 + 127, 0), which is m's binary32 exponent field
//       minus 2, not below 0; 255 when the block holds an infinity or a NaN
//   element = round(x * 2^(127 - s)), magnitudes above 6 becoming 6.
// The scaled value is below 8, so "above 6" is at most a third of a step over.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kernels.cuh"

namespace zsm {

enum MxType { kMxBf16 = 0, kMxF16 = 1, kMxF32 = 2 };  // mirrors ZERO_DTYPE_*
constexpr int kMxBlock = 32;

struct MxMatrix {
  uint8_t* codes;   // 16-byte aligned
  uint8_t* scales;
  int64_t rows, cols;
  int64_t code_pitch;   // bytes between rows, a multiple of 16
  int64_t scale_pitch;  // bytes between rows
};

inline int64_t mx_blocks(int64_t n) { return (n + kMxBlock - 1) / kMxBlock; }

// Division by a fixed 32-bit divisor of dividends below 2^31: the rounded-up
// reciprocal's high half, exact there because 2^(31 + l) (l = ceil(log2 d))
// exceeds the dividend times the reciprocal's rounding error.
struct FastDiv {
  uint32_t d, mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0, 0};
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  f.shift = l ? l - 1 : 0;
  f.mul = d == 1 ? 0 : (uint32_t)(((1ull << (31 + l)) + d - 1) / d);
  return f;
}

// Scale bytes in the tensor core's order ("pieces"), for matrices whose rows
// of scales are not 16-byte aligned: kMxPiece bytes for each 128 rows and 16
// blocks, row r's byte for block b at 512 (b / 4) + 16 (r % 32) +
// 4 (r / 32 % 4) + b % 4; 0 past the matrix (the codes there are 0 too, but a
// product with a NaN scale would not be).  Pieces of 128 rows follow one
// another, a row block's groups of 16 blocks first, in whole pairs of blocks.
constexpr int kMxPiece = 2048;
struct MxPieceArgs {
  const uint8_t* scales[2];
  int64_t pitch[2];
  int rows[2];
  uint8_t* out[2];
  int n;              // matrices
  int warps0, warps;  // 32-row parts of the first, of all
  int k_blocks, groups;
};

struct MxQuantArgs {
  const void* src;      // rows x cols of `type`, ld elements between rows; or an MX4 matrix:
  MxMatrix from;        //   (type ignored, codes set)
  int type;
  int64_t rows, cols, ld;
  MxMatrix out;         // blocks along the rows: rows x cols (codes null: not wanted)
  MxMatrix out_t;       // blocks down the columns: cols x rows (codes null: not wanted)
  int stochastic;
  uint64_t seed;
  MxPieceArgs pieces;   // written beside it when pieces.warps is not 0 (rows only)
};

// The backward pass of a linear layer's operands in one launch: dy along its
// rows and down its columns, x down its columns (both of `type`), w's transpose.
struct MxBackwardArgs {
  MxQuantArgs dy, x, w;
};

struct MxDequantArgs {
  MxMatrix in;
  void* dst;
  int type;
  int64_t ld;
};

// All-gather into N MX4 buffers.  The flat elements [lo, lo + n) come from
// src[i / shard] + i (one array for every owner when `uniform`); block k of
// the interval covers elements lo + 32 k and on.
struct MxGatherArgs {
  const uint16_t* src[kMaxRanks];
  uint8_t* codes[kMaxRanks];
  uint8_t* scales[kMaxRanks];
  int64_t lo, n, shard;
  int n_ranks, uniform, fmt;
};

// Reduce-scatter of N MX4 gradients of n elements to 16-bit means.
struct MxReduceArgs {
  const uint8_t* codes[kMaxRanks];
  const uint8_t* scales[kMaxRanks];
  uint16_t* shard_out;
  int64_t n;
  int n_ranks, accumulate, fmt;
  float inv_n;
  NormScratch ns;
};

// c[i][j] = sum over k of a[i][k] b[j][k], for all rows i of a and j of b.
struct MxMatmulArgs {
  MxMatrix a, b;
  void* out;
  int type;
  int64_t ld;
  void* workspace;  // mx_matmul_workspace bytes, 16-byte aligned
  int pdl;          // 1: programmatic launch: the grid before this one writes the operands
  int b_ready;      // 1: but not b, whose pieces (if it needs any) it writes into the workspace
  const void* x;    // when set, a's rows x cols as a dense matrix of x_type, which the kernel quantises itself
  int x_type;       //   (a's codes and scales are not used)
  int64_t x_ld;
};
constexpr int kMxFewRows = 16;  // rows of x that launch_mx_matmul can quantise itself

cudaError_t launch_mx_quantize(const MxQuantArgs& a, int sm_count, cudaStream_t s);
cudaError_t launch_mx_backward(const MxBackwardArgs& a, int sm_count, cudaStream_t s);
cudaError_t launch_mx_dequantize(const MxDequantArgs& a, int sm_count, cudaStream_t s);
cudaError_t launch_mx_gather(const MxGatherArgs& a, int sm_count, cudaStream_t s);
cudaError_t launch_mx_reduce(const MxReduceArgs& a, int sm_count, cudaStream_t s);
cudaError_t launch_mx_matmul(const MxMatmulArgs& a, int sm_count, cudaStream_t s);
// The same for one row of a (where mx_by_gemv says so), without the tensor cores or m.workspace.
bool mx_by_gemv(int64_t rows, int64_t cols);
cudaError_t launch_mx_gemv(const MxMatmulArgs& a, int sm_count, cudaStream_t s);
int64_t mx_matmul_workspace(const MxMatrix& a, const MxMatrix& b);
// b's part of the workspace as pieces to be written (none when its rows load as they lie).
bool mx_linear_pieces(const MxMatrix& b, void* workspace, MxPieceArgs* g);
int64_t mx_few_rows_workspace(const MxMatrix& b);  // with x instead of a
cudaError_t mx_matmul_errors(unsigned* count, cudaStream_t s);

// The message zero_last_error(NULL) returns to the calling thread.
void set_thread_error(const char* msg);

#ifdef __CUDACC__
namespace mx {

__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv& f) {
  return f.mul ? __umulhi(n, f.mul) >> f.shift : n;
}

// The scale byte of a block from the largest magnitude's binary32 pattern.
__device__ __forceinline__ uint32_t scale_code(uint32_t max_bits) {
  const uint32_t e = max_bits >> 23;
  return e == 255u ? 255u : (e < 2u ? 0u : e - 2u);
}

// 2^(127 - s); 0 for s = 255.  s of a finite block is at most 252, so the
// exponent field 254 - s is that of a normal number.
__device__ __forceinline__ float inverse_scale(uint32_t s) { return s == 255u ? 0.0f : __uint_as_float((254u - s) << 23); }

// 2^(s - 127): subnormal for s = 0, NaN for s = 255.
__device__ __forceinline__ float scale_value(uint32_t s) {
  return s == 0u ? __uint_as_float(0x00400000u) : s == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(s << 23);
}

// Eight scaled values to eight 4-bit elements, to nearest even (6 and above: 6).
__device__ __forceinline__ uint32_t encode8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Eight 4-bit elements to four half2 (exact).
__device__ __forceinline__ void decode8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ float2 half2_float2(uint32_t h) {
  __half2_raw r;
  r.x = (unsigned short)(h & 0xFFFFu);
  r.y = (unsigned short)(h >> 16);
  return __half22float2(__half2(r));
}

// Two binary32 products and sums at once.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)),
        "l"(reinterpret_cast<const uint64_t&>(c)));
  return d;
}

// Eight elements' values.
__device__ __forceinline__ void values8(uint32_t w, uint32_t s, float (&v)[8]) {
  uint32_t h[4];
  decode8(w, h);
  const float sc = scale_value(s);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 f = mul2(half2_float2(h[p]), make_float2(sc, sc));
    v[2 * p] = f.x, v[2 * p + 1] = f.y;
  }
}

// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", 2011): four words for one 128-bit counter and 64-bit key.
__device__ __forceinline__ uint4 philox(uint64_t counter, uint64_t key) {
  uint32_t c0 = (uint32_t)counter, c1 = (uint32_t)(counter >> 32), c2 = 0, c3 = 0;
  uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint32_t p_hi = __umulhi(c0, 0xD2511F53u), p_lo = c0 * 0xD2511F53u;
    const uint32_t q_hi = __umulhi(c2, 0xCD9E8D57u), q_lo = c2 * 0xCD9E8D57u;
    c0 = q_hi ^ c1 ^ k0;
    c1 = q_lo;
    c2 = p_hi ^ c3 ^ k1;
    c3 = p_lo;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// One element rounded stochastically: with t the scaled magnitude in units of
// its grid step and r a number of 16 bits, floor(t + r / 2^16), formed as
// (floor(2^16 t) + r) >> 16 so that every step is exact (t < 4, so 18 bits).
__device__ __forceinline__ uint32_t encode_stochastic(float v, uint32_t r) {
  const float a = fabsf(v);
  const float up = a < 2.0f ? 131072.0f : a < 4.0f ? 65536.0f : 32768.0f;  // 2^16 / step
  const uint32_t base = a < 2.0f ? 0u : a < 4.0f ? 2u : 4u;               // code of q steps = q + base
  const uint32_t q = ((uint32_t)(a * up) + r) >> 16;
  const uint32_t code = min(q + base, 7u);
  return code | ((__float_as_uint(v) >> 28) & 8u);
}

// Eight scaled values; call c (0..3) of block b gives the random numbers of
// its elements 8c .. 8c + 7, the low half of each word first.
__device__ __forceinline__ uint32_t encode8_stochastic(const float (&v)[8], uint64_t block, int c, uint64_t seed) {
  const uint4 w = philox(4ull * block + (uint64_t)c, seed);
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
  uint32_t out = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    out |= encode_stochastic(v[j], j & 1 ? r[j >> 1] >> 16 : r[j >> 1] & 0xFFFFu) << (4 * j);
  return out;
}

}  // namespace mx
#endif

}  // namespace zsm
