// Dense vectors of eight elements, their quantisation and their stores, shared
// by the kernels that walk rows (mx4.cu, mx8.cu, rms_norm.cu, embedding.cu) and
// the product that quantises its own operand (mx4_gemm.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "device_math.cuh"
#include "mx4.cuh"

namespace zsm {
namespace mx {

using namespace dev;

// The two 16-bit formats: two values rounded into a word, infinity's pattern.
template <class F>
struct Half;
template <>
struct Half<Bf16> {
  static constexpr uint32_t kInf = 0x7F80u;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162_raw r = __floats2bfloat162_rn(a, b);
    return (uint32_t)r.x | ((uint32_t)r.y << 16);
  }
};
template <>
struct Half<F16> {
  static constexpr uint32_t kInf = 0x7C00u;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2_raw r = __floats2half2_rn(a, b);
    return (uint32_t)r.x | ((uint32_t)r.y << 16);
  }
};

// Of two words of two elements each, the larger magnitudes (their signs are of no
// use; a NaN counts as larger than any number).
template <class F>
__device__ __forceinline__ uint32_t larger2(uint32_t a, uint32_t b);
template <>
__device__ __forceinline__ uint32_t larger2<Bf16>(uint32_t a, uint32_t b) {
  uint32_t m;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
  return m;
}
template <>
__device__ __forceinline__ uint32_t larger2<F16>(uint32_t a, uint32_t b) {
  uint32_t m;
  asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
  return m;
}

// Eight consecutive elements of a storage type, kept as loaded: their values,
// and the binary32 pattern of the largest magnitude (an infinity or NaN
// counts as larger than any number).
template <class F>
struct Vec16 {  // bf16 or binary16
  using raw = uint16_t;
  static constexpr int kUnits = 4;
  uint32_t w[4];
  __device__ __forceinline__ void load(const raw* p) {
    const uint4 x = ld_stream(p);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  }
  // The whole vector, or zeros: one predicated load, without a branch whose
  // end would wait for it.
  __device__ __forceinline__ void load_if(const raw* p, bool yes) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@q ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(w[0]), "=&r"(w[1]), "=&r"(w[2]), "=&r"(w[3])
        : "l"(p), "r"((int)yes)
        : "memory");
  }
  __device__ __forceinline__ void load(const raw* p, int64_t n) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = (2 * j < n ? (uint32_t)p[2 * j] : 0u) | (2 * j + 1 < n ? (uint32_t)p[2 * j + 1] << 16 : 0u);
  }
  __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0u; }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return larger2<F>(a, b); }
  static __device__ __forceinline__ float lo(uint32_t x) { return F::lo(x); }
  static __device__ __forceinline__ float hi(uint32_t x) { return F::hi(x); }
  __device__ __forceinline__ uint32_t max_bits() const {
    // 16-bit patterns without their signs order as their magnitudes do
    uint32_t m = larger(larger(w[0], w[1]), larger(w[2], w[3])) & 0x7FFF7FFFu;
    m = max(m & 0xFFFFu, m >> 16);
    return __float_as_uint(F::f32((uint16_t)m));
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[2 * j] = F::lo(w[j]), v[2 * j + 1] = F::hi(w[j]);
  }
};
struct Vec32 {  // binary32
  using raw = float;
  static constexpr int kUnits = 2;
  float x[8];
  __device__ __forceinline__ void load(const raw* p) {
    const float4 a = ld_stream(p), b = ld_stream(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  __device__ __forceinline__ void load_if(const raw* p, bool yes) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %9, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "mov.b32 %4, 0;\n\tmov.b32 %5, 0;\n\tmov.b32 %6, 0;\n\tmov.b32 %7, 0;\n\t"
        "@q ld.global.v4.f32 {%0, %1, %2, %3}, [%8];\n\t"
        "@q ld.global.v4.f32 {%4, %5, %6, %7}, [%8 + 16];\n\t}"
        : "=&f"(x[0]), "=&f"(x[1]), "=&f"(x[2]), "=&f"(x[3]), "=&f"(x[4]), "=&f"(x[5]), "=&f"(x[6]), "=&f"(x[7])
        : "l"(p), "r"((int)yes)
        : "memory");
  }
  __device__ __forceinline__ void load(const raw* p, int64_t n) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = j < n ? p[j] : 0.0f;
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 0.0f;
  }
  __device__ __forceinline__ uint32_t max_bits() const {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(x[j]) & 0x7FFFFFFFu);
    return m;
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = x[j];
  }
};

// vec: a whole vector's address is 16-byte aligned.
template <class V>
__device__ __forceinline__ void load8(V& x, const typename V::raw* p, int64_t n, int vec) {
  if (n >= 8 && vec) x.load(p);
  else if (n > 0) x.load(p, n);
  else x.clear();
}

// Eight products with a power of two, in pairs.
__device__ __forceinline__ void scale_by(float (&v)[8], float s) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 f = mul2(make_float2(v[j], v[j + 1]), make_float2(s, s));
    v[j] = f.x, v[j + 1] = f.y;
  }
}

// The codes of eight elements from their block's scale byte.  `block` and c
// (the vector's place in the block) number the random numbers.
template <bool kStochastic, class V>
__device__ __forceinline__ uint32_t encode(const V& x, uint32_t s, uint64_t block, int c, uint64_t seed) {
  float v[8];
  x.values(v);
  scale_by(v, inverse_scale(s));
  const uint32_t w = kStochastic ? encode8_stochastic(v, block, c, seed) : encode8(v);
  return s == 255u ? 0u : w;
}

__device__ __forceinline__ uint32_t max_of_four(uint32_t m) {  // over four neighbouring lanes
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  return max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
}

// One warp's part of the pieces: 32 rows, 16 blocks, a lane a row.
__device__ __forceinline__ void write_pieces(const MxPieceArgs& a, int w) {
  if (w >= a.warps) return;
  const int lane = threadIdx.x & 31, o = w >= a.warps0 ? 1 : 0;
  if (o) w -= a.warps0;
  const int g = w % a.groups, r32 = w / a.groups;
  const int64_t row = 32ll * r32 + lane;
  const int n = row < a.rows[o] ? min(a.k_blocks - 16 * g, 16) : 0;
  const uint8_t* p = a.scales[o] + (n > 0 ? row * a.pitch[o] + 16 * g : 0);
  uint32_t v[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (j < n) v[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
  uint8_t* out = a.out[o] + ((int64_t)(r32 >> 2) * a.groups + g) * kMxPiece + 16 * lane + 4 * (r32 & 3);
#pragma unroll
  for (int j = 0; j < 4; ++j) *reinterpret_cast<uint32_t*>(out + 512 * j) = v[j];
}

// ---------------------------------------------------------- element types --

// kFinite: the largest number, where an MX8 value may be over it.
struct TBf16 {
  static constexpr float kFinite = 0.0f;
  using V = Vec16<Bf16>;
  using raw = uint16_t;
  static __device__ __forceinline__ uint32_t pack(float a, float b) { return Half<Bf16>::pack(a, b); }
  static __device__ __forceinline__ raw rn(float x) { return Bf16::rn(x); }
};
struct TF16 {
  static constexpr float kFinite = 65504.0f;
  using V = Vec16<F16>;
  using raw = uint16_t;
  static __device__ __forceinline__ uint32_t pack(float a, float b) { return Half<F16>::pack(a, b); }
  static __device__ __forceinline__ raw rn(float x) { return F16::rn(x); }
};
struct TF32 {
  static constexpr float kFinite = 0.0f;
  using V = Vec32;
  using raw = float;
  static __device__ __forceinline__ raw rn(float x) { return x; }
};

// Eight elements rounded into n places (all eight, on a 16-byte boundary, when
// n >= 8 and vec).
template <class T>
__device__ __forceinline__ void store8(typename T::raw* p, const float (&v)[8], int64_t n, int vec) {
  using raw = typename T::raw;
  if (n >= 8 && vec) {
    if constexpr (sizeof(raw) == 2) {
      st_stream(p, make_uint4(T::pack(v[0], v[1]), T::pack(v[2], v[3]), T::pack(v[4], v[5]), T::pack(v[6], v[7])));
    } else {
      st_stream(p, make_float4(v[0], v[1], v[2], v[3]));
      st_stream(p + 4, make_float4(v[4], v[5], v[6], v[7]));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = T::rn(v[j]);
  }
}

// ------------------------------------------------------------------ launches --

inline int cap_grid(int64_t want, int cap) { return (int)std::max<int64_t>(1, std::min<int64_t>(want, cap)); }

inline bool aligned(const void* p, int64_t pitch_bytes) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)pitch_bytes) & 15u) == 0;
}

// Pieces of 256 columns over all rows; a matrix whose rows lie end to end in
// whole blocks is taken as one row, so that narrow rows fill the warps.
struct Pieces {
  int64_t rows, cols;
  FastDiv per_row;
  uint32_t units;
};
inline bool pieces_of(int64_t rows, int64_t cols, bool end_to_end, Pieces* p) {
  if (end_to_end) {
    cols *= rows;
    rows = 1;
  }
  const int64_t per = (cols + 255) / 256;
  // as FastDiv and the kernels' counters allow; more than 2^31 pieces of
  // whole rows are more memory than there is
  if (per * rows > 0x7FFFFFFFll) return false;
  *p = Pieces{rows, cols, fast_div((uint32_t)per), (uint32_t)(per * rows)};
  return true;
}

// CTAs to an SM of a streaming launch at most: a CTA that ends makes room for
// one whose loads go out at once (read-back of 8192 x 2048: 11.8 us with 8, the
// CTAs then walking on, 9.8 with 64).
constexpr int kWaves = 64;

}  // namespace mx
}  // namespace zsm
