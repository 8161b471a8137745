// A thread's eight columns of a row, and their loads and stores, for kernels
// that give a row to a group of threads (rms_norm.cu, embedding.cu).
#pragma once

#include "mx4_quant.cuh"
#include "mx8.cuh"

namespace zsm {
namespace mx {

// Neighbours where a row is made of whole, 16-byte aligned vectors of eight
// (kVec), every kStride-th column otherwise, so that a warp's loads of single
// elements are whole sectors and 32 columns, a block of an MX matrix, lie
// across its lanes.  Rows are given by their address and columns in 32 bits:
// these kernels are bound by instructions as much as by memory, and 64-bit
// products of rows and pitches for every access were a third of them.
template <bool kVec, int kStride>
struct Columns {
  uint32_t first, cols;
  __device__ __forceinline__ Columns(uint32_t base, uint32_t thread, uint32_t n)
      : first(base + (kVec ? 8 * thread : thread)), cols(n) {}
  __device__ __forceinline__ uint32_t at(int j) const { return kVec ? first + j : first + kStride * j; }
  __device__ __forceinline__ bool in(int j) const { return kVec ? first < cols : at(j) < cols; }
};

template <class F>
__device__ __forceinline__ void set(Vec16<F>& x, const uint16_t (&e)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) x.w[j] = pack2(e[2 * j], e[2 * j + 1]);
}
__device__ __forceinline__ void set(Vec32& x, const float (&e)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) x.x[j] = e[j];
}

// A matrix's row.
template <class T>
__device__ __forceinline__ const typename T::raw* row_of(const void* m, int64_t row, int64_t ld) {
  return static_cast<const typename T::raw*>(m) + row * ld;
}
template <class T>
__device__ __forceinline__ typename T::raw* row_of(void* m, int64_t row, int64_t ld) {
  return static_cast<typename T::raw*>(m) + row * ld;
}
struct Row8 {
  uint8_t *codes, *scales;
};
__device__ __forceinline__ Row8 row_of(const Mx8Matrix& m, int64_t row) {
  return {m.codes + row * m.code_pitch, m.scales + row * m.scale_pitch};
}

// The row's elements at a thread's columns, 0 past its end.
template <class V, bool kVec, int kStride>
__device__ __forceinline__ void load_columns(V& x, const typename V::raw* row, const Columns<kVec, kStride>& c) {
  if constexpr (kVec) {
    if (c.in(0)) x.load(row + c.first);
    else x.clear();
  } else {
    typename V::raw e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = c.in(j) ? __ldcs(row + c.at(j)) : typename V::raw(0);
    set(x, e);
  }
}

// A vector as it is.
template <class F, bool kVec, int kStride>
__device__ __forceinline__ void store_columns(uint16_t* row, const Columns<kVec, kStride>& c, const Vec16<F>& x) {
  if constexpr (kVec) {
    if (c.in(0)) st_stream(row + c.first, make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c.in(j)) row[c.at(j)] = (uint16_t)(x.w[j >> 1] >> (16 * (j & 1)));
  }
}
template <bool kVec, int kStride>
__device__ __forceinline__ void store_columns(float* row, const Columns<kVec, kStride>& c, const Vec32& x) {
  if constexpr (kVec) {
    if (c.in(0)) {
      st_stream(row + c.first, make_float4(x.x[0], x.x[1], x.x[2], x.x[3]));
      st_stream(row + c.first + 4, make_float4(x.x[4], x.x[5], x.x[6], x.x[7]));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c.in(j)) row[c.at(j)] = x.x[j];
  }
}

// Products of pairs.
__device__ __forceinline__ float2 pair(const float (&v)[8], int p) { return make_float2(v[2 * p], v[2 * p + 1]); }
__device__ __forceinline__ void scale8(float (&v)[8], float s) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 f = mul2(pair(v, p), make_float2(s, s));
    v[2 * p] = f.x, v[2 * p + 1] = f.y;
  }
}
__device__ __forceinline__ void times8(float (&v)[8], const float (&w)[8]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 f = mul2(pair(v, p), pair(w, p));
    v[2 * p] = f.x, v[2 * p + 1] = f.y;
  }
}

// A row's MX8 elements without their blocks' scales: eight neighbours.
__device__ __forceinline__ void elements8(uint2 w, float (&v)[8]) {
  uint32_t h[4];
  decode_e4m3(w.x, h[0], h[1]);
  decode_e4m3(w.y, h[2], h[3]);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 f = half2_float2(h[p]);
    v[2 * p] = f.x, v[2 * p + 1] = f.y;
  }
}

// An MX8 row's values at a thread's columns, 0 past its end, in multiples of
// `unit` (a power of two or any other number: one rounding).
template <bool kVec, int kStride>
__device__ __forceinline__ void load_columns8(const Row8& row, const Columns<kVec, kStride>& c, float unit, float (&v)[8]) {
  if constexpr (kVec) {
    uint2 w = make_uint2(0u, 0u);
    uint32_t s = 0u;
    if (c.in(0)) {
      w = __ldcs(reinterpret_cast<const uint2*>(row.codes + c.first));
      s = row.scales[c.first >> 5];
    }
    elements8(w, v);
    scale8(v, __fmul_rn(scale_value(s), unit));
  } else {
    uint32_t w[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j] = c.in(j) ? row.codes[c.at(j)] : 0u;
      s[j] = c.in(j) ? row.scales[c.at(j) >> 5] : 0u;
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      uint32_t h, none;
      decode_e4m3(w[j] | w[j + 1] << 8, h, none);
      const float2 f = half2_float2(h);
      v[j] = __fmul_rn(f.x, __fmul_rn(scale_value(s[j]), unit));
      v[j + 1] = __fmul_rn(f.y, __fmul_rn(scale_value(s[j + 1]), unit));
    }
  }
}

// A vector of a row, 0 past its end, into an MX8 row; v holds x's values.
// Called by whole warps whose columns are neighbours'.
template <class V, bool kVec, int kStride>
__device__ __forceinline__ void store_columns8(const Row8& row, const Columns<kVec, kStride>& c, const V& x,
                                               const float (&v)[8]) {
  const uint32_t padded = (c.cols + 31u) & ~31u;
  if constexpr (kVec) {
    const uint32_t s = scale_code8(max_of_four(x.max_bits()));
    if (c.first >= padded) return;
    *reinterpret_cast<uint2*>(row.codes + c.first) = encode8_mx8(v, s);
    if ((c.first & 31u) == 0) row.scales[c.first >> 5] = (uint8_t)s;
  } else {
    static_assert(kVec || kStride % 32 == 0, "a warp's columns are a block");
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t s = scale_code8(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v[j]) & 0x7FFFFFFFu));
      if (c.at(j) >= padded) continue;
      const float u = __fmul_rn(v[j], inverse_scale(s));
      row.codes[c.at(j)] = s == 255u ? 0 : (uint8_t)encode_e4m3(u, 0.0f, 0.0f, 0.0f);
      if ((c.at(j) & 31u) == 0) row.scales[c.at(j) >> 5] = (uint8_t)s;
    }
  }
}

// A vector of one of the three types at a thread's columns, 0 past its end.
template <bool kVec, int kStride>
__device__ __forceinline__ void load_weights(const void* w, int type, const Columns<kVec, kStride>& c, float (&v)[8]) {
  if constexpr (kVec) {
    if (type == kMxF32) {
      float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = a;
      if (c.in(0)) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + c.first);
        a = __ldg(p), b = __ldg(p + 1);
      }
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
      return;
    }
    uint4 a = make_uint4(0u, 0u, 0u, 0u);
    if (c.in(0)) a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + c.first));
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
    if (type == kMxBf16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[2 * j] = Bf16::lo(u[j]), v[2 * j + 1] = Bf16::hi(u[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[2 * j] = F16::lo(u[j]), v[2 * j + 1] = F16::hi(u[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = 0.0f;
      if (!c.in(j)) continue;
      if (type == kMxF32) {
        v[j] = __ldg(static_cast<const float*>(w) + c.at(j));
      } else {
        const uint16_t u = __ldg(static_cast<const uint16_t*>(w) + c.at(j));
        v[j] = type == kMxF16 ? F16::f32(u) : Bf16::f32(u);
      }
    }
  }
}

// x + y, rounded to their type.  Two 16-bit numbers' sum is exact in binary32
// unless one is below half a step of the other, so that rounding it through
// binary32 and rounding it at once, as the packed additions do, give the same.
__device__ __forceinline__ void add_to(Vec16<Bf16>& x, const Vec16<Bf16>& y) {
#pragma unroll
  for (int j = 0; j < 4; ++j) asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(x.w[j]) : "r"(y.w[j]));
}
__device__ __forceinline__ void add_to(Vec16<F16>& x, const Vec16<F16>& y) {
#pragma unroll
  for (int j = 0; j < 4; ++j) asm("add.rn.f16x2 %0, %0, %1;" : "+r"(x.w[j]) : "r"(y.w[j]));
}
__device__ __forceinline__ void add_to(Vec32& x, const Vec32& y) {
#pragma unroll
  for (int j = 0; j < 8; ++j) x.x[j] = __fadd_rn(x.x[j], y.x[j]);
}

// Eight values rounded into a vector of a type.
template <class F>
__device__ __forceinline__ void round_to(Vec16<F>& x, const float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) x.w[j] = Half<F>::pack(v[2 * j], v[2 * j + 1]);
}
__device__ __forceinline__ void round_to(Vec32& x, const float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) x.x[j] = v[j];
}

// Sixteen (or eight) bytes of global into shared memory, asynchronously; a
// thread's copies arrive in the order of its groups.
__device__ __forceinline__ void copy_async16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_async8(void* to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

}  // namespace mx
}  // namespace zsm
