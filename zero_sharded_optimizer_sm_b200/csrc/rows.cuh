// A thread's eight columns of a row, and their loads and stores, for kernels
// that give a row to a group of threads (rms_norm.cu, embedding.cu).
#pragma once

#include "mx4_quant.cuh"
#include "mx8.cuh"

namespace zsm {
namespace mx {

// Neighbours where a row's vectors of eight are 16-byte aligned (kVec), every
// kStride-th column otherwise, so that a warp's loads of single elements are
// whole sectors and 32 columns, a block of an MX matrix, lie across its lanes.
template <bool kVec, int kStride>
struct Columns {
  int64_t first, cols;
  __device__ __forceinline__ Columns(int64_t base, int thread, int64_t n)
      : first(base + (kVec ? 8 * thread : thread)), cols(n) {}
  __device__ __forceinline__ int64_t at(int j) const { return kVec ? first + j : first + kStride * j; }
  __device__ __forceinline__ bool in(int j) const { return at(j) < cols; }
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

// The row's elements at a thread's columns, 0 past its end.
template <class V, bool kVec, int kStride>
__device__ __forceinline__ void load_columns(V& x, const typename V::raw* row, const Columns<kVec, kStride>& c) {
  if constexpr (kVec) {
    load8(x, row + c.first, c.cols - c.first, 1);
  } else {
    typename V::raw e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = c.in(j) ? __ldcs(row + c.at(j)) : typename V::raw(0);
    set(x, e);
  }
}

template <class T, bool kVec, int kStride>
__device__ __forceinline__ void store_columns(typename T::raw* row, const Columns<kVec, kStride>& c, const float (&v)[8]) {
  if constexpr (kVec) {
    store8<T>(row + c.first, v, c.cols - c.first, 1);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c.in(j)) row[c.at(j)] = T::rn(v[j]);
  }
}

// The same of an MX8 row.
template <bool kVec, int kStride>
__device__ __forceinline__ void load_columns8(const Mx8Matrix& m, int64_t row, const Columns<kVec, kStride>& c, float (&v)[8]) {
  const uint8_t* codes = m.codes + row * m.code_pitch;
  const uint8_t* scales = m.scales + row * m.scale_pitch;
  if constexpr (kVec) {
    uint2 w = make_uint2(0u, 0u);
    uint32_t s = 0u;
    if (c.first < c.cols) {
      w = __ldcs(reinterpret_cast<const uint2*>(codes + c.first));
      s = scales[c.first >> 5];
    }
    values8_mx8(w, s, v);
  } else {
    uint32_t w[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j] = c.in(j) ? codes[c.at(j)] : 0u;
      s[j] = c.in(j) ? scales[c.at(j) >> 5] : 0u;
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      uint32_t h, none;
      decode_e4m3(w[j] | w[j + 1] << 8, h, none);
      const float2 f = half2_float2(h);
      v[j] = __fmul_rn(f.x, scale_value(s[j]));
      v[j + 1] = __fmul_rn(f.y, scale_value(s[j + 1]));
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (!c.in(j)) v[j] = 0.0f;  // (what fills up the last block is not the row's)
}

// Eight values, rounded to x's type in x, into an MX8 row.  Called by whole
// warps whose columns are neighbours'.
template <class V, bool kVec, int kStride>
__device__ __forceinline__ void store_columns8(const Mx8Matrix& m, int64_t row, int64_t nb, const Columns<kVec, kStride>& c,
                                               const V& x) {
  uint8_t* codes = m.codes + row * m.code_pitch;
  uint8_t* scales = m.scales + row * m.scale_pitch;
  float v[8];
  x.values(v);
  if constexpr (kVec) {
    const uint32_t s = scale_code8(max_of_four(x.max_bits()));
    const int64_t b = c.first >> 5;
    if (b >= nb) return;
    *reinterpret_cast<uint2*>(codes + c.first) = encode8_mx8(v, s);
    if ((c.first & 31) == 0) scales[b] = (uint8_t)s;
  } else {
    static_assert(kVec || kStride % 32 == 0, "a warp's columns are a block");
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t s = scale_code8(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v[j]) & 0x7FFFFFFFu));
      const int64_t b = c.at(j) >> 5;
      if (b >= nb) continue;
      const float u = __fmul_rn(v[j], inverse_scale(s));
      codes[c.at(j)] = s == 255u ? 0 : (uint8_t)encode_e4m3(u, 0.0f, 0.0f, 0.0f);
      if ((c.at(j) & 31) == 0) scales[b] = (uint8_t)s;
    }
  }
}

// A vector of one of the three types at a thread's columns, 0 past its end.
template <bool kVec, int kStride>
__device__ __forceinline__ void load_weights(const void* w, int type, const Columns<kVec, kStride>& c, float (&v)[8]) {
  const int64_t n = c.cols - c.first;
  if (kVec && n >= 8) {
    if (type == kMxF32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + c.first);
      const float4 a = __ldg(p), b = __ldg(p + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
      return;
    }
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + c.first));
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = type == kMxF16 ? F16::lo(u[j]) : Bf16::lo(u[j]);
      v[2 * j + 1] = type == kMxF16 ? F16::hi(u[j]) : Bf16::hi(u[j]);
    }
    return;
  }
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
