// A thread's eight columns of a row, and their loads and stores at any
// alignment, for kernels that give neighbouring vectors of a row to the lanes of
// a warp (mx8.cu, rms_norm.cu, embedding.cu).
#pragma once

#include "mx4_quant.cuh"
#include "mx8.cuh"

namespace zsm {
namespace mx {

// Eight neighbouring columns.  kWhole: the row is made of whole, 16-byte
// aligned vectors.  Rows are given by their address and columns in 32 bits:
// these kernels are bound by instructions as much as by memory, and 64-bit
// products of rows and pitches for every access were a third of them.
template <bool kWhole>
struct Columns {
  uint32_t first, cols;
  __device__ __forceinline__ Columns(uint32_t base, uint32_t vector, uint32_t n) : first(base + 8 * vector), cols(n) {}
  __device__ __forceinline__ bool any() const { return first < cols; }
  __device__ __forceinline__ bool in(int j) const { return kWhole ? first < cols : first + j < cols; }
};

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

// Rows that are not aligned (every row but the first of a matrix with an odd
// number of columns) are read in their aligned 16-byte words all the same: a
// lane reads the word that its vector begins in and the next one, most of
// which is in L1 then, and shifts the two by the row's offset, which is the
// same for all lanes.  (Loading a vector as eight elements took four times the
// instructions.)  A word may reach past the row's ends, into what lies before
// or after it in the matrix; those elements are dropped, whatever another
// block is writing there.  It never reaches past the matrix: such a word is
// read element by element.

// Words of kPer elements each, moved down by `by` elements (less than four words).
template <int kWords, int kPer>
__device__ __forceinline__ void shift_down(uint32_t (&w)[kWords], uint32_t by) {
#pragma unroll
  for (int i = 0; i + 2 < kWords; ++i) w[i] = by & (2u * kPer) ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i + 1 < kWords; ++i) w[i] = by & kPer ? w[i + 1] : w[i];
  if constexpr (kPer == 2) {
    const uint32_t bits = 16u * (by & 1u);
#pragma unroll
    for (int i = 0; i + 1 < kWords; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], bits);
  }
}

template <class V>
struct WordsOf;  // how a vector lies in words
template <class F>
struct WordsOf<Vec16<F>> {
  static constexpr int kN = 4, kPer = 2;
};
template <>
struct WordsOf<Vec32> {
  static constexpr int kN = 8, kPer = 1;
};
template <class V>
__device__ __forceinline__ uint32_t (&words(V& x))[WordsOf<V>::kN] {
  return reinterpret_cast<uint32_t(&)[WordsOf<V>::kN]>(x);
}
template <class V>
__device__ __forceinline__ const uint32_t (&words(const V& x))[WordsOf<V>::kN] {
  return reinterpret_cast<const uint32_t(&)[WordsOf<V>::kN]>(x);
}

// The elements by which a row is past a 16-byte boundary.
template <class raw>
__device__ __forceinline__ uint32_t offset_of(const raw* row) {
  return (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u) / (uint32_t)sizeof(raw);
}

// A matrix's memory, from its first to behind its last element.
struct Span {
  uintptr_t lo, hi;
  __device__ __forceinline__ bool holds(const uint4* word) const {
    return reinterpret_cast<uintptr_t>(word) >= lo && reinterpret_cast<uintptr_t>(word) + 16 <= hi;
  }
  // Whether all 16-byte words with an element of a row are the matrix's (of all
  // rows but the first and the last they are).
  template <class raw>
  __device__ __forceinline__ bool holds(const raw* row, uint32_t cols, uint32_t off) const {
    const uintptr_t from = reinterpret_cast<uintptr_t>(row) - sizeof(raw) * off;
    return from >= lo && from + sizeof(raw) * ((off + cols + (16 / sizeof(raw) - 1)) & ~(uint32_t)(16 / sizeof(raw) - 1)) <= hi;
  }
};
template <class T>
__device__ __forceinline__ Span span_of(const void* m, int64_t rows, int64_t cols, int64_t ld) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(m);
  return {lo, lo + sizeof(typename T::raw) * ((rows - 1) * ld + cols)};
}

// A vector as it was loaded: its words, and the ones after them for an
// unaligned row.
template <class V, bool kWhole>
struct Fetched {
  static constexpr int kN = WordsOf<V>::kN, kAll = kWhole ? kN : kN + 4;
  uint32_t w[kAll];
};

// Sixteen bytes at an aligned address, of which only those within the span are
// read.
template <int kPer>
__device__ __noinline__ uint4 load_within(uintptr_t at, Span m) {
  uint32_t e[4 * kPer];
#pragma unroll
  for (int j = 0; j < 4 * kPer; ++j) {
    const uintptr_t p = at + (4 / kPer) * j;
    e[j] = 0u;
    if (p >= m.lo && p < m.hi) e[j] = kPer == 2 ? *reinterpret_cast<const uint16_t*>(p) : *reinterpret_cast<const uint32_t*>(p);
  }
  if constexpr (kPer == 2) return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
  else return make_uint4(e[0], e[1], e[2], e[3]);
}

template <class V, bool kWhole>
__device__ __forceinline__ void fetch_columns(Fetched<V, kWhole>& f, const typename V::raw* row, const Columns<kWhole>& c,
                                              const Span& m) {
  constexpr int kN = Fetched<V, kWhole>::kN;
  if constexpr (kWhole) {
    V x;
    if (c.any()) x.load(row + c.first);
    else x.clear();
#pragma unroll
    for (int i = 0; i < kN; ++i) f.w[i] = words(x)[i];
  } else {
    const uint32_t off = offset_of(row);
    const bool inside = m.holds(row, c.cols, off);  // (the same for the whole warp)
    const uint4* from = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(row + c.first) & ~(uintptr_t)15);
    constexpr uint32_t kIn = 16 / sizeof(typename V::raw);
#pragma unroll
    for (int i = 0; i < kN / 4 + 1; ++i) {
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (c.first + kIn * i < c.cols + off) {  // the word holds an element of the row
        if (inside || m.holds(from + i)) x = from[i];
        else x = load_within<WordsOf<V>::kPer>(reinterpret_cast<uintptr_t>(from + i), m);
      }
      f.w[4 * i] = x.x, f.w[4 * i + 1] = x.y, f.w[4 * i + 2] = x.z, f.w[4 * i + 3] = x.w;
    }
  }
}

// The vector: 0 past the row's end.
template <class V, bool kWhole>
__device__ __forceinline__ void take_columns(V& x, Fetched<V, kWhole>& f, uint32_t off, const Columns<kWhole>& c) {
  constexpr int kN = Fetched<V, kWhole>::kN, kPer = WordsOf<V>::kPer;
  if constexpr (!kWhole) shift_down<kN + 4, kPer>(f.w, off);
#pragma unroll
  for (int i = 0; i < kN; ++i) words(x)[i] = f.w[i];
  if constexpr (!kWhole) {
    if (!c.in(7)) {
      const uint32_t left = c.any() ? c.cols - c.first : 0u;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        if (kPer * i >= (int)left) words(x)[i] = 0u;
        else if (kPer == 2 && 2 * i + 1 >= (int)left) words(x)[i] &= 0xFFFFu;
      }
    }
  }
}

template <class V, bool kWhole>
__device__ __forceinline__ void take_columns(V& x, Fetched<V, kWhole>& f, const typename V::raw* row, const Columns<kWhole>& c) {
  take_columns(x, f, kWhole ? 0u : offset_of(row), c);
}

// Both at once.
template <class V, bool kWhole>
__device__ __forceinline__ void load_columns(V& x, const typename V::raw* row, const Columns<kWhole>& c, const Span& m) {
  Fetched<V, kWhole> f;
  fetch_columns(f, row, c, m);
  take_columns(x, f, row, c);
}

// A vector as it is, into its row: an unaligned one's words are put together
// from two neighbouring lanes' vectors; what a warp's first and last lanes lack a
// neighbour for -- eight elements of 16 bits, four of 32 -- goes to as many lanes
// and out in one store; the row's last word goes element by element.  Called by
// whole warps, every kLanes of which have neighbouring vectors of a row.
__device__ __forceinline__ void store_whole(uint16_t* p, const uint32_t* w) {
  st_stream(p, make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void store_whole(float* p, const uint32_t* w) {
  // one 32-byte store where that is aligned: of two of 16 each would touch every sector of the warp's
  if ((reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
    asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
    return;
  }
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  __stcs(reinterpret_cast<uint4*>(p) + 1, make_uint4(w[4], w[5], w[6], w[7]));
}
template <class raw>
__device__ __forceinline__ void store_some(raw* p, const uint32_t* w, int from, int to) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j < from || j >= to) continue;
    if constexpr (sizeof(raw) == 2) p[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
    else p[j] = __uint_as_float(w[j]);
  }
}

template <int kLanes = 32, class V, bool kWhole>
__device__ __forceinline__ void store_columns(typename V::raw* row, const Columns<kWhole>& c, const V& x) {
  using raw = typename V::raw;
  constexpr int kN = WordsOf<V>::kN, kPer = WordsOf<V>::kPer;
  if constexpr (kWhole) {
    if (c.any()) store_whole(row + c.first, words(x));
  } else {
    static_assert(kLanes >= 8, "a word's elements have a lane each");
    const uint32_t off = offset_of(row), lane = threadIdx.x & (kLanes - 1);
    // (rows of one warp may begin at different offsets in their words)
    const uint32_t mask = kLanes == 32 ? 0xFFFFFFFFu : ((1u << (kLanes & 31)) - 1u) << (threadIdx.x & 31 & ~(kLanes - 1));
    const int there = (int)(c.cols - c.first);  // elements of the row from mine on (below 0: it ended before)
    if (off == 0) {
      if (there >= 8) store_whole(row + c.first, words(x));
      else store_some(row + c.first, words(x), 0, there);
      return;
    }
    // the neighbour's last elements before mine: of both vectors one after
    // another what is from 8 - off on
    uint32_t w[kN + 4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __shfl_up_sync(mask, words(x)[kN - 4 + i], 1, kLanes);
#pragma unroll
    for (int i = 0; i < kN; ++i) w[4 + i] = words(x)[i];
    shift_down<kN + 4, kPer>(w, 4 * kPer - off);
    raw* p = row + (int64_t)c.first - off;  // elements -off .. 7 - off of mine
    const int end = min(there + (int)off, 8);
    if (end == 8) {
      if (lane > 0) store_whole(p, w);
      else if constexpr (kN == 8) __stcs(reinterpret_cast<uint4*>(p) + 1, make_uint4(w[4], w[5], w[6], w[7]));
    } else if (end > 0) {
      store_some(p, w, lane > 0 ? 0 : (int)off, end);
    }
    // lane j: of the elements that begin the first lane's vector and end the last one's, in a word each, the jth
    constexpr uint32_t kIn = 16 / sizeof(raw);  // elements of a word
    const bool last = lane >= kIn - off;
    uint32_t e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t mine = lane == kLanes - 1 ? words(x)[kN - 4 + i] : words(x)[i];
      e[i] = __shfl_sync(mask, mine, last ? kLanes - 1 : 0, kLanes);
    }
    const int first_there = __shfl_sync(mask, there, 0, kLanes);
    const uint32_t at = last ? kLanes * 8 - kIn + lane : lane;  // from the first lane's first column on
    // (of a lane 0 whose word the row's end is in, the elements have gone out above)
    if (lane < kIn && (int)at < first_there && (last || first_there + (int)off >= 8)) {
      const uint32_t i = lane / kPer;
      const uint32_t v = i < 2 ? (i < 1 ? e[0] : e[1]) : (i < 3 ? e[2] : e[3]);
      raw* q = row + (c.first - 8 * lane) + at;
      if constexpr (kPer == 2) *q = (uint16_t)(v >> (16 * (lane & 1)));
      else *q = __uint_as_float(v);
    }
  }
}

// Pairs at once.  (The assembler rounds a packed product and the packed sum that
// takes it once, as a multiply-add, in spite of .rn on both: where the two meet
// the multiply-add is written, so that it does not depend on the code around.)
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
  return d;
}
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

__device__ __forceinline__ void plus8(float (&v)[8], const float (&w)[8]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 f = add2(pair(v, p), pair(w, p));
    v[2 * p] = f.x, v[2 * p + 1] = f.y;
  }
}

// v s + w
__device__ __forceinline__ void scale_plus8(float (&v)[8], float s, const float (&w)[8]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 f = fma2(pair(v, p), make_float2(s, s), pair(w, p));
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

// An MX8 row's codes and scale byte at a thread's columns.
struct Fetched8 {
  uint2 w;
  uint32_t s;
};
template <bool kWhole>
__device__ __forceinline__ void fetch_columns8(Fetched8& f, const Row8& row, const Columns<kWhole>& c) {
  f.w = make_uint2(0u, 0u), f.s = 0u;
  if (!c.any()) return;
  f.w = __ldcs(reinterpret_cast<const uint2*>(row.codes + c.first));
  f.s = row.scales[c.first >> 5];
}
// Its values, 0 past its end, in multiples of `unit` (a power of two or any
// other number: one rounding).
template <bool kWhole>
__device__ __forceinline__ void take_columns8(float (&v)[8], const Fetched8& f, const Columns<kWhole>& c, float unit) {
  elements8(f.w, v);
  scale8(v, __fmul_rn(scale_value(f.s), unit));
  if constexpr (!kWhole) {
    if (!c.in(7)) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!c.in(j)) v[j] = 0.0f;  // (what fills up the last block is not the row's)
    }
  }
}

// A vector of a row, 0 past its end, into an MX8 row; v holds x's values.
// Called by whole warps whose lanes have neighbouring vectors.
template <class V, bool kWhole>
__device__ __forceinline__ void store_columns8(const Row8& row, const Columns<kWhole>& c, const V& x, const float (&v)[8]) {
  const uint32_t s = scale_code8(max_of_four(x.max_bits()));
  if (c.first >= ((c.cols + 31u) & ~31u)) return;
  *reinterpret_cast<uint2*>(row.codes + c.first) = encode8_mx8(v, s);
  if ((c.first & 31u) == 0) row.scales[c.first >> 5] = (uint8_t)s;
}

// A vector of one of the three types at a thread's columns, 0 past its end.
// `vec`: it is 16-byte aligned.
template <bool kWhole>
__device__ __forceinline__ void load_weights(const void* w, int type, bool vec, const Columns<kWhole>& c, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  if (kWhole || (vec && c.in(7))) {
    if (!c.any()) return;
    if (type == kMxF32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + c.first);
      const float4 a = __ldg(p), b = __ldg(p + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
      return;
    }
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + c.first));
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
    if (type == kMxBf16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[2 * j] = Bf16::lo(u[j]), v[2 * j + 1] = Bf16::hi(u[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[2 * j] = F16::lo(u[j]), v[2 * j + 1] = F16::hi(u[j]);
    }
    return;
  }
  if constexpr (!kWhole) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!c.in(j)) continue;
      if (type == kMxF32) {
        v[j] = __ldg(static_cast<const float*>(w) + c.first + j);
      } else {
        const uint16_t u = __ldg(static_cast<const uint16_t*>(w) + c.first + j);
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
// (for words that a neighbour copies too)
__device__ __forceinline__ void copy_async16_shared(void* to, uintptr_t from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
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
