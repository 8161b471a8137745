// Root-mean-square norm, forward and backward (rms_norm.cuh has the formulas).
//
// Both are memory-bound: forward 2 to 4 values of the row's type and up to two
// MX8 bytes an element, backward 3 or 4.  Elements of rows of up to 16384 columns
// forward, 4096 backward, are read once: they stay in registers (forward) or
// shared memory (backward), as they were loaded, between the sum over the row and
// its use.  Longer rows are read twice.
#include <cuda_runtime.h>

#include <type_traits>

#include "rms_norm.cuh"
#include "rows.cuh"

namespace zsm {
namespace {

using namespace mx;

// ----------------------------------------------------------------- forward --

// The row's sum: of every 32 neighbouring vectors in binary32 in one order, of
// those in binary64 in theirs, so that its bits are the same whether a thread has
// one vector or two, and with them a row's results in every batch.  kLanes of a
// warp share the row (0: the block does); every thread of it gets the sum.  A
// warp adds up two sums in its halves, after one exchange: as many shuffles as
// for one.
template <int kLanes, int kSums>
__device__ __forceinline__ double group_sum(const float (&of)[kSums], float* smem) {
  static_assert(kSums == 1 || (kSums == 2 && (kLanes == 0 || kLanes == 32)), "halves of warps");
  const bool upper = kSums == 2 && (threadIdx.x & 16);
  float mine = upper ? of[kSums - 1] : of[0];
  if constexpr (kSums == 2) mine = __fadd_rn(mine, __shfl_xor_sync(0xFFFFFFFFu, upper ? of[0] : of[1], 16));
#pragma unroll
  for (int o = (kLanes ? kLanes / 2 : 16) / kSums; o > 0; o >>= 1) mine = __fadd_rn(mine, __shfl_xor_sync(0xFFFFFFFFu, mine, o));
  if constexpr (kLanes > 0) {
    if constexpr (kSums == 1) return (double)mine;
    return __dadd_rn((double)mine, (double)__shfl_xor_sync(0xFFFFFFFFu, mine, 16));
  }
  const uint32_t warps = blockDim.x / 32, n = warps * kSums;  // up to 32
  if ((threadIdx.x & (32 / kSums - 1)) == 0) smem[(upper ? warps : 0) + (threadIdx.x >> 5)] = mine;
  __syncthreads();
  // (a tree: every thread adding up all of them took 3 us more of 31 at 2048 x 8192)
  const uint32_t powers = n > 1 ? 1u << (32 - __clz(n - 1)) : 1u, w = threadIdx.x & (powers - 1);
  double v = w < n ? (double)smem[w] : 0.0;
  for (uint32_t o = powers / 2; o > 0; o >>= 1) v = __dadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// rstd = m^(-1/2), m = ss / cols + eps: the function's binary32 estimate and one
// Newton step in binary64, whose error is the square of the estimate's, rounded to
// binary32 once.  (y's rounding to 16 and then to 8 bits turns on rstd's last bit
// now and then.  The sum that m comes from is binary32's of 256 columns each: of
// normal numbers 8 rstd in a hundred of rows of 4096 are not the correctly rounded
// ones, 15 of rows of 512.)
__device__ __forceinline__ double root_of(double m) {
  const float r = rsqrtf((float)m);
  const double e = __fma_rn(-__dmul_rn(m, (double)r), (double)r, 1.0);
  return __fma_rn(__dmul_rn(0.5, e), (double)r, (double)r);
}

// Whether m is below 2^-100, 2^126 and more, infinite or not a number: near or past
// the ends of binary32, as the squares may have been.
__device__ __forceinline__ bool is_far(double m) {
  return (uint32_t)__double2hiint(m) - ((1023u - 100u) << 20) >= 226u << 20;
}
// rstd of any m: moved by a power of four.
__device__ __forceinline__ float far_root_of(double m) {
  if (isinf(m)) return 0.0f;
  const bool above = m > 1.0;
  return (float)__dmul_rn(root_of(__dmul_rn(m, above ? 0x1p-160 : 0x1p160)), above ? 0x1p-80 : 0x1p80);
}
// The squares of such a row are added up once more in units of 2^80 or 2^-80.
// Above, where one |h| is 2^64 or 256 are 2^60, no sum of up to 2^31 columns is
// infinite then; below, where the mean counts beside an eps of that size, no square
// that counts is lost.  (Binary16's squares, 2^-48 to 2^32, are right as
// they are.)
__device__ __forceinline__ float unit_of(double m) { return m > 1.0 ? 0x1p-80f : 0x1p80f; }
__device__ __forceinline__ double in_units(double ss, float unit) { return __dmul_rn(ss, unit < 1.0f ? 0x1p160 : 0x1p-160); }

// The addresses of a row of the operands and results.
template <class T>
struct NormRow {
  using raw = typename T::raw;
  const raw *x, *r;
  raw *h, *y;
  Row8 h8, y8;
  __device__ __forceinline__ NormRow(const RmsNormArgs& a, int64_t row)
      : x(row_of<T>(a.x, row, a.ld_x)), r(row_of<T>(a.residual, row, a.ld_residual)), h(row_of<T>(a.h, row, a.ld_h)),
        y(row_of<T>(a.y, row, a.ld_y)), h8(row_of(a.h8, row)), y8(row_of(a.y8, row)) {}
};

// Vectors of one row of h: x plus the residual, rounded to their type.  All
// loads go out before the first is waited for.
template <class T, bool kWhole, int kN>
__device__ __forceinline__ void load_h(const RmsNormArgs& a, const NormRow<T>& row, const Columns<kWhole> (&c)[kN],
                                       typename T::V (&x)[kN]) {
  Fetched<typename T::V, kWhole> fx[kN], fr[kN];
#pragma unroll
  for (int k = 0; k < kN; ++k) fetch_columns(fx[k], row.x, c[k], span_of<T>(a.x, a.rows, a.cols, a.ld_x));
  if (a.residual) {
#pragma unroll
    for (int k = 0; k < kN; ++k) fetch_columns(fr[k], row.r, c[k], span_of<T>(a.residual, a.rows, a.cols, a.ld_residual));
  }
#pragma unroll
  for (int k = 0; k < kN; ++k) take_columns(x[k], fx[k], row.x, c[k]);
  if (a.residual) {
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      typename T::V r;
      take_columns(r, fr[k], row.r, c[k]);
      add_to(x[k], r);
    }
  }
}

__device__ __forceinline__ float2 square_sum(const float (&v)[8], float2 ss) {
#pragma unroll
  for (int p = 0; p < 4; ++p) ss = fma2(pair(v, p), pair(v, p), ss);
  return ss;
}

// For a row that is far: a vector's squares in units, by a call, so that this rare
// way takes no registers from the other (inlined, 6000 x 2421 bf16 took 47.1 us
// instead of 46.2).
template <class V>
__device__ __noinline__ float far_squares(const V x, float unit) {
  float v[8];
  x.values(v);
  scale8(v, unit);
  const float2 ss = square_sum(v, make_float2(0.0f, 0.0f));
  return __fadd_rn(ss.x, ss.y);
}
// Of aligned rows the values are formed anew after it: kept in registers past it,
// 8192 x 4096 with all results took 59.7 us instead of 54.9.  (Unaligned ones have
// them in registers anyway.)
template <class V, int kN>
__device__ __forceinline__ void as_loaded(V (&x)[kN]) {
#pragma unroll
  for (int k = 0; k < kN; ++k)
#pragma unroll
    for (int i = 0; i < WordsOf<V>::kN; ++i) asm volatile("" : "+r"(words(x[k])[i]));
}

// All results of one vector of h.  Called by whole warps.
template <class T, int kLanes, class C>
__device__ __forceinline__ void finish(const RmsNormArgs& a, const NormRow<T>& row, const C& c, float rstd,
                                       const typename T::V& x) {
  float v[8], w[8];
  x.values(v);
  if (a.h) store_columns<kLanes>(row.h, c, x);
  if (a.h8.codes) store_columns8(row.h8, c, x, v);
  if (!a.y && !a.y8.codes) return;
  load_weights(a.weight, a.w_type, a.w_aligned, c, w);
  scale8(v, rstd);
  times8(v, w);
  typename T::V y;
  round_to(y, v);
  if (a.y) store_columns<kLanes>(row.y, c, y);
  if (a.y8.codes) {
    if (!isfinite(rstd)) {  // past the row x and w are 0, but 0 times this is not
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!c.in(j)) v[j] = 0.0f;
      round_to(y, v);
    }
    y.values(v);
    store_columns8(row.y8, c, y, v);
  }
}

// A block to a row, or kLanes of a warp, kChunks vectors of eight elements a
// thread; the host picks the block's threads to fit the row.  Blocks that end
// make room for others whose loads go out at once, so that nothing has to be
// fetched ahead: 8192 x 4096 bf16 with a residual and all results, 338 MB, takes
// 55 us, 52 at the copy's rate (with 64-bit addresses for every access and single
// products 70), issue slots 75 % busy; without MX8 41.7 of 41.0.  Rows of odd
// length, 6000 x 2421 binary16 with all results, take 46 of 22: instructions.  One
// token of 4096 takes 2.6, its launch and two trips to memory.
constexpr int kLanesThreads = 128;  // of a block whose warps have rows of their own
template <class T, bool kWhole, int kLanes, int kChunks>
__global__ void __launch_bounds__(kLanes ? kLanesThreads : 512) rms_norm_kernel(const __grid_constant__ RmsNormArgs a,
                                                                                const double inv_cols) {
  static_assert(kLanes % 4 == 0, "whole blocks of MX8");
  constexpr int kSums = kChunks == 4 ? 1 : kChunks;  // (of four a thread, each thread's at once: rows that always go so)
  __shared__ float smem[512 / 32 * kSums];
  const uint32_t group = kLanes ? kLanes : blockDim.x, t = kLanes ? threadIdx.x & (kLanes - 1) : threadIdx.x;
  const uint32_t number = kLanes ? blockIdx.x * (kLanesThreads / group) + threadIdx.x / group : blockIdx.x;
  const bool there = kLanes == 0 || number < (uint32_t)a.rows;  // past the end: a row of no columns, for the shuffles' sake
  const NormRow<T> row(a, there ? number : 0);
  const uint32_t cols = there ? (uint32_t)a.cols : 0u;
  using C = Columns<kWhole>;
  typename T::V x[kChunks];
  if constexpr (kChunks == 1) {
    const C c[1] = {C(0, t, cols)};
    load_h<T>(a, row, c, x);
  } else {
#pragma unroll
    for (int k = 0; k < kChunks; k += 2) {
      const C c[2] = {C(8 * group * k, t, cols), C(8 * group * (k + 1), t, cols)};
      load_h<T>(a, row, c, reinterpret_cast<typename T::V(&)[2]>(x[k]));
    }
  }
  float ss[kSums];
  float2 of = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    float v[8];
    x[k].values(v);
    of = square_sum(v, kSums == 1 ? of : make_float2(0.0f, 0.0f));
    ss[kSums == 1 ? 0 : k] = __fadd_rn(of.x, of.y);
  }
  const double m = __fma_rn(group_sum<kLanes>(ss, smem), inv_cols, (double)a.eps);
  float rstd;
  if (kLanes ? __any_sync(0xFFFFFFFFu, is_far(m)) : is_far(m)) {  // (whole warps, or the whole block)
    double far = m;
    if constexpr (!std::is_same<T, TF16>::value) {
      const float unit = unit_of(m);
      if constexpr (kWhole) as_loaded(x);
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const float f = far_squares(x[k], unit);
        ss[kSums == 1 ? 0 : k] = kSums == 1 && k > 0 ? __fadd_rn(ss[0], f) : f;
      }
      if constexpr (kLanes == 0) __syncthreads();  // (the first sum's shared memory)
      far = __fma_rn(in_units(group_sum<kLanes>(ss, smem), unit), inv_cols, (double)a.eps);
    }
    rstd = is_far(m) ? far_root_of(far) : (float)root_of(m);
  } else {
    rstd = (float)root_of(m);
  }
  if (a.rstd && t == 0 && there) a.rstd[number] = rstd;
#pragma unroll
  for (int k = 0; k < kChunks; ++k) finish<T, kLanes ? kLanes : 32>(a, row, C(8 * group * k, t, cols), rstd, x[k]);
}

// Rows too long for registers: read a second time (a thread reads its own
// elements before it writes results in their place).
constexpr int kLongThreads = 512;
template <class T, bool kWhole>
__global__ void __launch_bounds__(kLongThreads) rms_norm_long_kernel(const __grid_constant__ RmsNormArgs a,
                                                                     const double inv_cols) {
  __shared__ float smem[kLongThreads / 32];
  const NormRow<T> row(a, blockIdx.x);
  const uint32_t cols = (uint32_t)a.cols;
  using C = Columns<kWhole>;
  auto row_sum = [&](auto far, float unit) {  // (of a far row in units)
    float2 ss = make_float2(0.0f, 0.0f);
    for (uint32_t first = 0; first < cols; first += 8 * kLongThreads) {
      typename T::V x[1];
      const C c[1] = {C(first, threadIdx.x, cols)};
      float v[8];
      load_h<T>(a, row, c, x);
      x[0].values(v);
      if constexpr (decltype(far)::value) scale8(v, unit);
      ss = square_sum(v, ss);
    }
    float sum[1] = {__fadd_rn(ss.x, ss.y)};
    return group_sum<0>(sum, smem);
  };
  const double m = __fma_rn(row_sum(std::false_type(), 1.0f), inv_cols, (double)a.eps);
  float rstd;
  if (is_far(m)) {
    __syncthreads();  // (the sum's shared memory)
    const float unit = unit_of(m);
    rstd = far_root_of(__fma_rn(in_units(row_sum(std::true_type(), unit), unit), inv_cols, (double)a.eps));
  } else {
    rstd = (float)root_of(m);
  }
  if (a.rstd && threadIdx.x == 0) a.rstd[blockIdx.x] = rstd;
  for (uint32_t first = 0; first < cols; first += 8 * kLongThreads) {
    typename T::V x[1];
    const C c[1] = {C(first, threadIdx.x, cols)};
    load_h<T>(a, row, c, x);
    finish<T, 32>(a, row, c[0], rstd, x[0]);
  }
}

// ---------------------------------------------------------------- backward --

// A block walks over rows block, block + blocks, ... and keeps its columns'
// part of dw in registers; the parts go to the workspace, one row of it a
// block, and a second kernel adds them in order.
//
// The rows come through a ring in shared memory, two to four rows deep, by
// asynchronous copies: each thread fetches the words that it reads itself (of
// an unaligned row one more than it has, which its neighbour fetches too), so
// that nothing but its own copies has to be waited for, and the sum over a row
// -- the one place where the block's threads meet -- never holds up the loads of
// the next ones.  8192 x 4096 bf16 from the checkpoint, with dh: 50 us with dw's
// second kernel (36 at the copy's rate; with loads into registers 103): issue
// slots 65 % busy, the rest is the sum's chain of shuffles and a barrier a row.
// (Two vectors a thread in three blocks of 256 threads have a fifth fewer
// instructions and took 56: fewer warps to hide that chain behind.)
constexpr int64_t kSms = 148;
constexpr uint32_t kMaxThreads = 512;

// The longest rows that a block takes, a vector a thread; longer ones go through
// memory twice (see below).
constexpr int64_t kRingCols = 8 * kMaxThreads;

// Threads of a block, blocks to an SM (the kernel's registers allow 1024
// threads), and blocks at most: as many as are there at a time.
uint32_t threads_of(int64_t cols) { return (uint32_t)((cols + 255) / 256 * 32); }
uint32_t blocks_to_sm(int64_t cols) { return std::min(1024 / threads_of(cols), 16u); }
int64_t parts_of(int64_t rows, int64_t cols) {
  // four rows a block where that leaves every SM one: a block's start and its
  // part of dw cost as much as some rows do (1237 x 771: one row a block 14 us)
  const int64_t few = std::max((rows + 3) / 4, std::min(rows, kSms));
  return std::max<int64_t>(1, std::min(few, kSms * blocks_to_sm(cols)));
}

// Sum over the block in binary32 (smem holds two rounds' values, so that one
// barrier a round will do), or over the kLanes of a warp that share a row.
template <int kLanes>
__device__ __forceinline__ float block_sum(float v, float (*smem)[32], int round) {
#pragma unroll
  for (int o = kLanes ? kLanes / 2 : 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  if constexpr (kLanes > 0) return v;
  const uint32_t lane = threadIdx.x & 31, warps = blockDim.x / 32;
  if (warps == 1) return v;
  if (lane == 0) smem[round & 1][threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? smem[round & 1][lane] : 0.0f;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return __shfl_sync(0xFFFFFFFFu, v, 0);
}
static_assert(kMaxThreads <= 512, "sixteen warps at most are added");

// One vector's part of a row's sum of g xh, and of dw; dy becomes g.
__device__ __forceinline__ void add_vector(float (&dy)[8], const float (&xh)[8], const float (&w)[8], float2 (&acc)[4],
                                           float2& dot) {
#pragma unroll
  for (int p = 0; p < 4; ++p) acc[p] = fma2(pair(dy, p), pair(xh, p), acc[p]);
  times8(dy, w);
#pragma unroll
  for (int p = 0; p < 4; ++p) dot = fma2(pair(dy, p), pair(xh, p), dot);
}

// g - xh mean of one vector, in g's place.
__device__ __forceinline__ void dx_vector(float (&g)[8], const float (&xh)[8], float mean) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 d = fma2(pair(xh, p), make_float2(-mean, -mean), pair(g, p));
    g[2 * p] = d.x, g[2 * p + 1] = d.y;
  }
}

// The rows of a block at a time: of one warp, kLanes to a row, or (0) one.
__host__ __device__ constexpr int rows_at_once(int lanes) { return lanes ? 32 / lanes : 1; }

// dx of that, rounded: times rstd, plus dh (a vector of the type) if there is one.
template <class T, int kLanes, class C>
__device__ __forceinline__ void store_dx(typename T::raw* row, const C& c, float rstd, const typename T::V* dh, float (&v)[8]) {
  if (dh) {
    float u[8];
    dh->values(u);
    scale_plus8(v, rstd, u);
  } else {
    scale8(v, rstd);
  }
  typename T::V x;
  round_to(x, v);
  store_columns<kLanes>(row, c, x);
}

template <class C, class A>
__device__ __forceinline__ void store_part(float* out, const C& c, const A& acc) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c.in(j)) out[c.first + j] = j & 1 ? acc[j >> 1].y : acc[j >> 1].x;
}

// One row's stage of the ring: dy, dh, h of every thread's vectors, 16 bytes of
// each thread next to another's.
template <class T, bool kWhole, bool kMx8, bool kDh>
struct Ring {
  using V = typename T::V;
  using raw = typename T::raw;
  static constexpr int kWords = sizeof(raw) / 2 + (kWhole ? 0 : 1);  // 16-byte words fetched of a vector
  static constexpr uint32_t kPlanes = kWords * (1 + (kMx8 ? 0 : 1) + (kDh ? 1 : 0));
  // bytes of a stage for so many vectors, and where dh's and h's words begin
  static __host__ __device__ __forceinline__ uint32_t bytes(uint32_t vectors) { return vectors * (16 * kPlanes + (kMx8 ? 8 : 0)); }
  static __device__ __forceinline__ uint32_t dh_at(uint32_t vectors) { return 16 * kWords * vectors; }
  static __device__ __forceinline__ uint32_t h_at(uint32_t vectors) { return 16 * kWords * vectors * (kDh ? 2 : 1); }

  // The rows' addresses, moved on from row to row.
  struct Rows {
    const raw *dy, *dh, *h;
    const uint8_t* codes;
    __device__ __forceinline__ Rows(const RmsNormBackwardArgs& a, int64_t row)
        : dy(row_of<T>(a.dy, row, a.ld_dy)), dh(row_of<T>(a.dh, row, a.ld_dh)), h(row_of<T>(a.h, row, a.ld_h)),
          codes(a.h8.codes + row * a.h8.code_pitch) {}
    __device__ __forceinline__ void next(const RmsNormBackwardArgs& a, uint32_t step) {
      dy += step * a.ld_dy;
      if constexpr (kDh) dh += step * a.ld_dh;
      if constexpr (kMx8) codes += step * a.h8.code_pitch;
      else h += step * a.ld_h;
    }
  };

  static __device__ __forceinline__ void fetch16(uint8_t* to, uint32_t vectors, const raw* row, const Columns<kWhole>& c,
                                                 const void* m, uintptr_t m_end) {
    if constexpr (kWhole) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) copy_async16(to + 16 * i * vectors, row + c.first + 16 / (int)sizeof(raw) * i);
    } else {
      const Span span = {reinterpret_cast<uintptr_t>(m), m_end};
      const uint32_t off = offset_of(row);
      const bool inside = span.holds(row, c.cols, off);
      const uintptr_t from = reinterpret_cast<uintptr_t>(row + c.first) & ~(uintptr_t)15;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        if (c.first + 16 / (uint32_t)sizeof(raw) * i >= c.cols + off) break;
        if (inside || span.holds(reinterpret_cast<const uint4*>(from + 16 * i))) copy_async16_shared(to + 16 * i * vectors, from + 16 * i);
        else *reinterpret_cast<uint4*>(to + 16 * i * vectors) = load_within<WordsOf<V>::kPer>(from + 16 * i, span);
      }
    }
  }
  // Asks for a row if there is one; the group is there all the same.
  static __device__ __forceinline__ void fetch(const RmsNormBackwardArgs& a, const Rows& row, const Columns<kWhole>& c,
                                               bool there, uint8_t* to) {
    if (there && c.any()) {
      const uint32_t vectors = blockDim.x, v = threadIdx.x;
      fetch16(to + 16 * v, vectors, row.dy, c, a.dy, a.dy_end);
      if constexpr (kDh) fetch16(to + dh_at(vectors) + 16 * v, vectors, row.dh, c, a.dh, a.dh_end);
      if constexpr (kMx8) copy_async8(to + h_at(vectors) + 8 * v, row.codes + c.first);
      else fetch16(to + h_at(vectors) + 16 * v, vectors, row.h, c, a.h, a.h_end);
    }
    copy_async_commit();
  }
  // The elements by which row `row` of a matrix is past a 16-byte boundary.
  static __device__ __forceinline__ uint32_t offset(const void* m, uint32_t row, int64_t ld) {
    if constexpr (kWhole) return 0u;
    const uint32_t bytes = (uint32_t)reinterpret_cast<uintptr_t>(m) + row * ((uint32_t)ld * (uint32_t)sizeof(raw));
    return (bytes & 15u) / (uint32_t)sizeof(raw);
  }
  static __device__ __forceinline__ void read(const uint8_t* at, uint32_t vectors, uint32_t off, const Columns<kWhole>& c, V& x) {
    Fetched<V, kWhole> f;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const uint4 w = *reinterpret_cast<const uint4*>(at + 16 * i * vectors);
      f.w[4 * i] = w.x, f.w[4 * i + 1] = w.y, f.w[4 * i + 2] = w.z, f.w[4 * i + 3] = w.w;
    }
    take_columns(x, f, off, c);
  }
};

// xh and g stay in registers over the sum.  kLanes: a block of one warp, that many
// lanes to a row (0: the block to a row).
template <class T, bool kWhole, bool kMx8, bool kDh, int kLanes>
__global__ void __launch_bounds__(kMaxThreads, 2)
    rms_norm_backward_kernel(const __grid_constant__ RmsNormBackwardArgs a, const int stages) {
  using R = Ring<T, kWhole, kMx8, kDh>;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float smem[2][32];
  pdl_trigger();
  constexpr uint32_t kRows = rows_at_once(kLanes);
  const uint32_t lane = kLanes ? threadIdx.x % (32 / kRows) : threadIdx.x;
  const uint32_t first = blockIdx.x * kRows + (kLanes ? threadIdx.x / (32 / kRows) : 0);
  const uint32_t step = gridDim.x * kRows, rows = (uint32_t)a.rows, vectors = blockDim.x, size = R::bytes(vectors);
  const Columns<kWhole> c(0, lane, (uint32_t)a.cols);
  uint32_t ahead = first;  // the row to ask for
  typename R::Rows from(a, first);
  for (int s = 0; s < stages - 1; ++s, ahead += step) {
    R::fetch(a, from, c, ahead < rows, ring + s * size);
    from.next(a, step);
  }
  float2 acc[4];
  float w[8];
#pragma unroll
  for (int p = 0; p < 4; ++p) acc[p] = make_float2(0.0f, 0.0f);
  load_weights(a.weight, a.w_type, a.w_aligned, c, w);
  const float inv = __fdiv_rn(1.0f, (float)a.cols);
  // the row's statistics and scales, a row ahead
  const float* stats = a.rstd + first;
  const uint8_t* scales = a.h8.scales + first * a.h8.scale_pitch + (c.first >> 5);
  float next_rstd = 0.0f;
  uint32_t next_scale = 0u;
  if (first < rows) {
    next_rstd = *stats;
    if (kMx8 && c.any()) next_scale = *scales;
  }
  typename T::raw* to = row_of<T>(a.dx, first, a.ld_dx);
  uint32_t now = 0, later = (stages - 1) * size;  // the stages of this row and of the one to ask for
  int round = 0;
  for (uint32_t base = blockIdx.x * kRows; base < rows; base += step, ahead += step, ++round) {
    const uint32_t row = base + (first - blockIdx.x * kRows);
    const bool there = kRows == 1 || row < rows, mine = there && c.any();
    R::fetch(a, from, c, ahead < rows, ring + later);
    from.next(a, step);
    later = now;
    const uint8_t* stage = ring + now + 16 * threadIdx.x;
    now = now + size == stages * size ? 0 : now + size;
    const float rstd = next_rstd;
    const uint32_t scale = next_scale;
    stats += step;
    scales += step * a.h8.scale_pitch;
    if (row + step < rows) {
      next_rstd = *stats;
      if (kMx8 && c.any()) next_scale = *scales;
    }
    if (stages == 4) copy_async_wait<3>();
    else if (stages == 3) copy_async_wait<2>();
    else copy_async_wait<1>();
    float2 dot = make_float2(0.0f, 0.0f);
    float g[8], xh[8];
    typename T::V dh;
    if (mine) {
      typename T::V x;
      R::read(stage, vectors, R::offset(a.dy, row, a.ld_dy), c, x);
      x.values(g);
      if constexpr (kMx8) {
        take_columns8(xh, Fetched8{*reinterpret_cast<const uint2*>(stage + R::h_at(vectors) - 8 * threadIdx.x), scale}, c, rstd);
      } else {
        R::read(stage + R::h_at(vectors), vectors, R::offset(a.h, row, a.ld_h), c, x);
        x.values(xh);
        scale8(xh, rstd);
      }
      add_vector(g, xh, w, acc, dot);
    }
    const float mean = __fmul_rn(block_sum<kLanes>(__fadd_rn(dot.x, dot.y), smem, round), inv);
    if (mine) {
      dx_vector(g, xh, mean);
      if constexpr (kDh) R::read(stage + R::dh_at(vectors), vectors, R::offset(a.dh, row, a.ld_dh), c, dh);
    }
    // (an unaligned row's by whole warps; past the last row to one of no columns)
    const Columns<kWhole> of(0, lane, there ? (uint32_t)a.cols : 0u);
    if (!kWhole || mine) store_dx<T, kLanes ? kLanes : 32>(to, of, rstd, kDh ? &dh : nullptr, g);
    to += step * a.ld_dx;
  }
  if constexpr (kLanes > 0) {  // the warp's rows together
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1)
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        acc[p].x = __fadd_rn(acc[p].x, __shfl_xor_sync(0xFFFFFFFFu, acc[p].x, o));
        acc[p].y = __fadd_rn(acc[p].y, __shfl_xor_sync(0xFFFFFFFFu, acc[p].y, o));
      }
    if (threadIdx.x >= kLanes) return;
  }
  store_part(static_cast<float*>(a.workspace) + blockIdx.x * a.cols, c, acc);
}

// Longer rows: the rows' dot products first (into the workspace's head), then
// pieces of 1024 columns, as many blocks as fill the SMs.  The second reading of
// dy and h comes from L2 up to some 100 MB: 2048 x 8192 bf16 takes 40 us, 4088 x
// 4104 48.  (Two or four vectors a thread in the ring, whose blocks then are one
// to an SM: 46 and 59.)
constexpr int kDotThreads = 256;
constexpr int kWideThreads = 128;
int64_t wide_parts(int64_t rows, int64_t cols) {
  const int64_t slabs = (cols + 8 * kWideThreads - 1) / (8 * kWideThreads);
  return std::max<int64_t>(1, std::min(rows, 16 * kSms / slabs));
}
int64_t dots_floats(int64_t rows) { return (rows + 3) / 4 * 4; }

// dy and xh of a vector.
template <class T, bool kMx8, bool kWhole>
__device__ __forceinline__ void load_dy_xh(const RmsNormBackwardArgs& a, int64_t row, const Columns<kWhole>& c, float rstd,
                                           float (&dy)[8], float (&xh)[8]) {
  using V = typename T::V;
  const typename T::raw *at = row_of<T>(a.dy, row, a.ld_dy), *h_at = row_of<T>(a.h, row, a.ld_h);
  Fetched<V, kWhole> f, fh;
  Fetched8 f8;
  V x;
  fetch_columns(f, at, c, span_of<T>(a.dy, a.rows, a.cols, a.ld_dy));
  if constexpr (kMx8) fetch_columns8(f8, row_of(a.h8, row), c);
  else fetch_columns(fh, h_at, c, span_of<T>(a.h, a.rows, a.cols, a.ld_h));
  take_columns(x, f, at, c);
  x.values(dy);
  if constexpr (kMx8) {
    take_columns8(xh, f8, c, rstd);
  } else {
    take_columns(x, fh, h_at, c);
    x.values(xh);
    scale8(xh, rstd);
  }
}

template <class T, bool kWhole, bool kMx8>
__global__ void __launch_bounds__(kDotThreads) rms_norm_dots_kernel(const __grid_constant__ RmsNormBackwardArgs a) {
  using C = Columns<kWhole>;
  __shared__ float smem[2][32];
  pdl_trigger();
  const int64_t row = blockIdx.x;
  const uint32_t cols = (uint32_t)a.cols;
  const float rstd = a.rstd[row];
  float2 dot = make_float2(0.0f, 0.0f);
  for (uint32_t first = 0; first < cols; first += 8 * kDotThreads) {
    const C c(first, threadIdx.x, cols);
    float xh[8], w[8], d[8];
    float2 unused[4] = {};
    load_dy_xh<T, kMx8>(a, row, c, rstd, d, xh);
    load_weights(a.weight, a.w_type, a.w_aligned, c, w);
    add_vector(d, xh, w, unused, dot);
  }
  const float all = block_sum<0>(__fadd_rn(dot.x, dot.y), smem, 0);
  if (threadIdx.x == 0) static_cast<float*>(a.workspace)[row] = all;
}

template <class T, bool kWhole, bool kMx8>
__global__ void __launch_bounds__(kWideThreads) rms_norm_backward_wide_kernel(const __grid_constant__ RmsNormBackwardArgs a,
                                                                              const int64_t dots) {
  const Columns<kWhole> c(8u * kWideThreads * blockIdx.x, threadIdx.x, (uint32_t)a.cols);
  pdl_trigger();
  float2 acc[4] = {}, unused = make_float2(0.0f, 0.0f);
  float w[8];
  load_weights(a.weight, a.w_type, a.w_aligned, c, w);
  const float inv = __fdiv_rn(1.0f, (float)a.cols);
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    typename T::V dh;
    float xh[8], g[8];
    const float rstd = a.rstd[row];
    load_dy_xh<T, kMx8>(a, row, c, rstd, g, xh);
    if (a.dh) load_columns(dh, row_of<T>(a.dh, row, a.ld_dh), c, span_of<T>(a.dh, a.rows, a.cols, a.ld_dh));
    add_vector(g, xh, w, acc, unused);
    dx_vector(g, xh, __fmul_rn(static_cast<const float*>(a.workspace)[row], inv));
    store_dx<T, 32>(row_of<T>(a.dx, row, a.ld_dx), c, rstd, a.dh ? &dh : nullptr, g);
  }
  store_part(static_cast<float*>(a.workspace) + dots + blockIdx.y * a.cols, c, acc);
}

// dw from the parts: 32 columns a block, a warp every 32nd part of them, then
// the warps' sums in order.
constexpr int kDwWarps = 32;
__global__ void __launch_bounds__(32 * kDwWarps) rms_norm_dw_kernel(const float* parts, const int64_t n, const int64_t cols,
                                                                    void* dw, const int type) {
  __shared__ float smem[kDwWarps][33];
  const int x = threadIdx.x & 31, q = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + x;
  pdl_wait();
  float s = 0.0f;
  if (col < cols) {
    const float* from = parts + col;
#pragma unroll 8
    for (uint32_t p = q; p < (uint32_t)n; p += kDwWarps) s = __fadd_rn(s, __ldcg(from + p * cols));
  }
  smem[q][x] = s;
  __syncthreads();
  if (q || col >= cols) return;
#pragma unroll
  for (int k = 1; k < kDwWarps; ++k) s = __fadd_rn(s, smem[k][x]);
  if (type == kMxF32) static_cast<float*>(dw)[col] = s;
  else static_cast<uint16_t*>(dw)[col] = type == kMxF16 ? F16::rn(s) : Bf16::rn(s);
}

// ------------------------------------------------------------------ launch --

// As many lanes to a row as it has vectors, in powers of two, up to a warp's with
// two vectors each; above, a block of as many threads as the row has vectors, or
// half or a quarter of them.  Measured, bf16 with a residual and all results, us:
//   131072 x 128       a warp to a row 46, 16 lanes 28
//   32768 x 512        a block of one vector a thread 27.6, a warp of two 26.4
//   32263 x 520        one vector a thread 37.4, two 42.2 (whose threads have
//   21845 x 768        28.5 and 30.8               twice the row's vectors in part)
//   16384 x 1024       28.0 and 26.7, 8192 x 2048 29.3 and 26.5
//   4096 x 4096        32.7 and 27.8, four 30.0
//   2048 x 8192        two 30.8, four 35.9
// and while the SMs hold all rows' threads at once, latency counts:
//   64 x 512           a block of one 2.4, a warp of two 2.8; 4096 x 512 4.6, 4.4
//   64 x 2048          one 2.6, two 3.1; 2048 x 2048 8.0, 7.6
//   64 x 4096          one 3.0, two 3.4; 592 x 4096 5.6, 5.2
template <class T, bool kWhole>
cudaError_t forward(const RmsNormArgs& a, cudaStream_t s) {
  const double inv = 1.0 / (double)a.cols;
  const int64_t vectors = (a.cols + 7) / 8;
  auto blocks = [&](int lanes) { return (unsigned)((a.rows * lanes + kLanesThreads - 1) / kLanesThreads); };
  auto threads = [&](int64_t chunks) { return (unsigned)(((vectors + chunks - 1) / chunks + 31) / 32 * 32); };
  const unsigned rows = (unsigned)a.rows;
  const bool few = a.rows * vectors <= 148 * 1024;
  if (vectors <= 8) rms_norm_kernel<T, kWhole, 8, 1><<<blocks(8), kLanesThreads, 0, s>>>(a, inv);
  else if (vectors <= 16) rms_norm_kernel<T, kWhole, 16, 1><<<blocks(16), kLanesThreads, 0, s>>>(a, inv);
  else if (vectors <= 32) rms_norm_kernel<T, kWhole, 32, 1><<<blocks(32), kLanesThreads, 0, s>>>(a, inv);
  else if (vectors <= 64 && !few) rms_norm_kernel<T, kWhole, 32, 2><<<blocks(32), kLanesThreads, 0, s>>>(a, inv);
  else if (few ? vectors <= 512 : vectors <= 256 && threads(1) != 2 * threads(2)) rms_norm_kernel<T, kWhole, 0, 1><<<rows, threads(1), 0, s>>>(a, inv);
  else if (vectors <= 1024) rms_norm_kernel<T, kWhole, 0, 2><<<rows, threads(2), 0, s>>>(a, inv);
  else if (vectors <= 2048) rms_norm_kernel<T, kWhole, 0, 4><<<rows, threads(4), 0, s>>>(a, inv);
  else rms_norm_long_kernel<T, kWhole><<<rows, kLongThreads, 0, s>>>(a, inv);
  return cudaGetLastError();
}

template <class T>
cudaError_t forward(const RmsNormArgs& a, cudaStream_t s) {
  const int64_t b = sizeof(typename T::raw);
  auto fits = [&](const void* p, int64_t ld) { return !p || aligned(p, ld * b); };
  const bool whole = a.cols % 8 == 0 && fits(a.x, a.ld_x) && fits(a.residual, a.ld_residual) && fits(a.y, a.ld_y) &&
                     fits(a.h, a.ld_h) && a.w_aligned;
  return whole ? forward<T, true>(a, s) : forward<T, false>(a, s);
}

cudaError_t add_dw(const RmsNormBackwardArgs& a, int64_t first, int64_t parts, cudaStream_t s) {
  return launch_kernel(rms_norm_dw_kernel, (int)((a.cols + 31) / 32), 32 * kDwWarps, 0, s, true,
                       static_cast<const float*>(a.workspace) + first, parts, a.cols, a.dw, a.dw_type);
}

template <class T, bool kMx8, bool kWhole, bool kDh, int kLanes>
cudaError_t backward_ring(const RmsNormBackwardArgs& a, cudaStream_t s) {
  // as deep as lets the blocks of parts_of fit an SM together
  constexpr int kRoom = 220 * 1024, kRows = rows_at_once(kLanes);
  const uint32_t threads = threads_of(a.cols);
  const int stage = (int)Ring<T, kWhole, kMx8, kDh>::bytes(threads);
  const int stages = std::max(2, std::min(4, kRoom / (int)blocks_to_sm(a.cols) / stage));
  static_assert(2 * kMaxThreads * (3 * 48) <= kRoom, "two stages fit, of an unaligned binary32 row too");
  auto kernel = rms_norm_backward_kernel<T, kWhole, kMx8, kDh, kLanes>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRoom);
  if (e != cudaSuccess) return e;
  const int64_t parts = parts_of((a.rows + kRows - 1) / kRows, a.cols);
  kernel<<<(unsigned)parts, threads, stages * stage, s>>>(a, stages);
  const cudaError_t r = cudaGetLastError();
  return r == cudaSuccess ? add_dw(a, 0, parts, s) : r;
}

template <class T, bool kMx8, bool kWhole, bool kDh>
cudaError_t backward_ring(const RmsNormBackwardArgs& a, cudaStream_t s) {
  // (131072 x 128 bf16 from the checkpoint: 50 us with a warp to a row, 34 with 16 lanes)
  if (a.cols <= 64) return backward_ring<T, kMx8, kWhole, kDh, 8>(a, s);
  if (a.cols <= 128) return backward_ring<T, kMx8, kWhole, kDh, 16>(a, s);
  return backward_ring<T, kMx8, kWhole, kDh, 0>(a, s);
}

template <class T, bool kMx8, bool kWhole>
cudaError_t backward_wide(const RmsNormBackwardArgs& a, cudaStream_t s) {
  const int64_t dots = dots_floats(a.rows), parts = wide_parts(a.rows, a.cols);
  rms_norm_dots_kernel<T, kWhole, kMx8><<<(unsigned)a.rows, kDotThreads, 0, s>>>(a);
  const dim3 grid((unsigned)((a.cols + 8 * kWideThreads - 1) / (8 * kWideThreads)), (unsigned)parts);
  rms_norm_backward_wide_kernel<T, kWhole, kMx8><<<grid, kWideThreads, 0, s>>>(a, dots);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? add_dw(a, dots, parts, s) : e;
}

template <class T, bool kMx8, bool kWhole>
cudaError_t backward(const RmsNormBackwardArgs& a, cudaStream_t s) {
  if (a.cols > kRingCols) return backward_wide<T, kMx8, kWhole>(a, s);
  return a.dh ? backward_ring<T, kMx8, kWhole, true>(a, s) : backward_ring<T, kMx8, kWhole, false>(a, s);
}

template <class T, bool kMx8>
cudaError_t backward(const RmsNormBackwardArgs& a, cudaStream_t s) {
  const int64_t b = sizeof(typename T::raw);
  auto fits = [&](const void* p, int64_t ld) { return !p || aligned(p, ld * b); };
  const bool whole = a.cols % 8 == 0 && fits(a.dy, a.ld_dy) && fits(a.h, a.ld_h) && fits(a.dh, a.ld_dh) &&
                     fits(a.dx, a.ld_dx) && a.w_aligned;
  return whole ? backward<T, kMx8, true>(a, s) : backward<T, kMx8, false>(a, s);
}

template <class T>
cudaError_t backward(const RmsNormBackwardArgs& a, cudaStream_t s) {
  return a.h ? backward<T, false>(a, s) : backward<T, true>(a, s);
}

}  // namespace

int64_t rms_norm_backward_workspace(int64_t rows, int64_t cols) {
  return 4 * (cols <= kRingCols ? parts_of(rows, cols) * cols : dots_floats(rows) + wide_parts(rows, cols) * cols);
}

cudaError_t launch_rms_norm(const RmsNormArgs& a, int, cudaStream_t s) {
  switch (a.type) {
    case kMxBf16: return forward<TBf16>(a, s);
    case kMxF16: return forward<TF16>(a, s);
    case kMxF32: return forward<TF32>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_rms_norm_backward(const RmsNormBackwardArgs& a, int, cudaStream_t s) {
  switch (a.type) {
    case kMxBf16: return backward<TBf16>(a, s);
    case kMxF16: return backward<TF16>(a, s);
    case kMxF32: return backward<TF32>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace zsm
