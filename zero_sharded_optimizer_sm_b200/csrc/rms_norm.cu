// Root-mean-square norm, forward and backward (rms_norm.cuh has the formulas).
//
// Both are memory-bound: forward 2 to 4 values of the row's type and up to two
// MX8 bytes an element, backward 3 or 4.  A row's elements are read once: they
// stay in registers (forward) or shared memory (backward), as they were loaded,
// between the sum over the row and its use.
#include <cuda_runtime.h>

#include "rms_norm.cuh"
#include "rows.cuh"

namespace zsm {
namespace {

using namespace mx;

// Threads to a block: a block of more than 32 threads to a row has one row.
template <int kGroup>
constexpr int kBlockOf = kGroup > 128 ? kGroup : 128;

// ----------------------------------------------------------------- forward --

// Sum over the kGroup threads that share a row (a warp, or the whole block of
// kGroup threads), from a warp's binary32 sum on in binary64: every thread gets
// the same bits.
template <int kGroup>
__device__ __forceinline__ double group_sum(float mine, float* smem) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine = __fadd_rn(mine, __shfl_xor_sync(0xFFFFFFFFu, mine, o));
  if constexpr (kGroup == 32) return (double)mine;
  constexpr int kWarps = kGroup / 32;
  if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = mine;
  __syncthreads();
  double v = 0.0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v = __dadd_rn(v, (double)smem[w]);
  return v;
}

// (ss / cols + eps)^(-1/2), rounded once from binary64: the function's binary32
// estimate and one Newton step, whose error is the square of the estimate's.
// y's rounding to 16 and then to 8 bits turns on rstd's last bit now and then,
// so it is the correctly rounded one but for sums next to a tie.
__device__ __forceinline__ float rstd_of(double ss, double inv_cols, double eps) {
  const double m = __fma_rn(ss, inv_cols, eps);
  const float r = rsqrtf((float)m);
  const double e = __fma_rn(-__dmul_rn(m, (double)r), (double)r, 1.0);
  const float better = (float)__fma_rn(__dmul_rn(0.5, e), (double)r, (double)r);
  return isfinite((float)m) ? better : r;
}

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

// A vector of one row of h: x plus the residual, rounded to their type.
template <class T, class C>
__device__ __forceinline__ void load_h(const RmsNormArgs& a, const NormRow<T>& row, const C& c, typename T::V& x) {
  load_columns(x, row.x, c);
  if (a.residual) {
    typename T::V r;
    load_columns(r, row.r, c);
    add_to(x, r);
  }
}

__device__ __forceinline__ float2 square_sum(const float (&v)[8], float2 ss) {
#pragma unroll
  for (int p = 0; p < 4; ++p) ss = fma2(pair(v, p), pair(v, p), ss);
  return ss;
}

// All results of one vector of h.  Called by whole warps.
template <class T, class C>
__device__ __forceinline__ void finish(const RmsNormArgs& a, const NormRow<T>& row, const C& c, float rstd,
                                       const typename T::V& x) {
  float v[8], w[8];
  x.values(v);
  if (a.h) store_columns(row.h, c, x);
  if (a.h8.codes) store_columns8(row.h8, c, x, v);
  if (!a.y && !a.y8.codes) return;
  load_weights(a.weight, a.w_type, c, w);
  scale8(v, rstd);
  times8(v, w);
  typename T::V y;
  round_to(y, v);
  if (a.y) store_columns(row.y, c, y);
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

// kGroup threads to a row, kChunks vectors of eight elements a thread.
template <class T, bool kVec, int kGroup, int kChunks>
__global__ void __launch_bounds__(kBlockOf<kGroup>) rms_norm_kernel(const __grid_constant__ RmsNormArgs a,
                                                                    const double inv_cols) {
  constexpr int kRows = kBlockOf<kGroup> / kGroup;
  __shared__ float smem[32];
  const uint32_t number = blockIdx.x * kRows + (kRows > 1 ? threadIdx.x / kGroup : 0);
  if (number >= (uint32_t)a.rows) return;  // whole groups
  const NormRow<T> row(a, number);
  const uint32_t t = threadIdx.x % kGroup, cols = (uint32_t)a.cols;
  using C = Columns<kVec, kGroup>;
  typename T::V x[kChunks];
#pragma unroll
  for (int k = 0; k < kChunks; ++k) load_h<T>(a, row, C(8 * kGroup * k, t, cols), x[k]);
  float2 ss = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    float v[8];
    x[k].values(v);
    ss = square_sum(v, ss);
  }
  const float rstd = rstd_of(group_sum<kGroup>(__fadd_rn(ss.x, ss.y), smem), inv_cols, (double)a.eps);
  if (a.rstd && t == 0) a.rstd[number] = rstd;
#pragma unroll
  for (int k = 0; k < kChunks; ++k) finish<T>(a, row, C(8 * kGroup * k, t, cols), rstd, x[k]);
}

// Rows too long for registers: read a second time (a thread reads its own
// elements before it writes results in their place).
constexpr int kLongThreads = 512;
template <class T, bool kVec>
__global__ void __launch_bounds__(kLongThreads) rms_norm_long_kernel(const __grid_constant__ RmsNormArgs a,
                                                                     const double inv_cols) {
  __shared__ float smem[32];
  const NormRow<T> row(a, blockIdx.x);
  const uint32_t cols = (uint32_t)a.cols;
  using C = Columns<kVec, kLongThreads>;
  float2 ss = make_float2(0.0f, 0.0f);
  for (uint32_t first = 0; first < cols; first += 8 * kLongThreads) {
    typename T::V x;
    float v[8];
    load_h<T>(a, row, C(first, threadIdx.x, cols), x);
    x.values(v);
    ss = square_sum(v, ss);
  }
  const float rstd = rstd_of(group_sum<kLongThreads>(__fadd_rn(ss.x, ss.y), smem), inv_cols, (double)a.eps);
  if (a.rstd && threadIdx.x == 0) a.rstd[blockIdx.x] = rstd;
  for (uint32_t first = 0; first < cols; first += 8 * kLongThreads) {
    typename T::V x;
    const C c(first, threadIdx.x, cols);
    load_h<T>(a, row, c, x);
    finish<T>(a, row, c, rstd, x);
  }
}

// ---------------------------------------------------------------- backward --

// A block walks over rows block, block + blocks, ... and keeps its columns'
// part of dw in registers; the parts go to the workspace, one row of it a
// block, and a second kernel adds them in order.
//
// Rows whose vectors are aligned come through a ring in shared memory, kStages
// rows deep, by asynchronous copies: each thread fetches the elements that it
// reads itself, so that nothing but its own copies has to be waited for, and
// the sum over a row -- the one place where the block's threads meet -- never
// holds up the loads of the next ones.
constexpr int64_t kSms = 148;

// Blocks at most, for rows of so many columns: as many as are there at a time.
int64_t max_parts(int64_t cols) { return kSms * (cols <= 1024 ? 8 : cols <= 2048 ? 4 : cols <= 4096 ? 2 : 1); }
int64_t parts_of(int64_t rows, int64_t cols) { return std::max<int64_t>(1, std::min(rows, max_parts(cols))); }

// The longest rows that a block takes; longer ones go through memory twice.
int64_t wide_from(int type) { return type == kMxF32 ? 8192 : 16384; }

// Sum over the block (kGroup threads) in binary32; smem holds two rounds'
// values, so that one barrier a round will do.
template <int kGroup>
__device__ __forceinline__ float block_sum(float v, float (*smem)[32], int round) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  constexpr int kWarps = kGroup / 32;
  const int lane = threadIdx.x & 31;
  if (lane == 0) smem[round & 1][threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < kWarps ? smem[round & 1][lane] : 0.0f;
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return __shfl_sync(0xFFFFFFFFu, v, 0);
}

// One vector's part of a row's sum of g xh, and of dw; dy becomes g.
__device__ __forceinline__ void add_vector(float (&dy)[8], const float (&xh)[8], const float (&w)[8], float2 (&acc)[4],
                                           float2& dot) {
#pragma unroll
  for (int p = 0; p < 4; ++p) acc[p] = fma2(pair(dy, p), pair(xh, p), acc[p]);
  times8(dy, w);
#pragma unroll
  for (int p = 0; p < 4; ++p) dot = fma2(pair(dy, p), pair(xh, p), dot);
}

// dx of one vector, without dh, in g's place: rstd (g - xh mean).
__device__ __forceinline__ void dx_vector(float (&g)[8], const float (&xh)[8], float rstd, float mean) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 d = fma2(pair(xh, p), make_float2(-mean, -mean), pair(g, p));
    g[2 * p] = d.x, g[2 * p + 1] = d.y;
  }
  scale8(g, rstd);
}

// dx, rounded, with dh (a vector of the type) added if there is one.
template <class T, class C>
__device__ __forceinline__ void store_dx(typename T::raw* row, const C& c, const typename T::V* dh, float (&v)[8]) {
  if (dh) {
    float u[8];
    dh->values(u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fadd_rn(v[j], u[j]);
  }
  typename T::V x;
  round_to(x, v);
  store_columns(row, c, x);
}

template <class C, class A>
__device__ __forceinline__ void store_part(float* out, const C& c, const A& acc) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c.in(j)) out[c.at(j)] = j & 1 ? acc[j >> 1].y : acc[j >> 1].x;
}

// One row's stage of the ring: dy, h, dh of every thread's vectors, 16 bytes of
// each thread next to another's.
template <class T, int kGroup, int kChunks, bool kMx8, bool kDh>
struct Ring {
  using V = typename T::V;
  using raw = typename T::raw;
  static constexpr int kWords = sizeof(raw) / 2;        // 16-byte words of a vector
  static constexpr int kPlane = kGroup * kChunks * 16;  // bytes of one word of all vectors
  static constexpr int kH = kWords * kPlane;            // where h's begin
  static constexpr int kD = kH + (kMx8 ? kPlane / 2 : kWords * kPlane);
  static constexpr int kBytes = kD + (kDh ? kWords * kPlane : 0);

  // Asks for a row (none past the end; the group is there all the same).
  static __device__ __forceinline__ void fetch(const RmsNormBackwardArgs& a, int64_t row, uint8_t* to) {
    if (row < a.rows) {
      const raw* dy = row_of<T>(a.dy, row, a.ld_dy);
      const raw* h = row_of<T>(a.h, row, a.ld_h);
      const raw* dh = row_of<T>(a.dh, row, a.ld_dh);
      const uint8_t* h8 = a.h8.codes + row * a.h8.code_pitch;
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const uint32_t v = kGroup * k + threadIdx.x;
        if (8 * v >= (uint32_t)a.cols) break;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          constexpr int kIn = 16 / (int)sizeof(raw);
          copy_async16(to + i * kPlane + 16 * v, dy + 8 * v + kIn * i);
          if constexpr (!kMx8) copy_async16(to + kH + i * kPlane + 16 * v, h + 8 * v + kIn * i);
          if constexpr (kDh) copy_async16(to + kD + i * kPlane + 16 * v, dh + 8 * v + kIn * i);
        }
        if constexpr (kMx8) copy_async8(to + kH + 8 * v, h8 + 8 * v);
      }
    }
    copy_async_commit();
  }
  static __device__ __forceinline__ void read(const uint8_t* plane, int k, V& x) {
    const uint8_t* p = plane + 16 * (kGroup * k + threadIdx.x);
    uint4* w = reinterpret_cast<uint4*>(&x);
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = *reinterpret_cast<const uint4*>(p + i * kPlane);
  }
  // xh of a vector.
  static __device__ __forceinline__ void read_xh(const uint8_t* stage, int k, uint32_t scale, float rstd, float (&v)[8]) {
    if constexpr (kMx8) {
      elements8(*reinterpret_cast<const uint2*>(stage + kH + 8 * (kGroup * k + threadIdx.x)), v);
      scale8(v, __fmul_rn(scale_value(scale), rstd));
    } else {
      V x;
      read(stage + kH, k, x);
      x.values(v);
      scale8(v, rstd);
    }
  }
};

// A row's vectors are whole and aligned here.  One vector a thread: xh and g
// stay in registers over the sum; more: they are read and made a second time.
template <class T, int kGroup, int kChunks, bool kMx8, bool kDh, int kStages>
__global__ void __launch_bounds__(kGroup) rms_norm_backward_ring_kernel(const __grid_constant__ RmsNormBackwardArgs a) {
  using R = Ring<T, kGroup, kChunks, kMx8, kDh>;
  using C = Columns<true, kGroup>;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float smem[2][32];
  pdl_trigger();
  const int64_t step = gridDim.x;
  const uint32_t cols = (uint32_t)a.cols;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) R::fetch(a, blockIdx.x + s * step, ring + s * R::kBytes);
  float2 acc[kChunks][4];
  float w[8];
#pragma unroll
  for (int k = 0; k < kChunks; ++k)
#pragma unroll
    for (int p = 0; p < 4; ++p) acc[k][p] = make_float2(0.0f, 0.0f);
  if constexpr (kChunks == 1) load_weights(a.weight, a.w_type, C(0, threadIdx.x, cols), w);
  const float inv = __fdiv_rn(1.0f, (float)a.cols);
  // the row's statistics and scales, a row ahead
  float next_rstd = 0.0f;
  uint32_t scale[kChunks] = {}, next_scale[kChunks] = {};
  auto ahead = [&](int64_t row) {
    if (row >= a.rows) return;
    next_rstd = a.rstd[row];
    if constexpr (kMx8) {
      const uint8_t* scales = a.h8.scales + row * a.h8.scale_pitch;
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const C c(8 * kGroup * k, threadIdx.x, cols);
        if (c.in(0)) next_scale[k] = scales[c.first >> 5];
      }
    }
  };
  ahead(blockIdx.x);
  uint32_t now = 0, later = (kStages - 1) * R::kBytes;  // the stages of this row and of the one to ask for
  int round = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += step, ++round) {
    R::fetch(a, row + (kStages - 1) * step, ring + later);
    later = now;
    const uint8_t* stage = ring + now;
    now = now + R::kBytes == kStages * R::kBytes ? 0 : now + R::kBytes;
    const float rstd = next_rstd;
#pragma unroll
    for (int k = 0; k < kChunks; ++k) scale[k] = next_scale[k];
    ahead(row + step);
    copy_async_wait<kStages - 1>();
    float2 dot = make_float2(0.0f, 0.0f);
    float g[8], xh[8];
    auto vector = [&](int k, bool sums) {
      const C c(8 * kGroup * k, threadIdx.x, cols);
      typename T::V dy;
      R::read(stage, k, dy);
      dy.values(g);
      R::read_xh(stage, k, scale[k], rstd, xh);
      if constexpr (kChunks > 1) load_weights(a.weight, a.w_type, c, w);
      if (sums) add_vector(g, xh, w, acc[k], dot);
      else times8(g, w);
    };
#pragma unroll
    for (int k = 0; k < kChunks; ++k)
      if (C(8 * kGroup * k, threadIdx.x, cols).in(0)) vector(k, true);
    const float mean = __fmul_rn(block_sum<kGroup>(__fadd_rn(dot.x, dot.y), smem, round), inv);
    typename T::raw* to = row_of<T>(a.dx, row, a.ld_dx);
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      const C c(8 * kGroup * k, threadIdx.x, cols);
      if (!c.in(0)) break;
      if constexpr (kChunks > 1) vector(k, false);
      dx_vector(g, xh, rstd, mean);
      typename T::V dh;
      if constexpr (kDh) R::read(stage + R::kD, k, dh);
      store_dx<T>(to, c, kDh ? &dh : nullptr, g);
    }
  }
  float* out = static_cast<float*>(a.workspace) + blockIdx.x * a.cols;
#pragma unroll
  for (int k = 0; k < kChunks; ++k) store_part(out, C(8 * kGroup * k, threadIdx.x, cols), acc[k]);
}

// Rows of any alignment, straight from memory.
template <class T, bool kMx8, class C>
__device__ __forceinline__ void load_dy_xh(const RmsNormBackwardArgs& a, int64_t row, const C& c, float rstd,
                                           typename T::V& dy, float (&xh)[8]) {
  load_columns(dy, row_of<T>(a.dy, row, a.ld_dy), c);
  if constexpr (kMx8) {
    load_columns8(row_of(a.h8, row), c, rstd, xh);
  } else {
    typename T::V x;
    load_columns(x, row_of<T>(a.h, row, a.ld_h), c);
    x.values(xh);
    scale8(xh, rstd);
  }
}

template <class T, class C>
__device__ __forceinline__ void finish_dx(const RmsNormBackwardArgs& a, int64_t row, const C& c, float (&v)[8]) {
  typename T::V dh;
  if (a.dh) load_columns(dh, row_of<T>(a.dh, row, a.ld_dh), c);
  store_dx<T>(row_of<T>(a.dx, row, a.ld_dx), c, a.dh ? &dh : nullptr, v);
}

template <class T, int kGroup, int kChunks, bool kMx8>
__global__ void __launch_bounds__(kGroup) rms_norm_backward_kernel(const __grid_constant__ RmsNormBackwardArgs a) {
  using C = Columns<false, kGroup>;
  __shared__ float smem[2][32];
  pdl_trigger();
  const uint32_t cols = (uint32_t)a.cols;
  float2 acc[kChunks][4];
#pragma unroll
  for (int k = 0; k < kChunks; ++k)
#pragma unroll
    for (int p = 0; p < 4; ++p) acc[k][p] = make_float2(0.0f, 0.0f);
  const float inv = __fdiv_rn(1.0f, (float)a.cols);
  int round = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, ++round) {
    typename T::V dy[kChunks];
    float xh[kChunks][8], w[8], g[8];
    const float rstd = a.rstd[row];
    float2 dot = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < kChunks; ++k) load_dy_xh<T, kMx8>(a, row, C(8 * kGroup * k, threadIdx.x, cols), rstd, dy[k], xh[k]);
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      dy[k].values(g);
      load_weights(a.weight, a.w_type, C(8 * kGroup * k, threadIdx.x, cols), w);
      add_vector(g, xh[k], w, acc[k], dot);
    }
    const float mean = __fmul_rn(block_sum<kGroup>(__fadd_rn(dot.x, dot.y), smem, round), inv);
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      const C c(8 * kGroup * k, threadIdx.x, cols);
      if constexpr (kChunks > 1) {
        dy[k].values(g);
        load_weights(a.weight, a.w_type, c, w);
        times8(g, w);
      }
      dx_vector(g, xh[k], rstd, mean);
      finish_dx<T>(a, row, c, g);
    }
  }
  float* out = static_cast<float*>(a.workspace) + blockIdx.x * a.cols;
#pragma unroll
  for (int k = 0; k < kChunks; ++k) store_part(out, C(8 * kGroup * k, threadIdx.x, cols), acc[k]);
}

// Longer rows: the rows' dot products first (into the workspace's head), then
// pieces of 2048 columns.
constexpr int kWideThreads = 256;
constexpr int kWideParts = 64;
int64_t wide_parts(int64_t rows) { return std::max<int64_t>(1, std::min<int64_t>(rows, kWideParts)); }
int64_t dots_floats(int64_t rows) { return (rows + 3) / 4 * 4; }

template <class T, bool kVec, bool kMx8>
__global__ void __launch_bounds__(kWideThreads) rms_norm_dots_kernel(const __grid_constant__ RmsNormBackwardArgs a) {
  using C = Columns<kVec, kWideThreads>;
  __shared__ float smem[2][32];
  pdl_trigger();
  const int64_t row = blockIdx.x;
  const uint32_t cols = (uint32_t)a.cols;
  const float rstd = a.rstd[row];
  float2 dot = make_float2(0.0f, 0.0f);
  for (uint32_t first = 0; first < cols; first += 8 * kWideThreads) {
    const C c(first, threadIdx.x, cols);
    if (!c.in(0)) break;
    typename T::V dy;
    float xh[8], w[8], d[8];
    float2 unused[4] = {};
    load_dy_xh<T, kMx8>(a, row, c, rstd, dy, xh);
    load_weights(a.weight, a.w_type, c, w);
    dy.values(d);
    add_vector(d, xh, w, unused, dot);
  }
  const float all = block_sum<kWideThreads>(__fadd_rn(dot.x, dot.y), smem, 0);
  if (threadIdx.x == 0) static_cast<float*>(a.workspace)[row] = all;
}

template <class T, bool kVec, bool kMx8>
__global__ void __launch_bounds__(kWideThreads) rms_norm_backward_wide_kernel(const __grid_constant__ RmsNormBackwardArgs a,
                                                                              const int64_t dots) {
  const Columns<kVec, kWideThreads> c(8u * kWideThreads * blockIdx.x, threadIdx.x, (uint32_t)a.cols);
  pdl_trigger();
  if (!c.in(0)) return;
  float2 acc[4] = {}, unused = make_float2(0.0f, 0.0f);
  float w[8];
  load_weights(a.weight, a.w_type, c, w);
  const float inv = __fdiv_rn(1.0f, (float)a.cols);
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    typename T::V dy;
    float xh[8], g[8];
    const float rstd = a.rstd[row];
    load_dy_xh<T, kMx8>(a, row, c, rstd, dy, xh);
    dy.values(g);
    add_vector(g, xh, w, acc, unused);
    dx_vector(g, xh, rstd, __fmul_rn(static_cast<const float*>(a.workspace)[row], inv));
    finish_dx<T>(a, row, c, g);
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
#pragma unroll 8
    for (int64_t p = q; p < n; p += kDwWarps) s = __fadd_rn(s, __ldcg(parts + p * cols + col));
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

template <class T, bool kVec, int kGroup, int kChunks>
cudaError_t forward(const RmsNormArgs& a, cudaStream_t s) {
  constexpr int kRows = kBlockOf<kGroup> / kGroup;
  rms_norm_kernel<T, kVec, kGroup, kChunks><<<(unsigned)((a.rows + kRows - 1) / kRows), kBlockOf<kGroup>, 0, s>>>(
      a, 1.0 / (double)a.cols);
  return cudaGetLastError();
}

template <class T, bool kVec>
cudaError_t forward(const RmsNormArgs& a, cudaStream_t s) {
  if (a.cols <= 256) return forward<T, kVec, 32, 1>(a, s);
  if (a.cols <= 512) return forward<T, kVec, 32, 2>(a, s);
  if (a.cols <= 1024) return forward<T, kVec, 128, 1>(a, s);
  if (a.cols <= 2048) return forward<T, kVec, 256, 1>(a, s);
  if (a.cols <= 4096) return forward<T, kVec, 256, 2>(a, s);
  if (a.cols <= 8192) return forward<T, kVec, 512, 2>(a, s);
  if (a.cols <= 16384) return forward<T, kVec, 512, 4>(a, s);
  rms_norm_long_kernel<T, kVec><<<(unsigned)a.rows, kLongThreads, 0, s>>>(a, 1.0 / (double)a.cols);
  return cudaGetLastError();
}

template <class T>
cudaError_t forward(const RmsNormArgs& a, cudaStream_t s) {
  const int64_t b = sizeof(typename T::raw);
  auto fits = [&](const void* p, int64_t ld) { return !p || aligned(p, ld * b); };
  const bool vec = a.cols % 8 == 0 && fits(a.x, a.ld_x) && fits(a.residual, a.ld_residual) && fits(a.y, a.ld_y) && fits(a.h, a.ld_h) &&
                   aligned(a.weight, 0);
  return vec ? forward<T, true>(a, s) : forward<T, false>(a, s);
}

cudaError_t add_dw(const RmsNormBackwardArgs& a, int64_t first, int64_t parts, cudaStream_t s) {
  return launch_kernel(rms_norm_dw_kernel, (int)((a.cols + 31) / 32), 32 * kDwWarps, 0, s, true,
                       static_cast<const float*>(a.workspace) + first, parts, a.cols, a.dw, a.dw_type);
}

template <class T, bool kMx8, int kGroup, int kChunks, bool kDh>
cudaError_t backward_ring(const RmsNormBackwardArgs& a, int64_t parts, cudaStream_t s) {
  // as deep as lets the blocks of max_parts fit an SM together
  constexpr int kStage = Ring<T, kGroup, kChunks, kMx8, kDh>::kBytes;
  constexpr int kShare = 220 * 1024 / (kGroup <= 128 ? 8 : kGroup <= 256 ? 4 : kChunks == 1 ? 2 : 1);
  constexpr int kStages = kShare / kStage < 2 ? 2 : kShare / kStage > 5 ? 5 : kShare / kStage;
  static_assert(kStages * kStage <= 220 * 1024, "the ring fits");
  auto kernel = rms_norm_backward_ring_kernel<T, kGroup, kChunks, kMx8, kDh, kStages>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStages * kStage);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)parts, kGroup, kStages * kStage, s>>>(a);
  return cudaGetLastError();
}

template <class T, bool kMx8, int kGroup, int kChunks>
cudaError_t backward(const RmsNormBackwardArgs& a, bool vec, cudaStream_t s) {
  const int64_t parts = parts_of(a.rows, a.cols);
  cudaError_t e;
  if (vec) {
    e = a.dh ? backward_ring<T, kMx8, kGroup, kChunks, true>(a, parts, s)
             : backward_ring<T, kMx8, kGroup, kChunks, false>(a, parts, s);
  } else {
    rms_norm_backward_kernel<T, kGroup, kChunks, kMx8><<<(unsigned)parts, kGroup, 0, s>>>(a);
    e = cudaGetLastError();
  }
  return e == cudaSuccess ? add_dw(a, 0, parts, s) : e;
}

template <class T, bool kMx8, bool kVec>
cudaError_t backward_wide(const RmsNormBackwardArgs& a, cudaStream_t s) {
  const int64_t dots = dots_floats(a.rows), parts = wide_parts(a.rows);
  rms_norm_dots_kernel<T, kVec, kMx8><<<(unsigned)a.rows, kWideThreads, 0, s>>>(a);
  const dim3 grid((unsigned)((a.cols + 8 * kWideThreads - 1) / (8 * kWideThreads)), (unsigned)parts);
  rms_norm_backward_wide_kernel<T, kVec, kMx8><<<grid, kWideThreads, 0, s>>>(a, dots);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? add_dw(a, dots, parts, s) : e;
}

template <class T, bool kMx8>
cudaError_t backward(const RmsNormBackwardArgs& a, cudaStream_t s) {
  const int64_t b = sizeof(typename T::raw);
  auto fits = [&](const void* p, int64_t ld) { return !p || aligned(p, ld * b); };
  const bool vec = a.cols % 8 == 0 && fits(a.dy, a.ld_dy) && fits(a.h, a.ld_h) && fits(a.dh, a.ld_dh) &&
                   fits(a.dx, a.ld_dx) && aligned(a.weight, 0);
  if (a.cols > wide_from(a.type)) return vec ? backward_wide<T, kMx8, true>(a, s) : backward_wide<T, kMx8, false>(a, s);
  if (a.cols <= 256) return backward<T, kMx8, 32, 1>(a, vec, s);
  if (a.cols <= 512) return backward<T, kMx8, 64, 1>(a, vec, s);
  if (a.cols <= 1024) return backward<T, kMx8, 128, 1>(a, vec, s);
  if (a.cols <= 2048) return backward<T, kMx8, 256, 1>(a, vec, s);
  if (a.cols <= 4096) return backward<T, kMx8, 512, 1>(a, vec, s);
  if (a.cols <= 8192) return backward<T, kMx8, 512, 2>(a, vec, s);
  if constexpr (sizeof(typename T::raw) == 2) return backward<T, kMx8, 512, 4>(a, vec, s);
  return cudaErrorInvalidValue;
}

template <class T>
cudaError_t backward(const RmsNormBackwardArgs& a, cudaStream_t s) {
  return a.h ? backward<T, false>(a, s) : backward<T, true>(a, s);
}

}  // namespace

int64_t rms_norm_backward_workspace(int64_t rows, int64_t cols) {
  // for every type: binary32's rows go through memory twice from 8192 columns on
  const int64_t once = parts_of(rows, cols) * cols, twice = dots_floats(rows) + wide_parts(rows) * cols;
  return 4 * (cols <= wide_from(kMxF32) ? once : cols <= wide_from(kMxBf16) ? std::max(once, twice) : twice);
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
