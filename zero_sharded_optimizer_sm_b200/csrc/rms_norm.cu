// Root-mean-square norm, forward and backward (rms_norm.cuh has the formulas).
//
// Both are memory-bound: forward 2 to 4 values of the row's type and up to two
// MX8 bytes an element, backward 3 or 4.  A row's elements are read once: they
// stay in registers, as they were loaded, between the sum over the row and its
// use.
#include <cuda_runtime.h>

#include "mx4_quant.cuh"
#include "rms_norm.cuh"

namespace zsm {
namespace {

using namespace mx;

// n (at most 8) values of a vector of one of the three types, 0 past the end.
__device__ __forceinline__ void weights8(const void* w, int type, int64_t at, int64_t n, int vec, float (&v)[8]) {
  if (type == kMxF32) {
    const float* p = static_cast<const float*>(w) + at;
    if (n >= 8 && vec) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j < n ? __ldg(p + j) : 0.0f;
    }
    return;
  }
  const uint16_t* p = static_cast<const uint16_t*>(w) + at;
  uint32_t u[4];
  if (n >= 8 && vec) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
    u[0] = a.x, u[1] = a.y, u[2] = a.z, u[3] = a.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      u[j] = (2 * j < n ? (uint32_t)__ldg(p + 2 * j) : 0u) | (2 * j + 1 < n ? (uint32_t)__ldg(p + 2 * j + 1) << 16 : 0u);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = type == kMxF16 ? F16::lo(u[j]) : Bf16::lo(u[j]);
    v[2 * j + 1] = type == kMxF16 ? F16::hi(u[j]) : Bf16::hi(u[j]);
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

// Sum over the kGroup threads that share a row (a warp, or the whole block of
// kGroup threads); every one of them gets the same bits.
template <int kGroup>
__device__ __forceinline__ float group_sum(float v, float* smem) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  if constexpr (kGroup > 32) {
    constexpr int kWarps = kGroup / 32;
    const int lane = threadIdx.x & 31;
    __syncthreads();  // the last call's values have been read
    if (lane == 0) smem[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < kWarps ? smem[lane] : 0.0f;
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    v = __shfl_sync(0xFFFFFFFFu, v, 0);
  }
  return v;
}

__device__ __forceinline__ void store_mx8(const Mx8Matrix& m, int64_t row, int64_t col, int64_t nb, uint32_t s,
                                          const float (&v)[8]) {
  const int64_t b = col >> 5;
  if (b >= nb) return;
  *reinterpret_cast<uint2*>(m.codes + row * m.code_pitch + col) = encode8_mx8(v, s);
  if ((col & 31) == 0) m.scales[row * m.scale_pitch + b] = (uint8_t)s;
}

// ----------------------------------------------------------------- forward --

// Threads to a block: a block of more than 32 threads to a row has one row.
template <int kGroup>
constexpr int kBlockOf = kGroup > 128 ? kGroup : 128;

// The vectors of one row of h at a thread's column: x plus the residual,
// rounded to their type.
template <class T>
__device__ __forceinline__ void load_h(const RmsNormArgs& a, int64_t row, int64_t col, int vec, typename T::V& x) {
  using raw = typename T::raw;
  const int64_t n = a.cols - col;
  load8(x, static_cast<const raw*>(a.x) + row * a.ld_x + col, n, vec);
  if (a.residual) {
    typename T::V r;
    load8(r, static_cast<const raw*>(a.residual) + row * a.ld_residual + col, n, vec);
    float v[8], u[8];
    x.values(v);
    r.values(u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fadd_rn(v[j], u[j]);
    round_to(x, v);
  }
}

__device__ __forceinline__ float square_sum(const float (&v)[8], float ss) {
#pragma unroll
  for (int j = 0; j < 8; ++j) ss = __fmaf_rn(v[j], v[j], ss);
  return ss;
}

// All results of one vector of h.  Called by whole warps.
template <class T>
__device__ __forceinline__ void finish(const RmsNormArgs& a, int64_t row, int64_t col, int64_t nb, int vec, float rstd,
                                       const typename T::V& x) {
  using raw = typename T::raw;
  const int64_t n = a.cols - col;
  float v[8], w[8];
  x.values(v);
  if (a.h) store8<T>(static_cast<raw*>(a.h) + row * a.ld_h + col, v, n, vec);
  if (a.h8.codes) store_mx8(a.h8, row, col, nb, scale_code8(max_of_four(x.max_bits())), v);
  weights8(a.weight, a.w_type, col, n, vec, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(__fmul_rn(v[j], rstd), w[j]);
  if (a.y) store8<T>(static_cast<raw*>(a.y) + row * a.ld_y + col, v, n, vec);
  if (a.y8.codes) {
    typename T::V y;
    round_to(y, v);
    y.values(v);
    if (n < 8) {  // past the row: w is 0 there, but rstd need not be finite
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j >= n) v[j] = 0.0f;
      round_to(y, v);
    }
    store_mx8(a.y8, row, col, nb, scale_code8(max_of_four(y.max_bits())), v);
  }
}

__device__ __forceinline__ float rstd_of(float ss, int64_t cols, float eps) {
  return __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)cols), eps)));
}

// kGroup threads to a row, kChunks vectors of eight elements a thread.
template <class T, int kGroup, int kChunks>
__global__ void __launch_bounds__(kBlockOf<kGroup>) rms_norm_kernel(const __grid_constant__ RmsNormArgs a, const int vec) {
  constexpr int kRows = kBlockOf<kGroup> / kGroup;
  __shared__ float smem[32];
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kGroup;
  if (row >= a.rows) return;  // whole groups
  const int64_t nb = (a.cols + kMxBlock - 1) / kMxBlock;
  const int64_t c0 = 8 * (threadIdx.x % kGroup);
  typename T::V x[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) load_h<T>(a, row, c0 + 8 * kGroup * c, vec, x[c]);
  float ss = 0.0f;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    float v[8];
    x[c].values(v);
    ss = square_sum(v, ss);
  }
  const float rstd = rstd_of(group_sum<kGroup>(ss, smem), a.cols, a.eps);
  if (a.rstd && c0 == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) finish<T>(a, row, c0 + 8 * kGroup * c, nb, vec, rstd, x[c]);
}

// Rows too long for registers: read a second time (a thread reads its own
// elements before it writes results in their place).
constexpr int kLongThreads = 512;
template <class T>
__global__ void __launch_bounds__(kLongThreads) rms_norm_long_kernel(const __grid_constant__ RmsNormArgs a, const int vec) {
  __shared__ float smem[32];
  const int64_t row = blockIdx.x;
  const int64_t nb = (a.cols + kMxBlock - 1) / kMxBlock;
  float ss = 0.0f;
  for (int64_t col = 8 * threadIdx.x; col < a.cols; col += 8 * kLongThreads) {
    typename T::V x;
    float v[8];
    load_h<T>(a, row, col, vec, x);
    x.values(v);
    ss = square_sum(v, ss);
  }
  const float rstd = rstd_of(group_sum<kLongThreads>(ss, smem), a.cols, a.eps);
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
  for (int64_t first = 0; first < a.cols; first += 8 * kLongThreads) {  // whole warps take part
    const int64_t col = first + 8 * threadIdx.x;
    typename T::V x;
    load_h<T>(a, row, col, vec, x);
    finish<T>(a, row, col, nb, vec, rstd, x);
  }
}

// ---------------------------------------------------------------- backward --

// A block's group walks over rows group, group + groups, ... and keeps its
// columns' part of dw in registers; the parts go to the workspace, one row of
// it a block, and a second kernel adds them in order.
constexpr int64_t kParts = 592;          // blocks at most: 4 to an SM of 148
constexpr int64_t kWideCols = 16384;     // longer rows go through memory twice

int64_t parts_of(int64_t rows) { return std::max<int64_t>(1, std::min(rows, kParts)); }

template <class T, bool kMx8>
__device__ __forceinline__ void load_backward(const RmsNormBackwardArgs& a, int64_t row, int64_t col, int vec,
                                              typename T::V& dy, float (&h)[8]) {
  using raw = typename T::raw;
  const int64_t n = a.cols - col;
  load8(dy, static_cast<const raw*>(a.dy) + row * a.ld_dy + col, n, vec);
  if constexpr (kMx8) {
    uint2 w = make_uint2(0u, 0u);
    uint32_t s = 0u;
    if (n > 0) {
      w = __ldcs(reinterpret_cast<const uint2*>(a.h8.codes + row * a.h8.code_pitch + col));
      s = a.h8.scales[row * a.h8.scale_pitch + (col >> 5)];
    }
    values8_mx8(w, s, h);
    if (n < 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j >= n) h[j] = 0.0f;
    }
  } else {
    typename T::V x;
    load8(x, static_cast<const raw*>(a.h) + row * a.ld_h + col, n, vec);
    x.values(h);
  }
}

// dx of one vector: h here is xh, g = dy w.
template <class T>
__device__ __forceinline__ void store_dx(const RmsNormBackwardArgs& a, int64_t row, int64_t col, int vec, float rstd, float c,
                                         const float (&xh)[8], const float (&g)[8]) {
  using raw = typename T::raw;
  const int64_t n = a.cols - col;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(rstd, __fmaf_rn(-xh[j], c, g[j]));
  if (a.dh) {
    typename T::V d;
    float u[8];
    load8(d, static_cast<const raw*>(a.dh) + row * a.ld_dh + col, n, vec);
    d.values(u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fadd_rn(v[j], u[j]);
  }
  store8<T>(static_cast<raw*>(a.dx) + row * a.ld_dx + col, v, n, vec);
}

template <class T, int kGroup, int kChunks, bool kMx8>
__global__ void __launch_bounds__(kBlockOf<kGroup>) rms_norm_backward_kernel(const __grid_constant__ RmsNormBackwardArgs a,
                                                                               const int vec) {
  constexpr int kBlock = kBlockOf<kGroup>, kRows = kBlock / kGroup;
  __shared__ float smem[32];
  __shared__ float parts[kRows > 1 ? kRows * 8 * kGroup * kChunks : 1];
  const int64_t c0 = 8 * (threadIdx.x % kGroup);
  float acc[kChunks][8], w[kChunks][8];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    weights8(a.weight, a.w_type, c0 + 8 * kGroup * c, a.cols - (c0 + 8 * kGroup * c), vec, w[c]);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[c][j] = 0.0f;
  }
  const float inv = __fdiv_rn(1.0f, (float)a.cols);
  for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kGroup; row < a.rows; row += (int64_t)gridDim.x * kRows) {
    typename T::V dy[kChunks];
    float xh[kChunks][8];
    const float rstd = a.rstd[row];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) load_backward<T, kMx8>(a, row, c0 + 8 * kGroup * c, vec, dy[c], xh[c]);
    float dot = 0.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      float d[8];
      dy[c].values(d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (c0 + 8 * kGroup * c + j < a.cols) xh[c][j] = __fmul_rn(xh[c][j], rstd);  // (past the row 0, whatever rstd is)
        dot = __fmaf_rn(__fmul_rn(d[j], w[c][j]), xh[c][j], dot);
        acc[c][j] = __fmaf_rn(d[j], xh[c][j], acc[c][j]);
      }
    }
    const float mean = __fmul_rn(group_sum<kGroup>(dot, smem), inv);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      float g[8];
      dy[c].values(g);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = __fmul_rn(g[j], w[c][j]);
      store_dx<T>(a, row, c0 + 8 * kGroup * c, vec, rstd, mean, xh[c], g);
    }
  }
  float* out = static_cast<float*>(a.workspace) + blockIdx.x * a.cols;
  if constexpr (kRows > 1) {
    constexpr int kCols = 8 * kGroup * kChunks;
    float* mine = parts + (threadIdx.x / kGroup) * kCols;
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) mine[c0 + 8 * kGroup * c + j] = acc[c][j];
    __syncthreads();
    for (int col = threadIdx.x; col < kCols && col < a.cols; col += kBlock) {
      float s = parts[col];
#pragma unroll
      for (int r = 1; r < kRows; ++r) s = __fadd_rn(s, parts[r * kCols + col]);
      out[col] = s;
    }
  } else {
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c0 + 8 * kGroup * c + j < a.cols) out[c0 + 8 * kGroup * c + j] = acc[c][j];
  }
}

// Longer rows: the rows' dot products first (into the workspace's head), then
// pieces of 2048 columns.
constexpr int kWideThreads = 256;
constexpr int kWideParts = 64;
int64_t wide_parts(int64_t rows) { return std::max<int64_t>(1, std::min<int64_t>(rows, kWideParts)); }
int64_t dots_floats(int64_t rows) { return (rows + 3) / 4 * 4; }

template <class T, bool kMx8>
__global__ void __launch_bounds__(kWideThreads) rms_norm_dots_kernel(const __grid_constant__ RmsNormBackwardArgs a,
                                                                     const int vec) {
  __shared__ float smem[32];
  const int64_t row = blockIdx.x;
  const float rstd = a.rstd[row];
  float dot = 0.0f;
  for (int64_t col = 8 * threadIdx.x; col < a.cols; col += 8 * kWideThreads) {
    typename T::V dy;
    float h[8], w[8], d[8];
    load_backward<T, kMx8>(a, row, col, vec, dy, h);
    weights8(a.weight, a.w_type, col, a.cols - col, vec, w);
    dy.values(d);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col + j < a.cols) dot = __fmaf_rn(__fmul_rn(d[j], w[j]), __fmul_rn(h[j], rstd), dot);
  }
  dot = group_sum<kWideThreads>(dot, smem);
  if (threadIdx.x == 0) static_cast<float*>(a.workspace)[row] = dot;
}

template <class T, bool kMx8>
__global__ void __launch_bounds__(kWideThreads) rms_norm_backward_wide_kernel(const __grid_constant__ RmsNormBackwardArgs a,
                                                                              const int64_t dots, const int vec) {
  const int64_t col = 8 * ((int64_t)blockIdx.x * kWideThreads + threadIdx.x);
  if (col >= a.cols) return;
  float acc[8], w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
  weights8(a.weight, a.w_type, col, a.cols - col, vec, w);
  const float inv = __fdiv_rn(1.0f, (float)a.cols);
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    typename T::V dy;
    float xh[8], g[8];
    const float rstd = a.rstd[row];
    load_backward<T, kMx8>(a, row, col, vec, dy, xh);
    dy.values(g);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      xh[j] = __fmul_rn(xh[j], rstd);
      acc[j] = __fmaf_rn(g[j], xh[j], acc[j]);
      g[j] = __fmul_rn(g[j], w[j]);
    }
    store_dx<T>(a, row, col, vec, rstd, __fmul_rn(static_cast<const float*>(a.workspace)[row], inv), xh, g);
  }
  float* out = static_cast<float*>(a.workspace) + dots + blockIdx.y * a.cols;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (col + j < a.cols) out[col + j] = acc[j];
}

// dw from the parts: 32 columns a block, eight threads a column that take every
// eighth part, then their sums in order.
__global__ void __launch_bounds__(256) rms_norm_dw_kernel(const float* __restrict__ parts, const int64_t n, const int64_t cols,
                                                          void* dw, const int type) {
  __shared__ float smem[8][33];
  const int x = threadIdx.x & 31, q = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + x;
  float s = 0.0f;
  if (col < cols)
    for (int64_t p = q; p < n; p += 8) s = __fadd_rn(s, parts[p * cols + col]);
  smem[q][x] = s;
  __syncthreads();
  if (q || col >= cols) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) s = __fadd_rn(s, smem[k][x]);
  if (type == kMxF32) static_cast<float*>(dw)[col] = s;
  else static_cast<uint16_t*>(dw)[col] = type == kMxF16 ? F16::rn(s) : Bf16::rn(s);
}

// ------------------------------------------------------------------ launch --

template <class T, int kGroup, int kChunks>
cudaError_t forward(const RmsNormArgs& a, int vec, cudaStream_t s) {
  constexpr int kRows = kBlockOf<kGroup> / kGroup;
  rms_norm_kernel<T, kGroup, kChunks><<<(unsigned)((a.rows + kRows - 1) / kRows), kBlockOf<kGroup>, 0, s>>>(a, vec);
  return cudaGetLastError();
}

template <class T>
cudaError_t forward(const RmsNormArgs& a, cudaStream_t s) {
  const int64_t b = sizeof(typename T::raw);
  auto fits = [&](const void* p, int64_t ld) { return !p || aligned(p, ld * b); };
  const int vec = fits(a.x, a.ld_x) && fits(a.residual, a.ld_residual) && fits(a.y, a.ld_y) && fits(a.h, a.ld_h) &&
                  aligned(a.weight, 0);
  if (a.cols <= 256) return forward<T, 32, 1>(a, vec, s);
  if (a.cols <= 512) return forward<T, 32, 2>(a, vec, s);
  if (a.cols <= 1024) return forward<T, 128, 1>(a, vec, s);
  if (a.cols <= 2048) return forward<T, 256, 1>(a, vec, s);
  if (a.cols <= 4096) return forward<T, 256, 2>(a, vec, s);
  if (a.cols <= 8192) return forward<T, 512, 2>(a, vec, s);
  if (a.cols <= 16384) return forward<T, 512, 4>(a, vec, s);
  rms_norm_long_kernel<T><<<(unsigned)a.rows, kLongThreads, 0, s>>>(a, vec);
  return cudaGetLastError();
}

template <class T, bool kMx8, int kGroup, int kChunks>
cudaError_t backward(const RmsNormBackwardArgs& a, int vec, cudaStream_t s) {
  constexpr int kRows = kBlockOf<kGroup> / kGroup;
  const int64_t parts = std::min<int64_t>((a.rows + kRows - 1) / kRows, parts_of(a.rows));
  rms_norm_backward_kernel<T, kGroup, kChunks, kMx8><<<(unsigned)parts, kBlockOf<kGroup>, 0, s>>>(a, vec);
  rms_norm_dw_kernel<<<(unsigned)((a.cols + 31) / 32), 256, 0, s>>>(static_cast<const float*>(a.workspace), parts, a.cols,
                                                                    a.dw, a.dw_type);
  return cudaGetLastError();
}

template <class T, bool kMx8>
cudaError_t backward(const RmsNormBackwardArgs& a, cudaStream_t s) {
  const int64_t b = sizeof(typename T::raw);
  auto fits = [&](const void* p, int64_t ld) { return !p || aligned(p, ld * b); };
  const int vec = fits(a.dy, a.ld_dy) && fits(a.h, a.ld_h) && fits(a.dh, a.ld_dh) && fits(a.dx, a.ld_dx) &&
                  aligned(a.weight, 0);
  if (a.cols <= 256) return backward<T, kMx8, 32, 1>(a, vec, s);
  if (a.cols <= 512) return backward<T, kMx8, 32, 2>(a, vec, s);
  if (a.cols <= 1024) return backward<T, kMx8, 128, 1>(a, vec, s);
  if (a.cols <= 2048) return backward<T, kMx8, 256, 1>(a, vec, s);
  if (a.cols <= 4096) return backward<T, kMx8, 256, 2>(a, vec, s);
  if (a.cols <= 8192) return backward<T, kMx8, 512, 2>(a, vec, s);
  if (a.cols <= kWideCols) return backward<T, kMx8, 512, 4>(a, vec, s);
  const int64_t dots = dots_floats(a.rows), parts = wide_parts(a.rows);
  rms_norm_dots_kernel<T, kMx8><<<(unsigned)a.rows, kWideThreads, 0, s>>>(a, vec);
  const dim3 grid((unsigned)((a.cols + 8 * kWideThreads - 1) / (8 * kWideThreads)), (unsigned)parts);
  rms_norm_backward_wide_kernel<T, kMx8><<<grid, kWideThreads, 0, s>>>(a, dots, vec);
  rms_norm_dw_kernel<<<(unsigned)((a.cols + 31) / 32), 256, 0, s>>>(static_cast<const float*>(a.workspace) + dots, parts,
                                                                    a.cols, a.dw, a.dw_type);
  return cudaGetLastError();
}

template <class T>
cudaError_t backward(const RmsNormBackwardArgs& a, cudaStream_t s) {
  return a.h ? backward<T, false>(a, s) : backward<T, true>(a, s);
}

}  // namespace

int64_t rms_norm_backward_workspace(int64_t rows, int64_t cols) {
  return 4 * (cols > kWideCols ? dots_floats(rows) + wide_parts(rows) * cols : parts_of(rows) * cols);
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
