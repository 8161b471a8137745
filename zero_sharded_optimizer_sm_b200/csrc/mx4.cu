// MX4 quantisation, read-back, and the collectives that move MX4 data: the
// all-gather of the owners' 16-bit parameters into N ranks' MX4 buffers and
// the reduce-scatter of N ranks' MX4 gradients ("ZERO训练技术", sections
// "ZeRO-1" to "ZeRO-3", with a quarter of the bytes per element that moves).
//
// All are memory-bound streams: per element a 16-bit quantisation moves
// 2 + 17/32 bytes, the gather 2 + 17N/32 and the reduce 17N/32 + 2.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "device_math.cuh"
#include "mx4.cuh"

namespace zsm {
namespace {

using namespace dev;
using namespace mx;

struct TBf16 {
  using raw = uint16_t;
  static __device__ __forceinline__ float f32(raw h) { return Bf16::f32(h); }
  static __device__ __forceinline__ raw rn(float x) { return Bf16::rn(x); }
};
struct TF16 {
  using raw = uint16_t;
  static __device__ __forceinline__ float f32(raw h) { return F16::f32(h); }
  static __device__ __forceinline__ raw rn(float x) { return F16::rn(x); }
};
struct TF32 {
  using raw = float;
  static __device__ __forceinline__ float f32(raw x) { return x; }
  static __device__ __forceinline__ raw rn(float x) { return x; }
};

// Eight consecutive elements, of which the first n exist (the others are 0).
// vec: the address is 16-byte aligned whenever n = 8.
template <class T>
__device__ __forceinline__ void load8(const typename T::raw* p, int64_t n, bool vec, typename T::raw (&r)[8]) {
  if (vec && n >= 8) {
    if constexpr (sizeof(typename T::raw) == 2) {
      const uint4 w = ld_stream(reinterpret_cast<const uint16_t*>(p));
      const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r[2 * j] = (uint16_t)(x[j] & 0xFFFFu);
        r[2 * j + 1] = (uint16_t)(x[j] >> 16);
      }
    } else {
      const float4 a = ld_stream(reinterpret_cast<const float*>(p)), b = ld_stream(reinterpret_cast<const float*>(p) + 4);
      r[0] = a.x, r[1] = a.y, r[2] = a.z, r[3] = a.w, r[4] = b.x, r[5] = b.y, r[6] = b.z, r[7] = b.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = j < n ? p[j] : typename T::raw(0);
  }
}

template <class T>
__device__ __forceinline__ void store8(typename T::raw* p, int64_t n, bool vec, const float (&v)[8]) {
  if (vec && n >= 8) {
    if constexpr (sizeof(typename T::raw) == 2) {
      const uint16_t h[8] = {T::rn(v[0]), T::rn(v[1]), T::rn(v[2]), T::rn(v[3]),
                             T::rn(v[4]), T::rn(v[5]), T::rn(v[6]), T::rn(v[7])};
      st_stream(reinterpret_cast<uint16_t*>(p), pack8(h));
    } else {
      st_stream(reinterpret_cast<float*>(p), make_float4(v[0], v[1], v[2], v[3]));
      st_stream(reinterpret_cast<float*>(p) + 4, make_float4(v[4], v[5], v[6], v[7]));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = T::rn(v[j]);
  }
}

__device__ __forceinline__ uint32_t max_bits8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  return m;
}

// A quarter block (8 elements) held by one lane of four: its codes and, the
// same in the four lanes, the block's scale byte.  `block` and the lane's
// place in the block number the random numbers.
__device__ __forceinline__ uint32_t encode_quarter(float (&v)[8], int stochastic, uint64_t block, int c, uint64_t seed,
                                                   uint32_t& s) {
  uint32_t m = max_bits8(v);
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  s = scale_code(m);
  const float inv = inverse_scale(s);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], inv);
  const uint32_t w = stochastic ? encode8_stochastic(v, block, c, seed) : encode8(v);
  return s == 255u ? 0u : w;
}

// ---------------------------------------------------- quantise along rows --

// A warp takes 256 consecutive columns of one row at a time, a lane 8 of them
// and four lanes a block; kUnits such pieces are loaded before any is used.
constexpr int kRowThreads = 256;
constexpr int kUnits = 2;

template <class T>
__global__ void __launch_bounds__(kRowThreads) mx_rows_kernel(const __grid_constant__ MxQuantArgs a,
                                                              const FastDiv per_row, const uint32_t units, const int vec) {
  using raw = typename T::raw;
  const raw* src = static_cast<const raw*>(a.src);
  const uint32_t warps = gridDim.x * (kRowThreads / 32);
  const int lane = threadIdx.x & 31;
  const int64_t nb = (a.cols + kMxBlock - 1) / kMxBlock;
  for (uint32_t u0 = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); u0 < units; u0 += kUnits * warps) {
    raw x[kUnits][8];
    int64_t row[kUnits], col[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const uint32_t u = u0 + k * warps;
      if (u < units) {
        const uint32_t r = div_by(u, per_row);
        row[k] = r;
        col[k] = (int64_t)(u - r * per_row.d) * 256 + lane * 8;
        load8<T>(src + row[k] * a.ld + col[k], a.cols - col[k], vec, x[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      if (u0 + k * warps >= units) break;  // the same for the whole warp
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = T::f32(x[k][j]);
      const int64_t b = col[k] >> 5;
      uint32_t s;
      const uint32_t w = encode_quarter(v, a.stochastic, (uint64_t)(row[k] * nb + b), lane & 3, a.seed, s);
      if (b < nb) {
        *reinterpret_cast<uint32_t*>(a.out.codes + row[k] * a.out.code_pitch + (col[k] >> 1)) = w;
        if ((lane & 3) == 0) a.out.scales[row[k] * a.out.scale_pitch + b] = (uint8_t)s;
      }
    }
  }
}

// --------------------------------------- quantise down columns (and rows) --

// A CTA takes a tile of 128 rows and 64 columns: 16-byte loads (kept in
// registers for the blocks along the rows when those are wanted too) go
// through shared memory, from which a thread reads one block of 32 elements
// of one column.  Four neighbouring lanes take the four blocks of a column
// (64 contiguous bytes of the result).  Row r's eight chunks of 8 elements
// are rotated by r / 32 chunks, which puts the four blocks' reads on
// different banks.
constexpr int kTileRows = 128;
constexpr int kTileCols = 64;

template <class T, bool kFromMx>
__global__ void __launch_bounds__(256) mx_tile_kernel(const __grid_constant__ MxQuantArgs a, const uint32_t tiles_x,
                                                      const int vec) {
  using raw = typename T::raw;
  __shared__ __align__(16) raw tile[kTileRows][kTileCols];
  const raw* src = static_cast<const raw*>(a.src);
  const int64_t r0 = (int64_t)(blockIdx.x / tiles_x) * kTileRows;
  const int64_t c0 = (int64_t)(blockIdx.x % tiles_x) * kTileCols;
  const int t = threadIdx.x;
  const int cv = t & 7;
  const int64_t col = c0 + 8 * cv;
  raw x[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = r0 + (t >> 3) + 32 * i;
    const int64_t left = row < a.rows ? a.cols - col : 0;
    if constexpr (kFromMx) {
      // the elements' values are exact in bf16 (three significant bits and
      // the same exponent range as binary32)
      uint32_t h[4] = {0u, 0u, 0u, 0u};
      float sc = 0.0f;
      if (left > 0) {
        decode8(*reinterpret_cast<const uint32_t*>(a.from.codes + row * a.from.code_pitch + (col >> 1)), h);
        sc = scale_value(a.from.scales[row * a.from.scale_pitch + (col >> 5)]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = half2_float2(h[j]);
        x[i][2 * j] = T::rn(__fmul_rn(f.x, sc));
        x[i][2 * j + 1] = T::rn(__fmul_rn(f.y, sc));
      }
    } else {
      load8<T>(src + row * a.ld + col, left, vec, x[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (t >> 3) + 32 * i;
    raw* d = &tile[r][8 * ((cv + i) & 7)];
#pragma unroll
    for (int j = 0; j < 8; j += 16 / sizeof(raw)) {
      uint4 w;
      raw* p = reinterpret_cast<raw*>(&w);
#pragma unroll
      for (int k = 0; k < (int)(16 / sizeof(raw)); ++k) p[k] = x[i][j + k];
      *reinterpret_cast<uint4*>(d + j) = w;
    }
  }
  if (a.out.codes) {
    const int64_t nb = (a.cols + kMxBlock - 1) / kMxBlock, b = col >> 5;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = r0 + (t >> 3) + 32 * i;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = T::f32(x[i][j]);
      uint32_t s;
      const uint32_t w = encode_quarter(v, a.stochastic, (uint64_t)(row * nb + b), cv & 3, a.seed, s);
      if (row < a.rows && b < nb) {
        *reinterpret_cast<uint32_t*>(a.out.codes + row * a.out.code_pitch + (col >> 1)) = w;
        if ((cv & 3) == 0) a.out.scales[row * a.out.scale_pitch + b] = (uint8_t)s;
      }
    }
  }
  __syncthreads();
  const int64_t nbt = (a.rows + kMxBlock - 1) / kMxBlock;
  const int q = t & 3, c = t >> 2;
  const int64_t b = r0 / kMxBlock + q, oc = c0 + c;
  if (b >= nbt || oc >= a.cols) return;
  const int at = (c + 8 * q) & 63;
  float v[32];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    v[j] = T::f32(tile[32 * q + j][at]);
    m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  }
  const uint32_t s = scale_code(m);
  const float inv = inverse_scale(s);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = __fmul_rn(v[8 * k + j], inv);
    w[k] = a.stochastic ? encode8_stochastic(e, (uint64_t)(oc * nbt + b), k, a.seed) : encode8(e);
    if (s == 255u) w[k] = 0u;
  }
  *reinterpret_cast<uint4*>(a.out_t.codes + oc * a.out_t.code_pitch + 16 * b) = make_uint4(w[0], w[1], w[2], w[3]);
  a.out_t.scales[oc * a.out_t.scale_pitch + b] = (uint8_t)s;
}

// --------------------------------------------------------------- read back --

template <class T>
__global__ void __launch_bounds__(kRowThreads) mx_dequant_kernel(const __grid_constant__ MxDequantArgs a,
                                                                 const FastDiv per_row, const uint32_t units, const int vec) {
  using raw = typename T::raw;
  raw* dst = static_cast<raw*>(a.dst);
  const uint32_t warps = gridDim.x * (kRowThreads / 32);
  const int lane = threadIdx.x & 31;
  for (uint32_t u0 = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); u0 < units; u0 += kUnits * warps) {
    uint32_t w[kUnits], s[kUnits];
    int64_t row[kUnits], col[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const uint32_t u = u0 + k * warps;
      col[k] = a.in.cols;
      if (u < units) {
        const uint32_t r = div_by(u, per_row);
        row[k] = r;
        col[k] = (int64_t)(u - r * per_row.d) * 256 + lane * 8;
        if (col[k] < a.in.cols) {
          w[k] = *reinterpret_cast<const uint32_t*>(a.in.codes + row[k] * a.in.code_pitch + (col[k] >> 1));
          s[k] = a.in.scales[row[k] * a.in.scale_pitch + (col[k] >> 5)];
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      if (col[k] >= a.in.cols) continue;
      uint32_t h[4];
      decode8(w[k], h);
      const float sc = scale_value(s[k]);
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = half2_float2(h[j]);
        v[2 * j] = __fmul_rn(f.x, sc);
        v[2 * j + 1] = __fmul_rn(f.y, sc);
      }
      store8<T>(dst + row[k] * a.ld + col[k], a.in.cols - col[k], vec, v);
    }
  }
}

// -------------------------------------------------------------- all-gather --

// A lane quantises 8 of the owners' elements (four lanes a block) and writes
// the block's codes and scale to every rank.
template <class F>
__global__ void __launch_bounds__(kThreads) mx_gather_kernel(const __grid_constant__ MxGatherArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t n_blocks = (a.n + kMxBlock - 1) / kMxBlock;
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  // whole warps go round the loop together: the last block's missing lanes quantise zeros
  const int64_t n_lanes = ((n_blocks * 4 + 31) / 32) * 32;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n_lanes; i += stride) {
    const int64_t e = i * 8;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (e < a.n) {
      const uint16_t* src = a.uniform ? a.src[0] : a.src[(a.lo + e) / a.shard];
      x = ld_stream(src + a.lo + e);
    }
    float v[8] = {F::lo(x.x), F::hi(x.x), F::lo(x.y), F::hi(x.y), F::lo(x.z), F::hi(x.z), F::lo(x.w), F::hi(x.w)};
    uint32_t s;
    const uint32_t w = encode_quarter(v, 0, 0, 0, 0, s);
    if ((i >> 2) < n_blocks) {
      for (int r = 0; r < a.n_ranks; ++r) {
        *reinterpret_cast<uint32_t*>(a.codes[r] + 4 * i) = w;
        if ((lane & 3) == 0) a.scales[r][i >> 2] = (uint8_t)s;
      }
    }
  }
}

// ---------------------------------------------------------- reduce-scatter --

// A lane sums 8 elements (4 bytes of codes and the block's scale byte from
// each rank), in rank order.  element * scale is exact in binary32 (three
// significant bits), so the fused multiply-add rounds once, as adding the
// element's value does.
template <class F>
__global__ void __launch_bounds__(kThreads) mx_reduce_kernel(const __grid_constant__ MxReduceArgs a) {
  double sq = 0.0;
  unsigned long long nf = 0;
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  const int64_t n_vec = a.n / kVec;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n_vec; i += stride) {
    float acc[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) acc[j] = 0.0f;
    for (int r0 = 0; r0 < a.n_ranks; r0 += 8) {
      uint32_t w[8], s[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (r0 + k < a.n_ranks) {
          w[k] = __ldcs(reinterpret_cast<const uint32_t*>(a.codes[r0 + k]) + i);
          s[k] = a.scales[r0 + k][i >> 2];
        }
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (r0 + k < a.n_ranks) {
          uint32_t h[4];
          decode8(w[k], h);
          const float sc = scale_value(s[k]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = half2_float2(h[j]);
            acc[2 * j] = __fmaf_rn(f.x, sc, acc[2 * j]);
            acc[2 * j + 1] = __fmaf_rn(f.y, sc, acc[2 * j + 1]);
          }
        }
    }
    uint16_t g16[kVec];
    float g[kVec];
    mean_bf16<F>(acc, a.inv_n, g16, g, sq, nf);
    st_stream(a.shard_out + i * kVec, pack8(g16));
  }
  norm_epilogue<kThreads>(a.ns, sq, nf, a.accumulate);
}

int cap_grid(int64_t want, int cap) { return (int)std::max<int64_t>(1, std::min<int64_t>(want, cap)); }

bool aligned(const void* p, int64_t pitch_bytes) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)pitch_bytes) & 15u) == 0;
}

// Pieces of 256 columns over all rows; a matrix whose rows lie end to end in
// whole blocks is taken as one row, so that narrow rows fill the warps.
struct Pieces {
  int64_t rows, cols;
  FastDiv per_row;
  uint32_t units;
};
bool pieces_of(int64_t rows, int64_t cols, bool end_to_end, Pieces* p) {
  if (end_to_end) {
    cols *= rows;
    rows = 1;
  }
  const int64_t per = (cols + 255) / 256;
  if (per * rows > 0x7FFFFFFFll - (1 << 24)) return false;  // (rows * cols < 2^38)
  *p = Pieces{rows, cols, fast_div((uint32_t)per), (uint32_t)(per * rows)};
  return true;
}

template <class T>
cudaError_t quantize_rows(MxQuantArgs a, int sm_count, cudaStream_t s) {
  const bool flat = a.cols % kMxBlock == 0 && a.ld == a.cols && a.out.code_pitch == a.cols / 2 &&
                    a.out.scale_pitch == a.cols / kMxBlock;
  Pieces p;
  if (!pieces_of(a.rows, a.cols, flat, &p)) return cudaErrorInvalidValue;
  a.rows = p.rows, a.cols = p.cols;
  const int vec = aligned(a.src, flat ? 0 : a.ld * (int64_t)sizeof(typename T::raw)) ? 1 : 0;
  const int per_cta = kUnits * kRowThreads / 32;
  mx_rows_kernel<T><<<cap_grid((p.units + per_cta - 1) / per_cta, 8 * sm_count), kRowThreads, 0, s>>>(a, p.per_row,
                                                                                                     p.units, vec);
  return cudaGetLastError();
}

template <class T, bool kFromMx>
cudaError_t quantize_tiles(const MxQuantArgs& a, cudaStream_t s) {
  const int64_t tx = (a.cols + kTileCols - 1) / kTileCols, ty = (a.rows + kTileRows - 1) / kTileRows;
  if (tx * ty > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const int vec = kFromMx || aligned(a.src, a.ld * (int64_t)sizeof(typename T::raw)) ? 1 : 0;
  mx_tile_kernel<T, kFromMx><<<(unsigned)(tx * ty), 256, 0, s>>>(a, (uint32_t)tx, vec);
  return cudaGetLastError();
}

template <class T>
cudaError_t quantize_from(const MxQuantArgs& a, int sm_count, cudaStream_t s) {
  return a.out_t.codes ? quantize_tiles<T, false>(a, s) : quantize_rows<T>(a, sm_count, s);
}

template <class T>
cudaError_t dequantize_to(MxDequantArgs a, int sm_count, cudaStream_t s) {
  const bool flat = a.in.cols % kMxBlock == 0 && a.ld == a.in.cols && a.in.code_pitch == a.in.cols / 2 &&
                    a.in.scale_pitch == a.in.cols / kMxBlock;
  Pieces p;
  if (!pieces_of(a.in.rows, a.in.cols, flat, &p)) return cudaErrorInvalidValue;
  a.in.rows = p.rows, a.in.cols = p.cols;
  const int vec = aligned(a.dst, flat ? 0 : a.ld * (int64_t)sizeof(typename T::raw)) ? 1 : 0;
  const int per_cta = kUnits * kRowThreads / 32;
  mx_dequant_kernel<T><<<cap_grid((p.units + per_cta - 1) / per_cta, 8 * sm_count), kRowThreads, 0, s>>>(
      a, p.per_row, p.units, vec);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx_quantize(const MxQuantArgs& a, int sm_count, cudaStream_t s) {
  if (a.from.codes) return quantize_tiles<TBf16, true>(a, s);
  switch (a.type) {
    case kMxBf16: return quantize_from<TBf16>(a, sm_count, s);
    case kMxF16: return quantize_from<TF16>(a, sm_count, s);
    case kMxF32: return quantize_from<TF32>(a, sm_count, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_mx_dequantize(const MxDequantArgs& a, int sm_count, cudaStream_t s) {
  switch (a.type) {
    case kMxBf16: return dequantize_to<TBf16>(a, sm_count, s);
    case kMxF16: return dequantize_to<TF16>(a, sm_count, s);
    case kMxF32: return dequantize_to<TF32>(a, sm_count, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_mx_gather(const MxGatherArgs& a, int sm_count, cudaStream_t s) {
  const int grid = cap_grid((a.n / 8 + kThreads - 1) / kThreads + 1, 8 * sm_count);
  if (a.fmt == kFmtF16) mx_gather_kernel<F16><<<grid, kThreads, 0, s>>>(a);
  else mx_gather_kernel<Bf16><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_mx_reduce(const MxReduceArgs& a, int sm_count, cudaStream_t s) {
  const int grid = cap_grid((a.n / kVec + kThreads - 1) / kThreads, std::min(8 * sm_count, kMaxGrid));
  if (a.fmt == kFmtF16) mx_reduce_kernel<F16><<<grid, kThreads, 0, s>>>(a);
  else mx_reduce_kernel<Bf16><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace zsm
