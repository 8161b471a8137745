// MX8 quantisation and read-back: a layer's activations on their way into and
// out of what the backward pass keeps ("激活值" in the pages' accounting of
// memory; there 16 bits an element).
//
// Both are memory-bound streams: per 16-bit element 2 + 33/32 bytes.
#include <cuda_runtime.h>

#include "mx4_quant.cuh"
#include "mx8.cuh"

namespace zsm {
namespace {

using namespace mx;

constexpr int kRowThreads = 256;

// A warp takes 256 consecutive columns of one row at a time, a lane 8 of them
// and four lanes a block; V::kUnits such pieces go through each step side by
// side.
template <class V>
__global__ void __launch_bounds__(kRowThreads) mx8_quant_kernel(const __grid_constant__ Mx8QuantArgs a,
                                                                const FastDiv per_row, const uint32_t units, const int vec) {
  constexpr int kUnits = V::kUnits;
  const typename V::raw* src = static_cast<const typename V::raw*>(a.src);
  const uint32_t warps = gridDim.x * (kRowThreads / 32);
  const int lane = threadIdx.x & 31;
  const int64_t nb = (a.cols + kMxBlock - 1) / kMxBlock;
  for (uint32_t u0 = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); u0 < units; u0 += kUnits * warps) {
    V x[kUnits];
    uint32_t row[kUnits];
    int64_t col[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const uint32_t u = min(u0 + k * warps, units - 1);  // past the end: the last piece again, not stored
      row[k] = div_by(u, per_row);
      col[k] = (int64_t)(u - row[k] * per_row.d) * 256 + lane * 8;
      load8(x[k], src + row[k] * a.ld + col[k], a.cols - col[k], vec);
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const uint32_t s = scale_code8(max_of_four(x[k].max_bits()));
      const int64_t b = col[k] >> 5;
      float v[8];
      x[k].values(v);
      if (b < nb && u0 + k * warps < units) {
        *reinterpret_cast<uint2*>(a.out.codes + row[k] * a.out.code_pitch + col[k]) = encode8_mx8(v, s);
        if ((lane & 3) == 0) a.out.scales[row[k] * a.out.scale_pitch + b] = (uint8_t)s;
      }
    }
  }
}

template <class T>
__global__ void __launch_bounds__(kRowThreads) mx8_dequant_kernel(const __grid_constant__ Mx8DequantArgs a,
                                                                  const FastDiv per_row, const uint32_t units, const int vec) {
  using raw = typename T::raw;
  constexpr int kUnits = 4;
  raw* dst = static_cast<raw*>(a.dst);
  const uint32_t warps = gridDim.x * (kRowThreads / 32);
  const int lane = threadIdx.x & 31;
  for (uint32_t u0 = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); u0 < units; u0 += kUnits * warps) {
    uint32_t s[kUnits], row[kUnits];
    uint2 w[kUnits];
    int64_t col[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const uint32_t u = min(u0 + k * warps, units - 1);
      row[k] = div_by(u, per_row);
      col[k] = (int64_t)(u - row[k] * per_row.d) * 256 + lane * 8;
      const int64_t at = min(col[k], a.in.cols - 1);  // lanes past the row read its last block, and store nothing
      w[k] = __ldcs(reinterpret_cast<const uint2*>(a.in.codes + row[k] * a.in.code_pitch + (at & ~7ll)));
      s[k] = a.in.scales[row[k] * a.in.scale_pitch + (at >> 5)];
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      float v[8];
      values8_mx8(w[k], s[k], v);
      finite_in<T>(v);
      store8<T>(dst + row[k] * a.ld + col[k], v, u0 + k * warps < units ? a.in.cols - col[k] : 0, vec);
    }
  }
}

template <class V>
cudaError_t quantize_from(Mx8QuantArgs a, int sm_count, cudaStream_t s) {
  const bool flat = a.cols % kMxBlock == 0 && a.ld == a.cols && a.out.code_pitch == a.cols &&
                    a.out.scale_pitch == a.cols / kMxBlock;
  Pieces p;
  if (!pieces_of(a.rows, a.cols, flat, &p)) return cudaErrorInvalidValue;
  a.rows = p.rows, a.cols = p.cols;
  const int vec = aligned(a.src, flat ? 0 : a.ld * (int64_t)sizeof(typename V::raw)) ? 1 : 0;
  const int per_cta = V::kUnits * kRowThreads / 32;
  mx8_quant_kernel<V><<<cap_grid((p.units + per_cta - 1) / per_cta, kWaves * sm_count), kRowThreads, 0, s>>>(
      a, p.per_row, p.units, vec);
  return cudaGetLastError();
}

template <class T>
cudaError_t dequantize_to(Mx8DequantArgs a, int sm_count, cudaStream_t s) {
  const bool flat = a.in.cols % kMxBlock == 0 && a.ld == a.in.cols && a.in.code_pitch == a.in.cols &&
                    a.in.scale_pitch == a.in.cols / kMxBlock;
  Pieces p;
  if (!pieces_of(a.in.rows, a.in.cols, flat, &p)) return cudaErrorInvalidValue;
  a.in.rows = p.rows, a.in.cols = p.cols;
  const int vec = aligned(a.dst, flat ? 0 : a.ld * (int64_t)sizeof(typename T::raw)) ? 1 : 0;
  const int per_cta = 4 * kRowThreads / 32;
  mx8_dequant_kernel<T><<<cap_grid((p.units + per_cta - 1) / per_cta, kWaves * sm_count), kRowThreads, 0, s>>>(
      a, p.per_row, p.units, vec);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx8_quantize(const Mx8QuantArgs& a, int sm_count, cudaStream_t s) {
  switch (a.type) {
    case kMxBf16: return quantize_from<Vec16<Bf16>>(a, sm_count, s);
    case kMxF16: return quantize_from<Vec16<F16>>(a, sm_count, s);
    case kMxF32: return quantize_from<Vec32>(a, sm_count, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_mx8_dequantize(const Mx8DequantArgs& a, int sm_count, cudaStream_t s) {
  switch (a.type) {
    case kMxBf16: return dequantize_to<TBf16>(a, sm_count, s);
    case kMxF16: return dequantize_to<TF16>(a, sm_count, s);
    case kMxF32: return dequantize_to<TF32>(a, sm_count, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace zsm
