// MX8 quantisation and read-back: a layer's activations on their way into and
// out of what the backward pass keeps ("ZeRO：从优化器状态到残差状态的显存优化",
// section 3.1, counts them at 16 bits an element).
//
// Both are memory-bound streams: per 16-bit element 2 + 33/32 bytes.
#include <cuda_runtime.h>

#include "mx8.cuh"
#include "rows.cuh"

namespace zsm {
namespace {

using namespace mx;

constexpr int kRowThreads = 256;
constexpr int kUnits = 4;

// A warp takes up to kUnits pieces of 256 columns of one row, a lane eight columns
// of each and four lanes a block; they go through every step side by side.  Rows
// of odd length, 6000 x 2421 bf16, take 17 us to quantise and 15 to read back
// (7 each at the copy's rate; element by element 18 and 48): instructions, 70 %
// of the issue slots, for shifting unaligned words into place.
template <class T, bool kWhole>
__global__ void __launch_bounds__(kRowThreads) mx8_quant_kernel(const __grid_constant__ Mx8QuantArgs a,
                                                                const FastDiv per_row, const uint32_t units) {
  const uint32_t u = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (u >= units) return;
  const uint32_t number = div_by(u, per_row), first = (u - number * per_row.d) * (256 * kUnits), cols = (uint32_t)a.cols;
  const typename T::raw* row = row_of<T>(a.src, number, a.ld);
  const Row8 out = row_of(a.out, number);
  Fetched<typename T::V, kWhole> f[kUnits];
  const Span span = span_of<T>(a.src, a.rows, a.cols, a.ld);
#pragma unroll
  for (int k = 0; k < kUnits; ++k)
    if (first + 256 * k < cols) fetch_columns(f[k], row, Columns<kWhole>(first + 256 * k, lane, cols), span);
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    if (first + 256 * k >= cols) break;
    const Columns<kWhole> c(first + 256 * k, lane, cols);
    typename T::V x;
    float v[8];
    take_columns(x, f[k], row, c);
    x.values(v);
    store_columns8(out, c, x, v);
  }
}

template <class T, bool kWhole>
__global__ void __launch_bounds__(kRowThreads) mx8_dequant_kernel(const __grid_constant__ Mx8DequantArgs a,
                                                                  const FastDiv per_row, const uint32_t units) {
  const uint32_t u = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (u >= units) return;
  const uint32_t number = div_by(u, per_row), first = (u - number * per_row.d) * (256 * kUnits), cols = (uint32_t)a.in.cols;
  const Row8 in = row_of(a.in, number);
  typename T::raw* row = row_of<T>(a.dst, number, a.ld);
  Fetched8 f[kUnits];
#pragma unroll
  for (int k = 0; k < kUnits; ++k)
    if (first + 256 * k < cols) fetch_columns8(f[k], in, Columns<kWhole>(first + 256 * k, lane, cols));
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    if (first + 256 * k >= cols) break;
    float v[8];
    typename T::V x;
    elements8(f[k].w, v);
    scale8(v, scale_value(f[k].s));
    finite_in<T>(v);
    round_to(x, v);
    store_columns(row, Columns<kWhole>(first + 256 * k, lane, cols), x);
  }
}

// A matrix whose rows lie end to end in whole blocks, as most activations do,
// is one long row: a lane takes sixteen neighbouring elements, two lanes a
// block, and nothing but one address has to be worked out for them: 8192 x 4096
// bf16 quantised and read back in 29.7 us one after the other, its 203 MB at the
// copy's rate 31.0 (a lane to eight elements of a row: 36 to 39, three quarters
// of the issue slots busy, mostly with addresses).
constexpr int kFlat = 2;  // groups of 16 elements of a thread, side by side

// The index of a thread's group k.
__device__ __forceinline__ int64_t flat_at(int k) { return ((int64_t)blockIdx.x * kFlat + k) * kRowThreads + threadIdx.x; }

template <class T>
__device__ __forceinline__ void load16(typename T::V (&x)[2], const typename T::raw* p, bool wide) {
  if constexpr (sizeof(typename T::raw) == 2) {
    if (wide) {  // aligned to 32 bytes: one load
      uint32_t *a = words(x[0]), *b = words(x[1]);
      asm volatile("ld.global.cs.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                   : "l"(p)
                   : "memory");
      return;
    }
  }
  x[0].load(p);
  x[1].load(p + 8);
}
template <class T>
__device__ __forceinline__ void store16(typename T::raw* p, const typename T::V (&x)[2], bool wide) {
  if constexpr (sizeof(typename T::raw) == 2) {
    if (wide) {
      const uint32_t *a = words(x[0]), *b = words(x[1]);
      asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a[0]), "r"(a[1]), "r"(a[2]),
                   "r"(a[3]), "r"(b[0]), "r"(b[1]), "r"(b[2]), "r"(b[3])
                   : "memory");
      return;
    }
  }
  store_whole(p, words(x[0]));
  store_whole(p + 8, words(x[1]));
}

template <class T>
__global__ void __launch_bounds__(kRowThreads) mx8_quant_flat_kernel(const typename T::raw* src, uint8_t* codes,
                                                                     uint8_t* scales, const int64_t groups, const bool wide) {
  typename T::V x[kFlat][2];
#pragma unroll
  for (int k = 0; k < kFlat; ++k) {
    const int64_t i = flat_at(k);
    if (i < groups) load16<T>(x[k], src + 16 * i, wide);
    else x[k][0].clear(), x[k][1].clear();
  }
#pragma unroll
  for (int k = 0; k < kFlat; ++k) {
    const int64_t i = flat_at(k);
    uint32_t m = max(x[k][0].max_bits(), x[k][1].max_bits());
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    const uint32_t s = scale_code8(m);
    float v[8], u[8];
    x[k][0].values(v);
    x[k][1].values(u);
    const uint2 a = encode8_mx8(v, s), b = encode8_mx8(u, s);
    if (i < groups) {
      *reinterpret_cast<uint4*>(codes + 16 * i) = make_uint4(a.x, a.y, b.x, b.y);
      if ((i & 1) == 0) scales[i >> 1] = (uint8_t)s;
    }
  }
}

template <class T>
__global__ void __launch_bounds__(kRowThreads) mx8_dequant_flat_kernel(const uint8_t* codes, const uint8_t* scales,
                                                                       typename T::raw* dst, const int64_t groups,
                                                                       const bool wide) {
  uint4 w[kFlat];
  uint32_t s[kFlat];
#pragma unroll
  for (int k = 0; k < kFlat; ++k) {
    const int64_t i = flat_at(k);
    if (i >= groups) continue;
    w[k] = __ldcs(reinterpret_cast<const uint4*>(codes + 16 * i));
    s[k] = scales[i >> 1];
  }
#pragma unroll
  for (int k = 0; k < kFlat; ++k) {
    const int64_t i = flat_at(k);
    if (i >= groups) continue;
    const float sc = scale_value(s[k]);
    float v[8];
    typename T::V x[2];
    elements8(make_uint2(w[k].x, w[k].y), v);
    scale8(v, sc);
    finite_in<T>(v);
    round_to(x[0], v);
    elements8(make_uint2(w[k].z, w[k].w), v);
    scale8(v, sc);
    finite_in<T>(v);
    round_to(x[1], v);
    store16<T>(dst + 16 * i, x, wide);
  }
}

// The launch over an MX8 matrix, with a dense one beside it.
struct Launch {
  FastDiv per_row;
  uint32_t units;
  bool flat, whole, wide;
  unsigned grid;
  int64_t groups;
};
template <class T>
bool launch_of(const void* dense, int64_t ld, const Mx8Matrix& m, Launch* l) {
  const int64_t b = sizeof(typename T::raw);
  l->flat = m.cols % kMxBlock == 0 && ld == m.cols && m.code_pitch == m.cols && m.scale_pitch == m.cols / kMxBlock &&
            aligned(dense, 0);
  if (l->flat) {
    l->groups = m.rows * m.cols / 16;
    l->wide = (reinterpret_cast<uintptr_t>(dense) & 31u) == 0;
    const int64_t grid = (l->groups + kFlat * kRowThreads - 1) / (kFlat * kRowThreads);
    l->grid = (unsigned)grid;
    return grid <= 0x7FFFFFFFll;
  }
  const int64_t per = (m.cols + 256 * kUnits - 1) / (256 * kUnits), units = per * m.rows;
  l->per_row = fast_div((uint32_t)per), l->units = (uint32_t)units;
  l->whole = m.cols % 8 == 0 && aligned(dense, ld * b);
  l->grid = (unsigned)((units + kRowThreads / 32 - 1) / (kRowThreads / 32));
  // as FastDiv allows; more whole rows of so many columns are more memory than there is
  return units <= 0x7FFFFFFFll;
}

template <class T>
cudaError_t quantize_from(const Mx8QuantArgs& a, cudaStream_t s) {
  Launch l;
  if (!launch_of<T>(a.src, a.ld, a.out, &l)) return cudaErrorInvalidValue;
  if (l.flat)
    mx8_quant_flat_kernel<T><<<l.grid, kRowThreads, 0, s>>>(static_cast<const typename T::raw*>(a.src), a.out.codes,
                                                            a.out.scales, l.groups, l.wide);
  else if (l.whole) mx8_quant_kernel<T, true><<<l.grid, kRowThreads, 0, s>>>(a, l.per_row, l.units);
  else mx8_quant_kernel<T, false><<<l.grid, kRowThreads, 0, s>>>(a, l.per_row, l.units);
  return cudaGetLastError();
}

template <class T>
cudaError_t dequantize_to(const Mx8DequantArgs& a, cudaStream_t s) {
  Launch l;
  if (!launch_of<T>(a.dst, a.ld, a.in, &l)) return cudaErrorInvalidValue;
  if (l.flat)
    mx8_dequant_flat_kernel<T><<<l.grid, kRowThreads, 0, s>>>(a.in.codes, a.in.scales, static_cast<typename T::raw*>(a.dst),
                                                              l.groups, l.wide);
  else if (l.whole) mx8_dequant_kernel<T, true><<<l.grid, kRowThreads, 0, s>>>(a, l.per_row, l.units);
  else mx8_dequant_kernel<T, false><<<l.grid, kRowThreads, 0, s>>>(a, l.per_row, l.units);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx8_quantize(const Mx8QuantArgs& a, int, cudaStream_t s) {
  switch (a.type) {
    case kMxBf16: return quantize_from<TBf16>(a, s);
    case kMxF16: return quantize_from<TF16>(a, s);
    case kMxF32: return quantize_from<TF32>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_mx8_dequantize(const Mx8DequantArgs& a, int, cudaStream_t s) {
  switch (a.type) {
    case kMxBf16: return dequantize_to<TBf16>(a, s);
    case kMxF16: return dequantize_to<TF16>(a, s);
    case kMxF32: return dequantize_to<TF32>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace zsm
