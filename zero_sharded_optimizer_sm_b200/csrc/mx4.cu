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
#include <type_traits>

#include "device_math.cuh"
#include "mx4.cuh"
#include "mx4_quant.cuh"
#include "mx8.cuh"

namespace zsm {
namespace {

using namespace dev;
using namespace mx;

// ---------------------------------------------------- quantise along rows --

// A warp takes 256 consecutive columns of one row at a time, a lane 8 of them
// and four lanes a block; V::kUnits such pieces go through each step side by
// side, which hides the loads, the exchange between the four lanes and the
// conversions behind one another (8192 x 2048 bf16: 20 us one by one, 11.3 side
// by side; its 42 MB take 6.5 at the copy's rate).  No unit is at its limit
// then: by the counters the issue slots are 60 % used, the integer units 58 %,
// and 42 % of the warps that could be there are.  2048 x 6144 binary32 takes
// 10.7 us to nearest and 22.5 stochastically: the generator and its rounding
// double the instructions (integer units 67 %).
constexpr int kRowThreads = 256;

template <class V, bool kStochastic>
__global__ void __launch_bounds__(kRowThreads) mx_rows_kernel(const __grid_constant__ MxQuantArgs a,
                                                              const FastDiv per_row, const uint32_t units, const int vec,
                                                              const uint32_t ctas) {
  constexpr int kUnits = V::kUnits;
  pdl_trigger();
  if (blockIdx.x >= ctas) {  // the CTAs after those write another matrix's scale pieces
    write_pieces(a.pieces, (blockIdx.x - ctas) * (kRowThreads / 32) + (threadIdx.x >> 5));
    return;
  }
  const typename V::raw* src = static_cast<const typename V::raw*>(a.src);
  const uint32_t warps = ctas * (kRowThreads / 32);
  const int lane = threadIdx.x & 31;
  const int64_t nb = (a.cols + kMxBlock - 1) / kMxBlock;
  for (uint32_t u0 = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); u0 < units; u0 += kUnits * warps) {
    V x[kUnits];
    uint32_t row[kUnits], m[kUnits];
    int64_t col[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const uint32_t u = min(u0 + k * warps, units - 1);  // past the end: the last piece again, not stored
      row[k] = div_by(u, per_row);
      col[k] = (int64_t)(u - row[k] * per_row.d) * 256 + lane * 8;
      load8(x[k], src + row[k] * a.ld + col[k], a.cols - col[k], vec);
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) m[k] = x[k].max_bits();
#pragma unroll
    for (int k = 0; k < kUnits; ++k) m[k] = max(m[k], __shfl_xor_sync(0xFFFFFFFFu, m[k], 1));
#pragma unroll
    for (int k = 0; k < kUnits; ++k) m[k] = max(m[k], __shfl_xor_sync(0xFFFFFFFFu, m[k], 2));
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const uint32_t s = scale_code(m[k]);
      const int64_t b = col[k] >> 5;
      const uint32_t w = encode<kStochastic>(x[k], s, (uint64_t)(row[k] * nb + b), lane & 3, a.seed);
      if (b < nb && u0 + k * warps < units) {
        *reinterpret_cast<uint32_t*>(a.out.codes + row[k] * a.out.code_pitch + (col[k] >> 1)) = w;
        if ((lane & 3) == 0) a.out.scales[row[k] * a.out.scale_pitch + b] = (uint8_t)s;
      }
    }
  }
}

// --------------------------------------- quantise down columns (and rows) --

// A CTA takes a tile of 128 rows and 128 columns of 16-bit elements (64 of
// 32-bit ones): 16-byte loads, kept in registers for the blocks along the
// rows when those are wanted too, go through shared memory, from which a
// thread reads one block of 32 elements of each of the columns that share a
// 32-bit word.  Four neighbouring lanes take the four blocks of a column (64
// contiguous bytes of the result).  Row r's words are rotated by 8 (r / 32),
// which puts the four blocks' reads on different banks.
//
// 8192 x 2048 bf16 takes 10.2 us down the columns and 14.7 both ways (6.5 and
// 7.9 at the copy's rate): loads that all CTAs of a wave wait for at once
// (issue slots 48 % used, 41 % of the warps).  An MX4 matrix's transpose takes
// 13.5 of 2.7: its elements go through the tile as 16-bit values, at twice the
// instructions of a dense one's.
constexpr int kTileRows = 128;
constexpr int kTileWords = 64;  // 32-bit words of a tile's row

// What a tile is read from: a dense matrix, an MX4 one, an MX8 one.
enum Source { kDense, kFromMx4, kFromMx8 };

template <class V, Source kFrom, bool kRows, bool kStochastic>
__device__ __forceinline__ void quantize_tile(const MxQuantArgs& a, uint32_t index, uint32_t tiles_x, int vec,
                                              uint32_t (&tile)[kTileRows][kTileWords]) {
  using raw = typename V::raw;
  constexpr int kPer = 4 / sizeof(raw);           // columns in a word
  constexpr int kTileCols = kTileWords * kPer;
  constexpr int kVecs = kTileCols / 8;            // vectors of a tile's row
  constexpr int kLoads = kTileRows * kVecs / 256; // of a thread
  constexpr int kChunks = 2 / kPer;               // 16-byte chunks of a vector
  const raw* src = static_cast<const raw*>(a.src);
  const int64_t r0 = (int64_t)(index / tiles_x) * kTileRows;
  const int64_t c0 = (int64_t)(index % tiles_x) * kTileCols;
  const int t = threadIdx.x;
  const int cv = t % kVecs, rv = t / kVecs;
  const int64_t col = c0 + 8 * cv;
  V x[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int64_t row = r0 + rv + (256 / kVecs) * i;
    const int64_t left = row < a.rows ? a.cols - col : 0;
    if constexpr (kFrom != kDense) {
      // the elements' values are exact in bf16: three or four significant bits
      // and the same exponent range as binary32
      using Codes = typename std::conditional<kFrom == kFromMx4, uint32_t, uint2>::type;
      Codes w = {};
      uint32_t sc = 0u;
      if (left > 0) {
        w = *reinterpret_cast<const Codes*>(a.from.codes + row * a.from.code_pitch + (kFrom == kFromMx4 ? col >> 1 : col));
        sc = a.from.scales[row * a.from.scale_pitch + (col >> 5)];
      }
      float v[8];
      if constexpr (kFrom == kFromMx4) values8(w, sc, v);
      else values8_mx8(w, sc, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[i].w[j] = pack2(Bf16::rn(v[2 * j]), Bf16::rn(v[2 * j + 1]));
        if (2 * j + 1 >= left) x[i].w[j] = 2 * j >= left ? 0u : x[i].w[j] & 0xFFFFu;
      }
    } else {
      load8(x[i], src + row * a.ld + col, left, vec);
    }
  }
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = rv + (256 / kVecs) * i;
    const uint4* p = reinterpret_cast<const uint4*>(&x[i]);
#pragma unroll
    for (int k = 0; k < kChunks; ++k)
      *reinterpret_cast<uint4*>(&tile[r][4 * ((kChunks * cv + k + 2 * (r >> 5)) & 15)]) = p[k];
  }
  if constexpr (kRows) {
    const int64_t nb = (a.cols + kMxBlock - 1) / kMxBlock, b = col >> 5;
    uint32_t m[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) m[i] = x[i].max_bits();
#pragma unroll
    for (int i = 0; i < kLoads; ++i) m[i] = max_of_four(m[i]);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int64_t row = r0 + rv + (256 / kVecs) * i;
      const uint32_t s = scale_code(m[i]);
      const uint32_t w = encode<kStochastic>(x[i], s, (uint64_t)(row * nb + b), cv & 3, a.seed);
      if (row < a.rows && b < nb) {
        *reinterpret_cast<uint32_t*>(a.out.codes + row * a.out.code_pitch + (col >> 1)) = w;
        if ((cv & 3) == 0) a.out.scales[row * a.out.scale_pitch + b] = (uint8_t)s;
      }
    }
  }
  __syncthreads();
  const int64_t nbt = (a.rows + kMxBlock - 1) / kMxBlock;
  const int q = t & 3, word = t >> 2;
  const int64_t b = r0 / kMxBlock + q;
  const int64_t oc = c0 + kPer * word;
  if (b >= nbt || oc >= a.cols) return;
  const uint32_t* column = &tile[32 * q][(word + 8 * q) & (kTileWords - 1)];
  uint32_t x32[32];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    x32[j] = column[j * kTileWords];
    if constexpr (kPer == 2) m = V::larger(m, x32[j]);
    else m = max(m, x32[j] & 0x7FFFFFFFu);
  }
  m &= kPer == 2 ? 0x7FFF7FFFu : 0x7FFFFFFFu;
#pragma unroll
  for (int h = 0; h < kPer; ++h) {
    if (oc + h >= a.cols) break;
    auto value = [&](int j) -> float {
      if constexpr (kPer == 2) return h ? V::hi(x32[j]) : V::lo(x32[j]);
      else return __uint_as_float(x32[j]);
    };
    uint32_t top;
    if constexpr (kPer == 2) top = __float_as_uint(h ? V::hi(m) : V::lo(m));
    else top = m;
    const uint32_t s = scale_code(top);
    const float inv = inverse_scale(s);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = value(8 * k + j);
      scale_by(e, inv);
      w[k] = kStochastic ? encode8_stochastic(e, (uint64_t)((oc + h) * nbt + b), k, a.seed) : encode8(e);
      if (s == 255u) w[k] = 0u;
    }
    *reinterpret_cast<uint4*>(a.out_t.codes + (oc + h) * a.out_t.code_pitch + 16 * b) = make_uint4(w[0], w[1], w[2], w[3]);
    a.out_t.scales[(oc + h) * a.out_t.scale_pitch + b] = (uint8_t)s;
  }
}

template <class V, Source kFrom, bool kRows, bool kStochastic>
__global__ void __launch_bounds__(256, 4) mx_tile_kernel(const __grid_constant__ MxQuantArgs a, const uint32_t tiles_x,
                                                         const int vec) {
  __shared__ __align__(16) uint32_t tile[kTileRows][kTileWords];
  pdl_trigger();
  quantize_tile<V, kFrom, kRows, kStochastic>(a, blockIdx.x, tiles_x, vec, tile);
}

// The three matrices of a linear layer's backward pass, one after another in
// the grid.
struct TileCounts {
  uint32_t dy, x;           // CTAs of dy, of dy and x
  uint32_t dy_x, x_x, w_x;  // tiles along a row
  int dy_vec, x_vec;
};
template <class V, bool kStochastic, bool kX8>
__global__ void __launch_bounds__(256, 4) mx_backward_kernel(const __grid_constant__ MxBackwardArgs a, const TileCounts n) {
  __shared__ __align__(16) uint32_t tile[kTileRows][kTileWords];
  pdl_trigger();
  if (blockIdx.x < n.dy) quantize_tile<V, kDense, true, kStochastic>(a.dy, blockIdx.x, n.dy_x, n.dy_vec, tile);
  else if (blockIdx.x < n.x) {
    if constexpr (kX8) quantize_tile<Vec16<Bf16>, kFromMx8, false, false>(a.x, blockIdx.x - n.dy, n.x_x, 1, tile);
    else quantize_tile<V, kDense, false, false>(a.x, blockIdx.x - n.dy, n.x_x, n.x_vec, tile);
  } else quantize_tile<Vec16<Bf16>, kFromMx4, false, false>(a.w, blockIdx.x - n.x, n.w_x, 1, tile);
}

// --------------------------------------------------------------- read back --

// As mx_rows_kernel: a lane turns 4 bytes of codes into 8 elements, kUnits
// pieces of 256 columns side by side.
template <class T>
__global__ void __launch_bounds__(kRowThreads) mx_dequant_kernel(const __grid_constant__ MxDequantArgs a,
                                                                 const FastDiv per_row, const uint32_t units, const int vec) {
  using raw = typename T::raw;
  constexpr int kUnits = 4;
  raw* dst = static_cast<raw*>(a.dst);
  const uint32_t warps = gridDim.x * (kRowThreads / 32);
  const int lane = threadIdx.x & 31;
  for (uint32_t u0 = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); u0 < units; u0 += kUnits * warps) {
    uint32_t w[kUnits], s[kUnits], row[kUnits];
    int64_t col[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const uint32_t u = min(u0 + k * warps, units - 1);
      row[k] = div_by(u, per_row);
      col[k] = (int64_t)(u - row[k] * per_row.d) * 256 + lane * 8;
      const int64_t at = min(col[k], a.in.cols - 1);  // lanes past the row read its last block, and store nothing
      w[k] = __ldcs(reinterpret_cast<const uint32_t*>(a.in.codes + row[k] * a.in.code_pitch + ((at >> 3) << 2)));
      s[k] = a.in.scales[row[k] * a.in.scale_pitch + (at >> 5)];
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      float v[8];
      values8(w[k], s[k], v);
      const int64_t n = u0 + k * warps < units ? a.in.cols - col[k] : 0;
      raw* p = dst + row[k] * a.ld + col[k];
      store8<T>(p, v, n, vec);
    }
  }
}

// -------------------------------------------------------------- all-gather --

// A lane quantises a block of the owners' elements and writes its codes (16
// bytes) and scale to every rank: a warp's scales fill a sector, and there is
// nothing to exchange.  Eight ranks, 16.8M elements: 17.8 us, 5.9 TB/s of its
// 105 MB (four lanes to a block, with four bytes of codes each: 21.6).
template <class F>
__global__ void __launch_bounds__(kThreads) mx_gather_kernel(const __grid_constant__ MxGatherArgs a) {
  const int64_t n_blocks = (a.n + kMxBlock - 1) / kMxBlock;
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  for (int64_t b = (int64_t)blockIdx.x * kThreads + threadIdx.x; b < n_blocks; b += stride) {
    Vec16<F> x[4];
    uint32_t m = 0, w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t e = b * kMxBlock + 8 * k;
      const uint16_t* src = a.src[0];
      if (!a.uniform && e < a.n) src = a.src[(a.lo + e) / a.shard];
      x[k].load_if(src + a.lo + e, e < a.n);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) m = max(m, x[k].max_bits());
    const uint32_t s = scale_code(m);
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = encode<false>(x[k], s, 0, 0, 0);
    for (int r = 0; r < a.n_ranks; ++r) {
      *reinterpret_cast<uint4*>(a.codes[r] + 16 * b) = make_uint4(w[0], w[1], w[2], w[3]);
      a.scales[r][b] = (uint8_t)s;
    }
  }
}

// ---------------------------------------------------------- reduce-scatter --

// A lane sums 16 elements (8 bytes of codes and the block's scale byte from
// each rank), in rank order; eight ranks' loads are out at a time.
// element * scale is exact in binary32 (three significant bits), so the fused
// multiply-add rounds once, as adding the element's value does.
//
// What bounds it is mostly instructions (issue slots 65 % used by the counters,
// the integer units 56 %), so where the first ranks' scales for a block
// differ by no more than 2^4 -- nearly always, of gradients -- they are summed
// in binary16, two elements at a time: with 2^low the smallest scale every
// term is a whole number of 2^low / 2, up to 6 * 16 * 2, and eight of them
// stay below binary16's 2^11.  So neither that sum nor the one in binary32
// that it stands for rounds anything, and they are equal; only one conversion
// to binary32 is left for all ranks.  More ranks than that are added in
// binary32.
// Eight ranks, 16.8M elements: 25.1 us, 4.2 TB/s of its 105 MB (all in binary32
// 30.3, and 34.2 with the elements put together by integer operations instead
// of the conversion unit); four ranks 20.0.
// kWide ranks at a time; kFull: the ranks are a multiple of it.
constexpr uint32_t kNearScales = 4;
constexpr uint32_t kPlainScale = 240;  // up to it a rank's value, and what is added to it, stay finite
template <class F, int kWide, bool kFull>
__global__ void __launch_bounds__(kThreads, kWide == 8 ? 4 : 5) mx_reduce_kernel(const __grid_constant__ MxReduceArgs a) {
  double sq = 0.0;
  unsigned nf = 0;
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  const int64_t n_vec = (a.n + 15) / 16;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n_vec; i += stride) {
    float2 acc[8];  // pairs of neighbours
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = make_float2(0.0f, 0.0f);
    for (int r0 = 0; r0 < a.n_ranks; r0 += kWide) {
      uint2 w[kWide];
      uint32_t s[kWide], top, low;
#pragma unroll
      for (int k = 0; k < kWide; ++k) {
        w[k] = make_uint2(0u, 0u), s[k] = s[0];  // (rank r0 is there)
        if (kFull || r0 + k < a.n_ranks) {
          w[k] = __ldcs(reinterpret_cast<const uint2*>(a.codes[r0 + k]) + i);
          s[k] = __ldcs(a.scales[r0 + k] + (i >> 1));
        }
      }
      top = low = s[0];
#pragma unroll
      for (int k = 1; k < kWide; ++k) top = max(top, s[k]), low = min(low, s[k]);
      if (r0 == 0 && top <= kPlainScale && top - low <= kNearScales) {
        __half2 sum[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = __half2half2(__ushort_as_half(0));
#pragma unroll
        for (int k = 0; k < kWide; ++k)
          if (kFull || k < a.n_ranks) {
            uint32_t h[8];
            decode8(w[k].x, reinterpret_cast<uint32_t(&)[4]>(h[0]));
            decode8(w[k].y, reinterpret_cast<uint32_t(&)[4]>(h[4]));
            const uint32_t sc = (s[k] - low + 15u) * 0x04000400u;  // 2^(s - low), twice
#pragma unroll
            for (int j = 0; j < 8; ++j)
              sum[j] = __hfma2(reinterpret_cast<const __half2&>(h[j]), reinterpret_cast<const __half2&>(sc), sum[j]);
          }
        const float sc = scale_value(low);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = mul2(__half22float2(sum[j]), make_float2(sc, sc));
      } else if (top <= kPlainScale) {
#pragma unroll
        for (int k = 0; k < kWide; ++k)
          if (kFull || r0 + k < a.n_ranks) {
            uint32_t h[8];
            decode8(w[k].x, reinterpret_cast<uint32_t(&)[4]>(h[0]));
            decode8(w[k].y, reinterpret_cast<uint32_t(&)[4]>(h[4]));
            const float sc = scale_value(s[k]);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = fma2(half2_float2(h[j]), make_float2(sc, sc), acc[j]);
          }
      } else {  // a scale near the top of the range, or NaN
#pragma unroll 1
        for (int k = 0; k < kWide && r0 + k < a.n_ranks; ++k) {
          const uint2 wk = __ldcs(reinterpret_cast<const uint2*>(a.codes[r0 + k]) + i);
          const float sc = scale_value(a.scales[r0 + k][i >> 1]);
          uint32_t h[8];
          decode8(wk.x, reinterpret_cast<uint32_t(&)[4]>(h[0]));
          decode8(wk.y, reinterpret_cast<uint32_t(&)[4]>(h[4]));
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 v = half2_float2(h[j]);
            acc[j] = make_float2(__fadd_rn(acc[j].x, __fmul_rn(v.x, sc)), __fadd_rn(acc[j].y, __fmul_rn(v.y, sc)));
          }
        }
      }
    }
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      if (i * 16 + 8 * g >= a.n) break;
      uint32_t x[4], m = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = Half<F>::pack(__fmul_rn(acc[4 * g + j].x, a.inv_n), __fmul_rn(acc[4 * g + j].y, a.inv_n));
        m = __vmaxu2(m, x[j] & 0x7FFF7FFFu);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // each square is exact, so one rounding as with a separate product
        const double d = (double)F::lo(x[j]), e = (double)F::hi(x[j]);
        sq = __fma_rn(d, d, sq);
        sq = __fma_rn(e, e, sq);
      }
      if (max(m & 0xFFFFu, m >> 16) >= Half<F>::kInf) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          nf += ((x[j] & 0x7FFFu) >= Half<F>::kInf ? 1u : 0u) + ((x[j] >> 16 & 0x7FFFu) >= Half<F>::kInf ? 1u : 0u);
      }
      st_stream(a.shard_out + i * 16 + 8 * g, make_uint4(x[0], x[1], x[2], x[3]));
    }
  }
  norm_epilogue<kThreads>(a.ns, sq, (unsigned long long)nf, a.accumulate);
}

template <class V>
cudaError_t quantize_rows(MxQuantArgs a, int sm_count, cudaStream_t s) {
  const bool flat = a.cols % kMxBlock == 0 && a.ld == a.cols && a.out.code_pitch == a.cols / 2 &&
                    a.out.scale_pitch == a.cols / kMxBlock;
  Pieces p;
  if (!pieces_of(a.rows, a.cols, flat, &p)) return cudaErrorInvalidValue;
  a.rows = p.rows, a.cols = p.cols;
  const int vec = aligned(a.src, flat ? 0 : a.ld * (int64_t)sizeof(typename V::raw)) ? 1 : 0;
  const int per_cta = V::kUnits * kRowThreads / 32;
  const int grid = cap_grid((p.units + per_cta - 1) / per_cta, kWaves * sm_count);
  const int more = (a.pieces.warps + kRowThreads / 32 - 1) / (kRowThreads / 32);
  if (a.stochastic) mx_rows_kernel<V, true><<<grid + more, kRowThreads, 0, s>>>(a, p.per_row, p.units, vec, grid);
  else mx_rows_kernel<V, false><<<grid + more, kRowThreads, 0, s>>>(a, p.per_row, p.units, vec, grid);
  return cudaGetLastError();
}

template <class V, Source kFrom>
cudaError_t quantize_tiles(const MxQuantArgs& a, cudaStream_t s) {
  constexpr int kCols = kTileWords * 4 / (int)sizeof(typename V::raw);
  const int64_t tx = (a.cols + kCols - 1) / kCols, ty = (a.rows + kTileRows - 1) / kTileRows;
  if (tx * ty > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const int vec = kFrom != kDense || aligned(a.src, a.ld * (int64_t)sizeof(typename V::raw)) ? 1 : 0;
  const unsigned grid = (unsigned)(tx * ty);
  const uint32_t x = (uint32_t)tx;
  if constexpr (kFrom == kDense) {  // an MX4 matrix is only transposed
    if (a.out.codes) {
      if (a.stochastic) mx_tile_kernel<V, kFrom, true, true><<<grid, 256, 0, s>>>(a, x, vec);
      else mx_tile_kernel<V, kFrom, true, false><<<grid, 256, 0, s>>>(a, x, vec);
      return cudaGetLastError();
    }
  }
  if (a.stochastic) mx_tile_kernel<V, kFrom, false, true><<<grid, 256, 0, s>>>(a, x, vec);
  else mx_tile_kernel<V, kFrom, false, false><<<grid, 256, 0, s>>>(a, x, vec);
  return cudaGetLastError();
}

template <class V>
cudaError_t quantize_backward(const MxBackwardArgs& a, cudaStream_t s) {
  constexpr int kCols = kTileWords * 4 / (int)sizeof(typename V::raw), kCols16 = 2 * kTileWords;
  auto up = [](int64_t n, int64_t d) { return (n + d - 1) / d; };
  const bool x8 = a.x.from.codes != nullptr;
  const int64_t dx = up(a.dy.cols, kCols), xx = up(a.x.cols, x8 ? kCols16 : kCols), wx = up(a.w.cols, kCols16);
  const int64_t nd = dx * up(a.dy.rows, kTileRows), nx = xx * up(a.x.rows, kTileRows), nw = wx * up(a.w.rows, kTileRows);
  if (nd + nx + nw > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  TileCounts n;
  n.dy = (uint32_t)nd, n.x = (uint32_t)(nd + nx);
  n.dy_x = (uint32_t)dx, n.x_x = (uint32_t)xx, n.w_x = (uint32_t)wx;
  n.dy_vec = aligned(a.dy.src, a.dy.ld * (int64_t)sizeof(typename V::raw)) ? 1 : 0;
  n.x_vec = !x8 && aligned(a.x.src, a.x.ld * (int64_t)sizeof(typename V::raw)) ? 1 : 0;
  const unsigned grid = (unsigned)(nd + nx + nw);
  if (a.dy.stochastic) {
    if (x8) mx_backward_kernel<V, true, true><<<grid, 256, 0, s>>>(a, n);
    else mx_backward_kernel<V, true, false><<<grid, 256, 0, s>>>(a, n);
  } else {
    if (x8) mx_backward_kernel<V, false, true><<<grid, 256, 0, s>>>(a, n);
    else mx_backward_kernel<V, false, false><<<grid, 256, 0, s>>>(a, n);
  }
  return cudaGetLastError();
}

template <class V>
cudaError_t quantize_from(const MxQuantArgs& a, int sm_count, cudaStream_t s) {
  return a.out_t.codes ? quantize_tiles<V, kDense>(a, s) : quantize_rows<V>(a, sm_count, s);
}

template <class T>
cudaError_t dequantize_to(MxDequantArgs a, int sm_count, cudaStream_t s) {
  const bool flat = a.in.cols % kMxBlock == 0 && a.ld == a.in.cols && a.in.code_pitch == a.in.cols / 2 &&
                    a.in.scale_pitch == a.in.cols / kMxBlock;
  Pieces p;
  if (!pieces_of(a.in.rows, a.in.cols, flat, &p)) return cudaErrorInvalidValue;
  a.in.rows = p.rows, a.in.cols = p.cols;
  const int vec = aligned(a.dst, flat ? 0 : a.ld * (int64_t)sizeof(typename T::raw)) ? 1 : 0;
  const int per_cta = 4 * kRowThreads / 32;
  mx_dequant_kernel<T><<<cap_grid((p.units + per_cta - 1) / per_cta, kWaves * sm_count), kRowThreads, 0, s>>>(
      a, p.per_row, p.units, vec);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx_quantize(const MxQuantArgs& a, int sm_count, cudaStream_t s) {
  if (a.from.codes) return quantize_tiles<Vec16<Bf16>, kFromMx4>(a, s);  // an MX4 matrix's transpose
  switch (a.type) {
    case kMxBf16: return quantize_from<Vec16<Bf16>>(a, sm_count, s);
    case kMxF16: return quantize_from<Vec16<F16>>(a, sm_count, s);
    case kMxF32: return quantize_from<Vec32>(a, sm_count, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_mx_backward(const MxBackwardArgs& a, int sm_count, cudaStream_t s) {
  if (a.dy.type == a.x.type || a.x.from.codes) {
    switch (a.dy.type) {
      case kMxBf16: return quantize_backward<Vec16<Bf16>>(a, s);
      case kMxF16: return quantize_backward<Vec16<F16>>(a, s);
      case kMxF32: return quantize_backward<Vec32>(a, s);
      default: return cudaErrorInvalidValue;
    }
  }
  cudaError_t e = launch_mx_quantize(a.dy, sm_count, s);
  if (e == cudaSuccess) e = launch_mx_quantize(a.x, sm_count, s);
  return e == cudaSuccess ? launch_mx_quantize(a.w, sm_count, s) : e;
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
  const int grid = cap_grid((mx_blocks(a.n) + kThreads - 1) / kThreads, kWaves * sm_count);
  if (a.fmt == kFmtF16) mx_gather_kernel<F16><<<grid, kThreads, 0, s>>>(a);
  else mx_gather_kernel<Bf16><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_mx_reduce(const MxReduceArgs& a, int sm_count, cudaStream_t s) {
  // as many CTAs as are there at a time (with twice as many 0.8 us more)
  const int grid = cap_grid((a.n / 16 + kThreads) / kThreads, std::min((a.n_ranks > 4 ? 4 : 5) * sm_count, kMaxGrid));
  auto launch = [&](auto f) {
    using F = decltype(f);
    if (a.n_ranks % 8 == 0) mx_reduce_kernel<F, 8, true><<<grid, kThreads, 0, s>>>(a);
    else if (a.n_ranks > 4) mx_reduce_kernel<F, 8, false><<<grid, kThreads, 0, s>>>(a);
    else if (a.n_ranks == 4) mx_reduce_kernel<F, 4, true><<<grid, kThreads, 0, s>>>(a);
    else mx_reduce_kernel<F, 4, false><<<grid, kThreads, 0, s>>>(a);
  };
  if (a.fmt == kFmtF16) launch(F16{});
  else launch(Bf16{});
  return cudaGetLastError();
}

}  // namespace zsm
