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

// ----------------------------------------------------------------- forward --

// Sum over a warp, and from the warps' binary32 sums on in binary64 over the
// block (kWarp: a warp has its own row): every thread gets the same bits.
template <bool kWarp>
__device__ __forceinline__ double group_sum(float mine, float* smem) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine = __fadd_rn(mine, __shfl_xor_sync(0xFFFFFFFFu, mine, o));
  if constexpr (kWarp) return (double)mine;
  const uint32_t warps = blockDim.x / 32;
  if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = mine;
  __syncthreads();
  double v = 0.0;
#pragma unroll 4
  for (uint32_t w = 0; w < warps; ++w) v = __dadd_rn(v, (double)smem[w]);
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

// All results of one vector of h.  Called by whole warps.
template <class T, class C>
__device__ __forceinline__ void finish(const RmsNormArgs& a, const NormRow<T>& row, const C& c, float rstd,
                                       const typename T::V& x) {
  float v[8], w[8];
  x.values(v);
  if (a.h) store_columns(row.h, c, x);
  if (a.h8.codes) store_columns8(row.h8, c, x, v);
  if (!a.y && !a.y8.codes) return;
  load_weights(a.weight, a.w_type, a.w_aligned, c, w);
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

// A block to a row, or (kWarp) a warp, kChunks vectors of eight elements a
// thread; the host picks the block's threads to fit the row.  Blocks that end
// make room for others whose loads go out at once, so that nothing has to be
// fetched ahead: 8192 x 4096 bf16 with a residual and all results, 338 MB, takes
// 52 us, the copy's rate (with 64-bit addresses for every access and single
// products 70, issue slots 73 % busy; now 62 %); without MX8 41, the copy's rate
// too.  Rows of odd length, 6000 x 2421 binary16 with all results, take 46 of 22:
// instructions (75 %).  One token of 4096 takes 2.7, its launch and two trips to
// memory.
constexpr int kWarpRows = 4;  // of a block
template <class T, bool kWhole, bool kWarp, int kChunks>
__global__ void __launch_bounds__(kWarp ? 32 * kWarpRows : 512) rms_norm_kernel(const __grid_constant__ RmsNormArgs a,
                                                                                const double inv_cols) {
  __shared__ float smem[32];
  const uint32_t number = kWarp ? blockIdx.x * kWarpRows + threadIdx.x / 32 : blockIdx.x;
  if (kWarp && number >= (uint32_t)a.rows) return;
  const NormRow<T> row(a, number);
  const uint32_t group = kWarp ? 32 : blockDim.x, t = kWarp ? threadIdx.x & 31 : threadIdx.x;
  using C = Columns<kWhole>;
  typename T::V x[kChunks];
  if constexpr (kChunks == 1) {
    const C c[1] = {C(0, t, (uint32_t)a.cols)};
    load_h<T>(a, row, c, x);
  } else {
#pragma unroll
    for (int k = 0; k < kChunks; k += 2) {
      const C c[2] = {C(8 * group * k, t, (uint32_t)a.cols), C(8 * group * (k + 1), t, (uint32_t)a.cols)};
      load_h<T>(a, row, c, reinterpret_cast<typename T::V(&)[2]>(x[k]));
    }
  }
  float2 ss = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    float v[8];
    x[k].values(v);
    ss = square_sum(v, ss);
  }
  const float rstd = rstd_of(group_sum<kWarp>(__fadd_rn(ss.x, ss.y), smem), inv_cols, (double)a.eps);
  if (a.rstd && t == 0) a.rstd[number] = rstd;
#pragma unroll
  for (int k = 0; k < kChunks; ++k) finish<T>(a, row, C(8 * group * k, t, (uint32_t)a.cols), rstd, x[k]);
}

// Rows too long for registers: read a second time (a thread reads its own
// elements before it writes results in their place).
constexpr int kLongThreads = 512;
template <class T, bool kWhole>
__global__ void __launch_bounds__(kLongThreads) rms_norm_long_kernel(const __grid_constant__ RmsNormArgs a,
                                                                     const double inv_cols) {
  __shared__ float smem[32];
  const NormRow<T> row(a, blockIdx.x);
  const uint32_t cols = (uint32_t)a.cols;
  using C = Columns<kWhole>;
  float2 ss = make_float2(0.0f, 0.0f);
  for (uint32_t first = 0; first < cols; first += 8 * kLongThreads) {
    typename T::V x[1];
    const C c[1] = {C(first, threadIdx.x, cols)};
    float v[8];
    load_h<T>(a, row, c, x);
    x[0].values(v);
    ss = square_sum(v, ss);
  }
  const float rstd = rstd_of(group_sum<false>(__fadd_rn(ss.x, ss.y), smem), inv_cols, (double)a.eps);
  if (a.rstd && threadIdx.x == 0) a.rstd[blockIdx.x] = rstd;
  for (uint32_t first = 0; first < cols; first += 8 * kLongThreads) {
    typename T::V x[1];
    const C c[1] = {C(first, threadIdx.x, cols)};
    load_h<T>(a, row, c, x);
    finish<T>(a, row, c[0], rstd, x[0]);
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

// Threads of a block and vectors of a thread for rows of so many columns.
struct Shape {
  uint32_t threads, chunks;
};
Shape shape_of(int64_t cols) {
  const uint32_t vectors = (uint32_t)((cols + 7) / 8);
  const uint32_t chunks = vectors <= kMaxThreads ? 1 : vectors <= 2 * kMaxThreads ? 2 : 4;
  return {std::max(32u, ((vectors + chunks - 1) / chunks + 31) / 32 * 32), chunks};
}

// Blocks to an SM, and blocks at most: as many as are there at a time (the
// kernels' registers allow 1024 threads).
uint32_t blocks_to_sm(const Shape& p) { return std::max(1u, std::min(1024 / p.threads / p.chunks, 16u)); }
int64_t parts_of(int64_t rows, int64_t cols) {
  // four rows a block where that leaves every SM one: a block's start and its
  // part of dw cost as much as some rows do (1237 x 771: one row a block 14 us)
  const int64_t few = std::max((rows + 3) / 4, std::min(rows, kSms));
  return std::max<int64_t>(1, std::min(few, kSms * blocks_to_sm(shape_of(cols))));
}

// The longest rows of which two stages fit; longer ones go through memory twice.
int64_t wide_from(int type, bool whole) { return (type == kMxF32 ? 4096 : 8192) * (whole ? 2 : 1); }

// Sum over the block in binary32; smem holds two rounds' values, so that one
// barrier a round will do.
__device__ __forceinline__ float block_sum(float v, float (*smem)[32], int round) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
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

// dx of that, rounded: times rstd, plus dh (a vector of the type) if there is one.
template <class T, class C>
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
  store_columns(row, c, x);
}

template <class C, class A>
__device__ __forceinline__ void store_part(float* out, const C& c, const A& acc) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c.in(j)) out[c.first + j] = j & 1 ? acc[j >> 1].y : acc[j >> 1].x;
}

// One row's stage of the ring: dy, dh, h of every thread's vectors, 16 bytes of
// each thread next to another's.
template <class T, bool kWhole, int kChunks, bool kMx8, bool kDh>
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
    __device__ __forceinline__ void next(const RmsNormBackwardArgs& a) {
      const uint32_t step = gridDim.x;
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
  static __device__ __forceinline__ void fetch(const RmsNormBackwardArgs& a, const Rows& row, bool there, uint8_t* to) {
    if (there) {
      const uint32_t vectors = blockDim.x * kChunks;
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const uint32_t v = blockDim.x * k + threadIdx.x;
        const Columns<kWhole> c(0, v, (uint32_t)a.cols);
        if (!c.any()) break;
        fetch16(to + 16 * v, vectors, row.dy, c, a.dy, a.dy_end);
        if constexpr (kDh) fetch16(to + dh_at(vectors) + 16 * v, vectors, row.dh, c, a.dh, a.dh_end);
        if constexpr (kMx8) copy_async8(to + h_at(vectors) + 8 * v, row.codes + c.first);
        else fetch16(to + h_at(vectors) + 16 * v, vectors, row.h, c, a.h, a.h_end);
      }
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

// One vector a thread: xh and g stay in registers over the sum; more: they are
// read and made a second time.
template <class T, bool kWhole, int kChunks, bool kMx8, bool kDh>
__global__ void __launch_bounds__(kMaxThreads, kChunks == 1 ? 2 : 1)
    rms_norm_backward_kernel(const __grid_constant__ RmsNormBackwardArgs a, const int stages) {
  using R = Ring<T, kWhole, kChunks, kMx8, kDh>;
  using C = Columns<kWhole>;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float smem[2][32];
  pdl_trigger();
  const uint32_t step = gridDim.x, rows = (uint32_t)a.rows;
  const uint32_t cols = (uint32_t)a.cols, group = blockDim.x, vectors = group * kChunks, size = R::bytes(vectors);
  uint32_t ahead = blockIdx.x;  // the row to ask for
  typename R::Rows from(a, ahead);
  for (int s = 0; s < stages - 1; ++s, ahead += step) {
    R::fetch(a, from, ahead < rows, ring + s * size);
    from.next(a);
  }
  float2 acc[kChunks][4];
  float w[8];
#pragma unroll
  for (int k = 0; k < kChunks; ++k)
#pragma unroll
    for (int p = 0; p < 4; ++p) acc[k][p] = make_float2(0.0f, 0.0f);
  if constexpr (kChunks == 1) load_weights(a.weight, a.w_type, a.w_aligned, C(0, threadIdx.x, cols), w);
  const float inv = __fdiv_rn(1.0f, (float)a.cols);
  // the row's statistics and scales, a row ahead
  const float* stats = a.rstd + blockIdx.x;
  const uint8_t* scales = a.h8.scales + blockIdx.x * a.h8.scale_pitch;
  float next_rstd = 0.0f;
  uint32_t scale[kChunks] = {}, next_scale[kChunks] = {};
  auto look = [&]() {
    next_rstd = *stats;
    if constexpr (kMx8) {
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const C c(8 * group * k, threadIdx.x, cols);
        if (c.any()) next_scale[k] = scales[c.first >> 5];
      }
    }
  };
  look();
  typename T::raw* to = row_of<T>(a.dx, blockIdx.x, a.ld_dx);
  uint32_t now = 0, later = (stages - 1) * size;  // the stages of this row and of the one to ask for
  int round = 0;
  for (uint32_t row = blockIdx.x; row < rows; row += step, ahead += step, ++round) {
    R::fetch(a, from, ahead < rows, ring + later);
    from.next(a);
    later = now;
    const uint8_t* stage = ring + now;
    now = now + size == stages * size ? 0 : now + size;
    const float rstd = next_rstd;
#pragma unroll
    for (int k = 0; k < kChunks; ++k) scale[k] = next_scale[k];
    stats += step;
    scales += step * a.h8.scale_pitch;
    if (row + step < rows) look();
    if (stages == 4) copy_async_wait<3>();
    else if (stages == 3) copy_async_wait<2>();
    else copy_async_wait<1>();
    float2 dot = make_float2(0.0f, 0.0f);
    float g[8], xh[8];
    auto vector = [&](int k, const C& c, bool sums) {
      const uint32_t v = group * k + threadIdx.x;
      typename T::V x;
      R::read(stage + 16 * v, vectors, R::offset(a.dy, row, a.ld_dy), c, x);
      x.values(g);
      if constexpr (kMx8) {
        take_columns8(xh, Fetched8{*reinterpret_cast<const uint2*>(stage + R::h_at(vectors) + 8 * v), scale[k]}, c, rstd);
      } else {
        R::read(stage + R::h_at(vectors) + 16 * v, vectors, R::offset(a.h, row, a.ld_h), c, x);
        x.values(xh);
        scale8(xh, rstd);
      }
      if constexpr (kChunks > 1) load_weights(a.weight, a.w_type, a.w_aligned, c, w);
      if (sums) add_vector(g, xh, w, acc[k], dot);
      else times8(g, w);
    };
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      const C c(8 * group * k, threadIdx.x, cols);
      if (c.any()) vector(k, c, true);
    }
    const float mean = __fmul_rn(block_sum(__fadd_rn(dot.x, dot.y), smem, round), inv);
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      const C c(8 * group * k, threadIdx.x, cols);
      if (kWhole && !c.any()) break;
      typename T::V dh;
      if (c.any()) {
        if constexpr (kChunks > 1) vector(k, c, false);
        dx_vector(g, xh, mean);
        if constexpr (kDh)
          R::read(stage + R::dh_at(vectors) + 16 * (group * k + threadIdx.x), vectors, R::offset(a.dh, row, a.ld_dh), c, dh);
      }
      store_dx<T>(to, c, rstd, kDh ? &dh : nullptr, g);  // (by whole warps)
    }
    to += step * a.ld_dx;
  }
  float* out = static_cast<float*>(a.workspace) + blockIdx.x * a.cols;
#pragma unroll
  for (int k = 0; k < kChunks; ++k) store_part(out, C(8 * group * k, threadIdx.x, cols), acc[k]);
}

// Longer rows: the rows' dot products first (into the workspace's head), then
// pieces of 2048 columns.
constexpr int kWideThreads = 256;
constexpr int kWideParts = 64;
int64_t wide_parts(int64_t rows) { return std::max<int64_t>(1, std::min<int64_t>(rows, kWideParts)); }
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
__global__ void __launch_bounds__(kWideThreads) rms_norm_dots_kernel(const __grid_constant__ RmsNormBackwardArgs a) {
  using C = Columns<kWhole>;
  __shared__ float smem[2][32];
  pdl_trigger();
  const int64_t row = blockIdx.x;
  const uint32_t cols = (uint32_t)a.cols;
  const float rstd = a.rstd[row];
  float2 dot = make_float2(0.0f, 0.0f);
  for (uint32_t first = 0; first < cols; first += 8 * kWideThreads) {
    const C c(first, threadIdx.x, cols);
    float xh[8], w[8], d[8];
    float2 unused[4] = {};
    load_dy_xh<T, kMx8>(a, row, c, rstd, d, xh);
    load_weights(a.weight, a.w_type, a.w_aligned, c, w);
    add_vector(d, xh, w, unused, dot);
  }
  const float all = block_sum(__fadd_rn(dot.x, dot.y), smem, 0);
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
    store_dx<T>(row_of<T>(a.dx, row, a.ld_dx), c, rstd, a.dh ? &dh : nullptr, g);
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

// A warp to a row up to 512 columns; above, a block of as many threads as the
// row has vectors, or half or a quarter of them.
template <class T, bool kWhole>
cudaError_t forward(const RmsNormArgs& a, cudaStream_t s) {
  const double inv = 1.0 / (double)a.cols;
  const unsigned rows = (unsigned)a.rows, warps = (rows + kWarpRows - 1) / kWarpRows;
  const uint32_t vectors = (uint32_t)((a.cols + 7) / 8);
  auto threads = [&](uint32_t chunks) { return ((vectors + chunks - 1) / chunks + 31) / 32 * 32; };
  if (vectors <= 32) rms_norm_kernel<T, kWhole, true, 1><<<warps, 32 * kWarpRows, 0, s>>>(a, inv);
  else if (vectors <= 64) rms_norm_kernel<T, kWhole, true, 2><<<warps, 32 * kWarpRows, 0, s>>>(a, inv);
  else if (vectors <= 256) rms_norm_kernel<T, kWhole, false, 1><<<rows, threads(1), 0, s>>>(a, inv);
  else if (vectors <= 1024) rms_norm_kernel<T, kWhole, false, 2><<<rows, threads(2), 0, s>>>(a, inv);
  else if (vectors <= 2048) rms_norm_kernel<T, kWhole, false, 4><<<rows, threads(4), 0, s>>>(a, inv);
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

template <class T, bool kMx8, bool kWhole, int kChunks, bool kDh>
cudaError_t backward(const RmsNormBackwardArgs& a, const Shape& p, cudaStream_t s) {
  // as deep as lets the blocks of parts_of fit an SM together
  constexpr int kRoom = 220 * 1024;
  const int stage = (int)Ring<T, kWhole, kChunks, kMx8, kDh>::bytes(p.threads * kChunks);
  const int stages = std::max(2, std::min(4, kRoom / (int)blocks_to_sm(p) / stage));
  if (stages * stage > kRoom) return cudaErrorInvalidValue;
  auto kernel = rms_norm_backward_kernel<T, kWhole, kChunks, kMx8, kDh>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRoom);
  if (e != cudaSuccess) return e;
  const int64_t parts = parts_of(a.rows, a.cols);
  kernel<<<(unsigned)parts, p.threads, stages * stage, s>>>(a, stages);
  const cudaError_t r = cudaGetLastError();
  return r == cudaSuccess ? add_dw(a, 0, parts, s) : r;
}

template <class T, bool kMx8, bool kWhole, int kChunks>
cudaError_t backward(const RmsNormBackwardArgs& a, const Shape& p, cudaStream_t s) {
  return a.dh ? backward<T, kMx8, kWhole, kChunks, true>(a, p, s) : backward<T, kMx8, kWhole, kChunks, false>(a, p, s);
}

template <class T, bool kMx8, bool kWhole>
cudaError_t backward_wide(const RmsNormBackwardArgs& a, cudaStream_t s) {
  const int64_t dots = dots_floats(a.rows), parts = wide_parts(a.rows);
  rms_norm_dots_kernel<T, kWhole, kMx8><<<(unsigned)a.rows, kWideThreads, 0, s>>>(a);
  const dim3 grid((unsigned)((a.cols + 8 * kWideThreads - 1) / (8 * kWideThreads)), (unsigned)parts);
  rms_norm_backward_wide_kernel<T, kWhole, kMx8><<<grid, kWideThreads, 0, s>>>(a, dots);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? add_dw(a, dots, parts, s) : e;
}

template <class T, bool kMx8, bool kWhole>
cudaError_t backward(const RmsNormBackwardArgs& a, cudaStream_t s) {
  const Shape p = shape_of(a.cols);
  if (a.cols > wide_from(a.type, kWhole)) return backward_wide<T, kMx8, kWhole>(a, s);
  if (p.chunks == 1) return backward<T, kMx8, kWhole, 1>(a, p, s);
  if (p.chunks == 2) return backward<T, kMx8, kWhole, 2>(a, p, s);
  if constexpr (kWhole && sizeof(typename T::raw) == 2) return backward<T, kMx8, kWhole, 4>(a, p, s);
  return cudaErrorInvalidValue;
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
  // whatever the type and alignment, on which it depends whether rows go through memory twice
  const int64_t once = parts_of(rows, cols) * cols, twice = dots_floats(rows) + wide_parts(rows) * cols;
  return 4 * (cols <= wide_from(kMxF32, false) ? once : cols <= wide_from(kMxBf16, true) ? std::max(once, twice) : twice);
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
