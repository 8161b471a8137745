// Embedding lookup and its gradient (embedding.cuh has the formulas).
//
// The lookup is a gather of rows, memory-bound.  The gradient is bound by the
// table that it writes whole: the batch's rows are sorted by their token, so
// that each row of the table is summed in binary32 in the batch's order,
// rounded once, and written once -- the same bits on every run, which atomic
// additions would not give.
#include <cuda_runtime.h>

#include "embedding.cuh"
#include "mx4_quant.cuh"

namespace zsm {
namespace {

using namespace mx;

__device__ __forceinline__ int64_t token_at(const void* tokens, int bytes, int64_t i) {
  return bytes == 8 ? __ldg(static_cast<const long long*>(tokens) + i) : (int64_t)__ldg(static_cast<const int*>(tokens) + i);
}

// ------------------------------------------------------------------ lookup --

constexpr int kRowThreads = 256;
constexpr int kUnits = 4;

// A source of rows, eight elements at a time: a dense table of one of the
// three types, or an MX4 one.
template <class V>
struct Dense {
  static __device__ __forceinline__ void row8(const EmbeddingArgs& a, int64_t row, int64_t col, int vec, float (&v)[8]) {
    V x;
    const typename V::raw* p = static_cast<const typename V::raw*>(a.table) + row * a.ld + col;
    const int64_t n = a.cols - col;
    if (n >= 8 && vec) x.load_if(p, true);
    else if (n > 0) x.load(p, n);
    else x.clear();
    x.values(v);
  }
};
struct Mx4Rows {
  static __device__ __forceinline__ void row8(const EmbeddingArgs& a, int64_t row, int64_t col, int, float (&v)[8]) {
    uint32_t w = 0u, s = 0u;
    if (col < a.cols) {
      w = __ldg(reinterpret_cast<const uint32_t*>(a.from.codes + row * a.from.code_pitch + (col >> 1)));
      s = __ldg(a.from.scales + row * a.from.scale_pitch + (col >> 5));
    }
    values8(w, s, v);
  }
};

// A warp takes 256 consecutive columns of one token at a time, kUnits of them
// side by side.
template <class S, class T>
__global__ void __launch_bounds__(kRowThreads) embedding_kernel(const __grid_constant__ EmbeddingArgs a, const FastDiv per_row,
                                                                const uint32_t units, const int vec) {
  using raw = typename T::raw;
  const uint32_t warps = gridDim.x * (kRowThreads / 32);
  const int lane = threadIdx.x & 31;
  for (uint32_t u0 = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); u0 < units; u0 += kUnits * warps) {
    uint32_t t[kUnits];
    int64_t col[kUnits], token[kUnits];
    float v[kUnits][8];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const uint32_t u = min(u0 + k * warps, units - 1);
      t[k] = div_by(u, per_row);
      col[k] = (int64_t)(u - t[k] * per_row.d) * 256 + lane * 8;
      token[k] = token_at(a.tokens, a.token_bytes, t[k]);
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      if ((uint64_t)token[k] < (uint64_t)a.vocab) {
        S::row8(a, token[k], col[k], vec, v[k]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = 0.0f;
      }
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      if ((uint64_t)token[k] < (uint64_t)a.vocab) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = __fmul_rn(v[k][j], a.scale);
      }
      store8<T>(static_cast<raw*>(a.out) + t[k] * a.ld_out + col[k], v[k], u0 + k * warps < units ? a.cols - col[k] : 0, vec);
    }
  }
}

// -------------------------------------------------------------------- sort --

// The batch's positions ordered by token, equal tokens in the batch's order
// (padding counts as token `vocab`): a radix sort of 8 bits at a time from the
// lowest, each pass three kernels -- the digits' counts of every kChunk
// positions, their running sums (all chunks of a digit one after another), and
// each position to its place.
constexpr int kSortThreads = 256;
constexpr int kPer = 8;                            // positions of a thread
constexpr int kChunk = kSortThreads * kPer;
constexpr int kDigits = 256;

struct Sort {
  const void* tokens;  // the first pass's keys; null: keys_in, pos_in
  int token_bytes;
  int64_t vocab;
  const uint32_t *keys_in, *pos_in;
  uint32_t *keys_out, *pos_out;
  uint32_t* counts;  // [digit][chunk]
  uint32_t n, chunks;
  int shift;
};

__device__ __forceinline__ uint32_t key_at(const Sort& s, uint32_t i) {
  if (!s.tokens) return s.keys_in[i];
  const int64_t t = token_at(s.tokens, s.token_bytes, i);
  return (uint64_t)t < (uint64_t)s.vocab ? (uint32_t)t : (uint32_t)s.vocab;
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const __grid_constant__ Sort s) {
  __shared__ uint32_t count[kDigits];
  count[threadIdx.x] = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const uint32_t i = blockIdx.x * kChunk + k * kSortThreads + threadIdx.x;
    if (i < s.n) atomicAdd(&count[key_at(s, i) >> s.shift & (kDigits - 1)], 1u);
  }
  __syncthreads();
  s.counts[threadIdx.x * s.chunks + blockIdx.x] = count[threadIdx.x];
}

// Sum over the lower lanes, and of all, of a warp.
__device__ __forceinline__ uint32_t warp_before(uint32_t v, uint32_t& total) {
  const int lane = threadIdx.x & 31;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  total = __shfl_sync(0xFFFFFFFFu, x, 31);
  return x - v;
}

__global__ void __launch_bounds__(1024) sort_scan_kernel(uint32_t* counts, const uint32_t n) {
  __shared__ uint32_t sums[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t each = (n + 1023) / 1024, lo = min(threadIdx.x * each, n), hi = min(lo + each, n);
  uint32_t mine = 0, total;
  for (uint32_t i = lo; i < hi; ++i) mine += counts[i];
  uint32_t before = warp_before(mine, total);
  if (lane == 0) sums[warp] = total;
  __syncthreads();
  uint32_t all;
  const uint32_t part = warp_before(sums[lane], all);
  before += __shfl_sync(0xFFFFFFFFu, part, warp);
  for (uint32_t i = lo; i < hi; ++i) {
    const uint32_t c = counts[i];
    counts[i] = before;
    before += c;
  }
}

// A warp ranks 32 consecutive positions at a time: those of equal digit find
// one another, count from the warp's running count of it, and the warps' counts
// are put behind one another.
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const __grid_constant__ Sort s) {
  constexpr int kWarps = kSortThreads / 32;
  __shared__ uint32_t count[kWarps][kDigits];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int d = lane; d < kDigits; d += 32) count[warp][d] = 0;
  __syncwarp();
  const uint32_t first = blockIdx.x * kChunk + warp * 32 * kPer + lane;
  uint32_t key[kPer], rank[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) key[k] = first + 32 * k < s.n ? key_at(s, first + 32 * k) : 0xFFFFFFFFu;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const bool there = first + 32 * k < s.n;
    const uint32_t digit = there ? key[k] >> s.shift & (kDigits - 1) : kDigits;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, digit);
    const uint32_t before = __popc(same & ((1u << lane) - 1u));
    rank[k] = there ? count[warp][digit] + before : 0u;
    __syncwarp();
    if (there && before == 0) count[warp][digit] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  uint32_t at = s.counts[threadIdx.x * s.chunks + blockIdx.x];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const uint32_t c = count[w][threadIdx.x];
    count[w][threadIdx.x] = at;
    at += c;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const uint32_t i = first + 32 * k;
    if (i >= s.n) break;
    const uint32_t to = count[warp][key[k] >> s.shift & (kDigits - 1)] + rank[k];
    s.keys_out[to] = key[k];
    s.pos_out[to] = s.tokens ? i : s.pos_in[i];
  }
}

// ---------------------------------------------------------------- gradient --

// starts[v]: the first place of token v or a later one, for v = 0 .. vocab.
__global__ void __launch_bounds__(256) embedding_starts_kernel(const uint32_t* keys, const uint32_t n, const uint32_t vocab,
                                                               uint32_t* starts) {
  const uint32_t v = blockIdx.x * 256 + threadIdx.x;
  if (v > vocab) return;
  uint32_t lo = 0, hi = n;
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2;
    if (keys[mid] < v) lo = mid + 1;
    else hi = mid;
  }
  starts[v] = lo;
}

// A warp sums 256 columns of one row of the table.
template <class V, class T>
__global__ void __launch_bounds__(kRowThreads) embedding_sum_kernel(const __grid_constant__ EmbeddingBackwardArgs a,
                                                                    const uint32_t* starts, const uint32_t* pos,
                                                                    const uint32_t per_row, const int vec) {
  using raw = typename T::raw;
  const int64_t warps = (int64_t)gridDim.x * (kRowThreads / 32), units = a.vocab * per_row;
  const int lane = threadIdx.x & 31;
  for (int64_t u = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); u < units; u += warps) {
    const int64_t row = u / per_row, col = (u - row * per_row) * 256 + lane * 8, n = a.cols - col;
    const uint32_t lo = starts[row], hi = starts[row + 1];
    if (a.accumulate && lo == hi) continue;
    float acc[8], v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
    for (uint32_t i = lo; i < hi; ++i) {
      V x;
      load8(x, static_cast<const typename V::raw*>(a.dy) + (int64_t)pos[i] * a.ld_dy + col, n, vec);
      x.values(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = __fadd_rn(acc[j], v[j]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = __fmul_rn(acc[j], a.scale);
    raw* out = static_cast<raw*>(a.dtable) + row * a.ld + col;
    if (a.accumulate) {
      typename T::V x;
      load8(x, out, n, vec);
      x.values(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = __fadd_rn(acc[j], v[j]);
    }
    store8<T>(out, acc, n, vec);
  }
}

// ------------------------------------------------------------------ launch --

int64_t element_bytes(int type) { return type == kMxF32 ? 4 : 2; }

template <class S, class T>
cudaError_t lookup(const EmbeddingArgs& a, int sm_count, cudaStream_t s) {
  const int64_t per = (a.cols + 255) / 256;
  if (per * a.n > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const uint32_t units = (uint32_t)(per * a.n);
  const int vec = (a.from.codes || aligned(a.table, a.ld * element_bytes(a.type))) &&
                  aligned(a.out, a.ld_out * element_bytes(a.out_type));
  const int per_cta = kUnits * kRowThreads / 32;
  embedding_kernel<S, T><<<cap_grid((units + per_cta - 1) / per_cta, kWaves * sm_count), kRowThreads, 0, s>>>(
      a, fast_div((uint32_t)per), units, vec);
  return cudaGetLastError();
}

template <class S>
cudaError_t lookup(const EmbeddingArgs& a, int sm_count, cudaStream_t s) {
  switch (a.out_type) {
    case kMxBf16: return lookup<S, TBf16>(a, sm_count, s);
    case kMxF16: return lookup<S, TF16>(a, sm_count, s);
    case kMxF32: return lookup<S, TF32>(a, sm_count, s);
    default: return cudaErrorInvalidValue;
  }
}

template <class V, class T>
cudaError_t sum_rows(const EmbeddingBackwardArgs& a, const uint32_t* starts, const uint32_t* pos, int sm_count,
                     cudaStream_t s) {
  const int64_t per = (a.cols + 255) / 256;
  const int vec = aligned(a.dy, a.ld_dy * element_bytes(a.type)) && aligned(a.dtable, a.ld * element_bytes(a.dtable_type));
  embedding_sum_kernel<V, T><<<cap_grid((per * a.vocab + 7) / 8, kWaves * sm_count), kRowThreads, 0, s>>>(
      a, starts, pos, (uint32_t)per, vec);
  return cudaGetLastError();
}

template <class V>
cudaError_t sum_rows(const EmbeddingBackwardArgs& a, const uint32_t* starts, const uint32_t* pos, int sm_count,
                     cudaStream_t s) {
  switch (a.dtable_type) {
    case kMxBf16: return sum_rows<V, TBf16>(a, starts, pos, sm_count, s);
    case kMxF16: return sum_rows<V, TF16>(a, starts, pos, sm_count, s);
    case kMxF32: return sum_rows<V, TF32>(a, starts, pos, sm_count, s);
    default: return cudaErrorInvalidValue;
  }
}

// The workspace: two sets of keys and positions, the counts, the starts.
struct Space {
  int64_t keys[2], pos[2], counts, starts, bytes;
};
Space space_of(int64_t n, int64_t vocab) {
  Space p;
  int64_t at = 0;
  auto part = [&](int64_t words) {
    const int64_t here = at;
    at += (4 * words + 15) / 16 * 16;
    return here;
  };
  for (int k = 0; k < 2; ++k) p.keys[k] = part(n), p.pos[k] = part(n);
  p.counts = part(kDigits * ((n + kChunk - 1) / kChunk));
  p.starts = part(vocab + 1);
  p.bytes = at;
  return p;
}

}  // namespace

int64_t embedding_backward_workspace(int64_t n, int64_t vocab, int64_t) { return space_of(n, vocab).bytes; }

cudaError_t launch_embedding(const EmbeddingArgs& a, int sm_count, cudaStream_t s) {
  if (a.from.codes) return lookup<Mx4Rows>(a, sm_count, s);
  switch (a.type) {
    case kMxBf16: return lookup<Dense<Vec16<Bf16>>>(a, sm_count, s);
    case kMxF16: return lookup<Dense<Vec16<F16>>>(a, sm_count, s);
    case kMxF32: return lookup<Dense<Vec32>>(a, sm_count, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_embedding_backward(const EmbeddingBackwardArgs& a, int sm_count, cudaStream_t s) {
  const Space p = space_of(a.n, a.vocab);
  uint8_t* base = static_cast<uint8_t*>(a.workspace);
  auto words = [&](int64_t at) { return reinterpret_cast<uint32_t*>(base + at); };
  Sort sort = {};
  sort.tokens = a.tokens, sort.token_bytes = a.token_bytes;
  sort.vocab = a.vocab;
  sort.n = (uint32_t)a.n;
  sort.chunks = (uint32_t)((a.n + kChunk - 1) / kChunk);
  sort.counts = words(p.counts);
  int out = 0;
  for (int shift = 0; shift == 0 || a.vocab >> shift; shift += 8, out ^= 1) {
    sort.shift = shift;
    sort.keys_out = words(p.keys[out]), sort.pos_out = words(p.pos[out]);
    sort_count_kernel<<<sort.chunks, kSortThreads, 0, s>>>(sort);
    sort_scan_kernel<<<1, 1024, 0, s>>>(sort.counts, kDigits * sort.chunks);
    sort_place_kernel<<<sort.chunks, kSortThreads, 0, s>>>(sort);
    sort.tokens = nullptr;
    sort.keys_in = sort.keys_out, sort.pos_in = sort.pos_out;
  }
  embedding_starts_kernel<<<(unsigned)((a.vocab + 256) / 256), 256, 0, s>>>(sort.keys_in, sort.n, (uint32_t)a.vocab,
                                                                             words(p.starts));
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  switch (a.type) {
    case kMxBf16: return sum_rows<Vec16<Bf16>>(a, words(p.starts), sort.pos_in, sm_count, s);
    case kMxF16: return sum_rows<Vec16<F16>>(a, words(p.starts), sort.pos_in, sm_count, s);
    case kMxF32: return sum_rows<Vec32>(a, words(p.starts), sort.pos_in, sm_count, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace zsm
