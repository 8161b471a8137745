// Embedding lookup and its gradient (embedding.cuh has the formulas).
//
// The lookup is a gather of rows, memory-bound.  The gradient is bound by the
// table that it writes whole: the batch's rows are sorted by their token, so
// that each row of the table is summed in binary32, rounded once, and written
// once.  A token's rows are added in the batch's order as far as one warp adds
// them, and the sums of several warps after that; who adds what follows from the
// sizes and the tokens: the same bits on every run, which atomic additions would
// not give.
#include <cuda_runtime.h>

#include "embedding.cuh"
#include "rows.cuh"

namespace zsm {
namespace {

using namespace mx;

__device__ __forceinline__ int64_t token_at(const void* tokens, int bytes, int64_t i) {
  return bytes == 8 ? __ldg(static_cast<const long long*>(tokens) + i) : (int64_t)__ldg(static_cast<const int*>(tokens) + i);
}

// ------------------------------------------------------------------ lookup --

constexpr int kRowThreads = 256;
constexpr int kPieces = 4;  // of 256 columns

// A source of rows: a dense table of one of the three types, or an MX4 one.
template <class T, bool kWhole>
struct Dense {
  const typename T::raw* row;
  Span span;
  Fetched<typename T::V, kWhole> f[kPieces];
  __device__ __forceinline__ Dense(const EmbeddingArgs& a, int64_t r)
      : row(row_of<T>(a.table, r, a.ld)), span(span_of<T>(a.table, a.vocab, a.cols, a.ld)) {}
  __device__ __forceinline__ void load(int k, const Columns<kWhole>& c) { fetch_columns(f[k], row, c, span); }
  __device__ __forceinline__ void values(int k, const Columns<kWhole>& c, float scale, float (&v)[8]) {
    typename T::V x;
    take_columns(x, f[k], row, c);
    x.values(v);
    scale8(v, scale);
  }
};
template <bool kWhole>
struct Mx4Rows {
  const uint8_t *codes, *scales;
  uint32_t w[kPieces], s[kPieces];
  __device__ __forceinline__ Mx4Rows(const EmbeddingArgs& a, int64_t r)
      : codes(a.from.codes + r * a.from.code_pitch), scales(a.from.scales + r * a.from.scale_pitch) {}
  __device__ __forceinline__ void load(int k, const Columns<kWhole>& c) {
    w[k] = s[k] = 0u;
    if (!c.any()) return;
    w[k] = __ldg(reinterpret_cast<const uint32_t*>(codes + (c.first >> 1)));
    s[k] = __ldg(scales + (c.first >> 5));
  }
  __device__ __forceinline__ void values(int k, const Columns<kWhole>&, float scale, float (&v)[8]) const {
    values8(w[k], s[k], v);
    scale8(v, scale);
  }
};

// A warp takes up to kPieces pieces of 256 columns of one token, side by side: the
// token is read once for them.  8192 tokens of an MX4 table of 32000 x 4096 take
// 13.4 us, 74 MB of which 67 are written (11.3 at the copy's rate; a warp to
// scattered pieces of four tokens 21); rows of odd length, 8000 of 2421 bf16, 24
// of 12, bound by instructions (69 % of the issue slots).
template <class S, class T, bool kWhole>
__global__ void __launch_bounds__(kRowThreads) embedding_kernel(const __grid_constant__ EmbeddingArgs a, const FastDiv per_row,
                                                                const uint32_t units) {
  const uint32_t u = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (u >= units) return;
  const uint32_t t = div_by(u, per_row), first = (u - t * per_row.d) * (256 * kPieces), cols = (uint32_t)a.cols;
  const int64_t token = token_at(a.tokens, a.token_bytes, t);
  const bool there = (uint64_t)token < (uint64_t)a.vocab;
  typename T::raw* out = row_of<T>(a.out, t, a.ld_out);
  S source(a, there ? token : 0);
  if (there) {
#pragma unroll
    for (int k = 0; k < kPieces; ++k)
      if (first + 256 * k < cols) source.load(k, Columns<kWhole>(first + 256 * k, threadIdx.x & 31, cols));
  }
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    if (first + 256 * k >= cols) break;
    typename T::V x;
    x.clear();
    if (there) {
      float v[8];
      source.values(k, Columns<kWhole>(first + 256 * k, threadIdx.x & 31, cols), a.scale, v);
      round_to(x, v);
    }
    store_columns(out, Columns<kWhole>(first + 256 * k, threadIdx.x & 31, cols), x);
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

// ------------------------------------------------------ sort of one cluster --

// Batches of up to kClusterMax positions are sorted by one cluster of CTAs in
// one launch: every CTA keeps its part of the (token, position) pairs in shared
// memory, and a pass writes them to their places in the cluster's CTAs.  16384
// positions of 16-bit tokens take some 8 us, latency throughout: three barriers
// and two trips through the cluster's memory a pass.  (A whole call, 64 columns,
// this way and with three launches a pass: 16385 positions 29 and 38 us, 32768 33
// and 40, of 300000 rows 40 and 55, 65536 56 and 57.)
constexpr int kClusterThreads = 1024;
constexpr int kClusterWarps = kClusterThreads / 32;
constexpr int kClusterCtas = 8;
constexpr int kClusterBits = 9;                       // of a pass: two for up to 2^18 - 1 rows
constexpr int kClusterDigits = 1 << kClusterBits;
constexpr int kClusterPer = 8192;                     // positions of a CTA
constexpr int64_t kClusterMax = (int64_t)kClusterCtas * kClusterPer;

struct ClusterSort {
  const void* tokens;
  int token_bytes;
  uint32_t n, vocab;
  int ctas;        // of a cluster
  uint32_t per;    // positions of a CTA: a multiple of 1024
  int bits, passes;
  uint32_t *keys, *pos;
};

struct ClusterShared {
  uint16_t count[kClusterWarps][kClusterDigits];  // a warp's pairs of a digit, then those of the warps before it
  uint32_t all[kClusterDigits];                   // the CTA's pairs of a digit (read by the cluster)
  uint32_t base[kClusterDigits];                  // the place of the CTA's first pair of a digit
  uint32_t sums[kClusterWarps];
};
constexpr int kClusterSmem = (int)sizeof(ClusterShared) + 2 * kClusterPer * 8;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
}
// The address of `p` (this CTA's shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(const void* p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ uint32_t ld_cluster(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster(uint32_t at, uint2 v) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(v.x), "r"(v.y) : "memory");
}

__device__ __forceinline__ uint32_t key_of(int64_t token, uint32_t vocab) {
  return (uint64_t)token < (uint64_t)vocab ? (uint32_t)token : vocab;
}

__global__ void __launch_bounds__(kClusterThreads, 1) sort_cluster_kernel(const __grid_constant__ ClusterSort s) {
  extern __shared__ __align__(16) uint8_t smem[];
  pdl_trigger();
  ClusterShared& sh = *reinterpret_cast<ClusterShared*>(smem);
  uint2* pairs = reinterpret_cast<uint2*>(smem + sizeof(ClusterShared));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = s.ctas > 1 ? cluster_rank() : 0;
  const uint32_t mine = rank * s.per;                              // my first position
  const uint32_t rounds = s.per / kClusterThreads;                 // pairs of a lane
  const uint32_t left = s.n > mine ? min(s.n - mine, s.per) : 0u;  // my pairs
  const uint32_t first = warp * 32 * rounds + lane;
  for (uint32_t k = 0; k < rounds; ++k) {
    const uint32_t i = first + 32 * k;
    if (i < left) pairs[i] = make_uint2(key_of(token_at(s.tokens, s.token_bytes, mine + i), s.vocab), mine + i);
  }
  for (int pass = 0; pass < s.passes; ++pass) {
    const uint2* from = pairs + (pass & 1) * s.per;
    uint2* to = pairs + (~pass & 1) * s.per;
    const int shift = pass * s.bits;
    const uint32_t digits = 1u << s.bits;
    for (uint32_t d = lane; d < digits; d += 32) sh.count[warp][d] = 0;
    __syncwarp();
    uint32_t ranks[kClusterPer / kClusterThreads];
#pragma unroll
    for (uint32_t k = 0; k < kClusterPer / kClusterThreads; ++k) {
      if (k >= rounds) break;
      const uint32_t i = first + 32 * k;
      const uint32_t digit = i < left ? from[i].x >> shift & (digits - 1) : digits;
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, digit);
      const uint32_t before = __popc(same & ((1u << lane) - 1u));
      ranks[k] = i < left ? sh.count[warp][digit] + before : 0u;
      __syncwarp();
      if (i < left && before == 0) sh.count[warp][digit] += (uint16_t)__popc(same);
      __syncwarp();
    }
    __syncthreads();
    if (threadIdx.x < digits) {  // a digit's warps one behind another
      uint32_t sum = 0;
#pragma unroll 8
      for (int w = 0; w < kClusterWarps; ++w) {
        const uint32_t c = sh.count[w][threadIdx.x];
        sh.count[w][threadIdx.x] = (uint16_t)sum;
        sum += c;
      }
      sh.all[threadIdx.x] = sum;
    }
    if (s.ctas > 1) cluster_sync();
    else __syncthreads();
    // a digit's CTAs one behind another, behind the lower digits of all
    uint32_t total = 0, lower = 0;
    if (threadIdx.x < digits) {
      for (int c = 0; c < s.ctas; ++c) {
        const uint32_t v = s.ctas > 1 ? ld_cluster(in_cta(&sh.all[threadIdx.x], c)) : sh.all[threadIdx.x];
        if (c < (int)rank) lower += v;
        total += v;
      }
    }
    uint32_t of_warp;
    const uint32_t before = warp_before(total, of_warp);
    if (lane == 0) sh.sums[warp] = of_warp;
    __syncthreads();
    uint32_t ignored;
    const uint32_t part = warp_before(sh.sums[lane], ignored);
    const uint32_t below = __shfl_sync(0xFFFFFFFFu, part, warp);  // (whole warps, however few the digits)
    if (threadIdx.x < digits) sh.base[threadIdx.x] = lower + before + below;
    __syncthreads();
    const bool last = pass + 1 == s.passes;
#pragma unroll
    for (uint32_t k = 0; k < kClusterPer / kClusterThreads; ++k) {
      if (k >= rounds) break;
      const uint32_t i = first + 32 * k;
      if (i >= left) break;
      const uint2 v = from[i];
      const uint32_t digit = v.x >> shift & (digits - 1);
      const uint32_t at = sh.base[digit] + sh.count[warp][digit] + ranks[k];
      if (last) s.keys[at] = v.x, s.pos[at] = v.y;
      else if (s.ctas > 1) st_cluster(in_cta(to + at % s.per, at / s.per), v);
      else to[at] = v;
    }
    if (s.ctas > 1) cluster_sync();  // (also: nobody leaves while its counts may be read)
    else __syncthreads();
  }
}

// ---------------------------------------------------------------- gradient --

// The sorted rows of dy are summed in segments of `seg` consecutive places, a
// warp 256 columns of one segment, so that a token that fills half the batch
// takes no longer than any other half.  A token's run that lies within a
// segment is finished there; of a run that crosses into the next ones, every
// segment leaves its part in the workspace -- slot 0 where the run came in from
// the segment before, slot 1 where it begins -- and the join adds the parts in
// order.
//
// Half the warps of every CTA first clear the rows of the table that no token of
// the batch has -- most of the gradient's bytes, as a rule.  They look for the
// tokens in the batch itself and clear while the cluster sorts; for a batch that
// is longer than a cluster sorts, they search the sorted tokens instead.  The
// other half waits for the sort and walks over the units (a slab of a segment),
// so that a short call is the sort's latency, the sums' and the join's one after
// another (8192 tokens, 32000 x 768: 24 us, 9.4 at the copy's rate).  One CTA an
// SM: of two kinds of CTAs, the clearing ones came to lie in pairs on half the SMs
// and took 47 us for 206 MB instead of 36.
constexpr int kSumThreads = 1024;
constexpr int kBitRows = 1 << 15;

struct Clear {
  uint8_t* table;
  int64_t row_bytes, pitch_bytes;
  bool by_search, end_to_end;  // rows of one piece
  FastDiv by_row;              // a row's elements of 2 bytes
  uint32_t rows;               // of the table that a CTA looks after at a time
  uint32_t each, late, each_late;  // a CTA's rows, and the last CTAs', how many those are
};

struct Segments {
  const uint32_t *keys, *pos;
  float* parts;  // [segment][slot][pitch], the columns rounded up to eights
  int64_t pitch;
  uint32_t n, seg, count, slabs;
};

// A warp's 256 columns.
template <bool kWhole>
using Slab = Columns<kWhole>;

template <class T, bool kWhole>
__device__ __forceinline__ void finish_row(const EmbeddingBackwardArgs& a, int64_t row, const Slab<kWhole>& c,
                                           const float (&sum)[8]) {
  using raw = typename T::raw;
  raw* out = static_cast<raw*>(a.dtable) + row * a.ld;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = sum[j];
  typename T::V x;
  if (a.accumulate) {
    float u[8];
    load_columns(x, out, c, span_of<T>(a.dtable, a.vocab, a.cols, a.ld));
    x.values(u);
    scale_plus8(v, a.scale, u);
  } else {
    scale8(v, a.scale);
  }
  round_to(x, v);
  store_columns(out, c, x);
}

// One warp clears `bytes` bytes at p, an element's multiple.
__device__ __forceinline__ void clear_row(uint8_t* p, int64_t bytes) {
  const int lane = threadIdx.x & 31;
  const int64_t head = min((int64_t)(-reinterpret_cast<uintptr_t>(p) & 15u), bytes);
  if (2 * lane < head) *reinterpret_cast<uint16_t*>(p + 2 * lane) = 0;
  p += head, bytes -= head;
  const int64_t n = bytes / 16;
  uint4* q = reinterpret_cast<uint4*>(p);
#pragma unroll 4
  for (int64_t i = lane; i < n; i += 32) __stcs(q + i, make_uint4(0u, 0u, 0u, 0u));
  if (2 * lane < (int)(bytes & 15)) *reinterpret_cast<uint16_t*>(p + 16 * n + 2 * lane) = 0;
}

// The CTA's share of the rows without a token, by its first kThreads threads.
template <int kThreads>
__device__ __forceinline__ void clear_rows(const EmbeddingBackwardArgs& a, const Segments& g, const Clear& z, uint32_t* bits) {
  auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); };
  const uint32_t soon = gridDim.x - z.late, mine = blockIdx.x < soon ? z.each : z.each_late;
  const int64_t begin = (int64_t)min(blockIdx.x, soon) * z.each + (blockIdx.x < soon ? 0 : (int64_t)(blockIdx.x - soon) * mine);
  const int64_t end = min(a.vocab, begin + mine);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (z.by_search) pdl_wait();
  for (int64_t lo = begin; lo < end; lo += z.rows) {
    const uint32_t rows = (uint32_t)min(end - lo, (int64_t)z.rows);
    if (z.by_search) {
      for (uint32_t r = threadIdx.x; r < (rows + 31) / 32 * 32; r += kThreads) {
        const uint32_t v = (uint32_t)lo + r;
        uint32_t x = 0, y = g.n;
        while (x < y) {
          const uint32_t mid = x + (y - x) / 2;
          if (g.keys[mid] < v) x = mid + 1;
          else y = mid;
        }
        const uint32_t word = __ballot_sync(0xFFFFFFFFu, x < g.n && g.keys[x] == v);
        if (lane == 0) bits[r >> 5] = word;
      }
    } else {
      for (uint32_t i = threadIdx.x; i < (rows + 31) / 32; i += kThreads) bits[i] = 0;
      sync();
      constexpr int kTokens = 8;  // loads of a thread that are out at a time
      for (uint32_t i = threadIdx.x; i < g.n; i += kTokens * kThreads) {
        int64_t token[kTokens];
#pragma unroll
        for (int k = 0; k < kTokens; ++k) token[k] = i + k * kThreads < g.n ? token_at(a.tokens, a.token_bytes, i + k * kThreads) : -1;
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
          const uint64_t at = (uint64_t)token[k] - (uint64_t)lo;
          // (a token that fills half the batch is marked once, not in turn by every thread)
          if (at < rows && !(reinterpret_cast<volatile uint32_t*>(bits)[at >> 5] >> (at & 31) & 1u))
            atomicOr(&bits[at >> 5], 1u << (at & 31));
        }
      }
    }
    sync();
    auto present = [&](uint32_t r) { return (bits[r >> 5] >> (r & 31) & 1u) != 0; };
    if (z.end_to_end) {
      // the rows as one piece of memory, its aligned words shared out among all
      // threads: a warp to a row of its own was 13 us slower over 206 MB, for
      // memory that is written in 16 places of a CTA at a time
      uint8_t* from = z.table + lo * z.row_bytes;
      const uint32_t bytes = (uint32_t)(rows * z.row_bytes), head = (uint32_t)(-reinterpret_cast<uintptr_t>(from) & 15u);
      auto row_at = [&](uint32_t byte) { return div_by(byte >> 1, z.by_row); };
      auto clear_some = [&](uint32_t at, uint32_t to) {
        for (; at < to; at += 2)
          if (!present(row_at(at))) *reinterpret_cast<uint16_t*>(from + at) = 0;
      };
      if (threadIdx.x == 0) clear_some(0, min(head, bytes));
      if (bytes > head) {
        const uint32_t words = (bytes - head) / 16;
#pragma unroll 4
        for (uint32_t i = threadIdx.x; i < words; i += kThreads) {
          const uint32_t at = head + 16 * i, r = row_at(at);
          // the row of the word's last element: rows of a word or more, the same or the next
          const uint32_t last = z.row_bytes < 16 ? row_at(at + 14) : r + (at + 14 >= (r + 1) * (uint32_t)z.row_bytes);
          if (!present(r) && !present(last) && last - r < 2) __stcs(reinterpret_cast<uint4*>(from + at), make_uint4(0u, 0u, 0u, 0u));
          else if (r != last) clear_some(at, at + 16);
        }
        if (threadIdx.x == 0) clear_some(head + 16 * words, bytes);
      }
    } else {
      uint8_t* row = z.table + (lo + warp) * z.pitch_bytes;
      for (uint32_t r = warp; r < rows; r += (kThreads / 32), row += (kThreads / 32) * z.pitch_bytes)
        if (!present(r)) clear_row(row, z.row_bytes);
    }
    sync();
  }
}

// A part's row of the workspace, eight columns of it a lane.
__device__ __forceinline__ float* part_at(const Segments& g, uint32_t segment, int slot) {
  return g.parts + (2ll * segment + slot) * g.pitch;
}
__device__ __forceinline__ void load_part(const float* p, float (&v)[8]) {
  const float4 a = __ldcg(reinterpret_cast<const float4*>(p)), b = __ldcg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store_part(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// A slab of a segment.
template <class D, class T, bool kWhole>
__device__ __forceinline__ void sum_unit(const EmbeddingBackwardArgs& a, const Segments& g, const FastDiv& by_slabs,
                                         const uint32_t u) {
  // rows whose loads are out at a time, as many as 64 registers hold
  constexpr int kAhead = sizeof(typename D::raw) == 2 ? (kWhole ? 8 : 3) : (kWhole ? 4 : 2);
  using V = typename D::V;
  const int lane = threadIdx.x & 31;
  const uint32_t segment = div_by(u, by_slabs), slab = u - segment * g.slabs;
  const uint32_t lo = segment * g.seg, hi = min(lo + g.seg, g.n);
  const Slab<kWhole> c(256u * slab, lane, (uint32_t)a.cols);
  const uint32_t vocab = (uint32_t)a.vocab;
  uint32_t current = g.keys[lo];
  if (current == vocab) return;  // padding from here on
  bool inside = lo > 0 && g.keys[lo - 1] == current;  // the run came in from the segment before
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
  auto flush = [&](bool goes_on) {
    if (!inside && !goes_on) {
      finish_row<T, kWhole>(a, current, c, acc);
    } else {
      if (c.any()) store_part(part_at(g, segment, inside ? 0 : 1) + c.first, acc);
    }
  };
  bool padding = false;
  const Span span = span_of<D>(a.dy, a.n, a.cols, a.ld_dy);
  for (uint32_t at = lo; at < hi && !padding; at += 32) {
    const uint32_t many = min(hi - at, 32u);
    const uint32_t key = (uint32_t)lane < many ? g.keys[at + lane] : vocab;
    const uint32_t pos = (uint32_t)lane < many ? g.pos[at + lane] : 0u;
    for (uint32_t i = 0; i < many && !padding; i += kAhead) {
      Fetched<V, kWhole> f[kAhead];
      const typename D::raw* row[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {  // (of a place that is not summed the batch's first row)
        row[k] = row_of<D>(a.dy, __shfl_sync(0xFFFFFFFFu, pos, (i + k) & 31), a.ld_dy);
        fetch_columns(f[k], row[k], c, span);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const uint32_t next = __shfl_sync(0xFFFFFFFFu, key, (i + k) & 31);
        if (padding || i + k >= many) continue;
        if (next != current) {
          flush(false);
          inside = false;
          current = next;
          padding = next == vocab;
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
        }
        V x;
        float v[8];
        take_columns(x, f[k], row[k], c);
        x.values(v);
        plus8(acc, v);
      }
    }
  }
  if (!padding) flush(hi < g.n && g.keys[hi] == current);
}

template <class D, class T, bool kWhole>
__global__ void __launch_bounds__(kSumThreads, 1)
    embedding_segments_kernel(const __grid_constant__ EmbeddingBackwardArgs a, const __grid_constant__ Segments g,
                              const __grid_constant__ Clear z, const FastDiv by_slabs) {
  __shared__ uint32_t bits[kBitRows / 32];
  constexpr int kClearing = kSumThreads / 2;
  pdl_trigger();
  if (z.table && threadIdx.x < kClearing) clear_rows<kClearing>(a, g, z, bits);
  pdl_wait();  // (every thread, whether it takes a unit or not: the join relies on the sort's being over too)
  // the warps that do not clear: all of an accumulating call
  const uint32_t skip = z.table ? kClearing / 32 : 0, warps = kSumThreads / 32 - skip, warp = threadIdx.x >> 5;
  if (warp < skip) return;
  for (uint32_t u = blockIdx.x * warps + warp - skip; u < g.count * g.slabs; u += gridDim.x * warps)
    sum_unit<D, T, kWhole>(a, g, by_slabs, u);
}

// A warp looks after the run that begins in its segment and crosses into the
// next; runs over more than kShort segments are added by the whole CTA, a share
// of the parts a warp.
constexpr uint32_t kShort = 16;
constexpr int kJoinThreads = 256;

template <bool kWhole>
__device__ __forceinline__ void add_parts(const Segments& g, uint32_t from, uint32_t to, const Slab<kWhole>& c,
                                          float (&acc)[8]) {
  if (!c.any()) return;
#pragma unroll 8
  for (uint32_t s = from; s < to; ++s) {
    float v[8];
    load_part(part_at(g, s, 0) + c.first, v);
    plus8(acc, v);
  }
}

template <class T, bool kWhole>
__global__ void __launch_bounds__(kJoinThreads) embedding_join_kernel(const __grid_constant__ EmbeddingBackwardArgs a,
                                                                      const __grid_constant__ Segments g) {
  constexpr int kWarps = kJoinThreads / 32;
  __shared__ uint32_t ends[kWarps];
  __shared__ float sums[kWarps][8][32];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t slab = blockIdx.x % g.slabs, first = blockIdx.x / g.slabs * kWarps, segment = first + warp;
  const Slab<kWhole> c(256u * slab, lane, (uint32_t)a.cols);
  // the segment after the last of my run; 0: no run of mine
  uint32_t end = 0, key = 0;
  if (segment + 1 < g.count) {
    const uint32_t lo = segment * g.seg, hi = lo + g.seg;
    key = g.keys[hi - 1];
    const uint32_t before = lo ? g.keys[lo - 1] : ~0u, first_key = g.keys[lo], next = g.keys[hi];
    if (next == key && key != (uint32_t)a.vocab && (first_key != key || before != key)) {
      // the last segment that begins with the run's token: 32 segments ahead
      // in steps of 1, then of 32, 1024, ... until one does not, and back
      uint32_t last = segment + 1, step = 1;
      for (bool back = false;;) {
        const uint32_t s = last + (lane + 1) * step;
        const uint32_t ahead = __popc(__ballot_sync(0xFFFFFFFFu, s < g.count && g.keys[s * g.seg] == key));
        last += ahead * step;
        if (ahead < 32) back = true;
        if (back && step == 1) break;
        step = back ? step / 32 : step * 32;
      }
      end = last + 1;
    }
  }
  const bool is_long = end && end - segment > kShort;
  if (lane == 0) ends[warp] = is_long ? end : 0;
  float acc[8];
  if (end) {
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
    if (c.any()) load_part(part_at(g, segment, 1) + c.first, acc);
    if (!is_long) {
      add_parts<kWhole>(g, segment + 1, end, c, acc);
      finish_row<T, kWhole>(a, key, c, acc);
    }
  }
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) {
    const uint32_t to = ends[w];
    if (!to) continue;
    const uint32_t from = first + w + 1, each = (to - from + kWarps - 1) / kWarps;
    float part[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) part[j] = 0.0f;
    add_parts<kWhole>(g, min(from + warp * each, to), min(from + (warp + 1) * each, to), c, part);
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[warp][j][lane] = part[j];
    __syncthreads();
    if (warp == w) {
#pragma unroll
      for (int k = 0; k < kWarps; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = __fadd_rn(acc[j], sums[k][j][lane]);
      finish_row<T, kWhole>(a, key, c, acc);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------ a few tokens --

// Up to kFew tokens need no sort: a warp takes a position and a slab, looks
// through all tokens for an earlier one of its kind (whose warp it leaves the sum
// to) and for the later ones, and adds their rows in the batch's order; a token of
// more than kAlone positions is left to kShares warps of the CTA, every kShares-th
// of them each, whose sums are added in order -- as many whether half the warps
// clear or not, so that adding to zeros gives the bits that writing does.  As long
// as the warps have two units each at most; us for a whole call, here and sorted,
// spread tokens and one token over and over:
//   301 tokens, 5003 x 768 binary16      4.9 and 10.4, 8.3 and 11.0
//   512 tokens of the same               5.4 and 11.9, 10.1 and 11.5
//   512 tokens, 50304 x 1024 bf16        18.2 and 21.4, 19.6 and 24.3
//   128 tokens, 2000 x 8192 bf16         9.8 and 13.4, 10.2 and 16.1
//   301 tokens of the same (five units)  20.1 and 14.6, 17.8 and 16.4
// What bounds it is latency: the launch, the tokens, two searches, the rows.  (A
// warp alone for up to 16 positions instead of 32: tokens of a text, 301, 7.4 us
// instead of 6.2.)
constexpr uint32_t kFew = 512;
constexpr uint32_t kAlone = 32;
constexpr int kShareBits = 4;
constexpr uint32_t kShares = 1u << kShareBits;
static_assert(kFew <= kAlone * kShares && kShares <= kSumThreads / 64, "a share fits a warp's list, and there are as many warps");
bool few_tokens(int64_t n, int64_t cols) { return n <= kFew && n * ((cols + 255) / 256) <= 2 * 148 * (kSumThreads / 64); }

struct FewShared {
  uint32_t keys[kFew];
  uint32_t bits[kBitRows / 32];
  uint16_t lists[kSumThreads / 32][kAlone];  // a warp's positions, all or a share
  uint32_t longs[kSumThreads / 32];      // the warps' units that all are to add up, plus 1
  float sums[kShares][8][32];
};

// Sums the rows at the positions of a warp's list, in order.
template <class D, bool kWhole>
__device__ __forceinline__ void add_listed(const EmbeddingBackwardArgs& a, const uint16_t* list, uint32_t many,
                                           const Slab<kWhole>& c, float (&acc)[8]) {
  constexpr int kAhead = sizeof(typename D::raw) == 2 ? (kWhole ? 8 : 3) : (kWhole ? 4 : 2);
  using V = typename D::V;
  const Span span = span_of<D>(a.dy, a.n, a.cols, a.ld_dy);
  for (uint32_t i = 0; i < many; i += kAhead) {
    Fetched<V, kWhole> f[kAhead];
    const typename D::raw* row[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {  // (past the list's end its last row again, not summed)
      row[k] = row_of<D>(a.dy, list[min(i + k, many - 1)], a.ld_dy);
      fetch_columns(f[k], row[k], c, span);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (i + k >= many) break;
      V x;
      float v[8];
      take_columns(x, f[k], row[k], c);
      x.values(v);
      plus8(acc, v);
    }
  }
}

template <class D, class T, bool kWhole>
__global__ void __launch_bounds__(kSumThreads, 1)
    embedding_few_kernel(const __grid_constant__ EmbeddingBackwardArgs a, const __grid_constant__ Segments g,
                         const __grid_constant__ Clear z, const FastDiv by_slabs) {
  __shared__ FewShared sh;
  constexpr int kClearing = kSumThreads / 2;
  if (z.table && threadIdx.x < kClearing) {
    clear_rows<kClearing>(a, g, z, sh.bits);
    return;
  }
  const uint32_t skip = z.table ? kClearing / 32 : 0, warps = kSumThreads / 32 - skip, warp = (threadIdx.x >> 5) - skip;
  const uint32_t lane = threadIdx.x & 31, vocab = (uint32_t)a.vocab, chunks = (g.n + 31) / 32;
  auto sync = [&] { asm volatile("bar.sync 2, %0;" ::"r"(32 * warps) : "memory"); };
  for (uint32_t i = 32 * warp + lane; i < 32 * chunks; i += 32 * warps) {
    const int64_t t = i < g.n ? token_at(a.tokens, a.token_bytes, i) : -1;
    sh.keys[i] = (uint64_t)t < (uint64_t)a.vocab ? (uint32_t)t : vocab;
  }
  sync();
  uint16_t* list = sh.lists[warp];
  float acc[8];
  // a list of the positions of `key` from `from` on whose number among them is
  // the share's (of 2^shift), and how many there are
  auto collect = [&](uint32_t key, uint32_t from, uint32_t share, uint32_t shift) {
    uint32_t count = 0;
#pragma unroll 4
    for (uint32_t k = from / 32; k < chunks; ++k) {
      const uint32_t at = 32 * k + lane;
      const bool mine = sh.keys[at] == key;
      const uint32_t all = __ballot_sync(0xFFFFFFFFu, mine), nth = count + __popc(all & ((1u << lane) - 1u));
      if (mine && nth - (nth >> shift << shift) == share && nth >> shift < kAlone) list[nth >> shift] = (uint16_t)at;
      count += __popc(all);
    }
    __syncwarp();
    return count;
  };
  // units go round the CTAs first: a token's slabs to as many of them
  const uint32_t units = g.n * g.slabs;
  for (uint32_t round = 0; round * warps * gridDim.x < units; ++round) {
    const uint32_t u = blockIdx.x + gridDim.x * (warp + warps * round);
    uint32_t is_long = 0;
    if (u < units) {
      const uint32_t i = div_by(u, by_slabs), key = sh.keys[i];
      bool first = key != vocab;
      for (uint32_t k = 0; first && k <= i / 32; ++k)
        first = !__any_sync(0xFFFFFFFFu, 32 * k + lane < i && sh.keys[32 * k + lane] == key);
      if (first) {
        const uint32_t many = collect(key, i, 0, 0);
        if (many <= kAlone) {
          const Slab<kWhole> c(256u * (u - i * g.slabs), lane, (uint32_t)a.cols);
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
          add_listed<D, kWhole>(a, list, many, c, acc);
          finish_row<T, kWhole>(a, key, c, acc);
        } else {
          is_long = u + 1;
        }
        __syncwarp();
      }
    }
    if (lane == 0) sh.longs[warp] = is_long;
    sync();
    for (uint32_t w = 0; w < warps; ++w) {
      const uint32_t of = sh.longs[w];
      if (!of) continue;
      const uint32_t i = div_by(of - 1, by_slabs), key = sh.keys[i];
      const Slab<kWhole> c(256u * (of - 1 - i * g.slabs), lane, (uint32_t)a.cols);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
      if (warp < kShares) {
        const uint32_t all = collect(key, i, warp, kShareBits);
        if (all > warp) add_listed<D, kWhole>(a, list, (all - warp + kShares - 1) / kShares, c, acc);
#pragma unroll
        for (int j = 0; j < 8; ++j) sh.sums[warp][j][lane] = acc[j];
      }
      sync();
      if (warp == w) {
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = sh.sums[0][j][lane];
        for (uint32_t k = 1; k < kShares; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] = __fadd_rn(acc[j], sh.sums[k][j][lane]);
        finish_row<T, kWhole>(a, key, c, acc);
      }
      sync();
    }
    sync();  // (the list of long units is read by all before it is written again)
  }
}

// ------------------------------------------------------------------ launch --

int64_t element_bytes(int type) { return type == kMxF32 ? 4 : 2; }

template <template <bool> class S, class T>
cudaError_t lookup(const EmbeddingArgs& a, cudaStream_t s) {
  const int64_t per = (a.cols + 256 * kPieces - 1) / (256 * kPieces), units = per * a.n;
  if (units > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const bool whole = a.cols % 8 == 0 && (a.from.codes || aligned(a.table, a.ld * element_bytes(a.type))) &&
                     aligned(a.out, a.ld_out * element_bytes(a.out_type));
  const unsigned grid = (unsigned)((units + kRowThreads / 32 - 1) / (kRowThreads / 32));
  if (whole) embedding_kernel<S<true>, T, true><<<grid, kRowThreads, 0, s>>>(a, fast_div((uint32_t)per), (uint32_t)units);
  else embedding_kernel<S<false>, T, false><<<grid, kRowThreads, 0, s>>>(a, fast_div((uint32_t)per), (uint32_t)units);
  return cudaGetLastError();
}

template <template <bool> class S>
cudaError_t lookup(const EmbeddingArgs& a, cudaStream_t s) {
  switch (a.out_type) {
    case kMxBf16: return lookup<S, TBf16>(a, s);
    case kMxF16: return lookup<S, TF16>(a, s);
    case kMxF32: return lookup<S, TF32>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

template <bool kWhole>
using DenseBf16 = Dense<TBf16, kWhole>;
template <bool kWhole>
using DenseF16 = Dense<TF16, kWhole>;
template <bool kWhole>
using DenseF32 = Dense<TF32, kWhole>;

template <class D, class T, bool kWhole>
cudaError_t sum_rows(const EmbeddingBackwardArgs& a, const Segments& g, const Clear& z, int sm_count, cudaStream_t s) {
  if (few_tokens(g.n, a.cols)) {
    const unsigned grid = (unsigned)(z.table ? sm_count : std::min<int64_t>(sm_count, (int64_t)g.n * g.slabs));
    embedding_few_kernel<D, T, kWhole><<<grid, kSumThreads, 0, s>>>(a, g, z, fast_div(g.slabs));
    return cudaGetLastError();
  }
  const int64_t units = (int64_t)g.count * g.slabs;
  if (units > 0x7FFFFFF0ll) return cudaErrorInvalidValue;
  const int grid = z.table ? sm_count : (int)std::min<int64_t>(sm_count, units);
  cudaError_t e = launch_kernel(embedding_segments_kernel<D, T, kWhole>, grid, kSumThreads, 0, s, true, a, g, z,
                                fast_div(g.slabs));
  if (e != cudaSuccess || g.count == 1) return e;
  return launch_kernel(embedding_join_kernel<T, kWhole>, (int)((g.count + kJoinThreads / 32 - 1) / (kJoinThreads / 32) * g.slabs),
                       kJoinThreads, 0, s, true, a, g);
}

template <class D>
cudaError_t sum_rows(const EmbeddingBackwardArgs& a, const Segments& g, const Clear& z, int sm_count, cudaStream_t s) {
  const bool vec = a.cols % 8 == 0 && aligned(a.dy, a.ld_dy * element_bytes(a.type)) &&
                   aligned(a.dtable, a.ld * element_bytes(a.dtable_type));
  switch (a.dtable_type) {
    case kMxBf16: return vec ? sum_rows<D, TBf16, true>(a, g, z, sm_count, s) : sum_rows<D, TBf16, false>(a, g, z, sm_count, s);
    case kMxF16: return vec ? sum_rows<D, TF16, true>(a, g, z, sm_count, s) : sum_rows<D, TF16, false>(a, g, z, sm_count, s);
    case kMxF32: return vec ? sum_rows<D, TF32, true>(a, g, z, sm_count, s) : sum_rows<D, TF32, false>(a, g, z, sm_count, s);
    default: return cudaErrorInvalidValue;
  }
}

// Places of a segment, for a warp to add one after another: as many as leave
// every warp that the SMs hold a segment's slab, from 8 rows, whose loads go out
// together, to 128, whose parts take a sixteenth of dy's elements' number.
constexpr int64_t kManyWarps = 148 * 32;
uint32_t segment_of(int64_t n, int64_t cols) {
  const int64_t slabs = (cols + 255) / 256;
  uint32_t seg = 8;
  while (seg < 128 && 2 * seg * kManyWarps <= n * slabs) seg *= 2;
  return seg;
}

// The workspace: keys and positions (two sets and the counts for the sort of a
// long batch), the segments' parts.
int64_t pitch_of(int64_t cols) { return (cols + 7) / 8 * 8; }
struct Space {
  int64_t keys[2], pos[2], counts, parts, bytes;
};
Space space_of(int64_t n, int64_t cols) {
  Space p = {};
  if (few_tokens(n, cols)) return p;
  int64_t at = 0;
  auto part = [&](int64_t words) {
    const int64_t here = at;
    at += (4 * words + 15) / 16 * 16;
    return here;
  };
  const bool is_long = n > kClusterMax;
  for (int k = 0; k < (is_long ? 2 : 1); ++k) p.keys[k] = part(n), p.pos[k] = part(n);
  if (is_long) p.counts = part(kDigits * ((n + kChunk - 1) / kChunk));
  const int64_t seg = segment_of(n, cols), count = (n + seg - 1) / seg;
  p.parts = part(count > 1 ? 2 * count * pitch_of(cols) : 0);
  p.bytes = at;
  return p;
}

int bits_of(int64_t v) {
  int b = 0;
  while (v >> b) ++b;
  return b;
}

int cluster_ctas(int64_t n) { return n <= kClusterThreads ? 1 : n <= 2 * kClusterThreads ? 2 : n <= 4 * kClusterThreads ? 4 : kClusterCtas; }

// What a CTA clears while the cluster sorts.  The segments' CTAs start while it
// does; the last ones find its SMs taken and begin when it is done, so that they
// get so much less to clear (8192 tokens, 32000 x 768 bf16: 25.0 us, shared equally
// 26.2; 16384 tokens, 50304 x 2048: 61.2 and 61.8).
int64_t late_bytes(int64_t n) { return (4 + n / 4096) * 38000; }

cudaError_t sort_in_cluster(ClusterSort c, cudaStream_t s) {
  const int64_t thousands = (c.n + kClusterThreads - 1) / kClusterThreads;
  c.ctas = cluster_ctas(c.n);
  c.per = (uint32_t)((thousands + c.ctas - 1) / c.ctas) * kClusterThreads;
  const int bits = bits_of(c.vocab);
  c.passes = std::max(1, (bits + kClusterBits - 1) / kClusterBits);
  c.bits = std::max(1, (bits + c.passes - 1) / c.passes);
  const int smem = (int)sizeof(ClusterShared) + 2 * (int)c.per * 8;
  const cudaError_t e = cudaFuncSetAttribute(sort_cluster_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kClusterSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)c.ctas);
  cfg.blockDim = dim3(kClusterThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)c.ctas, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sort_cluster_kernel, c);
}

}  // namespace

int64_t embedding_backward_workspace(int64_t n, int64_t cols) { return space_of(n, cols).bytes; }

cudaError_t launch_embedding(const EmbeddingArgs& a, int, cudaStream_t s) {
  if (a.from.codes) return lookup<Mx4Rows>(a, s);
  switch (a.type) {
    case kMxBf16: return lookup<DenseBf16>(a, s);
    case kMxF16: return lookup<DenseF16>(a, s);
    case kMxF32: return lookup<DenseF32>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_embedding_backward(const EmbeddingBackwardArgs& a, int sm_count, cudaStream_t s) {
  const Space p = space_of(a.n, a.cols);
  uint8_t* base = static_cast<uint8_t*>(a.workspace);
  auto words = [&](int64_t at) { return reinterpret_cast<uint32_t*>(base + at); };
  Segments g = {};
  g.n = (uint32_t)a.n;
  g.seg = segment_of(a.n, a.cols);
  g.count = (uint32_t)((a.n + g.seg - 1) / g.seg);
  g.slabs = (uint32_t)((a.cols + 255) / 256);
  g.parts = reinterpret_cast<float*>(base + p.parts);
  g.pitch = pitch_of(a.cols);
  ClusterSort c = {};
  c.tokens = a.tokens, c.token_bytes = a.token_bytes;
  c.n = (uint32_t)a.n, c.vocab = (uint32_t)a.vocab;
  Clear z = {};
  if (!a.accumulate) {
    z.table = static_cast<uint8_t*>(a.dtable);
    z.row_bytes = a.cols * element_bytes(a.dtable_type);
    z.pitch_bytes = a.ld * element_bytes(a.dtable_type);
    z.by_search = a.n > kClusterMax;
    z.end_to_end = z.pitch_bytes == z.row_bytes;
    z.by_row = fast_div((uint32_t)(z.row_bytes / 2));
    // so many that their bytes are counted in 31 bits
    z.rows = (uint32_t)std::max<int64_t>(1, std::min<int64_t>(kBitRows, 0x7FFFFFF0ll / z.row_bytes));
    z.end_to_end = z.end_to_end && z.row_bytes <= 0x7FFFFFF0ll;
    if (a.n <= kClusterMax && !few_tokens(a.n, a.cols)) z.late = std::min(cluster_ctas(a.n), sm_count - 1);
    z.each_late = z.late ? (uint32_t)std::max<int64_t>(0, a.vocab / sm_count - late_bytes(a.n) / z.row_bytes) : 0;
    z.each = (uint32_t)((a.vocab - (int64_t)z.late * z.each_late + sm_count - z.late - 1) / (sm_count - z.late));
  }
  cudaError_t e = cudaSuccess;
  if (few_tokens(a.n, a.cols)) {  // (no sort)
  } else if (a.n <= kClusterMax) {
    c.keys = words(p.keys[0]), c.pos = words(p.pos[0]);
    e = sort_in_cluster(c, s);
  } else {
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
    c.keys = sort.keys_out, c.pos = sort.pos_out;
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  g.keys = c.keys, g.pos = c.pos;
  switch (a.type) {
    case kMxBf16: return sum_rows<TBf16>(a, g, z, sm_count, s);
    case kMxF16: return sum_rows<TF16>(a, g, z, sm_count, s);
    case kMxF32: return sum_rows<TF32>(a, g, z, sm_count, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace zsm
