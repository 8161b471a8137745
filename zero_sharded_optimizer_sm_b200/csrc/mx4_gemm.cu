// The MX4 product: out[i][j] = sum over k of a[i][k] b[j][k] for two MX4
// matrices with blocks along k, on the block-scaled 4-bit tensor-core path
// (tcgen05.mma kind::mxf4, one scale per 32 elements of either operand).
//
// Names below: P is the operand whose 128 rows of a tile are the TMEM lanes,
// Q the one whose BN rows are the TMEM columns; a is P in the plain
// orientation and Q in the swapped one (few rows of a, so that the 128 lanes
// are filled by b's).  A k tile is 256 elements: one 128-byte swizzled row of
// codes and 8 scale bytes per matrix row, four instructions of 64 elements.
//
// Roles of a CTA's warps: 0 loads codes (TMA); 1 copies scales from shared
// memory into TMEM and issues the products; 4-7 read the accumulator and
// store; 8-11 load scales.  The scales lie in memory one row after another,
// and the tensor core wants, for each 128 rows and 128 k elements, a 512-byte
// piece with row r's four bytes at 16 (r % 32) + 4 (r / 32): a thread loads
// 16 bytes of a row into registers and stores four words at their places.
//
// Few tiles and a long k: a cluster of up to 8 CTAs splits k, each CTA sends
// the columns another one owns into that one's shared memory, and the owner
// adds the parts in rank order -- no workspace, and the same bits every run.
//
// Every wait on a barrier is bounded; one that runs out sets a flag that
// zero_mx4_check reports, after the CTA's own copies have landed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "device_math.cuh"
#include "mx4.cuh"
#include "tma_pipe.cuh"

namespace zsm {
namespace {

using namespace pipe;

constexpr int kLanes = 128;            // rows of P in a tile
constexpr int kTileK = 256;            // elements of k in a stage
constexpr int kTileKBytes = kTileK / 2;
constexpr int kThreadsMm = 384;
constexpr int kLoaderWarps = 4;

__device__ unsigned g_mx_error;        // a bounded wait that ran out (zero_mx4_check)

struct MmArgs {
  const uint8_t* p_scales;
  const uint8_t* q_scales;
  int64_t p_scale_pitch, q_scale_pitch;
  int p_rows, q_rows, k_blocks, k_tiles;
  int p_align, q_align;  // 16, 8, 4 or 1: alignment of that operand's scale rows
  int p_tiles, n_tiles, split;
  void* out;
  int64_t p_stride, q_stride;  // elements between rows of P / of Q in the result
  int type, vec;               // vec: 32-byte stores along q are aligned
  int pdl;
};

__host__ __device__ constexpr int q_chunks(int bn) { return (bn + 127) / 128; }
// Bytes of one stage: codes of both operands, scale pieces of both (two per
// 128 rows), rounded up to the 1024 bytes a swizzled tile starts on.
__host__ __device__ constexpr int stage_codes(int bn) { return (kLanes + bn) * kTileKBytes; }
__host__ __device__ constexpr int stage_scales(int bn) { return 1024 * (1 + q_chunks(bn)); }
__host__ __device__ constexpr int stage_bytes(int bn) { return stage_codes(bn) + stage_scales(bn); }
// TMEM columns: the accumulator, then two sets of scales used by turns.
__host__ __device__ constexpr int scale_cols(int bn) { return 8 * (1 + q_chunks(bn)); }
__host__ __device__ constexpr int acc_cols(int bn) { return bn < 32 ? 32 : bn; }
__host__ __device__ constexpr int tmem_cols(int bn) {
  int need = acc_cols(bn) + 2 * scale_cols(bn), n = 32;
  while (n < need) n *= 2;
  return n;
}

// ------------------------------------------------------------ instructions --

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y)
      : "memory");
}

__device__ __forceinline__ void tmem_alloc(uint32_t* slot, int cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, int cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory descriptors: a K-major tile of 128-byte swizzled rows (groups
// of 8 rows 1024 bytes apart), and 32 unswizzled rows of 16 bytes (groups of
// 8 rows 128 bytes apart).
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (8ull << 32) | (1ull << 46);
}
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

// Instruction descriptor: both operands 4-bit (format 1), scales a power of
// two (bit 23), N / 8 at bit 17, M / 128 at bit 27, and which two of the four
// scale bytes of a TMEM column the 64 elements use (0 or 2) at bits 4 and 29.
__host__ __device__ constexpr uint32_t inst_desc(int n, uint32_t id, int m = 128) {
  return (id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(m >> 7) << 27) |
         (id << 29);
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t pd, uint64_t qd, uint32_t idesc, uint32_t ps, uint32_t qs,
                                    bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(pd), "l"(qd), "r"(idesc), "r"(ps), "r"(qs), "r"(accumulate ? 1 : 0)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// The same for a pair of CTAs: both hold a part of either operand in their
// shared memory and half of the accumulator's rows in their TMEM; one thread
// of the even CTA issues for both.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* slot, int cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t addr, int cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t pd, uint64_t qd, uint32_t idesc, uint32_t ps, uint32_t qs,
                                         bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(pd), "l"(qd), "r"(idesc), "r"(ps), "r"(qs), "r"(accumulate ? 1 : 0)
      : "memory");
}
// One arrival on that barrier of each of the pair's CTAs.
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// A load into this CTA's shared memory whose bytes count on a barrier of the
// pair's even CTA.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
      "%4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ uint32_t address_in(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
// mbar_try_wait for a barrier on which the other CTA's threads arrive too.
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A wait of at most kWaitCycles: 0 done, 1 ran out, 2 another role stopped.
// Bounded by the SM's own clock: a read of the global timer takes about a
// microsecond, which would be added to every wait that has to poll.
constexpr long long kWaitCycles = 4000000000ll;  // two seconds at 2 GHz
template <bool kCluster>
__device__ __forceinline__ int wait_bounded(uint64_t* bar, unsigned parity, volatile int* abort_flag) {
  auto done = [&] { return kCluster ? try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
  if (done()) return 0;
  const long long t0 = clock64();
  while (!done()) {
    if (*abort_flag) return 2;
    if (clock64() - t0 > kWaitCycles) return 1;
  }
  return 0;
}

// N consecutive accumulator columns of this warp's 32 lanes.
template <int N>
__device__ __forceinline__ void tmem_read(uint32_t addr, float (&v)[N]) {
  static_assert(N == 8 || N == 16 || N == 32, "built widths");
  uint32_t r[N];
  if constexpr (N == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
  } else if constexpr (N == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
  }
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}

// 24 consecutive columns of this warp's 32 lanes, from registers.
__device__ __forceinline__ void tmem_write24(uint32_t addr, const uint4 (&v)[6]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(addr),
      "r"(v[0].x), "r"(v[0].y), "r"(v[0].z), "r"(v[0].w), "r"(v[1].x), "r"(v[1].y), "r"(v[1].z), "r"(v[1].w),
      "r"(v[2].x), "r"(v[2].y), "r"(v[2].z), "r"(v[2].w), "r"(v[3].x), "r"(v[3].y), "r"(v[3].z), "r"(v[3].w)
      : "memory");
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr + 16),
               "r"(v[4].x), "r"(v[4].y), "r"(v[4].z), "r"(v[4].w), "r"(v[5].x), "r"(v[5].y), "r"(v[5].z), "r"(v[5].w)
               : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_remote(uint32_t addr, uint32_t rank, float v) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tst.shared::cluster.f32 [a], %2;\n\t}" ::"r"(addr),
      "r"(rank), "f"(v)
      : "memory");
}

// ------------------------------------------------------------------ stores --

template <class F>
__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
  return dev::pack2(F::rn(a), F::rn(b));
}

__device__ __forceinline__ void store_one(const MmArgs& a, int64_t at, float v) {
  if (a.type == kMxBf16) static_cast<uint16_t*>(a.out)[at] = dev::Bf16::rn(v);
  else if (a.type == kMxF16) static_cast<uint16_t*>(a.out)[at] = dev::F16::rn(v);
  else static_cast<float*>(a.out)[at] = v;
}

__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// N consecutive results along q of row p, starting at column q.
template <int N>
__device__ __forceinline__ void store_run(const MmArgs& a, int64_t p, int64_t q, const float (&v)[N]) {
  if (p >= a.p_rows) return;
  const int64_t at = p * a.p_stride + q * a.q_stride;
  if (N >= 16 && a.vec && q + N <= a.q_rows) {
    if (a.type == kMxF32) {
#pragma unroll
      for (int i = 0; i + 8 <= N; i += 8) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[i + j]);
        store32(static_cast<float*>(a.out) + at + i, w);
      }
    } else {
#pragma unroll
      for (int i = 0; i + 16 <= N; i += 16) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          w[j] = a.type == kMxBf16 ? pack_pair<dev::Bf16>(v[i + 2 * j], v[i + 2 * j + 1])
                                   : pack_pair<dev::F16>(v[i + 2 * j], v[i + 2 * j + 1]);
        store32(static_cast<uint16_t*>(a.out) + at + i, w);
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (q + i < a.q_rows) store_one(a, at + i * a.q_stride, v[i]);
}

// ------------------------------------------------------------ scale loader --

// 16 scale bytes (two k tiles) of a row of which the first n exist (the
// others are 0).  Words: rows 4-byte aligned and n a multiple of 4; every
// load is predicated and none sits in a branch, whose end would wait for it.
template <bool kWords>
__device__ __forceinline__ uint4 load_scales(const uint8_t* p, int n, int align) {
  if constexpr (kWords) {
    const bool all = align == 16 && n >= 16;
    const bool lo = !all && align >= 8 && n >= 8, hi = !all && align >= 8 && n >= 16;
    const bool w0 = !all && !lo && n >= 4, w1 = !all && !lo && n >= 8;
    const bool w2 = !all && !hi && n >= 12, w3 = !all && !hi && n >= 16;
    uint4 r;
    asm volatile(
        "{\n\t.reg .pred q, l, h, a, b, c, d;\n\t"
        "setp.ne.b32 q, %5, 0;\n\tsetp.ne.b32 l, %6, 0;\n\tsetp.ne.b32 h, %7, 0;\n\t"
        "setp.ne.b32 a, %8, 0;\n\tsetp.ne.b32 b, %9, 0;\n\tsetp.ne.b32 c, %10, 0;\n\tsetp.ne.b32 d, %11, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@q ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t"
        "@l ld.global.v2.b32 {%0, %1}, [%4];\n\t"
        "@h ld.global.v2.b32 {%2, %3}, [%4 + 8];\n\t"
        "@a ld.global.b32 %0, [%4];\n\t"
        "@b ld.global.b32 %1, [%4 + 4];\n\t"
        "@c ld.global.b32 %2, [%4 + 8];\n\t"
        "@d ld.global.b32 %3, [%4 + 12];\n\t}"
        : "=&r"(r.x), "=&r"(r.y), "=&r"(r.z), "=&r"(r.w)
        : "l"(p), "r"((int)all), "r"((int)lo), "r"((int)hi), "r"((int)w0), "r"((int)w1), "r"((int)w2), "r"((int)w3)
        : "memory");
    return r;
  } else {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (n > j) w[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__device__ __forceinline__ void st_word(uint32_t addr, uint32_t w) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(w) : "memory");
}

// A loader thread's whole run: the scale bytes of its R rows for every k tile
// of every tile, in order.  The loads are kAhead times two k tiles ahead of
// the stores (their latency under a full load of code copies is several k
// tiles long).  rows(tile, ptr) gives the R rows' starts (null: no such row),
// put(w) stores one k tile's two words of each row when its stage is free,
// and says whether to go on.  One warp's instructions between two k tiles
// are what bounds this, so everything that depends on the tile alone is kept.
template <int R, int kAhead, bool kWords, class Rows, class Put>
__device__ __forceinline__ void stream_scales(int first, int step, int n_tiles, int k0, int k1, int k_blocks, int align,
                                              Rows rows, Put put) {
  if (k0 >= k1 || first >= n_tiles) return;
  uint4 ring[kAhead][R];
  const uint8_t* ptr[R];
  int next = first, next_kt = k0;  // what is fetched next
  if (k0 & 1) align = min(align, 8);
  rows(first, ptr);
  auto fetch_next = [&](uint4 (&r)[R]) {
    if (next >= n_tiles) return;
    const int n = k_blocks - 8 * next_kt;
#pragma unroll
    for (int j = 0; j < R; ++j)
      r[j] = load_scales<kWords>(ptr[j] + 8 * next_kt, ptr[j] ? n : 0, align);
    next_kt += 2;
    if (next_kt >= k1) {
      next_kt = k0;
      next += step;
      if (next < n_tiles) rows(next, ptr);
    }
  };
#pragma unroll
  for (int u = 0; u < kAhead; ++u) fetch_next(ring[u]);
  int tile = first, kt = k0;
  while (true) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      uint2 w[R];
      uint4 now[R];
#pragma unroll
      for (int j = 0; j < R; ++j) {
        now[j] = ring[u][j];
        w[j] = make_uint2(now[j].x, now[j].y);
      }
      fetch_next(ring[u]);
      if (!put(w)) return;
      if (kt + 1 < k1) {
#pragma unroll
        for (int j = 0; j < R; ++j) w[j] = make_uint2(now[j].z, now[j].w);
        if (!put(w)) return;
      }
      kt += 2;
      if (kt >= k1) {
        kt = k0;
        tile += step;
        if (tile >= n_tiles) return;
      }
    }
  }
}

// ------------------------------------------------------------------ kernel --

template <int BN, int STAGES>
struct Shared {
  uint64_t codes_full[STAGES], scales_full[STAGES], empty[STAGES];
  uint64_t acc_full, acc_empty, drained;
  uint32_t tmem;
  int abort;
};

template <int BN, int STAGES>
__global__ void __launch_bounds__(kThreadsMm, BN <= 64 ? 2 : 1)
    mx_matmul_kernel(const __grid_constant__ CUtensorMap p_map, const __grid_constant__ CUtensorMap q_map,
                     const __grid_constant__ MmArgs a) {
  extern __shared__ uint8_t raw_smem[];
  __shared__ Shared<BN, STAGES> sh;
  constexpr int kQ = q_chunks(BN);
  constexpr int kStage = stage_bytes(BN);
  uint8_t* smem = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = a.split > 1 ? cluster_rank() : 0;
  const int k0 = (int)((int64_t)a.k_tiles * rank / a.split), k1 = (int)((int64_t)a.k_tiles * (rank + 1) / a.split);
  const int first = blockIdx.x / a.split, step = gridDim.x / a.split;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&sh.codes_full[s], 1);
      mbar_init(&sh.scales_full[s], kLoaderWarps);
      mbar_init(&sh.empty[s], 1);
    }
    mbar_init(&sh.acc_full, 1);
    mbar_init(&sh.acc_empty, 4);
    mbar_init(&sh.drained, 1);
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc(&sh.tmem, tmem_cols(BN));
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sh.tmem;
  volatile int* abort_flag = &sh.abort;
  auto wait = [&](uint64_t* bar, unsigned parity) -> bool {
    const int r = wait_bounded<false>(bar, parity, abort_flag);
    if (r == 1) {
      *abort_flag = 1;
      atomicOr(&g_mx_error, 1u);
    }
    return r == 0;
  };
  if (a.pdl) dev::pdl_wait();

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int tile = first; tile < a.n_tiles && ok; tile += step) {
        const int p0 = (tile % a.p_tiles) * kLanes, q0 = (tile / a.p_tiles) * BN;
        for (int kt = k0; kt < k1; ++kt, ++it) {
          const int s = it % STAGES;
          if (it >= STAGES && !(ok = wait(&sh.empty[s], ((it / STAGES) - 1) & 1))) break;
          uint8_t* st = smem + s * kStage;
          mbar_expect_tx(&sh.codes_full[s], (kLanes + BN) * kTileKBytes);
          tma_load_2d(st, &p_map, kt * kTileKBytes, p0, &sh.codes_full[s]);
          tma_load_2d(st + kLanes * kTileKBytes, &q_map, kt * kTileKBytes, q0, &sh.codes_full[s]);
        }
      }
      if (!ok)  // the copies in flight land before the CTA may end
        for (int j = it > STAGES ? it - STAGES : 0; j < it; ++j)
          mbar_wait(&sh.codes_full[j % STAGES], (j / STAGES) & 1);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int it = 0, n = 0;
      bool ok = true, issued = false;
      for (int tile = first; tile < a.n_tiles && ok; tile += step, ++n) {
        if (n > 0 && !(ok = wait(&sh.acc_empty, (n - 1) & 1))) break;
        fence_after();
        for (int kt = k0; kt < k1; ++kt, ++it) {
          const int s = it % STAGES;
          if (!(ok = wait(&sh.codes_full[s], (it / STAGES) & 1))) break;
          if (!(ok = wait(&sh.scales_full[s], (it / STAGES) & 1))) break;
          fence_after();
          const uint32_t base = smem_u32(smem + s * kStage);
          const uint32_t scales = base + stage_codes(BN);
          const uint32_t ts = tmem + acc_cols(BN) + (it & 1) * scale_cols(BN);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            copy_scales(ts + 4 * c, scale_desc(scales + 512 * c));
#pragma unroll
            for (int q = 0; q < kQ; ++q)
              copy_scales(ts + 8 + 4 * (c * kQ + q), scale_desc(scales + 1024 + 512 * (c * kQ + q)));
          }
          const uint64_t pd = tile_desc(base), qd = tile_desc(base + kLanes * kTileKBytes);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma(tmem, pd + 2 * j, qd + 2 * j, inst_desc(BN, (j & 1) * 2), ts + 4 * (j >> 1), ts + 8 + 4 * kQ * (j >> 1),
                kt > k0 || j > 0);
          issued = true;
          mma_commit(&sh.empty[s]);
        }
        if (ok) mma_commit(&sh.acc_full);
      }
      if (!ok && issued) {  // products in flight end before TMEM is freed
        mma_commit(&sh.drained);
        mbar_wait(&sh.drained, 0);
      }
    }
  } else if (warp >= 8) {
    // thread t: row t of P and rows t (and t + 128) of Q
    const int t = threadIdx.x - 256;  // 0..127
    const uint32_t at = 16u * (t & 31) + 4u * (t >> 5);
    int st = 0, turn = 0;  // the stage and whether it has been used before
    unsigned parity = 1;
    auto rows = [&](int tile, const uint8_t* (&ptr)[1 + kQ]) {
      const int64_t p = (int64_t)(tile % a.p_tiles) * kLanes + t, q = (int64_t)(tile / a.p_tiles) * BN + t;
      ptr[0] = p < a.p_rows ? a.p_scales + p * a.p_scale_pitch : nullptr;
#pragma unroll
      for (int j = 0; j < kQ; ++j)
        ptr[1 + j] = q + 128 * j < a.q_rows && t + 128 * j < BN ? a.q_scales + (q + 128 * j) * a.q_scale_pitch : nullptr;
    };
    auto put = [&](const uint2 (&w)[1 + kQ]) {
      if (turn && !__all_sync(0xFFFFFFFFu, wait(&sh.empty[st], parity))) return false;
      const uint32_t dst = smem_u32(smem) + st * kStage + stage_codes(BN) + at;
#pragma unroll
      for (int j = 0; j < 1 + kQ; ++j) {
        const uint32_t to = dst + (j == 0 ? 0 : 1024 + 512 * (j - 1));
        st_word(to, w[j].x);
        st_word(to + (j == 0 ? 512 : 512 * kQ), w[j].y);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.scales_full[st]);
      if (++st == STAGES) {
        st = 0;
        turn = 1;
        parity ^= 1;
      }
      return true;
    };
    const int align = min(a.p_align, a.q_align);
    constexpr int kAhead = BN <= 64 ? 2 : 4;
    if (align >= 4 && a.k_blocks % 4 == 0)
      stream_scales<1 + kQ, kAhead, true>(first, step, a.n_tiles, k0, k1, a.k_blocks, align, rows, put);
    else
      stream_scales<1 + kQ, 1, false>(first, step, a.n_tiles, k0, k1, a.k_blocks, align, rows, put);
  } else if (warp >= 4 && a.split == 1) {
    const int w = warp - 4;
    int n = 0;
    for (int tile = first; tile < a.n_tiles; tile += step, ++n) {
      if (!__all_sync(0xFFFFFFFFu, wait(&sh.acc_full, n & 1))) break;
      fence_after();
      const int64_t p = (int64_t)(tile % a.p_tiles) * kLanes + 32 * w + lane, q0 = (int64_t)(tile / a.p_tiles) * BN;
      constexpr int kStep = BN < 32 ? 8 : 32;
      for (int c = 0; c < BN; c += kStep) {
        float v[kStep];
        tmem_read<kStep>(tmem + ((uint32_t)(32 * w) << 16) + c, v);
        store_run<kStep>(a, p, q0 + c, v);
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.acc_empty);
    }
  }

  if (a.split > 1) {
    // Column c of the tile belongs to rank c / own; its part from rank r goes
    // to that rank's [r][c % own][lane], in the stages' memory, which every
    // CTA of the cluster has finished with after the first barrier.
    const int own = (BN + a.split - 1) / a.split;
    const int w = warp - 4;
    bool ok = true;
    if (warp >= 4 && warp < 8) {
      ok = __all_sync(0xFFFFFFFFu, wait(&sh.acc_full, 0));
      fence_after();
    }
    __syncwarp();
    cluster_sync();
    if (warp >= 4 && warp < 8 && ok) {
      constexpr int kStep = BN < 32 ? 8 : 32;
      const uint32_t base = smem_u32(smem);
      for (int c = 0; c < BN; c += kStep) {
        float v[kStep];
        tmem_read<kStep>(tmem + ((uint32_t)(32 * w) << 16) + c, v);
#pragma unroll
        for (int i = 0; i < kStep; ++i) {
          const uint32_t to = (uint32_t)(c + i) / own, at = (uint32_t)(c + i) % own;
          store_remote(base + 4u * ((rank * own + at) * kLanes + 32 * w + lane), to, v[i]);
        }
      }
    }
    __syncwarp();
    cluster_sync();
    if (warp >= 4 && warp < 8) {
      const float* part = reinterpret_cast<const float*>(smem);
      const int64_t p = (int64_t)(first % a.p_tiles) * kLanes + 32 * w + lane, q0 = (int64_t)(first / a.p_tiles) * BN;
      for (int i = 0; i < own; ++i) {
        const int c = rank * own + i;
        if (c >= BN || p >= a.p_rows || q0 + c >= a.q_rows) continue;
        float v = part[i * kLanes + 32 * w + lane];
        for (int r = 1; r < a.split; ++r) v = __fadd_rn(v, part[(r * own + i) * kLanes + 32 * w + lane]);
        store_one(a, p * a.p_stride + (q0 + c) * a.q_stride, v);
      }
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 1) tmem_free(tmem, tmem_cols(BN));
}

// ------------------------------------------------------- kernel, CTA pairs --

// Tiles of 256 x 256 by pairs of CTAs (one cluster of two per pair of SMs,
// walking the tiles): each CTA loads 128 rows of P and 128 of Q, and the
// pair's instruction reads both halves of Q, so that a stage brings 32 KB
// into each SM where a CTA alone (128 x 256) would need 48.  Every CTA keeps
// the scales of its own rows of P and of all 256 rows of Q.
//
// The scales come in the tensor core's order, from a workspace that
// mx_scale_pieces_kernel filled: the 1024 bytes of 128 rows and one k tile
// lie together, one row of the tensor map s_map.  (Warps
// that gather them from the rows while the products run could not keep up:
// 1900 cycles a k tile, of which the products need 512.)
//
// From the stage four warps of each CTA carry them on to TMEM (a thread's 16
// bytes of a piece are its lane's four columns).  The tensor core's own copy
// instruction takes 58 cycles for each 512 bytes in turn with the products:
// 350 cycles a k tile beside their 512.
//
// Two accumulators of 256 columns share 96 of TMEM's 512 with each other
// (the rest holds four sets of scales): the epilogue empties the shared
// columns first and lets the next tile start, then the others while it runs.
constexpr int kPairN = 256;
constexpr int kPairStages = 6;
constexpr int kPairCodes = 2 * kLanes * kTileKBytes;     // per CTA
constexpr int kPieces = 1024;                            // scale bytes of 128 rows and one k tile
constexpr int kPairStage = kPairCodes + 3 * kPieces;     // per CTA
constexpr int kPairThreads = 384;
constexpr int kPairSets = 4;
constexpr int kPairScaleCols = 24;
constexpr int kPairScales = 512 - kPairSets * kPairScaleCols;  // first column of the scales
constexpr int kPairSecond = kPairScales - kPairN;              // first column of the second accumulator
constexpr int kPairShared = kPairN - kPairSecond;              // columns in both
static_assert(kPairShared % 16 == 0 && kPairShared > 0, "the epilogue's order");
static_assert(kPairSets <= kPairStages, "a set is written again after its stage's products");

struct PairShared {
  uint64_t full[kPairStages], pieces_full[kPairStages], scales_full[kPairStages], empty[kPairStages];
  uint64_t acc_full[2], acc_empty, drained;
  uint32_t tmem;
  int abort;
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    mx_matmul_pair_kernel(const __grid_constant__ CUtensorMap p_map, const __grid_constant__ CUtensorMap q_map,
                          const __grid_constant__ CUtensorMap s_map, const __grid_constant__ MmArgs a) {
  extern __shared__ uint8_t raw_smem[];
  __shared__ PairShared sh;
  uint8_t* smem = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.pieces_full[s], 1);
      mbar_init(&sh.scales_full[s], 8);
      mbar_init(&sh.empty[s], 1);
    }
    mbar_init(&sh.acc_full[0], 1);
    mbar_init(&sh.acc_full[1], 1);
    mbar_init(&sh.acc_empty, 8);
    mbar_init(&sh.drained, 1);
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc_pair(&sh.tmem, 512);
  fence_before();
  __syncthreads();
  cluster_sync();
  fence_after();
  const uint32_t tmem = sh.tmem;
  volatile int* abort_flag = &sh.abort;
  auto wait = [&](uint64_t* bar, unsigned parity) -> bool {
    const int r = wait_bounded<true>(bar, parity, abort_flag);
    if (r == 1) {
      *abort_flag = 1;
      atomicOr(&g_mx_error, 1u);
    }
    return r == 0;
  };
  if (a.pdl) dev::pdl_wait();

  if (warp == 0) {
    if (lane == 0) {
      int it = 0, s = 0;
      unsigned parity = 1;
      bool ok = true;
      const uint32_t full = address_in(&sh.full[0], 0), mine = address_in(&sh.pieces_full[0], rank);
      for (int tile = first; tile < a.n_tiles && ok; tile += step) {
        const int pb = (tile % a.p_tiles) * 2, qb = (tile / a.p_tiles) * 2;  // blocks of 128 rows
        const int py = (pb + rank) * a.k_tiles, qy = (2 * a.p_tiles + qb) * a.k_tiles;  // their rows in s_map
        for (int kt = 0; kt < a.k_tiles; ++kt) {
          if (it >= kPairStages && !(ok = wait(&sh.empty[s], parity))) break;
          fence_proxy_async_smem();  // the scale warps' reads of the stage, before it is written again
          uint8_t* st = smem + s * kPairStage;
          if (rank == 0) mbar_expect_tx(&sh.full[s], 2 * kPairCodes);
          mbar_expect_tx(&sh.pieces_full[s], 3 * kPieces);
          uint8_t* sc = st + kPairCodes;
          tma_load_2d_pair(sc, &s_map, 0, py + kt, mine + 8 * s);
          tma_load_2d_pair(sc + kPieces, &s_map, 0, qy + kt, mine + 8 * s);
          tma_load_2d_pair(sc + 2 * kPieces, &s_map, 0, qy + a.k_tiles + kt, mine + 8 * s);
          tma_load_2d_pair(st, &p_map, kt * kTileKBytes, (pb + rank) * kLanes, full + 8 * s);
          tma_load_2d_pair(st + kLanes * kTileKBytes, &q_map, kt * kTileKBytes, (qb + rank) * kLanes, full + 8 * s);
          ++it;
          if (++s == kPairStages) {
            s = 0;
            parity ^= 1;
          }
        }
      }
      // the last products' arrivals here, before this CTA may end
      if (it < kPairStages) s = 0, parity = 0;
      for (int j = min(it, kPairStages); j > 0 && ok; --j) {
        ok = wait(&sh.empty[s], parity);
        if (++s == kPairStages) {
          s = 0;
          parity ^= 1;
        }
      }
      if (!ok && it > 0) {  // the copies in flight land long before this has passed
        const unsigned long long t0 = now_ns();
        while (now_ns() - t0 < 20000000ull) {
        }
      }
    }
  } else if (warp == 1 && rank == 0) {
    if (lane == 0) {
      int n = 0, s = 0, set = 0;
      unsigned parity = 0;
      bool ok = true, issued = false;
      const uint32_t base = smem_u32(smem);
      for (int tile = first; tile < a.n_tiles && ok; tile += step, ++n) {
        if (n > 0 && !(ok = wait(&sh.acc_empty, (n - 1) & 1))) break;
        fence_after();
        const uint32_t acc = tmem + (n & 1 ? kPairSecond : 0);
        for (int kt = 0; kt < a.k_tiles; ++kt) {
          if (!(ok = wait(&sh.full[s], parity))) break;
          if (!(ok = wait(&sh.scales_full[s], parity))) break;
          fence_after();
          const uint32_t at = base + s * kPairStage;
          const uint64_t pd = tile_desc(at), qd = tile_desc(at + kLanes * kTileKBytes);
          const uint32_t ts = tmem + kPairScales + set * kPairScaleCols;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_pair(acc, pd + 2 * j, qd + 2 * j, inst_desc(kPairN, (j & 1) * 2, 256), ts + 4 * (j >> 1),
                     ts + 8 + 8 * (j >> 1), kt > 0 || j > 0);
          issued = true;
          mma_commit_pair(&sh.empty[s]);
          if (++set == kPairSets) set = 0;
          if (++s == kPairStages) {
            s = 0;
            parity ^= 1;
          }
        }
        if (ok) mma_commit_pair(&sh.acc_full[n & 1]);
      }
      if (!ok && issued) {  // products in flight end before TMEM is freed
        mma_commit_pair(&sh.drained);
        mbar_wait(&sh.drained, 0);
      }
    }
  } else if (warp >= 4 && warp < 8) {
    const int w = warp - 4;
    int n = 0;
    for (int tile = first; tile < a.n_tiles; tile += step, ++n) {
      if (!__all_sync(0xFFFFFFFFu, wait(&sh.acc_full[n & 1], (n >> 1) & 1))) break;
      fence_after();
      const int64_t p = (int64_t)(tile % a.p_tiles) * 2 * kLanes + rank * kLanes + 32 * w + lane;
      const int64_t q0 = (int64_t)(tile / a.p_tiles) * kPairN;
      const uint32_t acc = tmem + ((uint32_t)(32 * w) << 16) + (n & 1 ? kPairSecond : 0);
      const int turn = n & 1 ? 0 : kPairSecond;  // this accumulator's first column that the other one shares
      for (int c = 0; c < kPairN; c += 16) {
        const int col = (turn + c) & (kPairN - 1);
        float v[16];
        tmem_read<16>(acc + col, v);
        if (c + 16 == kPairShared) {
          fence_before();
          __syncwarp();
          if (lane == 0) arrive_at(address_in(&sh.acc_empty, 0));
        }
        store_run<16>(a, p, q0 + col, v);
      }
      fence_before();
    }
  } else if (warp >= 8) {
    const int w = warp - 8;
    const int tiles = first < a.n_tiles ? (a.n_tiles - 1 - first) / step + 1 : 0;
    const int64_t total = (int64_t)tiles * a.k_tiles;
    const uint32_t ready = address_in(&sh.scales_full[0], 0);
    const uint32_t ts = tmem + ((uint32_t)(32 * w) << 16) + kPairScales;
    int s = 0, set = 0, s_old = 0;  // s_old: the stage whose products used this set before
    unsigned parity = 0, parity_old = 0;
    for (int64_t it = 0; it < total; ++it) {
      bool ok = wait(&sh.pieces_full[s], parity);
      if (it >= kPairSets) {
        ok = ok && wait(&sh.empty[s_old], parity_old);
        if (++s_old == kPairStages) {
          s_old = 0;
          parity_old ^= 1;
        }
      }
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      fence_after();
      const uint8_t* sc = smem + s * kPairStage + kPairCodes + 16 * lane;
      // columns: P's two pieces, then Q's of rows 0-127 and 128-255 for each half of the k tile
      uint4 v[6];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        v[c] = *reinterpret_cast<const uint4*>(sc + 512 * c);
        v[2 + 2 * c] = *reinterpret_cast<const uint4*>(sc + kPieces + 512 * c);
        v[3 + 2 * c] = *reinterpret_cast<const uint4*>(sc + 2 * kPieces + 512 * c);
      }
      tmem_write24(ts + set * kPairScaleCols, v);
      fence_before();
      __syncwarp();
      if (lane == 0) arrive_at(ready + 8 * s);
      if (++set == kPairSets) set = 0;
      if (++s == kPairStages) {
        s = 0;
        parity ^= 1;
      }
    }
  }
  fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA ends while the other may still reach its memory
  fence_after();
  if (warp == 1) tmem_free_pair(tmem, 512);
}

// The scales of both operands in the pair kernel's order: 1024 bytes for each
// 128 rows and k tile, row r's byte for block b of the tile at
// 512 (b / 4) + 16 (r % 32) + 4 (r / 32 % 4) + b % 4; 0 past the matrix (the
// codes there are 0 too, but a product with a NaN scale would not be).  A
// warp takes 32 rows and one k tile, a lane a row.
struct PieceArgs {
  const uint8_t* scales[2];
  int64_t pitch[2];
  int rows[2], align[2];
  uint8_t* out[2];
  int warps0, warps;  // 32-row pieces of the first operand, of both
  int k_blocks, k_tiles;
};

__global__ void __launch_bounds__(256) mx_scale_pieces_kernel(const __grid_constant__ PieceArgs a) {
  dev::pdl_wait();
  dev::pdl_trigger();
  const int lane = threadIdx.x & 31;
  int w = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w >= a.warps) return;
  const int o = w >= a.warps0 ? 1 : 0;
  if (o) w -= a.warps0;
  const int kt = w % a.k_tiles, r32 = w / a.k_tiles;
  const int64_t row = 32ll * r32 + lane;
  const int n = row < a.rows[o] ? min(a.k_blocks - 8 * kt, 8) : 0;
  const uint8_t* p = a.scales[o] + (n > 0 ? row * a.pitch[o] + 8 * kt : 0);
  uint32_t v[2] = {0u, 0u};
  if (a.align[o] >= 8 && n == 8) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    v[0] = x.x, v[1] = x.y;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) v[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
  }
  uint8_t* out = a.out[o] + ((int64_t)(r32 >> 2) * a.k_tiles + kt) * kPieces + 16 * lane + 4 * (r32 & 3);
  *reinterpret_cast<uint32_t*>(out) = v[0];
  *reinterpret_cast<uint32_t*>(out + 512) = v[1];
}

// -------------------------------------------------------------------- host --

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// The codes as a matrix of bytes; a box is 128 bytes of `rows` rows, swizzled.
bool codes_map(CUtensorMap* map, const MxMatrix& m, int rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)(mx_blocks(m.cols) * 16), (cuuint64_t)m.rows};
  const cuuint64_t strides[1] = {(cuuint64_t)m.code_pitch};
  const cuuint32_t box[2] = {kTileKBytes, (cuuint32_t)rows}, one[2] = {1, 1};
  return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, m.codes, dims, strides, box, one,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The large dynamic shared memory, opted into once per device (`opted`: a bit for each).
template <class K>
cudaError_t opt_in(K kernel, int bytes, std::atomic<uint64_t>& opted) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (bit && (opted.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) opted.fetch_or(bit, std::memory_order_release);
  return e;
}

// A workspace of scale pieces as rows of 1024 bytes.
bool pieces_map(CUtensorMap* map, uint8_t* pieces, int64_t rows) {
  const cuuint64_t dims[2] = {kPieces / 4, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {kPieces};
  const cuuint32_t box[2] = {kPieces / 4, 1}, one[2] = {1, 1};
  return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, pieces, dims, strides, box, one,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, int STAGES>
cudaError_t launch(const MxMatrix& p, const MxMatrix& q, MmArgs a, int sm_count, cudaStream_t s) {
  CUtensorMap pm, qm;
  if (!codes_map(&pm, p, kLanes) || !codes_map(&qm, q, BN)) return cudaErrorInvalidValue;
  constexpr int kSmem = STAGES * stage_bytes(BN) + 1024;
  static_assert(kSmem <= 227 * 1024 - 1024, "stages fit shared memory");
  static_assert(STAGES * stage_bytes(BN) >= (BN + 8) * kLanes * 4 || BN > 128, "the split's parts fit the stages");
  auto kernel = mx_matmul_kernel<BN, STAGES>;
  static std::atomic<uint64_t> opted{0};
  const cudaError_t e = opt_in(kernel, kSmem, opted);
  if (e != cudaSuccess) return e;
  a.p_tiles = (a.p_rows + kLanes - 1) / kLanes;
  const int64_t tiles = (int64_t)a.p_tiles * ((a.q_rows + BN - 1) / BN);
  if (tiles > 0x0FFFFFFF) return cudaErrorInvalidValue;
  a.n_tiles = (int)tiles;
  // one cluster (a CTA when k is not split) per tile, or one CTA per SM walking the tiles
  const int grid = a.split > 1 ? a.n_tiles * a.split : std::min<int>(a.n_tiles, sm_count * (BN <= 64 ? 2 : 1));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreadsMm);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (a.split > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = (unsigned)a.split;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (a.pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, pm, qm, a);
}

// Row blocks of 128 that the pair kernel reads for `rows` rows (whole pairs).
int64_t pair_blocks(int64_t rows) { return 2 * ((rows + 255) / 256); }

cudaError_t launch_pair(const MxMatrix& p, const MxMatrix& q, MmArgs a, uint8_t* workspace, int sm_count, cudaStream_t s) {
  PieceArgs g = {};
  g.scales[0] = a.p_scales, g.scales[1] = a.q_scales;
  g.pitch[0] = a.p_scale_pitch, g.pitch[1] = a.q_scale_pitch;
  g.rows[0] = a.p_rows, g.rows[1] = a.q_rows;
  g.align[0] = a.p_align, g.align[1] = a.q_align;
  CUtensorMap pm, qm, sm;
  const int64_t row = (int64_t)a.k_tiles * kPieces, pb = pair_blocks(p.rows), qb = pair_blocks(q.rows);
  if ((pb + qb) * 4 * a.k_tiles > 0x7FFFFFFF - 8) return cudaErrorInvalidValue;
  if (!codes_map(&pm, p, kLanes) || !codes_map(&qm, q, kLanes) || !pieces_map(&sm, workspace, (pb + qb) * a.k_tiles))
    return cudaErrorInvalidValue;
  g.out[0] = workspace, g.out[1] = workspace + pb * row;
  g.k_blocks = a.k_blocks, g.k_tiles = a.k_tiles;
  g.warps0 = (int)(pb * 4 * a.k_tiles), g.warps = (int)((pb + qb) * 4 * a.k_tiles);
  cudaError_t e = launch_kernel(mx_scale_pieces_kernel, (g.warps + 7) / 8, 256, 0, s, a.pdl != 0, g);
  if (e != cudaSuccess) return e;
  a.pdl = 1;
  constexpr int kSmem = kPairStages * kPairStage + 1024;
  static_assert(kSmem <= 227 * 1024 - 1024, "stages fit shared memory");
  static std::atomic<uint64_t> opted{0};
  e = opt_in(mx_matmul_pair_kernel, kSmem, opted);
  if (e != cudaSuccess) return e;
  a.p_tiles = (a.p_rows + 2 * kLanes - 1) / (2 * kLanes);
  const int64_t tiles = (int64_t)a.p_tiles * ((a.q_rows + kPairN - 1) / kPairN);
  if (tiles > 0x0FFFFFFF) return cudaErrorInvalidValue;
  a.n_tiles = (int)tiles;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)std::min<int64_t>(tiles, sm_count / 2));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mx_matmul_pair_kernel, pm, qm, sm, a);
}

}  // namespace

// Whether the product runs on CTA pairs: enough 256 x 256 tiles for half of them.
bool by_pairs(int64_t m, int64_t n, int sm_count) { return ((m + 255) / 256) * ((n + 255) / 256) >= sm_count / 4; }

int64_t mx_matmul_workspace(int64_t m, int64_t n, int64_t k, int sm_count) {
  if (!by_pairs(m, n, sm_count)) return 0;
  return (pair_blocks(m) + pair_blocks(n)) * ((mx_blocks(k) + 7) / 8) * kPieces;
}

cudaError_t launch_mx_matmul(const MxMatmulArgs& m, int sm_count, cudaStream_t s) {
  if (!encode_fn()) return cudaErrorNotSupported;
  // Many tiles: CTA pairs, a's rows as lanes, whose results go out 32 bytes at
  // a time along a row -- or b's rows as lanes where the result's rows are not
  // 32-byte aligned, which makes a warp's 32 lanes neighbours in memory.  Few
  // tiles: b's rows as lanes, narrower tiles, k split over a cluster.
  const int64_t row_bytes = m.ld * (m.type == kMxF32 ? 4 : 2);
  const bool aligned = ((reinterpret_cast<uintptr_t>(m.out) | (uintptr_t)row_bytes) & 31u) == 0;
  const bool many = by_pairs(m.a.rows, m.b.rows, sm_count);
  const bool swap = !many || !aligned;
  const MxMatrix& p = swap ? m.b : m.a;
  const MxMatrix& q = swap ? m.a : m.b;
  MmArgs a = {};
  a.p_scales = p.scales, a.q_scales = q.scales;
  a.p_scale_pitch = p.scale_pitch, a.q_scale_pitch = q.scale_pitch;
  a.p_rows = (int)p.rows, a.q_rows = (int)q.rows;
  a.k_blocks = (int)mx_blocks(p.cols);
  a.k_tiles = (a.k_blocks + 7) / 8;
  auto align = [](const MxMatrix& x) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(x.scales) | (uintptr_t)x.scale_pitch;
    return bits & 3u ? 1 : bits & 7u ? 4 : bits & 15u ? 8 : 16;
  };
  a.p_align = align(p), a.q_align = align(q);
  a.out = m.out, a.type = m.type, a.pdl = m.pdl;
  a.p_stride = swap ? 1 : m.ld, a.q_stride = swap ? m.ld : 1;
  a.vec = !swap;
  a.split = 1;
  if (many) return launch_pair(p, q, a, static_cast<uint8_t*>(m.workspace), sm_count, s);
  const int64_t p_tiles = (p.rows + kLanes - 1) / kLanes;
  auto split_for = [&](int bn, int slots) {
    const int64_t tiles = p_tiles * ((q.rows + bn - 1) / bn);
    const int64_t n = std::min<int64_t>(std::min<int64_t>(8, a.k_tiles), slots / tiles);
    a.split = (int)std::max<int64_t>(1, n);
  };
  if (q.rows <= 16) {
    split_for(16, 2 * sm_count);
    return launch<16, 5>(p, q, a, sm_count, s);
  }
  if (p_tiles * ((q.rows + 31) / 32) <= sm_count) {
    split_for(32, 2 * sm_count);
    return launch<32, 4>(p, q, a, sm_count, s);
  }
  if (p_tiles * ((q.rows + 63) / 64) <= sm_count) {
    split_for(64, 2 * sm_count);
    return launch<64, 4>(p, q, a, sm_count, s);
  }
  split_for(128, sm_count);
  return launch<128, 5>(p, q, a, sm_count, s);
}

// The flag of a bounded wait that ran out (current device), cleared as it is read (waits for `s`).
cudaError_t mx_matmul_error(unsigned* flag, cudaStream_t s) {
  cudaError_t e = cudaMemcpyFromSymbolAsync(flag, g_mx_error, sizeof *flag, 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && *flag) {
    const unsigned zero = 0;
    e = cudaMemcpyToSymbolAsync(g_mx_error, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  return e;
}

}  // namespace zsm
