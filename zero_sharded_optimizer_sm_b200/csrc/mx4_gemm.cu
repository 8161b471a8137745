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
// Roles of a CTA's warps: 0 loads codes and scales (TMA); 1 issues the
// products; 2-5 and 6-9 bring scales into TMEM; 6-9 read the accumulator and
// store (a warp reaches the 32 lanes of TMEM that its number modulo 4 says).
//
// Scales: the tensor core wants the four scale bytes that row r has for 128 k
// elements in lane r % 32 of every 32 lanes, column r / 32.  They come two k
// tiles (16 bytes of a row) at a time through shared memory, either as they
// lie -- 16 bytes of each of 128 rows, where the rows are 16-byte aligned --
// or, where they are not, from a workspace in which a small kernel has put
// the words in that order (scale pieces).  Each of the four warps then writes
// the same words to its own lanes, from registers: the copy instruction that
// would take them from shared memory runs in turn with the products, 58
// cycles for 512 bytes, 350 cycles a k tile of 256 x 256 beside the products'
// 512 (8192 x 4096 x 4096 took a fifth longer so).  Reading the rows with
// ordinary loads instead of TMA cost 1900 cycles a k tile, most of it the
// ordering of such stores before the tensor core's reads of shared memory.
//
// Few tiles and a long k: a cluster of up to 8 CTAs splits k, each CTA sends
// the columns another one owns into that one's shared memory, and the owner
// adds the parts in rank order -- no workspace, and the same bits every run.
//
// Every wait on a barrier is bounded; one that runs out is counted for
// zero_mx4_check, and the CTA ends after its own copies have landed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "device_math.cuh"
#include "mx4.cuh"
#include "mx4_quant.cuh"
#include "tma_pipe.cuh"

namespace zsm {
namespace {

using namespace pipe;

constexpr int kLanes = 128;            // rows of P in a tile
constexpr int kTileK = 256;            // elements of k in a stage
constexpr int kTileKBytes = kTileK / 2;
constexpr int kThreadsMm = 320;
constexpr int kScaleWarps = 4;

__device__ unsigned g_mx_errors;       // bounded waits that ran out, ever (zero_mx4_check)

struct MmArgs {
  int p_rows, q_rows, k_tiles;
  int p_pieces, q_pieces;  // 1: that operand's scales come as pieces
  const uint8_t* p_scales; // set: P's scales are read from their rows by the scale warps (dense Q only)
  int64_t p_scale_pitch;
  int p_align, k_blocks;   //   alignment of those rows: 8 or 4
  int p_tiles, n_tiles, split;
  void* out;
  int64_t p_stride, q_stride;  // elements between rows of P / of Q in the result
  int type, vec;               // vec: 32-byte stores along q are aligned (CTA pairs only)
  const void* x;               // Q as a dense matrix (kernels with a vector type V)
  int64_t x_ld;
  int x_cols, x_vec;           // x_vec: its vectors are 16-byte aligned
  int pdl;                     // launched early: the grid before this one writes (some of) the operands,
  int p_early;                 //   but not P and its scales
};

// A stage: the codes of both operands for one k tile.  A group of scales: 16
// bytes for each row (up to 128 of P, then of Q) for two k tiles.
__host__ __device__ constexpr int stage_bytes(int bn) { return (kLanes + bn) * kTileKBytes; }
constexpr int kGroup = kMxPiece;  // of 128 rows
// TMEM columns: the accumulator, then four sets of scales used by turns.
constexpr int kSets = 4;
constexpr int kScaleCols = 16;
__host__ __device__ constexpr int acc_cols(int bn) { return bn < 32 ? 32 : bn; }
__host__ __device__ constexpr int tmem_cols(int bn) {
  int need = acc_cols(bn) + kSets * kScaleCols, n = 32;
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

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
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

// Shared-memory descriptor of a K-major tile of 128-byte swizzled rows
// (groups of 8 rows 1024 bytes apart).
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
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
// An arrival on a barrier of either CTA, in order at CTA scope: what it
// announces is in TMEM, ordered by the tcgen05 fences.  (Release at cluster
// scope cost 1900 cycles an arrival.)
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A wait of at most kWaitCycles: 0 done, 1 ran out, 2 another role stopped.
// Bounded by the SM's own clock: a read of the global timer takes about a
// microsecond, which would be added to every wait that has to poll.
constexpr long long kWaitCycles = 4000000000ll;  // two seconds at 2 GHz
__device__ __forceinline__ int wait_bounded(uint64_t* bar, unsigned parity, volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return 0;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort_flag) return 2;
    if (clock64() - t0 > kWaitCycles) return 1;
  }
  return 0;
}
// Whether all of a team's 128 threads say yes (named barriers 1 and 2).
__device__ __forceinline__ bool all_of_team(int team, bool yes) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, %2, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((int)yes), "r"(team + 1)
      : "memory");
  return r != 0;
}
// Long enough for every copy in flight to have landed (after a failed wait only).
__device__ __forceinline__ void linger() {
  const long long t0 = clock64();
  while (clock64() - t0 < 40000000ll) {
  }
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

// 16 or 8 consecutive columns of this warp's 32 lanes, from registers.
__device__ __forceinline__ void tmem_write16(uint32_t addr, const uint4 (&v)[4]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(addr),
      "r"(v[0].x), "r"(v[0].y), "r"(v[0].z), "r"(v[0].w), "r"(v[1].x), "r"(v[1].y), "r"(v[1].z), "r"(v[1].w),
      "r"(v[2].x), "r"(v[2].y), "r"(v[2].z), "r"(v[2].w), "r"(v[3].x), "r"(v[3].y), "r"(v[3].z), "r"(v[3].w)
      : "memory");
}
__device__ __forceinline__ void tmem_write8(uint32_t addr, const uint4 (&v)[2]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr),
               "r"(v[0].x), "r"(v[0].y), "r"(v[0].z), "r"(v[0].w), "r"(v[1].x), "r"(v[1].y), "r"(v[1].z), "r"(v[1].w)
               : "memory");
}
__device__ __forceinline__ void tmem_wait_write() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

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

// N results along q of row p, starting at column q, one by one.
template <int N>
__device__ __forceinline__ void store_run(const MmArgs& a, int64_t p, int64_t q, const float (&v)[N]) {
  if (p >= a.p_rows) return;
  const int64_t at = p * a.p_stride + q * a.q_stride;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (q + i < a.q_rows) store_one(a, at + i * a.q_stride, v[i]);
}
// 16 of them, consecutive in memory and 32-byte aligned when a.vec.
__device__ __forceinline__ void store_wide(const MmArgs& a, int64_t p, int64_t q, const float (&v)[16]) {
  if (!a.vec || q + 16 > a.q_rows) return store_run(a, p, q, v);
  if (p >= a.p_rows) return;
  const int64_t at = p * a.p_stride + q;
  uint32_t w[8];
  if (a.type == kMxF32) {
#pragma unroll
    for (int i = 0; i < 16; i += 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[i + j]);
      store32(static_cast<float*>(a.out) + at + i, w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      w[j] = a.type == kMxBf16 ? pack_pair<dev::Bf16>(v[2 * j], v[2 * j + 1]) : pack_pair<dev::F16>(v[2 * j], v[2 * j + 1]);
    store32(static_cast<uint16_t*>(a.out) + at, w);
  }
}

// ------------------------------------------------------------------ scales --

// The four TMEM columns (rows lane, lane + 32, lane + 64, lane + 96) of half c
// of k tile h of a group, for a lane: from rows as they lie, m[j] holds row
// lane + 32 j's 16 bytes; from pieces, m[2 h + c] the four rows' words.
struct ScaleGroup {
  uint4 m[4];
  __device__ __forceinline__ void load(const uint8_t* group, int lane, bool pieces, int rows) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      m[j] = pieces || lane + 32 * j < rows ? *reinterpret_cast<const uint4*>(group + 16 * lane + 512 * j)
                                            : make_uint4(0u, 0u, 0u, 0u);
    if (!pieces) transpose();
  }
  __device__ __forceinline__ void transpose() {  // words [row][k] to [k][row]
    const uint4 r0 = m[0], r1 = m[1], r2 = m[2], r3 = m[3];
    m[0] = make_uint4(r0.x, r1.x, r2.x, r3.x);
    m[1] = make_uint4(r0.y, r1.y, r2.y, r3.y);
    m[2] = make_uint4(r0.z, r1.z, r2.z, r3.z);
    m[3] = make_uint4(r0.w, r1.w, r2.w, r3.w);
  }
};

// 16 scale bytes of a row, of which the first n exist (the others are 0), the
// row 8-byte (align 8) or 4-byte aligned.  But for a row's last odd blocks
// every load is predicated and none sits in a branch, whose end would wait
// for it.
__device__ __forceinline__ uint4 load_row(const uint8_t* p, int n, int align) {
  const bool lo = align >= 8 && n >= 8, hi = align >= 8 && n >= 16;
  const bool w0 = !lo && n >= 4, w1 = !lo && n >= 8, w2 = !hi && n >= 12, w3 = !hi && n >= 16;
  uint4 r;
  asm volatile(
      "{\n\t.reg .pred l, h, a, b, c, d;\n\t"
      "setp.ne.b32 l, %5, 0;\n\tsetp.ne.b32 h, %6, 0;\n\t"
      "setp.ne.b32 a, %7, 0;\n\tsetp.ne.b32 b, %8, 0;\n\tsetp.ne.b32 c, %9, 0;\n\tsetp.ne.b32 d, %10, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@l ld.global.v2.b32 {%0, %1}, [%4];\n\t"
      "@h ld.global.v2.b32 {%2, %3}, [%4 + 8];\n\t"
      "@a ld.global.b32 %0, [%4];\n\t"
      "@b ld.global.b32 %1, [%4 + 4];\n\t"
      "@c ld.global.b32 %2, [%4 + 8];\n\t"
      "@d ld.global.b32 %3, [%4 + 12];\n\t}"
      : "=&r"(r.x), "=&r"(r.y), "=&r"(r.z), "=&r"(r.w)
      : "l"(p), "r"((int)lo), "r"((int)hi), "r"((int)w0), "r"((int)w1), "r"((int)w2), "r"((int)w3)
      : "memory");
  if (n > 0 && n < 16 && (n & 3)) {  // the row's last block does not end a word
    uint32_t w = 0;
    for (int i = n & ~3; i < n; ++i) w |= (uint32_t)p[i] << (8 * (i & 3));
    if (n < 4) r.x = w;
    else if (n < 8) r.y = w;
    else if (n < 12) r.z = w;
    else r.w = w;
  }
  return r;
}

// The same for the BN rows that start at row `part` (a multiple of BN) of a
// 128-row piece: row part + lane + 32 j's words lie where its row number says.
template <int BN>
__device__ __forceinline__ void load_part(ScaleGroup& g, const uint8_t* piece, int lane, int part) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < (BN + 31) / 32; ++j) {
      const int r = part + lane + 32 * j;
      if (lane + 32 * j < BN)
        w[j] = *reinterpret_cast<const uint32_t*>(piece + 512 * k + 16 * (r & 31) + 4 * (r >> 5));
    }
    g.m[k] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__global__ void __launch_bounds__(256) mx_scale_pieces_kernel(const __grid_constant__ MxPieceArgs a) {
  mx::write_pieces(a, blockIdx.x * 8 + (threadIdx.x >> 5));
}

// ------------------------------------------------------------------ kernel --

template <int BN, int STAGES, int GROUPS>
struct Shared {
  uint64_t codes_full[STAGES], scales_full[STAGES], empty[STAGES];
  uint64_t group_full[GROUPS], group_empty[GROUPS];
  uint64_t acc_full, acc_empty, drained;
  uint32_t tmem;
  int abort;
  static_assert(kSets <= STAGES, "a set is written again after its stage's products");
};

// V: void when Q is an MX4 matrix; else the vector type of the dense matrix
// that Q is (at most 16 rows), which the scale warps quantise on its way: a
// warp takes every fourth row's 256 elements of the k tile, 8 a lane.
// kDirect (dense Q only): P's scales are read from their rows by those warps
// too, for rows that are 4-byte aligned but not 16 -- with few tokens another
// launch for pieces would cost more than the narrower loads.
//
// Two tokens through 12288 x 4096 (27 MB of weights) take 11.2 us, 2.4 TB/s:
// the chain of one k tile's steps in the scale warps (load, quantise, meet,
// write to TMEM, product) is about 0.6 us, and a CTA has 8 k tiles of it;
// k tiles beyond the fourth wait for their sets.  Small matrices are launch
// and first-load latency: 2304 x 768 with four tokens takes 5.2 us.
template <int BN, int STAGES, int GROUPS, class V, bool kDirect>
__global__ void __launch_bounds__(kThreadsMm, BN <= 64 && !std::is_same<V, mx::Vec32>::value ? 2 : 1)
    mx_matmul_kernel(const __grid_constant__ CUtensorMap p_map, const __grid_constant__ CUtensorMap q_map,
                     const __grid_constant__ CUtensorMap ps_map, const __grid_constant__ CUtensorMap qs_map,
                     const __grid_constant__ MmArgs a) {
  extern __shared__ uint8_t raw_smem[];
  __shared__ Shared<BN, STAGES, GROUPS> sh;
  constexpr bool kDense = !std::is_void<V>::value;
  __shared__ uint32_t x_scales[kDense ? 2 : 1][2][2 * kMxFewRows];  // a team's, of its k tiles by turns: a row's 8 bytes
  constexpr int kStage = stage_bytes(BN);
  uint8_t* smem = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
  uint8_t* group_smem = smem + STAGES * kStage;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = a.split > 1 ? cluster_rank() : 0;
  // this CTA's k tiles: whole groups
  const int groups = (a.k_tiles + 1) / 2;
  const int g0 = (int)((int64_t)groups * rank / a.split), g1 = (int)((int64_t)groups * (rank + 1) / a.split);
  const int k0 = 2 * g0, k1 = min(2 * g1, a.k_tiles);
  const int first = blockIdx.x / a.split, step = gridDim.x / a.split;
  constexpr bool by_group = !kDirect;  // scales through shared memory
  static_assert(kDense || !kDirect, "Q's scales come in groups");

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&sh.codes_full[s], 1);
      mbar_init(&sh.scales_full[s], kScaleWarps);
      mbar_init(&sh.empty[s], 1);
    }
    for (int g = 0; g < GROUPS; ++g) {
      mbar_init(&sh.group_full[g], 1);
      mbar_init(&sh.group_empty[g], kScaleWarps);
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
    const int r = wait_bounded(bar, parity, abort_flag);
    if (r == 1) {
      *abort_flag = 1;
      atomicAdd(&g_mx_errors, 1u);
    }
    return r == 0;
  };

  if (warp == 0) {
    if (lane == 0) {
      // P's part of a stage or group and Q's: the first ones of P go out
      // before the wait for the grid that writes Q.
      for (const CUtensorMap* map : {&p_map, &q_map, &ps_map, &qs_map}) prefetch_map(map);
      auto load_codes = [&](bool p, int tile, int kt, int s) {
        uint8_t* st = smem + s * kStage;
        if (p) tma_load_2d(st, &p_map, kt * kTileKBytes, (tile % a.p_tiles) * kLanes, &sh.codes_full[s]);
        else tma_load_2d(st + kLanes * kTileKBytes, &q_map, kt * kTileKBytes, (tile / a.p_tiles) * BN, &sh.codes_full[s]);
      };
      auto load_group = [&](bool p, int tile, int g, int s) {
        uint8_t* to = group_smem + s * 2 * kGroup + (p ? 0 : kGroup);
        const CUtensorMap* map = p ? &ps_map : &qs_map;
        const int row = p ? (tile % a.p_tiles) * kLanes : (tile / a.p_tiles) * BN;
        if (p ? a.p_pieces : a.q_pieces)  // Q's 128-row pieces: BN divides 128, see q_part
          tma_load_2d(to, map, 0, 2 * ((row / kLanes) * groups + g), &sh.group_full[s]);
        else tma_load_2d(to, map, 16 * g, row, &sh.group_full[s]);
      };
      const int q_bytes = kDense ? 0 : a.q_pieces ? kGroup : 16 * BN;
      constexpr int kCodes = kDense ? kLanes * kTileKBytes : stage_bytes(BN);
      const int early = a.pdl && a.p_early && first < a.n_tiles ? min(k1 - k0, STAGES) : 0;
      const int early_groups = by_group ? min((early + 1) / 2, GROUPS) : 0;
      for (int j = 0; j < early; ++j) {
        if (j % 2 == 0 && j / 2 < early_groups) {
          mbar_expect_tx(&sh.group_full[j / 2], kGroup + q_bytes);
          load_group(true, first, g0 + j / 2, j / 2);
        }
        mbar_expect_tx(&sh.codes_full[j], kCodes);
        load_codes(true, first, k0 + j, j);
      }
      if (a.pdl) dev::pdl_wait();
      int it = 0, s = 0, gt = 0, gs = 0;
      unsigned parity = 1, gparity = 1;
      bool ok = true;
      for (int tile = first; tile < a.n_tiles && ok; tile += step) {
        for (int kt = k0; kt < k1; ++kt) {
          if (by_group && ((kt - k0) & 1) == 0) {
            if (gt >= GROUPS && !(ok = wait(&sh.group_empty[gs], gparity))) break;
            fence_proxy_async_smem();  // the scale warps' reads of the group, before it is written again
            if (gt >= early_groups) {
              mbar_expect_tx(&sh.group_full[gs], kGroup + q_bytes);
              load_group(true, tile, kt / 2, gs);
            }
            if (!kDense) load_group(false, tile, kt / 2, gs);
            ++gt;
            if (++gs == GROUPS) {
              gs = 0;
              gparity ^= 1;
            }
          }
          if (it >= STAGES && !(ok = wait(&sh.empty[s], parity))) break;
          if (it >= early) {
            mbar_expect_tx(&sh.codes_full[s], kCodes);
            load_codes(true, tile, kt, s);
          }
          if (!kDense) load_codes(false, tile, kt, s);
          ++it;
          if (++s == STAGES) {
            s = 0;
            parity ^= 1;
          }
        }
      }
      if (!ok) linger();  // the copies in flight land before the CTA may end
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int it = 0, n = 0, s = 0;
      unsigned parity = 0;
      bool ok = true, issued = false;
      const uint32_t base = smem_u32(smem);
      for (int tile = first; tile < a.n_tiles && ok; tile += step, ++n) {
        if (n > 0 && !(ok = wait(&sh.acc_empty, (n - 1) & 1))) break;
        fence_after();
        for (int kt = k0; kt < k1; ++kt, ++it) {
          if (!(ok = wait(&sh.codes_full[s], parity))) break;
          if (!(ok = wait(&sh.scales_full[s], parity))) break;
          fence_after();
          const uint32_t at = base + s * kStage;
          const uint32_t ts = tmem + acc_cols(BN) + (it % kSets) * kScaleCols;
          const uint64_t pd = tile_desc(at), qd = tile_desc(at + kLanes * kTileKBytes);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma(tmem, pd + 2 * j, qd + 2 * j, inst_desc(BN, (j & 1) * 2), ts + 4 * (j >> 1), ts + 8 + 4 * (j >> 1),
                kt > k0 || j > 0);
          issued = true;
          mma_commit(&sh.empty[s]);
          if (++s == STAGES) {
            s = 0;
            parity ^= 1;
          }
        }
        if (ok) mma_commit(&sh.acc_full);
      }
      if (!ok && issued) {  // products in flight end before TMEM is freed
        mma_commit(&sh.drained);
        mbar_wait(&sh.drained, 0);
      }
    }
  } else {
    // Two teams of four warps (2-5, 6-9), a warp for each 32 lanes of TMEM,
    // take the groups of scales by turns; the second then stores the tile.
    const int team = warp < 6 ? 0 : 1, quarter = warp & 3;
    const uint32_t ts = tmem + ((uint32_t)(32 * quarter) << 16) + acc_cols(BN);
    int it = 0, s = 0, gs = 0, g_at = 0, old = 0;  // old: the stage whose products used this set of scales before
    unsigned gparity = 0, parity_old = 0;
    bool ok = true;
    // a dense Q's vectors of the next k tile (rows wq, wq + 4, ...), loaded one k tile ahead
    const int wq = (warp - 2) & 3;
    constexpr int kRowsOf = kDense ? kMxFewRows / kScaleWarps : 1;
    using Dense = typename std::conditional<kDense, V, mx::Vec32>::type;
    Dense next[kRowsOf];
    // The half of x_scales for the team's next k tile.  It turns with the k
    // tiles that the team itself takes -- both teams' count would bring the
    // same half twice running where a CTA walks tiles with an odd number of
    // them -- so that the team's meeting over the k tile between lies between
    // the reads of a half and the writes for its next use.
    int half = 0;
    const typename Dense::raw* x_at[kRowsOf];
#pragma unroll
    for (int i = 0; i < kRowsOf; ++i)
      x_at[i] = static_cast<const typename Dense::raw*>(a.x) + (wq + kScaleWarps * i) * a.x_ld + 8 * lane;
    auto fetch = [&](int kt) {
      const int left = a.x_cols - kTileK * kt - 8 * lane;
      const bool whole = left >= 8 && a.x_vec;
#pragma unroll
      for (int i = 0; i < kRowsOf; ++i) {
        if (wq + kScaleWarps * i >= a.q_rows) break;  // the same for the warp
        next[i].load_if(x_at[i] + kTileK * kt, whole);
        if (left > 0 && !whole) next[i].load(x_at[i] + kTileK * kt, left);
      }
    };
    if (kDense) {
      // the rows past Q's last stay zero in every stage
      for (int i = threadIdx.x - 64; i < STAGES * kMxFewRows * 8; i += kThreadsMm - 64)
        *reinterpret_cast<uint4*>(smem + i / (8 * kMxFewRows) * kStage + kLanes * kTileKBytes +
                                  16 * (i % (8 * kMxFewRows))) = make_uint4(0u, 0u, 0u, 0u);
      fence_proxy_async_smem();
      asm volatile("bar.sync 3, %0;" ::"n"(kThreadsMm - 64) : "memory");  // both teams
    }
    // P's scales straight from their rows, likewise ahead by a group
    ScaleGroup direct;
    auto fetch_scales = [&](int tile, int kt) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t row = (int64_t)(tile % a.p_tiles) * kLanes + lane + 32 * j;
        direct.m[j] = load_row(a.p_scales + row * a.p_scale_pitch + 8 * kt, row < a.p_rows ? a.k_blocks - 8 * kt : 0,
                               a.p_align);
      }
    };
    auto next_old = [&] {
      if (++old == STAGES) {
        old = 0;
        parity_old ^= 1;
      }
    };
    int n_tile = 0;
    for (int tile = first; tile < a.n_tiles && ok; tile += step, ++n_tile) {
      // Q's rows start inside a piece of 128 when BN is less: q_part turns lane + 32 j into them
      const int q_part = a.q_pieces ? (tile / a.p_tiles) * BN % kLanes : 0;
      const int mine0 = k0 + 2 * ((g_at ^ team) & 1);  // this team's first k tile
      if (mine0 < k1) {
        if (kDense) fetch(mine0);
        if (kDirect) fetch_scales(tile, mine0);
      }
      for (int kt = k0; kt < k1 && ok; kt += 2, ++g_at) {
        if ((g_at & 1) != team) {
          for (int h = 0; h < 2 && kt + h < k1; ++h, ++it) {
            if (it >= kSets) next_old();
            if (++s == STAGES) s = 0;
          }
          if (++gs == GROUPS) {
            gs = 0;
            gparity ^= 1;
          }
          continue;
        }
        ScaleGroup p, q;
        if (kDirect) {
          p = direct;
          p.transpose();
          if (kt + 4 < k1) fetch_scales(tile, kt + 4);
        } else {
          ok = __all_sync(0xFFFFFFFFu, wait(&sh.group_full[gs], gparity));
          if (!kDense && !ok) break;
        }
        const uint8_t* group = group_smem + gs * 2 * kGroup;
        if (by_group) p.load(group, lane, a.p_pieces, kLanes);
        if (kDense) q = ScaleGroup{};
        else if (!a.q_pieces || BN == kLanes) q.load(group + kGroup, lane, a.q_pieces, BN);
        else load_part<BN>(q, group + kGroup, lane, q_part);
        if (by_group) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.group_empty[gs]);
        }
        if (++gs == GROUPS) {
          gs = 0;
          gparity ^= 1;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (kt + h >= k1) break;
          if (it >= kSets) {  // the set is free, and with it (kSets <= STAGES) the stage
            ok = ok && __all_sync(0xFFFFFFFFu, wait(&sh.empty[old], parity_old));
            next_old();
          }
          if constexpr (kDense) {
            uint32_t* x_scale = x_scales[team][half];
            half ^= 1;
            if (ok) {
              uint8_t* to = smem + s * kStage + kLanes * kTileKBytes + 4 * (lane & 3);
              uint8_t* sc = reinterpret_cast<uint8_t*>(x_scale);
#pragma unroll
              for (int i = 0; i < kRowsOf; ++i) {
                const int row = wq + kScaleWarps * i;
                if (row >= a.q_rows) break;
                const uint32_t sb = mx::scale_code(mx::max_of_four(next[i].max_bits()));
                const uint32_t w = mx::encode<false>(next[i], sb, 0, 0, 0);
                *reinterpret_cast<uint32_t*>(to + 128 * row + 16 * ((lane >> 2) ^ (row & 7))) = w;  // swizzled as TMA does
                if ((lane & 3) == 0) sc[8 * row + (lane >> 2)] = (uint8_t)sb;
              }
              const int after = h == 0 && kt + 1 < k1 ? kt + 1 : kt + 4;
              if (after < k1) fetch(after);
              fence_proxy_async_smem();
            }
            ok = all_of_team(team, ok);  // the row's scales are there; or all four stop together
            if (ok) {
              q.m[2 * h].x = lane < a.q_rows ? x_scale[2 * lane] : 0u;
              q.m[2 * h + 1].x = lane < a.q_rows ? x_scale[2 * lane + 1] : 0u;
            }
          }
          if (!ok) break;
          fence_after();
          const uint4 v[4] = {p.m[2 * h], p.m[2 * h + 1], q.m[2 * h], q.m[2 * h + 1]};
          tmem_write16(ts + (it % kSets) * kScaleCols, v);
          tmem_wait_write();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.scales_full[s]);
          ++it;
          if (++s == STAGES) s = 0;
        }
      }
      if (team == 0 || a.split > 1) continue;
      ok = ok && __all_sync(0xFFFFFFFFu, wait(&sh.acc_full, n_tile & 1));
      if (kDense) ok = all_of_team(team, ok);
      if (!ok) break;
      fence_after();
      const int64_t p = (int64_t)(tile % a.p_tiles) * kLanes + 32 * quarter + lane, q0 = (int64_t)(tile / a.p_tiles) * BN;
      constexpr int kStep = BN < 32 ? 8 : 32;
      for (int c = 0; c < BN && q0 + c < a.q_rows; c += kStep) {
        float v[kStep];
        tmem_read<kStep>(tmem + ((uint32_t)(32 * quarter) << 16) + c, v);
        store_run<kStep>(a, p, q0 + c, v);
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.acc_empty);
    }
  }

  if (a.split > 1) {
    // Column c of the tile belongs to rank c / own (own = BN / split, a power
    // of two); its part from rank r goes to that rank's [r][c % own][lane], in
    // the stages' memory, which every CTA of the cluster has finished with
    // after the first barrier.
    const int shift = __ffs(BN / a.split) - 1, own = 1 << shift;
    const int w = warp & 3;
    bool ok = true;
    if (warp >= 6) {
      ok = __all_sync(0xFFFFFFFFu, wait(&sh.acc_full, 0));
      fence_after();
    }
    __syncwarp();
    cluster_sync();
    if (warp >= 6 && ok) {
      constexpr int kStep = BN < 32 ? 8 : 32;
      const uint32_t base = smem_u32(smem) + 4u * (rank * own * kLanes + 32 * w + lane);
      for (int c = 0; c < BN; c += kStep) {
        float v[kStep];
        tmem_read<kStep>(tmem + ((uint32_t)(32 * w) << 16) + c, v);
#pragma unroll
        for (int i = 0; i < kStep; ++i)
          store_remote(base + 4u * kLanes * ((c + i) & (own - 1)), (uint32_t)(c + i) >> shift, v[i]);
      }
    }
    __syncwarp();
    cluster_sync();
    if (warp >= 6) {
      const float* part = reinterpret_cast<const float*>(smem) + 32 * w + lane;
      const int64_t p = (int64_t)(first % a.p_tiles) * kLanes + 32 * w + lane, q0 = (int64_t)(first / a.p_tiles) * BN;
      for (int i = 0; i < own; ++i) {
        const int c = rank * own + i;
        if (p >= a.p_rows || q0 + c >= a.q_rows) break;
        float v = part[i * kLanes];
        for (int r = 1; r < a.split; ++r) v = __fadd_rn(v, part[(r * own + i) * kLanes]);
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
// Two accumulators of 256 columns share 96 of TMEM's 512 with each other
// (the rest holds four sets of scales): the epilogue empties the shared
// columns first and lets the next tile start, then the others while it runs.
//
// What bounds it is the way between L2 and the SMs, by the counters:
// 8192 x 4096 x 4096 (rows, rows, columns) loads 638 MB and stores 67 in 74 us
// at 1.72 GHz, 9.5 TB/s, with the tensor pipe 50 % active; 8192 x 8192 x 2048
// moves 9.0 TB/s in 86 us at 1.75 GHz, 41 % active.  The time goes with the
// clock that the power cap leaves: 72.8 us (3.8 PFLOP/s) in bursts of 12 and
// 77.1 back to back at 1.68 GHz on one GPU, 69 on another.
// Builds without the stores took 60 us where the whole took 69, without the
// products 53; at 8192 x 8192 x 2048 64.7 us without the stores of 87.5.
// Tried and left out: one change of the stores to TMA through shared memory,
// five stages, more shared columns and a second team of scale warps, 74 us
// where this took 69 (five stages alone: 71.1 and 70.2; the others were not
// measured apart, so what TMA stores by themselves would give is not known);
// the scales of both operands as pieces (no change in the kernel, 4 us more
// before it).
constexpr int kPairN = 256;
constexpr int kPairStages = 6;
constexpr int kPairCodes = 2 * kLanes * kTileKBytes;     // per CTA
constexpr int kPairGroups = 3;
constexpr int kPairGroup = 3 * kGroup;                   // per CTA: 128 rows of P, 256 of Q
constexpr int kPairThreads = kThreadsMm;
constexpr int kPairSets = 4;
constexpr int kPairScaleCols = 24;
constexpr int kPairScales = 512 - kPairSets * kPairScaleCols;  // first column of the scales
constexpr int kPairSecond = kPairScales - kPairN;              // first column of the second accumulator
constexpr int kPairShared = kPairN - kPairSecond;              // columns in both
static_assert(kPairShared % 16 == 0 && kPairShared > 0, "the epilogue's order");
static_assert(kPairSets <= kPairStages, "a set is written again after its stage's products");

struct PairShared {
  uint64_t full[kPairStages], scales_full[kPairStages], empty[kPairStages];
  uint64_t group_full[kPairGroups], group_empty[kPairGroups];
  uint64_t acc_full[2], acc_empty, drained;
  uint32_t tmem;
  int abort;
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    mx_matmul_pair_kernel(const __grid_constant__ CUtensorMap p_map, const __grid_constant__ CUtensorMap q_map,
                          const __grid_constant__ CUtensorMap ps_map, const __grid_constant__ CUtensorMap qs_map,
                          const __grid_constant__ MmArgs a) {
  extern __shared__ uint8_t raw_smem[];
  __shared__ PairShared sh;
  uint8_t* smem = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  uint8_t* group_smem = smem + kPairStages * kPairCodes;
  const int groups = (a.k_tiles + 1) / 2;
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.scales_full[s], 8);
      mbar_init(&sh.empty[s], 1);
    }
    for (int g = 0; g < kPairGroups; ++g) {
      mbar_init(&sh.group_full[g], 1);
      mbar_init(&sh.group_empty[g], kScaleWarps);
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
    const int r = wait_bounded(bar, parity, abort_flag);
    if (r == 1) {
      *abort_flag = 1;
      atomicAdd(&g_mx_errors, 1u);
    }
    return r == 0;
  };
  if (a.pdl) dev::pdl_wait();

  if (warp == 0) {
    if (lane == 0) {
      int it = 0, s = 0;
      unsigned parity = 1;
      bool ok = true;
      for (const CUtensorMap* map : {&p_map, &q_map, &ps_map, &qs_map}) prefetch_map(map);
      const uint32_t full = address_in(&sh.full[0], 0), mine = address_in(&sh.group_full[0], rank);
      int gt = 0, gs = 0;
      unsigned gparity = 1;
      auto load_group = [&](uint8_t* to, const CUtensorMap* map, int pieces, int block, int g, uint32_t bar) {
        if (pieces) tma_load_2d_pair(to, map, 0, 2 * (block * groups + g), bar);
        else tma_load_2d_pair(to, map, 16 * g, block * kLanes, bar);
      };
      for (int tile = first; tile < a.n_tiles && ok; tile += step) {
        const int pb = (tile % a.p_tiles) * 2, qb = (tile / a.p_tiles) * 2;  // blocks of 128 rows
        for (int kt = 0; kt < a.k_tiles; ++kt) {
          if ((kt & 1) == 0) {
            if (gt >= kPairGroups && !(ok = wait(&sh.group_empty[gs], gparity))) break;
            fence_proxy_async_smem();  // the scale warps' reads of the group, before it is written again
            mbar_expect_tx(&sh.group_full[gs], kPairGroup);
            uint8_t* to = group_smem + gs * kPairGroup;
            load_group(to, &ps_map, a.p_pieces, pb + rank, kt / 2, mine + 8 * gs);
            load_group(to + kGroup, &qs_map, a.q_pieces, qb, kt / 2, mine + 8 * gs);
            load_group(to + 2 * kGroup, &qs_map, a.q_pieces, qb + 1, kt / 2, mine + 8 * gs);
            ++gt;
            if (++gs == kPairGroups) {
              gs = 0;
              gparity ^= 1;
            }
          }
          if (it >= kPairStages && !(ok = wait(&sh.empty[s], parity))) break;
          uint8_t* st = smem + s * kPairCodes;
          if (rank == 0) mbar_expect_tx(&sh.full[s], 2 * kPairCodes);
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
      if (!ok) linger();  // the copies in flight land before the CTA may end
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
          const uint32_t at = base + s * kPairCodes;
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
  } else if (warp >= 6) {
    const int w = warp & 3;
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
        store_wide(a, p, q0 + col, v);
      }
      fence_before();
    }
  } else if (warp >= 2 && warp < 6) {
    const uint32_t ready = address_in(&sh.scales_full[0], 0);
    const uint32_t ts = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + kPairScales;
    int it = 0, s = 0, gs = 0, set = 0, old = 0;  // old: the stage whose products used this set before
    unsigned gparity = 0, parity_old = 0;
    bool ok = true;
    for (int tile = first; tile < a.n_tiles && ok; tile += step) {
      for (int kt = 0; kt < a.k_tiles && ok; kt += 2) {
        if (!(ok = __all_sync(0xFFFFFFFFu, wait(&sh.group_full[gs], gparity)))) break;
        ScaleGroup p, q, r;
        const uint8_t* group = group_smem + gs * kPairGroup;
        p.load(group, lane, a.p_pieces, kLanes);
        q.load(group + kGroup, lane, a.q_pieces, kLanes);
        r.load(group + 2 * kGroup, lane, a.q_pieces, kLanes);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.group_empty[gs]);
        if (++gs == kPairGroups) {
          gs = 0;
          gparity ^= 1;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (kt + h >= a.k_tiles) break;
          if (it >= kPairSets) {
            if (!(ok = __all_sync(0xFFFFFFFFu, wait(&sh.empty[old], parity_old)))) break;
            if (++old == kPairStages) {
              old = 0;
              parity_old ^= 1;
            }
          }
          fence_after();
          // columns: P's for each half of the k tile, then Q's of rows 0-127 and 128-255 for each half
          const uint4 v[4] = {p.m[2 * h], p.m[2 * h + 1], q.m[2 * h], r.m[2 * h]};
          const uint4 w[2] = {q.m[2 * h + 1], r.m[2 * h + 1]};
          tmem_write16(ts + set * kPairScaleCols, v);
          tmem_write8(ts + set * kPairScaleCols + 16, w);
          tmem_wait_write();
          fence_before();
          __syncwarp();
          if (lane == 0) arrive_at(ready + 8 * s);
          ++it;
          if (++set == kPairSets) set = 0;
          if (++s == kPairStages) s = 0;
        }
      }
    }
  }
  fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA ends while the other may still reach its memory
  fence_after();
  if (warp == 1) tmem_free_pair(tmem, 512);
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

// The scales as they lie -- boxes of 16 bytes of `rows` rows -- or, from a
// workspace of pieces, boxes of one piece (two rows of 1024 bytes).
bool scales_map(CUtensorMap* map, const MxMatrix& m, int rows, uint8_t* pieces, int64_t n_pieces) {
  if (pieces) {
    const cuuint64_t dims[2] = {kGroup / 8, (cuuint64_t)(2 * n_pieces)};
    const cuuint64_t strides[1] = {kGroup / 2};
    const cuuint32_t box[2] = {kGroup / 8, 2}, one[2] = {1, 1};
    return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, pieces, dims, strides, box, one,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  const cuuint64_t dims[2] = {(cuuint64_t)mx_blocks(m.cols), (cuuint64_t)m.rows};
  const cuuint64_t strides[1] = {(cuuint64_t)m.scale_pitch};
  const cuuint32_t box[2] = {16, (cuuint32_t)rows}, one[2] = {1, 1};
  return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, m.scales, dims, strides, box, one,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether a matrix's scale rows can be loaded as they lie (the tensor map's
// alignment).
bool rows_load(const MxMatrix& m) {
  return ((reinterpret_cast<uintptr_t>(m.scales) | (uintptr_t)m.scale_pitch) & 15u) == 0;
}
bool words_load(const MxMatrix& m) {
  return ((reinterpret_cast<uintptr_t>(m.scales) | (uintptr_t)m.scale_pitch) & 3u) == 0;
}
// Pieces of a matrix: blocks of 128 rows (whole pairs of them) times groups of two k tiles.
int64_t row_blocks(const MxMatrix& m) { return 2 * ((m.rows + 255) / 256); }
int64_t groups_of(const MxMatrix& m) { return (mx_blocks(m.cols) + 15) / 16; }
int64_t pieces_bytes(const MxMatrix& m) { return rows_load(m) ? 0 : row_blocks(m) * groups_of(m) * kGroup; }

// Adds a matrix's pieces to the kernel's work (warps -1: too many).
void add_pieces(MxPieceArgs* g, const MxMatrix& m, uint8_t* out) {
  if (!out || g->warps < 0) return;
  const int i = g->n++;
  g->groups = (int)groups_of(m);
  g->k_blocks = (int)mx_blocks(m.cols);
  g->scales[i] = m.scales, g->pitch[i] = m.scale_pitch, g->rows[i] = (int)m.rows, g->out[i] = out;
  const int64_t warps = g->warps + 4 * row_blocks(m) * g->groups;
  g->warps = warps > 0x7FFFFFFF - 8 ? -1 : (int)warps;
  if (i == 0) g->warps0 = g->warps;
}

struct Maps {
  CUtensorMap p, q, ps, qs;
};
bool make_maps(Maps* t, const MxMatrix& p, const MxMatrix& q, int q_rows, uint8_t* p_pieces, uint8_t* q_pieces) {
  return codes_map(&t->p, p, kLanes) && codes_map(&t->q, q, q_rows) &&
         scales_map(&t->ps, p, kLanes, p_pieces, row_blocks(p) * groups_of(p)) &&
         scales_map(&t->qs, q, q_rows, q_pieces, row_blocks(q) * groups_of(q));
}

template <class K>
cudaError_t launch_product(K kernel, int grid, int smem, int cluster, const Maps& t, const MmArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreadsMm);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = (unsigned)cluster;
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
  return cudaLaunchKernelEx(&cfg, kernel, t.p, t.q, t.ps, t.qs, a);
}

template <int BN, int STAGES, int GROUPS, class V = void, bool kDirect = false>
cudaError_t launch(const MxMatrix& p, const MxMatrix& q, MmArgs a, uint8_t* p_pieces, uint8_t* q_pieces, int sm_count,
                   cudaStream_t s) {
  constexpr int kSmem = STAGES * stage_bytes(BN) + GROUPS * 2 * kGroup + 1024;
  static_assert(kSmem <= (BN <= 64 ? 113 : 226) * 1024, "stages fit shared memory (twice for narrow tiles)");
  static_assert(STAGES * stage_bytes(BN) >= BN * kLanes * 4, "the split's parts fit the stages");
  static std::atomic<uint64_t> opted{0};
  const cudaError_t e = opt_in(mx_matmul_kernel<BN, STAGES, GROUPS, V, kDirect>, kSmem, opted);
  if (e != cudaSuccess) return e;
  static_assert(std::is_void<V>::value || BN == kMxFewRows, "a dense Q is one tile wide");
  Maps t;
  if (std::is_void<V>::value) {
    if (!make_maps(&t, p, q, BN, p_pieces, q_pieces)) return cudaErrorInvalidValue;
  } else {  // maps that are not used are P's codes'
    if (!codes_map(&t.p, p, kLanes)) return cudaErrorInvalidValue;
    t.q = t.ps = t.qs = t.p;
    if (!kDirect && !scales_map(&t.ps, p, kLanes, p_pieces, row_blocks(p) * groups_of(p))) return cudaErrorInvalidValue;
  }
  a.p_tiles = (a.p_rows + kLanes - 1) / kLanes;
  const int64_t tiles = (int64_t)a.p_tiles * ((a.q_rows + BN - 1) / BN);
  if (tiles > 0x0FFFFFFF) return cudaErrorInvalidValue;
  a.n_tiles = (int)tiles;
  // one cluster (a CTA when k is not split) per tile, or every SM's CTAs walking the tiles
  const int grid = a.split > 1 ? a.n_tiles * a.split : std::min<int>(a.n_tiles, sm_count * (BN <= 64 ? 2 : 1));
  return launch_product(mx_matmul_kernel<BN, STAGES, GROUPS, V, kDirect>, grid, kSmem, a.split, t, a, s);
}

cudaError_t launch_pair(const MxMatrix& p, const MxMatrix& q, MmArgs a, uint8_t* p_pieces, uint8_t* q_pieces, int sm_count,
                        cudaStream_t s) {
  constexpr int kSmem = kPairStages * kPairCodes + kPairGroups * kPairGroup + 1024;
  static_assert(kSmem <= 226 * 1024, "stages fit shared memory");
  static std::atomic<uint64_t> opted{0};
  const cudaError_t e = opt_in(mx_matmul_pair_kernel, kSmem, opted);
  if (e != cudaSuccess) return e;
  Maps t;
  if (!make_maps(&t, p, q, kLanes, p_pieces, q_pieces)) return cudaErrorInvalidValue;
  a.p_tiles = (a.p_rows + 2 * kLanes - 1) / (2 * kLanes);
  const int64_t tiles = (int64_t)a.p_tiles * ((a.q_rows + kPairN - 1) / kPairN);
  if (tiles > 0x0FFFFFFF) return cudaErrorInvalidValue;
  a.n_tiles = (int)tiles;
  return launch_product(mx_matmul_pair_kernel, 2 * (int)std::min<int64_t>(tiles, sm_count / 2), kSmem, 1, t, a, s);
}

// Whether the product runs on CTA pairs: more than 128 rows on both sides, and
// 256 x 256 tiles for half of the pairs.
bool by_pairs(int64_t m, int64_t n, int sm_count) {
  return std::min(m, n) > kLanes && ((m + 255) / 256) * ((n + 255) / 256) >= sm_count / 4;
}

}  // namespace

int64_t mx_matmul_workspace(const MxMatrix& a, const MxMatrix& b) { return pieces_bytes(a) + pieces_bytes(b); }
bool mx_linear_pieces(const MxMatrix& b, void* workspace, MxPieceArgs* g) {
  *g = MxPieceArgs{};
  if (rows_load(b)) return true;
  add_pieces(g, b, static_cast<uint8_t*>(workspace));
  return g->warps >= 0;
}
int64_t mx_few_rows_workspace(const MxMatrix& b) { return words_load(b) ? 0 : pieces_bytes(b); }

cudaError_t launch_mx_matmul(const MxMatmulArgs& m, int sm_count, cudaStream_t s) {
  if (mx_by_gemv(m.a.rows, m.a.cols)) return launch_mx_gemv(m, sm_count, s);
  if (!encode_fn()) return cudaErrorNotSupported;
  // Many tiles: CTA pairs, a's rows as lanes, whose results go out 32 bytes at
  // a time along a row -- or b's rows as lanes where the result's rows are not
  // 32-byte aligned, which makes a warp's 32 lanes neighbours in memory.  Few
  // tiles: b's rows as lanes, narrower tiles, k split over a cluster.
  const int64_t row_bytes = m.ld * (m.type == kMxF32 ? 4 : 2);
  const bool aligned = ((reinterpret_cast<uintptr_t>(m.out) | (uintptr_t)row_bytes) & 31u) == 0;
  const bool many = !m.x && by_pairs(m.a.rows, m.b.rows, sm_count);
  const bool swap = !many || !aligned;
  const MxMatrix& p = swap ? m.b : m.a;
  const MxMatrix& q = swap ? m.a : m.b;

  MmArgs a = {};
  a.p_rows = (int)p.rows, a.q_rows = (int)q.rows;
  a.k_tiles = (int)((mx_blocks(p.cols) + 7) / 8);
  a.out = m.out, a.type = m.type;
  a.p_stride = swap ? 1 : m.ld, a.q_stride = swap ? m.ld : 1;
  a.vec = !swap;
  a.split = 1;
  a.pdl = m.pdl;

  uint8_t* space = static_cast<uint8_t*>(m.workspace);
  uint8_t *p_pieces = nullptr, *q_pieces = nullptr;
  const bool direct = m.x && !rows_load(p) && words_load(p);
  if (direct) {
    a.p_scales = p.scales, a.p_scale_pitch = p.scale_pitch;
    a.p_align = (reinterpret_cast<uintptr_t>(p.scales) | (uintptr_t)p.scale_pitch) & 7u ? 4 : 8;
    a.k_blocks = (int)mx_blocks(p.cols);
  } else if (!rows_load(p)) {
    p_pieces = space, space += pieces_bytes(p);
  }
  if (!m.x && !rows_load(q)) q_pieces = space;
  a.p_pieces = p_pieces != nullptr, a.q_pieces = q_pieces != nullptr;
  if (p_pieces || q_pieces) {
    MxPieceArgs g = {};
    add_pieces(&g, p, p_pieces);
    add_pieces(&g, q, q_pieces);
    if (g.warps < 0) return cudaErrorInvalidValue;
    if (!m.b_ready) {
      mx_scale_pieces_kernel<<<(g.warps + 7) / 8, 256, 0, s>>>(g);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
      a.pdl = 1;
    }
  }
  a.p_early = swap && m.b_ready && !p_pieces && !q_pieces;

  if (many) return launch_pair(p, q, a, p_pieces, q_pieces, sm_count, s);
  const int64_t p_tiles = (p.rows + kLanes - 1) / kLanes;
  // a part of k has at least 4 k tiles (16 columns: 12288 x 4096, 192 CTAs
  // instead of 96: 15.2 -> 12.2 us) or 8, below which the exchange costs more
  auto split_for = [&](int bn, int slots) {
    const int64_t tiles = p_tiles * ((q.rows + bn - 1) / bn);
    const int64_t most = std::min<int64_t>(std::min<int64_t>(8, a.k_tiles / (bn == 16 ? 4 : 8)), slots / tiles);
    for (a.split = 1; 2 * a.split <= most;) a.split *= 2;
  };
  if (q.rows <= kMxFewRows) {
    split_for(16, 2 * sm_count);
    if (!m.x) return launch<16, 5, 3>(p, q, a, p_pieces, q_pieces, sm_count, s);
    a.x = m.x, a.x_ld = m.x_ld, a.x_cols = (int)q.cols;
    const int64_t bytes = m.x_ld * (m.x_type == kMxF32 ? 4 : 2);
    a.x_vec = ((reinterpret_cast<uintptr_t>(m.x) | (uintptr_t)bytes) & 15u) == 0;
    auto dense = [&](auto v) {
      using V = decltype(v);
      return direct ? launch<16, 5, 3, V, true>(p, q, a, p_pieces, q_pieces, sm_count, s)
                    : launch<16, 5, 3, V, false>(p, q, a, p_pieces, q_pieces, sm_count, s);
    };
    if (m.x_type == kMxBf16) return dense(mx::Vec16<dev::Bf16>{});
    if (m.x_type == kMxF16) return dense(mx::Vec16<dev::F16>{});
    return dense(mx::Vec32{});
  }
  if (p_tiles * ((q.rows + 31) / 32) <= sm_count) {
    split_for(32, 2 * sm_count);
    return launch<32, 4, 3>(p, q, a, p_pieces, q_pieces, sm_count, s);
  }
  if (p_tiles * ((q.rows + 63) / 64) <= sm_count) {
    split_for(64, 2 * sm_count);
    return launch<64, 4, 2>(p, q, a, p_pieces, q_pieces, sm_count, s);
  }
  split_for(128, sm_count);
  return launch<128, 6, 3>(p, q, a, p_pieces, q_pieces, sm_count, s);
}

// How many bounded waits have run out on the current device (waits for `s`).
cudaError_t mx_matmul_errors(unsigned* count, cudaStream_t s) {
  const cudaError_t e = cudaMemcpyFromSymbolAsync(count, g_mx_errors, sizeof *count, 0, cudaMemcpyDeviceToHost, s);
  return e == cudaSuccess ? cudaStreamSynchronize(s) : e;
}

}  // namespace zsm
