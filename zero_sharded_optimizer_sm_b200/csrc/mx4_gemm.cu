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
__host__ __device__ constexpr uint32_t inst_desc(int n, uint32_t id) {
  return (id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | (1u << 27) | (id << 29);
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

// N consecutive accumulator columns of this warp's 32 lanes.
template <int N>
__device__ __forceinline__ void tmem_read(uint32_t addr, float (&v)[N]) {
  static_assert(N == 8 || N == 32, "built widths");
  uint32_t r[N];
  if constexpr (N == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
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

// 16 scale bytes (two k tiles) of one row, of which the first n exist (the
// others are 0), by loads as wide as the rows' alignment allows.
__device__ __forceinline__ uint4 load_scales(const uint8_t* p, int n, int align) {
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  if (n >= 16 && align == 16) return *reinterpret_cast<const uint4*>(p);
  if (n >= 16 && align == 8) {
    const uint2 lo = *reinterpret_cast<const uint2*>(p), hi = *reinterpret_cast<const uint2*>(p + 8);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
  if (align >= 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n >= 4 * j + 4) w[j] = *reinterpret_cast<const uint32_t*>(p + 4 * j);
      else
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (n > 4 * j + i) w[j] |= (uint32_t)p[4 * j + i] << (8 * i);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (n > j) w[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void st_word(uint32_t addr, uint32_t w) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(w) : "memory");
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
    const int r = mbar_wait_or_abort(bar, parity, abort_flag, kWaitNs);
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
    // Thread t holds row t of P and rows t (and t + 128) of Q, two k tiles at
    // a time, the next two loaded before the present ones are stored.
    const int t = threadIdx.x - 256;  // 0..127
    const uint32_t at = 16u * (t & 31) + 4u * (t >> 5);
    uint4 cur[1 + kQ], nxt[1 + kQ];
    auto fetch = [&](int tile, int kt, uint4 (&r)[1 + kQ]) {
      const int left = a.k_blocks - 8 * kt, most = kt & 1 ? 8 : 16;
      const int64_t p = (int64_t)(tile % a.p_tiles) * kLanes + t, q = (int64_t)(tile / a.p_tiles) * BN + t;
      r[0] = load_scales(a.p_scales + p * a.p_scale_pitch + 8 * kt, p < a.p_rows ? left : 0, min(a.p_align, most));
#pragma unroll
      for (int j = 0; j < kQ; ++j)
        r[1 + j] = load_scales(a.q_scales + (q + 128 * j) * a.q_scale_pitch + 8 * kt,
                               q + 128 * j < a.q_rows && t + 128 * j < BN ? left : 0,
                               min(a.q_align, most));
    };
    int it = 0;
    bool ok = true;
    if (first < a.n_tiles && k0 < k1) fetch(first, k0, nxt);
    for (int tile = first; tile < a.n_tiles && ok; tile += step) {
      for (int kt = k0; kt < k1 && ok; kt += 2) {
#pragma unroll
        for (int j = 0; j < 1 + kQ; ++j) cur[j] = nxt[j];
        if (kt + 2 < k1) fetch(tile, kt + 2, nxt);
        else if (tile + step < a.n_tiles) fetch(tile + step, k0, nxt);
        for (int h = 0; h < 2 && kt + h < k1; ++h, ++it) {
          const int s = it % STAGES;
          if (it >= STAGES &&
              !(ok = __all_sync(0xFFFFFFFFu, wait(&sh.empty[s], ((it / STAGES) - 1) & 1))))
            break;  // the whole warp
          const uint32_t dst = smem_u32(smem + s * kStage) + stage_codes(BN) + at;
          st_word(dst, h ? cur[0].z : cur[0].x);
          st_word(dst + 512, h ? cur[0].w : cur[0].y);
#pragma unroll
          for (int j = 0; j < kQ; ++j) {
            st_word(dst + 1024 + 512 * j, h ? cur[1 + j].z : cur[1 + j].x);
            st_word(dst + 1024 + 512 * (kQ + j), h ? cur[1 + j].w : cur[1 + j].y);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.scales_full[s]);
        }
      }
    }
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

template <int BN, int STAGES>
cudaError_t launch(const MxMatrix& p, const MxMatrix& q, MmArgs a, int sm_count, cudaStream_t s) {
  CUtensorMap pm, qm;
  if (!codes_map(&pm, p, kLanes) || !codes_map(&qm, q, BN)) return cudaErrorInvalidValue;
  constexpr int kSmem = STAGES * stage_bytes(BN) + 1024;
  static_assert(kSmem <= 227 * 1024 - 1024, "stages fit shared memory");
  static_assert(STAGES * stage_bytes(BN) >= (BN + 8) * kLanes * 4 || BN > 128, "the split's parts fit the stages");
  auto kernel = mx_matmul_kernel<BN, STAGES>;
  // the large dynamic shared memory is opted into once per device
  static std::atomic<uint64_t> opted{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!bit || !(opted.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    opted.fetch_or(bit, std::memory_order_release);
  }
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

}  // namespace

cudaError_t launch_mx_matmul(const MxMatmulArgs& m, int sm_count, cudaStream_t s) {
  if (!encode_fn()) return cudaErrorNotSupported;
  // Plain orientation, 128 x 256 tiles, when they give every SM one; below
  // that the swapped one (a's rows are the columns of the tile), where the
  // parts of a split k end in stores that run along the result's rows.
  const bool swap = ((m.a.rows + kLanes - 1) / kLanes) * ((m.b.rows + 255) / 256) < sm_count;
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
  const int64_t row_bytes = m.ld * (m.type == kMxF32 ? 4 : 2);
  a.vec = !swap && ((reinterpret_cast<uintptr_t>(m.out) | (uintptr_t)row_bytes) & 31u) == 0;
  a.split = 1;
  if (!swap) return launch<256, 4>(p, q, a, sm_count, s);
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
