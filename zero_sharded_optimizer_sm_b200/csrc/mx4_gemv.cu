// The MX4 product of one row of a (a token): out[i] = sum over k of a[k] b[i][k],
// a dense (quantised on its way) or MX4.
//
// Such a product reads b once and uses each element once, so it streams b
// through registers instead of the tensor core, whose tiles need TMA, their
// scales brought into place and an epilogue.  A warp takes a row of b, a lane
// one block of 32 at a time (16 bytes, the next step's on their way); a's
// blocks lie in shared memory as binary16.  A product of two elements is a
// whole number of quarters up to 36, and eight of them one after another at
// most 1152 quarters: binary16, with 11 bits, sums them exactly, and binary32
// the four such sums of a block.  Each block's sum times its two scales is
// added in binary32 in the lane, the lanes' sums by a fixed tree: the same
// bits every time.
//
// One token, weights not in L2 (us, here and on the tensor cores): 768 x 768
// 2.2 and 5.1, 2304 x 768 2.2 and 5.0, 8192 x 2048 4.4 and 6.9, 12288 x 4096
// 8.2 and 10.9, 50304 x 2048 13.6 and 15.0.  The large ones wait for nothing
// alone: at 12288 x 4096 the counters have the issue slots 66 % used (a lane's
// block has 16 conversions, 16 multiply-adds, the loads, the sums and scales),
// the busiest unit 42 %, DRAM 29 %, the rest latency of the loads and of shared
// memory.  With two rows of a beside each other
// 12288 x 4096 took 12.8 us and with four 27, the tensor cores 11 for both, so
// two tokens are theirs.  Two CTAs of 512 threads to an SM, not four of 256
// or one of 1024: each quantises the whole of a, which 16384 columns make
// 2.6 us longer with four, and one waits for it (2304 x 768: 2.7).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "device_math.cuh"
#include "mx4.cuh"
#include "mx4_quant.cuh"

namespace zsm {
namespace {

using namespace dev;
using namespace mx;

constexpr int kGemvThreads = 512;
constexpr int kGemvCtas = 2;                // to an SM
constexpr int kGemvWarps = kGemvThreads / 32;
constexpr int kGemvBlocks = 2;              // of a row, to a lane and step
constexpr int kStep = 32 * kGemvBlocks;     // blocks to a warp's step
constexpr int kStepBytes = kStep * 68;      // a's share of shared memory for them: codes as halves, scales
constexpr int kMaxGemvBytes = 48 * 1024;    // without a launch attribute: 22528 columns
constexpr uint32_t kNan = 1u << 20;         // the scale of a block that is not a number

struct GemvArgs {
  MxMatrix b;
  MxMatrix a;     // one row, when x is null
  const void* x;  // or its dense values
  int x_vec;
  void* out;
  int type;
};

__device__ __forceinline__ __half2 as_half2(uint32_t v) { return *reinterpret_cast<const __half2*>(&v); }

__device__ __forceinline__ uint4 load_if(const uint8_t* p, bool yes) {
  uint4 r;
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@q ld.global.cs.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(r.x), "=&r"(r.y), "=&r"(r.z), "=&r"(r.w)
      : "l"(p), "r"((int)yes)
      : "memory");
  return r;
}
__device__ __forceinline__ uint32_t load_byte_if(const uint8_t* p, bool yes) {  // or the scale 1
  uint32_t r;
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\tmov.b32 %0, 127;\n\t@q ld.global.u8 %0, [%1];\n\t}"
               : "=&r"(r)
               : "l"(p), "r"((int)yes)
               : "memory");
  return r;
}

// One block's term: its sum of products times 2^(sw - 127) and 2^sx.
__device__ __forceinline__ float add_block(float acc, float sum, uint32_t sw, uint32_t sx) {
  const uint32_t e = sw + sx;  // a power of two's exponent field
  if (e - 1u < 254u && sw != 255u) return __fmaf_rn(sum, __uint_as_float(e << 23), acc);
  if (sw == 255u || (int)sx > 1000) return __uint_as_float(0x7FC00000u);
  if (sum == 0.0f) return acc;
  const double p = (double)sum * __hiloint2double((int)((e + (1023u - 127u)) << 20), 0);
  return __fadd_rn(acc, (float)p);
}

// V: the vector type of a dense a, or void.
template <class V>
__global__ void __launch_bounds__(kGemvThreads, kGemvCtas) mx_gemv_kernel(const __grid_constant__ GemvArgs a) {
  // a's blocks by steps: word q's elements of a lane's block j, 16 bytes a
  // lane (so that q and j are constants in an address); then all scales
  extern __shared__ uint4 space[];
  const int nb = (int)((a.b.cols + kMxBlock - 1) / kMxBlock);
  const int steps = (nb + kStep - 1) / kStep;
  uint32_t* xs = reinterpret_cast<uint32_t*>(space + steps * kStep * 4);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t row = (int64_t)blockIdx.x * kGemvWarps + warp;
  const int row_step = gridDim.x * kGemvWarps;

  // the next step's codes and scales in b
  const uint8_t* codes = a.b.codes + row * a.b.code_pitch + 16 * lane;
  const uint8_t* scales = a.b.scales + row * a.b.scale_pitch + lane;
  const int64_t code_hop = row_step * a.b.code_pitch - (int64_t)(steps - 1) * kStep * 16;
  const int64_t scale_hop = row_step * a.b.scale_pitch - (int64_t)(steps - 1) * kStep;
  uint4 w[kGemvBlocks];
  uint32_t s[kGemvBlocks];
  auto load = [&](int left) {  // blocks left in the row, from this lane's on
#pragma unroll
    for (int j = 0; j < kGemvBlocks; ++j) {
      w[j] = load_if(codes + 512 * j, left > 32 * j);
      s[j] = load_byte_if(scales + 32 * j, left > 32 * j);
    }
  };
  load(row < a.b.rows ? nb - lane : 0);

  for (int c0 = 32 * warp; c0 < steps * kStep * 4; c0 += kGemvThreads) {
    const int c = c0 + lane, block = c >> 2;
    const bool live = block < nb;
    uint32_t word = 0, sc = 127;
    if constexpr (std::is_void<V>::value) {
      if (live) {
        word = *reinterpret_cast<const uint32_t*>(a.a.codes + 4 * c);
        sc = a.a.scales[block];
        if (sc == 255u) word = 0;
      }
    } else {
      V x;
      x.clear();
      if (live) load8(x, static_cast<const typename V::raw*>(a.x) + 8 * c, a.b.cols - 8 * c, a.x_vec);
      sc = scale_code(max_of_four(x.max_bits()));
      word = encode<false>(x, sc, 0, 0, 0);
      if (!live) sc = 127;
    }
    uint32_t h[4];
    decode8(word, h);
    space[(block >> 5) * 128 + (c & 3) * 32 + (block & 31)] = make_uint4(h[0], h[1], h[2], h[3]);
    if ((c & 3) == 0) xs[block] = (sc == 255u ? kNan : sc) - 127u;
  }
  __syncthreads();

  for (; row < a.b.rows; row += row_step) {
    float acc = 0.0f;
    const uint4* xv = space + lane;
    const uint32_t* xsc = xs + lane;
    for (int left = nb; left > 0; left -= kStep, xv += kStep * 4, xsc += kStep) {
      uint4 c[kGemvBlocks];
      uint32_t sw[kGemvBlocks];
#pragma unroll
      for (int j = 0; j < kGemvBlocks; ++j) c[j] = w[j], sw[j] = s[j];
      if (left > kStep) {
        codes += 16 * kStep, scales += kStep;
        load(left - kStep - lane);
      } else {
        codes += code_hop, scales += scale_hop;
        load(row + row_step < a.b.rows ? nb - lane : 0);
      }
#pragma unroll
      for (int j = 0; j < kGemvBlocks; ++j) {
        if (j > 0 && left <= 32 * j) break;
        const uint32_t word[4] = {c[j].x, c[j].y, c[j].z, c[j].w};
        __half2 sum[2];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t h[4];
          decode8(word[q], h);
          const uint4 v = xv[(4 * j + q) * 32];
          __half2 r = q & 1 ? __hfma2(as_half2(h[0]), as_half2(v.x), sum[q >> 1]) : __hmul2(as_half2(h[0]), as_half2(v.x));
          r = __hfma2(as_half2(h[1]), as_half2(v.y), r);
          r = __hfma2(as_half2(h[2]), as_half2(v.z), r);
          sum[q >> 1] = __hfma2(as_half2(h[3]), as_half2(v.w), r);
        }
        const float2 u = __half22float2(sum[0]), v = __half22float2(sum[1]);
        acc = add_block(acc, (u.x + u.y) + (v.x + v.y), sw[j], xsc[32 * j]);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc = __fadd_rn(acc, __shfl_xor_sync(0xFFFFFFFFu, acc, o));
    if (lane == 0) {
      if (a.type == kMxBf16) static_cast<uint16_t*>(a.out)[row] = Bf16::rn(acc);
      else if (a.type == kMxF16) static_cast<uint16_t*>(a.out)[row] = F16::rn(acc);
      else static_cast<float*>(a.out)[row] = acc;
    }
  }
}

int64_t gemv_bytes(int64_t cols) { return (mx_blocks(cols) + kStep - 1) / kStep * kStepBytes; }

template <class V>
cudaError_t launch_gemv(const GemvArgs& a, int sm_count, cudaStream_t s) {
  const int grid = (int)std::min<int64_t>((a.b.rows + kGemvWarps - 1) / kGemvWarps, kGemvCtas * sm_count);
  mx_gemv_kernel<V><<<grid, kGemvThreads, gemv_bytes(a.b.cols), s>>>(a);
  return cudaGetLastError();
}

}  // namespace

bool mx_by_gemv(int64_t rows, int64_t cols) { return rows == 1 && gemv_bytes(cols) <= kMaxGemvBytes; }

cudaError_t launch_mx_gemv(const MxMatmulArgs& m, int sm_count, cudaStream_t s) {
  GemvArgs a = {};
  a.b = m.b, a.a = m.a;
  a.x = m.x, a.x_vec = (reinterpret_cast<uintptr_t>(m.x) & 15u) == 0;
  a.out = m.out, a.type = m.type;
  if (!m.x) return launch_gemv<void>(a, sm_count, s);
  if (m.x_type == kMxBf16) return launch_gemv<Vec16<Bf16>>(a, sm_count, s);
  if (m.x_type == kMxF16) return launch_gemv<Vec16<F16>>(a, sm_count, s);
  return launch_gemv<Vec32>(a, sm_count, s);
}

}  // namespace zsm
