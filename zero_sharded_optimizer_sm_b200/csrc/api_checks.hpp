// Argument checks shared by the entry points that need no context.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "../../include/zero_sm.h"
#include "mx4.cuh"

namespace zsm {
namespace api {

inline zero_status fail(zero_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  zsm::set_thread_error(buf);
  return s;
}

inline zero_status cuda_fail(cudaError_t e, const char* what) {
  return fail(ZERO_ECUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

constexpr int64_t kMaxDim = 0x7FFFFFFF - 255;  // row and column numbers of a tile stay in 32 bits

inline int elem_bytes(int32_t dtype) { return dtype == ZERO_DTYPE_F32 ? 4 : 2; }

inline zero_status check_dtype(int32_t dtype) {
  if (dtype != ZERO_DTYPE_BF16 && dtype != ZERO_DTYPE_F16 && dtype != ZERO_DTYPE_F32)
    return fail(ZERO_EINVAL, "unknown dtype %d", dtype);
  return ZERO_OK;
}

inline zero_status check_dense(const char* name, const void* p, int32_t dtype, int64_t rows, int64_t cols, int64_t ld) {
  const zero_status st = check_dtype(dtype);
  if (st != ZERO_OK) return st;
  if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim)
    return fail(ZERO_EINVAL, "%s: %lld x %lld is out of range", name, (long long)rows, (long long)cols);
  if (rows == 0 || cols == 0) return ZERO_OK;
  if (!p || (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(elem_bytes(dtype) - 1)))
    return fail(ZERO_EINVAL, "%s is null or not aligned to its elements", name);
  if (ld < cols && rows > 1)
    return fail(ZERO_EINVAL, "%s: %lld elements between rows of %lld", name, (long long)ld, (long long)cols);
  return ZERO_OK;
}

inline zero_status check_mx4(const char* name, const zero_mx4* m) {
  if (!m) return fail(ZERO_EINVAL, "%s is NULL", name);
  if (m->rows < 0 || m->cols < 0 || m->rows > kMaxDim || m->cols > kMaxDim)
    return fail(ZERO_EINVAL, "%s: %lld x %lld is out of range", name, (long long)m->rows, (long long)m->cols);
  if (m->rows == 0 || m->cols == 0) return ZERO_OK;
  const int64_t nb = zsm::mx_blocks(m->cols);
  if (!m->codes || (reinterpret_cast<uintptr_t>(m->codes) & 15u) || !m->scales)
    return fail(ZERO_EINVAL, "%s: codes must be 16-byte aligned and neither codes nor scales NULL", name);
  if (m->code_pitch % 16 || m->code_pitch < 16 * nb)
    return fail(ZERO_EINVAL, "%s: code_pitch %lld must be a multiple of 16, at least 16 * %lld blocks", name,
                (long long)m->code_pitch, (long long)nb);
  if (m->scale_pitch < nb)
    return fail(ZERO_EINVAL, "%s: scale_pitch %lld is less than the row's %lld blocks", name, (long long)m->scale_pitch,
                (long long)nb);
  return ZERO_OK;
}

inline zero_status check_mx8(const char* name, const zero_mx8* m) {
  if (!m) return fail(ZERO_EINVAL, "%s is NULL", name);
  if (m->rows < 0 || m->cols < 0 || m->rows > kMaxDim || m->cols > kMaxDim)
    return fail(ZERO_EINVAL, "%s: %lld x %lld is out of range", name, (long long)m->rows, (long long)m->cols);
  if (m->rows == 0 || m->cols == 0) return ZERO_OK;
  const int64_t nb = zsm::mx_blocks(m->cols);
  if (!m->codes || (reinterpret_cast<uintptr_t>(m->codes) & 15u) || !m->scales)
    return fail(ZERO_EINVAL, "%s: codes must be 16-byte aligned and neither codes nor scales NULL", name);
  if (m->code_pitch % 16 || m->code_pitch < 32 * nb)
    return fail(ZERO_EINVAL, "%s: code_pitch %lld must be a multiple of 16, at least 32 * %lld blocks", name,
                (long long)m->code_pitch, (long long)nb);
  if (m->scale_pitch < nb)
    return fail(ZERO_EINVAL, "%s: scale_pitch %lld is less than the row's %lld blocks", name, (long long)m->scale_pitch,
                (long long)nb);
  return ZERO_OK;
}

inline MxMatrix matrix(const zero_mx4& m) {
  return {static_cast<uint8_t*>(m.codes), static_cast<uint8_t*>(m.scales), m.rows, m.cols, m.code_pitch, m.scale_pitch};
}
inline MxMatrix matrix8(const zero_mx8& m) {
  return {static_cast<uint8_t*>(m.codes), static_cast<uint8_t*>(m.scales), m.rows, m.cols, m.code_pitch, m.scale_pitch};
}

// SMs of the current device, asked for once per device.
inline cudaError_t sm_count(int* n) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (*n = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && dev < 64) known[dev].store(*n, std::memory_order_relaxed);
  return e;
}

inline zero_status check_workspace(const void* workspace, int64_t have, int64_t need) {
  if (need > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u) || have < need))
    return fail(ZERO_EINVAL, "the workspace must be 16-byte aligned and of at least %lld bytes (%lld given)",
                (long long)need, (long long)have);
  return ZERO_OK;
}

// A result that is a sum over no elements: zeros.
inline zero_status zero_fill(void* out, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, cudaStream_t s) {
  const int es = elem_bytes(dtype);
  const cudaError_t e = cudaMemset2DAsync(out, (size_t)(rows > 1 ? ld : cols) * es, 0, (size_t)cols * es, (size_t)rows, s);
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "clearing the result");
}

}  // namespace api
}  // namespace zsm
