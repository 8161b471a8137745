// Entry points of the operators around a layer's products: 8-bit checkpoints
// (zero_mx8_*), the norm and the embedding.  Argument checks and launches.
#include <cuda_runtime.h>

#include <cmath>

#include "../../include/zero_sm.h"
#include "api_checks.hpp"
#include "embedding.cuh"
#include "mx8.cuh"
#include "rms_norm.cuh"

static_assert(ZERO_MX8_BLOCK == zsm::kMxBlock, "block length");

namespace {

using namespace zsm::api;

zero_status launched(cudaError_t e, const char* what) { return e == cudaSuccess ? ZERO_OK : cuda_fail(e, what); }

// An optional matrix of the operation's type.
zero_status check_optional(const char* name, const void* p, int32_t dtype, int64_t rows, int64_t cols, int64_t ld) {
  return p ? check_dense(name, p, dtype, rows, cols, ld) : ZERO_OK;
}

zero_status check_vector(const char* name, const void* p, int32_t dtype, int64_t n) {
  return check_dense(name, p, dtype, 1, n, n);
}

zero_status check_shape8(const char* name, const zero_mx8* m, int64_t rows, int64_t cols) {
  const zero_status st = check_mx8(name, m);
  if (st != ZERO_OK) return st;
  if (m->rows != rows || m->cols != cols)
    return fail(ZERO_EINVAL, "%s is not %lld x %lld", name, (long long)rows, (long long)cols);
  return ZERO_OK;
}

zero_status check_tokens(const void* tokens, int32_t token_bytes, int64_t n, int64_t vocab) {
  if (token_bytes != 4 && token_bytes != 8)
    return fail(ZERO_EINVAL, "tokens of %d bytes: 4 or 8 are needed", token_bytes);
  if (n < 0 || n > kMaxDim) return fail(ZERO_EINVAL, "%lld tokens: out of range", (long long)n);
  if (vocab < 0 || vocab > kMaxDim) return fail(ZERO_EINVAL, "a vocabulary of %lld: out of range", (long long)vocab);
  if (n && (!tokens || (reinterpret_cast<uintptr_t>(tokens) & (uintptr_t)(token_bytes - 1))))
    return fail(ZERO_EINVAL, "tokens is null or not aligned to its elements");
  return ZERO_OK;
}

zero_status check_scale(double scale) {
  return std::isfinite((float)scale) ? ZERO_OK : fail(ZERO_EINVAL, "scale %g is not a finite binary32 number", scale);
}

}  // namespace

extern "C" {

zero_status zero_mx8_quantize(const void* src, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, const zero_mx8* out,
                              void* stream) {
  zero_status st = check_dense("src", src, dtype, rows, cols, ld);
  if (st != ZERO_OK) return st;
  if ((st = check_shape8("out", out, rows, cols)) != ZERO_OK) return st;
  if (rows == 0 || cols == 0) return ZERO_OK;
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  const zsm::Mx8QuantArgs a = {src, dtype, rows, cols, rows > 1 ? ld : cols, matrix8(*out)};
  return launched(zsm::launch_mx8_quantize(a, sms, static_cast<cudaStream_t>(stream)), "MX8 quantise launch");
}

zero_status zero_mx8_dequantize(const zero_mx8* in, void* dst, int32_t dtype, int64_t ld, void* stream) {
  zero_status st = check_mx8("in", in);
  if (st != ZERO_OK) return st;
  if ((st = check_dense("dst", dst, dtype, in->rows, in->cols, ld)) != ZERO_OK) return st;
  if (in->rows == 0 || in->cols == 0) return ZERO_OK;
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  const zsm::Mx8DequantArgs a = {matrix8(*in), dst, dtype, in->rows > 1 ? ld : in->cols};
  return launched(zsm::launch_mx8_dequantize(a, sms, static_cast<cudaStream_t>(stream)), "MX8 read-back launch");
}

zero_status zero_rms_norm(const void* x, const void* residual, int32_t dtype, int64_t rows, int64_t cols, int64_t ld_x,
                          int64_t ld_residual, const void* weight, int32_t weight_dtype, double eps, void* y, int64_t ld_y,
                          void* h, int64_t ld_h, const zero_mx8* y8, const zero_mx8* h8, float* rstd, void* stream) {
  zero_status st = check_dense("x", x, dtype, rows, cols, ld_x);
  if (st != ZERO_OK) return st;
  if ((st = check_optional("residual", residual, dtype, rows, cols, ld_residual)) != ZERO_OK) return st;
  if ((st = check_vector("weight", weight, weight_dtype, cols)) != ZERO_OK) return st;
  if (!(eps > 0.0) || !std::isfinite((float)eps) || (float)eps == 0.0f)
    return fail(ZERO_EINVAL, "eps %g must be a positive binary32 number", eps);
  if ((st = check_optional("y", y, dtype, rows, cols, ld_y)) != ZERO_OK) return st;
  if ((st = check_optional("h", h, dtype, rows, cols, ld_h)) != ZERO_OK) return st;
  if (y8 && (st = check_shape8("y8", y8, rows, cols)) != ZERO_OK) return st;
  if (h8 && (st = check_shape8("h8", h8, rows, cols)) != ZERO_OK) return st;
  if (reinterpret_cast<uintptr_t>(rstd) & 3u) return fail(ZERO_EINVAL, "rstd is not aligned to its elements");
  if (rows && cols == 0 && rstd) {  // the mean of nothing: not a number (four bytes of 0xFF are one)
    const cudaError_t e = cudaMemsetAsync(rstd, 0xFF, sizeof(float) * (size_t)rows, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "rows without columns");
  }
  if (rows == 0 || cols == 0) return ZERO_OK;  // (the results' addresses may be null then)
  if (!y && !h && !y8 && !h8 && !rstd) return fail(ZERO_EINVAL, "no result is given");
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  zsm::RmsNormArgs a = {};
  a.x = x, a.residual = residual, a.type = dtype;
  a.rows = rows, a.cols = cols;
  const bool one = rows == 1;
  a.ld_x = one ? cols : ld_x, a.ld_residual = one ? cols : ld_residual;
  a.weight = weight, a.w_type = weight_dtype, a.w_aligned = (reinterpret_cast<uintptr_t>(weight) & 15u) == 0;
  a.eps = (float)eps;
  a.y = y, a.ld_y = one ? cols : ld_y;
  a.h = h, a.ld_h = one ? cols : ld_h;
  if (y8) a.y8 = matrix8(*y8);
  if (h8) a.h8 = matrix8(*h8);
  a.rstd = rstd;
  return launched(zsm::launch_rms_norm(a, sms, static_cast<cudaStream_t>(stream)), "norm launch");
}

zero_status zero_rms_norm_backward_workspace(int64_t rows, int64_t cols, int64_t* bytes) {
  if (!bytes) return fail(ZERO_EINVAL, "bytes is NULL");
  *bytes = 0;
  if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim)
    return fail(ZERO_EINVAL, "%lld x %lld is out of range", (long long)rows, (long long)cols);
  if (rows && cols) *bytes = zsm::rms_norm_backward_workspace(rows, cols);
  return ZERO_OK;
}

zero_status zero_rms_norm_backward(const void* dy, int32_t dtype, int64_t rows, int64_t cols, int64_t ld_dy, const void* h,
                                   int64_t ld_h, const zero_mx8* h8, const void* weight, int32_t weight_dtype,
                                   const float* rstd, const void* dh, int64_t ld_dh, void* dx, int64_t ld_dx, void* dw,
                                   int32_t dw_dtype, void* workspace, int64_t workspace_bytes, void* stream) {
  zero_status st = check_dense("dy", dy, dtype, rows, cols, ld_dy);
  if (st != ZERO_OK) return st;
  if (h && h8) return fail(ZERO_EINVAL, "both h and h8 are given");
  if (h8) st = check_shape8("h8", h8, rows, cols);
  else st = check_dense("h", h, dtype, rows, cols, ld_h);
  if (st != ZERO_OK) return st;
  if ((st = check_vector("weight", weight, weight_dtype, cols)) != ZERO_OK) return st;
  if (cols && (st = check_vector("rstd", rstd, ZERO_DTYPE_F32, rows)) != ZERO_OK) return st;
  if ((st = check_optional("dh", dh, dtype, rows, cols, ld_dh)) != ZERO_OK) return st;
  if ((st = check_dense("dx", dx, dtype, rows, cols, ld_dx)) != ZERO_OK) return st;
  if ((st = check_vector("dw", dw, dw_dtype, cols)) != ZERO_OK) return st;
  if (cols == 0) return ZERO_OK;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) return zero_fill(dw, dw_dtype, 1, cols, cols, s);
  if ((st = check_workspace(workspace, workspace_bytes, zsm::rms_norm_backward_workspace(rows, cols))) != ZERO_OK) return st;
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  zsm::RmsNormBackwardArgs a = {};
  const bool one = rows == 1;
  a.dy = dy, a.type = dtype;
  a.rows = rows, a.cols = cols;
  a.ld_dy = one ? cols : ld_dy;
  a.h = h, a.ld_h = one ? cols : ld_h;
  if (h8) a.h8 = matrix8(*h8);
  a.weight = weight, a.w_type = weight_dtype, a.w_aligned = (reinterpret_cast<uintptr_t>(weight) & 15u) == 0;
  a.rstd = rstd;
  a.dh = dh, a.ld_dh = one ? cols : ld_dh;
  const int64_t size = elem_bytes(dtype);
  auto end = [&](const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) + size * ((rows - 1) * ld + cols); };
  a.dy_end = end(dy, a.ld_dy), a.h_end = end(h, a.ld_h), a.dh_end = end(dh, a.ld_dh);
  a.dx = dx, a.ld_dx = one ? cols : ld_dx;
  a.dw = dw, a.dw_type = dw_dtype;
  a.workspace = workspace;
  return launched(zsm::launch_rms_norm_backward(a, sms, s), "norm backward launch");
}

zero_status zero_embedding(const void* tokens, int32_t token_bytes, int64_t n, const void* table, int32_t dtype, int64_t vocab,
                           int64_t cols, int64_t ld, const zero_mx4* table4, double scale, void* out, int32_t out_dtype,
                           int64_t ld_out, void* stream) {
  zero_status st = check_tokens(tokens, token_bytes, n, vocab);
  if (st != ZERO_OK) return st;
  if (table && table4) return fail(ZERO_EINVAL, "both table and table4 are given");
  if (table4) {
    if ((st = check_mx4("table4", table4)) != ZERO_OK) return st;
    if (table4->rows != vocab || table4->cols != cols)
      return fail(ZERO_EINVAL, "table4 is not %lld x %lld", (long long)vocab, (long long)cols);
  } else if ((st = check_dense("table", table, dtype, vocab, cols, ld)) != ZERO_OK) {
    return st;
  }
  if ((st = check_scale(scale)) != ZERO_OK) return st;
  if ((st = check_dense("out", out, out_dtype, n, cols, ld_out)) != ZERO_OK) return st;
  if (n == 0 || cols == 0) return ZERO_OK;
  // (an MX4 table's codes, by which the launch knows it, may be null here)
  if (vocab == 0) return zero_fill(out, out_dtype, n, cols, ld_out, static_cast<cudaStream_t>(stream));
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  zsm::EmbeddingArgs a = {};
  a.tokens = tokens, a.token_bytes = token_bytes;
  a.n = n, a.vocab = vocab, a.cols = cols;
  a.table = table, a.type = dtype, a.ld = vocab > 1 ? ld : cols;
  if (table4) a.from = matrix(*table4);
  a.scale = (float)scale;
  a.out = out, a.out_type = out_dtype, a.ld_out = n > 1 ? ld_out : cols;
  return launched(zsm::launch_embedding(a, sms, static_cast<cudaStream_t>(stream)), "embedding launch");
}

zero_status zero_embedding_backward_workspace(int64_t n, int64_t vocab, int64_t cols, int64_t* bytes) {
  if (!bytes) return fail(ZERO_EINVAL, "bytes is NULL");
  *bytes = 0;
  if (n < 0 || vocab < 0 || cols < 0 || n > kMaxDim || vocab > kMaxDim || cols > kMaxDim)
    return fail(ZERO_EINVAL, "%lld tokens, %lld x %lld: out of range", (long long)n, (long long)vocab, (long long)cols);
  if (n && vocab && cols) *bytes = zsm::embedding_backward_workspace(n, cols);
  return ZERO_OK;
}

zero_status zero_embedding_backward(const void* dy, int32_t dtype, int64_t n, int64_t cols, int64_t ld_dy, const void* tokens,
                                    int32_t token_bytes, int64_t vocab, double scale, void* dtable, int32_t dtable_dtype,
                                    int64_t ld, int32_t accumulate, void* workspace, int64_t workspace_bytes, void* stream) {
  zero_status st = check_tokens(tokens, token_bytes, n, vocab);
  if (st != ZERO_OK) return st;
  if ((st = check_dense("dy", dy, dtype, n, cols, ld_dy)) != ZERO_OK) return st;
  if ((st = check_scale(scale)) != ZERO_OK) return st;
  if ((st = check_dense("dtable", dtable, dtable_dtype, vocab, cols, ld)) != ZERO_OK) return st;
  if (accumulate != 0 && accumulate != 1) return fail(ZERO_EINVAL, "accumulate %d: 0 or 1 is needed", accumulate);
  if (vocab == 0 || cols == 0) return ZERO_OK;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n == 0) return accumulate ? ZERO_OK : zero_fill(dtable, dtable_dtype, vocab, cols, ld, s);
  if ((st = check_workspace(workspace, workspace_bytes, zsm::embedding_backward_workspace(n, cols))) != ZERO_OK)
    return st;
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  zsm::EmbeddingBackwardArgs a = {};
  a.dy = dy, a.type = dtype;
  a.n = n, a.cols = cols, a.ld_dy = n > 1 ? ld_dy : cols;
  a.tokens = tokens, a.token_bytes = token_bytes;
  a.vocab = vocab, a.scale = (float)scale;
  a.dtable = dtable, a.dtable_type = dtable_dtype, a.ld = vocab > 1 ? ld : cols;
  a.accumulate = accumulate;
  a.workspace = workspace;
  return launched(zsm::launch_embedding_backward(a, sms, s), "embedding backward launch");
}

}  // extern "C"
