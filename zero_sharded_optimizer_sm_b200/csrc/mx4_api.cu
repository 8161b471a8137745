// Entry points of the MX4 operators that need no context (zero_mx4_*):
// argument checks and launches.  The collectives' are in zero_api.cu.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "../../include/zero_sm.h"
#include "mx4.cuh"
#include "mx4_errors.hpp"

static_assert(ZERO_DTYPE_BF16 == zsm::kMxBf16 && ZERO_DTYPE_F16 == zsm::kMxF16 && ZERO_DTYPE_F32 == zsm::kMxF32,
              "element types");
static_assert(ZERO_MX4_BLOCK == zsm::kMxBlock, "block length");

namespace {

zero_status fail(zero_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  zsm::set_thread_error(buf);
  return s;
}

zero_status cuda_fail(cudaError_t e, const char* what) {
  return fail(ZERO_ECUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

constexpr int64_t kMaxDim = 0x7FFFFFFF - 255;  // row and column numbers of a tile stay in 32 bits

int elem_bytes(int32_t dtype) { return dtype == ZERO_DTYPE_F32 ? 4 : 2; }

zero_status check_dtype(int32_t dtype) {
  if (dtype != ZERO_DTYPE_BF16 && dtype != ZERO_DTYPE_F16 && dtype != ZERO_DTYPE_F32)
    return fail(ZERO_EINVAL, "unknown dtype %d", dtype);
  return ZERO_OK;
}

zero_status check_dense(const char* name, const void* p, int32_t dtype, int64_t rows, int64_t cols, int64_t ld) {
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

zero_status check_mx4(const char* name, const zero_mx4* m) {
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

zsm::MxMatrix matrix(const zero_mx4& m) {
  return {static_cast<uint8_t*>(m.codes), static_cast<uint8_t*>(m.scales), m.rows, m.cols, m.code_pitch, m.scale_pitch};
}

// SMs of the current device, asked for once per device.
cudaError_t sm_count(int* n) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (*n = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && dev < 64) known[dev].store(*n, std::memory_order_relaxed);
  return e;
}

zero_status check_rounding(int32_t rounding) {
  if (rounding != ZERO_MX4_NEAREST && rounding != ZERO_MX4_STOCHASTIC)
    return fail(ZERO_EINVAL, "unknown rounding %d", rounding);
  return ZERO_OK;
}

zero_status check_workspace(const void* workspace, int64_t have, int64_t need) {
  if (need > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u) || have < need))
    return fail(ZERO_EINVAL, "the workspace must be 16-byte aligned and of at least %lld bytes (%lld given)",
                (long long)need, (long long)have);
  return ZERO_OK;
}

int64_t align16(int64_t n) { return (n + 15) / 16 * 16; }

zero_status matmul(const zero_mx4& a, const zero_mx4& b, void* out, int32_t dtype, int64_t ld, void* workspace, int pdl,
                   int b_ready, int sms, cudaStream_t s) {
  zsm::MxMatmulArgs m = {};
  m.a = matrix(a);
  m.b = matrix(b);
  m.out = out;
  m.type = dtype;
  m.ld = a.rows == 1 ? std::max<int64_t>(ld, b.rows) : ld;
  m.workspace = workspace;
  m.pdl = pdl;
  m.b_ready = b_ready;
  const cudaError_t e = zsm::launch_mx_matmul(m, sms, s);
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "MX4 product launch");
}

// zero_mx4_linear's workspace: x's codes, its scales (rows of 16-byte
// multiples) unless the rows are few, then the product's own part.
zero_mx4 quantised_x(uint8_t* at, int64_t tokens, int64_t inputs) {
  const int64_t nb = zsm::mx_blocks(inputs);
  return {at, at ? at + tokens * 16 * nb : nullptr, tokens, inputs, 16 * nb, align16(nb)};
}
int64_t linear_own(int64_t tokens, int64_t inputs) {
  const int64_t nb = zsm::mx_blocks(inputs);
  return tokens * (16 * nb + align16(nb));
}
int64_t linear_need(int64_t tokens, const zero_mx4* w) {
  if (tokens <= zsm::kMxFewRows) return zsm::mx_few_rows_workspace(matrix(*w));  // x is quantised in the product
  return linear_own(tokens, w->cols) + zsm::mx_matmul_workspace(matrix(quantised_x(nullptr, tokens, w->cols)), matrix(*w));
}

// zero_mx4_linear_backward's workspace: dy, its transpose and x's and w's, each
// with rows of scales of 16-byte multiples.
struct Backward {
  zero_mx4 dy, dy_t, x_t, w_t;
  int64_t bytes;
};
Backward backward_parts(uint8_t* at, int64_t tokens, int64_t o, int64_t k) {
  Backward p;
  int64_t used = 0;
  auto part = [&](int64_t rows, int64_t cols) {
    const zero_mx4 m = quantised_x(at ? at + used : nullptr, rows, cols);
    used += linear_own(rows, cols);
    return m;
  };
  p.dy = part(tokens, o);
  p.dy_t = part(o, tokens);
  p.x_t = part(k, tokens);
  p.w_t = part(k, o);
  p.bytes = used;
  return p;
}

// A product over no elements: zeros.
zero_status zero_fill(void* out, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, cudaStream_t s) {
  const int es = elem_bytes(dtype);
  const cudaError_t e = cudaMemset2DAsync(out, (size_t)(rows > 1 ? ld : cols) * es, 0, (size_t)cols * es, (size_t)rows, s);
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "clearing the product");
}

}  // namespace

extern "C" {

zero_status zero_mx4_quantize(const void* src, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, int32_t rounding,
                              uint64_t seed, const zero_mx4* out, const zero_mx4* out_t, void* stream) {
  zero_status st = check_dense("src", src, dtype, rows, cols, ld);
  if (st != ZERO_OK) return st;
  if ((st = check_rounding(rounding)) != ZERO_OK) return st;
  if (!out && !out_t) return fail(ZERO_EINVAL, "neither out nor out_t is given");
  if (out && (st = check_mx4("out", out)) != ZERO_OK) return st;
  if (out_t && (st = check_mx4("out_t", out_t)) != ZERO_OK) return st;
  if (out && (out->rows != rows || out->cols != cols))
    return fail(ZERO_EINVAL, "out is not %lld x %lld", (long long)rows, (long long)cols);
  if (out_t && (out_t->rows != cols || out_t->cols != rows))
    return fail(ZERO_EINVAL, "out_t is not %lld x %lld", (long long)cols, (long long)rows);
  if (rows == 0 || cols == 0) return ZERO_OK;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  zsm::MxQuantArgs a = {};
  a.src = src;
  a.type = dtype;
  a.rows = rows, a.cols = cols, a.ld = rows > 1 ? ld : cols;
  if (out) a.out = matrix(*out);
  if (out_t) a.out_t = matrix(*out_t);
  a.stochastic = rounding == ZERO_MX4_STOCHASTIC;
  a.seed = seed;
  e = zsm::launch_mx_quantize(a, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "MX4 quantise launch");
}

zero_status zero_mx4_transpose(const zero_mx4* in, int32_t rounding, uint64_t seed, const zero_mx4* out, void* stream) {
  zero_status st = check_mx4("in", in);
  if (st != ZERO_OK) return st;
  if ((st = check_mx4("out", out)) != ZERO_OK) return st;
  if ((st = check_rounding(rounding)) != ZERO_OK) return st;
  if (out->rows != in->cols || out->cols != in->rows)
    return fail(ZERO_EINVAL, "out is not %lld x %lld", (long long)in->cols, (long long)in->rows);
  if (in->rows == 0 || in->cols == 0) return ZERO_OK;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  zsm::MxQuantArgs a = {};
  a.from = matrix(*in);
  a.rows = in->rows, a.cols = in->cols;
  a.out_t = matrix(*out);
  a.stochastic = rounding == ZERO_MX4_STOCHASTIC;
  a.seed = seed;
  e = zsm::launch_mx_quantize(a, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "MX4 transpose launch");
}

zero_status zero_mx4_dequantize(const zero_mx4* in, void* dst, int32_t dtype, int64_t ld, void* stream) {
  zero_status st = check_mx4("in", in);
  if (st != ZERO_OK) return st;
  if ((st = check_dense("dst", dst, dtype, in->rows, in->cols, ld)) != ZERO_OK) return st;
  if (in->rows == 0 || in->cols == 0) return ZERO_OK;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  zsm::MxDequantArgs a = {matrix(*in), dst, dtype, in->rows > 1 ? ld : in->cols};
  e = zsm::launch_mx_dequantize(a, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "MX4 read-back launch");
}

zero_status zero_mx4_matmul_workspace(const zero_mx4* a, const zero_mx4* b, int64_t* bytes) {
  if (!bytes) return fail(ZERO_EINVAL, "bytes is NULL");
  *bytes = 0;
  zero_status st = check_mx4("a", a);
  if (st != ZERO_OK) return st;
  if ((st = check_mx4("b", b)) != ZERO_OK) return st;
  if (a->rows && b->rows && a->cols) *bytes = zsm::mx_matmul_workspace(matrix(*a), matrix(*b));
  return ZERO_OK;
}

zero_status zero_mx4_matmul(const zero_mx4* a, const zero_mx4* b, void* out, int32_t dtype, int64_t ld, void* workspace,
                            int64_t workspace_bytes, void* stream) {
  zero_status st = check_mx4("a", a);
  if (st != ZERO_OK) return st;
  if ((st = check_mx4("b", b)) != ZERO_OK) return st;
  if (a->cols != b->cols)
    return fail(ZERO_EINVAL, "a has %lld columns, b %lld", (long long)a->cols, (long long)b->cols);
  if ((st = check_dense("out", out, dtype, a->rows, b->rows, ld)) != ZERO_OK) return st;
  if (a->rows == 0 || b->rows == 0) return ZERO_OK;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->cols == 0) return zero_fill(out, dtype, a->rows, b->rows, ld, s);
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  const int64_t need = zsm::mx_matmul_workspace(matrix(*a), matrix(*b));
  if ((st = check_workspace(workspace, workspace_bytes, need)) != ZERO_OK) return st;
  return matmul(*a, *b, out, dtype, ld, workspace, 0, 0, sms, s);
}

zero_status zero_mx4_linear_workspace(int64_t tokens, const zero_mx4* w, int64_t* bytes) {
  if (!bytes) return fail(ZERO_EINVAL, "bytes is NULL");
  *bytes = 0;
  const zero_status st = check_mx4("w", w);
  if (st != ZERO_OK) return st;
  if (tokens < 0 || tokens > kMaxDim) return fail(ZERO_EINVAL, "%lld tokens", (long long)tokens);
  if (tokens && w->rows && w->cols) {
    *bytes = linear_need(tokens, w);
  }
  return ZERO_OK;
}

zero_status zero_mx4_linear(const void* x, int32_t dtype, int64_t tokens, int64_t ld, const zero_mx4* w, void* y,
                            int32_t y_dtype, int64_t ld_y, void* workspace, int64_t workspace_bytes, void* stream) {
  zero_status st = check_mx4("w", w);
  if (st != ZERO_OK) return st;
  if ((st = check_dense("x", x, dtype, tokens, w->cols, ld)) != ZERO_OK) return st;
  if ((st = check_dense("y", y, y_dtype, tokens, w->rows, ld_y)) != ZERO_OK) return st;
  if (tokens == 0 || w->rows == 0) return ZERO_OK;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (w->cols == 0) return zero_fill(y, y_dtype, tokens, w->rows, ld_y, s);
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  const int64_t own = linear_own(tokens, w->cols);
  uint8_t* at = static_cast<uint8_t*>(workspace);
  zero_mx4 xq = quantised_x(at, tokens, w->cols);
  st = check_workspace(workspace, workspace_bytes, linear_need(tokens, w));
  if (st != ZERO_OK) return st;
  if (tokens <= zsm::kMxFewRows) {
    zsm::MxMatmulArgs m = {};
    m.a = matrix(xq);
    m.b = matrix(*w);
    m.out = y, m.type = y_dtype;
    m.ld = tokens == 1 ? std::max<int64_t>(ld_y, w->rows) : ld_y;
    m.workspace = at;
    m.x = x, m.x_type = dtype;
    m.x_ld = tokens == 1 ? w->cols : ld;
    const cudaError_t er = zsm::launch_mx_matmul(m, sms, s);
    return er == cudaSuccess ? ZERO_OK : cuda_fail(er, "MX4 product launch");
  }
  // one launch quantises x and, where they are needed, writes w's scale pieces
  zsm::MxQuantArgs q = {};
  q.src = x, q.type = dtype;
  q.rows = tokens, q.cols = w->cols, q.ld = ld;
  q.out = matrix(xq);
  if (!zsm::mx_linear_pieces(matrix(*w), at + own, &q.pieces)) return cuda_fail(cudaErrorInvalidValue, "MX4 scale pieces");
  const cudaError_t er = zsm::launch_mx_quantize(q, sms, s);
  if (er != cudaSuccess) return cuda_fail(er, "MX4 quantise launch");
  return matmul(xq, *w, y, y_dtype, ld_y, at + own, 1, 1, sms, s);
}

zero_status zero_mx4_linear_backward_workspace(int64_t tokens, const zero_mx4* w, int64_t* bytes) {
  if (!bytes) return fail(ZERO_EINVAL, "bytes is NULL");
  *bytes = 0;
  const zero_status st = check_mx4("w", w);
  if (st != ZERO_OK) return st;
  if (tokens < 0 || tokens > kMaxDim) return fail(ZERO_EINVAL, "%lld tokens", (long long)tokens);
  if (tokens && w->rows && w->cols) *bytes = backward_parts(nullptr, tokens, w->rows, w->cols).bytes;
  return ZERO_OK;
}

zero_status zero_mx4_linear_backward(const void* dy, int32_t dy_dtype, int64_t ld_dy, const void* x, int32_t x_dtype,
                                     int64_t ld_x, int64_t tokens, const zero_mx4* w, int32_t rounding, uint64_t seed,
                                     void* dx, int32_t dx_dtype, int64_t ld_dx, void* dw, int32_t dw_dtype, int64_t ld_dw,
                                     void* workspace, int64_t workspace_bytes, void* stream) {
  zero_status st = check_mx4("w", w);
  if (st != ZERO_OK) return st;
  const int64_t o = w->rows, k = w->cols;
  if ((st = check_dense("dy", dy, dy_dtype, tokens, o, ld_dy)) != ZERO_OK) return st;
  if ((st = check_dense("x", x, x_dtype, tokens, k, ld_x)) != ZERO_OK) return st;
  if ((st = check_rounding(rounding)) != ZERO_OK) return st;
  if ((st = check_dense("dx", dx, dx_dtype, tokens, k, ld_dx)) != ZERO_OK) return st;
  if ((st = check_dense("dw", dw, dw_dtype, o, k, ld_dw)) != ZERO_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (k == 0) return ZERO_OK;
  if (tokens == 0) return o ? zero_fill(dw, dw_dtype, o, k, ld_dw, s) : ZERO_OK;
  if (o == 0) return zero_fill(dx, dx_dtype, tokens, k, ld_dx, s);
  const Backward p = backward_parts(static_cast<uint8_t*>(workspace), tokens, o, k);
  if ((st = check_workspace(workspace, workspace_bytes, p.bytes)) != ZERO_OK) return st;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  zsm::MxBackwardArgs a = {};
  a.dy.src = dy, a.dy.type = dy_dtype;
  a.dy.rows = tokens, a.dy.cols = o, a.dy.ld = tokens > 1 ? ld_dy : o;
  a.dy.out = matrix(p.dy), a.dy.out_t = matrix(p.dy_t);
  a.dy.stochastic = rounding == ZERO_MX4_STOCHASTIC, a.dy.seed = seed;
  a.x.src = x, a.x.type = x_dtype;
  a.x.rows = tokens, a.x.cols = k, a.x.ld = tokens > 1 ? ld_x : k;
  a.x.out_t = matrix(p.x_t);
  a.w.from = matrix(*w);
  a.w.rows = o, a.w.cols = k;
  a.w.out_t = matrix(p.w_t);
  e = zsm::launch_mx_backward(a, sms, s);
  if (e != cudaSuccess) return cuda_fail(e, "MX4 backward quantise launch");
  if ((st = matmul(p.dy, p.w_t, dx, dx_dtype, ld_dx, nullptr, 1, 0, sms, s)) != ZERO_OK) return st;
  return matmul(p.dy_t, p.x_t, dw, dw_dtype, ld_dw, nullptr, 1, 0, sms, s);
}

zero_status zero_mx4_check(void* stream) {
  unsigned count = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = zsm::mx_matmul_errors(&count, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "reading the MX4 products' error count");
  if (!zsm::mx_errors_are_news(dev, count)) return ZERO_OK;
  return fail(ZERO_ECUDA, "a bounded wait in an MX4 product kernel ran out: the product's result is invalid");
}

}  // extern "C"
