// C ABI of the operators beside the layer (include/epoch.h): argument checks
// and launches. Nothing here keeps state between calls.
#include <cmath>

#include "common.cuh"
#include "layer.h"

using namespace epoch;

namespace {

cudaStream_t S(epoch_stream s) { return reinterpret_cast<cudaStream_t>(s); }

bool dtype_ok(int32_t d) { return d == EPOCH_F32 || d == EPOCH_BF16; }
bool on(const void *p, size_t align) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (align - 1)) == 0; }
size_t size_of(int32_t d) { return d == EPOCH_BF16 ? 2 : 4; }
bool of_type(const void *p, int32_t d) { return on(p, size_of(d)); }
bool of_type_or_null(const void *p, int32_t d) { return p == nullptr || of_type(p, d); }
bool stride_ok(int64_t stride, int32_t n_rows, int64_t width) {
  return n_rows <= 1 || (stride >= width && stride <= (INT64_MAX >> 4) / n_rows);
}

// Bytes of an argument: `rows` runs of `width`, `stride` apart (none where the pointer is null).
struct Rows {
  const char *at;
  int64_t rows, width, stride;
  Rows(const void *p, int64_t n, int64_t w, int64_t s, size_t size)
      : at(static_cast<const char *>(p)), rows(p ? n : 0), width(w * static_cast<int64_t>(size)),
        stride(n > 1 ? s * static_cast<int64_t>(size) : width) {}
  Rows(const void *p, int64_t n, size_t size) : Rows(p, 1, n, n, size) {}
  const char *end() const { return at + (rows - 1) * stride + width; }
  // the other's bytes row by row, so its type too
  bool same(const Rows &o) const { return at == o.at && rows == o.rows && width == o.width && stride == o.stride; }
};
int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b != 0 && a < 0); }
// Whether two arguments share a byte: columns of one buffer side by side, or rows of it in turn, do not.
bool overlap(const Rows &a, const Rows &b) {
  if (a.rows == 0 || b.rows == 0 || a.end() <= b.at || b.end() <= a.at) return false;
  if (a.rows > b.rows) return overlap(b, a);
  const int64_t d = b.at - a.at;  // row j of b starts at d + j * b.stride from a's first
  auto meets = [&](int64_t start) {  // a's row there: rows j that end behind its start and start before its end
    const int64_t lo = floor_div(start - d - b.width, b.stride) + 1, hi = floor_div(start + a.width - d - 1, b.stride);
    return (lo > 0 ? lo : 0) <= (hi < b.rows - 1 ? hi : b.rows - 1);
  };
  // Equal strides: with as many rows or fewer, a row of a meets one of b where the first or the last one does.
  if (a.stride == b.stride) return meets(0) || meets((a.rows - 1) * a.stride);
  for (int64_t i = 0; i < a.rows; ++i)
    if (meets(i * a.stride)) return true;
  return false;
}

epoch_status status_of(cudaError_t e) { return e == cudaSuccess ? EPOCH_OK : EPOCH_ECUDA; }

constexpr int32_t kMaxHidden = 1 << 20;

// Checks the arguments of a product and puts them together (m > 0).
epoch_status product(const void *a, const float *a_scales, const void *b, const float *b_scales, const int32_t *offsets,
                     int32_t n_groups, int32_t m, int32_t n, int32_t k, void *y, int64_t y_stride, int32_t out_dtype,
                     GemmArgs *g) {
  if (m < 0 || n < 1 || k < 16 || k % 16 || k > (1 << 30) || n_groups < 1 || n_groups > 1024 || !dtype_ok(out_dtype))
    return EPOCH_EINVAL;
  if (offsets == nullptr ? n_groups != 1 : !on(offsets, 4)) return EPOCH_EINVAL;
  if (static_cast<int64_t>(n_groups) * n > INT32_MAX - 256 || m > INT32_MAX - 256) return EPOCH_EINVAL;
  if (m == 0) return EPOCH_OK;
  if (!on(a, 16) || !on(b, 16) || !on(a_scales, 4) || !on(b_scales, 4) || !of_type(y, out_dtype) ||
      !stride_ok(y_stride, m, n))
    return EPOCH_EINVAL;
  const int64_t kb = (k + 127) / 128, nb = (n + 127) / 128, rows = m;
  const Rows result(y, m, n, y_stride, size_of(out_dtype));
  if (overlap(result, Rows(a, rows * k, 1)) || overlap(result, Rows(a_scales, rows * kb, 4)) ||
      overlap(result, Rows(b, static_cast<int64_t>(n_groups) * n * k, 1)) ||
      overlap(result, Rows(b_scales, n_groups * nb * kb, 4)) || overlap(result, Rows(offsets, n_groups + 1, 4)))
    return EPOCH_EINVAL;
  *g = GemmArgs{};
  g->a = a;
  g->b = b;
  g->sa = a_scales;
  g->sb = b_scales;
  g->offsets = offsets;
  g->out = y;
  g->out_stride = y_stride;
  g->m = m;
  g->N = n;
  g->K = k;
  g->n_groups = n_groups;
  g->out_bf16 = out_dtype == EPOCH_BF16;
  return EPOCH_OK;
}

}  // namespace

extern "C" {

epoch_status epoch_norm_before(const void *x, int64_t x_stride, int32_t x_dtype, const void *weight, int32_t par_dtype,
                               int32_t n_rows, int32_t hidden, float eps, void *out, int64_t out_stride,
                               int32_t out_dtype, epoch_stream stream) {
  if (n_rows < 0 || hidden < 1 || hidden > kMaxHidden || !dtype_ok(x_dtype) || !dtype_ok(par_dtype) ||
      !dtype_ok(out_dtype) || !std::isfinite(eps) || eps < 0.f)
    return EPOCH_EINVAL;
  if (!of_type(weight, par_dtype)) return EPOCH_EINVAL;
  if (n_rows == 0) return EPOCH_OK;
  if (!of_type(x, x_dtype) || !of_type(out, out_dtype) || !stride_ok(x_stride, n_rows, hidden) ||
      !stride_ok(out_stride, n_rows, hidden))
    return EPOCH_EINVAL;
  const Rows in(x, n_rows, hidden, x_stride, size_of(x_dtype)), result(out, n_rows, hidden, out_stride, size_of(out_dtype));
  if ((overlap(result, in) && !result.same(in)) || overlap(result, Rows(weight, hidden, size_of(par_dtype))))
    return EPOCH_EINVAL;
  NormArgs a = {};
  a.residual = x;
  a.residual_stride = x_stride;
  a.weight = weight;
  a.out = out;
  a.out_stride = out_stride;
  a.n_rows = n_rows;
  a.hidden = hidden;
  a.act_bf16 = out_dtype == EPOCH_BF16;
  a.res_bf16 = x_dtype == EPOCH_BF16;
  a.par_bf16 = par_dtype == EPOCH_BF16;
  a.eps = eps;
  return status_of(launch_block_norm(a, false, S(stream)));
}

epoch_status epoch_norm_after(const epoch_norm_after_args *p, epoch_stream stream) {
  if (p == nullptr || p->n_rows < 0 || p->hidden < 1 || p->hidden > kMaxHidden || !dtype_ok(p->dtype) ||
      !dtype_ok(p->residual_dtype) || !dtype_ok(p->par_dtype) || !std::isfinite(p->eps) || p->eps < 0.f)
    return EPOCH_EINVAL;
  if (p->gate_kind < EPOCH_GATE_NONE || p->gate_kind > EPOCH_GATE_FULL) return EPOCH_EINVAL;
  if (!of_type_or_null(p->weight, p->par_dtype) || !of_type_or_null(p->scale, p->par_dtype) ||
      !of_type_or_null(p->next_weight, p->par_dtype))
    return EPOCH_EINVAL;
  if (p->gate_kind == EPOCH_GATE_CHANNEL && !of_type(p->gate, p->par_dtype)) return EPOCH_EINVAL;
  const int32_t n = p->n_rows, h = p->hidden;
  if (n == 0) return EPOCH_OK;
  if ((p->next_weight == nullptr) != (p->next_out == nullptr)) return EPOCH_EINVAL;
  if (!of_type(p->block, p->dtype) || !of_type(p->residual, p->residual_dtype) || !of_type(p->out, p->residual_dtype) ||
      !of_type_or_null(p->next_out, p->dtype))
    return EPOCH_EINVAL;
  if (p->gate_kind == EPOCH_GATE_FULL && (!of_type(p->gate, p->dtype) || !stride_ok(p->gate_stride, n, h)))
    return EPOCH_EINVAL;
  if (!stride_ok(p->block_stride, n, h) || !stride_ok(p->residual_stride, n, h) || !stride_ok(p->out_stride, n, h) ||
      (p->next_out != nullptr && !stride_ok(p->next_stride, n, h)))
    return EPOCH_EINVAL;
  // An output may be an input of its type and rows: a thread reads its elements of a row before it writes them.
  const size_t sa = size_of(p->dtype), sr = size_of(p->residual_dtype), sp = size_of(p->par_dtype);
  const bool full = p->gate_kind == EPOCH_GATE_FULL;
  const Rows block(p->block, n, h, p->block_stride, sa), residual(p->residual, n, h, p->residual_stride, sr);
  const Rows gate(full ? p->gate : nullptr, n, h, p->gate_stride, sa);
  const Rows outs[2] = {Rows(p->out, n, h, p->out_stride, sr), Rows(p->next_out, n, h, p->next_stride, sa)};
  const void *params[4] = {p->weight, p->scale, p->next_weight, p->gate_kind == EPOCH_GATE_CHANNEL ? p->gate : nullptr};
  if (overlap(outs[0], outs[1])) return EPOCH_EINVAL;
  for (const Rows &o : outs) {
    for (const Rows *in : {&block, &residual, &gate})
      if (overlap(o, *in) && !o.same(*in)) return EPOCH_EINVAL;
    for (const void *q : params)
      if (overlap(o, Rows(q, h, sp))) return EPOCH_EINVAL;
  }
  NormArgs a = {};
  a.block = p->block;
  a.residual = p->residual;
  a.weight = p->weight;
  a.gate = p->gate_kind == EPOCH_GATE_NONE ? nullptr : p->gate;
  a.scale = p->scale;
  a.next_weight = p->next_weight;
  a.out = p->out;
  a.next_out = p->next_out;
  a.block_stride = p->block_stride;
  a.residual_stride = p->residual_stride;
  a.gate_stride = p->gate_stride;
  a.out_stride = p->out_stride;
  a.next_stride = p->next_stride;
  a.n_rows = n;
  a.hidden = h;
  a.act_bf16 = p->dtype == EPOCH_BF16;
  a.res_bf16 = p->residual_dtype == EPOCH_BF16;
  a.par_bf16 = p->par_dtype == EPOCH_BF16;
  a.gate_kind = p->gate_kind;
  a.gate_sigmoid = p->gate_sigmoid ? 1 : 0;
  a.residual_scale = p->residual_scale;
  a.eps = p->eps;
  return status_of(launch_block_norm(a, true, S(stream)));
}

epoch_status epoch_fp8_quantize(const void *x, int64_t x_stride, int32_t dtype, const int32_t *rows, int32_t n_rows,
                                int32_t n_src, int32_t cols, int32_t swiglu, void *q, float *scales,
                                epoch_stream stream) {
  if (n_rows < 0 || n_src < 0 || cols < 1 || cols > (1 << 30) || !dtype_ok(dtype)) return EPOCH_EINVAL;
  if (n_rows == 0) return EPOCH_OK;
  if (rows == nullptr && n_src != n_rows) return EPOCH_EINVAL;
  const int64_t blocks = static_cast<int64_t>(n_rows) * ((cols + 127) / 128);
  if (blocks > INT32_MAX) return EPOCH_EINVAL;
  if ((n_src > 0 && !of_type(x, dtype)) || (rows != nullptr && !on(rows, 4)) || q == nullptr || !on(scales, 4) ||
      !stride_ok(x_stride, n_src, static_cast<int64_t>(cols) * (swiglu ? 2 : 1)))
    return EPOCH_EINVAL;
  const int64_t wide = static_cast<int64_t>(cols) * (swiglu ? 2 : 1);
  const Rows in(n_src ? x : nullptr, n_src, wide, x_stride, size_of(dtype)), index(rows, n_rows, 4);
  const Rows values(q, static_cast<int64_t>(n_rows) * cols, 1), factors(scales, blocks, 4);
  if (overlap(values, in) || overlap(factors, in) || overlap(values, index) || overlap(factors, index) ||
      overlap(values, factors))
    return EPOCH_EINVAL;
  QuantArgs a = {};
  a.x = x;
  a.rows = rows;
  a.q = static_cast<uint8_t *>(q);
  a.scales = scales;
  a.x_stride = x_stride;
  a.n_rows = n_rows;
  a.n_src = n_src;
  a.cols = cols;
  a.swiglu = swiglu ? 1 : 0;
  return status_of(launch_fp8_quant(a, dtype == EPOCH_BF16, S(stream)));
}

epoch_status epoch_fp8_quantize_weight(const void *w, int32_t dtype, int32_t n_mats, int32_t n, int32_t k, void *q,
                                       float *scales, epoch_stream stream) {
  if (!dtype_ok(dtype) || n_mats < 0 || n_mats > 65535 || n < 1 || n > (1 << 22) || k < 1 || k > (1 << 22))
    return EPOCH_EINVAL;
  if (n_mats == 0) return EPOCH_OK;
  if (!of_type(w, dtype) || q == nullptr || !on(scales, 4)) return EPOCH_EINVAL;
  const int64_t count = static_cast<int64_t>(n_mats) * n * k;
  const Rows in(w, count, size_of(dtype)), values(q, count, 1);
  const Rows factors(scales, static_cast<int64_t>(n_mats) * ((n + 127) / 128) * ((k + 127) / 128), 4);
  if (overlap(values, in) || overlap(factors, in) || overlap(values, factors)) return EPOCH_EINVAL;
  return status_of(launch_fp8_quant_weight(w, dtype == EPOCH_BF16, n_mats, n, k, static_cast<uint8_t *>(q), scales,
                                           S(stream)));
}

epoch_status epoch_fp8_matmul(const void *a, const float *a_scales, const void *b, const float *b_scales,
                              const int32_t *offsets, int32_t n_groups, int32_t m, int32_t n, int32_t k, void *y,
                              int64_t y_stride, int32_t out_dtype, epoch_stream stream) {
  GemmArgs g;
  const epoch_status st = product(a, a_scales, b, b_scales, offsets, n_groups, m, n, k, y, y_stride, out_dtype, &g);
  if (st != EPOCH_OK || m == 0) return st;
  return status_of(launch_fp8_gemm(g, S(stream)));
}

epoch_status epoch_test_fp8_timeout(const void *a, const float *a_scales, const void *b, const float *b_scales,
                                    const int32_t *offsets, int32_t n_groups, int32_t m, int32_t n, int32_t k, void *y,
                                    int64_t y_stride, int32_t out_dtype, int64_t timeout_ns, epoch_stream stream) {
  GemmArgs g;
  const epoch_status st = product(a, a_scales, b, b_scales, offsets, n_groups, m, n, k, y, y_stride, out_dtype, &g);
  if (st != EPOCH_OK) return st;
  if (timeout_ns < 1000 || timeout_ns > 5000000000ll || m == 0 ||
      fp8_gemm_kernel(offsets ? n_groups : 0, m, n, num_sms()) == 0)
    return EPOCH_EINVAL;
  return status_of(launch_fp8_gemm(g, S(stream), timeout_ns, 16));
}

int32_t epoch_fp8_matmul_kernel(int32_t n_groups, int32_t m, int32_t n, int32_t n_sms) {
  if (m < 0 || n < 1 || n_groups < 0 || n_groups > 1024 || n_sms < 0) return -1;
  return fp8_gemm_kernel(n_groups, m, n, n_sms ? n_sms : num_sms());
}

epoch_status epoch_ops_status(int32_t clear, epoch_stream stream, uint32_t *word_out) {
  uint32_t *at = ops_error_word();
  uint32_t word = 0;
  if (at == nullptr || cudaMemcpyAsync(&word, at, sizeof(word), cudaMemcpyDeviceToHost, S(stream)) != cudaSuccess ||
      cudaStreamSynchronize(S(stream)) != cudaSuccess)
    return EPOCH_ECUDA;
  if (clear && word && cudaMemsetAsync(at, 0, sizeof(word), S(stream)) != cudaSuccess) return EPOCH_ECUDA;
  if (word_out) *word_out = word;
  if (word & EPOCH_DEVERR_TIMEOUT) return EPOCH_ETIMEOUT;
  return word ? EPOCH_EDEVICE : EPOCH_OK;
}

}  // extern "C"
