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
epoch_status status_of(cudaError_t e) { return e == cudaSuccess ? EPOCH_OK : EPOCH_ECUDA; }

constexpr int32_t kMaxHidden = 1 << 20;

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

epoch_status epoch_norm_after(const void *block, int64_t block_stride, int32_t dtype, const void *residual,
                              int64_t residual_stride, int32_t residual_dtype, const void *weight, const void *gate,
                              int64_t gate_stride, int32_t gate_kind, int32_t gate_sigmoid, const void *scale,
                              float residual_scale, const void *next_weight, int32_t par_dtype, int32_t n_rows,
                              int32_t hidden, float eps, void *out, int64_t out_stride, void *next_out,
                              int64_t next_stride, epoch_stream stream) {
  if (n_rows < 0 || hidden < 1 || hidden > kMaxHidden || !dtype_ok(dtype) || !dtype_ok(residual_dtype) ||
      !dtype_ok(par_dtype) || !std::isfinite(eps) || eps < 0.f)
    return EPOCH_EINVAL;
  if (gate_kind < EPOCH_GATE_NONE || gate_kind > EPOCH_GATE_FULL) return EPOCH_EINVAL;
  if (!of_type_or_null(weight, par_dtype) || !of_type_or_null(scale, par_dtype) ||
      !of_type_or_null(next_weight, par_dtype))
    return EPOCH_EINVAL;
  if (gate_kind == EPOCH_GATE_CHANNEL && !of_type(gate, par_dtype)) return EPOCH_EINVAL;
  if (n_rows == 0) return EPOCH_OK;
  if ((next_weight == nullptr) != (next_out == nullptr)) return EPOCH_EINVAL;
  if (!of_type(block, dtype) || !of_type(residual, residual_dtype) || !of_type(out, residual_dtype) ||
      !of_type_or_null(next_out, dtype))
    return EPOCH_EINVAL;
  if (gate_kind == EPOCH_GATE_FULL && (!of_type(gate, dtype) || !stride_ok(gate_stride, n_rows, hidden)))
    return EPOCH_EINVAL;
  if (!stride_ok(block_stride, n_rows, hidden) || !stride_ok(residual_stride, n_rows, hidden) ||
      !stride_ok(out_stride, n_rows, hidden) || (next_out != nullptr && !stride_ok(next_stride, n_rows, hidden)))
    return EPOCH_EINVAL;
  NormArgs a = {};
  a.block = block;
  a.residual = residual;
  a.weight = weight;
  a.gate = gate_kind == EPOCH_GATE_NONE ? nullptr : gate;
  a.scale = scale;
  a.next_weight = next_weight;
  a.out = out;
  a.next_out = next_out;
  a.block_stride = block_stride;
  a.residual_stride = residual_stride;
  a.gate_stride = gate_stride;
  a.out_stride = out_stride;
  a.next_stride = next_stride;
  a.n_rows = n_rows;
  a.hidden = hidden;
  a.act_bf16 = dtype == EPOCH_BF16;
  a.res_bf16 = residual_dtype == EPOCH_BF16;
  a.par_bf16 = par_dtype == EPOCH_BF16;
  a.gate_kind = gate_kind;
  a.gate_sigmoid = gate_sigmoid ? 1 : 0;
  a.residual_scale = residual_scale;
  a.eps = eps;
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
  return status_of(launch_fp8_quant_weight(w, dtype == EPOCH_BF16, n_mats, n, k, static_cast<uint8_t *>(q), scales,
                                           S(stream)));
}

epoch_status epoch_fp8_matmul(const void *a, const float *a_scales, const void *b, const float *b_scales,
                              const int32_t *offsets, int32_t n_groups, int32_t m, int32_t n, int32_t k, void *y,
                              int64_t y_stride, int32_t out_dtype, epoch_stream stream) {
  if (m < 0 || n < 1 || k < 16 || k % 16 || n_groups < 1 || n_groups > 1024 || !dtype_ok(out_dtype))
    return EPOCH_EINVAL;
  if (offsets == nullptr ? n_groups != 1 : !on(offsets, 4)) return EPOCH_EINVAL;
  if (static_cast<int64_t>(n_groups) * n > INT32_MAX - 256 || m > INT32_MAX - 256) return EPOCH_EINVAL;
  if (m == 0) return EPOCH_OK;
  if (!on(a, 16) || !on(b, 16) || !on(a_scales, 4) || !on(b_scales, 4) || !of_type(y, out_dtype) ||
      !stride_ok(y_stride, m, n))
    return EPOCH_EINVAL;
  GemmArgs g = {};
  g.a = a;
  g.b = b;
  g.sa = a_scales;
  g.sb = b_scales;
  g.offsets = offsets;
  g.out = y;
  g.out_stride = y_stride;
  g.m = m;
  g.N = n;
  g.K = k;
  g.n_groups = n_groups;
  g.out_bf16 = out_dtype == EPOCH_BF16;
  return status_of(launch_fp8_gemm(g, S(stream)));
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
