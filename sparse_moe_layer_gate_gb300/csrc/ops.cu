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

// Bytes that no output may share: whether any two of them do, or one shares some with an input.
template <int N, int M> bool clash(const Rows (&outs)[N], const Rows (&ins)[M]) {
  for (int i = 0; i < N; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return true;
    for (const Rows &in : ins)
      if (overlap(outs[i], in)) return true;
  }
  return false;
}

bool fp4_format(int32_t f) { return f == EPOCH_FP4_NVFP4 || f == EPOCH_FP4_MXFP4; }
int64_t fp4_scale_bytes(int32_t format, int64_t rows, int64_t cols) {
  return (cols + 255) / 256 * rows * (format == EPOCH_FP4_NVFP4 ? 16 : 8);
}

// Checks the arguments of a product of experts and puts them together (m > 0).
epoch_status expert_product(const epoch_expert_args *p, ExpertGemmArgs *g) {
  if (p == nullptr || p->kind < EPOCH_EXPERT_F32 || p->kind > EPOCH_EXPERT_MXFP4 || !dtype_ok(p->out_dtype))
    return EPOCH_EINVAL;
  const bool fp4 = p->kind >= EPOCH_EXPERT_NVFP4;
  const int32_t unit = fp4 ? 32 : p->kind == EPOCH_EXPERT_BF16 ? 8 : 4;
  if (p->m < 0 || p->n < 1 || p->k < unit || p->k % unit || p->k > (1 << 30) || p->n_groups < 1 || p->n_groups > 1024 ||
      p->n_src < 0 || !std::isfinite(p->scale))
    return EPOCH_EINVAL;
  if ((p->swiglu && p->n % 2) || (fp4 && p->rows != nullptr) || (p->rows == nullptr && p->n_src != p->m))
    return EPOCH_EINVAL;
  if (p->offsets == nullptr ? p->n_groups != 1 : !on(p->offsets, 4)) return EPOCH_EINVAL;
  const int64_t weights = static_cast<int64_t>(p->n_groups) * p->n;
  if (weights > INT32_MAX - 256 || p->m > INT32_MAX - 256 || p->n_src > INT32_MAX - 256) return EPOCH_EINVAL;
  if (p->m == 0) return EPOCH_OK;
  const size_t in_size = p->kind == EPOCH_EXPERT_F32 ? 4 : 2;
  const int64_t out_n = p->swiglu ? p->n / 2 : p->n, k_row = fp4 ? p->k / 2 : p->k;
  if ((p->n_src > 0 && !on(p->a, 16)) || !on(p->b, 16) || !of_type(p->y, p->out_dtype) || !stride_ok(p->y_stride, p->m, out_n) ||
      (p->rows != nullptr && !on(p->rows, 4)) || (p->group_scale != nullptr && !on(p->group_scale, 4)))
    return EPOCH_EINVAL;
  if (fp4 && (!on(p->a_scales, 16) || !on(p->b_scales, 16))) return EPOCH_EINVAL;
  int64_t a_stride = k_row;
  if (!fp4 && p->n_src > 1) {
    a_stride = p->a_stride;
    if (!stride_ok(a_stride, p->n_src, p->k) || a_stride * static_cast<int64_t>(in_size) % 16 ||
        a_stride >= (1ll << 40) / static_cast<int64_t>(in_size))
      return EPOCH_EINVAL;
  }
  const int32_t format = p->kind == EPOCH_EXPERT_NVFP4 ? EPOCH_FP4_NVFP4 : EPOCH_FP4_MXFP4;
  const size_t size = fp4 ? 1 : in_size;
  const Rows outs[1] = {Rows(p->y, p->m, out_n, p->y_stride, size_of(p->out_dtype))};
  const Rows ins[7] = {Rows(p->n_src ? p->a : nullptr, p->n_src, k_row, a_stride, size),
                       Rows(p->b, weights * k_row, size),
                       Rows(p->offsets, p->n_groups + 1, 4),
                       Rows(p->rows, p->m, 4),
                       Rows(p->group_scale, p->n_groups, 4),
                       Rows(fp4 ? p->a_scales : nullptr, fp4_scale_bytes(format, p->m, p->k), 1),
                       Rows(fp4 ? p->b_scales : nullptr, fp4_scale_bytes(format, weights, p->k), 1)};
  if (clash(outs, ins)) return EPOCH_EINVAL;
  *g = ExpertGemmArgs{};
  g->a = p->a;
  g->b = p->b;
  g->sa = static_cast<const uint8_t *>(p->a_scales);
  g->sb = static_cast<const uint8_t *>(p->b_scales);
  g->offsets = p->offsets;
  g->rows = p->rows;
  g->group_scale = p->group_scale;
  g->out = p->y;
  g->a_stride = a_stride;
  g->out_stride = p->y_stride;
  g->scale = p->scale;
  g->m = p->m;
  g->n_src = p->n_src;
  g->N = p->n;
  g->K = p->k;
  g->n_groups = p->n_groups;
  g->kind = p->kind;
  g->swiglu = p->swiglu ? 1 : 0;
  g->out_bf16 = p->out_dtype == EPOCH_BF16;
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

size_t epoch_route_workspace_bytes(int32_t n_tok, int32_t n_experts) {
  if (n_tok < 1 || n_experts < 1 || n_experts > 1024) return 0;
  return router_workspace(n_tok, n_experts);
}

epoch_status epoch_route(const epoch_route_args *p, epoch_stream stream) {
  if (p == nullptr || p->n_tok < 0 || p->n_experts < 1 || p->n_experts > 1024 || p->top_k < 1 || p->top_k > 16 ||
      p->top_k > p->n_experts || !dtype_ok(p->dtype) ||
      (p->router != EPOCH_ROUTER_SOFTMAX && p->router != EPOCH_ROUTER_SIGMOID_GROUP))
    return EPOCH_EINVAL;
  const int64_t edges = static_cast<int64_t>(p->n_tok) * p->top_k;
  if (edges > INT32_MAX - 256) return EPOCH_EINVAL;
  const bool sigmoid = p->router == EPOCH_ROUTER_SIGMOID_GROUP;
  if (!sigmoid && p->bias != nullptr) return EPOCH_EINVAL;
  if (sigmoid && (p->n_group < 1 || p->n_group > 32 || p->n_experts % p->n_group || p->topk_group < 1 ||
                  p->topk_group > p->n_group || (p->bias != nullptr && !on(p->bias, 4))))
    return EPOCH_EINVAL;
  if (!on(p->offsets, 4)) return EPOCH_EINVAL;
  if (p->n_tok == 0) {  // an empty worklist
    return status_of(cudaMemsetAsync(p->offsets, 0, sizeof(int32_t) * (p->n_experts + 1), S(stream)));
  }
  if (!of_type(p->logits, p->dtype) || !stride_ok(p->logits_stride, p->n_tok, p->n_experts) || !on(p->sel, 4) ||
      !on(p->weights, 4) || !on(p->positions, 4) || !on(p->slots, 4))
    return EPOCH_EINVAL;
  const size_t need = router_workspace(p->n_tok, p->n_experts);
  if (need > 0 && (!on(p->workspace, 4) || p->workspace_bytes < need)) return EPOCH_EINVAL;
  const Rows outs[6] = {Rows(p->sel, edges, 4),   Rows(p->weights, edges, 4),
                        Rows(p->positions, edges, 4), Rows(p->slots, edges, 4),
                        Rows(p->offsets, p->n_experts + 1, 4), Rows(need ? p->workspace : nullptr, static_cast<int64_t>(need), 1)};
  const Rows ins[4] = {Rows(p->logits, p->n_tok, p->n_experts, p->logits_stride, size_of(p->dtype)),
                       Rows(p->bias, p->n_experts, 4), Rows(p->live, p->n_tok, 1), Rows(p->eligible, p->n_experts, 1)};
  if (clash(outs, ins)) return EPOCH_EINVAL;
  RouteArgs a = {};
  a.logits = p->logits;
  a.bias = p->bias;
  a.live = p->live;
  a.eligible = p->eligible;
  a.sel = p->sel;
  a.weights = p->weights;
  a.positions = p->positions;
  a.offsets = p->offsets;
  a.slots = p->slots;
  a.counts = static_cast<int32_t *>(p->workspace);
  a.logits_stride = p->logits_stride;
  a.n_tok = p->n_tok;
  a.n_experts = p->n_experts;
  a.top_k = p->top_k;
  a.bf16 = p->dtype == EPOCH_BF16;
  a.sigmoid = sigmoid;
  a.n_group = sigmoid ? p->n_group : 1;
  a.topk_group = sigmoid ? p->topk_group : 1;
  a.raw_weights = p->raw_weights ? 1 : 0;
  return status_of(launch_router(a, S(stream)));
}

epoch_status epoch_combine(const epoch_combine_args *p, epoch_stream stream) {
  if (p == nullptr || p->n_tok < 0 || p->n_edges < 0 || p->hidden < 1 || p->hidden > kMaxHidden || p->k < 1 || p->k > 64 ||
      !dtype_ok(p->dtype) || !dtype_ok(p->residual_dtype) || !dtype_ok(p->out_dtype))
    return EPOCH_EINVAL;
  const int64_t n = p->n_tok, h = p->hidden;
  if (n * h > (1ll << 38)) return EPOCH_EINVAL;
  if (n == 0) return EPOCH_OK;
  if ((p->n_edges > 0 && !of_type(p->edges, p->dtype)) || !of_type_or_null(p->shared, p->dtype) ||
      !of_type_or_null(p->residual, p->residual_dtype) || !of_type(p->out, p->out_dtype) || !on(p->slots, 4) || !on(p->weights, 4))
    return EPOCH_EINVAL;
  if (!stride_ok(p->edges_stride, p->n_edges, h) || (p->shared && !stride_ok(p->shared_stride, p->n_tok, h)) ||
      (p->residual && !stride_ok(p->residual_stride, p->n_tok, h)) || !stride_ok(p->out_stride, p->n_tok, h))
    return EPOCH_EINVAL;
  const size_t sd = size_of(p->dtype), sr = size_of(p->residual_dtype);
  const Rows out(p->out, n, h, p->out_stride, size_of(p->out_dtype));
  const Rows outs[1] = {out};
  const Rows ins[3] = {Rows(p->n_edges ? p->edges : nullptr, p->n_edges, h, p->edges_stride, sd), Rows(p->slots, n * p->k, 4),
                       Rows(p->weights, n * p->k, 4)};
  if (clash(outs, ins)) return EPOCH_EINVAL;
  // A thread reads its elements of these before it writes them.
  for (const Rows &in : {Rows(p->shared, n, h, p->shared_stride, sd), Rows(p->residual, n, h, p->residual_stride, sr)})
    if (overlap(out, in) && !out.same(in)) return EPOCH_EINVAL;
  CombineArgs a = {};
  a.edges = p->edges;
  a.shared = p->shared;
  a.residual = p->residual;
  a.slots = p->slots;
  a.weights = p->weights;
  a.out = p->out;
  a.edges_stride = p->edges_stride;
  a.shared_stride = p->shared_stride;
  a.residual_stride = p->residual_stride;
  a.out_stride = p->out_stride;
  a.n_tok = n;
  a.n_edges = p->n_edges;
  a.hidden = p->hidden;
  a.k = p->k;
  a.residual_bf16 = p->residual_dtype == EPOCH_BF16;
  a.out_bf16 = p->out_dtype == EPOCH_BF16;
  return status_of(launch_combine_edges(a, p->dtype == EPOCH_BF16, S(stream)));
}

epoch_status epoch_fp4_quantize(const void *x, int64_t x_stride, int32_t dtype, const int32_t *rows, int32_t n_rows,
                                int32_t n_src, int32_t cols, int32_t swiglu, int32_t format, float tensor_scale, void *q,
                                void *scales, epoch_stream stream) {
  if (n_rows < 0 || n_src < 0 || cols < 32 || cols % 32 || cols > (1 << 30) || !dtype_ok(dtype) || !fp4_format(format))
    return EPOCH_EINVAL;
  const float inv = 1.0f / tensor_scale;
  if (!(tensor_scale > 0.f) || !std::isfinite(tensor_scale) || !std::isfinite(inv) || inv == 0.f ||
      (format == EPOCH_FP4_MXFP4 && tensor_scale != 1.0f))
    return EPOCH_EINVAL;
  if (n_rows == 0) return EPOCH_OK;
  if (rows == nullptr && n_src != n_rows) return EPOCH_EINVAL;
  if (static_cast<int64_t>(n_rows) * ((cols + 255) / 256) > INT32_MAX) return EPOCH_EINVAL;
  const int64_t wide = static_cast<int64_t>(cols) * (swiglu ? 2 : 1);
  if ((n_src > 0 && !of_type(x, dtype)) || (rows != nullptr && !on(rows, 4)) || !on(q, 16) || !on(scales, 16) ||
      !stride_ok(x_stride, n_src, wide))
    return EPOCH_EINVAL;
  const Rows outs[2] = {Rows(q, static_cast<int64_t>(n_rows) * cols / 2, 1), Rows(scales, fp4_scale_bytes(format, n_rows, cols), 1)};
  const Rows ins[2] = {Rows(n_src ? x : nullptr, n_src, wide, x_stride, size_of(dtype)), Rows(rows, n_rows, 4)};
  if (clash(outs, ins)) return EPOCH_EINVAL;
  Fp4QuantArgs a = {};
  a.x = x;
  a.rows = rows;
  a.q = static_cast<uint8_t *>(q);
  a.scales = static_cast<uint8_t *>(scales);
  a.x_stride = x_stride;
  a.n_rows = n_rows;
  a.n_src = n_src;
  a.cols = cols;
  a.swiglu = swiglu ? 1 : 0;
  a.inv_scale = inv;
  return status_of(launch_fp4_quant(a, dtype == EPOCH_BF16, format == EPOCH_FP4_NVFP4, S(stream)));
}

epoch_status epoch_fp4_quantize_weight(const void *w, int32_t dtype, int32_t n_mats, int32_t n, int32_t k, int32_t format,
                                       void *q, void *scales, float *tensor_scales, epoch_stream stream) {
  if (!dtype_ok(dtype) || !fp4_format(format) || n_mats < 0 || n_mats > 65535 || n < 1 || n > (1 << 22) || k < 32 || k % 32 ||
      k > (1 << 22))
    return EPOCH_EINVAL;
  if (n_mats == 0) return EPOCH_OK;
  const int64_t rows = static_cast<int64_t>(n_mats) * n;
  if (rows * ((k + 255) / 256) > INT32_MAX) return EPOCH_EINVAL;
  if (!of_type(w, dtype) || !on(q, 16) || !on(scales, 16) || !on(tensor_scales, 4)) return EPOCH_EINVAL;
  const Rows outs[3] = {Rows(q, rows * k / 2, 1), Rows(scales, fp4_scale_bytes(format, rows, k), 1), Rows(tensor_scales, n_mats, 4)};
  const Rows ins[1] = {Rows(w, rows * k, size_of(dtype))};
  if (clash(outs, ins)) return EPOCH_EINVAL;
  Fp4QuantArgs a = {};
  a.x = w;
  a.q = static_cast<uint8_t *>(q);
  a.scales = static_cast<uint8_t *>(scales);
  a.x_stride = k;
  a.n_rows = a.n_src = rows;
  a.mat_rows = n;
  a.cols = k;
  a.inv_scale = 1.0f;
  return status_of(launch_fp4_quant_weight(a, n_mats, dtype == EPOCH_BF16, format == EPOCH_FP4_NVFP4, tensor_scales, S(stream)));
}

epoch_status epoch_fp4_dequantize(const void *q, const void *scales, int32_t format, int32_t n_mats, int32_t n, int32_t k,
                                  float scale, const float *group_scale, void *out, int64_t out_stride, int32_t out_dtype,
                                  epoch_stream stream) {
  if (!dtype_ok(out_dtype) || !fp4_format(format) || n_mats < 0 || n < 0 || k < 32 || k % 32 || k > (1 << 30) || !std::isfinite(scale))
    return EPOCH_EINVAL;
  const int64_t rows = static_cast<int64_t>(n_mats) * n;
  if (rows == 0) return EPOCH_OK;
  if (rows > INT32_MAX || rows * ((k + 255) / 256) > INT32_MAX) return EPOCH_EINVAL;
  if (!on(q, 16) || !on(scales, 16) || (group_scale != nullptr && !on(group_scale, 4)) || !of_type(out, out_dtype) ||
      !stride_ok(out_stride, static_cast<int32_t>(rows), k))
    return EPOCH_EINVAL;
  const Rows outs[1] = {Rows(out, rows, k, out_stride, size_of(out_dtype))};
  const Rows ins[3] = {Rows(q, rows * k / 2, 1), Rows(scales, fp4_scale_bytes(format, rows, k), 1), Rows(group_scale, n_mats, 4)};
  if (clash(outs, ins)) return EPOCH_EINVAL;
  Fp4DequantArgs a = {};
  a.q = static_cast<const uint8_t *>(q);
  a.scales = static_cast<const uint8_t *>(scales);
  a.group_scale = group_scale;
  a.out = out;
  a.n_rows = rows;
  a.mat_rows = n;
  a.out_stride = out_stride;
  a.cols = k;
  a.scale = scale;
  return status_of(launch_fp4_dequant(a, out_dtype == EPOCH_BF16, format == EPOCH_FP4_NVFP4, S(stream)));
}

epoch_status epoch_expert_matmul(const epoch_expert_args *p, epoch_stream stream) {
  ExpertGemmArgs g;
  const epoch_status st = expert_product(p, &g);
  if (st != EPOCH_OK || p->m == 0) return st;
  if (g.kind == EPOCH_EXPERT_F32) return status_of(launch_expert_simt(g, S(stream)));
  const bool few = expert_few(g.kind != EPOCH_EXPERT_BF16, g.offsets ? g.n_groups : 0, g.m, g.N, num_sms());
  return status_of(few ? launch_expert_few(g, S(stream)) : launch_expert_gemm(g, S(stream)));
}

epoch_status epoch_test_expert_timeout(const epoch_expert_args *p, int64_t timeout_ns, epoch_stream stream) {
  ExpertGemmArgs g;
  const epoch_status st = expert_product(p, &g);
  if (st != EPOCH_OK) return st;
  if (timeout_ns < 1000 || timeout_ns > 5000000000ll || p->m == 0 || g.kind == EPOCH_EXPERT_F32) return EPOCH_EINVAL;
  return status_of(launch_expert_gemm(g, S(stream), timeout_ns, 16));
}

int32_t epoch_expert_matmul_kernel(int32_t kind, int32_t n_groups, int32_t m, int32_t n, int32_t k, int32_t n_sms) {
  if (kind < EPOCH_EXPERT_F32 || kind > EPOCH_EXPERT_MXFP4 || m < 0 || n < 1 || k < 1 || n_groups < 0 || n_groups > 1024 || n_sms < 0)
    return -1;
  const int sms = n_sms ? n_sms : num_sms();
  const bool fp4 = kind != EPOCH_EXPERT_BF16;
  return kind == EPOCH_EXPERT_F32 || expert_few(fp4, n_groups, m, n, sms) ? 0 : expert_gemm_kernel(fp4, n_groups, m, n, sms);
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
