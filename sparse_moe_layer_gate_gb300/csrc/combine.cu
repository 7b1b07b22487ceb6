// The weighted sum of each position's edges, with the shared experts' output and the residual stream:
//
//   y[t] = sum_j weights[t, j] * edges[slots[t, j]] (+ shared[t]) (+ residual[t])
//
// in fp32, j ascending, rounded once. A negative slot adds nothing (a position that was routed to fewer
// experts); one past the last edge makes the row NaN. Bound by the edges' bytes: eight columns a
// thread, the edges' loads of four j together on their way.
#include "common.cuh"
#include "layer.h"

namespace epoch {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
  uint4 u;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[4 * h]), "=f"(v[4 * h + 1]), "=f"(v[4 * h + 2]), "=f"(v[4 * h + 3])
                 : "l"(p + 4 * h));
}
template <typename T, int C> __device__ __forceinline__ void load_c(const T *p, float (&v)[C]) {
  if constexpr (C == 8) load8(p, v);
  else v[0] = to_f32(p[0]);
}
__device__ __forceinline__ void store_c(__nv_bfloat16 *p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_c(float *p, const float (&v)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
template <typename T> __device__ __forceinline__ void store_c(T *p, const float (&v)[1]) { p[0] = from_f32<T>(v[0]); }

template <typename T, int C> __device__ __forceinline__ void add_row(const void *base, int bf16, int64_t at, float (&y)[C]) {
  float v[C];
  if (bf16) load_c<__nv_bfloat16, C>(static_cast<const __nv_bfloat16 *>(base) + at, v);
  else load_c<float, C>(static_cast<const float *>(base) + at, v);
#pragma unroll
  for (int i = 0; i < C; ++i) y[i] += v[i];
}

// C columns a thread: 8 where every row starts on a 16-byte boundary, else 1.
template <typename T, int C> __global__ void __launch_bounds__(kThreads) k_combine_edges(const CombineArgs a, unsigned pieces) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t t = i / pieces;
  if (t >= a.n_tok) return;
  const int c = static_cast<int>(i - t * pieces) * C;
  const T *edges = static_cast<const T *>(a.edges) + c;
  const int32_t *slots = a.slots + t * a.k;
  const float *weights = a.weights + t * a.k;
  float y[C];
#pragma unroll
  for (int q = 0; q < C; ++q) y[q] = 0.f;
  bool bad = false;
  constexpr int kTogether = 4;
  for (int j0 = 0; j0 < a.k; j0 += kTogether) {
    float v[kTogether][C], w[kTogether];
#pragma unroll
    for (int j = 0; j < kTogether; ++j) {
      const int slot = j0 + j < a.k ? __ldg(slots + j0 + j) : -1;
      const bool in = slot >= 0 && slot < a.n_edges;
      bad = bad || slot >= a.n_edges;
      w[j] = in ? __ldg(weights + j0 + j) : 0.f;
#pragma unroll
      for (int q = 0; q < C; ++q) v[j][q] = 0.f;
      if (in) load_c<T, C>(edges + slot * a.edges_stride, v[j]);
    }
#pragma unroll
    for (int j = 0; j < kTogether; ++j)
#pragma unroll
      for (int q = 0; q < C; ++q) y[q] = fmaf(w[j], v[j][q], y[q]);
  }
  if (a.shared) add_row<T, C>(a.shared, sizeof(T) == 2, t * a.shared_stride + c, y);
  if (a.residual) add_row<T, C>(a.residual, a.residual_bf16, t * a.residual_stride + c, y);
  if (bad)
#pragma unroll
    for (int q = 0; q < C; ++q) y[q] = __uint_as_float(0x7FC00000u);
  if (a.out_bf16) store_c(static_cast<__nv_bfloat16 *>(a.out) + t * a.out_stride + c, y);
  else store_c(static_cast<float *>(a.out) + t * a.out_stride + c, y);
}

template <typename T> cudaError_t launch_type(const CombineArgs &a, bool vec, cudaStream_t s) {
  const int64_t pieces = vec ? a.hidden / 8 : a.hidden, grid = (a.n_tok * pieces + kThreads - 1) / kThreads;
  if (vec) k_combine_edges<T, 8><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a, static_cast<unsigned>(pieces));
  else k_combine_edges<T, 1><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a, static_cast<unsigned>(pieces));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_combine_edges(const CombineArgs &a, bool bf16, cudaStream_t s) {
  auto on16 = [](const void *p, int64_t rows, int64_t stride, int size) {
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (rows <= 1 || stride * size % 16 == 0));
  };
  const int size = bf16 ? 2 : 4;
  const bool vec = a.hidden % 8 == 0 && on16(a.edges, a.n_edges, a.edges_stride, size) &&
                   on16(a.shared, a.n_tok, a.shared_stride, size) &&
                   on16(a.residual, a.n_tok, a.residual_stride, a.residual_bf16 ? 2 : 4) &&
                   on16(a.out, a.n_tok, a.out_stride, a.out_bf16 ? 2 : 4);
  return bf16 ? launch_type<__nv_bfloat16>(a, vec, s) : launch_type<float>(a, vec, s);
}

}  // namespace epoch
