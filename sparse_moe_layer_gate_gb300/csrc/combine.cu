// The weighted sum of each position's edges, with the shared experts' output and the residual stream:
//
//   y[t] = sum_j weights[t, j] * edges[slots[t, j]] (+ shared[t]) (+ residual[t])
//
// in fp32, j ascending, rounded once. A negative slot adds nothing (a position that was routed to fewer
// experts); one past the last edge makes the row NaN. Bound by the edges' bytes: a thread takes up to eight
// columns, by vectors as wide as the rows' alignment allows, with the edges' loads of four j together on
// their way; slots and weights are read once for all of its columns (8192 positions of 8 edges by 4096
// columns in bf16: 100 us, 6.0 TB/s). bf16 rows off 16-byte boundaries come by aligned vectors too, which
// are shifted (2000 positions of 8 edges by 2779 columns: 23.7 us; by elements 69).
#include "common.cuh"
#include "layer.h"

namespace epoch {

namespace {

constexpr int kThreads = 256;

// C elements from a boundary of their size (at most 16 bytes) on.
template <int C> __device__ __forceinline__ void load_c(const __nv_bfloat16 *p, float (&v)[C]) {
  uint32_t w[C > 1 ? C / 2 : 1];
  if constexpr (C == 8)
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
  else if constexpr (C == 4)
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
  else if constexpr (C == 2)
    asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(w[0]) : "l"(p));
  if constexpr (C == 1) {
    v[0] = __bfloat162float(*p);
  } else {
#pragma unroll
    for (int i = 0; i < C / 2; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
template <int C> __device__ __forceinline__ void load_c(const float *p, float (&v)[C]) {
  if constexpr (C >= 4) {
#pragma unroll
    for (int h = 0; h < C / 4; ++h)
      asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v[4 * h]), "=f"(v[4 * h + 1]), "=f"(v[4 * h + 2]), "=f"(v[4 * h + 3])
                   : "l"(p + 4 * h));
  } else if constexpr (C == 2) {
    asm volatile("ld.global.L1::no_allocate.v2.f32 {%0, %1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "l"(p));
  } else {
    v[0] = *p;
  }
}
template <int C> __device__ __forceinline__ void store_c(__nv_bfloat16 *p, const float (&v)[C]) {
  if constexpr (C == 1) {
    *p = __float2bfloat16_rn(v[0]);
  } else {
    uint32_t w[C / 2];
#pragma unroll
    for (int i = 0; i < C / 2; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    if constexpr (C == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (C == 4) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(p) = w[0];
  }
}
template <int C> __device__ __forceinline__ void store_c(float *p, const float (&v)[C]) {
  if constexpr (C >= 4) {
#pragma unroll
    for (int h = 0; h < C / 4; ++h) reinterpret_cast<float4 *>(p)[h] = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
  } else if constexpr (C == 2) {
    *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
  } else {
    *p = v[0];
  }
}

template <int C> __device__ __forceinline__ void add_row(const void *base, int bf16, int64_t at, float (&y)[C]) {
  float v[C];
  if (bf16) load_c<C>(static_cast<const __nv_bfloat16 *>(base) + at, v);
  else load_c<C>(static_cast<const float *>(base) + at, v);
#pragma unroll
  for (int i = 0; i < C; ++i) y[i] += v[i];
}

// A thread takes 8 / C vectors of C columns of a row, `lanes` threads a row.
template <typename T, int C> __global__ void __launch_bounds__(kThreads, 4) k_combine_edges(const CombineArgs a, unsigned lanes) {
  constexpr int V = 8 / C;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t t = i / lanes;
  if (t >= a.n_tok) return;
  const int c0 = static_cast<int>(i - t * lanes) * C, step = static_cast<int>(lanes) * C;
  const int32_t *slots = a.slots + t * a.k;
  const float *weights = a.weights + t * a.k;
  float y[V][C];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int q = 0; q < C; ++q) y[v][q] = 0.f;
  bool bad = false;
  constexpr int kTogether = 4;
  for (int j0 = 0; j0 < a.k; j0 += kTogether) {
    float x[kTogether][V][C], w[kTogether];
#pragma unroll
    for (int j = 0; j < kTogether; ++j) {
      const int slot = j0 + j < a.k ? __ldg(slots + j0 + j) : -1;
      const bool in = slot >= 0 && slot < a.n_edges;
      bad = bad || slot >= a.n_edges;
      w[j] = in ? __ldg(weights + j0 + j) : 0.f;
      const T *edge = static_cast<const T *>(a.edges) + c0 + (in ? slot : 0) * a.edges_stride;
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int q = 0; q < C; ++q) x[j][v][q] = 0.f;
        if (in && (V == 1 || c0 + v * step < a.hidden)) load_c<C>(edge + v * step, x[j][v]);
      }
    }
#pragma unroll
    for (int j = 0; j < kTogether; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int q = 0; q < C; ++q) y[v][q] = fmaf(w[j], x[j][v][q], y[v][q]);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = c0 + v * step;
    if (V > 1 && c >= a.hidden) break;
    if (a.shared) add_row<C>(a.shared, sizeof(T) == 2, t * a.shared_stride + c, y[v]);
    if (a.residual) add_row<C>(a.residual, a.residual_bf16, t * a.residual_stride + c, y[v]);
    if (bad)
#pragma unroll
      for (int q = 0; q < C; ++q) y[v][q] = __uint_as_float(0x7FC00000u);
    if (a.out_bf16) store_c<C>(static_cast<__nv_bfloat16 *>(a.out) + t * a.out_stride + c, y[v]);
    else store_c<C>(static_cast<float *>(a.out) + t * a.out_stride + c, y[v]);
  }
}

// Eight values of a bf16 row from column c0 on (from -7 on; c0 < hidden), whatever 2-byte boundary they start on: the two
// aligned vectors that hold them, shifted. A vector without a column of the row is not read; of the others only lie
// columns of the row in use. (No vector crosses into a page that the row has no part of.)
__device__ __forceinline__ void load_shifted(const __nv_bfloat16 *row, int c0, int hidden, uint32_t (&w)[8], int *off) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(row + c0);
  const uint4 *from = reinterpret_cast<const uint4 *>(at & ~static_cast<uintptr_t>(15));
  *off = static_cast<int>(at & 15u) / 2;
  const int first = c0 - *off;
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 0u;
  if (first + 8 > 0) asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(from));
  if (*off > 0 && first + 8 < hidden)
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "l"(from + 1));
}
__device__ __forceinline__ void shift(uint32_t (&w)[8], int off, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = off & 4 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = off & 2 ? w[i + 1] : w[i];
  const unsigned pick = off & 1 ? 0x5432u : 0x3210u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = __byte_perm(w[i], w[i + 1], pick);
    v[2 * i] = __uint_as_float(u << 16);
    v[2 * i + 1] = __uint_as_float(u & 0xFFFF0000u);
  }
}

// bf16 edges whose rows start or end off 16-byte boundaries: a thread takes the eight columns of 16 or 32 aligned bytes of the
// output row, so that lanes' stores are whole vectors too.
__global__ void __launch_bounds__(kThreads, 4) k_combine_shifted(const CombineArgs a, unsigned lanes) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t t = i / lanes;
  if (t >= a.n_tok) return;
  const uintptr_t out = reinterpret_cast<uintptr_t>(a.out) + t * a.out_stride * (a.out_bf16 ? 2 : 4);
  const int c0 = static_cast<int>(i - t * lanes) * 8 - static_cast<int>(out & 15u) / (a.out_bf16 ? 2 : 4);
  if (c0 >= a.hidden) return;
  const int32_t *slots = a.slots + t * a.k;
  const float *weights = a.weights + t * a.k;
  const __nv_bfloat16 *edges = static_cast<const __nv_bfloat16 *>(a.edges);
  float y[8] = {};
  bool bad = false;
  constexpr int kTogether = 4;
  for (int j0 = 0; j0 < a.k; j0 += kTogether) {
    uint32_t x[kTogether][8];
    float w[kTogether];
    int off[kTogether];
#pragma unroll
    for (int j = 0; j < kTogether; ++j) {
      const int slot = j0 + j < a.k ? __ldg(slots + j0 + j) : -1;
      const bool in = slot >= 0 && slot < a.n_edges;
      bad = bad || slot >= a.n_edges;
      w[j] = 0.f;
      off[j] = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) x[j][q] = 0u;
      if (in) {
        w[j] = __ldg(weights + j0 + j);
        load_shifted(edges + slot * a.edges_stride, c0, a.hidden, x[j], &off[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < kTogether; ++j) {
      float v[8];
      shift(x[j], off[j], v);
#pragma unroll
      for (int q = 0; q < 8; ++q) y[q] = fmaf(w[j], v[q], y[q]);
    }
  }
  auto add = [&](const void *base, bool bf16, int64_t at) {
    float v[8];
    if (bf16) {
      uint32_t x[8];
      int off;
      load_shifted(static_cast<const __nv_bfloat16 *>(base) + at, c0, a.hidden, x, &off);
      shift(x, off, v);
    } else {
      const float *row = static_cast<const float *>(base) + at;
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = c0 + q >= 0 && c0 + q < a.hidden ? row[c0 + q] : 0.f;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) y[q] += v[q];
  };
  if (a.shared) add(a.shared, true, t * a.shared_stride);
  if (a.residual) add(a.residual, a.residual_bf16, t * a.residual_stride);
  if (bad)
#pragma unroll
    for (int q = 0; q < 8; ++q) y[q] = __uint_as_float(0x7FC00000u);
  const bool whole = c0 >= 0 && c0 + 8 <= a.hidden;
  if (a.out_bf16) {
    __nv_bfloat16 *to = reinterpret_cast<__nv_bfloat16 *>(out) + c0;
    if (whole) {
      store_c<8>(to, y);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (c0 + q >= 0 && c0 + q < a.hidden) to[q] = __float2bfloat16_rn(y[q]);
    }
  } else {
    float *to = reinterpret_cast<float *>(out) + c0;
    if (whole) {
      store_c<8>(to, y);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (c0 + q >= 0 && c0 + q < a.hidden) to[q] = y[q];
    }
  }
}

template <typename T, int C> cudaError_t launch_columns(const CombineArgs &a, cudaStream_t s) {
  const int64_t lanes = (a.hidden + 7) / 8, grid = (a.n_tok * lanes + kThreads - 1) / kThreads;
  k_combine_edges<T, C><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a, static_cast<unsigned>(lanes));
  return cudaGetLastError();
}
template <typename T> cudaError_t launch_type(const CombineArgs &a, int c, cudaStream_t s) {
  if (c == 8) return launch_columns<T, 8>(a, s);
  if (c == 4) return launch_columns<T, 4>(a, s);
  return c == 2 ? launch_columns<T, 2>(a, s) : launch_columns<T, 1>(a, s);
}

}  // namespace

cudaError_t launch_combine_edges(const CombineArgs &a, bool bf16, cudaStream_t s) {
  // Columns of a vector: the most, up to 8, for which every row of every tensor and the row's end lie on the vector's
  // size (16 bytes at most).
  int c = 8;
  while (c > 1 && a.hidden % c) c /= 2;
  auto fits = [&](const void *p, int64_t rows, int64_t stride, int size) {
    if (p == nullptr) return;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(p) | (rows > 1 ? static_cast<uintptr_t>(stride * size) : 0u);
    while (c > 1 && bits % (c * size < 16 ? c * size : 16)) c /= 2;
  };
  fits(a.edges, a.n_edges, a.edges_stride, bf16 ? 2 : 4);
  fits(a.shared, a.n_tok, a.shared_stride, bf16 ? 2 : 4);
  fits(a.residual, a.n_tok, a.residual_stride, a.residual_bf16 ? 2 : 4);
  fits(a.out, a.n_tok, a.out_stride, a.out_bf16 ? 2 : 4);
  if (!bf16) return launch_type<float>(a, c, s);
  if (c == 8) return launch_columns<__nv_bfloat16, 8>(a, s);
  const int64_t lanes = (a.hidden + 14) / 8, grid = (a.n_tok * lanes + kThreads - 1) / kThreads;
  k_combine_shifted<<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a, static_cast<unsigned>(lanes));
  return cudaGetLastError();
}

}  // namespace epoch
