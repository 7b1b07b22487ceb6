// Quantisation to 8-bit floating point (e4m3) with a scale for each block of
// 128 consecutive columns: of rows (optionally gathered by a worklist, or the
// SwiGLU of a gate | up pair), and of weight matrices in blocks of 128 x 128.
//
//   s = max(max|x| / 448, 2^-126) over the block,  q = e4m3(x * (1 / s))
//
// 448 is the largest finite e4m3 value. The maximum is taken on the bit
// patterns of |x|, so a NaN (whose pattern is above infinity's) makes its
// block's scale NaN, and an infinity makes it infinite: either way every
// product with the block is NaN instead of a finite wrong number. The lower
// bound keeps 1 / s finite; a block of zeros gets q = 0.
#include "common.cuh"
#include "fp8.cuh"
#include "layer.h"

namespace epoch {

namespace {

constexpr int kQuantThreads = 256;

template <bool VEC> __device__ __forceinline__ void load8(const __nv_bfloat16 *p, int n, float (&v)[8]) {
  if constexpr (VEC) {
    uint4 u;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? __bfloat162float(p[i]) : 0.f;
  }
}
template <bool VEC> __device__ __forceinline__ void load8(const float *p, int n, float (&v)[8]) {
  if constexpr (VEC) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v[4 * h]), "=f"(v[4 * h + 1]), "=f"(v[4 * h + 2]), "=f"(v[4 * h + 3])
                   : "l"(p + 4 * h));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.f;
  }
}

// Sixteen threads take a block of a row, eight columns each; a CTA takes U times
// sixteen consecutive blocks, U of them (their row indices first, then their
// columns) on their way at once: a block is a chain of two loads, five shuffles and a
// store. 8192 gathered rows of 2048: 13.9 us with U = 1.
template <typename T, bool SWIGLU, bool VEC, int U>
__global__ void __launch_bounds__(kQuantThreads) k_fp8_quant(const QuantArgs a, int kb_n) {
  constexpr int kHalves = kQuantThreads / 16;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kHalves * U);
  const int64_t row0 = first / kb_n;
  const unsigned at0 = static_cast<unsigned>(first - row0 * kb_n) + (threadIdx.x >> 4);
  int64_t src[U];
  float v[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = row0 + (at0 + u * kHalves) / static_cast<unsigned>(kb_n);
    src[u] = row;
    if (a.rows != nullptr && row < a.n_rows) src[u] = __ldg(a.rows + row);
  }
  auto place = [&](int u, int64_t *row, int *kb, int *c, int *n) {
    const unsigned at = at0 + u * kHalves, r = at / static_cast<unsigned>(kb_n);
    *row = row0 + r;
    *kb = static_cast<int>(at - r * kb_n);
    *c = *kb * 128 + (threadIdx.x & 15) * 8;
    *n = *row < a.n_rows && *c < a.cols ? min(a.cols - *c, 8) : 0;
  };
#pragma unroll
  for (int u = 0; u < U; ++u) {
    int64_t row;
    int kb, c, n;
    place(u, &row, &kb, &c, &n);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
    // an index out of range is never followed: its scales are NaN
    if (n > 0 && src[u] >= 0 && src[u] < a.n_src) {
      const T *p = static_cast<const T *>(a.x) + src[u] * a.x_stride + c;
      load8<VEC>(p, n, v[u]);
      if constexpr (SWIGLU) {
        float w[8];
        load8<VEC>(p + a.cols, n, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = silu(v[u][i]) * w[i];
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    int64_t row;
    int kb, c, n;
    place(u, &row, &kb, &c, &n);
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[u][i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    float s = fp8_scale(m);
    if (src[u] < 0 || src[u] >= a.n_src) s = __uint_as_float(0x7FC00000u);
    if (row < a.n_rows && (threadIdx.x & 15) == 0) a.scales[row * kb_n + kb] = s;
    if (n == 0) continue;
    const float inv = 1.0f / s;
    uint8_t *q = a.q + row * a.cols + c;
    const uint2 out = make_uint2(fp8_pack4(v[u][0] * inv, v[u][1] * inv, v[u][2] * inv, v[u][3] * inv),
                                 fp8_pack4(v[u][4] * inv, v[u][5] * inv, v[u][6] * inv, v[u][7] * inv));
    if constexpr (VEC) {
      *reinterpret_cast<uint2 *>(q) = out;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) q[i] = static_cast<uint8_t>((i < 4 ? out.x : out.y) >> (8 * (i & 3)));
    }
  }
}

// One CTA per 128 x 128 block of a weight matrix [n][k]; blockIdx.z: the matrix.
template <typename T>
__global__ void __launch_bounds__(256) k_fp8_quant_weight(const T *w, int64_t n, int64_t k, uint8_t *q, float *scales) {
  __shared__ unsigned s_max[8];
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 128, c0 = static_cast<int64_t>(blockIdx.x) * 128;
  const int64_t base = static_cast<int64_t>(blockIdx.z) * n * k;
  const int64_t c = c0 + (threadIdx.x & 127);
  unsigned m = 0;
  for (int i = threadIdx.x >> 7; i < 128; i += 2) {
    const int64_t r = r0 + i;
    if (r < n && c < k) {
      const unsigned b = __float_as_uint(to_f32(w[base + r * k + c])) & 0x7FFFFFFFu;
      m = b > m ? b : m;
    }
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if (lane_id() == 0) s_max[warp_id()] = m;
  __syncthreads();
  for (int i = 0; i < 8; ++i) m = s_max[i] > m ? s_max[i] : m;
  const float s = fp8_scale(m);
  if (threadIdx.x == 0)
    scales[(static_cast<int64_t>(blockIdx.z) * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x] = s;
  const float inv = 1.0f / s;
  for (int i = threadIdx.x >> 7; i < 128; i += 2) {
    const int64_t r = r0 + i;
    if (r < n && c < k)
      q[base + r * k + c] = static_cast<uint8_t>(fp8_pack4(to_f32(w[base + r * k + c]) * inv, 0.f, 0.f, 0.f) & 0xFFu);
  }
}

template <typename T, bool SWIGLU, bool VEC> cudaError_t launch_blocks(const QuantArgs &a, cudaStream_t s) {
  const int kb = (a.cols + 127) / 128;
  const int64_t blocks = a.n_rows * kb, per = kQuantThreads / 16;
  // four blocks at once where that still leaves every SM eight CTAs
  if (blocks >= 4 * per * 8 * num_sms())
    k_fp8_quant<T, SWIGLU, VEC, 4><<<static_cast<unsigned>((blocks + 4 * per - 1) / (4 * per)), kQuantThreads, 0, s>>>(a, kb);
  else
    k_fp8_quant<T, SWIGLU, VEC, 1><<<static_cast<unsigned>((blocks + per - 1) / per), kQuantThreads, 0, s>>>(a, kb);
  return cudaGetLastError();
}
template <typename T> cudaError_t launch_rows(const QuantArgs &a, bool vec, cudaStream_t s) {
  if (a.swiglu) return vec ? launch_blocks<T, true, true>(a, s) : launch_blocks<T, true, false>(a, s);
  return vec ? launch_blocks<T, false, true>(a, s) : launch_blocks<T, false, false>(a, s);
}

}  // namespace

cudaError_t launch_fp8_quant(const QuantArgs &a, bool bf16, cudaStream_t s) {
  // eight columns at a time where every block of eight starts on a 16-byte (q: 8-byte) boundary
  const bool vec = a.cols % 8 == 0 && (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && a.x_stride % 8 == 0 &&
                   (reinterpret_cast<uintptr_t>(a.q) & 7u) == 0;
  return bf16 ? launch_rows<__nv_bfloat16>(a, vec, s) : launch_rows<float>(a, vec, s);
}

cudaError_t launch_fp8_quant_weight(const void *w, bool bf16, int64_t mats, int64_t n, int64_t k, uint8_t *q,
                                    float *scales, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((k + 127) / 128), static_cast<unsigned>((n + 127) / 128),
                  static_cast<unsigned>(mats));
  if (bf16)
    k_fp8_quant_weight<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16 *>(w), n, k, q, scales);
  else
    k_fp8_quant_weight<<<grid, 256, 0, s>>>(static_cast<const float *>(w), n, k, q, scales);
  return cudaGetLastError();
}

}  // namespace epoch
