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

// Sixteen threads take one block of a row, eight columns each; a CTA takes
// sixteen consecutive blocks (rows of the output in order, so a CTA reads 4 KB
// of consecutive bf16 when the rows are).
template <typename T, bool SWIGLU, bool VEC>
__global__ void __launch_bounds__(kQuantThreads) k_fp8_quant(const QuantArgs a, int kb_n) {
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kQuantThreads / 16);
  const int64_t row0 = first / kb_n;
  const int at = static_cast<int>(first - row0 * kb_n) + (threadIdx.x >> 4);
  const int64_t row = row0 + at / kb_n;
  const int kb = at % kb_n;
  const int c = kb * 128 + (threadIdx.x & 15) * 8;
  const bool on = row < a.n_rows;
  const int n = on && c < a.cols ? (a.cols - c < 8 ? a.cols - c : 8) : 0;
  int64_t src = row;
  if (a.rows != nullptr && on) src = a.rows[row];
  const bool bad = src < 0 || src >= a.n_src;  // never read: its scales are NaN
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  if (n > 0 && !bad) {
    const T *p = static_cast<const T *>(a.x) + src * a.x_stride + c;
    load8<VEC>(p, n, v);
    if constexpr (SWIGLU) {
      float u[8];
      load8<VEC>(p + a.cols, n, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = silu(v[i]) * u[i];
    }
  }
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const unsigned b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
    m = b > m ? b : m;
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const unsigned b = __shfl_xor_sync(0xffffffffu, m, o);
    m = b > m ? b : m;
  }
  float s = fp8_scale(m);
  if (bad) s = __uint_as_float(0x7FC00000u);
  if (!on) return;
  if ((threadIdx.x & 15) == 0) a.scales[row * kb_n + kb] = s;
  if (n == 0) return;
  const float inv = 1.0f / s;
  uint8_t *q = a.q + row * a.cols + c;
  if (VEC || n == 8) {
    const uint2 out = make_uint2(fp8_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                                 fp8_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
    if (VEC) {
      *reinterpret_cast<uint2 *>(q) = out;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = static_cast<uint8_t>((i < 4 ? out.x : out.y) >> (8 * (i & 3)));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) q[i] = static_cast<uint8_t>(fp8_pack4(v[i] * inv, 0.f, 0.f, 0.f) & 0xFFu);
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

template <typename T> cudaError_t launch_rows(const QuantArgs &a, bool vec, cudaStream_t s) {
  const int kb = (a.cols + 127) / 128;
  const int64_t per = kQuantThreads / 16;
  const int64_t grid = (a.n_rows * kb + per - 1) / per;
  const unsigned g = static_cast<unsigned>(grid);
  if (a.swiglu) {
    if (vec) k_fp8_quant<T, true, true><<<g, kQuantThreads, 0, s>>>(a, kb);
    else k_fp8_quant<T, true, false><<<g, kQuantThreads, 0, s>>>(a, kb);
  } else {
    if (vec) k_fp8_quant<T, false, true><<<g, kQuantThreads, 0, s>>>(a, kb);
    else k_fp8_quant<T, false, false><<<g, kQuantThreads, 0, s>>>(a, kb);
  }
  return cudaGetLastError();
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
