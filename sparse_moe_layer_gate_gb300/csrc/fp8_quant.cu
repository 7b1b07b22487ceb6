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

__device__ __forceinline__ void load16(const __nv_bfloat16 *p, float (&v)[16], unsigned &m) {
  uint4 u[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u[h].x), "=r"(u[h].y), "=r"(u[h].z), "=r"(u[h].w)
                 : "l"(p + 8 * h));
  const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
  uint32_t big = 0;  // largest magnitudes of the low and of the high halves
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    big = __vmaxu2(big, w[i] & 0x7FFF7FFFu);
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  m = max(big << 16, big & 0xFFFF0000u);
}
__device__ __forceinline__ void load16(const float *p, float (&v)[16], unsigned &m) {
#pragma unroll
  for (int h = 0; h < 4; ++h)
    asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[4 * h]), "=f"(v[4 * h + 1]), "=f"(v[4 * h + 2]), "=f"(v[4 * h + 3])
                 : "l"(p + 4 * h));
  m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
}

// Rows of whole 16-column pieces: eight threads take a block, sixteen columns
// each, and a CTA a tile of 2^tx blocks of a row x 32 / 2^tx rows, where 2^tx is the
// largest power of two (up to 32) that divides a row's blocks: places follow by
// shifts: 8.7 us at 8192 gathered rows of 2048 (2.5 TB/s of rows read and bytes
// written), where eight columns a thread and places by division took 13.9. Fewer
// instructions paid there, but they fill 46 % of the issue slots and the largest stall
// is the loads': a thread has one piece of one row on its way, and that latency is what
// is left. 65536 rows in their own order take 70 us, 86 % of the copy rate.
template <typename T, bool SWIGLU>
__global__ void __launch_bounds__(kQuantThreads) k_fp8_quant_wide(const QuantArgs a, int kb_n, int tx) {
  const unsigned tiles_x = static_cast<unsigned>(kb_n) >> tx;
  const unsigned ty = blockIdx.x / tiles_x;
  const int local = threadIdx.x >> 3;
  const int kb = static_cast<int>((blockIdx.x - ty * tiles_x) << tx) + (local & ((1 << tx) - 1));
  const int64_t row = static_cast<int64_t>(ty) * (32 >> tx) + (local >> tx);
  if (row >= a.n_rows) return;  // a block's eight threads leave together
  const unsigned lanes = 0xFFu << (threadIdx.x & 24);
  const int c = kb * 128 + (threadIdx.x & 7) * 16;
  int64_t src = row;
  if (a.rows != nullptr) src = __ldg(a.rows + row);
  const bool bad = src < 0 || src >= a.n_src;  // never followed: its scales are NaN
  const bool in = c < a.cols;
  float v[16];
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.f;
  if (in && !bad) {
    const T *p = static_cast<const T *>(a.x) + src * a.x_stride + c;
    load16(p, v, m);
    if constexpr (SWIGLU) {
      float u[16];
      unsigned unused;
      load16(p + a.cols, u, unused);
      m = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        v[i] = silu(v[i]) * u[i];
        m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
      }
    }
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(lanes, m, o));
  const float s = bad ? __uint_as_float(0x7FC00000u) : fp8_scale(m);
  if ((threadIdx.x & 7) == 0) a.scales[row * kb_n + kb] = s;
  if (!in) return;
  const float inv = 1.0f / s;
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = fp8_pack4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
  *reinterpret_cast<uint4 *>(a.q + row * a.cols + c) = make_uint4(q[0], q[1], q[2], q[3]);
}

// Eight consecutive elements from a 16-byte boundary on.
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
  const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// Any row: sixteen threads take a block, eight columns each; a CTA takes sixteen
// consecutive blocks. VEC: eight columns at a time (8192 rows of 2040, bf16: 20.1 us by
// single elements, 14.4 so).
template <typename T, bool SWIGLU, bool VEC>
__global__ void __launch_bounds__(kQuantThreads) k_fp8_quant(const QuantArgs a, int kb_n) {
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kQuantThreads / 16);
  const int64_t row0 = first / kb_n;
  const unsigned at = static_cast<unsigned>(first - row0 * kb_n) + (threadIdx.x >> 4), r = at / static_cast<unsigned>(kb_n);
  const int64_t row = row0 + r;
  const int kb = static_cast<int>(at - r * kb_n), c = kb * 128 + (threadIdx.x & 15) * 8;
  const bool on = row < a.n_rows;
  const int n = on && c < a.cols ? min(a.cols - c, 8) : 0;
  int64_t src = row;
  if (a.rows != nullptr && on) src = __ldg(a.rows + row);
  const bool bad = src < 0 || src >= a.n_src;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  if (n > 0 && !bad) {
    const T *p = static_cast<const T *>(a.x) + src * a.x_stride + c;
    if constexpr (VEC) {
      load8(p, v);
      if constexpr (SWIGLU) {
        float u[8];
        load8(p + a.cols, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = silu(v[i]) * u[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) v[i] = to_f32(p[i]);
      if constexpr (SWIGLU) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < n) v[i] = silu(v[i]) * to_f32(p[a.cols + i]);
      }
    }
  }
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (!on) return;
  const float s = bad ? __uint_as_float(0x7FC00000u) : fp8_scale(m);
  if ((threadIdx.x & 15) == 0) a.scales[row * kb_n + kb] = s;
  const float inv = 1.0f / s;
  uint8_t *q = a.q + row * a.cols + c;
  if constexpr (VEC) {
    if (n > 0)
      *reinterpret_cast<uint2 *>(q) = make_uint2(fp8_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                                                 fp8_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) q[i] = static_cast<uint8_t>(fp8_pack4(v[i] * inv, 0.f, 0.f, 0.f) & 0xFFu);
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

template <typename T, bool SWIGLU> cudaError_t launch_blocks(const QuantArgs &a, int per, cudaStream_t s) {
  const int kb = (a.cols + 127) / 128;
  if (per == 16) {
    int tx = 0;
    while (tx < 5 && (kb >> tx) % 2 == 0) ++tx;
    const int64_t rows = 32 >> tx, grid = (a.n_rows + rows - 1) / rows * (kb >> tx);
    k_fp8_quant_wide<T, SWIGLU><<<static_cast<unsigned>(grid), kQuantThreads, 0, s>>>(a, kb, tx);
  } else {
    const int64_t blocks = kQuantThreads / 16, grid = (a.n_rows * kb + blocks - 1) / blocks;
    if (per == 8) k_fp8_quant<T, SWIGLU, true><<<static_cast<unsigned>(grid), kQuantThreads, 0, s>>>(a, kb);
    else k_fp8_quant<T, SWIGLU, false><<<static_cast<unsigned>(grid), kQuantThreads, 0, s>>>(a, kb);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_quant(const QuantArgs &a, bool bf16, cudaStream_t s) {
  // sixteen or eight columns at a time where every such piece starts on a 16-byte boundary (of q, on one of its size)
  const int64_t per16 = bf16 ? 8 : 4;
  const uintptr_t q = reinterpret_cast<uintptr_t>(a.q);
  const bool on16 = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && (a.n_src <= 1 || a.x_stride % per16 == 0);
  const int per = on16 && a.cols % 16 == 0 && (q & 15u) == 0 ? 16 : on16 && a.cols % 8 == 0 && (q & 7u) == 0 ? 8 : 1;
  if (a.swiglu) return bf16 ? launch_blocks<__nv_bfloat16, true>(a, per, s) : launch_blocks<float, true>(a, per, s);
  return bf16 ? launch_blocks<__nv_bfloat16, false>(a, per, s) : launch_blocks<float, false>(a, per, s);
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
