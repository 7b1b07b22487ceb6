// Quantisation to 4-bit floating point (e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) with
// a scale for each block of consecutive columns, of rows (optionally gathered by a worklist, or the
// SwiGLU of a gate | up pair) and of weight matrices, and back.
//
//   nvfp4: blocks of 16, v' = v / t for a tensor scale t, s = e4m3(min(max|v'| / 6, 448)), at least
//          2^-9 (the smallest e4m3 value: a block of zeros divides by it), q = e2m1(v' / s)
//   mxfp4: blocks of 32, s = 2^(floor(log2 max|v|) - 2) within e8m0's range, q = e2m1(v / s)
//
// Both roundings are to nearest even of the exact quotients: s has four bits, so a border between
// two codes times s is exact in fp32, and a quotient that fp32 cannot tell from a border is decided
// by the remainder's sign. A block that holds a NaN or an infinity gets a NaN scale, so that every
// product with it is NaN. Scales lie by blocks of 256 columns, [ceil(K / 256)][rows][16 or 8], with
// zeros behind the last column.
#include <cmath>

#include <cuda_fp16.h>

#include "common.cuh"
#include "layer.h"

namespace epoch {

namespace {

constexpr int kThreads = 256;

// Sixteen consecutive elements from a 16-byte boundary on, and the bits of their largest magnitude.
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
__device__ __forceinline__ unsigned largest(const float (&v)[16]) {
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}
__device__ __forceinline__ void load16(const float *p, float (&v)[16], unsigned &m) {
#pragma unroll
  for (int h = 0; h < 4; ++h)
    asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[4 * h]), "=f"(v[4 * h + 1]), "=f"(v[4 * h + 2]), "=f"(v[4 * h + 3])
                 : "l"(p + 4 * h));
  m = largest(v);
}
// The same at any alignment.
template <typename T> __device__ __forceinline__ void load16_any(const T *p, float (&v)[16], unsigned &m) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = to_f32(p[i]);
  m = largest(v);
}

// Eight values to e2m1 (round to nearest even, out of range to the largest), the first in the lowest four bits.
__device__ __forceinline__ uint32_t pack8(const float *v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// e4m3 of m / 6 (m finite, >= 0), rounded once and kept within [2^-9, 448]. The quotient in fp32 may round onto a
// border between two e4m3 values; the remainder tells on which side of it m / 6 lies.
__device__ __forceinline__ uint32_t nv_scale(float m, float *s) {
  float q = m / 6.0f;
  const float rest = fmaf(-6.0f, q, m);
  if (rest > 0.f) q = __uint_as_float(__float_as_uint(q) | 1u);
  else if (rest < 0.f && (__float_as_uint(q) & 1u) == 0u) q = __uint_as_float(__float_as_uint(q) - 1u);
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.f), "f"(q));
  uint32_t b = two & 0xFFu;
  if (b == 0u) b = 1u;
  const uint32_t e = b >> 3, f = b & 7u;  // e4m3: bias 7; e = 0: f * 2^-9
  *s = e ? __uint_as_float(((e + 120u) << 23) | (f << 20)) : static_cast<float>(f) * 0x1p-9f;
  return b;
}

// Codes of v / s, inv = 1 / s. Quotients are taken to twelve bits, which leaves every border between codes (three bits)
// as it is and, where v has eight bits (EXACT false), keeps all others on their side of it: v and a border times s
// differ by 2^-8 or more of them. EXACT: a quotient that landed on a border moves off it by the sign of its remainder.
template <bool EXACT> __device__ __forceinline__ void nv_codes(const float (&v)[16], float s, float inv, uint32_t (&q)[2]) {
  float t[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    uint32_t b = (__float_as_uint(v[i] * inv) + 0x800u) & 0xFFFFF000u;
    if constexpr (EXACT) {
      const float at = __uint_as_float(b), rest = fmaf(-at, s, v[i]);
      // away from zero where v is beyond at * s, towards it where it is short of it
      if (rest != 0.f && at != 0.f) b = (rest > 0.f) == (at > 0.f) ? b + 1u : b - 1u;
    }
    t[i] = __uint_as_float(b);
  }
  q[0] = pack8(t);
  q[1] = pack8(t + 8);
}

// Sixteen columns a thread; sixteen threads take a block of 256 columns of a row and a CTA sixteen
// such blocks in order. ALIGNED: pieces start on 16-byte boundaries. EXACT: see nv_codes (else the tensor scale is a
// power of two and goes into the factor of the quotients).
template <typename T, bool NV, bool SWIGLU, bool ALIGNED, bool EXACT>
__global__ void __launch_bounds__(kThreads) k_fp4_quant(const Fp4QuantArgs a, unsigned kb_n) {
  const unsigned at = blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4);  // blocks of 256 columns: less than 2^31 + 16
  const int64_t row = at / kb_n;
  const unsigned kb = at - static_cast<unsigned>(row) * kb_n, piece = threadIdx.x & 15u;
  const int c = static_cast<int>(kb * 256 + piece * 16);
  const bool on = row < a.n_rows, in = on && c < a.cols;
  int64_t src = row, mat = 0;
  if (a.rows != nullptr && on) src = __ldg(a.rows + row);
  const bool bad = src < 0 || src >= a.n_src;  // never followed: its scales are NaN
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.f;
  float inv = a.inv_scale;
  if (a.amax != nullptr && on) {
    mat = static_cast<unsigned>(row) / static_cast<unsigned>(a.mat_rows);
    inv = 1.0f / fp4_tensor_scale(a.amax[mat]);
  }
  unsigned m = 0;
  if (in && !bad) {
    const T *p = static_cast<const T *>(a.x) + src * a.x_stride + c;
    if constexpr (ALIGNED) load16(p, v, m);
    else load16_any(p, v, m);
    if constexpr (SWIGLU) {
      float u[16];
      unsigned unused;
      if constexpr (ALIGNED) load16(p + a.cols, u, unused);
      else load16_any(p + a.cols, u, unused);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = silu(v[i]) * u[i];
      m = largest(v);
    }
  }
  uint32_t q[2], code;
  if constexpr (NV) {
    float s;
    if constexpr (EXACT) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] *= inv;
      m = largest(v);
    }
    const bool spoilt = m >= 0x7F800000u;
    code = nv_scale(spoilt ? 0.f : EXACT ? __uint_as_float(m) : __uint_as_float(m) * inv, &s);
    if (spoilt || bad) code = 0x7Fu;
    nv_codes<EXACT>(v, s, EXACT ? 1.0f / s : 1.0f / s * inv, q);
  } else {
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    // floor(log2 m) - 2, biased by 127: the exponent field less two, for subnormal m the least
    const int e = max(static_cast<int>(m >> 23) - 2, 0);
    code = m >= 0x7F800000u || bad ? 0xFFu : static_cast<uint32_t>(e);
    const float up = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);  // 2^(127 - e), normal for e <= 253
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= up;
    q[0] = pack8(v);
    q[1] = pack8(v + 8);
  }
  if (!on) return;
  if (!in) code = 0u;
  constexpr int kPer = NV ? 16 : 8;
  if (NV || (piece & 1u) == 0u) {
    const int64_t rows = a.amax ? a.mat_rows : a.n_rows, i = a.amax ? row - mat * rows : row;
    a.scales[((mat * kb_n + kb) * rows + i) * kPer + (NV ? piece : piece >> 1)] = static_cast<uint8_t>(code);
  }
  if (in) *reinterpret_cast<uint2 *>(a.q + (row * a.cols + c) / 2) = make_uint2(q[0], q[1]);
}

// Largest |x| of each matrix, as bit patterns (a NaN's are above infinity's).
template <typename T, bool ALIGNED> __global__ void __launch_bounds__(kThreads) k_fp4_amax(const T *w, int64_t count, uint32_t *amax) {
  __shared__ uint32_t s_max[kThreads / 32];
  const T *p = w + static_cast<int64_t>(blockIdx.y) * count;
  uint32_t m = 0;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * 16; i < count;
       i += static_cast<int64_t>(gridDim.x) * kThreads * 16) {
    float v[16];
    unsigned here;
    if constexpr (ALIGNED) load16(p + i, v, here);
    else load16_any(p + i, v, here);
    m = max(m, here);
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if (lane_id() == 0) s_max[warp_id()] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kThreads / 32; ++i) m = max(m, s_max[i]);
    atomicMax(amax + blockIdx.y, m);  // a maximum: the order does not matter
  }
}

__global__ void k_fp4_tensor_scales(uint32_t *amax, int n, int nv) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) reinterpret_cast<float *>(amax)[i] = nv ? fp4_tensor_scale(amax[i]) : 1.0f;
}

// Sixteen columns a thread, in the order of k_fp4_quant.
template <typename T, bool NV>
__global__ void __launch_bounds__(kThreads) k_fp4_dequant(const Fp4DequantArgs a, unsigned kb_n) {
  const unsigned at = blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4);  // blocks of 256 columns: less than 2^31 + 16
  const int64_t row = at / kb_n;
  const unsigned kb = at - static_cast<unsigned>(row) * kb_n, piece = threadIdx.x & 15u;
  const int c = static_cast<int>(kb * 256 + piece * 16);
  if (row >= a.n_rows || c >= a.cols) return;
  const int64_t mat = static_cast<unsigned>(row) / static_cast<unsigned>(a.mat_rows), i = row - mat * a.mat_rows;
  constexpr int kPer = NV ? 16 : 8;
  const uint2 q = __ldg(reinterpret_cast<const uint2 *>(a.q + (row * a.cols + c) / 2));
  const uint32_t b = __ldg(a.scales + ((mat * kb_n + kb) * a.mat_rows + i) * kPer + (NV ? piece : piece >> 1));
  float s;
  if constexpr (NV) {
    const uint32_t e = (b >> 3) & 15u, f = b & 7u;
    s = e ? __uint_as_float(((e + 120u) << 23) | (f << 20)) : static_cast<float>(f) * 0x1p-9f;
    if ((b & 0x7Fu) == 0x7Fu) s = __uint_as_float(0x7FC00000u);
    if (b & 0x80u) s = -s;
  } else {
    s = b == 0xFFu ? __uint_as_float(0x7FC00000u) : b ? __uint_as_float(b << 23) : 0x1p-127f;
  }
  s *= a.group_scale ? a.scale * __ldg(a.group_scale + mat) : a.scale;
  float v[16];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t p[4];  // pairs in fp16, which holds e2m1's values
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
        : "r"(h ? q.y : q.x));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&p[j]));
      v[8 * h + 2 * j] = f.x * s;
      v[8 * h + 2 * j + 1] = f.y * s;
    }
  }
  T *out = static_cast<T *>(a.out) + row * a.out_stride + c;
  if (a.wide) {
    if constexpr (sizeof(T) == 2) {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t *>(&h);
      }
      reinterpret_cast<uint4 *>(out)[0] = make_uint4(w[0], w[1], w[2], w[3]);
      reinterpret_cast<uint4 *>(out)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        reinterpret_cast<float4 *>(out)[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) out[j] = from_f32<T>(v[j]);
  }
}

template <typename T, bool NV, bool SWIGLU, bool EXACT> cudaError_t launch_one(const Fp4QuantArgs &a, bool aligned, cudaStream_t s) {
  const int64_t kb = (a.cols + 255) / 256, grid = (a.n_rows * kb + kThreads / 16 - 1) / (kThreads / 16);
  const unsigned g = static_cast<unsigned>(grid), k = static_cast<unsigned>(kb);
  if (aligned) k_fp4_quant<T, NV, SWIGLU, true, EXACT><<<g, kThreads, 0, s>>>(a, k);
  else k_fp4_quant<T, NV, SWIGLU, false, EXACT><<<g, kThreads, 0, s>>>(a, k);
  return cudaGetLastError();
}
// Whether dividing by t only moves exponents (and the quotient's factor 1 / s / t stays in range).
bool power_of_two(float inv) {
  int e;
  return std::frexp(inv, &e) == 0.5f && e > -100 && e < 100;
}
template <typename T> cudaError_t launch_type(const Fp4QuantArgs &a, bool nv, bool aligned, cudaStream_t s) {
  if (!nv) return a.swiglu ? launch_one<T, false, true, true>(a, aligned, s) : launch_one<T, false, false, true>(a, aligned, s);
  if (a.swiglu) return launch_one<T, true, true, true>(a, aligned, s);
  if constexpr (sizeof(T) == 2) {
    // (a matrix's own scale may be any power of two)
    if (a.amax == nullptr && power_of_two(a.inv_scale)) return launch_one<T, true, false, false>(a, aligned, s);
  }
  return launch_one<T, true, false, true>(a, aligned, s);
}

}  // namespace

cudaError_t launch_fp4_quant(const Fp4QuantArgs &a, bool bf16, bool nv, cudaStream_t s) {
  // every piece of sixteen columns on a 16-byte boundary
  const bool aligned = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && (a.n_src <= 1 || a.x_stride % (bf16 ? 8 : 4) == 0);
  return bf16 ? launch_type<__nv_bfloat16>(a, nv, aligned, s) : launch_type<float>(a, nv, aligned, s);
}

cudaError_t launch_fp4_quant_weight(Fp4QuantArgs a, int n_mats, bool bf16, bool nv, float *tensor_scales, cudaStream_t s) {
  uint32_t *amax = reinterpret_cast<uint32_t *>(tensor_scales);
  cudaError_t e = cudaMemsetAsync(amax, 0, sizeof(uint32_t) * n_mats, s);
  if (e != cudaSuccess) return e;
  const int64_t count = a.mat_rows * a.cols;  // a multiple of 32
  if (nv) {
    const bool aligned = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0;
    const int64_t want = (count / 16 + kThreads - 1) / kThreads, most = (8 * num_sms() + n_mats - 1) / n_mats;
    const dim3 grid(static_cast<unsigned>(want < most ? want : most), static_cast<unsigned>(n_mats));
    if (bf16) {
      const auto *w = static_cast<const __nv_bfloat16 *>(a.x);
      if (aligned) k_fp4_amax<__nv_bfloat16, true><<<grid, kThreads, 0, s>>>(w, count, amax);
      else k_fp4_amax<__nv_bfloat16, false><<<grid, kThreads, 0, s>>>(w, count, amax);
    } else {
      const auto *w = static_cast<const float *>(a.x);
      if (aligned) k_fp4_amax<float, true><<<grid, kThreads, 0, s>>>(w, count, amax);
      else k_fp4_amax<float, false><<<grid, kThreads, 0, s>>>(w, count, amax);
    }
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  a.amax = amax;  // (zero for mxfp4, which takes no tensor scale)
  e = launch_fp4_quant(a, bf16, nv, s);
  if (e != cudaSuccess) return e;
  k_fp4_tensor_scales<<<(n_mats + 255) / 256, 256, 0, s>>>(amax, n_mats, nv);
  return cudaGetLastError();
}

cudaError_t launch_fp4_dequant(Fp4DequantArgs a, bool bf16, bool nv, cudaStream_t s) {
  const int64_t kb = (a.cols + 255) / 256, grid = (a.n_rows * kb + kThreads / 16 - 1) / (kThreads / 16);
  a.wide = (reinterpret_cast<uintptr_t>(a.out) & 15u) == 0 && (a.n_rows <= 1 || a.out_stride % (bf16 ? 8 : 4) == 0);
  const unsigned g = static_cast<unsigned>(grid), k = static_cast<unsigned>(kb);
  if (bf16) {
    if (nv) k_fp4_dequant<__nv_bfloat16, true><<<g, kThreads, 0, s>>>(a, k);
    else k_fp4_dequant<__nv_bfloat16, false><<<g, kThreads, 0, s>>>(a, k);
  } else {
    if (nv) k_fp4_dequant<float, true><<<g, kThreads, 0, s>>>(a, k);
    else k_fp4_dequant<float, false><<<g, kThreads, 0, s>>>(a, k);
  }
  return cudaGetLastError();
}

}  // namespace epoch
