// Quantisation to 4-bit floating point (e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) with
// a scale for each block of consecutive columns, of rows (optionally gathered by a worklist, or the
// SwiGLU of a gate | up pair) and of weight matrices, and back.
//
//   nvfp4: blocks of 16, v' = v * (1 / t) for a tensor scale t, s = e4m3(min(max|v'| / 6, 448)), at least
//          2^-9 (the smallest e4m3 value: a block of zeros divides by it), q = e2m1(v' / s)
//   mxfp4: blocks of 32, s = 2^(floor(log2 max|v|) - 2) within e8m0's range, q = e2m1(v / s)
//
// Both roundings are to nearest even of the exact quotients: a border between two codes times s, or
// between two scales times 6, is exact in fp32, and a quotient next to a border is decided by the
// remainder's sign. A block that holds a NaN or an infinity gets a NaN scale, so that every
// product with it is NaN. Scales lie by blocks of 256 columns, [ceil(K / 256)][rows][16 or 8], with
// zeros behind the last column.
//
// One pass: a thread keeps its columns (32, or 8 of them where few blocks leave places on the device empty) in registers, and lanes
// that share a block exchange its maximum. Bound by the instructions of the exact rounding (70 % of the issue slots), the
// way back by latency: 8192 rows of 2048 gathered from bf16 to nvfp4 and back take 14.4 us (about 7 each way), their bytes
// 5.8 (2 and 6.4 by themselves). Weights, 256 x 1024 x 2048 in bf16: mxfp4 193 us (7.1 TB/s), nvfp4 631, whose tensor scales
// cost a pass before, and whose quotients by any power of two the exact rounding of fp32.
#include <cfloat>
#include <cmath>

#include <cuda_fp16.h>

#include "common.cuh"
#include "layer.h"

namespace epoch {

namespace {

constexpr int kThreads = 256;

// N words from global memory, in the widest accesses that `align` bytes allow (elements of T at the least). Accesses of
// 32 bytes take whole sectors however far apart the lanes' are.
template <typename T, int N> __device__ __forceinline__ void load_words(const T *p, int align, uint32_t (&w)[N]) {
  const char *at = reinterpret_cast<const char *>(p);
  if (N % 8 == 0 && align >= 32) {
#pragma unroll
    for (int h = 0; h + 8 <= N; h += 8)
      asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[h]), "=r"(w[h + 1]), "=r"(w[h + 2]), "=r"(w[h + 3]), "=r"(w[h + 4]), "=r"(w[h + 5]), "=r"(w[h + 6]),
                     "=r"(w[h + 7])
                   : "l"(at + 4 * h));
  } else if (align >= 16) {
#pragma unroll
    for (int h = 0; h < N; h += 4)
      asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[h]), "=r"(w[h + 1]), "=r"(w[h + 2]), "=r"(w[h + 3])
                   : "l"(at + 4 * h));
  } else if constexpr (sizeof(T) == 2) {
    const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = __ldg(q + 2 * i) | (static_cast<uint32_t>(__ldg(q + 2 * i + 1)) << 16);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t *>(p) + i);
  }
}
template <int N> __device__ __forceinline__ void store_words(void *p, int align, const uint32_t (&w)[N]) {
  char *at = static_cast<char *>(p);
  if (N % 8 == 0 && align >= 32) {
#pragma unroll
    for (int h = 0; h + 8 <= N; h += 8)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at + 4 * h), "r"(w[h]), "r"(w[h + 1]),
                   "r"(w[h + 2]), "r"(w[h + 3]), "r"(w[h + 4]), "r"(w[h + 5]), "r"(w[h + 6]), "r"(w[h + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int h = 0; h < N; h += 4) *reinterpret_cast<uint4 *>(at + 4 * h) = make_uint4(w[h], w[h + 1], w[h + 2], w[h + 3]);
  }
}
// Words of T as values.
template <typename T, int N> __device__ __forceinline__ void open_words(const uint32_t (&w)[N], float *v) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (sizeof(T) == 2) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      v[i] = __uint_as_float(w[i]);
    }
  }
}
// Bits of the largest magnitude of N values.
template <int N> __device__ __forceinline__ unsigned largest(const float *v) {
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
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

// Quotients decide between neighbours of few bits: codes meet at three bits, scales at five. They are taken to twelve
// bits, by factors that are off by a few steps of 2^-23, so that an exact quotient on a border is found there. A
// quotient that was near a border and not on it moves off it by the sign of its remainder (`rest`, exact).
__device__ __forceinline__ uint32_t to_twelve(float q) { return (__float_as_uint(q) + 0x800u) & 0xFFFFF000u; }
__device__ __forceinline__ float off_border(uint32_t b, float rest) {
  const float at = __uint_as_float(b);
  // away from zero where the dividend is beyond the border, towards it where it is short of it
  if (rest != 0.f && at != 0.f) b = (rest > 0.f) == (at > 0.f) ? b + 1u : b - 1u;
  return __uint_as_float(b);
}

__device__ __forceinline__ float open_e4m3(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(b)));
  return __low2float(*reinterpret_cast<const __half2 *>(&h));
}

// e4m3 of m / 6 (finite, >= 0), rounded once and kept within [2^-9, 448].
__device__ __forceinline__ uint32_t nv_scale(float m) {
  const uint32_t b = to_twelve(m * (1.0f / 6.0f));
  const float q = off_border(b, fmaf(-6.0f, __uint_as_float(b), m));
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.f), "f"(fmaxf(q, 0x1p-9f)));
  return two;
}

__device__ __forceinline__ float reciprocal_near(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

// Where a thread works: C columns of the blocks of 256 columns of rows, which threads take in order.
template <int C> struct Piece {
  unsigned row, kb;
  int part, c;
  __device__ explicit Piece(unsigned kb_n) {
    const unsigned at = blockIdx.x * (kThreads * C / 256) + threadIdx.x / (256 / C);  // less than 2^31 + 32
    row = at / kb_n;
    kb = at - row * kb_n;
    part = threadIdx.x & (256 / C - 1);
    c = static_cast<int>(kb * 256) + part * C;
  }
};

__device__ __noinline__ float silu_any(float g) { return silu(g); }
// silu(g) u of eight values, to the bit what the division gives (compared for every fp32 g). The quotient g / d, d = 1 + exp(-g), comes from a
// reciprocal improved once and the remainder of a first quotient, which rounds as the division does where nothing
// overflows or becomes subnormal (Markstein, Computation of elementary functions on the IBM RISC System/6000, 1990);
// other values take the division, whose branches for every element cost three times the kernel's time (6461 rows of
// 2784 columns to mxfp4: 58 us).
__device__ __forceinline__ void silu_of(float *v, const float *u) {
  float q[8];
  bool plain = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float g = v[i], size = fabsf(g), d = 1.0f + expf(-g);
    plain = plain && size < 1e30f && d < 1e30f && (size > 1e-25f || g == 0.0f);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    r = fmaf(fmaf(-d, r, 1.0f), r, r);
    q[i] = g * r;
    q[i] = g == 0.0f ? g : fmaf(fmaf(-d, q[i], g), r, q[i]);
  }
  if (!plain)
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = silu_any(v[i]);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = q[i] * u[i];
}

// C: 32 columns a thread where there are many (the work for a scale and for addresses is then shared by most), 8 where
// there are few (four times the threads). EXACT false: the elements have eight bits, so a quotient that is not on a
// border differs from it by 2^-8 of it or more, and the tensor scale is a power of two, which goes into the factor of
// the quotients.
template <typename T, bool NV, bool SWIGLU, bool EXACT, int C>
__global__ void __launch_bounds__(kThreads) k_fp4_quant(const Fp4QuantArgs a, unsigned kb_n, int align) {
  constexpr int kB = NV && C == 32 ? 2 : 1, kPer = C / kB;  // blocks of a thread and their columns here
  constexpr int kWords = C * static_cast<int>(sizeof(T)) / 4;
  const Piece<C> p(kb_n);
  const bool row_there = p.row < a.n_rows, in = row_there && p.c < a.cols;
  int64_t src = p.row;
  unsigned mat = 0;
  if (a.rows != nullptr && row_there) src = __ldg(a.rows + p.row);
  const bool bad = src < 0 || src >= a.n_src;  // never followed: its scales are NaN
  float v[C], inv = a.inv_scale;
  if (a.amax != nullptr && row_there) {
    mat = p.row / static_cast<unsigned>(a.mat_rows);
    inv = 1.0f / fp4_tensor_scale(a.amax[mat]);
  }
  uint32_t w[kWords];
#pragma unroll
  for (int i = 0; i < kWords; ++i) w[i] = 0u;
  const T *x = static_cast<const T *>(a.x) + src * a.x_stride + p.c;
  if (in && !bad) load_words(x, align, w);
  if constexpr (SWIGLU) {
    uint32_t y[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) y[i] = 0u;
    if (in && !bad) load_words(x + a.cols, align, y);
    float u[C];
    open_words<T>(w, v);
    open_words<T>(y, u);
#pragma unroll
    for (int i = 0; i < C; i += 8) silu_of(v + i, u + i);
  } else {
    open_words<T>(w, v);
  }
  unsigned m[kB];  // of v: a maximum times 1 / t is the maximum of the v'
#pragma unroll
  for (int b = 0; b < kB; ++b) {
    if constexpr (sizeof(T) == 2 && !SWIGLU) {
      uint32_t big = 0;  // largest magnitudes of the low and of the high halves
#pragma unroll
      for (int i = 0; i < kPer / 2; ++i) big = __vmaxu2(big, w[b * kPer / 2 + i] & 0x7FFF7FFFu);
      m[b] = max(big << 16, big & 0xFFFF0000u);
    } else {
      m[b] = largest<kPer>(v + b * kPer);
    }
    if constexpr (C == 8) {  // a block is two threads', or four
      m[b] = max(m[b], __shfl_xor_sync(0xffffffffu, m[b], 1));
      if constexpr (!NV) m[b] = max(m[b], __shfl_xor_sync(0xffffffffu, m[b], 2));
    }
  }
  if (!row_there) return;
  const int64_t rows = a.amax ? a.mat_rows : a.n_rows, block = (static_cast<int64_t>(mat) * kb_n + p.kb) * rows + (p.row - mat * rows);
  uint32_t code = 0u;
#pragma unroll
  for (int b = 0; b < kB; ++b) {
    const bool spoilt = m[b] >= 0x7F800000u || bad;
    float *y = v + b * kPer;
    if constexpr (NV) {
      const float most = __uint_as_float(m[b]) * inv;
      const uint32_t c = nv_scale(spoilt ? 0.f : fminf(most, FLT_MAX));
      const float s = open_e4m3(c), r = reciprocal_near(s) * (EXACT ? 1.0f : inv);
      if constexpr (EXACT) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) y[i] *= inv;
        if (most > FLT_MAX)  // beyond fp32: the largest codes, as beyond e4m3
#pragma unroll
          for (int i = 0; i < kPer; ++i) y[i] = fminf(fmaxf(y[i], -FLT_MAX), FLT_MAX);
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t t = to_twelve(y[i] * r);
        y[i] = EXACT ? off_border(t, fmaf(-__uint_as_float(t), s, y[i])) : __uint_as_float(t);
      }
      code |= (spoilt ? 0x7Fu : c) << (8 * b);
    } else {
      // floor(log2 m) - 2, biased by 127: the exponent field less two, for subnormal m the least
      const int e = max(static_cast<int>(m[b] >> 23) - 2, 0);
      const float scale = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);  // 2^(127 - e), normal for e <= 253
#pragma unroll
      for (int i = 0; i < kPer; ++i) y[i] *= scale;
      code = spoilt ? 0xFFu : e;
    }
  }
  if (!in) code = 0u;
  if constexpr (C == 32 && NV) reinterpret_cast<uint16_t *>(a.scales)[block * 8 + p.part] = static_cast<uint16_t>(code);
  else if constexpr (C == 32) a.scales[block * 8 + p.part] = static_cast<uint8_t>(code);
  else if constexpr (NV) { if ((p.part & 1) == 0) a.scales[block * 16 + (p.part >> 1)] = static_cast<uint8_t>(code); }
  else { if ((p.part & 3) == 0) a.scales[block * 8 + (p.part >> 2)] = static_cast<uint8_t>(code); }
  if (!in) return;
  uint8_t *q = a.q + (static_cast<int64_t>(p.row) * a.cols + p.c) / 2;
  if constexpr (C == 32) *reinterpret_cast<uint4 *>(q) = make_uint4(pack8(v), pack8(v + 8), pack8(v + 16), pack8(v + 24));
  else *reinterpret_cast<uint32_t *>(q) = pack8(v);
}

// Largest |x| of each matrix, as bit patterns (a NaN's are above infinity's).
template <typename T> __global__ void __launch_bounds__(kThreads) k_fp4_amax(const T *w, int64_t count, uint32_t *amax, int align) {
  __shared__ uint32_t s_max[kThreads / 32];
  const T *p = w + static_cast<int64_t>(blockIdx.y) * count;
  uint32_t m = 0;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * 8; i < count;
       i += static_cast<int64_t>(gridDim.x) * kThreads * 8) {
    uint32_t w[2 * sizeof(T)];
    float v[8];
    load_words(p + i, align, w);
    open_words<T>(w, v);
    m = max(m, largest<8>(v));
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

// In the order of k_fp4_quant. A code's value times its scale is exact in fp32 (mxfp4: an eighth of it, so that the largest
// are finite), and only then multiplied by the factor: zeros stay zeros whatever the scale and factor.
template <typename T, bool NV, int C>
__global__ void __launch_bounds__(kThreads) k_fp4_dequant(const Fp4DequantArgs a, unsigned kb_n) {
  constexpr int kCodes = C / 8, kWords = C * static_cast<int>(sizeof(T)) / 4;
  const Piece<C> p(kb_n);
  if (p.row >= a.n_rows || p.c >= a.cols) return;
  const unsigned mat = p.row / static_cast<unsigned>(a.mat_rows);
  const int64_t block = (static_cast<int64_t>(mat) * kb_n + p.kb) * a.mat_rows + (p.row - mat * a.mat_rows);
  const uint8_t *at = a.q + (static_cast<int64_t>(p.row) * a.cols + p.c) / 2;
  uint32_t q[kCodes], code;
  if constexpr (C == 32) {
    const uint4 u = __ldg(reinterpret_cast<const uint4 *>(at));
    q[0] = u.x, q[1] = u.y, q[2] = u.z, q[3] = u.w;
    code = NV ? __ldg(reinterpret_cast<const uint16_t *>(a.scales) + block * 8 + p.part) : __ldg(a.scales + block * 8 + p.part);
  } else {
    q[0] = __ldg(reinterpret_cast<const uint32_t *>(at));
    code = __ldg(a.scales + block * (NV ? 16 : 8) + (p.part >> (NV ? 1 : 2)));
  }
  float f = a.group_scale ? a.scale * __ldg(a.group_scale + mat) : a.scale;
  float s[2];
  if constexpr (NV) {
    s[0] = open_e4m3(code);
    s[1] = open_e4m3(code >> 8);
  } else {
    s[0] = s[1] = code == 0xFFu ? __uint_as_float(0x7FC00000u) : code ? __uint_as_float(code << 23) : 0x1p-127f;
    if (fabsf(f) < 0x1p120f) {  // (beyond it a value of 2^128 has an infinite product either way)
      f *= 8.f;
      s[0] = s[1] *= 0.125f;
    }
  }
  uint32_t o[kWords];
#pragma unroll
  for (int h = 0; h < kCodes; ++h) {
    uint32_t d[4];  // pairs in fp16, which holds e2m1's values
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(q[h]));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&d[j]));
      const float y0 = x.x * s[h / 2] * f, y1 = x.y * s[h / 2] * f;
      if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(y0, y1);
        o[4 * h + j] = *reinterpret_cast<const uint32_t *>(&t);
      } else {
        o[8 * h + 2 * j] = __float_as_uint(y0);
        o[8 * h + 2 * j + 1] = __float_as_uint(y1);
      }
    }
  }
  T *out = static_cast<T *>(a.out) + static_cast<int64_t>(p.row) * a.out_stride + p.c;
  if (a.align >= 16) {
    store_words(out, a.align, o);
  } else if constexpr (sizeof(T) == 2) {
    uint16_t *e = reinterpret_cast<uint16_t *>(out);
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      e[2 * i] = static_cast<uint16_t>(o[i]);
      e[2 * i + 1] = static_cast<uint16_t>(o[i] >> 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kWords; ++i) reinterpret_cast<uint32_t *>(out)[i] = o[i];
  }
}

// Whether threads of 32 columns still fill the device (several warps a scheduler).
bool many(int64_t blocks) { return blocks >= 64ll * num_sms(); }
unsigned ctas(int64_t blocks, int c) { return static_cast<unsigned>((blocks + kThreads * c / 256 - 1) / (kThreads * c / 256)); }
// Bytes on which every row and piece starts: 32, 16 or less.
int align_of(const void *p, int64_t rows, int64_t stride, int size) {
  const uintptr_t bits = reinterpret_cast<uintptr_t>(p) | (rows > 1 ? static_cast<uintptr_t>(stride * size) : 0u);
  return bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : 0;
}

template <typename T, bool NV, bool SWIGLU, bool EXACT> cudaError_t launch_one(const Fp4QuantArgs &a, int align, cudaStream_t s) {
  const int64_t kb = (a.cols + 255) / 256, blocks = a.n_rows * kb;
  const unsigned k = static_cast<unsigned>(kb);
  if (many(blocks)) k_fp4_quant<T, NV, SWIGLU, EXACT, 32><<<ctas(blocks, 32), kThreads, 0, s>>>(a, k, align);
  else k_fp4_quant<T, NV, SWIGLU, EXACT, 8><<<ctas(blocks, 8), kThreads, 0, s>>>(a, k, align);
  return cudaGetLastError();
}
template <typename T, bool NV> cudaError_t launch_back(const Fp4DequantArgs &a, cudaStream_t s) {
  const int64_t kb = (a.cols + 255) / 256, blocks = a.n_rows * kb;
  const unsigned k = static_cast<unsigned>(kb);
  if (many(blocks)) k_fp4_dequant<T, NV, 32><<<ctas(blocks, 32), kThreads, 0, s>>>(a, k);
  else k_fp4_dequant<T, NV, 8><<<ctas(blocks, 8), kThreads, 0, s>>>(a, k);
  return cudaGetLastError();
}
// Whether dividing by t only moves exponents (and the quotient's factor 1 / s / t stays in range).
bool power_of_two(float inv) {
  int e;
  return std::frexp(inv, &e) == 0.5f && e > -100 && e < 100;
}
template <typename T> cudaError_t launch_type(const Fp4QuantArgs &a, bool nv, int align, cudaStream_t s) {
  if (!nv) return a.swiglu ? launch_one<T, false, true, true>(a, align, s) : launch_one<T, false, false, true>(a, align, s);
  if (a.swiglu) return launch_one<T, true, true, true>(a, align, s);
  if constexpr (sizeof(T) == 2) {
    // (a matrix's own scale may be any power of two)
    if (a.amax == nullptr && power_of_two(a.inv_scale)) return launch_one<T, true, false, false>(a, align, s);
  }
  return launch_one<T, true, false, true>(a, align, s);
}

}  // namespace

cudaError_t launch_fp4_quant(const Fp4QuantArgs &a, bool bf16, bool nv, cudaStream_t s) {
  // (the up half of a SwiGLU starts a.cols elements on, a multiple of 64 bytes)
  const int align = align_of(a.x, a.n_src, a.x_stride, bf16 ? 2 : 4);
  return bf16 ? launch_type<__nv_bfloat16>(a, nv, align, s) : launch_type<float>(a, nv, align, s);
}

cudaError_t launch_fp4_quant_weight(Fp4QuantArgs a, int n_mats, bool bf16, bool nv, float *tensor_scales, cudaStream_t s) {
  uint32_t *amax = reinterpret_cast<uint32_t *>(tensor_scales);
  cudaError_t e = cudaMemsetAsync(amax, 0, sizeof(uint32_t) * n_mats, s);
  if (e != cudaSuccess) return e;
  const int64_t count = a.mat_rows * a.cols;  // a multiple of 32
  if (nv) {
    const bool aligned = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0;
    const int64_t want = (count / 8 + kThreads - 1) / kThreads, most = (8 * num_sms() + n_mats - 1) / n_mats;
    const dim3 grid(static_cast<unsigned>(want < most ? want : most), static_cast<unsigned>(n_mats));
    if (bf16) k_fp4_amax<<<grid, kThreads, 0, s>>>(static_cast<const __nv_bfloat16 *>(a.x), count, amax, aligned ? 16 : 0);
    else k_fp4_amax<<<grid, kThreads, 0, s>>>(static_cast<const float *>(a.x), count, amax, aligned ? 16 : 0);
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
  a.align = align_of(a.out, a.n_rows, a.out_stride, bf16 ? 2 : 4);
  if (bf16) return nv ? launch_back<__nv_bfloat16, true>(a, s) : launch_back<__nv_bfloat16, false>(a, s);
  return nv ? launch_back<float, true>(a, s) : launch_back<float, false>(a, s);
}

}  // namespace epoch
