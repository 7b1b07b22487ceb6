// RMS norms before and after a block, fused with the block's gate, the
// residual scale and the next block's norm.
//
//   before:  h  = rms(x) * w
//   after:   r' = s * r + g * z,   z = rms(b) * w   (w absent: z = b)
//            h' = rms(r') * w_next (w_next present), from r' before its rounding
//   rms(v) = v / sqrt(mean(v^2) + eps)
//
// Every value is held in fp32 from its load to its store: one rounding per
// output. Rows are independent and move through registers once (read r, b and a
// per-element gate, write r' and h'), so the bytes of the rows bound the time.
#include <cmath>

#include "common.cuh"
#include "layer.h"

namespace epoch {

namespace {

template <typename T> struct Vec8;  // eight consecutive elements
template <> struct Vec8<__nv_bfloat16> {
  uint4 a;
};
template <> struct Vec8<float> {
  float4 a, b;
};

__device__ __forceinline__ void unpack2(uint32_t u, float &lo, float &hi) {
  lo = __uint_as_float(u << 16);
  hi = __uint_as_float(u & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// E consecutive elements at p as fp32: E = 8 with 16-byte loads, E = 1 scalar.
// Streamed: rows are read once and need no place in L1.
template <int E> __device__ __forceinline__ void load_row(const __nv_bfloat16 *p, float (&v)[E]) {
  if constexpr (E == 8) {
    uint4 u;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(p));
    unpack2(u.x, v[0], v[1]);
    unpack2(u.y, v[2], v[3]);
    unpack2(u.z, v[4], v[5]);
    unpack2(u.w, v[6], v[7]);
  } else {
    v[0] = __bfloat162float(*p);
  }
}
template <int E> __device__ __forceinline__ void load_row(const float *p, float (&v)[E]) {
  if constexpr (E == 8) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v[4 * h]), "=f"(v[4 * h + 1]), "=f"(v[4 * h + 2]), "=f"(v[4 * h + 3])
                   : "l"(p + 4 * h));
  } else {
    v[0] = *p;
  }
}
template <int E> __device__ __forceinline__ void store_row(__nv_bfloat16 *p, const float (&v)[E]) {
  if constexpr (E == 8)
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
  else
    *p = __float2bfloat16_rn(v[0]);
}
template <int E> __device__ __forceinline__ void store_row(float *p, const float (&v)[E]) {
  if constexpr (E == 8) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *p = v[0];
  }
}
// Per-channel parameters, fp32 or bf16; every row reads them, so they stay cached.
template <int E> __device__ __forceinline__ void load_par(const void *p, int bf16, int c, float (&v)[E]) {
  if constexpr (E == 8) {
    if (bf16) {
      const uint4 u = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + c));
      unpack2(u.x, v[0], v[1]);
      unpack2(u.y, v[2], v[3]);
      unpack2(u.z, v[4], v[5]);
      unpack2(u.w, v[6], v[7]);
    } else {
      const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + c);
      const float4 a = __ldg(q), b = __ldg(q + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
  } else {
    v[0] = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[c]) : static_cast<const float *>(p)[c];
  }
}

// Sum of v over the `warps` warps of this thread's row (warp `w` of them;
// row_sums: their slots in shared memory). Every thread of the CTA calls it.
__device__ __forceinline__ float row_sum(float v, int warps, int w, float *row_sums) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (warps == 1) return v;
  if (lane_id() == 0) row_sums[w] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < warps; ++i) s += row_sums[i];
  __syncthreads();
  return s;
}

__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + expf(-g)); }

// A row belongs to `tpr` consecutive threads; thread p of them holds columns
// E * (p + i * tpr) .. + E, i < VPT, in registers (VPT = 0: H is larger than
// the registers hold, and every pass reads the row again -- from L2 or L1, and
// only elements that the same thread writes at the end, so out may be r).
template <typename TA, typename TR, bool AFTER, int E, int VPT>
__global__ void __launch_bounds__(512, E * VPT <= 16 ? 2 : 1) k_block_norm(const NormArgs a, int tpr) {
  __shared__ float sums[32];
  const int p = threadIdx.x & (tpr - 1);
  const int warps = tpr >> 5, w = p >> 5;
  float *row_sums = sums + (threadIdx.x >> 5) - w;
  const int rpb = blockDim.x / tpr;
  const float inv_h = 1.0f / static_cast<float>(a.hidden);
  const int step = E * tpr;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * rpb; r0 < a.n_rows; r0 += static_cast<int64_t>(gridDim.x) * rpb) {
    const int64_t row = r0 + threadIdx.x / tpr;
    const bool on = row < a.n_rows;
    const TR *res = static_cast<const TR *>(a.residual) + row * a.residual_stride;
    const TA *blk = static_cast<const TA *>(a.block) + row * a.block_stride;
    const TA *gate = static_cast<const TA *>(a.gate) + (a.gate_kind == 2 ? row * a.gate_stride : 0);
    // r' of columns c .. c + E from the block's values and the row's factor
    auto merge = [&](int c, const float (&b)[E], const float (&r)[E], float k, float (&o)[E]) {
      float z[E], t[E];
#pragma unroll
      for (int j = 0; j < E; ++j) z[j] = b[j];
      if (a.weight) {
        load_par<E>(a.weight, a.par_bf16, c, t);
#pragma unroll
        for (int j = 0; j < E; ++j) z[j] = z[j] * k * t[j];
      }
      if (a.gate_kind) {
        if (a.gate_kind == 2) load_row<E>(gate + c, t);
        else load_par<E>(a.gate, a.par_bf16, c, t);
        if (a.gate_sigmoid) {
#pragma unroll
          for (int j = 0; j < E; ++j) t[j] = sigmoid(t[j]);
        }
#pragma unroll
        for (int j = 0; j < E; ++j) z[j] *= t[j];
      }
      if (a.scale) {
        load_par<E>(a.scale, a.par_bf16, c, t);
#pragma unroll
        for (int j = 0; j < E; ++j) o[j] = r[j] * t[j] + z[j];
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j) o[j] = r[j] * a.residual_scale + z[j];
      }
    };
    auto scaled = [&](int c, const float (&v)[E], float k, const void *weight, TA *dst) {
      float t[E], o[E];
      load_par<E>(weight, a.par_bf16, c, t);
#pragma unroll
      for (int j = 0; j < E; ++j) o[j] = v[j] * k * t[j];
      store_row<E>(dst + c, o);
    };
    if constexpr (VPT > 0) {
      float r[VPT][E], b[AFTER ? VPT : 1][E];
      float sq = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = E * p + i * step;
        const bool in = on && c < a.hidden;
#pragma unroll
        for (int j = 0; j < E; ++j) r[i][j] = 0.f;
        if (in) load_row<E>(res + c, r[i]);
        if constexpr (AFTER) {
#pragma unroll
          for (int j = 0; j < E; ++j) b[i][j] = 0.f;
          if (in) load_row<E>(blk + c, b[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < E; ++j) {
          const float v = AFTER ? b[AFTER ? i : 0][j] : r[i][j];
          sq += v * v;
        }
      if constexpr (!AFTER) {
        const float k = rsqrtf(row_sum(sq, warps, w, row_sums) * inv_h + a.eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int c = E * p + i * step;
          if (on && c < a.hidden) scaled(c, r[i], k, a.weight, static_cast<TA *>(a.out) + row * a.out_stride);
        }
      } else {
        float k = 1.f;
        if (a.weight) k = rsqrtf(row_sum(sq, warps, w, row_sums) * inv_h + a.eps);
        sq = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int c = E * p + i * step;
          if (!on || c >= a.hidden) continue;
          float o[E];
          merge(c, b[i], r[i], k, o);
          store_row<E>(static_cast<TR *>(a.out) + row * a.out_stride + c, o);
#pragma unroll
          for (int j = 0; j < E; ++j) {
            r[i][j] = o[j];
            sq += o[j] * o[j];
          }
        }
        if (a.next_weight) {
          k = rsqrtf(row_sum(sq, warps, w, row_sums) * inv_h + a.eps);
#pragma unroll
          for (int i = 0; i < VPT; ++i) {
            const int c = E * p + i * step;
            if (on && c < a.hidden)
              scaled(c, r[i], k, a.next_weight, static_cast<TA *>(a.next_out) + row * a.next_stride);
          }
        }
      }
    } else {
      float v[E], b[E], o[E];
      float k = 1.f, sq = 0.f;
      if (!AFTER || a.weight) {
        for (int c = E * p; on && c < a.hidden; c += step) {
          if constexpr (AFTER) load_row<E>(blk + c, v);
          else load_row<E>(res + c, v);
#pragma unroll
          for (int j = 0; j < E; ++j) sq += v[j] * v[j];
        }
        k = rsqrtf(row_sum(sq, warps, w, row_sums) * inv_h + a.eps);
      }
      if constexpr (!AFTER) {
        for (int c = E * p; on && c < a.hidden; c += step) {
          load_row<E>(res + c, v);
          scaled(c, v, k, a.weight, static_cast<TA *>(a.out) + row * a.out_stride);
        }
      } else {
        float k2 = 0.f;
        if (a.next_weight) {
          sq = 0.f;
          for (int c = E * p; on && c < a.hidden; c += step) {
            load_row<E>(blk + c, b);
            load_row<E>(res + c, v);
            merge(c, b, v, k, o);
#pragma unroll
            for (int j = 0; j < E; ++j) sq += o[j] * o[j];
          }
          k2 = rsqrtf(row_sum(sq, warps, w, row_sums) * inv_h + a.eps);
        }
        for (int c = E * p; on && c < a.hidden; c += step) {
          load_row<E>(blk + c, b);
          load_row<E>(res + c, v);
          merge(c, b, v, k, o);
          store_row<E>(static_cast<TR *>(a.out) + row * a.out_stride + c, o);
          if (a.next_weight) scaled(c, o, k2, a.next_weight, static_cast<TA *>(a.next_out) + row * a.next_stride);
        }
      }
    }
  }
}

template <typename TA, typename TR, bool AFTER, int E, int VPT>
cudaError_t launch(const NormArgs &a, int tpr, cudaStream_t s) {
  const int threads = tpr < 128 ? 128 : tpr;
  const int rpb = threads / tpr;
  const int64_t blocks = (a.n_rows + rpb - 1) / rpb;
  const int64_t most = static_cast<int64_t>(num_sms()) * (2048 / threads) * 8;
  k_block_norm<TA, TR, AFTER, E, VPT><<<static_cast<unsigned>(blocks < most ? blocks : most), threads, 0, s>>>(a, tpr);
  return cudaGetLastError();
}

template <typename TA, typename TR, bool AFTER, int E>
cudaError_t choose(const NormArgs &a, cudaStream_t s) {
  // threads of a row: enough for 16 values each; 32 values each from 16 warps on
  const int64_t per = 16;
  int tpr = 32;
  while (tpr < 512 && tpr * per < a.hidden) tpr *= 2;
  const int64_t vpt = (a.hidden + static_cast<int64_t>(tpr) * E - 1) / (static_cast<int64_t>(tpr) * E);
  if (vpt * E <= 8) return launch<TA, TR, AFTER, E, 8 / E>(a, tpr, s);
  if (vpt * E <= 16) return launch<TA, TR, AFTER, E, 16 / E>(a, tpr, s);
  if (vpt * E <= 32) return launch<TA, TR, AFTER, E, 32 / E>(a, tpr, s);
  return launch<TA, TR, AFTER, E, 0>(a, 512, s);
}

template <bool AFTER, int E> cudaError_t by_type(const NormArgs &a, cudaStream_t s) {
  using bf = __nv_bfloat16;
  if (a.act_bf16) return a.res_bf16 ? choose<bf, bf, AFTER, E>(a, s) : choose<bf, float, AFTER, E>(a, s);
  return a.res_bf16 ? choose<float, bf, AFTER, E>(a, s) : choose<float, float, AFTER, E>(a, s);
}

// Eight elements of a row are loaded at once where every row of the tensor
// starts on a 16-byte boundary.
bool wide(const void *p, int64_t stride, int64_t n_rows, bool bf16) {
  const int64_t per16 = bf16 ? 8 : 4;
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (n_rows <= 1 || stride % per16 == 0));
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs &a, bool after, cudaStream_t s) {
  const bool w8 = a.hidden % 8 == 0 && wide(a.block, a.block_stride, a.n_rows, a.act_bf16) &&
                  wide(a.residual, a.residual_stride, a.n_rows, a.res_bf16) &&
                  wide(a.weight, 0, 1, a.par_bf16) && wide(a.scale, 0, 1, a.par_bf16) &&
                  wide(a.next_weight, 0, 1, a.par_bf16) &&
                  (a.gate_kind == 2 ? wide(a.gate, a.gate_stride, a.n_rows, a.act_bf16)
                                    : wide(a.gate, 0, 1, a.par_bf16)) &&
                  wide(a.out, a.out_stride, a.n_rows, after ? a.res_bf16 : a.act_bf16) &&
                  wide(a.next_out, a.next_stride, a.n_rows, a.act_bf16);
  if (after) return w8 ? by_type<true, 8>(a, s) : by_type<true, 1>(a, s);
  return w8 ? by_type<false, 8>(a, s) : by_type<false, 1>(a, s);
}

}  // namespace epoch
