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
// per-element gate, write r' and h'), so the bytes of the rows bound the time: 16384 rows
// of 4096 (fp32 r, r' and bf16 b, h') take 141 us at 5.7 TB/s; a few rows take the launch
// and two dependent sums, 2.0 us for norm_before of one row of 2048.
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

__device__ __forceinline__ Vec8<__nv_bfloat16> load_vec(const __nv_bfloat16 *p) {
  Vec8<__nv_bfloat16> v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.a.x), "=r"(v.a.y), "=r"(v.a.z), "=r"(v.a.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ Vec8<float> load_vec(const float *p) {
  Vec8<float> v;
  asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.a.x), "=f"(v.a.y), "=f"(v.a.z), "=f"(v.a.w)
               : "l"(p));
  asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.b.x), "=f"(v.b.y), "=f"(v.b.z), "=f"(v.b.w)
               : "l"(p + 4));
  return v;
}
__device__ __forceinline__ void unpack_vec(const Vec8<__nv_bfloat16> &u, float (&v)[8]) {
  unpack2(u.a.x, v[0], v[1]);
  unpack2(u.a.y, v[2], v[3]);
  unpack2(u.a.z, v[4], v[5]);
  unpack2(u.a.w, v[6], v[7]);
}
__device__ __forceinline__ void unpack_vec(const Vec8<float> &u, float (&v)[8]) {
  v[0] = u.a.x, v[1] = u.a.y, v[2] = u.a.z, v[3] = u.a.w;
  v[4] = u.b.x, v[5] = u.b.y, v[6] = u.b.z, v[7] = u.b.w;
}

// E consecutive elements at p as fp32: E = 8 with 16-byte loads, E = 1 scalar.
// Streamed: rows are read once and need no place in L1.
template <int E, typename T> __device__ __forceinline__ void load_row(const T *p, float (&v)[E]) {
  if constexpr (E == 8) unpack_vec(load_vec(p), v);
  else v[0] = to_f32(*p);
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
// row_sums: their slots in shared memory, two sets 32 apart that consecutive sums
// alternate between, so each needs one barrier). Every thread of the CTA calls it.
__device__ __forceinline__ float row_sum(float v, int warps, int w, float *row_sums, int &turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (warps == 1) return v;
  float *at = row_sums + 32 * turn;
  turn ^= 1;
  if (lane_id() == 0) at[w] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < warps; ++i) s += at[i];
  return s;
}

__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + expf(-g)); }

// A row belongs to `tpr` consecutive threads (whole warps); thread p of them holds columns
// E * (p + i * tpr) .. + E, i < VPT, in registers (VPT = 0: H is larger than
// the registers hold, and every pass reads the row again -- from L2 or L1, and
// only elements that the same thread writes at the end, so out may be r).
template <typename TA, typename TR, bool AFTER, int E, int VPT>
__global__ void __launch_bounds__(512, E == 8 && VPT <= 2 ? 2 : 1) k_block_norm(const NormArgs a, int tpr) {
  __shared__ float sums[64];
  int turn = 0;
  const int p = threadIdx.x % tpr;
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
        const float k = rsqrtf(row_sum(sq, warps, w, row_sums, turn) * inv_h + a.eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int c = E * p + i * step;
          if (on && c < a.hidden) scaled(c, r[i], k, a.weight, static_cast<TA *>(a.out) + row * a.out_stride);
        }
      } else {
        float k = 1.f;
        if (a.weight) k = rsqrtf(row_sum(sq, warps, w, row_sums, turn) * inv_h + a.eps);
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
          k = rsqrtf(row_sum(sq, warps, w, row_sums, turn) * inv_h + a.eps);
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
        k = rsqrtf(row_sum(sq, warps, w, row_sums, turn) * inv_h + a.eps);
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
          k2 = rsqrtf(row_sum(sq, warps, w, row_sums, turn) * inv_h + a.eps);
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

// Rows of at most 4096 columns: a CTA stays, every thread keeps its eight columns'
// parameters in registers (they cost more loads than the rows themselves: up to four
// fp32 values a column), and the next row is on its way while this one is summed up.
// VEC: the eight columns are neighbours and come in 16-byte loads. Else (rows of an odd
// length start anywhere) they lie tpr apart, so a warp's scalar loads are neighbours.
// FULL: the gate has a value for each row and column, and is read with the row.
// THREADS: scalar rows of up to 8192 columns take a CTA of up to 1024 threads each (vector
// rows gain nothing from that: 2432 of 8192 took 58 us so, 56 by short CTAs).
constexpr int kStayThreads = 512;

template <bool VEC, typename T> struct Row8;
template <typename T> struct Row8<true, T> {
  Vec8<T> v;
  __device__ __forceinline__ void load(const T *row, int c, int, int) { v = load_vec(row + c); }
  __device__ __forceinline__ void get(int, int, int, float (&o)[8]) const { unpack_vec(v, o); }
};
template <typename T> struct Row8<false, T> {
  T v[8];
  __device__ __forceinline__ void load(const T *row, int c, int tpr, int hidden) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j * tpr < hidden) v[j] = row[c + j * tpr];
  }
  __device__ __forceinline__ void get(int c, int tpr, int hidden, float (&o)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = c + j * tpr < hidden ? to_f32(v[j]) : 0.f;
  }
};

template <typename TA, typename TR, bool AFTER, bool FULL, bool VEC, int THREADS>
__global__ void __launch_bounds__(THREADS, VEC && THREADS == kStayThreads ? 2 : 1) k_block_norm_stay(const NormArgs a, int tpr) {
  __shared__ float sums[64];
  int turn = 0;
  const int p = threadIdx.x % tpr, c = VEC ? 8 * p : p;
  const int warps = tpr >> 5, w = p >> 5;
  float *row_sums = sums + (threadIdx.x >> 5) - w;
  const int rpb = blockDim.x / tpr;
  const float inv_h = 1.0f / static_cast<float>(a.hidden);
  const bool in = c < a.hidden;
  float wt[8], sc[8], nw[8], gt[8];
  auto params = [&](const void *from, float (&o)[8]) {
    if constexpr (VEC) {
      load_par<8>(from, a.par_bf16, c, o);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float one[1];
        if (c + j * tpr < a.hidden) {
          load_par<1>(from, a.par_bf16, c + j * tpr, one);
          o[j] = one[0];
        }
      }
    }
  };
  auto put = [&](auto *row, const float (&o)[8]) {
    if constexpr (VEC) {
      store_row<8>(row + c, o);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float one[1] = {o[j]};
        if (c + j * tpr < a.hidden) store_row<1>(row + c + j * tpr, one);
      }
    }
  };
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    wt[j] = gt[j] = 1.f;
    sc[j] = a.residual_scale;
    nw[j] = 0.f;
  }
  if (in) {
    if (a.weight) params(a.weight, wt);
    if constexpr (AFTER) {
      if (!FULL && a.gate_kind == 1) {
        params(a.gate, gt);
        if (a.gate_sigmoid) {
#pragma unroll
          for (int j = 0; j < 8; ++j) gt[j] = sigmoid(gt[j]);
        }
      }
      if (a.scale) params(a.scale, sc);
      if (a.next_weight) params(a.next_weight, nw);
    }
  }
  Row8<VEC, TR> r_next;
  Row8<VEC, TA> b_next, g_next;
  auto fetch = [&](int64_t row) {
    if (!in || row >= a.n_rows) return;
    r_next.load(static_cast<const TR *>(a.residual) + row * a.residual_stride, c, tpr, a.hidden);
    if constexpr (AFTER) b_next.load(static_cast<const TA *>(a.block) + row * a.block_stride, c, tpr, a.hidden);
    if constexpr (FULL) g_next.load(static_cast<const TA *>(a.gate) + row * a.gate_stride, c, tpr, a.hidden);
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * rpb;
  const int64_t mine = threadIdx.x / tpr;
  fetch(static_cast<int64_t>(blockIdx.x) * rpb + mine);
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * rpb; r0 < a.n_rows; r0 += step) {
    const int64_t row = r0 + mine;
    const bool on = in && row < a.n_rows;
    float r[8], b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = b[j] = 0.f;
    if (on) {
      r_next.get(c, tpr, a.hidden, r);
      if constexpr (AFTER) b_next.get(c, tpr, a.hidden, b);
    }
    float sq = 0.f, k = 1.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sq += AFTER ? b[j] * b[j] : r[j] * r[j];
    if constexpr (AFTER) {
      if constexpr (FULL) {
        float g[8];
        if (on) {
          g_next.get(c, tpr, a.hidden, g);
#pragma unroll
          for (int j = 0; j < 8; ++j) b[j] *= a.gate_sigmoid ? sigmoid(g[j]) : g[j];
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r[j] *= sc[j];
        b[j] *= FULL ? wt[j] : wt[j] * gt[j];
      }
    }
    fetch(row + step);
    if (!AFTER || a.weight) k = rsqrtf(row_sum(sq, warps, w, row_sums, turn) * inv_h + a.eps);
    if constexpr (!AFTER) {
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] *= k * wt[j];
      if (on) put(static_cast<TA *>(a.out) + row * a.out_stride, r);
    } else {
      sq = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r[j] = fmaf(b[j], k, r[j]);
        sq += r[j] * r[j];
      }
      if (on) put(static_cast<TR *>(a.out) + row * a.out_stride, r);
      if (a.next_weight) {
        k = rsqrtf(row_sum(on ? sq : 0.f, warps, w, row_sums, turn) * inv_h + a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] *= k * nw[j];
        if (on) put(static_cast<TA *>(a.next_out) + row * a.next_stride, r);
      }
    }
  }
}

template <typename TA, typename TR, bool AFTER, bool VEC, int THREADS>
cudaError_t launch_stay(const NormArgs &a, int tpr, cudaStream_t s) {
  const int rpb = THREADS / tpr, threads = tpr * rpb;
  const int64_t blocks = (a.n_rows + rpb - 1) / rpb;
  const int64_t most = static_cast<int64_t>(num_sms()) * (VEC && THREADS == kStayThreads ? 2 : 1);
  const unsigned grid = static_cast<unsigned>(blocks < most ? blocks : most);
  if (AFTER && a.gate_kind == 2) k_block_norm_stay<TA, TR, AFTER, AFTER, VEC, THREADS><<<grid, threads, 0, s>>>(a, tpr);
  else k_block_norm_stay<TA, TR, AFTER, false, VEC, THREADS><<<grid, threads, 0, s>>>(a, tpr);
  return cudaGetLastError();
}

template <typename TA, typename TR, bool AFTER, int E, int VPT>
cudaError_t launch(const NormArgs &a, int tpr, cudaStream_t s) {
  const int rpb = tpr < 128 ? 128 / tpr : 1, threads = tpr * rpb;
  const int64_t blocks = (a.n_rows + rpb - 1) / rpb;
  const int64_t most = static_cast<int64_t>(num_sms()) * (2048 / threads) * 8;
  k_block_norm<TA, TR, AFTER, E, VPT><<<static_cast<unsigned>(blocks < most ? blocks : most), threads, 0, s>>>(a, tpr);
  return cudaGetLastError();
}

template <typename TA, typename TR, bool AFTER, int E>
cudaError_t choose(const NormArgs &a, cudaStream_t s) {
  {
    // The staying CTAs pay for their parameters once, and eight columns a thread are the
    // shorter way through a row. Between one and three rows for each row's place on the
    // device their last turn is half empty. norm_after of bf16 z, fp32 r, a gate and h', us
    // by short CTAs / staying ones (n, the rows for a place):
    //   H = 2048   304, 1/2: 4.45 / 3.89    608, 1: 5.22 / 5.16   1216, 2: 7.57 / 7.83
    //             1824, 3: 12.96 / 10.60   2432, 4: 15.39 / 13.16   9728, 16: 47.3 / 42.0
    //   H = 4096   152, 1/2: 4.53 / 3.90    608, 2: 7.76 / 8.22    912, 3: 13.41 / 11.24
    // Scalar rows stay always: 20000 of 1001 take 175 / 69, 1216 of 2047 27 / 10, 2432 of 5761 176 / 104.
    const int wide = (a.hidden + 255) / 256 * 32;
    if (wide <= kStayThreads) {
      const int64_t places = 2ll * num_sms() * (kStayThreads / wide);
      if (E == 1 || a.n_rows <= places || a.n_rows >= 3 * places)
        return launch_stay<TA, TR, AFTER, E == 8, kStayThreads>(a, wide, s);
    }
    if constexpr (E == 1)
      if (wide <= 2 * kStayThreads) return launch_stay<TA, TR, AFTER, false, 2 * kStayThreads>(a, wide, s);
  }
  // threads of a row: whole warps, enough for 16 values each; more values from 16 warps on
  const int want = (a.hidden + 511) / 512 * 32, tpr = want < 512 ? want : 512;
  const int64_t vpt = (a.hidden + static_cast<int64_t>(tpr) * E - 1) / (static_cast<int64_t>(tpr) * E);
  if constexpr (E == 8) {  // scalar rows of so few columns stay
    if (vpt == 1) return launch<TA, TR, AFTER, E, 1>(a, tpr, s);
    if (vpt == 2) return launch<TA, TR, AFTER, E, 2>(a, tpr, s);
  }
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
