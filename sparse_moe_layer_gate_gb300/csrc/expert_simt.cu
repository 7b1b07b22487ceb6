// fp32 products of the routed experts, grouped by expert, on the FFMA pipes (the tensor cores have no
// fp32 operands, and TF32's ten bits would lose what an fp32 layer keeps). The formula is that of
// expert_gemm.cu; sums are fp32, in ascending k.
//
// Tiles of 128 or 32 rows x 128 columns, sixteen columns of K at a time through two places in shared
// memory, each thread 8 (2) x 8 sums as pairs for the packed fp32 multiply-add. With swiglu a tile's
// columns are 64 gate and 64 up rows of the weights: a thread's columns 4 and 4 of them. Short tiles
// where groups have few rows. Bound by the FFMA pipes at many rows.
#include "common.cuh"
#include "layer.h"
#include "tiles.cuh"

namespace epoch {

namespace {

constexpr int kCols = 128, kDepth = 16, kThreads = 256, kPad = 4;

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ void fma2(uint64_t &acc, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}

template <int ROWS> __global__ void __launch_bounds__(kThreads) k_expert_simt(const ExpertGemmArgs a, int nt_n) {
  constexpr int TM = ROWS / 16;                      // rows of a thread
  constexpr int LA = ROWS * kDepth / 4 / kThreads;   // float4 loads of a thread for the rows (ROWS 32: half the threads)
  constexpr int LB = kCols * kDepth / 4 / kThreads;
  __shared__ __align__(16) float s_a[2][kDepth][ROWS + kPad], s_b[2][kDepth][kCols + kPad];
  __shared__ int s_start[kMaxGroups + 1], s_cum[kMaxGroups + 1];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  if (a.offsets != nullptr) {
    if (warp_id() == 0) group_tiles(a.offsets, a.n_groups, a.m, ROWS, s_start, s_cum);
  } else if (tid == 0) {
    s_start[0] = 0;
    s_start[1] = a.m;
    s_cum[0] = 0;
    s_cum[1] = (a.m + ROWS - 1) / ROWS;
  }
  __syncthreads();
  TileWalk walk(s_start, s_cum, a.offsets ? a.n_groups : 1, nt_n, ROWS, 0);
  const int half_n = a.N / 2, out_n = a.swiglu ? half_n : a.N;
  const float *x = static_cast<const float *>(a.a), *w = static_cast<const float *>(a.b);
  for (int t = blockIdx.x; t < walk.total; t += gridDim.x) {
    int e, row0, rows, nt;
    walk.at(t, &e, &row0, &rows, &nt);
    rows = min(rows, ROWS);
    // where this thread's pieces come from: rows and weights that do not exist are zeros
    const float *pa[LA > 0 ? LA : 1], *pb[LB];
    const int kq = (tid & 3) * 4;  // columns of K
#pragma unroll
    for (int i = 0; i < (LA > 0 ? LA : 1); ++i) {
      const int r = (tid >> 2) + 64 * i;
      pa[i] = nullptr;
      if (r < rows) {
        int64_t src = row0 + r;
        if (a.rows != nullptr) src = __ldg(a.rows + row0 + r);
        if (a.rows == nullptr || (src >= 0 && src < a.n_src)) pa[i] = x + src * a.a_stride + kq;
      }
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
      const int j = (tid >> 2) + 64 * i;
      const int n = !a.swiglu ? nt * kCols + j : j < 64 ? nt * 64 + j : half_n + nt * 64 + j - 64;
      const bool there = a.swiglu ? nt * 64 + (j & 63) < half_n : n < a.N;
      pb[i] = there ? w + (static_cast<int64_t>(e) * a.N + n) * a.K + kq : nullptr;
    }
    float4 ra[LA > 0 ? LA : 1], rb[LB];
    auto load = [&](int k0) {
      const bool in = k0 + kq < a.K;
#pragma unroll
      for (int i = 0; i < (LA > 0 ? LA : 1); ++i)
        ra[i] = in && pa[i] ? __ldg(reinterpret_cast<const float4 *>(pa[i] + k0)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < LB; ++i)
        rb[i] = in && pb[i] ? __ldg(reinterpret_cast<const float4 *>(pb[i] + k0)) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    auto put = [&](int s) {
#pragma unroll
      for (int i = 0; i < (LA > 0 ? LA : 1); ++i) {
        const int r = (tid >> 2) + 64 * i;
        if (ROWS >= 64 || r < ROWS) {
          s_a[s][kq][r] = ra[i].x, s_a[s][kq + 1][r] = ra[i].y, s_a[s][kq + 2][r] = ra[i].z, s_a[s][kq + 3][r] = ra[i].w;
        }
      }
#pragma unroll
      for (int i = 0; i < LB; ++i) {
        const int j = (tid >> 2) + 64 * i;
        s_b[s][kq][j] = rb[i].x, s_b[s][kq + 1][j] = rb[i].y, s_b[s][kq + 2][j] = rb[i].z, s_b[s][kq + 3][j] = rb[i].w;
      }
    };
    uint64_t acc[TM][4];  // columns 4 tx .. + 3 and 64 + 4 tx .. + 3, in pairs
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0ull;
    load(0);
    __syncthreads();  // the tile before has been read
    put(0);
    const int steps = (a.K + kDepth - 1) / kDepth;
    for (int s = 0; s < steps; ++s) {
      if (s + 1 < steps) load((s + 1) * kDepth);
      __syncthreads();
      const int b = s & 1;
#pragma unroll
      for (int k = 0; k < kDepth; ++k) {
        const float4 b0 = *reinterpret_cast<const float4 *>(&s_b[b][k][4 * tx]);
        const float4 b1 = *reinterpret_cast<const float4 *>(&s_b[b][k][64 + 4 * tx]);
        const uint64_t bb[4] = {pack2(b0.x, b0.y), pack2(b0.z, b0.w), pack2(b1.x, b1.y), pack2(b1.z, b1.w)};
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const float v = s_a[b][k][ty * TM + i];
          const uint64_t vv = pack2(v, v);
#pragma unroll
          for (int j = 0; j < 4; ++j) fma2(acc[i][j], vv, bb[j]);
        }
      }
      if (s + 1 < steps) put(b ^ 1);
    }
    float f = a.scale;
    if (a.group_scale != nullptr) f *= __ldg(a.group_scale + e);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int r = ty * TM + i;
      if (r >= rows) continue;
      float fr = f;
      if (a.rows != nullptr) {
        const int src = __ldg(a.rows + row0 + r);
        if (src < 0 || src >= a.n_src) fr = __uint_as_float(0x7FC00000u);
      }
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 u = unpack2(acc[i][j]);
        v[2 * j] = u.x * fr;
        v[2 * j + 1] = u.y * fr;
      }
      const int64_t at = static_cast<int64_t>(row0 + r) * a.out_stride;
      auto put_out = [&](int n, float y) {
        if (n >= out_n) return;
        if (a.out_bf16) static_cast<__nv_bfloat16 *>(a.out)[at + n] = __float2bfloat16_rn(y);
        else static_cast<float *>(a.out)[at + n] = y;
      };
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (a.swiglu) {
          put_out(nt * 64 + 4 * tx + j, silu(v[j]) * v[4 + j]);
        } else {
          put_out(nt * kCols + 4 * tx + j, v[j]);
          put_out(nt * kCols + 64 + 4 * tx + j, v[4 + j]);
        }
      }
    }
  }
}

template <int ROWS> cudaError_t launch_rows(const ExpertGemmArgs &a, cudaStream_t s) {
  const int nt = (a.N + kCols - 1) / kCols;  // with swiglu 64 columns of each half
  const int64_t groups = a.n_groups < a.m ? a.n_groups : a.m;
  const int64_t tiles = (a.offsets ? a.m / ROWS + groups : (a.m + ROWS - 1) / ROWS) * nt;
  const int64_t most = 4ll * num_sms();
  k_expert_simt<ROWS><<<static_cast<unsigned>(tiles < most ? tiles : most), kThreads, 0, s>>>(a, nt);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert_simt(const ExpertGemmArgs &a, cudaStream_t s) {
  const int64_t groups = a.offsets ? a.n_groups : 1;
  return a.m <= 64 * groups ? launch_rows<32>(a, s) : launch_rows<128>(a, s);
}

}  // namespace epoch
