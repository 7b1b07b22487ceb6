// fp32 products of the routed experts, grouped by expert, on the FFMA pipes (the tensor cores have no
// fp32 operands, and TF32's ten bits would lose what an fp32 layer keeps). The formula is that of
// expert_gemm.cu; sums are fp32, in ascending k.
//
// Many rows (k_expert_simt): tiles of 128 or 64 rows x 128 columns, sixteen columns of K at a time through two
// places in shared memory, each thread 8 or 4 x 8 sums as pairs for the packed fp32 multiply-add. With swiglu a
// tile's columns are 64 gate and 64 up rows of the weights: a thread's columns 4 and 4 of them. Bound by
// the FFMA pipes (8192 x 2048 x 2048 over 8 experts 1.44 ms, 48 TFLOP/s).
//
// Few rows (k_expert_stream): bound by the weights' bytes and by latency. A warp takes four rows of weights
// (two gate and two up) and eight tokens: its lanes share K out, each keeps all 32 sums, and the sums meet
// by exchanges that halve them at every step.
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
  constexpr int TM = ROWS / 16;                     // rows of a thread
  constexpr int LA = ROWS * kDepth / 4 / kThreads;  // float4 loads of a thread for the rows
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
    const float *pa[LA], *pb[LB];
    const int kq = (tid & 3) * 4;  // columns of K
#pragma unroll
    for (int i = 0; i < LA; ++i) {
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
    float4 ra[LA], rb[LB];
    auto load = [&](int k0) {
      const bool in = k0 + kq < a.K;
#pragma unroll
      for (int i = 0; i < LA; ++i)
        ra[i] = in && pa[i] ? __ldg(reinterpret_cast<const float4 *>(pa[i] + k0)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < LB; ++i)
        rb[i] = in && pb[i] ? __ldg(reinterpret_cast<const float4 *>(pb[i] + k0)) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    auto put = [&](int s) {
#pragma unroll
      for (int i = 0; i < LA; ++i) {
        const int r = (tid >> 2) + 64 * i;
        s_a[s][kq][r] = ra[i].x, s_a[s][kq + 1][r] = ra[i].y, s_a[s][kq + 2][r] = ra[i].z, s_a[s][kq + 3][r] = ra[i].w;
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

constexpr int kTokens = 8;  // rows of a warp's unit

// The sums of 2^n values that every lane holds a part of: lane l ends with value l >> (5 - n) of them, by exchanges in
// which each lane passes half of its values on.
template <int N> __device__ __forceinline__ float meet(float (&v)[N]) {
  const int lane = lane_id();
  int o = 16;
#pragma unroll
  for (int n = N / 2; n >= 1; n /= 2, o /= 2) {
    const bool high = lane & o;
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const float send = high ? v[j] : v[j + n], keep = high ? v[j + n] : v[j];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
#pragma unroll
  for (; o >= 1; o /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}

// One unit with at most R tokens.
template <int R>
__device__ __forceinline__ void stream_unit(const ExpertGemmArgs &a, int e, int row0, int rows, int nt) {
  const int lane = lane_id(), warp = warp_id(), half_n = a.N / 2, out_n = a.swiglu ? half_n : a.N;
  const float *x = static_cast<const float *>(a.n_src > 0 ? a.a : a.b);
  const float *px[R], *pw[4];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    int64_t src = row0 + min(r, rows - 1);  // (rows that do not exist repeat one that does)
    if (a.rows != nullptr) src = __ldg(a.rows + src);
    if (src < 0 || src >= a.n_src) src = 0;  // never followed; the result is NaN
    px[r] = x + src * a.a_stride;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = a.swiglu ? (i & 2 ? half_n : 0) + min(nt * 16 + warp * 2 + (i & 1), half_n - 1) : min(nt * 32 + warp * 4 + i, a.N - 1);
    pw[i] = static_cast<const float *>(a.b) + (static_cast<int64_t>(e) * a.N + n) * a.K;
  }
  uint64_t acc[4][R];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < R; ++r) acc[i][r] = 0ull;
#pragma unroll 2
  for (int k = lane * 4; k < a.K; k += 128) {
    float4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(w[i].x), "=f"(w[i].y), "=f"(w[i].z), "=f"(w[i].w) : "l"(pw[i] + k));
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float4 v = __ldg(reinterpret_cast<const float4 *>(px[r] + k));
      const uint64_t lo = pack2(v.x, v.y), hi = pack2(v.z, v.w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        fma2(acc[i][r], pack2(w[i].x, w[i].y), lo);
        fma2(acc[i][r], pack2(w[i].z, w[i].w), hi);
      }
    }
  }
  float v[4 * R];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float2 f = unpack2(acc[i][r]);
      v[i * R + r] = f.x + f.y;
    }
  float y = meet(v);
  constexpr int kSame = 32 / (4 * R);  // lanes with the same value
  const int at = lane / kSame, i = at / R, r = at % R;
  float f = a.scale;
  if (a.group_scale != nullptr) f *= __ldg(a.group_scale + e);
  if (a.rows != nullptr && r < rows) {
    const int src = __ldg(a.rows + row0 + r);
    if (src < 0 || src >= a.n_src) f = __uint_as_float(0x7FC00000u);
  }
  y *= f;
  int n = nt * 32 + warp * 4 + i;
  if (a.swiglu) {
    const float up = __shfl_xor_sync(0xffffffffu, y, 16);  // rows 2 and 3 are the up rows of 0 and 1
    y = silu(y) * up;
    n = i < 2 ? nt * 16 + warp * 2 + i : out_n;
  }
  if (lane % kSame != 0 || r >= rows || n >= out_n) return;
  const int64_t to = static_cast<int64_t>(row0 + r) * a.out_stride + n;
  if (a.out_bf16) static_cast<__nv_bfloat16 *>(a.out)[to] = __float2bfloat16_rn(y);
  else static_cast<float *>(a.out)[to] = y;
}

__global__ void __launch_bounds__(kThreads, 2) k_expert_stream(const ExpertGemmArgs a, int nt_n) {
  __shared__ int s_start[kMaxGroups + 1], s_cum[kMaxGroups + 1];
  if (a.offsets != nullptr) {
    if (warp_id() == 0) group_tiles(a.offsets, a.n_groups, a.m, kTokens, s_start, s_cum);
  } else if (threadIdx.x == 0) {
    s_start[0] = 0;
    s_start[1] = a.m;
    s_cum[0] = 0;
    s_cum[1] = (a.m + kTokens - 1) / kTokens;
  }
  __syncthreads();
  TileWalk walk(s_start, s_cum, a.offsets ? a.n_groups : 1, nt_n, kTokens, 0);
  for (int t = blockIdx.x; t < walk.total; t += gridDim.x) {
    int e, row0, rows, nt;
    walk.at(t, &e, &row0, &rows, &nt);
    rows = min(rows, kTokens);
    if (rows == 1) stream_unit<1>(a, e, row0, rows, nt);
    else if (rows == 2) stream_unit<2>(a, e, row0, rows, nt);
    else if (rows <= 4) stream_unit<4>(a, e, row0, rows, nt);
    else stream_unit<8>(a, e, row0, rows, nt);
  }
}

}  // namespace

cudaError_t launch_expert_simt(const ExpertGemmArgs &a, cudaStream_t s) {
  const int64_t groups = a.offsets ? (a.n_groups < a.m ? a.n_groups : a.m) : 1, sms = num_sms();
  const int64_t nt = (a.N + kCols - 1) / kCols;  // with swiglu 64 columns of each half
  const int64_t nb = (a.N + 31) / 32;
  auto tiles = [&](int64_t rows) { return groups > 1 ? a.m / rows + groups : (a.m + rows - 1) / rows; };
  // The least of three estimates in nanoseconds. A step of 16 columns takes a tile of 64 rows 1000 (loads, and few CTAs)
  // or, with many, its SM 880 a tile; one of 128 rows 1700 or 1640; a unit of the streaming kernel some 6 and 0.0225 a column.
  // (us by streaming, 64 and 128 rows: 1024 x 512 x 512 39, 35, 57; 1315 rows over 17 experts of 152 x 352 18, 26, 40;
  // 2048 over 64 of 512 x 256 59, 33, 53; 8192 over 8 of 2048 x 2048 5197, 1573, 1437.)
  const double steps = (a.K + kDepth - 1) / kDepth;
  auto time_of = [&](int64_t rows, double one, double each) {
    const double many = each * static_cast<double>(tiles(rows) * nt) / static_cast<double>(sms);
    return 2000.0 + steps * (many > one ? many : one);
  };
  const double low = time_of(64, 1000.0, 880.0), tall = time_of(128, 1700.0, 1640.0);
  const double stream = 6000.0 + static_cast<double>(tiles(kTokens) * nb) * (6.0 + 0.0225 * a.K);
  auto grid = [&](int64_t n, int64_t most) { return static_cast<unsigned>(n < most ? n : most); };
  if (stream <= low && stream <= tall) k_expert_stream<<<grid(tiles(kTokens) * nb, 8 * sms), kThreads, 0, s>>>(a, static_cast<int>(nb));
  else if (low <= tall) k_expert_simt<64><<<grid(tiles(64) * nt, 4 * sms), kThreads, 0, s>>>(a, static_cast<int>(nt));
  else k_expert_simt<128><<<grid(tiles(128) * nt, 4 * sms), kThreads, 0, s>>>(a, static_cast<int>(nt));
  return cudaGetLastError();
}

}  // namespace epoch
