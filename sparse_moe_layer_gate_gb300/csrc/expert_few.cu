// Products of the routed experts on few rows: the formula of expert_gemm.cu, bf16 or 4-bit operands, where the
// weights' bytes and latency bound the time and the tensor cores idle either way.
//
// A CTA takes 16 rows of weights (with swiglu 8 gate and 8 up rows) and up to 16 rows of a group. Its eight warps
// share K out in pieces of 64 (bf16) or 256 columns, load both operands from global memory straight
// into the fragments of mma.sync.m16n8k16, and add their sums up through shared memory. The order of the products within a
// sum is free, so a lane takes 16 bytes that lie together and spreads them over consecutive products: both operands by
// the same rule. The tiles of expert_gemm.cu go through K one block of 64 or 256 columns after the other, at some 200 ns
// each, so this kernel serves where all its units are on the device at once. One row of 4096 x 4096: bf16 9.6 us (tiles
// 17.2), nvfp4 6.1 (8.5), mxfp4 7.6 (8.3); of 2048 x 8192 12.4 (28.7), 6.9 (13.0), 8.9 (12.3); of 512 x 512 4.1 (6.7). Bound by
// latency (launch, the first loads, eight warps' sums), and with 4-bit operands by the instructions that open them.
//
// 4-bit operands become fp16 (nvfp4) or bf16 (mxfp4) values with their scales in them, exactly: an e2m1 value has two
// bits, an e4m3 scale four, and fp16's eleven hold both; an e8m0 scale is a power of two, and bf16 has the range of all of
// them (values are an eighth of their size, so that the largest fit too; the sums are freed of that at the end).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "layer.h"
#include "tiles.cuh"

namespace epoch {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kTokens = 16;

// c += a b^T on 16 rows x 8 columns, 16 deep.
template <bool HALF> __device__ __forceinline__ void mma_16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (HALF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load_once(const void *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Eight e2m1 values (a word) times their scale as four pairs of 16-bit values. nvfp4: neighbours, by the conversion to fp16.
// mxfp4: columns (3, 7), (2, 6), (1, 5), (0, 4); an e2m1 value's bits at the top of a bf16's mantissa and below are that
// value x 2^-126, subnormal ones included.
template <bool NV> __device__ __forceinline__ void open_fp4(uint32_t w, uint32_t scale, uint32_t (&v)[4]) {
  if constexpr (NV) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&v[i]), *reinterpret_cast<const __half2 *>(&scale));
      v[i] = *reinterpret_cast<const uint32_t *>(&y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t t = w << (4 * i), bits = (t & 0x80008000u) | ((t >> 6) & 0x01C001C0u), up = 0x7E807E80u;  // 2^126
      const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&bits), *reinterpret_cast<const __nv_bfloat162 *>(&up));
      const __nv_bfloat162 y = __hmul2(x, *reinterpret_cast<const __nv_bfloat162 *>(&scale));
      v[i] = *reinterpret_cast<const uint32_t *>(&y);
    }
  }
}
// A scale's bits as the pair of factors that open_fp4 takes: its value, or for mxfp4 an eighth of it, so that values and
// factors of every e8m0 scale are bf16's.
constexpr float kMxBack = 64.f;
__device__ __forceinline__ uint32_t nv_factor(uint32_t e4m3) {  // fp16 has the same mantissa bits and more below
  e4m3 &= 0x7Fu;
  const __half y = __hmul(__ushort_as_half(static_cast<unsigned short>(e4m3 << 7)), __ushort_as_half(0x5C00));  // its bits are 2^-8 of it
  return e4m3 == 0x7Fu ? 0x7E007E00u : static_cast<uint32_t>(__half_as_ushort(y)) * 0x10001u;
}
__device__ __forceinline__ uint32_t mx_factor(uint32_t e8m0) {  // 2^(e - 130)
  const uint32_t bits = e8m0 == 255u ? 0x7FC0u : e8m0 > 3u ? (e8m0 - 3u) << 7 : 8u << e8m0;
  return bits * 0x10001u;
}

// A warp's piece of one row: 64 bf16 columns or 256 e2m1 columns, of which lane q of a group of four has two
// runs of 16 bytes, and the runs' scales.
template <int FP4> struct Piece {
  uint4 v[2];
  uint32_t s[2];
};
// Piece `it` of a row at p, its scales at s (a block's apart by s_block bytes).
template <int FP4, bool ONCE> __device__ __forceinline__ void load_piece(Piece<FP4> &r, const uint8_t *p, const uint8_t *s, int64_t s_block, int it, int q, int64_t bytes) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t at = static_cast<int64_t>(it) * 128 + 64 * h + 16 * q;
    if (at < bytes) {
      r.v[h] = ONCE ? load_once(p + at) : __ldg(reinterpret_cast<const uint4 *>(p + at));
      if constexpr (FP4 == 4) r.s[h] = __ldg(reinterpret_cast<const uint16_t *>(s + it * s_block + 8 * h) + q);
      if constexpr (FP4 == 2) r.s[h] = __ldg(s + it * s_block + 4 * h + q);
    } else {
      r.v[h] = make_uint4(0u, 0u, 0u, 0u);
      r.s[h] = 0u;
    }
  }
}
// Run h of a piece as the 16-bit values of its products: word j of four is part j of the run, eight columns
// as four pairs (4-bit), or one pair (bf16).
template <int FP4> __device__ __forceinline__ void open_part(const Piece<FP4> &r, int h, int j, uint32_t (&v)[4]) {
  const uint32_t w = j == 0 ? r.v[h].x : j == 1 ? r.v[h].y : j == 2 ? r.v[h].z : r.v[h].w;
  if constexpr (FP4 == 4) open_fp4<true>(w, nv_factor(j < 2 ? r.s[h] & 0xFFu : r.s[h] >> 8), v);
  else open_fp4<false>(w, mx_factor(r.s[h]), v);
}

template <int FP4, bool TALL>
__device__ __forceinline__ void few_unit(const ExpertGemmArgs &a, int kb_n, int e, int row0, int rows, int nt, float (*s_part)[256]) {
  constexpr int kAhead = FP4 ? 2 : 4;  // pieces on their way
  const int lane = lane_id(), warp = warp_id(), g = lane >> 2, q = lane & 3;
  const int half_n = a.N / 2;
  const int64_t bytes = FP4 ? a.K / 2 : 2ll * a.K;  // of a row: up to 2^31
  const int64_t row_bytes = FP4 ? a.K / 2 : 2 * a.a_stride;
  const uint8_t *base = static_cast<const uint8_t *>(a.n_src > 0 ? a.a : a.b), *px[2], *psx[2], *pw[2], *psw[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int64_t src = row0 + min(g + 8 * i, rows - 1);  // (rows that do not exist repeat one that does)
    if (FP4 == 0 && a.rows != nullptr) src = __ldg(a.rows + src);
    if (src < 0 || src >= a.n_src) src = 0;  // never followed; the result is NaN
    px[i] = base + src * row_bytes;
    psx[i] = a.sa + src * (4 * FP4);
    const int n = a.swiglu ? i * half_n + min(nt * 8 + g, half_n - 1) : min(nt * 16 + 8 * i + g, a.N - 1);
    pw[i] = static_cast<const uint8_t *>(a.b) + (static_cast<int64_t>(e) * a.N + n) * bytes;
    psw[i] = a.sb + (static_cast<int64_t>(e) * kb_n * a.N + n) * (4 * FP4);
  }
  const int64_t sx_block = static_cast<int64_t>(a.m) * (4 * FP4), sw_block = static_cast<int64_t>(a.N) * (4 * FP4);
  const int pieces = static_cast<int>((bytes + 127) / 128);
  float sum[2][4] = {};
  for (int it0 = warp; it0 < pieces; it0 += kWarps * kAhead) {
    Piece<FP4> w[kAhead][2];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) load_piece<FP4, true>(w[u][i], pw[i], psw[i], sw_block, it0 + u * kWarps, q, bytes);
    float acc[2][4] = {};
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (it0 + u * kWarps >= pieces) break;
      Piece<FP4> x[2];
#pragma unroll
      for (int i = 0; i < (TALL ? 2 : 1); ++i) load_piece<FP4, false>(x[i], px[i], psx[i], sx_block, it0 + u * kWarps, q, bytes);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (FP4 == 0) {
          const uint4 lo = x[0].v[h], hi = TALL ? x[1].v[h] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            mma_16<false>(acc[i], lo.x, hi.x, lo.y, hi.y, w[u][i].v[h].x, w[u][i].v[h].y);
            mma_16<false>(acc[i], lo.z, hi.z, lo.w, hi.w, w[u][i].v[h].z, w[u][i].v[h].w);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t lo[4], hi[4] = {};
            open_part(x[0], h, j, lo);
            if (TALL) open_part(x[1], h, j, hi);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t b[4];
              open_part(w[u][i], h, j, b);
              mma_16<FP4 == 4>(acc[i], lo[0], hi[0], lo[1], hi[1], b[0], b[1]);
              mma_16<FP4 == 4>(acc[i], lo[2], hi[2], lo[3], hi[3], b[2], b[3]);
            }
          }
        }
      }
    }
    // the tensor core's own sums are of 256 (4-bit: 512) columns
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) sum[i][c] += acc[i][c];
  }
  // value (row, column) of the unit: lane 4 (row % 8) + (column % 8) / 2 of tile column / 8 has it as value 2 (row / 8) + column % 2
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) s_part[warp][(g + 8 * (c >> 1)) * 16 + 8 * i + 2 * q + (c & 1)] = sum[i][c];
  __syncthreads();
  const int tid = threadIdx.x, row = tid >> 4, col = tid & 15;
  if (row < rows && !(a.swiglu && col >= 8)) {
    float f = a.scale * (FP4 == 2 ? kMxBack : 1.f);
    if (a.group_scale != nullptr) f *= __ldg(a.group_scale + e);
    if (FP4 == 0 && a.rows != nullptr) {
      const int src = __ldg(a.rows + row0 + row);
      if (src < 0 || src >= a.n_src) f = __uint_as_float(0x7FC00000u);
    }
    float y = 0.f, up = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      y += s_part[k][tid];
      if (a.swiglu) up += s_part[k][tid + 8];
    }
    y *= f;
    int n = nt * 16 + col, out_n = a.N;
    if (a.swiglu) {
      y = silu(y) * (up * f);
      n = nt * 8 + col;
      out_n = half_n;
    }
    if (n < out_n) {
      const int64_t to = static_cast<int64_t>(row0 + row) * a.out_stride + n;
      if (a.out_bf16) static_cast<__nv_bfloat16 *>(a.out)[to] = __float2bfloat16_rn(y);
      else static_cast<float *>(a.out)[to] = y;
    }
  }
  __syncthreads();
}

template <int FP4> __global__ void __launch_bounds__(kThreads, 2) k_expert_few(const ExpertGemmArgs a, int nt_n, int kb_n) {
  __shared__ int s_start[kMaxGroups + 1], s_cum[kMaxGroups + 1];
  __shared__ float s_part[kWarps][256];
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
    if (rows <= 8) few_unit<FP4, false>(a, kb_n, e, row0, rows, nt, s_part);
    else few_unit<FP4, true>(a, kb_n, e, row0, rows, nt, s_part);
  }
}

}  // namespace

// n_groups 0: dense. Units that are all on the device at once: a second round costs more than the tiles' way through K
// (one row of 16384 x 2048: bf16 18.6 us, tiles 16.2; nvfp4 11.0 and 7.6). Each unit of 4-bit operands opens its rows again,
// so more than one unit of rows is left to the tiles (64 of 2048 x 8192: nvfp4 19.1 and 13.0, mxfp4 27.4 and 11.7).
bool expert_few(bool fp4, int n_groups, int64_t m, int64_t N, int sms) {
  const int64_t groups = n_groups < m ? n_groups : m;
  const int64_t units = (groups > 1 ? m / kTokens + groups : (m + kTokens - 1) / kTokens) * ((N + 15) / 16);
  return units <= 2ll * sms && (!fp4 || m <= kTokens);
}

cudaError_t launch_expert_few(const ExpertGemmArgs &a, cudaStream_t s) {
  const int64_t groups = a.offsets ? (a.n_groups < a.m ? a.n_groups : a.m) : 1;
  const int nt = a.swiglu ? (a.N / 2 + 7) / 8 : (a.N + 15) / 16, kb_n = (a.K + 255) / 256;
  const int64_t units = (groups > 1 ? a.m / kTokens + groups : (a.m + kTokens - 1) / kTokens) * nt, most = 2ll * num_sms();
  const unsigned grid = static_cast<unsigned>(units < most ? units : most);
  if (a.kind == EPOCH_EXPERT_BF16) k_expert_few<0><<<grid, kThreads, 0, s>>>(a, nt, kb_n);
  else if (a.kind == EPOCH_EXPERT_NVFP4) k_expert_few<4><<<grid, kThreads, 0, s>>>(a, nt, kb_n);
  else k_expert_few<2><<<grid, kThreads, 0, s>>>(a, nt, kb_n);
  return cudaGetLastError();
}

}  // namespace epoch
