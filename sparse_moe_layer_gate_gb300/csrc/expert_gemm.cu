// Matrix products of the routed experts, dense or grouped by expert, on bf16 rows or on
// 4-bit (e2m1) operands with a scale for each 16 or 32 columns:
//
//   y[i, n] = s_e * sum_k a[i, k] * w[e, n, k],   offsets[e] <= i < offsets[e + 1]
//
// and, with swiglu, z[i, n] = silu(y[i, n]) * y[i, N / 2 + n]. Row i of a bf16 product may be row
// rows[i] of x (a worklist's positions). Sums are the tensor cores' fp32 accumulators of some blocks of K, added up in
// fp32; the factors s_e and the SwiGLU are applied to them in fp32 and the result is rounded once. For bf16 results the
// SwiGLU has the fast exponential and quotient: off by less than 2^-16 for gates down to -80, a 256th of the rounding that
// follows, and 0 for gates below -87, where silu is less than 2^-119 (the precise ones make an epilogue longer than the
// products of K = 512: 8192 rows over 8 experts of 4096 x 512 43 us, with these 30).
//
// Tiles of 128 rows x 256, 128, 64 or 32 columns, or of 256 x 256 by two CTAs whose tensor cores
// read both halves of the weights. A producer warp streams 128-byte-wide operand tiles (64 bf16 or
// 256 e2m1 columns) by TMA through a ring in shared memory, four more warps the gathered rows; an MMA
// warp issues the tcgen05 products into TMEM; eight epilogue warps take a finished accumulator into
// registers, free it, and store under the next tile's products. With swiglu a tile's columns are
// half gate and half up rows of the weights, so that both halves of an output meet in one thread.
//
// 4-bit operands: the tensor core multiplies by both scales itself and reads them from TMEM, where
// 32 rows x 4 scales take a column of 32 lanes. Scales lie in memory by blocks of 256 columns,
// [K / 256][rows][16 or 8], so that the rows of a tile are one run wherever it starts. Up to three warps
// bring them into shared memory in the order of TMEM (lane l of row group c), from which the MMA
// thread copies them ahead of the products that use them.
//
// What bounds it: with few rows an expert the weights' bytes (256 rows over 256 experts of 1024 x 2048, bf16 with swiglu: 94 us,
// 6.3 TB/s; 8192 rows, mxfp4: 53 us, 5.7 TB/s). With many, bf16: what an SM takes in from L2 for a tile of 128 rows, and the
// power limit (65536 gathered rows over 64 experts of 2048 x 2048: 405 us in a graph, 1.36 PFLOP/s; 450 called back to back);
// 4-bit: the scales leave room for one
// accumulator of 256 columns, so products wait while it is read (8192 x 4096 x 4096: 55 us, 5.0 PFLOP/s), and products are 64
// deep, at four times the bf16 rate; the form 96 deep, at six times, is not used. Registers: a thread of the epilogue holds 128
// sums of a tile of 256 columns, so there the compiler spills some (bytes stored: bf16 single 84 and pairs 292, nvfp4 96 and 52,
// mxfp4 112 and 68).
#include <cstring>
#include <mutex>

#include "common.cuh"
#include "layer.h"
#include "tiles.cuh"

namespace epoch {

namespace {

constexpr int kEpiWarps = 8;
// Four warpgroups: the epilogue's two, one for producer and MMA, and the helpers (4-bit operands: scales; gathered rows).
// The launch's 128 registers a thread are handed over: 88 to the last two, 168 to the epilogue's, whose values alone
// take 128 (2 * 88 + 2 * 168 = 4 * 128).
constexpr int kThreads = 32 * (kEpiWarps + 8);
constexpr int kRegsLaunch = 128, kRegsFew = 88, kRegsMany = 168;
constexpr int kRow = 128;  // bytes of an operand row of a stage: one swizzle row

struct ExpertParams {
  CUtensorMap a[3];  // boxes of 32, 64, 128 rows
  CUtensorMap b;     // boxes of half a tile's columns (pairs: 128)
  CUtensorMap out;   // boxes of 128 bytes x 32 rows of the output (pairs)
  ExpertGemmArgs g;
  int kb_n, nt_n;    // K blocks, tiles along N
  int out_n;         // columns of the output
  int align;         // bytes on which output rows start: 32, 16 or less
  int bulk;          // the output has a tensor map: its rows start and end on 16-byte boundaries
  int reuse;         // weights are read by several row tiles
  int acc_kb;        // K blocks (an even number) that an accumulator sums before it is added to the fp32 sums in registers
  uint32_t *err;
  int64_t timeout_ns;
  uint32_t hold;  // bytes that a stage waits for beyond its copies': 0, but for the test of waits that run out
};

// Tiles are BN columns wide. FP4 0: bf16; 4 or 2: e2m1 with 16 or 8 scales a row in 256 columns, in so many chunks
// of 4 scales.
template <int FP4, int BN, bool PAIR> struct Tile {
  static_assert(!PAIR || BN == 256, "pairs work on 256 columns");
  static constexpr int bm = PAIR ? 2 * kBm : kBm;
  static constexpr int b_rows = PAIR ? BN / 2 : BN;
  static constexpr int box_b = BN == 256 ? 128 : BN / 2;  // rows of a copy of weights
  static constexpr int operands = (kBm + b_rows) * kRow;
  static constexpr int groups_b = BN == 256 ? 2 : 1;      // 128-row groups of the weights' scales
  static constexpr int scale_bytes = (1 + groups_b) * FP4 * 512;
  static constexpr int stage = operands + scale_bytes;
  static constexpr int places = PAIR ? kEpiWarps * 8192 : 0;  // two places of 32 rows x 128 bytes of the output a warp
  static constexpr int fit = (220 * 1024 - places) / stage;
  static constexpr int stages = fit < 8 ? fit : 8;
  // TMEM: accumulators, then four places for the scales of a stage (the copies and the products of one thread
  // complete in order; four let a copy be well ahead of them)
  static constexpr int bufs = FP4 && BN == 256 ? 1 : 2;
  static constexpr int cols_b = BN == 256 ? 8 : 4;        // TMEM columns of a chunk of the weights' scales
  static constexpr int place = FP4 * (4 + cols_b);
  static constexpr int need = bufs * BN + 4 * place;
  static constexpr int tmem = need <= 64 ? 64 : need <= 128 ? 128 : need <= 256 ? 256 : 512;
  static constexpr int smem = 1024 + stages * stage + places;
};

// Shape M x N, fp32 accumulator, both operands K-major.
template <int FP4> __host__ __device__ constexpr uint32_t idesc_of(int M, int N) {
  if (FP4 == 0) return idesc_bf16_f32(M, N);
  return (1u << 7) | (1u << 10)                       // A and B: e2m1
         | (static_cast<uint32_t>(N >> 3) << 17) | (FP4 == 2 ? 1u << 23 : 0u)  // scales: e8m0, else e4m3
         | (static_cast<uint32_t>(M >> 4) << 24);
}

template <int FP4, bool PAIR>
__device__ __forceinline__ void mma(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sa, uint32_t sb,
                                    uint32_t accumulate) {
#define EPOCH_MMA_SCALED(GROUP, VEC)                                                             \
  asm volatile(                                                                                  \
      "{\n\t.reg .pred p;\n\t"                                                                   \
      "setp.ne.b32 p, %6, 0;\n\t"                                                                \
      "tcgen05.mma.cta_group::" GROUP ".kind::mxf4nvf4.block_scale.scale_vec::" VEC " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d), \
      "l"(ad), "l"(bd), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)                            \
      : "memory")
  if constexpr (FP4 == 0) {
    if constexpr (PAIR)
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "setp.ne.b32 p, %4, 0;\n\t"
          "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
          "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate)
          : "memory");
    else
      tc_mma_bf16(d, ad, bd, idesc, accumulate);
  } else if constexpr (FP4 == 4) {
    if constexpr (PAIR) EPOCH_MMA_SCALED("2", "4X");
    else EPOCH_MMA_SCALED("1", "4X");
  } else {
    if constexpr (PAIR) EPOCH_MMA_SCALED("2", "2X");
    else EPOCH_MMA_SCALED("1", "2X");
  }
#undef EPOCH_MMA_SCALED
}

// 32 rows of 16 bytes from shared memory to a run of four TMEM columns, in all four quarters of the lanes (of both
// CTAs' TMEM, each from its own shared memory).
template <bool PAIR> __device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr) {
  const uint64_t desc = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 32) |
                        (static_cast<uint64_t>(1) << 46);  // no swizzle, groups of eight rows 128 bytes apart
  if constexpr (PAIR) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// 16 bytes from global to shared memory, of which `size` are read (the others are zeros).
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int size) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}

template <int Q> __device__ __forceinline__ void load_cols(uint32_t at, float (&v)[Q]) {
  if constexpr (Q == 8) tmem_ld8(at, v);
  else if constexpr (Q == 16) tmem_ld16(at, v);
  else if constexpr (Q == 32) tmem_ld32(at, v);
  else {
    tmem_ld32(at, reinterpret_cast<float (&)[32]>(v[0]));
    tmem_ld32(at + 32, reinterpret_cast<float (&)[32]>(v[32]));
  }
}

// The words of a row that starts on no 16-byte boundary, `n` elements of SIZE bytes from `dst` on: up to the next boundary in
// pieces, then whole vectors of what is left, shifted, and pieces at the end. (A lane has a row: element stores write 32
// sectors an instruction.)
template <int SIZE, int W> __device__ __forceinline__ void store_shifted(uint8_t *dst, int n, uint32_t (&w)[W]) {
  constexpr int kPer = 16 / SIZE;  // elements of a vector
  const int head = static_cast<int>((16u - (reinterpret_cast<uintptr_t>(dst) & 15u)) & 15u) / SIZE;
  if (n > W * 4 / SIZE) n = W * 4 / SIZE;
  if (n < head) {
#pragma unroll
    for (int i = 0; i < kPer - 1; ++i)
      if (i < n) {
        if constexpr (SIZE == 2) reinterpret_cast<uint16_t *>(dst)[i] = static_cast<uint16_t>(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
        else reinterpret_cast<uint32_t *>(dst)[i] = w[i];
      }
    return;
  }
  if constexpr (SIZE == 2) {
    const bool odd = head & 1;
    if (odd) *reinterpret_cast<uint16_t *>(dst) = static_cast<uint16_t>(w[0]);
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = __byte_perm(w[i], i + 1 < W ? w[i + 1] : 0u, odd ? 0x5432u : 0x3210u);
    if (odd) dst += 2;
  }
  const bool one = head & (4 / SIZE), two = head & (8 / SIZE);  // words before the boundary
  if (one) *reinterpret_cast<uint32_t *>(dst) = w[0];
#pragma unroll
  for (int i = 0; i + 1 < W; ++i) w[i] = one ? w[i + 1] : w[i];
  if (one) dst += 4;
  if (two) *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
#pragma unroll
  for (int i = 0; i + 2 < W; ++i) w[i] = two ? w[i + 2] : w[i];
  if (two) dst += 8;
  n -= head;
#pragma unroll
  for (int i = 0; i < W / 4; ++i) {
    const int left = n - i * kPer;
    uint8_t *to = dst + 16 * i;
    const uint32_t *u = w + 4 * i;
    if (left >= kPer) {
      *reinterpret_cast<uint4 *>(to) = make_uint4(u[0], u[1], u[2], u[3]);
    } else if (left > 0) {
      const bool b8 = left & (8 / SIZE), b4 = left & (4 / SIZE);
      const uint32_t x = b8 ? u[2] : u[0], y = b8 ? u[3] : u[1];
      if (b8) *reinterpret_cast<uint2 *>(to) = make_uint2(u[0], u[1]);
      if (b8) to += 8;
      if (b4) *reinterpret_cast<uint32_t *>(to) = x;
      if constexpr (SIZE == 2) {
        if (b4) to += 4;
        if (left & 1) *reinterpret_cast<uint16_t *>(to) = static_cast<uint16_t>(b4 ? y : x);
      }
    }
  }
}

// Q consecutive values of an output row from column n0 on, `n` of which exist, in accesses of `align` bytes: 32 (whole
// sectors) or 16; less: shifted to 16.
template <int Q, int WORDS> __device__ __forceinline__ void store_cols(void *row, int n0, int n, const float (&v)[Q], bool bf16, int align) {
  constexpr int kRun = Q < 16 ? Q : 16;
  if (align < 16) {  // WORDS at a time: all of a run's would not fit into the registers
    constexpr int kHalves = Q < 2 * WORDS ? Q : 2 * WORDS, kWords = Q < WORDS ? Q : WORDS;
    if (bf16) {
#pragma unroll
      for (int j = 0; j < Q; j += kHalves) {
        uint32_t w[kHalves / 2];
#pragma unroll
        for (int i = 0; i < kHalves / 2; ++i) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[j + 2 * i], v[j + 2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        if (j < n) store_shifted<2>(static_cast<uint8_t *>(row) + 2 * (n0 + j), n - j, w);
      }
    } else {
#pragma unroll
      for (int j = 0; j < Q; j += kWords) {
        uint32_t w[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = __float_as_uint(v[j + i]);
        if (j < n) store_shifted<4>(static_cast<uint8_t *>(row) + 4 * (n0 + j), n - j, w);
      }
    }
    return;
  }
  if (bf16) {
    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(row) + n0;
#pragma unroll
    for (int j = 0; j < Q; j += kRun) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < kRun / 2; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[j + 2 * i], v[j + 2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
      }
      if (kRun == 16 && align >= 32 && j + 16 <= n) {
        store32(dst + j, w);
        continue;
      }
#pragma unroll
      for (int c = 0; c < kRun; c += 8) {
        if (j + c + 8 <= n) {
          *reinterpret_cast<uint4 *>(dst + j + c) = make_uint4(w[c / 2], w[c / 2 + 1], w[c / 2 + 2], w[c / 2 + 3]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (j + c + i < n)
              reinterpret_cast<uint16_t *>(dst)[j + c + i] = static_cast<uint16_t>(i & 1 ? w[(c + i) / 2] >> 16 : w[(c + i) / 2]);
        }
      }
    }
  } else {
    float *dst = static_cast<float *>(row) + n0;
#pragma unroll
    for (int j = 0; j < Q; j += 8) {
      if (align >= 32 && j + 8 <= n) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[j + i]);
        store32(dst + j, w);
        continue;
      }
#pragma unroll
      for (int c = j; c < j + 8; c += 4) {
        if (c + 4 <= n) {
          *reinterpret_cast<float4 *>(dst + c) = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
        } else {
#pragma unroll
          for (int i = c; i < c + 4; ++i)
            if (i < n) dst[i] = v[i];
        }
      }
    }
  }
}

// 64 columns of 32 rows, a row a lane, by bulk stores from the warp's two places in shared memory in turn: they run under
// the next tile's products, and leave the load and store units to the helpers. (Rows' own stores of 32 bytes took a
// fifth of the 4-bit product's time at 8192 x 4096 x 4096: the scales' loads waited behind them.)
__device__ __forceinline__ void bulk_run(const CUtensorMap *map, uint8_t *places, uint32_t &turn, int n0, int row, int out_n,
                                         const float (&v)[64], bool bf16) {
  const int lane = lane_id(), per = bf16 ? 64 : 32;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if ((bf16 && h == 1) || n0 + per * h >= out_n) break;
    uint8_t *place = places + (turn & 1u) * 4096;
    ++turn;
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");  // what was here has left
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 8; ++c) {  // 16 bytes at a time, in the 128-byte swizzle
      uint32_t w[4];
      if (bf16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 t = __floats2bfloat162_rn(v[8 * c + 2 * j], v[8 * c + 2 * j + 1]);
          w[j] = *reinterpret_cast<const uint32_t *>(&t);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __float_as_uint(v[32 * h + 4 * c + j]);
      }
      *reinterpret_cast<uint4 *>(place + lane * 128 + ((c ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                       reinterpret_cast<uint64_t>(map)),
                   "r"(n0 + per * h), "r"(row), "r"(smem_u32(place))
                   : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  }
}

template <int FP4, int BN, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) k_expert_gemm(const __grid_constant__ ExpertParams p) {
  using G = Tile<FP4, BN, PAIR>;
  constexpr int Q = BN / 4;                                        // columns of one of a thread's two runs
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[3 * G::stages + 2 * G::bufs];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int s_start[kMaxGroups + 1], s_cum[kMaxGroups + 1];
  const int warp = warp_id(), lane = lane_id();
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const int cta = PAIR ? blockIdx.x >> 1 : blockIdx.x, ctas = PAIR ? gridDim.x >> 1 : gridDim.x;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t *const ring_ptr = smem_raw + (ring - smem_u32(smem_raw));
  const uint32_t full = smem_u32(bars), empty = full + 8 * G::stages, tfull = empty + 8 * G::stages,
                 tempty = tfull + 8 * G::bufs, ready = tempty + 8 * G::bufs;
  const bool gather = FP4 == 0 && p.g.rows != nullptr;
  const int helpers = FP4 ? 1 + G::groups_b : gather ? 4 : 0;  // warps that write a stage beside the copies
  if (warp == 0) {
    if constexpr (PAIR) {
      tmem_alloc_pair(smem_u32(&s_tmem), G::tmem);
    } else {
      tmem_alloc(smem_u32(&s_tmem), G::tmem);
      tmem_relinquish();
    }
  } else if (warp == 1) {
    if (p.g.offsets != nullptr) {
      group_tiles(p.g.offsets, p.g.n_groups, p.g.m, G::bm, s_start, s_cum);
    } else if (lane == 0) {
      s_start[0] = 0;
      s_start[1] = p.g.m;
      s_cum[0] = 0;
      s_cum[1] = (p.g.m + G::bm - 1) / G::bm;
    }
  } else if (warp == 2 && lane == 0) {
    s_abort = 0;
    for (int i = 0; i < G::stages; ++i) {
      // the copies' bytes, this CTA's helpers, and for the second CTA's one warp that waits for them
      mbar_init(full + 8 * i, 1 + helpers + (PAIR && helpers ? 1 : 0));
      mbar_init(empty + 8 * i, 1);
      mbar_init(ready + 8 * i, helpers ? helpers : 1);
    }
    for (int i = 0; i < G::bufs; ++i) {
      mbar_init(tfull + 8 * i, 1);
      mbar_init(tempty + 8 * i, PAIR ? 2 * kEpiWarps : kEpiWarps);  // accumulators read (both CTAs')
    }
    mbar_fence_init();
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) {
    cluster_arrive();
    cluster_wait();
  }
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  volatile int *abort = &s_abort;
  TileWalk walk(s_start, s_cum, p.g.offsets ? p.g.n_groups : 1, p.nt_n, G::bm, rank);
  const int half_n = p.g.N / 2;

  // warps 0 .. 7: epilogue; 8: producer; 9: MMA; 12 .. 15: helpers
  if (warp >= kEpiWarps) {
    give_registers<kRegsFew>();
    if (warp == kEpiWarps) {  // ------------------------------------------------ producer
      const uint64_t keep = policy_evict_last(), pass = policy_evict_first();
      const uint64_t wpol = p.reuse ? keep : pass;
      const uint32_t counts = PAIR ? mapa_shared(full, 0) : full;  // the barriers that the copies count on
      constexpr int kCols = FP4 ? kRow : kRow / 2;                 // tensor map elements of an operand row
      uint32_t it = 0, st = 0, phase = 1;
      bool ok = true;
      for (int t = cta; ok && t < walk.total; t += ctas) {
        int e, row0, rows, nt;
        walk.at(t, &e, &row0, &rows, &nt);
        // single CTAs load the smallest box that holds their rows
        const int box = PAIR || rows > 64 ? 2 : rows > 32 ? 1 : 0;
        const uint32_t a_bytes = gather ? 0u : PAIR ? kBm * kRow : (32u << box) * kRow;
        const uint32_t bytes = (PAIR ? 2 : 1) * (a_bytes + G::b_rows * kRow) + p.hold;
        int b0, b1;  // first rows of the two copies of weights
        if (p.g.swiglu) {
          b0 = e * p.g.N + nt * (BN / 2);
          b1 = b0 + half_n;
          if (PAIR && rank) b0 = b1;
        } else {
          b0 = e * p.g.N + nt * BN + rank * G::b_rows;
          b1 = b0 + G::box_b;
        }
        for (int kb = 0; kb < p.kb_n; ++kb, ++it) {
          ok = warp_wait(empty + 8 * st, phase, abort, p.err, p.timeout_ns);
          if (!ok) break;
          const uint32_t dst = ring + st * G::stage, bar = counts + 8 * st;
          if (elect_one()) {
            if (rank == 0) mbar_arrive_expect_tx(full + 8 * st, bytes);
            if (!gather) load_box<PAIR>(dst, &p.a[box], kb * kCols, row0, bar, keep);
            load_box<PAIR>(dst + kBm * kRow, &p.b, kb * kCols, b0, bar, wpol);
            if constexpr (!PAIR) load_box<PAIR>(dst + kBm * kRow + G::box_b * kRow, &p.b, kb * kCols, b1, bar, wpol);
          }
          __syncwarp();
          if (++st == G::stages) {
            st = 0;
            phase ^= 1u;
          }
        }
      }
      // no exit with copies in flight: the last stages' copies (both CTAs' count here) have landed before the end
      if (rank == 0)
        for (uint32_t i = it > G::stages ? it - G::stages : 0; i < it; ++i) {
          int done = 0;
          wait_for(full + 8 * (i % G::stages), (i / G::stages) & 1u, &done, p.err, p.timeout_ns);
        }
    } else if (FP4 != 0 && warp >= kEpiWarps + 4 && warp < kEpiWarps + 4 + helpers) {  // scales, a group of 128 rows a warp
      constexpr int kPer = FP4 * 4;            // scales of a row in a stage
      constexpr int kAhead = FP4 == 4 ? 3 : 5;  // stages whose scales are on their way, the next tile's among them
      const int group = warp - kEpiWarps - 4;   // 0: a's rows; 1, 2: the weights'
      const uint32_t filled = PAIR && rank ? ready : full;
      const int steps = walk.total > cta ? (walk.total - cta + ctas - 1) / ctas * p.kb_n : 0;
      const int64_t step = static_cast<int64_t>(group == 0 ? p.g.m : p.g.N) * kPer;  // bytes between K blocks
      const uint8_t *src[4];
      int fetch_t = cta, fetch_kb = 0;  // what is loaded next
      uint32_t v[kAhead][4][FP4 ? FP4 : 1];
      auto load = [&](uint32_t (&u)[4][FP4 ? FP4 : 1]) {
        if (fetch_t >= walk.total) return;
        if (fetch_kb == 0) {
          int e, row0, rows, nt;
          walk.at(fetch_t, &e, &row0, &rows, &nt);
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // rows that do not exist read one that does
            const int r = 32 * c + lane;
            if (group == 0) {
              src[c] = p.g.sa + static_cast<int64_t>(min(row0 + r, p.g.m - 1)) * kPer;
            } else {
              const int j = min((group - 1) * 128 + r, BN - 1);
              const int n = !p.g.swiglu ? nt * BN + j : j < BN / 2 ? nt * (BN / 2) + j : half_n + nt * (BN / 2) + j - BN / 2;
              src[c] = p.g.sb + (static_cast<int64_t>(e) * p.kb_n * p.g.N + min(n, p.g.N - 1)) * kPer;
            }
          }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if constexpr (FP4 == 4) {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(src[c]));
            u[c][0] = x.x, u[c][1] = x.y, u[c][2] = x.z, u[c][3] = x.w;
          } else if constexpr (FP4 == 2) {
            const uint2 x = __ldg(reinterpret_cast<const uint2 *>(src[c]));
            u[c][0] = x.x, u[c][1] = x.y;
          }
          src[c] += step;
        }
        if (++fetch_kb == p.kb_n) {
          fetch_kb = 0;
          fetch_t += ctas;
        }
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) load(v[i]);
      uint32_t st = 0, phase = 1;
      bool ok = true;
      for (int n = 0; ok && n < steps; n += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (n + i >= steps) break;
          ok = warp_wait(empty + 8 * st, phase, abort, p.err, p.timeout_ns);
          if (!ok) break;
          uint8_t *dst = ring_ptr + st * G::stage + G::operands + group * FP4 * 512 + lane * 16;
#pragma unroll
          for (int k = 0; k < FP4; ++k)
            *reinterpret_cast<uint4 *>(dst + k * 512) = make_uint4(v[i][0][k], v[i][1][k], v[i][2][k], v[i][3][k]);
          __syncwarp();
          if (lane == 0) mbar_arrive(filled + 8 * st);
          load(v[i]);
          if (++st == G::stages) {
            st = 0;
            phase ^= 1u;
          }
        }
      }
    } else if (FP4 == 0 && gather && warp >= kEpiWarps + 4) {  // gathered rows, every fourth four of them a warp
      // Eight lanes copy an operand row in the 128-byte swizzle. (Copies of four rows an instruction by TMA took 80
      // clocks each, which bound tiles of many rows at 0.5 PFLOP/s.)
      constexpr int kLag = 2;  // stages between a copy and its arrival
      const int w = warp - kEpiWarps - 4, chunk = lane & 7;
      // without a row of x every index is out of range: a row of the weights stands in
      const __nv_bfloat16 *base = static_cast<const __nv_bfloat16 *>(p.g.n_src > 0 ? p.g.a : p.g.b);
      const uint32_t filled = PAIR && rank ? ready : full;
      uint32_t it = 0, st = 0, phase = 1;
      bool ok = true;
      auto arrive = [&](uint32_t i) {  // this warp's copies of stage i have landed
        __syncwarp();
        if (lane == 0) mbar_arrive(filled + 8 * (i % G::stages));
      };
      int from[8], rows = 0, next_rows = 0;  // the next tile's rows of x are read while this one's are copied
      auto look = [&](int t) {
        if (t >= walk.total) return;
        int e, row0, nt;
        walk.at(t, &e, &row0, &next_rows, &nt);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 4 * (4 * i + w) + (lane >> 3);
          from[i] = r < next_rows ? __ldg(p.g.rows + row0 + r) : 0;
        }
      };
      look(cta);
      for (int t = cta; ok && t < walk.total; t += ctas) {
        const __nv_bfloat16 *src[8];
        rows = next_rows;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // an index out of range is never followed; whatever is read instead, the result is NaN
          const int x = from[i] < 0 || from[i] >= p.g.n_src ? 0 : from[i];
          src[i] = base + x * p.g.a_stride + 8 * chunk;
        }
        look(t + ctas);
        for (int kb = 0; kb < p.kb_n; ++kb, ++it) {
          ok = warp_wait(empty + 8 * st, phase, abort, p.err, p.timeout_ns);
          if (!ok) break;
          const int size = kb * 64 + 8 * chunk < p.g.K ? 16 : 0;  // zeros behind the last column
          // rows 16 i + 4 w + lane / 8: the chunk's place in the swizzle is the same in all of them
          const int r0 = 4 * w + (lane >> 3);
          const uint32_t dst = ring + st * G::stage + r0 * kRow + ((chunk ^ (r0 & 7)) << 4);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (16 * i < rows) copy16(dst + 16 * i * kRow, src[i] + (size ? kb * 64 : 0), size);
          asm volatile("cp.async.commit_group;" ::: "memory");
          if (it >= kLag) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kLag) : "memory");
            arrive(it - kLag);
          }
          if (++st == G::stages) {
            st = 0;
            phase ^= 1u;
          }
        }
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      if (ok)
        for (uint32_t i = it > kLag ? it - kLag : 0; i < it; ++i) arrive(i);
    } else if (PAIR && warp == kEpiWarps + 1 && rank == 1) {  // ---------------- the second CTA's helpers, to the first
      // The fence between the helpers' writes and the tensor core's reads waits for every access of its warp, the helpers'
      // loads ahead among them, so it is a warp without accesses that makes it, here as in the first CTA.
      if (helpers) {
        const uint32_t filled = mapa_shared(full, 0);
        uint32_t st = 0, phase = 0;
        bool ok = true;
        for (int t = cta; ok && t < walk.total; t += ctas)
          for (int kb = 0; kb < p.kb_n; ++kb) {
            ok = warp_wait(ready + 8 * st, phase, abort, p.err, p.timeout_ns);
            if (!ok) break;
            fence_proxy_async_smem();
            if (lane == 0) arrive_cluster(filled + 8 * st);
            __syncwarp();
            if (++st == G::stages) {
              st = 0;
              phase ^= 1u;
            }
          }
      }
    } else if (warp == kEpiWarps + 1 && rank == 0) {  // ------------------------ MMA
      // The warp stays together and one elected lane issues, so that descriptors and barriers are uniform values. Two
      // stages a turn: a turn costs this warp some 300 clocks beside its products' 512 a stage (waits that are over,
      // fences, the election), which bound small tiles.
      constexpr uint32_t idesc = idesc_of<FP4>(G::bm, BN);
      constexpr bool kTwo = G::stages >= 6;
      uint32_t it = 0, st = 0, phase = 0, seq = 0;  // seq: accumulators begun
      bool ok = true;
      for (int t = cta; ok && t < walk.total; t += ctas) {
        for (int kb = 0, part = 0; kb < p.kb_n;) {
          const uint32_t buf = seq % G::bufs;
          // (accumulators of fewer K blocks take an even number of them)
          const int two = kTwo && kb + 1 < p.kb_n;
          const uint32_t st1 = st + 1 == G::stages ? 0 : st + 1, phase1 = st1 ? phase : phase ^ 1u;
          const bool r0 = mbar_try_wait(full + 8 * st, phase), r1 = !two || mbar_try_wait(full + 8 * st1, phase1);
          const bool r2 = part > 0 || mbar_try_wait(tempty + 8 * buf, ((seq / G::bufs) & 1u) ^ 1u);
          if (!__all_sync(0xffffffffu, r0 && r1 && r2)) {
            ok = (part > 0 || warp_wait(tempty + 8 * buf, ((seq / G::bufs) & 1u) ^ 1u, abort, p.err, p.timeout_ns)) &&
                 warp_wait(full + 8 * st, phase, abort, p.err, p.timeout_ns) &&
                 (!two || warp_wait(full + 8 * st1, phase1, abort, p.err, p.timeout_ns));
            if (!ok) break;
          }
          if (helpers) fence_proxy_async_smem();
          tc_fence_after();
          const bool last = part + 1 + two == p.acc_kb || kb + 1 + two == p.kb_n;
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (i == 1 && !two) break;
              const uint32_t src = ring + (i ? st1 : st) * G::stage;
              const uint64_t ad = sw128_kmajor_desc(src), bd = sw128_kmajor_desc(src + kBm * kRow);
              const uint32_t sa = tmem + G::bufs * BN + ((it + i) & 3u) * G::place, sb = sa + 4 * FP4;
              if constexpr (FP4 != 0) {
#pragma unroll
                for (int k = 0; k < FP4; ++k) {
                  copy_scales<PAIR>(sa + 4 * k, src + G::operands + k * 512);
#pragma unroll
                  for (int g = 0; g < G::groups_b; ++g)
                    copy_scales<PAIR>(sb + G::cols_b * k + 4 * g, src + G::operands + ((1 + g) * FP4 + k) * 512);
                }
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) {  // 32 bytes of columns an instruction
                // two products share a chunk of e8m0 scales: the second takes its upper half
                const int chunk = FP4 == 2 ? k / 2 : k;
                const uint32_t id = FP4 == 2 && (k & 1) ? idesc | (2u << 4) | (2u << 29) : idesc;
                mma<FP4, PAIR>(tmem + buf * BN, ad + 2 * k, bd + 2 * k, id, sa + 4 * chunk, sb + G::cols_b * chunk,
                               part > 0 || i > 0 || k > 0);
              }
              commit<PAIR>(empty + 8 * (i ? st1 : st));
            }
            if (last) commit<PAIR>(tfull + 8 * buf);
          }
          __syncwarp();
          kb += 1 + two;
          it += 1 + two;
          part = last ? 0 : part + 1 + two;
          seq += last;
          const uint32_t next = st + 1 + two;
          st = next < G::stages ? next : next - G::stages;
          if (next >= G::stages) phase ^= 1u;
        }
      }
      // no exit with products in flight: the last stages have been read
      for (uint32_t i = it > G::stages ? it - G::stages : 0; i < it; ++i) {
        int done = 0;
        wait_for(empty + 8 * (i % G::stages), (i / G::stages) & 1u, &done, p.err, p.timeout_ns);
      }
    }
  } else {  // ------------------------------------------------------------------ epilogue
    take_registers<kRegsMany>();
    const uint32_t read = PAIR ? mapa_shared(tempty, 0) : tempty;  // the barriers that the MMA thread waits on
    const int quarter = warp & 3, half = warp >> 2;  // TMEM lanes 32 quarter .. + 32, half of the columns
    const bool swiglu = p.g.swiglu != 0, bf16 = p.g.out_bf16 != 0;
    const int c0 = swiglu ? half * Q : half * 2 * Q, c1 = swiglu ? BN / 2 + half * Q : c0 + Q;
    const size_t size = bf16 ? 2 : 4;
    constexpr int kPiece = FP4 ? 8 : Q < 32 ? Q : 32;  // (what registers are left beside the scales' code)
    uint32_t seq = 0, turn = 0;
    uint8_t *const places = ring_ptr + G::stages * G::stage + warp * 8192;
    bool ok = true;
    for (int t = cta; ok && t < walk.total; t += ctas) {
      int e, row0, rows, nt;
      walk.at(t, &e, &row0, &rows, &nt);
      const int row = row0 + quarter * 32 + lane;
      const bool on = quarter * 32 + lane < rows;
      const int n0 = (swiglu ? nt * (BN / 2) : nt * BN) + c0;  // output column of the first run
      float s = p.g.scale;
      if (p.g.group_scale != nullptr) s *= __ldg(p.g.group_scale + e);
      if (on && p.g.rows != nullptr) {
        const int r = __ldg(p.g.rows + row);
        if (r < 0 || r >= p.g.n_src) s = __uint_as_float(0x7FC00000u);
      }
      float v0[Q], v1[Q];
      const bool any = quarter * 32 < rows && n0 < p.out_n;  // this warp holds an element of the tile
      uint32_t src = 0;
      auto begin = [&]() {  // the next accumulator is whole
        const uint32_t buf = seq % G::bufs;
        ok = __all_sync(0xffffffffu, wait_for(tfull + 8 * buf, (seq / G::bufs) & 1u, abort, p.err, p.timeout_ns));
        tc_fence_after();
        src = tmem + buf * BN + (static_cast<uint32_t>(quarter * 32) << 16);
      };
      auto end = [&]() {  // and has been read
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR) arrive_cluster(read + 8 * (seq % G::bufs));
          else mbar_arrive(read + 8 * (seq % G::bufs));
        }
        ++seq;
      };
      begin();
      if (!ok) break;
      if (any) {
        load_cols<Q>(src + c0, v0);
        load_cols<Q>(src + c1, v1);
        tmem_ld_wait();
      }
      end();
      for (int kb = p.acc_kb; kb < p.kb_n; kb += p.acc_kb) {
        begin();
        if (!ok) break;
        if (any) {
#pragma unroll
          for (int j = 0; j < Q; j += kPiece) {
            float w[kPiece];
            load_cols<kPiece>(src + c0 + j, w);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < kPiece; ++i) v0[j + i] += w[i];
            load_cols<kPiece>(src + c1 + j, w);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < kPiece; ++i) v1[j + i] += w[i];
          }
        }
        end();
      }
      if (!ok) break;
      if (!any) continue;
      // A warp whose 32 rows all exist; rows behind a group's last one belong to another tile.
      const bool bulk = PAIR && p.bulk && rows >= quarter * 32 + 32;
      if (!bulk && !on) continue;
      void *dst = static_cast<uint8_t *>(p.g.out) + static_cast<int64_t>(row) * p.g.out_stride * size;
      if (swiglu) {
        if (bf16) {
#pragma unroll
          for (int j = 0; j < Q; ++j) v0[j] = silu_fast(v0[j] * s) * (v1[j] * s);
        } else {
#pragma unroll
          for (int j = 0; j < Q; ++j) v0[j] = silu(v0[j] * s) * (v1[j] * s);
        }
        if constexpr (PAIR) {
          if (bulk) {
            bulk_run(&p.out, places, turn, n0, row0 + quarter * 32, p.out_n, v0, bf16);
            continue;
          }
        }
        store_cols<Q, PAIR ? 8 : 16>(dst, n0, p.out_n - n0, v0, bf16, p.align);
      } else {
#pragma unroll
        for (int j = 0; j < Q; ++j) {
          v0[j] *= s;
          v1[j] *= s;
        }
        if constexpr (PAIR) {
          if (bulk) {
            bulk_run(&p.out, places, turn, n0, row0 + quarter * 32, p.out_n, v0, bf16);
            bulk_run(&p.out, places, turn, n0 + Q, row0 + quarter * 32, p.out_n, v1, bf16);
            continue;
          }
        }
        store_cols<Q, PAIR ? 8 : 16>(dst, n0, p.out_n - n0, v0, bf16, p.align);
        if (n0 + Q < p.out_n) store_cols<Q, PAIR ? 8 : 16>(dst, n0 + Q, p.out_n - n0 - Q, v1, bf16, p.align);
      }
    }
  }
  if constexpr (PAIR) {  // no exit with stores still reading shared memory
    if (warp < kEpiWarps && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) {  // the other CTA may still reach this one's barriers
    cluster_arrive();
    cluster_wait();
  }
  if (warp == 0) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem, G::tmem);
    else tmem_dealloc(tmem, G::tmem);
  }
}

template <int FP4, int BN, bool PAIR> cudaError_t launch_tile(ExpertParams &p, cudaStream_t s) {
  using G = Tile<FP4, BN, PAIR>;
  auto *fn = &k_expert_gemm<FP4, BN, PAIR>;
  static std::mutex mu;
  static int resident[64] = {};  // CTAs that a device holds at once; -1: the kernel cannot run there
  int dev = 0, most = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = G::smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 1 : 0;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (resident[dev] == 0) {
      cudaFuncAttributes fa;
      e = cudaFuncGetAttributes(&fa, fn);
      if (e != cudaSuccess) return e;
      // the warpgroups hand registers over within what the launch holds
      if (fa.numRegs < kRegsLaunch) return cudaErrorInvalidConfiguration;
      e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, G::smem);
      if (e != cudaSuccess) return e;
      int n = num_sms();
      if (PAIR) {
        cfg.gridDim = dim3(static_cast<unsigned>(num_sms() / 2 * 2));
        e = cudaOccupancyMaxActiveClusters(&n, fn, &cfg);
        if (e != cudaSuccess) return e;
        n *= 2;
      }
      resident[dev] = n;
    }
    most = resident[dev];
  }
  if (most < (PAIR ? 2 : 1)) return cudaErrorNotSupported;
  p.nt_n = (p.g.N + BN - 1) / BN;
  // row tiles: at most one partial tile a group beyond the full ones
  const int64_t mt = p.g.offsets ? p.g.m / G::bm + (p.g.n_groups < p.g.m ? p.g.n_groups : p.g.m) : (p.g.m + G::bm - 1) / G::bm;
  const int64_t ctas = mt * p.nt_n * (PAIR ? 2 : 1);
  cfg.gridDim = dim3(static_cast<unsigned>(ctas < most ? ctas : most));
  return cudaLaunchKernelEx(&cfg, fn, p);
}

template <int FP4> cudaError_t launch_kind(ExpertParams &p, int kernel, cudaStream_t s) {
  if (kernel == kExpertPairs) return launch_tile<FP4, 256, true>(p, s);
  if (kernel == 256) return launch_tile<FP4, 256, false>(p, s);
  if (kernel == 128) return launch_tile<FP4, 128, false>(p, s);
  if (kernel == 64) return launch_tile<FP4, 64, false>(p, s);
  return launch_tile<FP4, 32, false>(p, s);
}

}  // namespace

// The tiles a product takes: the columns of a tile of single CTAs, kExpertPairs tiles of CTA pairs. n_groups 0: dense.
// The one whose rounds of tiles take the least time, by the nanoseconds that a K block of each took with many tiles
// (64 groups, 32768 rows by 2048 x 2048). Wide tiles are bound by what an SM takes in from L2 (about 50 bytes a clock),
// narrow ones by the MMA warp's turns. A group is expected to end in the middle of a tile.
int expert_gemm_kernel(bool fp4, int n_groups, int64_t m, int64_t N, int sms) {
  const int64_t E = n_groups ? (n_groups < m ? n_groups : m) : 1;
  auto tiles = [&](int64_t rows) {
    const int64_t t = E > 1 ? m / rows + (E + 1) / 2 : (m + rows - 1) / rows;
    return t > E ? t : E;
  };
  static const int64_t kCost[5][3] = {{256, 420, 790}, {128, 250, 555}, {64, 197, 430}, {32, 190, 390}, {kExpertPairs, 405, 600}};
  int bn = 256;
  int64_t best = INT64_MAX;
  for (const auto &c : kCost) {
    const bool pairs = c[0] == kExpertPairs;
    if (pairs && sms < 2) continue;
    const int64_t n = tiles(pairs ? 256 : kBm) * ((N + (pairs ? 256 : c[0]) - 1) / (pairs ? 256 : c[0])), at_once = pairs ? sms / 2 : sms;
    const int64_t t = (n + at_once - 1) / at_once * c[fp4 ? 2 : 1];
    if (t < best) {
      best = t;
      bn = static_cast<int>(c[0]);
    }
  }
  return bn;
}

cudaError_t launch_expert_gemm(const ExpertGemmArgs &a, cudaStream_t s, int64_t timeout_ns, uint32_t hold) {
  const bool fp4 = a.kind != EPOCH_EXPERT_BF16;
  const int kernel = expert_gemm_kernel(fp4, a.offsets ? a.n_groups : 0, a.m, a.N, num_sms());
  ExpertParams p;
  memset(&p, 0, sizeof(p));
  p.g = a;
  p.kb_n = (a.K + (fp4 ? 255 : 63)) / (fp4 ? 256 : 64);
  p.out_n = a.swiglu ? a.N / 2 : a.N;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(a.out) | static_cast<uintptr_t>(a.m > 1 ? a.out_stride * (a.out_bf16 ? 2 : 4) : 0);
  p.align = bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : 0;
  const int64_t E = a.offsets ? a.n_groups : 1;
  p.reuse = a.m > kBm * E;
  // The tensor core's sums are truncated, by 0.8 of a step of fp32 a product on the average, and so drift where terms have
  // one sign: over 65536 bf16 columns (4096 products) by 4e-4 of the result. So fp32 results add up accumulators of four
  // blocks (16 products: 4e-7, or 1.1e-6 where the terms range over many octaves), with 4-bit operands of eight (32: 1e-7 and
  // 6.5e-7, since the terms have few bits; 8192 x 4096 x 4096 nvfp4 64 us, in one accumulator 61, by four blocks 71). bf16
  // results add up accumulators of 64 blocks (256 products: 1.5e-5 and 2.4e-5, an 80th of half a step of bf16 at most; four
  // blocks would cost a prompt's bf16 product a tenth of its time).
  p.acc_kb = a.out_bf16 ? 64 : fp4 ? 8 : 4;
  p.err = ops_error_word();
  p.timeout_ns = timeout_ns;
  p.hold = hold;
  if (p.err == nullptr || !tma_encode_init()) return cudaErrorInitializationError;
  const uint64_t k_row = fp4 ? a.K / 2 : a.K;
  const uint32_t b_box = kernel == kExpertPairs || kernel == 256 ? 128 : kernel / 2;
  bool ok = encode_operand(&p.b, a.b, !fp4, k_row, E * a.N, k_row, b_box);
  if (a.rows == nullptr) {
    // the boxes that some tile's rows may ask for
    const bool pairs = kernel == kExpertPairs, partial = a.offsets != nullptr || a.m % kBm != 0;
    if (pairs || a.m > 64) ok = ok && encode_operand(&p.a[2], a.a, !fp4, k_row, a.m, a.a_stride, 128);
    if (!pairs && partial && a.m > 32) ok = ok && encode_operand(&p.a[1], a.a, !fp4, k_row, a.m, a.a_stride, 64);
    if (!pairs && partial) ok = ok && encode_operand(&p.a[0], a.a, !fp4, k_row, a.m, a.a_stride, 32);
  }
  // Bulk stores end a row on a 16-byte boundary: with another width they would write zeros into the columns behind it.
  const int per16 = a.out_bf16 ? 8 : 4;
  if (ok && kernel == kExpertPairs && (reinterpret_cast<uintptr_t>(a.out) & 15u) == 0 && a.out_stride % per16 == 0 &&
      p.out_n % per16 == 0) {
    ok = encode_rows(&p.out, a.out, a.out_bf16, p.out_n, a.m, a.out_stride);
    p.bulk = 1;
  }
  if (!ok) return cudaErrorInvalidValue;
  if (a.kind == EPOCH_EXPERT_BF16) return launch_kind<0>(p, kernel, s);
  return a.kind == EPOCH_EXPERT_NVFP4 ? launch_kind<4>(p, kernel, s) : launch_kind<2>(p, kernel, s);
}

}  // namespace epoch
