// Matrix product of e4m3 operands with a scale for each block of 128, dense or
// grouped by expert:
//
//   y[m, n] = sum over K blocks b of  sa[m, b] * sb[e, n / 128, b] * sum_{k in b} a[m, k] * w[e, n, k]
//
// where row m belongs to expert e of offsets[e] <= m < offsets[e + 1] (dense:
// one expert). Products of a K block are summed by the tensor cores; the
// scaled sums of the blocks are kept in fp32 registers and rounded once.
//
// Many rows (k_fp8_gemm): tiles of 128 rows x BN columns. A producer warp
// streams 128-byte-wide (one K block) operand tiles by TMA through a ring in
// shared memory, an MMA warp issues tcgen05 products of one K block into one of
// two TMEM accumulators, and eight epilogue warps read the other accumulator,
// scale it and add it to their registers: the promotion of one block runs under
// the products of the next.
//
// Few rows (k_fp8_small): bound by the weights' bytes; sixteen weight rows per
// CTA go from global memory straight into mma.sync fragments (see below).
#include <atomic>
#include <cstring>
#include <mutex>

#include "common.cuh"
#include "fp8.cuh"
#include "layer.h"

namespace epoch {

namespace {

constexpr int kBm = 128;
constexpr int kBk = 128;  // one scale block; 128 bytes: one swizzle row
constexpr int kEpiWarps = 8;
// Three warpgroups: producer, MMA and two warps for the scales, and the epilogue's two.
// The launch's 168 registers a thread are handed over: 56 to the first group,
// 224 to the others, whose sums alone take 128 (56 + 2 * 224 = 3 * 168).
constexpr int kThreads = 32 * (kEpiWarps + 4);
constexpr int kRegsFew = 56, kRegsMany = 224;
constexpr int kMaxGroups = 1024;

struct GemmParams {
  CUtensorMap a[3];  // boxes of 32, 64, 128 rows
  CUtensorMap b;     // boxes of BN rows
  GemmArgs g;
  int kb_n, nb_n, nt_n;  // K blocks, N scale blocks, N tiles
  uint32_t *err;
  int64_t timeout_ns;
};

// Shape N x M of kind::f8f6f4 with e4m3 operands, fp32 accumulator, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void tc_mma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

template <int R> __device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R> __device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}

// Two fp32 sums in a register pair; acc += v * s on both at once.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ void fma_pair(uint64_t &acc, uint64_t v, uint64_t s) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(s));
}
template <int N> __device__ __forceinline__ void add_scaled(uint64_t *acc, const float (&v)[N], uint64_t s) {
#pragma unroll
  for (int j = 0; j < N / 2; ++j) fma_pair(acc[j], pair(v[2 * j], v[2 * j + 1]), s);
}

// First rows of the groups, in ascending order and within [0, m] whatever the
// caller's offsets hold (start, E + 1 entries), and the number of row tiles
// before each group (cum, E + 1 entries). One warp; E <= kMaxGroups.
__device__ void group_tiles(const int32_t *offsets, int E, int m, int tile, int *start, int *cum) {
  const int lane = lane_id(), per = (E + 32) / 32;  // entries of offsets [0, E] per lane
  const int lo = lane * per, hi = min(lo + per, E + 1);
  int mx = 0;
  for (int i = lo; i < hi; ++i) {
    const int o = min(max(__ldg(offsets + i), 0), m);
    mx = max(mx, o);
    start[i] = mx;
  }
  int pre = mx;  // largest entry up to this lane's
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, pre, o);
    if (lane >= o) pre = max(pre, y);
  }
  pre = __shfl_up_sync(0xffffffffu, pre, 1);
  if (lane == 0) pre = 0;
  for (int i = lo; i < hi; ++i) start[i] = max(start[i], pre);
  __syncwarp();
  int n = 0;
  for (int i = lo; i < min(hi, E); ++i) n += (start[i + 1] - start[i] + tile - 1) / tile;
  int sum = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += y;
  }
  int at = sum - n;
  for (int i = lo; i < hi; ++i) {
    cum[i] = at;
    if (i < E) at += (start[i + 1] - start[i] + tile - 1) / tile;
  }
  __syncwarp();
}

// The tiles of one role: tile t of the launch is row tile t / nt_n (groups in
// order) and column tile t % nt_n, so neighbouring CTAs share their rows.
struct TileWalk {
  const int *start, *cum;
  int E, nt_n, e, total;
  __device__ TileWalk(const int *s, const int *c, int E_, int nt) : start(s), cum(c), E(E_), nt_n(nt), e(0) {
    total = cum[E] * nt_n;
  }
  __device__ void at(int t, int *group, int *row0, int *rows, int *nt) {
    const int mt = t / nt_n;
    *nt = t - mt * nt_n;
    while (cum[e + 1] <= mt) ++e;
    *group = e;
    *row0 = start[e] + (mt - cum[e]) * kBm;
    *rows = min(kBm, start[e + 1] - *row0);
  }
};

template <int BN> struct Geo {
  static constexpr int stage = (kBm + BN) * kBk;
  static constexpr int stages = BN == 256 ? 4 : 6;
  static constexpr int bufs = 512 / BN;  // TMEM accumulators
  static constexpr int smem = 1024 + stages * stage;
};

template <int BN, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) k_fp8_gemm(const __grid_constant__ GemmParams p) {
  using G = Geo<BN>;
  constexpr int kCols = BN / 2;  // columns of an epilogue warpgroup
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * G::stages + 2 * G::bufs];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ float s_scale[G::bufs][2][kBm];  // a's scale times b's, for each row and epilogue half
  __shared__ int s_start[kMaxGroups + 1], s_cum[kMaxGroups + 1];
  const int warp = warp_id(), lane = lane_id();
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t full = smem_u32(bars), empty = full + 8 * G::stages, tfull = empty + 8 * G::stages,
                 tempty = tfull + 8 * G::bufs;
  if (warp == 0) {
    tmem_alloc(smem_u32(&s_tmem), 512);
    tmem_relinquish();
  } else if (warp == 1) {
    if (p.g.offsets != nullptr) {
      group_tiles(p.g.offsets, p.g.n_groups, p.g.m, kBm, s_start, s_cum);
    } else if (lane == 0) {
      s_start[0] = 0;
      s_start[1] = p.g.m;
      s_cum[0] = 0;
      s_cum[1] = (p.g.m + kBm - 1) / kBm;
    }
  } else if (warp == 2 && lane == 0) {
    s_abort = 0;
    for (int i = 0; i < G::stages; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < G::bufs; ++i) {
      mbar_init(tfull + 8 * i, 2);  // the products, and the scales
      mbar_init(tempty + 8 * i, kEpiWarps);
    }
    mbar_fence_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  volatile int *abort = &s_abort;
  TileWalk walk(s_start, s_cum, p.g.offsets ? p.g.n_groups : 1, p.nt_n);

  // warps 0 .. 7: epilogue; 8: producer; 9: MMA; 10, 11: scales
  if (warp >= kEpiWarps) {
    give_registers<kRegsFew>();
    if (warp == kEpiWarps && lane == 0) {  // ----------------------------------- producer
      const uint64_t keep = policy_evict_last(), pass = policy_evict_first();
      // weights of a tile's columns are read once per row tile; with one row tile a group they stream through
      const uint64_t wpol = p.g.offsets ? pass : keep;
      uint32_t it = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < walk.total; t += gridDim.x) {
        int e, row0, rows, nt;
        walk.at(t, &e, &row0, &rows, &nt);
        const int box = rows <= 32 ? 0 : rows <= 64 ? 1 : 2;
        const CUtensorMap *ma = p.g.offsets ? &p.a[box] : &p.a[2];
        const uint32_t bytes = ((p.g.offsets ? 32u << box : 128u) + BN) * kBk;
        const int brow = e * p.g.N + nt * BN;
        for (int kb = 0; kb < p.kb_n; ++kb, ++it) {
          const uint32_t st = it % G::stages, ph = (it / G::stages) & 1u;
          if (!mbar_wait_bounded(empty + 8 * st, ph ^ 1u, abort, p.err, p.timeout_ns)) {
            ok = false;
            break;
          }
          const uint32_t dst = ring + st * G::stage;
          mbar_arrive_expect_tx(full + 8 * st, bytes);
          tma_load_2d(dst, ma, kb * kBk, row0, full + 8 * st, keep);
          tma_load_2d(dst + kBm * kBk, &p.b, kb * kBk, brow, full + 8 * st, wpol);
        }
      }
      // no exit with copies in flight: the last stages' copies have landed before the CTA ends
      for (uint32_t i = it > G::stages ? it - G::stages : 0; i < it; ++i) {
        int done = 0;
        mbar_wait_bounded(full + 8 * (i % G::stages), (i / G::stages) & 1u, &done, p.err, p.timeout_ns);
      }
    } else if (warp >= kEpiWarps + 2) {  // ------------------------------------- scales, every other K block a warp
      uint32_t it = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < walk.total; t += gridDim.x) {
        int e, row0, rows, nt;
        walk.at(t, &e, &row0, &rows, &nt);
        const float *sa[4], *sb[2];
        float fa[4], fb[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) sa[i] = p.g.sa + static_cast<int64_t>(row0 + min(32 * i + lane, rows - 1)) * p.kb_n;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          sb[i] = p.g.sb + (static_cast<int64_t>(e) * p.nb_n + min((nt * BN + i * kCols) / kFp8Block, p.nb_n - 1)) * p.kb_n;
        auto load = [&](int kb) {
          kb = min(kb, p.kb_n - 1);
#pragma unroll
          for (int i = 0; i < 4; ++i) fa[i] = __ldg(sa[i] + kb);
#pragma unroll
          for (int i = 0; i < 2; ++i) fb[i] = __ldg(sb[i] + kb);
        };
        const int first = static_cast<int>((it ^ static_cast<uint32_t>(warp)) & 1u);
        load(first);
        for (int kb = first; kb < p.kb_n; kb += 2) {
          const uint32_t i = it + kb, buf = i % G::bufs;
          ok = mbar_wait_bounded(tempty + 8 * buf, ((i / G::bufs) & 1u) ^ 1u, abort, p.err, p.timeout_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) s_scale[buf][h][32 * j + lane] = fa[j] * fb[h];
          __syncwarp();
          if (lane == 0) mbar_arrive(tfull + 8 * buf);
          load(kb + 2);
        }
        it += p.kb_n;
      }
    } else if (warp == kEpiWarps + 1 && lane == 0) {  // ------------------------ MMA
      constexpr uint32_t idesc = idesc_e4m3_f32(kBm, BN);
      uint32_t it = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < walk.total; t += gridDim.x) {
        for (int kb = 0; kb < p.kb_n; ++kb, ++it) {
          const uint32_t st = it % G::stages, buf = it % G::bufs;
          if (!mbar_wait_bounded(full + 8 * st, (it / G::stages) & 1u, abort, p.err, p.timeout_ns) ||
              !mbar_wait_bounded(tempty + 8 * buf, ((it / G::bufs) & 1u) ^ 1u, abort, p.err, p.timeout_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t src = ring + st * G::stage;
          const uint64_t ad = sw128_kmajor_desc(src), bd = sw128_kmajor_desc(src + kBm * kBk);
#pragma unroll
          for (int k = 0; k < kBk / 32; ++k)  // 32 columns (32 bytes) per instruction
            tc_mma_e4m3(tmem + buf * BN, ad + 2 * k, bd + 2 * k, idesc, k > 0);
          tc_commit(empty + 8 * st);
          tc_commit(tfull + 8 * buf);
        }
      }
      // no exit with products in flight: the last accumulators are complete
      for (uint32_t i = it > G::bufs ? it - G::bufs : 0; i < it; ++i) {
        int done = 0;
        mbar_wait_bounded(tfull + 8 * (i % G::bufs), (i / G::bufs) & 1u, &done, p.err, p.timeout_ns);
      }
    }
  } else {  // ------------------------------------------------------------------ epilogue
    take_registers<kRegsMany>();
    const int quarter = warp & 3, half = warp >> 2;  // TMEM lanes 32 quarter .. + 32, columns kCols half .. + kCols
    uint32_t it = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < walk.total; t += gridDim.x) {
      int e, row0, rows, nt;
      walk.at(t, &e, &row0, &rows, &nt);
      const int r = quarter * 32 + lane, row = row0 + r;
      const int n0 = nt * BN + half * kCols;
      const bool on = r < rows && n0 < p.g.N;
      const bool any = quarter * 32 < rows && n0 < p.g.N;  // this warp holds a row of the tile
      uint64_t acc[kCols / 2];
#pragma unroll
      for (int c = 0; c < kCols / 2; ++c) acc[c] = 0ull;
      for (int kb = 0; kb < p.kb_n; ++kb, ++it) {
        const uint32_t buf = it % G::bufs;
        ok = mbar_wait_bounded(tfull + 8 * buf, (it / G::bufs) & 1u, abort, p.err, p.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (any) {
          // 32 columns are on their way from TMEM while the 32 before them are added
          tc_fence_after();
          const uint32_t src = tmem + buf * BN + half * kCols + (static_cast<uint32_t>(quarter * 32) << 16);
          const float s = s_scale[buf][half][r];
          const uint64_t s2 = pair(s, s);
          float v[2][32];
          tmem_ld32(src, v[0]);
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c) {
            tmem_ld_wait();
            if (c + 1 < kCols / 32) tmem_ld32(src + 32 * (c + 1), v[(c + 1) & 1]);
            else tc_fence_before();
            if (c + 1 == kCols / 32) {
              __syncwarp();
              if (lane == 0) mbar_arrive(tempty + 8 * buf);
            }
            add_scaled(acc + 16 * c, v[c & 1], s2);
          }
        } else {
          __syncwarp();
          if (lane == 0) mbar_arrive(tempty + 8 * buf);
        }
      }
      if (ok && on) {
        const int n = min(kCols, p.g.N - n0);
        if constexpr (BF16) {
          __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.g.out) + static_cast<int64_t>(row) * p.g.out_stride + n0;
          if (p.g.wide_out && n == kCols) {
#pragma unroll
            for (int c = 0; c < kCols / 2; c += 4) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 f = unpair(acc[c + j]);
                const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
                w[j] = *reinterpret_cast<const uint32_t *>(&h);
              }
              *reinterpret_cast<uint4 *>(dst + 2 * c) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
#pragma unroll
            for (int c = 0; c < kCols / 2; ++c) {
              const float2 f = unpair(acc[c]);
              if (2 * c < n) dst[2 * c] = __float2bfloat16_rn(f.x);
              if (2 * c + 1 < n) dst[2 * c + 1] = __float2bfloat16_rn(f.y);
            }
          }
        } else {
          float *dst = static_cast<float *>(p.g.out) + static_cast<int64_t>(row) * p.g.out_stride + n0;
          if (p.g.wide_out && n == kCols) {
#pragma unroll
            for (int c = 0; c < kCols / 2; c += 2) {
              const float2 f = unpair(acc[c]), h = unpair(acc[c + 1]);
              *reinterpret_cast<float4 *>(dst + 2 * c) = make_float4(f.x, f.y, h.x, h.y);
            }
          } else {
#pragma unroll
            for (int c = 0; c < kCols / 2; ++c) {
              const float2 f = unpair(acc[c]);
              if (2 * c < n) dst[2 * c] = f.x;
              if (2 * c + 1 < n) dst[2 * c + 1] = f.y;
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ few rows
// A CTA takes sixteen weight rows of one expert and splits K over its warps;
// the warps' sums meet in shared memory in warp order. The weights stream from
// global memory into mma.sync fragments: the order of the products of a K block
// is free, so thread (g, t) of a warp holds sixteen consecutive bytes of row g
// and of row g + 8 (columns 16 t .. of a 64-column step) and the same columns of
// token g, which are the operands of two m16n8k32 products without any shuffle.
constexpr int kSmallWarps = 8;
constexpr int kSmallTokens = 64;  // rows of one call (8 token tiles)

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 load16(const void *p, bool ok) {
  uint4 u = make_uint4(0u, 0u, 0u, 0u);
  if (ok)
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(p));
  return u;
}

template <int NT, bool BF16>
__global__ void __launch_bounds__(32 * kSmallWarps) k_fp8_small(const GemmArgs a, int kb_n, int nb_n) {
  __shared__ float s_part[kSmallWarps][NT][128];
  __shared__ int s_start[kMaxGroups + 1], s_cum[kMaxGroups + 1];
  const int warp = warp_id(), lane = lane_id(), g = lane >> 2, t = lane & 3;
  const int E = a.offsets ? a.n_groups : 1;
  if (a.offsets != nullptr) {
    if (warp == 0) group_tiles(a.offsets, E, a.m, kSmallTokens, s_start, s_cum);
  } else if (threadIdx.x == 0) {
    s_start[0] = 0;
    s_start[1] = a.m;
    s_cum[0] = 0;
    s_cum[1] = 1;
  }
  __syncthreads();
  const int nt_n = (a.N + 15) / 16;
  const int units = s_cum[E] * nt_n;
  int e = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int mt = u / nt_n, n0 = (u - mt * nt_n) * 16;
    while (s_cum[e + 1] <= mt) ++e;
    const int row0 = s_start[e], rows = s_start[e + 1] - row0;  // m <= kSmallTokens: one tile a group
    const uint8_t *w = static_cast<const uint8_t *>(a.b) + (static_cast<int64_t>(e) * a.N + n0 + g) * a.K + 16 * t;
    const bool w0 = n0 + g < a.N, w1 = n0 + g + 8 < a.N;
    const float *sb = a.sb + (static_cast<int64_t>(e) * nb_n + n0 / kFp8Block) * kb_n;
    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    for (int kb = warp; kb < kb_n; kb += kSmallWarps) {
      uint4 wa[2], wb[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = kb * kFp8Block + 64 * h;
        const bool in = k + 16 * t < a.K;
        wa[h] = load16(w + k, w0 && in);
        wb[h] = load16(w + k + static_cast<int64_t>(8) * a.K, w1 && in);
      }
      const float sw = __ldg(sb + kb);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if (i * 8 >= rows) break;
        const int tok = i * 8 + g;
        const uint8_t *x = static_cast<const uint8_t *>(a.a) + static_cast<int64_t>(row0 + tok) * a.K + 16 * t;
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = kb * kFp8Block + 64 * h;
          uint4 xv = make_uint4(0u, 0u, 0u, 0u);
          if (tok < rows && k + 16 * t < a.K) xv = __ldg(reinterpret_cast<const uint4 *>(x + k));
          mma_e4m3(part, wa[h].x, wb[h].x, wa[h].y, wb[h].y, xv.x, xv.y);
          mma_e4m3(part, wa[h].z, wb[h].z, wa[h].w, wb[h].w, xv.z, xv.w);
        }
        const int c0 = i * 8 + 2 * t;
        const float s0 = c0 < rows ? __ldg(a.sa + static_cast<int64_t>(row0 + c0) * kb_n + kb) * sw : 0.f;
        const float s1 = c0 + 1 < rows ? __ldg(a.sa + static_cast<int64_t>(row0 + c0 + 1) * kb_n + kb) * sw : 0.f;
        acc[i][0] = fmaf(part[0], s0, acc[i][0]);
        acc[i][1] = fmaf(part[1], s1, acc[i][1]);
        acc[i][2] = fmaf(part[2], s0, acc[i][2]);
        acc[i][3] = fmaf(part[3], s1, acc[i][3]);
      }
    }
    // sums of the warps: value v of a token tile is weight row v / 8, token v % 8
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      float *d = s_part[warp][i];
      d[g * 8 + 2 * t] = acc[i][0];
      d[g * 8 + 2 * t + 1] = acc[i][1];
      d[(g + 8) * 8 + 2 * t] = acc[i][2];
      d[(g + 8) * 8 + 2 * t + 1] = acc[i][3];
    }
    __syncthreads();
    for (int v = threadIdx.x; v < NT * 128; v += blockDim.x) {
      // consecutive threads: consecutive columns of one row of the output
      const int tok = v >> 4, n = v & 15;
      const int at = n * 8 + (tok & 7);
      if (tok < rows && n0 + n < a.N) {
        float y = 0.f;
#pragma unroll
        for (int q = 0; q < kSmallWarps; ++q) y += s_part[q][tok >> 3][at];
        const int64_t o = static_cast<int64_t>(row0 + tok) * a.out_stride + n0 + n;
        if constexpr (BF16) static_cast<__nv_bfloat16 *>(a.out)[o] = __float2bfloat16_rn(y);
        else static_cast<float *>(a.out)[o] = y;
      }
    }
    __syncthreads();
  }
}

static __device__ uint32_t g_ops_error;  // device error word of the calls that belong to no layer

uint32_t *ops_error_address(int device) {
  static std::mutex mu;
  static uint32_t *addr[64] = {};
  if (device < 0 || device >= 64) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (addr[device] == nullptr) {
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, g_ops_error) != cudaSuccess) return nullptr;
    addr[device] = static_cast<uint32_t *>(p);
  }
  return addr[device];
}

template <int BN, bool BF16> cudaError_t launch_tc(GemmParams &p, cudaStream_t s) {
  using G = Geo<BN>;
  auto *fn = &k_fp8_gemm<BN, BF16>;
  static std::atomic<uint64_t> ready{0};  // devices whose copy of the kernel has its shared memory raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load() & bit)) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, G::smem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit);
  }
  p.nt_n = (p.g.N + BN - 1) / BN;
  // row tiles: at most one partial tile a group beyond the full ones
  const int64_t mt = p.g.offsets ? p.g.m / kBm + p.g.n_groups : (p.g.m + kBm - 1) / kBm;
  const int64_t tiles = mt * p.nt_n;
  const int grid = static_cast<int>(tiles < num_sms() ? tiles : num_sms());
  fn<<<grid, kThreads, G::smem, s>>>(p);
  return cudaGetLastError();
}

template <int NT> cudaError_t launch_small(const GemmArgs &a, int kb_n, int nb_n, cudaStream_t s) {
  const int64_t groups = a.offsets ? (a.n_groups < a.m ? a.n_groups : a.m) : 1;
  const int64_t units = groups * ((a.N + 15) / 16);
  const int64_t most = static_cast<int64_t>(num_sms()) * 4;
  const unsigned grid = static_cast<unsigned>(units < most ? units : most);
  if (a.out_bf16) k_fp8_small<NT, true><<<grid, 32 * kSmallWarps, 0, s>>>(a, kb_n, nb_n);
  else k_fp8_small<NT, false><<<grid, 32 * kSmallWarps, 0, s>>>(a, kb_n, nb_n);
  return cudaGetLastError();
}

}  // namespace

uint32_t *ops_error_word() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess ? ops_error_address(dev) : nullptr;
}

cudaError_t launch_fp8_gemm(const GemmArgs &a, cudaStream_t s) {
  const int kb_n = (a.K + kBk - 1) / kBk, nb_n = (a.N + kFp8Block - 1) / kFp8Block;
  if (a.m <= kSmallTokens) {
    if (a.m <= 8) return launch_small<1>(a, kb_n, nb_n, s);
    if (a.m <= 16) return launch_small<2>(a, kb_n, nb_n, s);
    if (a.m <= 32) return launch_small<4>(a, kb_n, nb_n, s);
    return launch_small<8>(a, kb_n, nb_n, s);
  }
  GemmParams p;
  memset(&p, 0, sizeof(p));
  p.g = a;
  p.g.wide_out = (reinterpret_cast<uintptr_t>(a.out) & 15u) == 0 && a.out_stride % (a.out_bf16 ? 8 : 4) == 0;
  p.kb_n = kb_n;
  p.nb_n = nb_n;
  p.err = ops_error_word();
  p.timeout_ns = 2000000000ll;
  if (p.err == nullptr || !tma_encode_init()) return cudaErrorInitializationError;
  const int bn = 256;
  const int64_t E = a.offsets ? a.n_groups : 1;
  bool ok = encode_kmajor_8bit(&p.a[2], a.a, a.K, a.m, 128) && encode_kmajor_8bit(&p.b, a.b, a.K, E * a.N, bn);
  if (ok && a.offsets)
    ok = encode_kmajor_8bit(&p.a[0], a.a, a.K, a.m, 32) && encode_kmajor_8bit(&p.a[1], a.a, a.K, a.m, 64);
  if (!ok) return cudaErrorInvalidValue;
  return a.out_bf16 ? launch_tc<256, true>(p, s) : launch_tc<256, false>(p, s);
}

}  // namespace epoch
