// Matrix product of e4m3 operands with a scale for each block of 128, dense or
// grouped by expert:
//
//   y[m, n] = sum over K blocks b of  sa[m, b] * sb[e, n / 128, b] * sum_{k in b} a[m, k] * w[e, n, k]
//
// where row m belongs to expert e of offsets[e] <= m < offsets[e + 1] (dense:
// one expert). Products of a K block are summed by the tensor cores; the
// scaled sums of the blocks are kept in fp32 registers and rounded once.
//
// Many rows (k_fp8_gemm): tiles of 128 rows x 256, 128, 64 or 32 columns, or of
// 256 x 256 by two CTAs whose tensor cores read both halves of the weights. A
// producer warp streams 128-byte-wide (one K block) operand tiles by TMA through
// a ring in shared memory, an MMA warp issues the tcgen05 products of one K block
// into one of two (narrow tiles: four) TMEM accumulators, and eight epilogue
// warps read the other, scale it and add it to their registers: the promotion of
// one block runs under the products of the next. What bounds it: TMEM serves one
// side at a time, so the reading of an accumulator (256 clocks at 256 columns)
// adds to its products (512) and a K block of a pair takes about 790 clocks;
// narrow tiles are taken where a round of wide ones would leave SMs idle.
// 8192 x 4096 x 4096 to bf16 95 us (2.9 PFLOP/s), to fp32 104 us; 256 experts of
// 1024 x 2048 with 8192 rows 93 us, where the weights' bytes bound it (6.1 TB/s). K is
// not split: 17 to 128 rows by 4096 x 4096 take 11 us, since 128 CTAs walk all of K.
//
// Few rows (k_fp8_small): bound by the weights' bytes; sixteen weight rows per
// CTA go from global memory straight into mma.sync fragments (see below). One row
// by 4096 x 2048: 3.1 us.
#include <cstring>
#include <mutex>

#include "common.cuh"
#include "fp8.cuh"
#include "layer.h"
#include "tiles.cuh"

namespace epoch {

namespace {

constexpr int kBk = 128;  // one scale block; 128 bytes: one swizzle row
constexpr int kEpiWarps = 8;
// Three warpgroups: producer, MMA and two warps for the scales, and the epilogue's two.
// The launch's 168 registers a thread are handed over: 56 to the first group,
// 224 to the others, whose sums alone take 128 (56 + 2 * 224 = 3 * 168).
constexpr int kThreads = 32 * (kEpiWarps + 4);
constexpr int kRegsFew = 56, kRegsMany = 224;

struct GemmParams {
  CUtensorMap a[3];  // boxes of 32, 64, 128 rows
  CUtensorMap b;     // boxes of the rows that a CTA loads
  CUtensorMap out;   // boxes of 128 bytes x 32 rows of the output (pairs)
  GemmArgs g;
  int kb_n, nb_n, nt_n;  // K blocks, N scale blocks, N tiles
  uint32_t *err;
  int64_t timeout_ns;
  uint32_t hold;  // bytes that a stage waits for beyond its copies': 0, but for the test of waits that run out
};

// Shape N x M of kind::f8f6f4 with e4m3 operands, fp32 accumulator, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
template <bool PAIR>
__device__ __forceinline__ void tc_mma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
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

__device__ __forceinline__ void load_tmem(uint32_t at, float (&v)[32]) { tmem_ld32(at, v); }
__device__ __forceinline__ void load_tmem(uint32_t at, float (&v)[16]) { tmem_ld16(at, v); }

// Tiles are BN columns wide. PAIR (BN = 256): two CTAs take 256 rows, each its own
// 128 rows of a and half of the weights' rows, which the products of both read.
template <int BN, bool PAIR> struct Geo {
  static_assert(!PAIR || BN == 256, "pairs work on 256 columns");
  static constexpr int bm = PAIR ? 2 * kBm : kBm;
  static constexpr int b_rows = PAIR ? BN / 2 : BN;
  static constexpr int stage = (kBm + b_rows) * kBk;
  static constexpr int stages = BN == 256 ? 4 : BN == 128 ? 6 : 8;
  static constexpr int bufs = BN == 256 ? 2 : 4;                           // TMEM accumulators
  static constexpr int tmem = bufs * BN;                                   // their columns
  static constexpr int out_bytes = PAIR ? kBm * BN * 2 : 0;                // 8 KB of the output a warp, on their way
  static constexpr int smem = 1024 + stages * stage + out_bytes;
};

template <int BN, bool PAIR, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) k_fp8_gemm(const __grid_constant__ GemmParams p) {
  using G = Geo<BN, PAIR>;
  constexpr int kCols = BN / 2;  // columns of an epilogue warpgroup
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * G::stages + 3 * G::bufs];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ float s_scale[G::bufs][2][kBm];  // a's scale times b's, for each row and epilogue half
  __shared__ int s_start[kMaxGroups + 1], s_cum[kMaxGroups + 1];
  const int warp = warp_id(), lane = lane_id();
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const int cta = PAIR ? blockIdx.x >> 1 : blockIdx.x, ctas = PAIR ? gridDim.x >> 1 : gridDim.x;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t full = smem_u32(bars), empty = full + 8 * G::stages, tfull = empty + 8 * G::stages,
                 tempty = tfull + 8 * G::bufs, sempty = tempty + 8 * G::bufs;
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
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < G::bufs; ++i) {
      mbar_init(tfull + 8 * i, 2);  // the products, and the scales
      mbar_init(tempty + 8 * i, PAIR ? 2 * kEpiWarps : kEpiWarps);  // accumulators read (both CTAs')
      mbar_init(sempty + 8 * i, kEpiWarps);                         // this CTA's scales read
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

  // warps 0 .. 7: epilogue; 8: producer; 9: MMA; 10, 11: scales
  if (warp >= kEpiWarps) {
    give_registers<kRegsFew>();
    if (warp == kEpiWarps) {  // ------------------------------------------------ producer
      const uint64_t keep = policy_evict_last(), pass = policy_evict_first();
      // weights of a tile's columns are read once per row tile; with one row tile a group they stream through
      const uint64_t wpol = p.g.offsets ? pass : keep;
      const uint32_t counts = PAIR ? mapa_shared(full, 0) : full;  // the barriers that the copies count on
      uint32_t it = 0, st = 0, phase = 1;
      bool ok = true;
      for (int t = cta; ok && t < walk.total; t += ctas) {
        int e, row0, rows, nt;
        walk.at(t, &e, &row0, &rows, &nt);
        // single CTAs load the smallest box that holds their rows
        const int box = PAIR || rows > 64 ? 2 : rows > 32 ? 1 : 0;
        const uint32_t bytes = (PAIR ? 2 * G::stage : ((32u << box) + BN) * kBk) + p.hold;
        const int brow = e * p.g.N + nt * BN + rank * G::b_rows;
        for (int kb = 0; kb < p.kb_n; ++kb, ++it) {
          ok = warp_wait(empty + 8 * st, phase, abort, p.err, p.timeout_ns);
          if (!ok) break;
          if (elect_one()) {
            const uint32_t dst = ring + st * G::stage;
            if (rank == 0) mbar_arrive_expect_tx(full + 8 * st, bytes);
            load_box<PAIR>(dst, &p.a[box], kb * kBk, row0, counts + 8 * st, keep);
            load_box<PAIR>(dst + kBm * kBk, &p.b, kb * kBk, brow, counts + 8 * st, wpol);
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
    } else if (warp >= kEpiWarps + 2) {  // ------------------------------------- scales, every other K block a warp
      uint32_t it = 0;
      bool ok = true;
      for (int t = cta; ok && t < walk.total; t += ctas) {
        int e, row0, rows, nt;
        walk.at(t, &e, &row0, &rows, &nt);
        const float *sa[4], *sb[2];
        float fa[4], fb[2];
#pragma unroll
        for (int i = 0; i < 4; ++i)  // rows behind the last one read a row that exists
          sa[i] = p.g.sa + static_cast<int64_t>(min(row0 + 32 * i + lane, p.g.m - 1)) * p.kb_n;
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
          ok = warp_wait(sempty + 8 * buf, ((i / G::bufs) & 1u) ^ 1u, abort, p.err, p.timeout_ns);
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
    } else if (warp == kEpiWarps + 1 && rank == 0) {  // ------------------------ MMA
      // The warp stays together and one elected lane issues: descriptors and barriers are then uniform values, which
      // the instructions take as they are. (From a single lane's branch, with the stage by division, a K block took
      // this warp 920 clocks at 256 x 256, against 512 of products.)
      constexpr uint32_t idesc = idesc_e4m3_f32(G::bm, BN);
      uint32_t it = 0, st = 0, phase = 0;
      bool ok = true;
      for (int t = cta; ok && t < walk.total; t += ctas) {
        for (int kb = 0; kb < p.kb_n; ++kb, ++it) {
          const uint32_t buf = it % G::bufs;
          const uint32_t free = ((it / G::bufs) & 1u) ^ 1u;
          const bool loaded = mbar_try_wait(full + 8 * st, phase), read = mbar_try_wait(tempty + 8 * buf, free);
          if (!__all_sync(0xffffffffu, loaded && read)) {
            ok = warp_wait(full + 8 * st, phase, abort, p.err, p.timeout_ns) &&
                 warp_wait(tempty + 8 * buf, free, abort, p.err, p.timeout_ns);
            if (!ok) break;
          }
          tc_fence_after();
          const uint32_t src = ring + st * G::stage;
          const uint64_t ad = sw128_kmajor_desc(src), bd = sw128_kmajor_desc(src + kBm * kBk);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kBk / 32; ++k)  // 32 columns (32 bytes) per instruction
              tc_mma_e4m3<PAIR>(tmem + buf * BN, ad + 2 * k, bd + 2 * k, idesc, k > 0);
            commit<PAIR>(tfull + 8 * buf);
            commit<PAIR>(empty + 8 * st);
          }
          __syncwarp();
          if (++st == G::stages) {
            st = 0;
            phase ^= 1u;
          }
        }
      }
      // no exit with products in flight: the last accumulators are complete
      for (uint32_t i = it > G::bufs ? it - G::bufs : 0; i < it; ++i) {
        int done = 0;
        wait_for(tfull + 8 * (i % G::bufs), (i / G::bufs) & 1u, &done, p.err, p.timeout_ns);
      }
    }
  } else {  // ------------------------------------------------------------------ epilogue
    take_registers<kRegsMany>();
    const uint32_t read = PAIR ? mapa_shared(tempty, 0) : tempty;  // the barriers that the MMA thread waits on
    auto release = [&](uint32_t buf) {
      __syncwarp();
      if (lane != 0) return;
      if constexpr (PAIR) arrive_cluster(read + 8 * buf);
      else mbar_arrive(read + 8 * buf);
      mbar_arrive(sempty + 8 * buf);
    };
    const int quarter = warp & 3, half = warp >> 2;  // TMEM lanes 32 quarter .. + 32, columns kCols half .. + kCols
    uint32_t it = 0;
    bool ok = true;
    for (int t = cta; ok && t < walk.total; t += ctas) {
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
        if constexpr (PAIR) ok = warp_wait(tfull + 8 * buf, (it / G::bufs) & 1u, abort, p.err, p.timeout_ns);
        else ok = __all_sync(0xffffffffu, wait_for(tfull + 8 * buf, (it / G::bufs) & 1u, abort, p.err, p.timeout_ns));
        if (!ok) break;
        if (any) {
          // The accumulator is free for the products after the next ones as soon as its last columns are on their
          // way, so loads go in two rounds of two (a load answers after 200 clocks and more) and the sums follow.
          tc_fence_after();
          const uint32_t src = tmem + buf * BN + half * kCols + (static_cast<uint32_t>(quarter * 32) << 16);
          constexpr int kLoad = kCols < 32 ? kCols : 32;
          float v0[kLoad], v1[kLoad];
          load_tmem(src, v0);
          if constexpr (kCols > 32) load_tmem(src + 32, v1);
          const float s = s_scale[buf][half][r];
          const uint64_t s2 = pair(s, s);
          tmem_ld_wait();
          if constexpr (kCols == 128) {
            add_scaled(acc, v0, s2);
            load_tmem(src + 64, v0);
            add_scaled(acc + 16, v1, s2);
            load_tmem(src + 96, v1);
            tmem_ld_wait();
          }
          tc_fence_before();
          release(buf);
          add_scaled(acc + (kCols == 128 ? 32 : 0), v0, s2);
          if constexpr (kCols > 32) add_scaled(acc + (kCols == 128 ? 48 : 16), v1, s2);
        } else {
          release(buf);
        }
      }
      // A pair's warp whose 32 rows all exist leaves its part to bulk stores, which run under the next tile's products
      // (rows behind a group's last one belong to another tile: such a warp stores row by row). They take 128 bytes of
      // each row at a time, from two places in shared memory in turn.
      bool stored = false;
      if constexpr (PAIR) {
        if (ok && p.g.bulk_out && rows >= quarter * 32 + 32 && n0 < p.g.N) {
          stored = true;
          // columns of a part, and parts of one commit: a bf16 warp's two fit the two places, four of fp32 take turns
          constexpr int kPart = BF16 ? 64 : 32, kTogether = BF16 ? 2 : 1;
          uint8_t *places = smem_raw + (ring - smem_u32(smem_raw)) + G::stages * G::stage + warp * 8192;
#pragma unroll
          for (int h0 = 0; h0 < kCols / kPart; h0 += kTogether) {
            if (n0 + kPart * h0 >= p.g.N) break;
            // What was here has left. A tile begins with the first place whichever the last one ended with (one part or
            // three of fp32 at the last columns of N: the first), so all of that tile's stores have to have read theirs.
            if (lane == 0) {
              if (h0 == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
              else asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(2 / kTogether - 1) : "memory");
            }
            __syncwarp();
#pragma unroll
            for (int h = h0; h < h0 + kTogether; ++h) {
#pragma unroll
              for (int c = 0; c < 8; ++c) {  // 16 bytes at a time, in the 128-byte swizzle
                uint32_t w[4];
                if constexpr (BF16) {
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    const float2 f = unpair(acc[32 * h + 4 * c + j]);
                    const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
                    w[j] = *reinterpret_cast<const uint32_t *>(&v);
                  }
                } else {
#pragma unroll
                  for (int j = 0; j < 2; ++j) {
                    const float2 f = unpair(acc[16 * h + 2 * c + j]);
                    w[2 * j] = __float_as_uint(f.x);
                    w[2 * j + 1] = __float_as_uint(f.y);
                  }
                }
                *reinterpret_cast<uint4 *>(places + (h & 1) * 4096 + lane * 128 + ((c ^ (lane & 7)) << 4)) =
                    make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
#pragma unroll
              for (int h = h0; h < h0 + kTogether; ++h)
                if (n0 + kPart * h < p.g.N)
                  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                                   reinterpret_cast<uint64_t>(&p.out)),
                               "r"(n0 + kPart * h), "r"(row0 + quarter * 32), "r"(smem_u32(places) + 4096 * (h & 1))
                               : "memory");
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
          }
        }
      }
      if (ok && on && !stored) {
        const int n = min(kCols, p.g.N - n0);
        if constexpr (BF16) {
          __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.g.out) + static_cast<int64_t>(row) * p.g.out_stride + n0;
          if (p.g.wide_out && n == kCols) {
#pragma unroll
            for (int c = 0; c < kCols / 2; c += 8) {
              uint32_t w[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float2 f = unpair(acc[c + j]);
                const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
                w[j] = *reinterpret_cast<const uint32_t *>(&h);
              }
              store32(dst + 2 * c, w);
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
            for (int c = 0; c < kCols / 2; c += 4) {
              uint32_t w[8];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 f = unpair(acc[c + j]);
                w[2 * j] = __float_as_uint(f.x);
                w[2 * j + 1] = __float_as_uint(f.y);
              }
              store32(dst + 2 * c, w);
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
  if constexpr (PAIR) {  // no exit with stores still reading shared memory
    if (warp < kEpiWarps && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
  }
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
    for (int kb0 = warp; kb0 < kb_n; kb0 += 2 * kSmallWarps) {
      uint4 wa[2][2], wb[2][2];  // two blocks' weights on their way together
      float sw[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int kb = kb0 + b * kSmallWarps;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = kb * kFp8Block + 64 * h;
          const bool in = k + 16 * t < a.K;  // false for a block behind the last one
          wa[b][h] = load16(w + k, w0 && in);
          wb[b][h] = load16(w + k + static_cast<int64_t>(8) * a.K, w1 && in);
        }
        sw[b] = kb < kb_n ? __ldg(sb + kb) : 0.f;
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int kb = kb0 + b * kSmallWarps;
        if (kb >= kb_n) break;
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
            mma_e4m3(part, wa[b][h].x, wb[b][h].x, wa[b][h].y, wb[b][h].y, xv.x, xv.y);
            mma_e4m3(part, wa[b][h].z, wb[b][h].z, wa[b][h].w, wb[b][h].w, xv.z, xv.w);
          }
          const int c0 = i * 8 + 2 * t;
          const float s0 = c0 < rows ? __ldg(a.sa + static_cast<int64_t>(row0 + c0) * kb_n + kb) * sw[b] : 0.f;
          const float s1 = c0 + 1 < rows ? __ldg(a.sa + static_cast<int64_t>(row0 + c0 + 1) * kb_n + kb) * sw[b] : 0.f;
          acc[i][0] = fmaf(part[0], s0, acc[i][0]);
          acc[i][1] = fmaf(part[1], s1, acc[i][1]);
          acc[i][2] = fmaf(part[2], s0, acc[i][2]);
          acc[i][3] = fmaf(part[3], s1, acc[i][3]);
        }
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

template <int BN, bool PAIR, bool BF16> cudaError_t launch_tc(GemmParams &p, cudaStream_t s) {
  using G = Geo<BN, PAIR>;
  auto *fn = &k_fp8_gemm<BN, PAIR, BF16>;
  static std::mutex mu;
  static int resident[64] = {};  // CTAs that a device holds at once
  int dev = 0, most = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
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
    if (resident[dev & 63] == 0) {
      e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, G::smem);
      if (e != cudaSuccess) return e;
      int n = num_sms();
      if (PAIR) {
        cfg.gridDim = dim3(static_cast<unsigned>(num_sms() / 2 * 2));
        e = cudaOccupancyMaxActiveClusters(&n, fn, &cfg);
        if (e != cudaSuccess) return e;
        n *= 2;
      }
      resident[dev & 63] = n;
    }
    most = resident[dev & 63];
  }
  if (most < (PAIR ? 2 : 1)) return cudaErrorNotSupported;
  p.nt_n = (p.g.N + BN - 1) / BN;
  // row tiles: at most one partial tile a group beyond the full ones
  const int64_t mt = p.g.offsets ? p.g.m / G::bm + p.g.n_groups : (p.g.m + G::bm - 1) / G::bm;
  const int64_t ctas = mt * p.nt_n * (PAIR ? 2 : 1);
  cfg.gridDim = dim3(static_cast<unsigned>(ctas < most ? ctas : most));
  return cudaLaunchKernelEx(&cfg, fn, p);
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

// The kernel a product takes: 0 the one for few rows, else the columns of a tile of single CTAs, kFp8Pairs tiles of CTA
// pairs. n_groups 0: dense.
int fp8_gemm_kernel(int n_groups, int64_t m, int64_t N, int sms) {
  // Few rows: the weights' bytes and latency bound the time. Rows of one expert cost mma.sync products (4096 x 4096:
  // 6.2 us at 8 rows, 8.1 at 16, 14 at 32, where the tiles below take 13), rows of several experts hardly.
  if (m <= (n_groups ? kSmallTokens : 16)) return 0;
  const int64_t E = n_groups ? n_groups : 1;
  // The tile: the one whose rounds of tiles take the least time, by the clocks that a K block of each took. Pairs
  // need groups that fill 256 rows.
  const int64_t mt = m / kBm + (n_groups ? (E < m ? E : m) : (m % kBm != 0));
  auto cost = [&](int64_t tiles, int64_t at_once, int64_t clocks) { return (tiles + at_once - 1) / at_once * clocks; };
  int bn = 256;
  int64_t best = cost(mt * ((N + 255) / 256), sms, 1000);
  const int64_t narrow[3][2] = {{128, 720}, {64, 600}, {32, 560}};
  for (const auto &c : narrow) {
    const int64_t t = cost(mt * ((N + c[0] - 1) / c[0]), sms, c[1]);
    if (t < best) {
      best = t;
      bn = static_cast<int>(c[0]);
    }
  }
  if (m >= 256 * E && sms >= 2) {
    const int64_t tiles = (m / 256 + (n_groups ? E : m % 256 != 0)) * ((N + 255) / 256);
    if (cost(tiles, sms / 2, 800) <= best) return kFp8Pairs;
  }
  return bn;
}

cudaError_t launch_fp8_gemm(const GemmArgs &a, cudaStream_t s, int64_t timeout_ns, uint32_t hold) {
  const int kb_n = (a.K + kBk - 1) / kBk, nb_n = (a.N + kFp8Block - 1) / kFp8Block;
  const int kernel = fp8_gemm_kernel(a.offsets ? a.n_groups : 0, a.m, a.N, num_sms());
  if (kernel == 0) {
    if (a.m <= 8) return launch_small<1>(a, kb_n, nb_n, s);
    if (a.m <= 16) return launch_small<2>(a, kb_n, nb_n, s);
    if (a.m <= 32) return launch_small<4>(a, kb_n, nb_n, s);
    return launch_small<8>(a, kb_n, nb_n, s);
  }
  GemmParams p;
  memset(&p, 0, sizeof(p));
  p.g = a;
  p.g.wide_out = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0 && a.out_stride % (a.out_bf16 ? 16 : 8) == 0;
  p.kb_n = kb_n;
  p.nb_n = nb_n;
  p.err = ops_error_word();
  p.timeout_ns = timeout_ns;
  p.hold = hold;
  if (p.err == nullptr || !tma_encode_init()) return cudaErrorInitializationError;
  const int64_t E = a.offsets ? a.n_groups : 1;
  const bool pairs = kernel == kFp8Pairs;
  const uint32_t b_rows = pairs ? Geo<256, true>::b_rows : kernel;
  bool ok = encode_kmajor_8bit(&p.a[2], a.a, a.K, a.m, 128) && encode_kmajor_8bit(&p.b, a.b, a.K, E * a.N, b_rows);
  if (ok && !pairs && (a.offsets || a.m % kBm != 0))
    ok = encode_kmajor_8bit(&p.a[0], a.a, a.K, a.m, 32) && encode_kmajor_8bit(&p.a[1], a.a, a.K, a.m, 64);
  // Bulk stores end a row on a 16-byte boundary: with another N they write zeros into the columns behind it.
  const int per16 = a.out_bf16 ? 8 : 4;
  if (ok && pairs && (reinterpret_cast<uintptr_t>(a.out) & 15u) == 0 && a.out_stride % per16 == 0 && a.N % per16 == 0) {
    ok = encode_rows(&p.out, a.out, a.out_bf16, a.N, a.m, a.out_stride);
    p.g.bulk_out = 1;
  }
  if (!ok) return cudaErrorInvalidValue;
  if (pairs) return a.out_bf16 ? launch_tc<256, true, true>(p, s) : launch_tc<256, true, false>(p, s);
  if (kernel == 256) return a.out_bf16 ? launch_tc<256, false, true>(p, s) : launch_tc<256, false, false>(p, s);
  if (kernel == 128) return a.out_bf16 ? launch_tc<128, false, true>(p, s) : launch_tc<128, false, false>(p, s);
  if (kernel == 64) return a.out_bf16 ? launch_tc<64, false, true>(p, s) : launch_tc<64, false, false>(p, s);
  return a.out_bf16 ? launch_tc<32, false, true>(p, s) : launch_tc<32, false, false>(p, s);
}

}  // namespace epoch
