// Tiles of rows grouped by expert on the 5th-generation tensor cores: what the
// products of 8-bit, 4-bit and bf16 operands share. Bounded waits of a warp, the
// forms of the tensor core's instructions for two CTAs that work on one tile, and
// the walk over the tiles of groups whose sizes stand on the device.
#pragma once

#include "common.cuh"

namespace epoch {

constexpr int kBm = 128;  // rows of a CTA's tile
constexpr int kMaxGroups = 1024;

// mbar_wait_bounded for the short waits of these kernels, all on their critical path:
// the clock is first read after 256 attempts, not after the first.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int *abort, uint32_t *err,
                                         int64_t timeout_ns) {
  uint64_t t0 = 0;
  for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
    if ((i & 255u) != 0u) continue;
    if (*abort) return false;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) {
      t0 = now;
    } else if (now - t0 > static_cast<uint64_t>(timeout_ns)) {
      set_error(err, EPOCH_DEVERR_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
  return true;
}
// The whole warp waits; a phase that is complete already (the usual case, and then
// the loop's overhead is what counts) costs one attempt and a vote.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort, uint32_t *err,
                                          int64_t timeout_ns) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_for(bar, parity, abort, err, timeout_ns));
}

// True for one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// Forms for two CTAs that work on one tile (a cluster of two; their shared memory
// and TMEM are laid out alike). TMEM is allocated and freed by a warp of each; the
// first CTA's MMA thread issues the products of both, and its commit arrives on
// the barriers of both; copies of both count on the first CTA's barrier.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
template <bool PAIR> __device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    tc_commit(bar);
}
template <bool PAIR>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, int32_t c0, int32_t c1, uint32_t bar,
                                         uint64_t policy) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar), "l"(policy)
        : "memory");
  else
    tma_load_2d(dst, map, c0, c1, bar, policy);
}
// Arrives on a barrier of another CTA of the cluster (or its own; address from
// mapa_shared), after TMEM reads that have returned: nothing in memory has to be
// released to the other CTA (a release at cluster scope waits for every access of
// the warp, which made the whole product twice as slow).
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

template <int R> __device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R> __device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}

// A thread's 32 bytes of its own row: a whole sector (16-byte stores of halves of
// sectors took a fifth of the product's time at 8192 x 4096 x 4096).
__device__ __forceinline__ void store32(void *p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// First rows of the groups, in ascending order and within [0, m] whatever the
// caller's offsets hold (start, E + 1 entries), and the number of row tiles
// before each group (cum, E + 1 entries). One warp; E <= kMaxGroups.
__device__ inline void group_tiles(const int32_t *offsets, int E, int m, int tile, int *start, int *cum) {
  const int lane = lane_id(), per = (E + 32) / 32;  // entries of offsets [0, E] per lane
  const int lo = lane * per, hi = min(lo + per, E + 1);
#pragma unroll 4
  for (int i = lane; i <= E; i += 32) start[i] = min(max(__ldg(offsets + i), 0), m);
  __syncwarp();
  int mx = 0;
  for (int i = lo; i < hi; ++i) {
    mx = max(mx, start[i]);
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
// order) and column tile t % nt_n, so neighbouring CTAs share their rows. The
// CTA's rows of the tile are `rows` (0 or less: none) from row0 on.
struct TileWalk {
  const int *start, *cum;
  int E, nt_n, bm, first, e, total;
  __device__ TileWalk(const int *s, const int *c, int E_, int nt, int bm_, int rank)
      : start(s), cum(c), E(E_), nt_n(nt), bm(bm_), first(rank * kBm), e(0) {
    total = cum[E] * nt_n;
  }
  __device__ void at(int t, int *group, int *row0, int *rows, int *nt) {
    const int mt = t / nt_n;
    *nt = t - mt * nt_n;
    // the last group that starts at or before the tile, by halves (hundreds between two tiles may be empty)
    for (int hi = cum[e + 1] <= mt ? E - 1 : e; e < hi;) {
      const int mid = (e + hi + 1) / 2;
      if (cum[mid] <= mt) e = mid;
      else hi = mid - 1;
    }
    *group = e;
    *row0 = start[e] + (mt - cum[e]) * bm + first;
    *rows = min(kBm, start[e + 1] - *row0);
  }
};

}  // namespace epoch
