// The whole MoE layer for a few tokens in one launch: router, top-k, routed and
// shared SwiGLU experts, weighted sum (epoch_moe_few).
//
//   G = x W_r^T (+ b);  S_t, w_t = the layer's router rule over every expert
//   y_t = sum_{e in S_t} w_te W_down,e (silu(W_gate,e x_t) * (W_up,e x_t)) + sum_shared (+ x_t)
//
// With at most 64 tokens the bytes of the selected experts' weights bound the
// time, so the kernel is built around reading each of them from memory once,
// straight into registers, with loads always in flight. (Eight tokens share a
// reading; an expert of more has its rows read again from L2 for every eight: 43
// tokens on 12 experts take 2.8 times their floor, a block on 47 experts 1.5 times.) One CTA per SM
// stays for the whole call; its phases are separated by grid barriers:
//
//   0. router logits, and the shared experts' activations, which need no routing;
//      -- barrier --  every CTA takes every token's top-k for itself, one a warp
//      (more than 16 tokens: one a CTA, and one more barrier), and sorts the edges
//      by expert in shared memory;
//   1. activations a = silu(gate) * up of every (token, expert) edge;
//      -- barrier --  (the first down weights are already in flight)
//   2. down products, fp32 per edge;
//      -- barrier --
//   3. y: the edges' sums in selection order.
//
// A group of warps works on 16 weight rows and splits K. Thread (g, t) of a warp
// (g = lane / 4, t = lane % 4) loads 16 consecutive bytes of row g and of row g + 8
// (64 bytes of a row by four threads): the order of the products along K is
// free, so these are operand fragments of two m16n8k16 products as they come, and
// the same bytes of eight tokens' rows are the other operand. In phase 1 rows
// 0-7 are gate rows and rows 8-15 the up rows of the same eight columns, so one
// tile of sums holds both halves of the SwiGLU.
//
// Sums are split into a fixed number of parts that meet in a fixed order, and a
// token is a column of its own in every product, so a token's result is the same
// bits whatever its neighbours and however often it is computed. Rounding: the
// activations of bf16 layers, which are an operand of the tensor core, to two bf16
// values each (16 bits), and y; everything else is fp32.
//
// fp32 layers run the same schedule with FFMA in place of the tensor core.
//
// Measured (H 2048, 256 experts of 512 columns, 8 and 1 shared a token, bf16;
// weights from memory): 1 token 21.6 us, of which 8 us are phases 1 and 2 and
// 1.1 us each barrier; 32 tokens (47 experts) 66 us at 4.6 TB/s, phase 1 at 7
// and phase 2 at 5.2 TB/s (its activations are as many bytes as its weights, phase
// 1's tokens half of them). Reading a unit's rows only (no products, no barriers)
// reaches 6.1 to 6.4 TB/s at 400 MB with these loads. Other ways for the two parts of
// the activations, at 32 tokens where this one took 67 us: the second parts read where they
// are used 75, tokens' rows asked for one chunk ahead and not two 71, two tiles of
// weight rows for a group's activations 68.
#include <atomic>
#include <cfloat>
#include <climits>
#include <cstring>

#include "common.cuh"
#include "layer.h"
#include "topk.cuh"

namespace epoch {

namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxEdges = kFewTokens * 16;

// ------------------------------------------------------------------ element types
template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
  static constexpr int step = 32, per = 8;  // columns of a K step (64 bytes of a row), and of a thread in it
  static constexpr int steps = 4;           // K steps loaded together: a chunk
  static constexpr int acc = 4;             // fp32 sums a thread keeps of a 16 x 8 tile while adding along K
};
template <> struct Elem<float> {
  static constexpr int step = 16, per = 4;
  static constexpr int steps = 2;           // its sums and the tokens' columns need the registers of the other two
  static constexpr int acc = 16;            // rows g and g + 8 of all eight tokens (this thread's columns only)
};

__device__ __forceinline__ uint4 load_weights(const void *p, bool ok) {
  uint4 u = make_uint4(0u, 0u, 0u, 0u);
  if (ok)
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(p));
  return u;
}
// Token rows, through L1: x, which nobody writes during the call, and (FRESH)
// activations that other SMs wrote before the grid barrier, whose acquire makes
// plain loads see them.
template <bool FRESH> __device__ __forceinline__ uint4 load_tokens(const void *p) {
  uint4 u;
  if constexpr (FRESH)
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p) : "memory");
  else
    u = __ldg(static_cast<const uint4 *>(p));
  return u;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Barrier of the `warps` warps of group `id` (hardware barrier id + 1 where there is more than one).
__device__ __forceinline__ void group_sync(int id, int warps) {
  if (warps == 1) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(warps * 32) : "memory");
}

// Grid barrier in two halves. Every CTA arrives once on *ctr (zero before the
// launch's first arrival); the wait ends when `want` have (the grid, but for the test of
// a wait that runs out), or gives up (false). Loads issued between the halves do not
// hold the arrival back.
__device__ __forceinline__ void grid_arrive(int32_t *ctr) {
  __syncthreads();
  if (threadIdx.x == 0) asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(ctr) : "memory");
}
__device__ bool grid_wait(const int32_t *ctr, int32_t want, uint32_t *err, int64_t timeout_ns) {
  __shared__ int s_ok;
  if (threadIdx.x == 0) {
    auto seen = [&] {
      int32_t v;
      asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(ctr) : "memory");
      return v;
    };
    int ok = 1;
    if (seen() < want) {
      const uint64_t t0 = globaltimer_ns();
      for (uint32_t i = 1; seen() < want; ++i)
        if ((i & 7u) == 0u && globaltimer_ns() - t0 > static_cast<uint64_t>(timeout_ns)) {
          set_error(err, EPOCH_DEVERR_TIMEOUT);
          ok = 0;
          break;
        }
    }
    s_ok = ok;
  }
  __syncthreads();
  return s_ok != 0;
}

// A unit's share of one warp, as a thread sees it: its columns of weight rows g
// and g + 8 (rows behind the last one read it again: their sums go nowhere), the
// row of its token g (behind the last token one repeats: every token is a column
// of its own), and the warp's K steps, a whole number of chunks.
struct Share {
  const char *p0, *p1;
  int row;           // where the token's row starts
  int count;         // tokens of the unit, at most 8
  int step, end, k;  // K steps, columns of a row
};

// FRESH: the tokens' rows are activations, in bf16 layers of two parts each, whose
// registers leave fewer for the weights on their way.
template <typename T, bool FRESH> struct Chunk {
  static constexpr int n = FRESH && sizeof(T) == 2 ? Elem<T>::steps / 2 : Elem<T>::steps;  // K steps
  uint4 a[n], b[n];                                     // weight rows g and g + 8
  uint4 v[sizeof(T) == 2 ? (FRESH ? 2 * n : n) : 1];  // token row g (bf16)
};

// Whether columns of a K step that a thread holds exist: rows of bf16 layers are
// a whole number of chunks.
template <typename T> __device__ __forceinline__ bool in_row(int c, int k) { return sizeof(T) == 2 || c < k; }

template <typename T, bool FRESH>
__device__ __forceinline__ void load_rows(const Share &w, int step, Chunk<T, FRESH> &c) {
  const int c0 = step * Elem<T>::step, ct = c0 + (lane_id() & 3) * Elem<T>::per;
  const char *p0 = w.p0 + static_cast<int64_t>(c0) * sizeof(T), *p1 = w.p1 + static_cast<int64_t>(c0) * sizeof(T);
#pragma unroll
  for (int j = 0; j < c.n; ++j) {
    const bool in = in_row<T>(ct + j * Elem<T>::step, w.k);
    c.a[j] = load_weights(p0 + 64 * j, in);
    c.b[j] = load_weights(p1 + 64 * j, in);
  }
}
template <typename T, bool FRESH>
__device__ __forceinline__ void load_token(const Share &w, int step, const T *x, Chunk<T, FRESH> &c) {
  const int c0 = step * Elem<T>::step + (lane_id() & 3) * Elem<T>::per;
  if constexpr (sizeof(T) == 2 && FRESH) {
    const T *row = x + w.row + 2 * c0;  // eight leading parts, then their eight rests
#pragma unroll
    for (int j = 0; j < c.n; ++j)
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(c.v[2 * j].x), "=r"(c.v[2 * j].y), "=r"(c.v[2 * j].z), "=r"(c.v[2 * j].w),
                     "=r"(c.v[2 * j + 1].x), "=r"(c.v[2 * j + 1].y), "=r"(c.v[2 * j + 1].z), "=r"(c.v[2 * j + 1].w)
                   : "l"(row + 2 * j * Elem<T>::step)
                   : "memory");
  } else if constexpr (sizeof(T) == 2) {
    const T *row = x + w.row + c0;
#pragma unroll
    for (int j = 0; j < c.n; ++j) c.v[j] = load_tokens<FRESH>(row + j * Elem<T>::step);
  }
}

// Adds a chunk's products to the sums. The fp32 form reads the tokens' rows here,
// four tokens' loads on their way together: a thread's sums are of every token.
template <typename T, bool FRESH>
__device__ __forceinline__ void add_chunk(const Share &w, int step, const Chunk<T, FRESH> &c, const T *x,
                                          float (&acc)[Elem<T>::acc]) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int j = 0; j < c.n * (FRESH ? 2 : 1); ++j) {
      const uint4 &a = c.a[FRESH ? j / 2 : j], &b = c.b[FRESH ? j / 2 : j];
      mma_bf16(acc, a.x, b.x, a.y, b.y, c.v[j].x, c.v[j].y);
      mma_bf16(acc, a.z, b.z, a.w, b.w, c.v[j].z, c.v[j].w);
    }
  } else {
    const int c0 = step * Elem<T>::step + (lane_id() & 3) * Elem<T>::per;
#pragma unroll
    for (int n = 0; n < 8; n += 4) {
      if (n >= w.count) break;
      uint4 v[4][Elem<T>::steps];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const T *row = x + __shfl_sync(0xffffffffu, w.row, 4 * (n + m)) + c0;
#pragma unroll
        for (int j = 0; j < Elem<T>::steps; ++j) {
          v[m][j] = make_uint4(0u, 0u, 0u, 0u);
          if (in_row<T>(c0 + j * Elem<T>::step, w.k)) v[m][j] = load_tokens<FRESH>(row + j * Elem<T>::step);
        }
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        float s = acc[n + m], q = acc[8 + n + m];
#pragma unroll
        for (int j = 0; j < Elem<T>::steps; ++j) {
          const float v0 = __uint_as_float(v[m][j].x), v1 = __uint_as_float(v[m][j].y),
                      v2 = __uint_as_float(v[m][j].z), v3 = __uint_as_float(v[m][j].w);
          s = fmaf(__uint_as_float(c.a[j].x), v0, s);
          s = fmaf(__uint_as_float(c.a[j].y), v1, s);
          s = fmaf(__uint_as_float(c.a[j].z), v2, s);
          s = fmaf(__uint_as_float(c.a[j].w), v3, s);
          q = fmaf(__uint_as_float(c.b[j].x), v0, q);
          q = fmaf(__uint_as_float(c.b[j].y), v1, q);
          q = fmaf(__uint_as_float(c.b[j].z), v2, q);
          q = fmaf(__uint_as_float(c.b[j].w), v3, q);
        }
        acc[n + m] = s;
        acc[8 + n + m] = q;
      }
    }
  }
}

// Part `part` of column col of an activation row. bf16 keeps eight columns' leading
// parts and then what is left of each, together 16 bits of a value (activations rounded
// to one bf16 raised y's error against 64 bits from 0.0017 to 0.0025 of its size);
// infinities leave nothing. The sixteen parts are one sector.
__device__ __forceinline__ void put_act(float *row, int col, int, float v) { row[col] = v; }
__device__ __forceinline__ void put_act(__nv_bfloat16 *row, int col, int part, float v) {
  if (part) {
    const float lead = __bfloat162float(__float2bfloat16_rn(v));
    v = fabsf(lead) <= FLT_MAX ? v - lead : 0.f;
  }
  row[(col >> 3) * 16 + part * 8 + (col & 7)] = __float2bfloat16_rn(v);
}

// A warp's sums to shared memory as [16 rows][8 tokens].
template <typename T> __device__ __forceinline__ void put_tile(float *d, const float (&acc)[Elem<T>::acc]) {
  const int lane = lane_id(), g = lane >> 2, t = lane & 3;
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<float2 *>(d + g * 8 + 2 * t) = make_float2(acc[0], acc[1]);
    *reinterpret_cast<float2 *>(d + (g + 8) * 8 + 2 * t) = make_float2(acc[2], acc[3]);
  } else {
#pragma unroll
    for (int n = 0; n < 8; ++n) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float s = acc[8 * h + n];  // over the four threads of the row
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        if (t == 0) d[(g + 8 * h) * 8 + n] = s;
      }
    }
  }
}

// Runs the units u = first, first + stride, ... < n of one phase on a group of
// `warps` warps (this warp is number `w` of group `gid`). Partial sums meet in
// `part` ([2][warps][128], alternating halves, so one group barrier a unit),
// from which `finish` takes them. Two chunks are always on their way: a chunk's
// registers are loaded again, with the unit's next columns or the next unit's
// first, as soon as its products are issued. `ready` runs once, after the first
// weights are asked for and before any token's row: the wait for the grid
// barrier before the phase, if any.
template <typename T, bool FRESH, typename Locate, typename Finish, typename Ready>
__device__ __forceinline__ bool run_units(int first, int stride, int n, int w, int warps, int gid, float *part,
                                          const T *x, Locate locate, Finish finish, Ready ready) {
  Chunk<T, FRESH> c0, c1;
  constexpr int kSteps = Chunk<T, FRESH>::n;
  Share cur;
  int u = first;
  if (u < n) {
    locate(u, w, warps, cur);
    if (cur.step < cur.end) load_rows<T, FRESH>(cur, cur.step, c0);
    if (cur.step + kSteps < cur.end) load_rows<T, FRESH>(cur, cur.step + kSteps, c1);
  }
  if (!ready()) return false;
  if (u < n) {
    if (cur.step < cur.end) load_token<T, FRESH>(cur, cur.step, x, c0);
    if (cur.step + kSteps < cur.end) load_token<T, FRESH>(cur, cur.step + kSteps, x, c1);
  }
  int half = 0;
  while (u < n) {
    float acc[Elem<T>::acc];
#pragma unroll
    for (int j = 0; j < Elem<T>::acc; ++j) acc[j] = 0.f;
    const int un = u + stride;
    Share now = cur;
    do {
      int ns = now.step + 2 * kSteps;  // what the registers hold next
      if (now.step < now.end) add_chunk<T, FRESH>(now, now.step, c0, x, acc);
      if (ns >= now.end) {
        cur.end = 0;  // nothing left to load
        if (un < n) locate(un, w, warps, cur);
        ns = cur.step;
      }
      if (ns < cur.end) {
        load_rows<T, FRESH>(cur, ns, c0);
        load_token<T, FRESH>(cur, ns, x, c0);
      }
      if (now.step + kSteps < now.end) add_chunk<T, FRESH>(now, now.step + kSteps, c1, x, acc);
      if (ns + kSteps < cur.end) {
        load_rows<T, FRESH>(cur, ns + kSteps, c1);
        load_token<T, FRESH>(cur, ns + kSteps, x, c1);
      }
      now.step += 2 * kSteps;
    } while (now.step < now.end);
    float *mine = part + (half * warps) * 128;
    put_tile<T>(mine + w * 128, acc);
    group_sync(gid, warps);
    finish(u, now.count, mine);
    half ^= 1;
    u = un;
  }
  return true;
}

// Warps of a group in phases 1 and 2, for rows of `bytes` bytes: at most four, and
// no more than leave each of them 512 bytes of a row (two chunks of bf16, four of fp32).
__device__ __forceinline__ int split_of(int bytes) { return bytes >= 2048 ? 4 : bytes >= 1024 ? 2 : 1; }

struct FewParams {
  Dims d;
  Weights w;
  FewWork ws;
  const void *x;
  void *y;
  uint32_t *err;
  int n_tok;
  int hold;  // grid barrier that waits for one CTA more than there are (a test's), or -1
};

// Routing tables of a CTA, in shared memory. A job is at most eight tokens of an
// expert: its units cost the same whatever the routing, and the weights that the
// jobs of a busy expert share come from memory once and from L2 the other times.
struct Routes {
  int16_t sel[kMaxEdges];   // expert of edge t * k + j
  float wgt[kMaxEdges];     // its weight
  int16_t list[kMaxEdges];  // edges by expert,
  int16_t tok[kMaxEdges];   // and their tokens
  int16_t job_expert[kMaxEdges], job_first[kMaxEdges], job_n[kMaxEdges];
  uint32_t mask[1024][2];   // tokens of each expert
  int16_t first[1024];      // its first entry in list
  int32_t warp_sum[kWarps];
  int32_t n_jobs;
};

// Group rule of the sigmoid router (see warp_group_limit) over the scores c of
// every expert, lane l holding the EPL consecutive ones from l * EPL on: clears ok
// outside the chosen groups. Where a group is the experts of 1, 2, 4, .. lanes
// these merge their two best; otherwise the groups are taken one by one, without a
// branch (10 tokens, 4 groups of 35: 25.9 us a call; warp_group_limit, which counts
// eligible experts and divides for each, 37.2).
template <int EPL>
__device__ __forceinline__ void limit_groups(const float (&c)[EPL], bool (&ok)[EPL], const Dims &d) {
  constexpr unsigned kAll = 0xffffffffu;
  const int gs = d.E / d.n_group, lanes = gs / EPL, lane = lane_id();
  if (gs % EPL != 0 || (lanes & (lanes - 1)) != 0) {
    int8_t id[EPL];  // group of each expert (32 groups at most)
    int at = lane * EPL / gs, left = gs - (lane * EPL - at * gs);
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      id[j] = static_cast<int8_t>(min(at, 31));  // lanes behind the last expert hold no key
      if (--left == 0) {
        ++at;
        left = gs;
      }
    }
    float score = -INFINITY;  // lane g: group g's
    for (int g = 0; g < d.n_group; ++g) {
      unsigned k1 = 0u, k2 = 0u;  // this lane's two best keys of the group
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const unsigned q = ok[j] && id[j] == g ? order_key(c[j]) : 0u;
        k2 = max(k2, min(k1, q));
        k1 = max(k1, q);
      }
      const unsigned m1 = __reduce_max_sync(kAll, k1);
      const unsigned holder = __ffs(__ballot_sync(kAll, k1 == m1)) - 1;
      const unsigned m2 = __reduce_max_sync(kAll, lane == holder ? k2 : k1);
      if (lane == g) score = m2 == 0u ? key_value(m1) : key_value(m1) + key_value(m2);
    }
    int rank = 0;
    for (int g = 0; g < d.n_group; ++g) {
      const float o = __shfl_sync(kAll, score, g);
      rank += o > score || (o == score && g < lane);
    }
    const unsigned chosen = __ballot_sync(kAll, lane < d.n_group && (rank < d.topk_group || rank * gs < d.k));
#pragma unroll
    for (int j = 0; j < EPL; ++j) ok[j] = ok[j] && (chosen >> id[j] & 1u);
    return;
  }
  unsigned k1 = 0u, k2 = 0u;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const unsigned q = ok[j] ? order_key(c[j]) : 0u;
    k2 = max(k2, min(k1, q));
    k1 = max(k1, q);
  }
  for (int o = 1; o < lanes; o <<= 1) {
    const unsigned q1 = __shfl_xor_sync(kAll, k1, o), q2 = __shfl_xor_sync(kAll, k2, o);
    k2 = max(max(k2, q2), min(k1, q1));
    k1 = max(k1, q1);
  }
  // a lane past the last expert holds no key, and its score ranks behind every group's
  const float score = k1 == 0u ? -INFINITY : k2 == 0u ? key_value(k1) : key_value(k1) + key_value(k2);
  const int mine = lane / lanes;
  int rank = 0;
  for (int g = 0; g < d.n_group; ++g) {
    const float o = __shfl_sync(kAll, score, g * lanes);
    rank += o > score || (o == score && g < mine);
  }
  const bool open = rank < d.topk_group || rank * gs < d.k;
#pragma unroll
  for (int j = 0; j < EPL; ++j) ok[j] = ok[j] && open;
}

// Top-k of one warp's scores (lane l holds the EPL consecutive experts from
// l * EPL on; order: score, then lower id first). On return the lane that holds
// selection j < k has *rank = j, its expert and its score; the others a rank of k
// or more. Every lane's best key is ranked among the lanes' bests; the k-th of
// them is a bound that the k best keys reach and few others do. Those are
// compacted into `scratch` (32 entries of this warp) and ranked against each
// other. All steps but the last are without loops or branches: a selection is
// a chain of latencies (k rounds of a warp maximum took 2100 clocks for 8 of 256).
template <int EPL>
__device__ __forceinline__ void rank_topk(const float (&c)[EPL], const bool (&ok)[EPL], int k, int *rank, int *sel,
                                          float *val, uint2 *scratch) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = lane_id();
  unsigned key[EPL];  // 0: not eligible (every key of a score is above it)
#pragma unroll
  for (int j = 0; j < EPL; ++j) key[j] = ok[j] ? order_key(c[j]) : 0u;
  unsigned best = 0u;
#pragma unroll
  for (int j = 0; j < EPL; ++j) best = max(best, key[j]);
  int r = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) r += __shfl_sync(kAll, best, i) >= best + (i < lane ? 0u : 1u);
  const unsigned holder = __ballot_sync(kAll, r == k - 1);
  const unsigned bound = max(__shfl_sync(kAll, best, __ffs(holder) - 1), 1u);
  unsigned pass[EPL];
  int total = 0, at[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) pass[j] = __ballot_sync(kAll, key[j] >= bound);
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    at[j] = total + __popc(pass[j] & ((1u << lane) - 1u));
    total += __popc(pass[j]);
  }
  if (total > 32) {  // many equal keys, or most of the experts selected
    *sel = -1;
    warp_topk_rounds<EPL>(key, k, sel, val);
    *rank = *sel < 0 ? k : lane;
    return;
  }
  if (lane >= total) scratch[lane] = make_uint2(0u, 0u);
#pragma unroll
  for (int j = 0; j < EPL; ++j)
    if (key[j] >= bound) scratch[at[j]] = make_uint2(key[j], ~static_cast<unsigned>(lane * EPL + j));
  __syncwarp();
  auto order = [](uint2 q) { return static_cast<uint64_t>(q.x) << 32 | q.y; };
  const uint2 own = scratch[lane];
  int rk = lane < total ? 0 : k;
  for (int i = 0; i < total; i += 8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) rk += order(scratch[i + j]) > order(own);
  }
  *rank = rk;
  *sel = static_cast<int>(~own.y);
  *val = key_value(own.x);
  __syncwarp();
}

// Top-k of token t by one warp, by the layer's router rule over every expert
// (see epoch_layer_config), from the logits row in global memory: lane l owns
// the EPL consecutive experts from l * EPL on. Writes the k experts and weights.
template <int EPL>
__device__ __noinline__ void select_token(const FewParams &p, int t, uint2 *scratch, int16_t *sel_out, float *wgt_out) {
  constexpr unsigned kAll = 0xffffffffu;
  const Dims &d = p.d;
  const int lane = lane_id(), E = d.E, k = d.k, lo = lane * EPL;
  const float *row = p.ws.logits + static_cast<size_t>(t) * E;
  float v[EPL], c[EPL];
  bool ok[EPL];
  if (EPL % 4 == 0 && (E & 3) == 0) {
#pragma unroll
    for (int j = 0; j < EPL / 4 * 4; j += 4) {
      const float4 q = lo + j < E ? __ldcg(reinterpret_cast<const float4 *>(row + lo + j))
                                  : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      v[j] = q.x, v[j + 1] = q.y, v[j + 2] = q.z, v[j + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) v[j] = lo + j < E ? __ldcg(row + lo + j) : -INFINITY;
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    ok[j] = lo + j < E;
    c[j] = v[j];
  }
  if (d.router != 0) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) c[j] = ok[j] ? __ldg(p.w.b_router + lo + j) : 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) c[j] += 1.f / (1.f + expf(-v[j]));
    if (d.topk_group < d.n_group) limit_groups<EPL>(c, ok, d);
  }
  int rank, sel;
  float val;
  rank_topk<EPL>(c, ok, k, &rank, &sel, &val, scratch);
  const bool mine = rank < k;
  float num = 0.f, den = 0.f;
  if (d.router == 0) {
    // the largest selected logit is the row's largest: every expert is eligible
    const float top = __shfl_sync(kAll, val, __ffs(__ballot_sync(kAll, rank == 0)) - 1);
    if (mine) num = expf(val - top);
    if (d.raw_weights) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) den += lo + j < E ? expf(v[j] - top) : 0.f;
    }
  } else {
    if (mine) num = 1.f / (1.f + expf(-__ldcg(row + sel)));
  }
  if (!d.raw_weights) den = num;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(kAll, den, o);
  if (d.raw_weights && d.router != 0) den = 1.f;
  if (mine) {
    sel_out[rank] = static_cast<int16_t>(sel);
    wgt_out[rank] = num / den;
  }
}

// Edges sorted by expert, then token, and the jobs, from the selections (all
// threads; r.mask is zero). Every CTA has to come to the same jobs: an edge's place
// follows from its expert's token mask, which no order of atomics changes.
__device__ void build_routes(const FewParams &p, Routes &r) {
  const int E = p.d.E, k = p.d.k, edges = p.n_tok * k, lane = lane_id(), warp = warp_id();
  if (p.n_tok == 1) {  // one edge an expert: nothing to sort
    if (threadIdx.x < k) {
      r.list[threadIdx.x] = r.job_first[threadIdx.x] = static_cast<int16_t>(threadIdx.x);
      r.tok[threadIdx.x] = 0;
      r.job_expert[threadIdx.x] = r.sel[threadIdx.x];
      r.job_n[threadIdx.x] = 1;
    }
    if (threadIdx.x == 0) r.n_jobs = k;
    __syncthreads();
    return;
  }
  for (int i = threadIdx.x; i < edges; i += kThreads) {
    const int t = i / k;
    atomicOr(&r.mask[r.sel[i]][t >> 5], 1u << (t & 31));
  }
  __syncthreads();
  // thread i holds experts 2 i and 2 i + 1; running sums of (jobs << 16 | edges)
  static_assert(2 * kThreads >= 1024, "two experts a thread");
  const int e0 = 2 * threadIdx.x;
  auto count = [&](int e) { return e < E ? __popc(r.mask[e][0]) + __popc(r.mask[e][1]) : 0; };
  const int c0 = count(e0), c1 = count(e0 + 1);
  const int own = (((c0 + 7) >> 3) + ((c1 + 7) >> 3)) << 16 | (c0 + c1);
  int sum = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += y;
  }
  if (lane == 31) r.warp_sum[warp] = sum;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const int y = r.warp_sum[i];
    before += i < warp ? y : 0;
    all += y;
  }
  sum += before - own;
  int job = sum >> 16, at = sum & 0xFFFF;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int c = j ? c1 : c0;
    if (c > 0) r.first[e0 + j] = static_cast<int16_t>(at);
    for (int q = 0; q < c; q += 8) {
      r.job_expert[job] = static_cast<int16_t>(e0 + j);
      r.job_first[job] = static_cast<int16_t>(at + q);
      r.job_n[job++] = static_cast<int16_t>(min(8, c - q));
    }
    at += c;
  }
  if (threadIdx.x == 0) r.n_jobs = all >> 16;
  __syncthreads();
  for (int i = threadIdx.x; i < edges; i += kThreads) {
    const int t = i / k, e = r.sel[i];
    const int q = r.first[e] + (t >= 32 ? __popc(r.mask[e][0]) : 0) + __popc(r.mask[e][t >> 5] & ((1u << (t & 31)) - 1u));
    r.list[q] = static_cast<int16_t>(i);
    r.tok[q] = static_cast<int16_t>(t);
  }
  __syncthreads();
}

template <typename T> __global__ void __launch_bounds__(kThreads, 1) k_moe_few(const __grid_constant__ FewParams p) {
  __shared__ __align__(16) float part[2 * kWarps * 128];  // partial sums of the units; the selection's scratch between the phases
  __shared__ Routes r;
  const Dims &d = p.d;
  const int warp = warp_id(), lane = lane_id(), g = lane >> 2, t = lane & 3;
  const int H = d.H, I = d.I, E = d.E, k = d.k, nt = p.n_tok, nt8 = (nt + 7) / 8;
  constexpr int per = Elem<T>::per, chunk = Elem<T>::step * Elem<T>::steps, steps = Elem<T>::steps;
  const T *x = static_cast<const T *>(p.x);
  // Scratch rows are whole 32-byte sectors, so that no store touches part of one (which L2 would complete from
  // memory first: a barrier after such stores costs 3 to 5 us more).
  constexpr int parts = sizeof(T) == 2 ? 2 : 1;  // of an activation
  const int Ia = few_row(I) * parts, Is = few_row(d.I_s) * parts, Ho = few_row(H);
  T *act = static_cast<T *>(p.ws.act);     // row of edge e at e * Ia,
  const int act_sh = p.n_tok * k * Ia;     // of shared expert s and token t at act_sh + (s * n_tok + t) * Is

  auto wait = [&](int b) {
    return grid_wait(p.ws.ctr + b, static_cast<int32_t>(gridDim.x) + (p.hold == b), p.err, d.timeout_ns);
  };
  auto split = [&](Share &o, int cols, int w, int warps) {
    const int chunks = (cols + chunk - 1) / chunk;
    o.k = cols;
    o.step = chunks * w / warps * steps;
    o.end = chunks * (w + 1) / warps * steps;
  };
  auto sum = [&](const float *mine, int warps, int tok, int row) {
    float s = 0.f;
    const float *q = mine + row * 8 + tok;
    for (int i = 0; i < warps; ++i) s += q[i * 128];
    return s;
  };
  auto at_row = [&](const void *base, int64_t row, int64_t cols) {
    return reinterpret_cast<const char *>(static_cast<const T *>(base) + row * cols + t * per);
  };

  // phase 0: router tiles of 16 experts, then shared tiles of 8 activation columns; eight tokens a unit
  const int n_router = (E + 15) / 16, sh8 = d.n_sh ? (d.I_s + 7) / 8 : 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) p.ws.ctr[3] = 0;  // no CTA reaches the last barrier before this one passes the first
  // the places that activations go to, in L2: stores to lines that are not there cost a block of 32 tokens 1.4 us
  const int64_t act_bytes = (static_cast<int64_t>(act_sh) + static_cast<int64_t>(d.n_sh) * nt * Is) * sizeof(T);
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * 128; i < act_bytes; i += static_cast<int64_t>(gridDim.x) * kThreads * 128)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char *>(act) + i));
  if (threadIdx.x < 16 && blockIdx.x / nt8 * 16 + threadIdx.x < E)  // the bias of this CTA's experts, needed at the end of the tile
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.w.b_router + blockIdx.x / nt8 * 16 + threadIdx.x));
  run_units<T, false>(
      blockIdx.x, gridDim.x, (n_router + d.n_sh * sh8) * nt8, warp, kWarps, 0, part, x,
      [&](int u, int wi, int ws, Share &o) {
        const int v = u / nt8, tok0 = (u - v * nt8) * 8;
        split(o, H, wi, ws);
        o.count = min(8, nt - tok0);
        o.row = min(tok0 + g, nt - 1) * H;
        if (v < n_router) {
          o.p0 = at_row(p.w.w_router, min(v * 16 + g, E - 1), H);
          o.p1 = at_row(p.w.w_router, min(v * 16 + g + 8, E - 1), H);
        } else {
          const int s = (v - n_router) / sh8, c = min((v - n_router - s * sh8) * 8 + g, d.I_s - 1);
          o.p0 = at_row(p.w.ws_gate, static_cast<int64_t>(s) * d.I_s + c, H);
          o.p1 = at_row(p.w.ws_up, static_cast<int64_t>(s) * d.I_s + c, H);
        }
      },
      [&](int u, int count, const float *mine) {
        const int v = u / nt8, tok0 = (u - v * nt8) * 8, q = threadIdx.x;
        if (v < n_router) {
          const int tok = q >> 4, e = v * 16 + (q & 15);
          if (tok < count && e < E)
            p.ws.logits[static_cast<size_t>(tok0 + tok) * E + e] =
                (d.router == 0 ? __ldg(p.w.b_router + e) : 0.f) + sum(mine, kWarps, tok, q & 15);
        } else {
          const int s = (v - n_router) / sh8, tok = q / (8 * parts), col = (v - n_router - s * sh8) * 8 + (q & 7);
          if (tok < count && col < Is / parts)
            put_act(act + act_sh + (s * nt + tok0 + tok) * Is, col, q >> 3 & (parts - 1),
                    silu(sum(mine, kWarps, tok, q & 7)) * sum(mine, kWarps, tok, (q & 7) + 8));
        }
      },
      [] { return true; });
  grid_arrive(p.ws.ctr);
  for (int e = threadIdx.x; e < E; e += kThreads) r.mask[e][0] = r.mask[e][1] = 0u;
  uint2 *scratch = reinterpret_cast<uint2 *>(part) + warp * 32;
  auto select = [&](int tok, int16_t *sel, float *wgt) {
    if (E <= 64) select_token<2>(p, tok, scratch, sel, wgt);
    else if (E <= 256) select_token<8>(p, tok, scratch, sel, wgt);
    else select_token<32>(p, tok, scratch, sel, wgt);
  };
  // One warp runs the selection on whatever the logits hold by now, so that its code is in the instruction cache
  // when the barrier opens (its results are written again below).
  if (warp == 1 && nt <= kWarps) select(0, r.sel, r.wgt);
  if (!wait(0)) return;

  if (nt <= kWarps) {
    if (warp < nt) select(warp, r.sel + warp * k, r.wgt + warp * k);
    __syncthreads();
  } else {
    // shared out over the CTAs
    const int tok = blockIdx.x + warp * gridDim.x;
    if (tok < nt) select(tok, p.ws.sel + tok * k, p.ws.wgt + tok * k);
    grid_arrive(p.ws.ctr + 1);
    if (!wait(1)) return;
    for (int i = threadIdx.x; i < nt * k; i += kThreads) {
      // in range even where a call that gave up left its barriers half counted
      r.sel[i] = static_cast<int16_t>(min(max(static_cast<int>(__ldcg(p.ws.sel + i)), 0), E - 1));
      r.wgt[i] = __ldcg(p.ws.wgt + i);
    }
    __syncthreads();
  }
  build_routes(p, r);

  // phase 1: routed activations, 8 columns of a job's expert a unit
  const int i8 = (I + 7) / 8;
  int warps = split_of(H * static_cast<int>(sizeof(T))), grp = warp / warps, w = warp % warps;
  int gthread = threadIdx.x - grp * warps * 32;
  run_units<T, false>(
      grp * gridDim.x + blockIdx.x, gridDim.x * (kWarps / warps), r.n_jobs * i8, w, warps, grp,
      part + grp * 2 * warps * 128, x,
      [&](int u, int wi, int ws, Share &o) {
        const int j = u / i8, c = min((u - j * i8) * 8 + g, I - 1);
        split(o, H, wi, ws);
        o.count = r.job_n[j];
        o.row = r.tok[r.job_first[j] + min(g, o.count - 1)] * H;
        o.p0 = at_row(p.w.w_gate, static_cast<int64_t>(r.job_expert[j]) * I + c, H);
        o.p1 = at_row(p.w.w_up, static_cast<int64_t>(r.job_expert[j]) * I + c, H);
      },
      [&](int u, int count, const float *mine) {
        const int j = u / i8;
        for (int v = gthread; v < count * 8 * parts; v += warps * 32) {
          const int tok = v / (8 * parts), c = v & 7, col = (u - j * i8) * 8 + c;
          if (col < Ia / parts)  // the last sector whole: columns behind I hold copies that nobody reads
            put_act(act + r.list[r.job_first[j] + tok] * Ia, col, v >> 3 & (parts - 1),
                    silu(sum(mine, warps, tok, c)) * sum(mine, warps, tok, c + 8));
        }
      },
      [] { return true; });
  grid_arrive(p.ws.ctr + 2);

  // phase 2: 16 rows of H of a job's expert (after the routed jobs, eight tokens
  // of a shared expert each) a unit; rows of the fp32 sums: edge e at row e,
  // shared expert s and token t at n_tok * k + s * n_tok + t
  const int h16 = (H + 15) / 16;
  warps = split_of(I * static_cast<int>(sizeof(T)));
  grp = warp / warps;
  w = warp % warps;
  gthread = threadIdx.x - grp * warps * 32;
  const bool in_time = run_units<T, true>(
      grp * gridDim.x + blockIdx.x, gridDim.x * (kWarps / warps), (r.n_jobs + d.n_sh * nt8) * h16, w, warps, grp,
      part + grp * 2 * warps * 128, act,
      [&](int u, int wi, int ws, Share &o) {
        const int j = u / h16, row = (u - j * h16) * 16 + g;
        if (j < r.n_jobs) {
          split(o, I, wi, ws);
          o.count = r.job_n[j];
          o.row = r.list[r.job_first[j] + min(g, o.count - 1)] * Ia;
          o.p0 = at_row(p.w.w_down, static_cast<int64_t>(r.job_expert[j]) * H + min(row, H - 1), I);
          o.p1 = at_row(p.w.w_down, static_cast<int64_t>(r.job_expert[j]) * H + min(row + 8, H - 1), I);
        } else {
          const int s = (j - r.n_jobs) / nt8, tok0 = (j - r.n_jobs - s * nt8) * 8;
          split(o, d.I_s, wi, ws);
          o.count = min(8, nt - tok0);
          o.row = act_sh + (s * nt + min(tok0 + g, nt - 1)) * Is;
          o.p0 = at_row(p.w.ws_down, static_cast<int64_t>(s) * H + min(row, H - 1), d.I_s);
          o.p1 = at_row(p.w.ws_down, static_cast<int64_t>(s) * H + min(row + 8, H - 1), d.I_s);
        }
      },
      [&](int u, int count, const float *mine) {
        const int j = u / h16, sj = j - r.n_jobs;
        for (int v = gthread; v < count * 16; v += warps * 32) {
          const int tok = v >> 4, c = v & 15, col = (u - j * h16) * 16 + c;
          const int at = sj < 0 ? r.list[r.job_first[j] + tok] : nt * k + sj / nt8 * nt + sj % nt8 * 8 + tok;
          if (col < Ho) __stcg(p.ws.out + static_cast<size_t>(at) * Ho + col, sum(mine, warps, tok, c));
        }
      },
      [&] { return wait(2); });
  if (!in_time) return;
  grid_arrive(p.ws.ctr + 3);
  if (!wait(3)) return;
  if (blockIdx.x == 0 && threadIdx.x < 3) p.ws.ctr[threadIdx.x] = 0;  // every CTA has left these barriers

  // y, four columns a thread, edges in selection order
  const int h4 = H / 4;
  for (int v = blockIdx.x * kThreads + threadIdx.x; v < nt * h4; v += gridDim.x * kThreads) {
    const int tok = v / h4, col = (v - tok * h4) * 4;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    auto add = [&](int first, int n, const float *wgt) {  // rows first, first + n_rows.. of the expert outputs
#pragma unroll 8
      for (int j = 0; j < n; ++j) {
        const float4 q = __ldcg(reinterpret_cast<const float4 *>(p.ws.out + static_cast<size_t>(first + j * (wgt ? 1 : nt)) * Ho + col));
        const float f = wgt ? wgt[j] : 1.f;
        s[0] = fmaf(f, q.x, s[0]);
        s[1] = fmaf(f, q.y, s[1]);
        s[2] = fmaf(f, q.z, s[2]);
        s[3] = fmaf(f, q.w, s[3]);
      }
    };
    add(tok * k, k, r.wgt + tok * k);
    add(nt * k + tok, d.n_sh, nullptr);
    const size_t at = static_cast<size_t>(tok) * H + col;
    T o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = from_f32<T>(d.residual ? s[j] + to_f32(x[at + j]) : s[j]);
    if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2 *>(static_cast<T *>(p.y) + at) = *reinterpret_cast<const uint2 *>(o);
    else *reinterpret_cast<uint4 *>(static_cast<T *>(p.y) + at) = *reinterpret_cast<const uint4 *>(o);
  }
}

template <typename T> cudaError_t launch(const FewParams &p, cudaStream_t s) {
  auto *fn = &k_moe_few<T>;
  static std::atomic<uint64_t> ready{0};  // devices whose copy of the kernel has its carveout set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load() & bit)) {
    // tokens' rows are read through L1, which gets what the tables and partial sums leave
    e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxL1);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit);
  }
  // Cooperative: the grid's CTAs are resident together or the launch fails, which the grid barriers need.
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(num_sms()));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

}  // namespace

cudaError_t launch_moe_few(const Dims &d, const Weights &w, const FewWork &ws, const void *x, void *y, int n_tok,
                           int bf16, int hold, uint32_t *err, cudaStream_t s) {
  FewParams p;
  p.d = d;
  p.w = w;
  p.ws = ws;
  p.x = x;
  p.y = y;
  p.err = err;
  p.n_tok = n_tok;
  p.hold = hold;
  return bf16 ? launch<__nv_bfloat16>(p, s) : launch<float>(p, s);
}

}  // namespace epoch
