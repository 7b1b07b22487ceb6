// The whole MoE layer for a few tokens in one launch: router, top-k, routed and
// shared SwiGLU experts, weighted sum (epoch_moe_few).
//
//   G = x W_r^T (+ b);  S_t, w_t = the layer's router rule over every expert
//   y_t = sum_{e in S_t} w_te W_down,e (silu(W_gate,e x_t) * (W_up,e x_t)) + sum_shared (+ x_t)
//
// With at most 64 tokens the bytes of the selected experts' weights bound the
// time, so the kernel is built around reading each of them once, from global
// memory straight into registers, with loads always in flight. One CTA per SM
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
// fp32 layers run the same schedule with FFMA in place of the tensor core.
#include <atomic>
#include <climits>
#include <cstring>

#include "common.cuh"
#include "layer.h"
#include "topk.cuh"

namespace epoch {

namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kSteps = 4;    // K steps (64 bytes of a row) loaded together
constexpr int kMaxEdges = kFewTokens * 16;

// ------------------------------------------------------------------ element types
template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
  static constexpr int step = 32, per = 8;  // columns of a K step, and of a thread in it
  static constexpr int acc = 4;             // fp32 sums a thread keeps of a 16 x 8 tile while adding along K
};
template <> struct Elem<float> {
  static constexpr int step = 16, per = 4;
  static constexpr int acc = 16;  // rows g and g + 8 of all eight tokens (this thread's columns only)
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
// launch's first arrival); the wait ends when all have, or gives up (false).
// Loads issued between the halves do not hold the arrival back.
__device__ __forceinline__ void grid_arrive(int32_t *ctr) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(ctr, 1);
  }
}
__device__ bool grid_wait(const int32_t *ctr, uint32_t *err, int64_t timeout_ns) {
  __shared__ int s_ok;
  if (threadIdx.x == 0) {
    const int32_t want = static_cast<int32_t>(gridDim.x);
    auto seen = [&] {
      int32_t v;
      asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(ctr) : "memory");
      return v;
    };
    int ok = 1;
    if (seen() < want) {
      const uint64_t t0 = globaltimer_ns();
      for (uint32_t i = 1; seen() < want; ++i)
        if ((i & 63u) == 0u && globaltimer_ns() - t0 > static_cast<uint64_t>(timeout_ns)) {
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

// Sixteen weight rows of one unit, as this thread sees them: its columns of rows
// g and g + 8 (rows behind the last one read it again: their sums go nowhere),
// and its warp's K steps, a whole number of chunks.
struct WeightRows {
  const char *p0, *p1;
  int step, end, k;  // K steps of this warp, columns of a row
};

// Whether columns of a K step that a thread holds exist: rows of bf16 layers are
// a whole number of chunks.
template <typename T> __device__ __forceinline__ bool in_row(int c, int k) { return sizeof(T) == 2 || c < k; }

template <typename T>
__device__ __forceinline__ void load_chunk(const WeightRows &w, int step, uint4 (&a)[kSteps], uint4 (&b)[kSteps]) {
  const int c0 = step * Elem<T>::step, ct = c0 + (lane_id() & 3) * Elem<T>::per;
  const char *p0 = w.p0 + static_cast<int64_t>(c0) * sizeof(T), *p1 = w.p1 + static_cast<int64_t>(c0) * sizeof(T);
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    const bool in = in_row<T>(ct + j * Elem<T>::step, w.k);
    a[j] = load_weights(p0 + 64 * j, in);
    b[j] = load_weights(p1 + 64 * j, in);
  }
}

// Adds the products of a loaded chunk with tokens' rows to the sums: rows[i] is
// where the row of this thread's token of tile i starts in x (tiles behind the
// last token repeat one: every token is a column of its own), of `count` tokens.
template <typename T, int NT, bool FRESH>
__device__ __forceinline__ void add_chunk(int step, int k, const uint4 (&a)[kSteps], const uint4 (&b)[kSteps],
                                          const T *x, const int (&rows)[NT], int count,
                                          float (&acc)[NT][Elem<T>::acc]) {
  const int c0 = step * Elem<T>::step + (lane_id() & 3) * Elem<T>::per;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if (8 * i >= count) break;
      const T *row = x + rows[i] + c0;
      uint4 v[kSteps];
#pragma unroll
      for (int j = 0; j < kSteps; ++j) v[j] = load_tokens<FRESH>(row + j * Elem<T>::step);
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        mma_bf16(acc[i], a[j].x, b[j].x, a[j].y, b[j].y, v[j].x, v[j].y);
        mma_bf16(acc[i], a[j].z, b[j].z, a[j].w, b[j].w, v[j].z, v[j].w);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int n = 0; n < 8; n += 2) {  // two tokens' loads on their way together
        if (8 * i + n >= count) break;
        uint4 v[2][kSteps];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const T *row = x + __shfl_sync(0xffffffffu, rows[i], 4 * (n + m)) + c0;  // token n + m of the tile
#pragma unroll
          for (int j = 0; j < kSteps; ++j) {
            v[m][j] = make_uint4(0u, 0u, 0u, 0u);
            if (in_row<T>(c0 + j * Elem<T>::step, k)) v[m][j] = load_tokens<FRESH>(row + j * Elem<T>::step);
          }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          float s = acc[i][n + m], q = acc[i][8 + n + m];
#pragma unroll
          for (int j = 0; j < kSteps; ++j) {
            const float v0 = __uint_as_float(v[m][j].x), v1 = __uint_as_float(v[m][j].y),
                        v2 = __uint_as_float(v[m][j].z), v3 = __uint_as_float(v[m][j].w);
            s = fmaf(__uint_as_float(a[j].x), v0, s);
            s = fmaf(__uint_as_float(a[j].y), v1, s);
            s = fmaf(__uint_as_float(a[j].z), v2, s);
            s = fmaf(__uint_as_float(a[j].w), v3, s);
            q = fmaf(__uint_as_float(b[j].x), v0, q);
            q = fmaf(__uint_as_float(b[j].y), v1, q);
            q = fmaf(__uint_as_float(b[j].z), v2, q);
            q = fmaf(__uint_as_float(b[j].w), v3, q);
          }
          acc[i][n + m] = s;
          acc[i][8 + n + m] = q;
        }
      }
    }
  }
}

// A warp's sums of tile i to shared memory as [16 rows][8 tokens].
template <typename T> __device__ __forceinline__ void put_tile(float *d, const float (&acc)[Elem<T>::acc]) {
  const int lane = lane_id(), g = lane >> 2, t = lane & 3;
  if constexpr (sizeof(T) == 2) {
    d[g * 8 + 2 * t] = acc[0];
    d[g * 8 + 2 * t + 1] = acc[1];
    d[(g + 8) * 8 + 2 * t] = acc[2];
    d[(g + 8) * 8 + 2 * t + 1] = acc[3];
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
// `warps` warps (this warp is number `w` of group `gid`). A unit with more
// tokens than NT tiles hold streams its weights once for each 8 NT tokens (the
// later times from L2). Partial sums meet in `part` ([2][warps][NT][128],
// alternating halves, so one group barrier each), from which `finish` takes
// them. Two chunks of weights are always on their way: a chunk's registers are
// loaded again, with the unit's next columns or the next unit's first, as soon
// as its products are issued. `ready` runs once, after the first loads are
// issued: the wait for the grid barrier before the phase, if any.
template <typename T, int NT, bool FRESH, typename Weights, typename Tokens, typename Finish, typename Ready>
__device__ __forceinline__ bool run_units(int first, int stride, int n, int w, int warps, int gid, float *part,
                                          const T *x, Weights weights, Tokens tokens, Finish finish, Ready ready) {
  uint4 a0[kSteps], b0[kSteps], a1[kSteps], b1[kSteps];
  WeightRows cur;
  int u = first, tok0 = 0;
  if (u < n) {
    weights(u, w, warps, cur);
    if (cur.step < cur.end) load_chunk<T>(cur, cur.step, a0, b0);
    if (cur.step + kSteps < cur.end) load_chunk<T>(cur, cur.step + kSteps, a1, b1);
  }
  if (!ready()) return false;
  int half = 0;
  while (u < n) {
    int rows[NT];
    const int left = tokens(u, tok0, rows);  // this thread's token rows, and how many tokens there are from tok0 on
    const int count = min(left, 8 * NT);
    float acc[NT][Elem<T>::acc];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < Elem<T>::acc; ++j) acc[i][j] = 0.f;
    const bool last = left <= 8 * NT;
    const int un = last ? u + stride : u;
    const int end = cur.end;
    int step = cur.step;
    do {
      int ns = step + 2 * kSteps;  // what the registers hold next
      const int s1 = step + kSteps, k0 = cur.k;
      if (step < end) add_chunk<T, NT, FRESH>(step, k0, a0, b0, x, rows, count, acc);
      step = ns;
      if (ns >= end) {
        cur.end = 0;  // nothing left to load
        if (un < n) weights(un, w, warps, cur);
        ns = cur.step;
      }
      if (ns < cur.end) load_chunk<T>(cur, ns, a0, b0);
      if (s1 < end) add_chunk<T, NT, FRESH>(s1, k0, a1, b1, x, rows, count, acc);
      if (ns + kSteps < cur.end) load_chunk<T>(cur, ns + kSteps, a1, b1);
    } while (step < end);
    float *mine = part + (static_cast<size_t>(half) * warps) * (NT * 128);
#pragma unroll
    for (int i = 0; i < NT; ++i)
      if (8 * i < count) put_tile<T>(mine + (w * NT + i) * 128, acc[i]);
    group_sync(gid, warps);
    finish(u, tok0, count, last, mine);
    half ^= 1;
    u = un;
    tok0 = last ? 0 : tok0 + 8 * NT;
  }
  return true;
}

// Warps of a group in phases 1 and 2, for rows of `chunks` chunks: at most four,
// and no more than leave each of them the two chunks it keeps in flight.
__device__ __forceinline__ int split_of(int chunks) { return chunks >= 8 ? 4 : chunks >= 4 ? 2 : 1; }

struct FewParams {
  Dims d;
  Weights w;
  FewWork ws;
  const void *x;
  void *y;
  uint32_t *err;
  int n_tok;
};

// Routing tables of a CTA, in shared memory.
struct Routes {
  int16_t sel[kMaxEdges];   // expert of edge t * k + j
  float wgt[kMaxEdges];     // its weight
  int16_t list[kMaxEdges];  // edges by expert,
  int16_t tok[kMaxEdges];   // and their tokens
  int16_t rank[kMaxEdges];
  int32_t first[1025];      // first entry of each hit expert in list
  int16_t hit[1024];        // hit experts
  int32_t cnt[1024];
  int32_t warp_sum[kWarps];
  int32_t n_hit;
  int16_t turn[1024];       // order of phase 1: hit experts
  int16_t deal[1024 + 8];   // order of phase 2 within a row tile: hit expert, or n_hit + shared expert
};

// Group rule of the sigmoid router (see warp_group_limit) over the scores c of
// every expert, lane l holding the EPL consecutive ones from l * EPL on: clears ok
// outside the chosen groups. Where a group is the experts of 1, 2, 4, .. lanes
// these merge their two best; otherwise the general form of warp_group_limit runs.
template <int EPL>
__device__ __forceinline__ void limit_groups(const float (&c)[EPL], bool (&ok)[EPL], const Dims &d) {
  constexpr unsigned kAll = 0xffffffffu;
  const int gs = d.E / d.n_group, lanes = gs / EPL, lane = lane_id();
  if (gs % EPL != 0 || (lanes & (lanes - 1)) != 0) {
    warp_group_limit<EPL>(c, ok, d.E, d.n_group, d.topk_group, d.k);
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
// a chain of latencies (2100 clocks as k rounds of a warp maximum).
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
  if ((E & 3) == 0) {
#pragma unroll
    for (int j = 0; j < EPL; j += 4) {
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

// Edges sorted by expert, from the selections (all threads; r.cnt is zero). The
// order of an expert's edges does not matter: each is a column of its own everywhere.
__device__ void build_routes(const FewParams &p, Routes &r) {
  const int E = p.d.E, k = p.d.k, edges = p.n_tok * k, lane = lane_id(), warp = warp_id();
  if (p.n_tok == 1) {  // one edge an expert: nothing to sort
    if (threadIdx.x <= k) r.first[threadIdx.x] = threadIdx.x;
    if (threadIdx.x < k) {
      r.hit[threadIdx.x] = r.sel[threadIdx.x];
      r.list[threadIdx.x] = static_cast<int16_t>(threadIdx.x);
      r.tok[threadIdx.x] = 0;
    }
    if (threadIdx.x == 0) r.n_hit = k;
    __syncthreads();
    return;
  }
  for (int i = threadIdx.x; i < edges; i += kThreads) r.rank[i] = static_cast<int16_t>(atomicAdd(&r.cnt[r.sel[i]], 1));
  __syncthreads();
  // thread i holds experts 2 i and 2 i + 1; running sums of (hit experts << 16 | edges)
  static_assert(2 * kThreads >= 1024, "two experts a thread");
  const int e0 = 2 * threadIdx.x;
  const int c0 = e0 < E ? r.cnt[e0] : 0, c1 = e0 + 1 < E ? r.cnt[e0 + 1] : 0;
  const int own = ((c0 > 0) + (c1 > 0)) << 16 | (c0 + c1);
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
  int hit = sum >> 16, at = sum & 0xFFFF;
  if (c0 > 0) {
    r.first[hit] = at;
    r.hit[hit++] = static_cast<int16_t>(e0);
    r.cnt[e0] = at;  // now the expert's first entry
    at += c0;
  }
  if (c1 > 0) {
    r.first[hit] = at;
    r.hit[hit] = static_cast<int16_t>(e0 + 1);
    r.cnt[e0 + 1] = at;
  }
  if (threadIdx.x == 0) {
    r.n_hit = all >> 16;
    r.first[all >> 16] = edges;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < edges; i += kThreads) {
    const int q = r.cnt[r.sel[i]] + r.rank[i];
    r.list[q] = static_cast<int16_t>(i);
    r.tok[q] = static_cast<int16_t>(i / k);
  }
  __syncthreads();
}

// Orders in which the phases take the experts, dearest first where they differ:
// an expert costs its weights and, per 8 tokens, the tokens' rows and products.
// Phase 1 deals its units out in turns, so a group gets one of each price.
// Phase 2 gives a group a run of neighbours in `deal`: the experts, by price,
// dealt into `columns` columns that stand one after another, so that any run
// of a column's length holds one of each price too. All threads.
__device__ void order_by_cost(const FewParams &p, Routes &r, int columns) {
  const int n_hit = r.n_hit, all = n_hit + p.d.n_sh;
  auto tiles = [&](int h) { return ((h < n_hit ? r.first[h + 1] - r.first[h] : p.n_tok) + 7) >> 3; };
  const int q = all / columns, rem = all % columns;
  int place[3], rank[3];  // up to 1024 + 8 entries
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int h = threadIdx.x + i * kThreads;
    rank[i] = h;
    if (h < all && p.n_tok > 8) {
      const int mine = tiles(h);
      rank[i] = 0;
      for (int o = 0; o < all; ++o) {
        const int other = tiles(o);
        rank[i] += other > mine || (other == mine && o < h);
      }
    }
    const int c = rank[i] % columns;
    place[i] = c * q + min(c, rem) + rank[i] / columns;
    if (h < all) r.deal[place[i]] = static_cast<int16_t>(h);
  }
  if (p.n_tok <= 8) {
    for (int h = threadIdx.x; h < n_hit; h += kThreads) r.turn[h] = static_cast<int16_t>(h);
  } else {
    // ranks among the hit experts alone: without the shared ones before them
    for (int h = threadIdx.x; h < n_hit; h += kThreads) {
      const int at = rank[h / kThreads] - (((p.n_tok + 7) >> 3) > tiles(h) ? p.d.n_sh : 0);
      r.turn[at] = static_cast<int16_t>(h);
    }
  }
  __syncthreads();
}

template <typename T, int NT> __global__ void __launch_bounds__(kThreads, 1) k_moe_few(const __grid_constant__ FewParams p) {
  extern __shared__ float part[];  // partial sums of the units; the selection's scratch between the phases
  __shared__ Routes r;
  const Dims &d = p.d;
  const int warp = warp_id(), lane = lane_id(), g = lane >> 2, t = lane & 3;
  const int H = d.H, I = d.I, E = d.E, k = d.k, nt = p.n_tok;
  constexpr int per = Elem<T>::per, step = Elem<T>::step;
  const T *x = static_cast<const T *>(p.x);
  T *act = static_cast<T *>(p.ws.act);     // row of edge e at e * I,
  const int act_sh = p.n_tok * k * I;      // of shared expert s and token t at act_sh + (s * n_tok + t) * I_s

  auto split = [&](WeightRows &o, int cols, int w, int warps) {
    const int chunks = (cols + step * kSteps - 1) / (step * kSteps);
    o.k = cols;
    o.step = chunks * w / warps * kSteps;
    o.end = chunks * (w + 1) / warps * kSteps;
  };
  auto sum = [&](const float *mine, int warps, int tok, int row) {
    float s = 0.f;
    const float *q = mine + (tok >> 3) * 128 + row * 8 + (tok & 7);
    for (int i = 0; i < warps; ++i) s += q[i * NT * 128];
    return s;
  };

  // phase 0: router tiles of 16 experts, then shared tiles of 8 activation columns
  const int n_router = (E + 15) / 16, sh8 = d.n_sh ? (d.I_s + 7) / 8 : 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) p.ws.ctr[3] = 0;  // no CTA reaches the last barrier before this one passes the first
  if (threadIdx.x < 16 && blockIdx.x * 16 + threadIdx.x < E)  // the bias of this CTA's experts, needed at the end of the tile
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.w.b_router + blockIdx.x * 16 + threadIdx.x));
  run_units<T, NT, false>(
      blockIdx.x, gridDim.x, n_router + d.n_sh * sh8, warp, kWarps, 0, part, x,
      [&](int u, int wi, int warps, WeightRows &o) {
        split(o, H, wi, warps);
        if (u < n_router) {
          const T *base = static_cast<const T *>(p.w.w_router) + t * per;
          o.p0 = reinterpret_cast<const char *>(base + static_cast<int64_t>(min(u * 16 + g, E - 1)) * H);
          o.p1 = reinterpret_cast<const char *>(base + static_cast<int64_t>(min(u * 16 + g + 8, E - 1)) * H);
        } else {
          const int s = (u - n_router) / sh8, c = min((u - n_router - s * sh8) * 8 + g, d.I_s - 1);
          const int64_t at = (static_cast<int64_t>(s) * d.I_s + c) * H + t * per;
          o.p0 = reinterpret_cast<const char *>(static_cast<const T *>(p.w.ws_gate) + at);
          o.p1 = reinterpret_cast<const char *>(static_cast<const T *>(p.w.ws_up) + at);
        }
      },
      [&](int, int tok0, int (&rows)[NT]) {
#pragma unroll
        for (int i = 0; i < NT; ++i) rows[i] = min(tok0 + 8 * i + g, nt - 1) * H;
        return nt - tok0;
      },
      [&](int u, int tok0, int count, bool, const float *mine) {
        if (u < n_router) {
          for (int v = threadIdx.x; v < count * 16; v += kThreads) {
            const int tok = v >> 4, e = u * 16 + (v & 15);
            if (e < E)
              p.ws.logits[static_cast<size_t>(tok0 + tok) * E + e] =
                  (d.router == 0 ? __ldg(p.w.b_router + e) : 0.f) + sum(mine, kWarps, tok, v & 15);
          }
          return;
        }
        const int s = (u - n_router) / sh8, col0 = (u - n_router - s * sh8) * 8;
        for (int v = threadIdx.x; v < count * 8; v += kThreads) {
          const int tok = v >> 3, c = v & 7;
          if (col0 + c < d.I_s)
            act[act_sh + (s * nt + tok0 + tok) * d.I_s + col0 + c] =
                from_f32<T>(silu(sum(mine, kWarps, tok, c)) * sum(mine, kWarps, tok, c + 8));
        }
      },
      [] { return true; });
  grid_arrive(p.ws.ctr);
  for (int e = threadIdx.x; e < E; e += kThreads) r.cnt[e] = 0;
  if (!grid_wait(p.ws.ctr, p.err, d.timeout_ns)) return;

  uint2 *scratch = reinterpret_cast<uint2 *>(part) + warp * 32;
  auto select = [&](int tok, int16_t *sel, float *wgt) {
    if (E <= 256) select_token<8>(p, tok, scratch, sel, wgt);
    else select_token<32>(p, tok, scratch, sel, wgt);
  };
  if (nt <= kWarps) {
    if (warp < nt) select(warp, r.sel + warp * k, r.wgt + warp * k);
    __syncthreads();
  } else {
    // shared out over the CTAs
    const int tok = blockIdx.x + warp * gridDim.x;
    if (tok < nt) select(tok, p.ws.sel + tok * k, p.ws.wgt + tok * k);
    grid_arrive(p.ws.ctr + 1);
    if (!grid_wait(p.ws.ctr + 1, p.err, d.timeout_ns)) return;
    for (int i = threadIdx.x; i < nt * k; i += kThreads) {
      r.sel[i] = __ldcg(p.ws.sel + i);
      r.wgt[i] = __ldcg(p.ws.wgt + i);
    }
    __syncthreads();
  }
  build_routes(p, r);

  const int h16 = (H + 15) / 16;
  const int warps2 = split_of(I / (step * kSteps)), n_groups = gridDim.x * (kWarps / warps2);
  order_by_cost(p, r, max(1, (n_groups + h16 - 1) / h16));

  // phase 1: routed activations, 8 columns of an expert a unit
  const int i8 = (I + 7) / 8;
  int warps = split_of(H / (step * kSteps)), grp = warp / warps, w = warp % warps;
  int gthread = threadIdx.x - grp * warps * 32;
  run_units<T, NT, false>(
      grp * gridDim.x + blockIdx.x, gridDim.x * (kWarps / warps), r.n_hit * i8, w, warps, grp,
      part + static_cast<size_t>(grp) * 2 * warps * NT * 128, x,
      [&](int u, int wi, int ws, WeightRows &o) {
        const int at_h = u / i8, h = r.turn[at_h], c = min((u - at_h * i8) * 8 + g, I - 1);
        const int64_t at = (static_cast<int64_t>(r.hit[h]) * I + c) * H + t * per;
        split(o, H, wi, ws);
        o.p0 = reinterpret_cast<const char *>(static_cast<const T *>(p.w.w_gate) + at);
        o.p1 = reinterpret_cast<const char *>(static_cast<const T *>(p.w.w_up) + at);
      },
      [&](int u, int tok0, int (&rows)[NT]) {
        const int h = r.turn[u / i8], f = r.first[h] + tok0, n = r.first[h + 1] - f;
#pragma unroll
        for (int i = 0; i < NT; ++i) rows[i] = r.tok[f + min(8 * i + g, n - 1)] * H;
        return n;
      },
      [&](int u, int tok0, int count, bool, const float *mine) {
        const int at_h = u / i8, f = r.first[r.turn[at_h]] + tok0;
        for (int v = gthread; v < count * 8; v += warps * 32) {
          const int tok = v >> 3, c = v & 7, col = (u - at_h * i8) * 8 + c;
          if (col < I)
            act[r.list[f + tok] * I + col] = from_f32<T>(silu(sum(mine, warps, tok, c)) * sum(mine, warps, tok, c + 8));
        }
      },
      [] { return true; });
  grid_arrive(p.ws.ctr + 2);

  // phase 2: 16 rows of H of an expert (routed, then shared) a unit; rows of
  // the fp32 sums: edge e at row e, shared expert s and token t at n_tok * k + s * n_tok + t.
  const int experts = r.n_hit + d.n_sh;
  warps = warps2;
  grp = warp / warps;
  w = warp % warps;
  gthread = threadIdx.x - grp * warps * 32;
  const int64_t group = grp * gridDim.x + blockIdx.x;
  const int lo = static_cast<int>(experts * h16 * group / n_groups);
  const int hi = static_cast<int>(experts * h16 * (group + 1) / n_groups);
  run_units<T, NT, true>(
      lo, 1, hi, w, warps, grp, part + static_cast<size_t>(grp) * 2 * warps * NT * 128, act,
      [&](int u, int wi, int ws, WeightRows &o) {
        const int tile = u / experts, h = r.deal[u - tile * experts], row = tile * 16 + g;
        const bool shared = h >= r.n_hit;
        const int cols = shared ? d.I_s : I;
        const T *base = static_cast<const T *>(shared ? p.w.ws_down : p.w.w_down) +
                        static_cast<int64_t>(shared ? h - r.n_hit : r.hit[h]) * H * cols + t * per;
        split(o, cols, wi, ws);
        o.p0 = reinterpret_cast<const char *>(base + static_cast<int64_t>(min(row, H - 1)) * cols);
        o.p1 = reinterpret_cast<const char *>(base + static_cast<int64_t>(min(row + 8, H - 1)) * cols);
      },
      [&](int u, int tok0, int (&rows)[NT]) {
        const int h = r.deal[u % experts];
        if (h >= r.n_hit) {
#pragma unroll
          for (int i = 0; i < NT; ++i)
            rows[i] = act_sh + ((h - r.n_hit) * nt + min(tok0 + 8 * i + g, nt - 1)) * d.I_s;
          return nt - tok0;
        }
        const int f = r.first[h] + tok0, n = r.first[h + 1] - f;
#pragma unroll
        for (int i = 0; i < NT; ++i) rows[i] = r.list[f + min(8 * i + g, n - 1)] * I;
        return n;
      },
      [&](int u, int tok0, int count, bool last, const float *mine) {
        const int tile = u / experts, h = r.deal[u - tile * experts];
        const bool shared = h >= r.n_hit;
        for (int v = gthread; v < count * 16; v += warps * 32) {
          const int tok = tok0 + (v >> 4), c = v & 15, col = tile * 16 + c;
          const int at = shared ? nt * k + (h - r.n_hit) * nt + tok : r.list[r.first[h] + tok];
          if (col < H) __stcg(p.ws.out + static_cast<size_t>(at) * H + col, sum(mine, warps, v >> 4, c));
        }
      },
      [&] { return grid_wait(p.ws.ctr + 2, p.err, d.timeout_ns); });
  grid_arrive(p.ws.ctr + 3);
  if (!grid_wait(p.ws.ctr + 3, p.err, d.timeout_ns)) return;
  if (blockIdx.x == 0 && threadIdx.x < 3) p.ws.ctr[threadIdx.x] = 0;  // every CTA has left these barriers

  // y, four columns a thread, edges in selection order
  const int h4 = H / 4;
  for (int v = blockIdx.x * kThreads + threadIdx.x; v < nt * h4; v += gridDim.x * kThreads) {
    const int tok = v / h4, col = (v - tok * h4) * 4;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    auto add = [&](int first, int n, const float *wgt) {  // rows first, first + n_rows.. of the expert outputs
#pragma unroll 8
      for (int j = 0; j < n; ++j) {
        const float4 q = __ldcg(reinterpret_cast<const float4 *>(p.ws.out + static_cast<size_t>(first + j * (wgt ? 1 : nt)) * H + col));
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

template <typename T, int NT> cudaError_t launch(const FewParams &p, cudaStream_t s) {
  auto *fn = &k_moe_few<T, NT>;
  static std::atomic<uint64_t> ready{0};  // devices whose copy of the kernel has its shared memory raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  constexpr int smem = 2 * kWarps * NT * 128 * sizeof(float);
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load() & bit)) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    // tokens' rows are read through L1, which gets what the partial sums leave
    if (e == cudaSuccess)
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
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

// Token tiles a thread's registers hold: up to 32 tokens of bf16 layers (16
// fp32 sums), 16 of fp32 layers (32 sums).
cudaError_t by_tokens(const FewParams &p, bool bf16, cudaStream_t s) {
  if (bf16) {
    if (p.n_tok <= 8) return launch<__nv_bfloat16, 1>(p, s);
    if (p.n_tok <= 16) return launch<__nv_bfloat16, 2>(p, s);
    return launch<__nv_bfloat16, 4>(p, s);
  }
  return p.n_tok <= 8 ? launch<float, 1>(p, s) : launch<float, 2>(p, s);
}

}  // namespace

cudaError_t launch_moe_few(const Dims &d, const Weights &w, const FewWork &ws, const void *x, void *y, int n_tok,
                           int bf16, uint32_t *err, cudaStream_t s) {
  FewParams p;
  p.d = d;
  p.w = w;
  p.ws = ws;
  p.x = x;
  p.y = y;
  p.err = err;
  p.n_tok = n_tok;
  return by_tokens(p, bf16 != 0, s);
}

}  // namespace epoch
