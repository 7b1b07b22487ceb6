// A router by itself: from logits to each position's experts and weights and to the worklist that the
// products grouped by expert take (expert-major, positions ascending), without running any expert.
//
// One warp a position: the lanes hold consecutive experts' logits, and the k best are found by rounds
// of a warp maximum. Positions of a CTA are marked in a word of bits for each expert, so that an
// edge's place among the CTA's is a population count, whatever order the warps come in. A second
// kernel adds what earlier CTAs and lower experts hold: every CTA reads all CTAs' counts (40 KB at
// 16384 positions and 256 experts) rather than wait for one that adds them up. Up to 32 positions
// one CTA does both. What bounds it: latency up to some thousand positions, then the instructions of
// the ranking (650 a position of 256 experts by softmax, 1050 by sigmoid under the group rule), not the logits' bytes:
// 16384 positions take 20.5 and 31.6 us, their bytes 2.8; one position takes 5.5. A lane holds 2, 4, 8, 16 or 32
// experts, the fewest that reach all of them: what it does for each is most of the work (8192 positions of 512 experts,
// sigmoid in two groups: 27 us with 16 a lane, 84 with 32; of 128 experts 18 with four, 29 with eight).
//
// The sigmoid router's order is that of sigmoid(G) + bias in 64 bits, equal ones by lower id. It is decided in fp32
// where neighbours are further apart than fp32's roundings can move them; for the positions where they
// are not (2 in 1000 with 256 experts, fp32 logits or a bias for each expert) the entries near the border are ranked once
// more in 64 bits. bf16 logits without a bias tie far more often, two positions in five: 16384 positions of 256 experts in
// groups take 40 us, with fp32 logits or a bias 30.
#include <climits>

#include "common.cuh"
#include "layer.h"
#include "topk.cuh"

namespace epoch {

namespace {

constexpr int kPass = 128;  // most positions of a CTA's pass

// Logit e of a row.
__device__ __forceinline__ float logit(const void *row, bool bf16, int e) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(row)[e]) : __ldg(static_cast<const float *>(row) + e);
}
// A lane's EPL consecutive logits as they lie in memory, so that a row's loads can be on their way while the row before
// is ranked: fp32 bits, or with whole vectors of bf16 pairs in the first half. vec: rows start on 16-byte boundaries.
template <int EPL> struct Raw {
  uint32_t w[EPL];
};
template <int EPL> __device__ __forceinline__ bool whole(bool vec, int E) { return EPL % 4 == 0 && vec && lane_id() * EPL + EPL <= E; }
template <int EPL> __device__ __forceinline__ void load_raw(const void *row, bool bf16, int E, bool vec, Raw<EPL> &r) {
  const int e0 = lane_id() * EPL;
  if constexpr (EPL % 4 == 0) {
    if (whole<EPL>(vec, E)) {
      if (bf16 && EPL == 4) {
        const uint2 u = __ldg(reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(row) + e0));
        r.w[0] = u.x, r.w[1] = u.y;
      } else if (bf16) {
#pragma unroll
        for (int q = 0; q < EPL / 8; ++q) {
          const uint4 u = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(row) + e0) + q);
          r.w[4 * q] = u.x, r.w[4 * q + 1] = u.y, r.w[4 * q + 2] = u.z, r.w[4 * q + 3] = u.w;
        }
      } else {
#pragma unroll
        for (int q = 0; q < EPL / 4; ++q) {
          const uint4 u = __ldg(reinterpret_cast<const uint4 *>(static_cast<const float *>(row) + e0) + q);
          r.w[4 * q] = u.x, r.w[4 * q + 1] = u.y, r.w[4 * q + 2] = u.z, r.w[4 * q + 3] = u.w;
        }
      }
      return;
    }
  }
#pragma unroll
  for (int c = 0; c < EPL; ++c) r.w[c] = e0 + c < E ? __float_as_uint(logit(row, bf16, e0 + c)) : 0xFF800000u;  // -inf behind the last
}
template <int EPL> __device__ __forceinline__ void open_raw(const Raw<EPL> &r, bool bf16, int E, bool vec, float (&v)[EPL]) {
  if (bf16 && whole<EPL>(vec, E)) {
#pragma unroll
    for (int c = 0; c < EPL; ++c) v[c] = __uint_as_float(c & 1 ? r.w[c / 2] & 0xFFFF0000u : r.w[c / 2] << 16);
  } else {
#pragma unroll
    for (int c = 0; c < EPL; ++c) v[c] = __uint_as_float(r.w[c]);
  }
}

// Unsigned key with the order of a number: -0 as +0, above the keys of -inf and of negative NaNs (at most kLowest) and
// below those of positive NaNs (above kHighest).
constexpr unsigned kLowest = 0x007FFFFFu, kHighest = 0xFF800000u;  // of -inf and of inf
__device__ __forceinline__ unsigned number_key(float v) {
  const int b = __float_as_int(v + 0.0f);
  return static_cast<unsigned>(b ^ ((b >> 31) | static_cast<int>(0x80000000u)));
}

// The k best of the warp's entries, lane l owning the EPL consecutive ids from l * EPL on: key 0 is no entry, equal
// keys go by lower id. Entry j < k ends up in scratch[j] (.x the key, .y the id; 0 and -1 where there is none).
// `scratch`: 32 entries of the warp's own.
//
// The k-th of the best keys of half lanes (of their different values: a bound that may be lower, not higher) bounds the
// k best entries from below: only entries at or above it, some ten, are ranked against one another, one a lane. (By whole
// lanes' bests half of the experts in half of the lanes, as the group rule leaves them, let twice as many through.)
template <int EPL>
__device__ __forceinline__ void best_of(const unsigned (&key)[EPL], int k, uint2 *scratch) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = lane_id();
  unsigned lo = 0u, hi = 0u, bound = 1u;  // bests of the lane's two halves
#pragma unroll
  for (int c = 0; c < EPL / 2; ++c) {
    lo = max(lo, key[c]);
    hi = max(hi, key[EPL / 2 + c]);
  }
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const unsigned m = __reduce_max_sync(kAll, max(lo, hi));
    bound = max(m, 1u);  // 0: fewer than k different bests, all entries count
    if (lo == m) lo = 0u;
    if (hi == m) hi = 0u;
  }
  unsigned pass = 0u;
#pragma unroll
  for (int c = 0; c < EPL; ++c) pass |= key[c] >= bound ? 1u << c : 0u;
  const int n = __popc(pass);
  int sum = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kAll, sum, o);
    if (lane >= o) sum += y;
  }
  const int total = __shfl_sync(kAll, sum, 31);
  if (__any_sync(kAll, total > 32)) {  // many equal keys, or k lanes with several of the best
    int id = -1;
    float v;
    warp_topk_rounds<EPL>(key, k, &id, &v);
    scratch[lane] = make_uint2(id >= 0 ? order_key(v) : 0u, static_cast<unsigned>(id));
    __syncwarp();
    return;
  }
  uint2 *to = scratch + (sum - n);
#pragma unroll
  for (int c = 0; c < EPL; ++c)
    if ((pass >> c) & 1u) *to++ = make_uint2(key[c], static_cast<unsigned>(lane * EPL + c));
  __syncwarp();
  const uint2 mine = scratch[lane < total ? lane : 0];  // ascending ids
  int rank = 0;
#pragma unroll 4
  for (int i = 0; i < total; ++i) {
    const unsigned o = scratch[i].x;
    rank += o > mine.x || (o == mine.x && i < lane);
  }
  __syncwarp();
  if (lane < total) scratch[rank] = mine;
  else scratch[lane] = make_uint2(0u, 0xffffffffu);
  __syncwarp();
}

// Selection score of an expert in 64 bits, and its place in an order of integers (0: none; a NaN ranks with -inf).
__device__ __forceinline__ double score_exact(const RouteArgs &a, float g, int e) {
  return 1.0 / (1.0 + exp(-static_cast<double>(g))) + (a.bias != nullptr ? static_cast<double>(__ldg(a.bias + e)) : 0.0);
}
__device__ __forceinline__ unsigned long long order_exact(double v) {
  if (v != v) v = -INFINITY;
  const long long b = __double_as_longlong(v + 0.0);
  return static_cast<unsigned long long>(b < 0 ? ~b : b | static_cast<long long>(1ull << 63));
}
__device__ __forceinline__ double value_exact(unsigned long long key) {  // 0 for none
  const long long b = static_cast<long long>(key);
  return key ? __longlong_as_double(b < 0 ? b & 0x7FFFFFFFFFFFFFFFll : ~b) : 0.0;
}
// Largest of the warp's keys (0: none) and the lowest lane that holds it.
__device__ __forceinline__ unsigned long long warp_best(unsigned long long v, int *lane) {
  const unsigned hi = __reduce_max_sync(0xffffffffu, static_cast<unsigned>(v >> 32));
  const unsigned lo = __reduce_max_sync(0xffffffffu, static_cast<unsigned>(v >> 32) == hi ? static_cast<unsigned>(v) : 0u);
  const unsigned long long best = (static_cast<unsigned long long>(hi) << 32) | lo;
  *lane = __ffs(__ballot_sync(0xffffffffu, v == best)) - 1;
  return best;
}

// Candidates of one position, at most one a lane in ascending id, ranked in 64 bits: lane j < k gets the id of rank j.
__device__ __noinline__ int rank_exact(const RouteArgs &a, const void *row, int e, int k) {
  unsigned long long left = e >= 0 ? order_exact(score_exact(a, logit(row, a.bf16 != 0, e), e)) : 0ull;
  int sel = -1;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    int win;
    const unsigned long long best = warp_best(left, &win);
    const int id = __shfl_sync(0xffffffffu, e, win);
    if (best == 0ull) break;
    if (lane_id() == j) sel = id;
    if (lane_id() == win) left = 0ull;
  }
  return sel;
}

// The whole selection of one position in 64 bits, where groups' scores are too near or too many experts are: lane j < k
// gets expert j, or -1. `can` has a bit for each of the lane's EPL experts. Rare, and slow.
template <int EPL> __device__ __noinline__ int select_exact(const RouteArgs &a, const void *row, unsigned can) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = lane_id(), gs = a.n_experts / a.n_group;
  unsigned long long key[EPL];
#pragma unroll 1
  for (int q = 0; q < EPL; ++q) {
    const int e = lane * EPL + q;
    key[q] = (can >> q) & 1u ? order_exact(score_exact(a, logit(row, a.bf16 != 0, e), e)) : 0ull;
  }
  if (a.topk_group < a.n_group) {
    double score = 0.0;  // lane i: group i's
    int held = 0;
#pragma unroll 1
    for (int i = 0; i < a.n_group; ++i) {
      unsigned long long k1 = 0ull, k2 = 0ull;
      int n = 0;
#pragma unroll 1
      for (int q = 0; q < EPL; ++q) {
        const unsigned long long v = (lane * EPL + q) / gs == i ? key[q] : 0ull;
        n += v != 0ull;
        if (v > k1) k2 = k1, k1 = v;
        else if (v > k2) k2 = v;
      }
      n = static_cast<int>(__reduce_add_sync(kAll, static_cast<unsigned>(n)));
      int win, unused;
      const unsigned long long m1 = warp_best(k1, &win), m2 = warp_best(lane == win ? k2 : k1, &unused);
      if (lane == i) score = value_exact(m1) + value_exact(m2), held = n;
    }
    int rank = 0, before = 0;
#pragma unroll 1
    for (int i = 0; i < a.n_group; ++i) {
      const double s = __shfl_sync(kAll, score, i);
      const int h = __shfl_sync(kAll, held, i);
      if (h > 0 && (s > score || (s == score && i < lane))) ++rank, before += h;
    }
    const unsigned chosen = __ballot_sync(kAll, lane < a.n_group && held > 0 && (rank < a.topk_group || before < a.top_k));
#pragma unroll 1
    for (int q = 0; q < EPL; ++q)
      if (!((chosen >> (((lane * EPL + q) / gs) & 31)) & 1u)) key[q] = 0ull;
  }
  int sel = -1;
#pragma unroll 1
  for (int j = 0; j < a.top_k; ++j) {
    unsigned long long v = 0ull;
    int at = 0;
#pragma unroll 1
    for (int q = 0; q < EPL; ++q)
      if (key[q] > v) v = key[q], at = q;
    int win;
    const unsigned long long best = warp_best(v, &win);
    const int id = __shfl_sync(kAll, lane * EPL + at, win);
    if (best == 0ull) break;
    if (lane == j) sel = id;
    if (lane == win) key[at] = 0ull;
  }
  return sel;
}

// sigmoid in fp32 for the selection, off by less than 4e-7: the exponential's 2 + 1.2 |g| steps of 2^-23 reach the
// result by s (1 - s) of them (less than one step), the sum's and the reciprocal's 2 steps and a half by s.
__device__ __forceinline__ float sigmoid_near(float g) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
  return s;
}
// Whether two selection scores are apart whatever fp32 made of them: sigmoid as above, the sum with the bias half a
// step of the result.
__device__ __forceinline__ bool apart(float a, float b) { return fabsf(a - b) > 1.2e-6f + 2.5e-7f * fmaxf(fabsf(a), fabsf(b)); }
// How far fp32 may have put a group's score from that of its two best, a + b: two sigmoids, 8e-7, and half a step of each
// term, of their sum and of the ends of score -+ group_reach, each at most 2^-24 (|a| + |b|). The terms' sizes count and
// not the sum's, which is small where the biases cancel.
__device__ __forceinline__ float group_reach(float a, float b) { return 1.2e-6f + 2.5e-7f * (fabsf(a) + fabsf(b)); }

// Weights where every selected sigmoid lies below exp(kLowLogit), which their sum then shows, over this thread's edges (of
// rows from row0 on): quotients of the sigmoids over the largest (see sigmoid_over). Logits up to kNoScore have a score of 0 in
// 64 bits too (exp(-g) overflows): their order is that of the ids, and the weights of a position that selects no other are
// 0 / 0. Out of the loop over the edges, which a call in it would slow down (16384 positions, softmax: 20.1 us, 20.8 with it).
constexpr float kLowSum = 4e-8f, kNoScore = -709.7827f;
__device__ __noinline__ void low_weights(const RouteArgs &a, const uint8_t *rows, int64_t row_bytes, const int16_t *ids, const float2 *stat,
                                         float *weights, int edges) {
  const int k = a.top_k;
  for (int i = threadIdx.x; i < edges; i += blockDim.x) {
    const int r = i / k;
    const int16_t *id = ids + r * k;
    const uint8_t *row = rows + r * row_bytes;
    if (ids[i] < 0) continue;
    float most = -INFINITY, sum = stat[r].y;
    for (int j = 0; j < k; ++j)
      if (id[j] >= 0) most = fmaxf(most, logit(row, a.bf16 != 0, id[j]));
    for (int j = 0; j < k; ++j)
      if (id[j] >= 0) sum += sigmoid_over(logit(row, a.bf16 != 0, id[j]), most);
    if (most < kLowLogit) weights[i] = most <= kNoScore ? __uint_as_float(0x7FC00000u) : sigmoid_over(logit(row, a.bf16 != 0, ids[i]), most) / sum;
  }
}

// Ids of the entries that lanes have marked (bits of their EPL), in ascending order one a lane from scratch on; how many
// there are, of which at most 32 fit.
template <int EPL> __device__ __forceinline__ int gather_marked(unsigned marked, uint2 *scratch) {
  const int lane = lane_id(), n = __popc(marked);
  int sum = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += y;
  }
  const int total = __shfl_sync(0xffffffffu, sum, 31);
  __syncwarp();
  if (__all_sync(0xffffffffu, total <= 32)) {
    int to = sum - n;
#pragma unroll
    for (int q = 0; q < EPL; ++q)
      if ((marked >> q) & 1u) scratch[to++].y = static_cast<unsigned>(lane * EPL + q);
  }
  __syncwarp();
  return total;
}

// The topk_group best groups (a bit each) by the entries that could be one of their two best, at most one a lane, in 64
// bits. Every expert is an entry.
__device__ __noinline__ unsigned groups_exact(const RouteArgs &a, const void *row, int e, int gs) {
  const int lane = lane_id(), mine = e >= 0 ? e / gs : -1;
  const unsigned long long key = e >= 0 ? order_exact(score_exact(a, logit(row, a.bf16 != 0, e), e)) : 0ull;
  unsigned long long score = 0ull;  // lane i: group i's, as a key
#pragma unroll 1
  for (int i = 0; i < a.n_group; ++i) {
    const unsigned long long v = mine == i ? key : 0ull;
    int win, unused;
    const unsigned long long m1 = warp_best(v, &win), m2 = warp_best(lane == win ? 0ull : v, &unused);
    if (lane == i) score = order_exact(value_exact(m1) + value_exact(m2));
  }
  unsigned chosen = 0u;
#pragma unroll 1
  for (int i = 0; i < a.topk_group; ++i) {
    int win;
    warp_best(score, &win);  // the lowest of equal ones
    chosen |= 1u << win;
    if (lane == win) score = 0ull;
  }
  return chosen;
}

// limit_groups for a position whose every expert is an entry: a group is 2^i lanes (`span`), whose two best are merged.
template <int EPL>
__device__ __forceinline__ bool limit_groups_fast(unsigned (&key)[EPL], const RouteArgs &a, int span, const void *row, uint2 *scratch) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = lane_id(), shift = 31 - __clz(span);
  unsigned k1 = key[0], k2 = 0u;
#pragma unroll
  for (int q = 1; q < EPL; ++q) {
    k2 = max(k2, min(k1, key[q]));
    k1 = max(k1, key[q]);
  }
  for (int o = 1; o < span; o <<= 1) {
    const unsigned o1 = __shfl_xor_sync(kAll, k1, o), o2 = __shfl_xor_sync(kAll, k2, o);
    k2 = max(max(k2, o2), min(k1, o1));
    k1 = max(k1, o1);
  }
  const float first = key_value(k1), second = key_value(k2), score = first + second, off = group_reach(first, second);
  const unsigned mine = number_key(score);
  // rounds of the best group left; equal ones go together (and are then too near, or all chosen)
  unsigned left = mine, bound = 0u;
#pragma unroll 4
  for (int i = 0; i < a.topk_group; ++i) {
    bound = __reduce_max_sync(kAll, left);
    if (left == bound) left = 0u;
  }
  bool in = mine >= bound;
  // the least that a chosen group's score can be and the most of another's (an infinite one leaves no certainty: NaN is least)
  const unsigned low = __reduce_min_sync(kAll, in ? order_key(score - off) : 0xffffffffu);
  const unsigned high = __reduce_max_sync(kAll, in ? 0u : order_key(score + off));
  if (!__all_sync(kAll, __popc(__ballot_sync(kAll, in)) == a.topk_group << shift && low > high)) {
    unsigned near = 0u;
#pragma unroll
    for (int q = 0; q < EPL; ++q) {
      const float v = key_value(key[q]);
      if (!(v < second && apart(v, second))) near |= 1u << q;
    }
    const int total = gather_marked<EPL>(near, scratch);
    if (__any_sync(kAll, total > 32)) return false;
    const unsigned chosen = groups_exact(a, row, lane < total ? static_cast<int>(scratch[lane].y) : -1, EPL << shift);
    __syncwarp();
    in = (chosen >> (lane >> shift)) & 1u;
  }
  if (!in)
#pragma unroll
    for (int q = 0; q < EPL; ++q) key[q] = 0u;
  return true;
}

// The groups that a position may search (clears keys outside them); false where fp32 cannot tell.
template <int EPL> __device__ __noinline__ bool limit_groups(unsigned *key, const RouteArgs &a) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = lane_id(), gs = a.n_experts / a.n_group;
  float score = -INFINITY, off = 0.f;  // lane i: group i's, and how far it may be off
  int held = 0;
  for (int i = 0; i < a.n_group; ++i) {
    unsigned k1 = 0u, k2 = 0u;
    int n = 0;
    const int lo = i * gs - lane * EPL, hi = lo + gs;  // the group's entries of this lane
#pragma unroll
    for (int q = 0; q < EPL; ++q) {
      const unsigned v = q >= lo && q < hi ? key[q] : 0u;
      n += v != 0u;
      k2 = max(k2, min(k1, v));
      k1 = max(k1, v);
    }
    const unsigned m1 = __reduce_max_sync(kAll, k1);
    const unsigned hold = __ballot_sync(kAll, k1 == m1);
    const unsigned m2 = __reduce_max_sync(kAll, lane == __ffs(hold) - 1 ? k2 : k1);
    n = static_cast<int>(__reduce_add_sync(kAll, static_cast<unsigned>(n)));
    if (lane == i) {
      const float first = key_value(m1), second = m2 == 0u ? 0.f : key_value(m2);
      held = n;
      score = m1 == 0u ? -INFINITY : first + second;
      off = group_reach(first, second);
    }
  }
  const bool there = lane < a.n_group && held > 0;
  int rank = 0, before = 0;
#pragma unroll 4
  for (int i = 0; i < a.n_group; ++i) {
    const float s = __shfl_sync(kAll, score, i);
    const int h = __shfl_sync(kAll, held, i);
    if (h > 0 && (s > score || (s == score && i < lane))) ++rank, before += h;
  }
  const unsigned chosen = __ballot_sync(kAll, there && (rank < a.topk_group || before < a.top_k));
  const unsigned others = __ballot_sync(kAll, there) & ~chosen;
  // A chosen and an unchosen group must be apart: the least chosen and the best other. Where more than topk_group are
  // taken, because those hold fewer than k, so many groups are chosen whatever their order only if all hold as many;
  // else their order counts too.
  const unsigned low = __reduce_min_sync(kAll, (chosen >> lane) & 1u ? order_key(score - off) : 0xffffffffu);
  const unsigned high = __reduce_max_sync(kAll, (others >> lane) & 1u ? order_key(score + off) : 0u);
  const bool alike = __reduce_max_sync(kAll, there ? held : 0) == __reduce_min_sync(kAll, there ? held : INT_MAX);
  bool sure = low > high;  // (without others high is 0)
  if (__any_sync(kAll, __popc(chosen) > a.topk_group && !alike)) {
    bool close = false;  // to the score of any other group
    for (int i = 0; i < a.n_group; ++i) {
      const float s = __shfl_sync(kAll, score, i), o = __shfl_sync(kAll, off, i);
      const int h = __shfl_sync(kAll, held, i);
      close = close || (h > 0 && i != lane && !(fabsf(s - score) > o + off));
    }
    sure = !__any_sync(kAll, ((chosen >> lane) & 1u) && close);
  }
#pragma unroll
  for (int q = 0; q < EPL; ++q)
    if (!((chosen >> (((lane * EPL + q) / gs) & 31)) & 1u)) key[q] = 0u;
  return sure;
}

// One position by one warp: selection j goes to id[j] (-1: none) and, with the softmax router, its logit to val[j]; stat
// gets what its weights need besides: the softmax's largest logit and, where they are raw, its sum over all experts;
// else 0, or NaN where a logit is (which spoils the weights). `eligible` has a bit for each of the lane's experts,
// bias their biases (up to sixteen).
template <int EPL>
__device__ __forceinline__ void route_row(const RouteArgs &a, const void *row, float (&v)[EPL], unsigned eligible,
                                          const float (&bias)[EPL], uint2 *scratch, int16_t *id, float *val, float2 *stat) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = lane_id(), k = a.top_k;
  unsigned key[EPL], can = eligible;
  unsigned low = 0xffffffffu, high = 0u;
#pragma unroll
  for (int c = 0; c < EPL; ++c) {
    key[c] = number_key(v[c]);
    low = min(low, key[c]);
    high = max(high, key[c]);
  }
  // -inf (behind the last expert too), NaN and masks are rare in a lane of whole experts
  float spoilt = 0.f;
  const bool clean = __all_sync(kAll, low > kLowest && high <= kHighest && eligible == (EPL == 32 ? 0xffffffffu : (1u << (EPL & 31)) - 1u));
  if (!clean) {
    bool nan = false;
#pragma unroll
    for (int c = 0; c < EPL; ++c) {
      if (key[c] < kLowest || key[c] > kHighest) {  // a NaN ranks with -inf, but can be selected
        nan = true;
        key[c] = kLowest;
      } else if (key[c] == kLowest) {
        can &= ~(1u << c);
      }
      if (!((can >> c) & 1u)) key[c] = 0u;
    }
    if (__any_sync(kAll, nan)) spoilt = __uint_as_float(0x7FC00000u);
  }
  if (!a.sigmoid) {
    best_of<EPL>(key, k, scratch);
    if (lane < k) {
      const uint2 e = scratch[lane];
      id[lane] = static_cast<int16_t>(e.y);
      val[lane] = key_value(e.x);
    }
    float top = key_value(scratch[0].x), sum = spoilt;
    if (a.raw_weights) {  // probabilities over all experts, eligible or not
      float m = v[0];
#pragma unroll
      for (int c = 1; c < EPL; ++c) m = fmaxf(m, v[c]);
      top = key_value(__reduce_max_sync(kAll, order_key(m)));
#pragma unroll
      for (int c = 0; c < EPL; ++c) sum += lane * EPL + c < a.n_experts ? expf(v[c] - top) : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    }
    if (lane == 0) *stat = make_float2(top, sum);
    __syncwarp();
    return;
  }
  unsigned most = 0u;
#pragma unroll
  for (int q = 0; q < EPL; ++q) {
    const int e = lane * EPL + q;
    v[q] = sigmoid_near(v[q]) + (EPL <= 16 ? bias[q] : a.bias != nullptr && e < a.n_experts ? __ldg(a.bias + e) : 0.f);
    const unsigned place = number_key(v[q]);
    key[q] = key[q] == 0u ? 0u : place;
    most = max(most, place - kLowest - 1u);
  }
  // NaN and -inf of a logit or a bias rank lowest
  const bool numbers = __all_sync(kAll, most < kHighest - kLowest);
  if (!numbers)
#pragma unroll
    for (int q = 0; q < EPL; ++q) key[q] = key[q] == 0u ? 0u : key[q] < kLowest || key[q] > kHighest ? kLowest : key[q];
  int sel = -1;
  bool sure = true;
  if (a.topk_group < a.n_group) {
    const int gs = a.n_experts / a.n_group, span = gs / EPL;
    if (clean && numbers && gs % EPL == 0 && (span & (span - 1)) == 0 && a.topk_group * gs >= k) sure = limit_groups_fast<EPL>(key, a, span, row, scratch);
    else sure = limit_groups<EPL>(key, a);
  }
  if (__all_sync(kAll, sure)) {
    // one more than asked for, so that the last border is seen too
    best_of<EPL>(key, k + 1, scratch);
    const uint2 mine = scratch[min(lane, k)], after = scratch[min(lane + 1, k)];
    sel = static_cast<int>(mine.y);
    if (__any_sync(kAll, lane < k && after.x != 0u && !apart(key_value(mine.x), key_value(after.x)))) {
      // Every entry that could be among the k: those not surely below the k-th, in 64 bits.
      const uint2 kth = scratch[k - 1];
      const float edge = key_value(kth.x);
      unsigned near = 0u;
#pragma unroll
      for (int q = 0; q < EPL; ++q)
        if (key[q] != 0u && (kth.x == 0u || !(v[q] < edge && apart(v[q], edge)))) near |= 1u << q;
      const int total = gather_marked<EPL>(near, scratch);
      sure = total <= 32;
      if (__all_sync(kAll, sure)) sel = rank_exact(a, row, lane < total ? static_cast<int>(scratch[lane].y) : -1, k);
    }
  }
  if (!__all_sync(kAll, sure)) sel = select_exact<EPL>(a, row, can);
  if (lane < k) id[lane] = static_cast<int16_t>(sel);
  if (lane == 0) *stat = make_float2(0.f, spoilt);
  __syncwarp();
}

// First entries of the experts (offsets, E + 1 values in shared memory) from their totals; all threads of the CTA.
__device__ __forceinline__ void scan_totals(const int *total, int E, int *offsets, int *s_warp) {
  const int tid = threadIdx.x, lane = lane_id(), warp = warp_id(), warps = blockDim.x >> 5;
  int carry = 0;
  for (int base = 0; base < E; base += blockDim.x) {
    const int e = base + tid, n = e < E ? total[e] : 0;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    int all = lane < warps ? s_warp[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, all, o);
      if (lane >= o) all += y;
    }
    const int below = __shfl_sync(0xffffffffu, all, warp > 0 ? warp - 1 : 0);
    if (e < E) offsets[e] = carry + (warp > 0 ? below : 0) + sum - n;
    carry += __shfl_sync(0xffffffffu, all, 31);
    __syncthreads();
  }
  if (tid == 0) offsets[E] = carry;
  __syncthreads();
}

// Counts of CTAs of one pass lie by expert, a byte each, in rows of whole vectors.
__host__ __device__ constexpr int byte_row(int ctas) { return (ctas + 15) & ~15; }
// The first n bytes of a word.
__device__ __forceinline__ uint32_t low_bytes(int n) { return n >= 4 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << (8 * n)) - 1u; }

// Selection, weights and, in slots, each edge's place among its CTA's edges of the expert; the CTA's counts. The only
// CTA of a grid (with one pass) finishes the worklist too. Selecting takes a warp a position; what follows takes a
// thread an edge.
template <int EPL, int THREADS>
__global__ void __launch_bounds__(THREADS) k_router_select(const RouteArgs a, int passes, int pass) {
  constexpr int kE = EPL * 32;
  constexpr bool kAhead = EPL <= 16;  // the next position's logits are on their way (wider lanes have no registers for it)
  __shared__ uint32_t s_bits[kPass / 32][kE];
  __shared__ int s_count[kE], s_off[kE + 1], s_warp[32];
  __shared__ uint2 s_scratch[THREADS / 32][32];
  __shared__ float s_val[kPass * 16];
  __shared__ int16_t s_id[kPass * 16];
  __shared__ float2 s_stat[kPass];
  // (The warp's number by a shuffle: the compiler then knows that the warp takes every branch on it together. Where it
  // does not, each warp maximum becomes a loop.)
  const int tid = threadIdx.x, threads = blockDim.x, lane = lane_id(), warp = __shfl_sync(0xffffffffu, warp_id(), 0), warps = threads >> 5;
  const int E = a.n_experts, k = a.top_k, words = (pass + 31) / 32;
  const unsigned by_k = (65536u + k - 1) / k;  // i / k = i * by_k >> 16 for i < 2048
  const bool vec = a.vec != 0, bf16 = a.bf16 != 0, one = gridDim.x == 1 && passes == 1;
  const int64_t row_bytes = a.logits_stride * (bf16 ? 2 : 4);
  const uint8_t *logits = static_cast<const uint8_t *>(a.logits);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * passes * pass;
  Raw<EPL> raw;
  bool live = true;
  auto fetch = [&](int64_t t, int64_t end) {
    if (t >= end) return;
    live = a.live == nullptr || __ldg(a.live + t) != 0;
    load_raw<EPL>(logits + t * row_bytes, bf16, E, vec, raw);
  };
  if (kAhead) fetch(first + warp, min(first + pass, static_cast<int64_t>(a.n_tok)));
  for (int i = tid; i < E; i += threads) {
    s_count[i] = 0;
    for (int w = 0; w < words; ++w) s_bits[w][i] = 0u;
  }
  unsigned eligible = 0u;
  float bias[EPL];
#pragma unroll
  for (int c = 0; c < EPL; ++c) {
    const int e = lane * EPL + c;
    if (e < E && (a.eligible == nullptr || __ldg(a.eligible + e) != 0)) eligible |= 1u << c;
    bias[c] = kAhead && e < E && a.bias != nullptr ? __ldg(a.bias + e) : 0.f;
  }
  pdl_trigger();
  for (int p = 0; p < passes; ++p) {
    const int64_t t0 = first + static_cast<int64_t>(p) * pass;
    if (t0 >= a.n_tok) break;
    const int rows = static_cast<int>(min(static_cast<int64_t>(pass), a.n_tok - t0)), edges = rows * k;
    for (int r = warp; r < rows; r += warps) {
      if (!kAhead || (p > 0 && r == warp)) fetch(t0 + r, t0 + rows);
      float v[EPL];
      open_raw<EPL>(raw, bf16, E, vec, v);
      const bool on = __any_sync(0xffffffffu, live);
      if (kAhead) fetch(t0 + r + warps, t0 + rows);
      if (on) {
        route_row<EPL>(a, logits + (t0 + r) * row_bytes, v, eligible, bias, s_scratch[warp], s_id + r * k, s_val + r * k, s_stat + r);
      } else if (lane < k) {
        s_id[r * k + lane] = -1;
      }
    }
    __syncthreads();
    // the weights' terms, a thread an edge; the selections as bits
    for (int i = tid; i < edges; i += threads) {
      const int r = static_cast<int>(i * by_k >> 16), e = s_id[i];
      float x = 0.f;
      if (e >= 0) {
        atomicOr(&s_bits[r >> 5][e], 1u << (r & 31));
        x = a.sigmoid ? sigmoid_over(logit(logits + (t0 + r) * row_bytes, bf16, e), 0.f) : expf(s_val[i] - s_stat[r].x);
      }
      s_val[i] = x;
    }
    __syncthreads();
    if (one) {  // totals, and with them the first places
      for (int i = tid; i < E; i += threads) {
        int n = 0;
        for (int w = 0; w < words; ++w) n += __popc(s_bits[w][i]);
        s_count[i] = n;
      }
      __syncthreads();
      scan_totals(s_count, E, s_off, s_warp);
      for (int i = tid; i <= E; i += threads) a.offsets[i] = s_off[i];
      for (int64_t i = s_off[E] + tid; i < static_cast<int64_t>(a.n_tok) * k; i += threads) a.positions[i] = -1;
    }
    const int *base = one ? s_off : s_count;
    bool low = false;
    for (int i = tid; i < edges; i += threads) {
      const int r = static_cast<int>(i * by_k >> 16), e = s_id[i];
      const int64_t at = t0 * k + i;
      int place = -1;
      float w = 0.f;
      if (e >= 0) {
        float sum = s_stat[r].y;
        if (!a.raw_weights)
          for (int j = 0; j < k; ++j) sum += s_val[r * k + j];
        if (a.raw_weights && a.sigmoid) w = s_val[i] + sum;
        else w = s_val[i] / sum, low = low || sum < kLowSum;  // (softmax's are 1 or more)
        place = base[e];
        for (int q = 0; q < (r >> 5); ++q) place += __popc(s_bits[q][e]);
        place += __popc(s_bits[r >> 5][e] & ((1u << (r & 31)) - 1u));
        if (one) a.positions[place] = static_cast<int>(t0 + r);
      }
      a.sel[at] = e;
      a.weights[at] = w;
      a.slots[at] = place;
    }
    if (low) low_weights(a, logits + t0 * row_bytes, row_bytes, s_id, s_stat, a.weights + t0 * k, edges);
    if (one) return;
    __syncthreads();
    for (int i = tid; i < E; i += threads) {
      int n = s_count[i];
      for (int w = 0; w < words; ++w) {
        n += __popc(s_bits[w][i]);
        s_bits[w][i] = 0u;
      }
      s_count[i] = n;
    }
    __syncthreads();
  }
  if (passes == 1) {  // at most 128: a byte
    uint8_t *at = reinterpret_cast<uint8_t *>(a.counts) + blockIdx.x;
    for (int i = tid; i < E; i += threads) at[static_cast<int64_t>(i) * byte_row(gridDim.x)] = static_cast<uint8_t>(s_count[i]);
  } else {
    for (int i = tid; i < E; i += threads) a.counts[static_cast<int64_t>(blockIdx.x) * E + i] = s_count[i];
  }
}

// Places: what lower experts and earlier CTAs hold is added to every edge's place.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) k_router_place(const RouteArgs a, int passes, int pass) {
  __shared__ int s_total[1024], s_before[1024], s_off[1025], s_warp[THREADS / 32];
  const int tid = threadIdx.x, E = a.n_experts, k = a.top_k;
  for (int i = tid; i < E; i += THREADS) s_total[i] = s_before[i] = 0;
  __syncthreads();
  pdl_wait();
  // threads of one expert share the CTAs out
  const int per = max(1, THREADS / E), ctas = gridDim.x, mine = blockIdx.x;
  for (int i = tid; i < E * per; i += THREADS) {
    int e;
    unsigned total = 0u, before = 0u;
    if (passes == 1) {
      const int row = byte_row(ctas);
      e = i / per;
      for (int b = 16 * (i % per); b < ctas; b += 16 * per) {
        const uint4 v = __ldcg(reinterpret_cast<const uint4 *>(reinterpret_cast<const uint8_t *>(a.counts) + static_cast<int64_t>(e) * row + b));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          total = __dp4a(w[q] & low_bytes(ctas - b - 4 * q), 0x01010101u, total);
          before = __dp4a(w[q] & low_bytes(mine - b - 4 * q), 0x01010101u, before);
        }
      }
    } else {
      e = i % E;
      const int part = i / E;
#pragma unroll 8
      for (int b = part; b < ctas; b += per) {
        const unsigned n = __ldcg(a.counts + static_cast<int64_t>(b) * E + e);
        total += n;
        before += b < mine ? n : 0u;
      }
    }
    if (per == 1) {
      s_total[e] = static_cast<int>(total);
      s_before[e] = static_cast<int>(before);
    } else {
      atomicAdd(&s_total[e], static_cast<int>(total));
      atomicAdd(&s_before[e], static_cast<int>(before));
    }
  }
  __syncthreads();
  scan_totals(s_total, E, s_off, s_warp);
  if (mine == 0)
    for (int i = tid; i <= E; i += THREADS) a.offsets[i] = s_off[i];
  for (int i = tid; i < E; i += THREADS) s_before[i] += s_off[i];
  __syncthreads();
  const int64_t all = static_cast<int64_t>(a.n_tok) * k, span = static_cast<int64_t>(passes) * pass * k;
  const int64_t lo = mine * span, hi = min(lo + span, all);
  for (int64_t i = lo + tid; i < hi; i += THREADS) {
    const int sel = __ldcg(a.sel + i);
    if (sel < 0) continue;  // its slot is -1 already
    const int slot = __ldcg(a.slots + i) + s_before[sel];
    a.slots[i] = slot;
    a.positions[slot] = static_cast<int>(i / k);
  }
  for (int64_t i = s_off[E] + static_cast<int64_t>(mine) * THREADS + tid; i < all; i += static_cast<int64_t>(ctas) * THREADS)
    a.positions[i] = -1;
}

struct Split {
  int ctas, passes, pass;
};
// Up to 32 positions a single CTA and launch. Beyond, passes of 8 to 128 positions dealt evenly to all SMs: the rows of a
// CTA take turns at its issue slots, so that few in many CTAs are soonest done (128 positions of 256 experts, softmax: 8.9
// us by passes of 8, 12 by 32, 17 by one CTA; the sigmoid router under the group rule 11.9, 17 and 27). Shorter passes gain
// nothing, as every CTA reads all CTAs' counts. (Up to 32 one CTA takes at most 2 us longer than two launches would, and
// saves the second launch's host time of 4.)
Split split_of(int64_t n, int sms) {
  if (n <= 32) return {1, 1, 32};
  const int64_t most = static_cast<int64_t>(kPass) * sms, passes = (n + most - 1) / most, places = passes * sms;
  const int64_t even = ((n + places - 1) / places + 3) & ~3ll, pass = even < 8 ? 8 : even > kPass ? kPass : even;
  return {static_cast<int>((n + passes * pass - 1) / (passes * pass)), static_cast<int>(passes), static_cast<int>(pass)};
}

template <int EPL> cudaError_t launch_select(const RouteArgs &a, const Split &sp, cudaStream_t s) {
  constexpr int kThreads = EPL <= 8 ? 1024 : 512;
  // a few positions: as many warps as they need, and at least eight for the experts' totals
  const int rows = a.n_tok < sp.pass ? a.n_tok : sp.pass, threads = 32 * rows < 256 ? 256 : 32 * rows;
  k_router_select<EPL, kThreads><<<sp.ctas, threads < kThreads ? threads : kThreads, 0, s>>>(a, sp.passes, sp.pass);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (sp.ctas == 1 && sp.passes == 1)) return e;
  RouteArgs b = a;
  int passes = sp.passes, pass = sp.pass;
  void *args[3] = {&b, &passes, &pass};
  return launch_kernel(reinterpret_cast<const void *>(&k_router_place<1024>), dim3(sp.ctas), dim3(1024), 0, s, args, true);
}

}  // namespace

size_t router_workspace(int64_t n_tok, int n_experts) {
  const Split sp = split_of(n_tok, num_sms());
  if (sp.passes > 1) return static_cast<size_t>(sp.ctas) * n_experts * sizeof(int32_t);
  return sp.ctas == 1 ? 0 : static_cast<size_t>(byte_row(sp.ctas)) * n_experts + 12;  // from a 4-byte boundary to one of 16
}

cudaError_t launch_router(RouteArgs a, cudaStream_t s) {
  const int per16 = a.bf16 ? 8 : 4;
  a.vec = (reinterpret_cast<uintptr_t>(a.logits) & 15u) == 0 && (a.n_tok <= 1 || a.logits_stride % per16 == 0);
  const Split sp = split_of(a.n_tok, num_sms());
  if (sp.passes == 1) a.counts = reinterpret_cast<int32_t *>((reinterpret_cast<uintptr_t>(a.counts) + 15) & ~static_cast<uintptr_t>(15));
  if (a.n_experts <= 64) return launch_select<2>(a, sp, s);
  if (a.n_experts <= 128) return launch_select<4>(a, sp, s);
  if (a.n_experts <= 256) return launch_select<8>(a, sp, s);
  if (a.n_experts <= 512) return launch_select<16>(a, sp, s);
  return launch_select<32>(a, sp, s);
}

}  // namespace epoch
