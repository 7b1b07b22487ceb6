// A router by itself: from logits to each position's experts and weights and to the worklist that the
// products grouped by expert take (expert-major, positions ascending), without running any expert.
//
// One warp a position: the lanes hold consecutive experts' logits, and the k best are ranked in
// registers (topk.cuh). Positions of a CTA are marked in a word of bits for each expert, so that an
// edge's place among the CTA's is a population count, whatever order the warps come in. A second
// kernel adds what earlier CTAs and lower experts hold: every CTA reads all CTAs' counts (64 KB at
// 16384 positions and 256 experts) rather than wait for one that adds them up. Up to 128 positions
// one CTA does both. What bounds it: latency up to some thousand positions, then the instructions of
// the ranking (some 350 a position and warp), not the logits' bytes.
//
// The sigmoid router's order is that of sigmoid(G) + bias in exact arithmetic. It is decided in fp32
// where neighbours are further apart than fp32's roundings can move them, and once more in 64 bits
// for the positions where they are not (about 2 in 1000 with 256 experts).
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
// logits of a lane's EPL consecutive experts; -inf behind the last. vec: rows start on 16-byte boundaries.
template <int EPL> __device__ __forceinline__ void row_logits(const void *row, bool bf16, int E, bool vec, float (&v)[EPL]) {
  const int e0 = lane_id() * EPL;
  if constexpr (EPL % 8 == 0) {
    if (vec && e0 + EPL <= E) {
      if (bf16) {
#pragma unroll
        for (int q = 0; q < EPL / 8; ++q) {
          const uint4 u = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(row) + e0) + q);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[8 * q + 2 * i] = __uint_as_float(w[i] << 16);
            v[8 * q + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
          }
        }
      } else {
#pragma unroll
        for (int q = 0; q < EPL / 4; ++q) {
          const float4 a = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(row) + e0) + q);
          v[4 * q] = a.x, v[4 * q + 1] = a.y, v[4 * q + 2] = a.z, v[4 * q + 3] = a.w;
        }
      }
      return;
    }
  }
#pragma unroll
  for (int c = 0; c < EPL; ++c) v[c] = e0 + c < E ? logit(row, bf16, e0 + c) : -INFINITY;
}

__device__ __forceinline__ double shfl_double(double v, int lane) { return __shfl_sync(0xffffffffu, v, lane); }

// Largest (value, lowest id) of the warp; id < 0: nothing.
__device__ __forceinline__ void warp_best(double &v, int &id) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double w = __shfl_xor_sync(0xffffffffu, v, o);
    const int j = __shfl_xor_sync(0xffffffffu, id, o);
    if (j >= 0 && (id < 0 || w > v || (w == v && j < id))) v = w, id = j;
  }
}

// The selection of one position by sigmoid(G) + bias in 64 bits: lane j < k gets expert j, or -1.
template <int EPL>
__device__ __noinline__ int select_exact(const float *g, const bool *can, const RouteArgs &a) {
  const int lane = lane_id(), E = a.n_experts, gs = E / a.n_group;
  double c[EPL];
  bool ok[EPL];
#pragma unroll 1
  for (int q = 0; q < EPL; ++q) {
    const int e = lane * EPL + q;
    ok[q] = can[q];
    c[q] = 1.0 / (1.0 + exp(-static_cast<double>(g[q]))) + (a.bias != nullptr && e < E ? static_cast<double>(__ldg(a.bias + e)) : 0.0);
    if (c[q] != c[q]) c[q] = -INFINITY;  // a NaN ranks with -inf
  }
  if (a.topk_group < a.n_group) {
    double score = 0.0;  // lane i: group i's
    int held = 0;
#pragma unroll 1
    for (int i = 0; i < a.n_group; ++i) {
      double sum = 0.0;
      int first = -1, n = 0;
#pragma unroll 1
      for (int q = 0; q < EPL; ++q) n += ok[q] && (lane * EPL + q) / gs == i;
      n = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(n)));
#pragma unroll 1
      for (int r = 0; r < 2; ++r) {
        double v = -INFINITY;
        int id = -1;
#pragma unroll 1
        for (int q = 0; q < EPL; ++q) {
          const int e = lane * EPL + q;
          if (ok[q] && e / gs == i && e != first && (id < 0 || c[q] > v)) v = c[q], id = e;
        }
        warp_best(v, id);
        if (id >= 0) sum += v;
        first = id;
      }
      if (lane == i) score = sum, held = n;
    }
    int rank = 0, before = 0;
#pragma unroll 1
    for (int i = 0; i < a.n_group; ++i) {
      const double s = shfl_double(score, i);
      const int h = __shfl_sync(0xffffffffu, held, i);
      if (h > 0 && (s > score || (s == score && i < lane))) ++rank, before += h;
    }
    const unsigned chosen = __ballot_sync(0xffffffffu, lane < a.n_group && held > 0 && (rank < a.topk_group || before < a.top_k));
#pragma unroll 1
    for (int q = 0; q < EPL; ++q) {
      const int i = (lane * EPL + q) / gs;
      if (ok[q] && !((chosen >> (i & 31)) & 1u)) ok[q] = false;
    }
  }
  int sel = -1;
#pragma unroll 1
  for (int j = 0; j < a.top_k; ++j) {
    double v = -INFINITY;
    int id = -1;
#pragma unroll 1
    for (int q = 0; q < EPL; ++q)
      if (ok[q] && (id < 0 || c[q] > v)) v = c[q], id = lane * EPL + q;
    warp_best(v, id);
    if (lane == j) sel = id;
#pragma unroll 1
    for (int q = 0; q < EPL; ++q)
      if (lane * EPL + q == id) ok[q] = false;
  }
  return sel;
}

// Whether two selection scores are apart whatever fp32 made of them: sigmoid is off by at most 4 steps of 2^-23 (expf
// 2, a sum and a quotient), the sum with the bias by half a step of the result; a group's score is the sum of two.
__device__ __forceinline__ bool apart(float a, float b) {
  return fabsf(a - b) > 4e-6f + 8e-7f * fmaxf(fabsf(a), fabsf(b));
}

// The groups that a position may search (clears ok outside them); false where fp32 cannot tell.
template <int EPL>
__device__ __forceinline__ bool limit_groups(const float (&c)[EPL], bool (&ok)[EPL], const RouteArgs &a) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = lane_id(), gs = a.n_experts / a.n_group;
  float score = -INFINITY;  // lane i: group i's
  int held = 0;
  for (int i = 0; i < a.n_group; ++i) {
    unsigned k1 = 0u, k2 = 0u;
    int n = 0;
    const int lo = i * gs - lane * EPL, hi = lo + gs;  // the group's entries of this lane
#pragma unroll
    for (int q = 0; q < EPL; ++q) {
      const unsigned key = ok[q] && q >= lo && q < hi ? order_key(c[q]) : 0u;
      n += key != 0u;
      k2 = max(k2, min(k1, key));
      k1 = max(k1, key);
    }
    const unsigned m1 = __reduce_max_sync(kAll, k1);
    const unsigned hold = __ballot_sync(kAll, k1 == m1 && k1 != 0u);
    const unsigned m2 = __reduce_max_sync(kAll, hold && lane == __ffs(hold) - 1 ? k2 : k1);
    n = static_cast<int>(__reduce_add_sync(kAll, static_cast<unsigned>(n)));
    if (lane == i) {
      held = n;
      score = m1 == 0u ? -INFINITY : m2 == 0u ? key_value(m1) : key_value(m1) + key_value(m2);
    }
  }
  const bool there = lane < a.n_group && held > 0;
  int rank = 0, before = 0;
  for (int i = 0; i < a.n_group; ++i) {
    const float s = __shfl_sync(kAll, score, i);
    const int h = __shfl_sync(kAll, held, i);
    if (h > 0 && (s > score || (s == score && i < lane))) ++rank, before += h;
  }
  const unsigned chosen = __ballot_sync(kAll, there && (rank < a.topk_group || before < a.top_k));
  // A chosen and an unchosen group must be apart; where more than topk_group are taken, their order counts too.
  bool sure = __popc(chosen) <= a.topk_group;
  for (int i = 0; i < a.n_group; ++i) {
    const float s = __shfl_sync(kAll, score, i);
    const int h = __shfl_sync(kAll, held, i);
    const bool other = there && h > 0 && (((chosen >> i) ^ (chosen >> lane)) & 1u);
    sure = sure && !(other && !apart(s, score));
  }
#pragma unroll
  for (int q = 0; q < EPL; ++q)
    if (ok[q] && !((chosen >> (((lane * EPL + q) / gs) & 31)) & 1u)) ok[q] = false;
  return __all_sync(kAll, sure);
}

// One position by one warp: lane j < top_k gets its expert (-1: none) and weight.
template <int EPL>
__device__ __forceinline__ void route_row(const RouteArgs &a, int64_t t, bool vec, const bool (&eligible)[EPL], uint2 *scratch,
                                          int *sel_out, float *w_out) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = lane_id(), k = a.top_k;
  float v[EPL];
  bool ok[EPL];
  const bool bf16 = a.bf16 != 0;
  const void *row = static_cast<const uint8_t *>(a.logits) + t * a.logits_stride * (bf16 ? 2 : 4);
  row_logits<EPL>(row, bf16, a.n_experts, vec, v);
  bool nan = false;
#pragma unroll
  for (int c = 0; c < EPL; ++c) {
    ok[c] = eligible[c] && v[c] != -INFINITY;
    nan = nan || v[c] != v[c];
  }
  int sel;
  float val, w;
  if (!a.sigmoid) {
    warp_topk<EPL>(v, ok, k, &sel, &val, scratch);
    const bool on = lane < k && sel >= 0;
    float top, sum;
    if (a.raw_weights) {  // probabilities over all experts, eligible or not
      float m = v[0];
#pragma unroll
      for (int c = 1; c < EPL; ++c) m = fmaxf(m, v[c]);
      top = key_value(__reduce_max_sync(kAll, order_key(m)));
      sum = 0.f;
#pragma unroll
      for (int c = 0; c < EPL; ++c) sum += lane * EPL + c < a.n_experts ? expf(v[c] - top) : 0.f;
    } else {
      top = __shfl_sync(kAll, val, 0);
      sum = on ? expf(val - top) : 0.f;
    }
    w = on ? expf(val - top) : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    w = on ? w / sum : 0.f;
  } else {
    float c[EPL];
    bool open[EPL];
#pragma unroll
    for (int q = 0; q < EPL; ++q) {
      const int e = lane * EPL + q;
      c[q] = 1.0f / (1.0f + expf(-v[q])) + (a.bias != nullptr && e < a.n_experts ? __ldg(a.bias + e) : 0.f);
      open[q] = ok[q];
    }
    bool sure = true;
    if (a.topk_group < a.n_group) sure = limit_groups<EPL>(c, open, a);
    if (sure) {
      // one more than asked for, so that the last border is seen too
      warp_topk<EPL>(c, open, k + 1, &sel, &val, scratch);
      const float next = __shfl_down_sync(kAll, val, 1);
      const int after = __shfl_down_sync(kAll, sel, 1);
      bool far = true, tied = false;
      if (lane < k && sel >= 0 && after >= 0 && !apart(val, next)) {
        // equal logits and equal biases are equal scores, in the order of their ids
        const float b0 = a.bias ? __ldg(a.bias + sel) : 0.f, b1 = a.bias ? __ldg(a.bias + after) : 0.f;
        far = tied = logit(row, bf16, sel) == logit(row, bf16, after) && b0 == b1;
      }
      if (__ballot_sync(kAll, tied) >> (k - 1) & 1u) {
        // a tie at the last border: nothing else may be near it, or it could belong before both
        const int at = __shfl_sync(kAll, sel, k - 1);
        const float edge = __shfl_sync(kAll, val, k - 1), g = logit(row, bf16, at), b = a.bias ? __ldg(a.bias + at) : 0.f;
#pragma unroll
        for (int q = 0; q < EPL; ++q) {
          const int e = lane * EPL + q;
          if (open[q] && !apart(c[q], edge)) far = far && v[q] == g && (a.bias == nullptr || __ldg(a.bias + e) == b);
        }
      }
      sure = __all_sync(kAll, far);
    }
    if (!sure) sel = select_exact<EPL>(v, ok, a);
    const bool on = lane < k && sel >= 0;
    const float g = on ? logit(row, bf16, sel) : 0.f;
    w = on ? 1.0f / (1.0f + expf(-g)) : 0.f;
    if (!a.raw_weights) {
      float sum = w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
      w = on ? w / sum : 0.f;
    }
  }
  if (__any_sync(kAll, nan) && sel >= 0) w = __uint_as_float(0x7FC00000u);  // a NaN among a position's logits spoils its weights
  *sel_out = lane < k ? sel : -1;
  *w_out = w;
}

// First entries of the experts (offsets, E + 1 values in shared memory) from their totals; all threads of the CTA.
template <int THREADS> __device__ __forceinline__ void scan_totals(const int *total, int E, int *offsets, int *s_warp) {
  const int tid = threadIdx.x, lane = lane_id(), warp = warp_id();
  constexpr int kWarps = THREADS / 32;
  int carry = 0;
  for (int base = 0; base < E; base += THREADS) {
    const int e = base + tid, n = e < E ? total[e] : 0;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    int add = carry;
    for (int w = 0; w < kWarps; ++w) {
      const int s = s_warp[w];
      if (w < warp) add += s;
      carry += s;
    }
    if (e < E) offsets[e] = add + sum - n;
    __syncthreads();
  }
  if (tid == 0) offsets[E] = carry;
  __syncthreads();
}

// Selection, weights and, in slots, each edge's place among its CTA's edges of the expert; the CTA's counts. The only
// CTA of a grid (with one pass) finishes the worklist too.
template <int EPL, int THREADS>
__global__ void __launch_bounds__(THREADS) k_router_select(const RouteArgs a, int passes, int pass) {
  constexpr int kWarps = THREADS / 32, kRows = kPass / kWarps;  // positions of a warp in a full pass
  constexpr int kE = EPL * 32;
  __shared__ uint32_t s_bits[kPass / 32][kE];
  __shared__ int s_count[kE], s_off[kE + 1], s_warp[kWarps];
  __shared__ uint2 s_scratch[kWarps][32];
  const int tid = threadIdx.x, lane = lane_id(), warp = warp_id(), E = a.n_experts, k = a.top_k;
  const int words = pass / 32;
  const bool vec = a.vec != 0, one = gridDim.x == 1 && passes == 1;
  for (int i = tid; i < kE; i += THREADS) {
    s_count[i] = 0;
#pragma unroll
    for (int w = 0; w < kPass / 32; ++w) s_bits[w][i] = 0u;
  }
  bool eligible[EPL];
#pragma unroll
  for (int c = 0; c < EPL; ++c) {
    const int e = lane * EPL + c;
    eligible[c] = e < E && (a.eligible == nullptr || __ldg(a.eligible + e) != 0);
  }
  const int64_t first = static_cast<int64_t>(blockIdx.x) * passes * pass;
  pdl_trigger();
  for (int p = 0; p < passes; ++p) {
    const int64_t t0 = first + static_cast<int64_t>(p) * pass;
    if (t0 >= a.n_tok) break;
    __syncthreads();  // the words are clear
    int sel[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = i * kWarps + warp;
      const int64_t t = t0 + r;
      sel[i] = -1;
      if (r >= pass || t >= a.n_tok) continue;
      float w = 0.f;
      if (a.live == nullptr || __ldg(a.live + t) != 0) route_row<EPL>(a, t, vec, eligible, s_scratch[warp], &sel[i], &w);
      if (lane < k) {
        a.sel[t * k + lane] = sel[i];
        a.weights[t * k + lane] = w;
        if (sel[i] >= 0) atomicOr(&s_bits[r >> 5][sel[i]], 1u << (r & 31));
      }
    }
    __syncthreads();
    int place[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = i * kWarps + warp;
      const int64_t t = t0 + r;
      place[i] = -1;
      if (r >= pass || t >= a.n_tok || lane >= k) continue;
      if (sel[i] >= 0) {
        place[i] = s_count[sel[i]];
        for (int w = 0; w < (r >> 5); ++w) place[i] += __popc(s_bits[w][sel[i]]);
        place[i] += __popc(s_bits[r >> 5][sel[i]] & ((1u << (r & 31)) - 1u));
      }
      if (!one) a.slots[t * k + lane] = place[i];
    }
    __syncthreads();
    for (int i = tid; i < E; i += THREADS) {
      int n = s_count[i];
      for (int w = 0; w < words; ++w) {
        n += __popc(s_bits[w][i]);
        s_bits[w][i] = 0u;
      }
      s_count[i] = n;
    }
    if (one) {
      __syncthreads();
      scan_totals<THREADS>(s_count, E, s_off, s_warp);
      for (int i = tid; i <= E; i += THREADS) a.offsets[i] = s_off[i];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = i * kWarps + warp;
        const int64_t t = t0 + r;
        if (r >= pass || t >= a.n_tok || lane >= k) continue;
        const int slot = sel[i] >= 0 ? s_off[sel[i]] + place[i] : -1;
        a.slots[t * k + lane] = slot;
        if (slot >= 0) a.positions[slot] = static_cast<int>(t);
      }
      for (int64_t i = s_off[E] + tid; i < static_cast<int64_t>(a.n_tok) * k; i += THREADS) a.positions[i] = -1;
    }
  }
  if (!one) {
    __syncthreads();
    for (int i = tid; i < E; i += THREADS)
      a.counts[static_cast<int64_t>(blockIdx.x) * E + i] = s_count[i];
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
    const int e = i % E, part = i / E;
    int total = 0, before = 0;
#pragma unroll 8
    for (int b = part; b < ctas; b += per) {
      const int n = __ldcg(a.counts + static_cast<int64_t>(b) * E + e);
      total += n;
      before += b < mine ? n : 0;
    }
    if (per == 1) {
      s_total[e] = total;
      s_before[e] = before;
    } else {
      atomicAdd(&s_total[e], total);
      atomicAdd(&s_before[e], before);
    }
  }
  __syncthreads();
  scan_totals<THREADS>(s_total, E, s_off, s_warp);
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
// Passes of 32, 64 or 128 positions, the shortest with which one pass of every SM takes all; a single CTA up to 128.
Split split_of(int64_t n, int sms) {
  Split s;
  s.pass = n <= kPass || n > 64ll * sms ? kPass : n > 32ll * sms ? 64 : 32;
  if (n <= 32) s.pass = 32;
  else if (n <= 64) s.pass = 64;
  const int64_t all = (n + s.pass - 1) / s.pass;
  s.passes = static_cast<int>((all + sms - 1) / sms);
  s.ctas = static_cast<int>((all + s.passes - 1) / s.passes);
  return s;
}

template <int EPL> cudaError_t launch_select(const RouteArgs &a, const Split &sp, cudaStream_t s) {
  constexpr int kThreads = EPL <= 8 ? 1024 : 512;
  k_router_select<EPL, kThreads><<<sp.ctas, kThreads, 0, s>>>(a, sp.passes, sp.pass);
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
  return sp.ctas == 1 && sp.passes == 1 ? 0 : static_cast<size_t>(sp.ctas) * n_experts * sizeof(int32_t);
}

cudaError_t launch_router(RouteArgs a, cudaStream_t s) {
  const int per16 = a.bf16 ? 8 : 4;
  a.vec = (reinterpret_cast<uintptr_t>(a.logits) & 15u) == 0 && (a.n_tok <= 1 || a.logits_stride % per16 == 0);
  const Split sp = split_of(a.n_tok, num_sms());
  if (a.n_experts <= 64) return launch_select<2>(a, sp, s);
  if (a.n_experts <= 256) return launch_select<8>(a, sp, s);
  return launch_select<32>(a, sp, s);
}

}  // namespace epoch
