// Routing to many experts: scores, a balance bias, expert groups, top-k, gates and the dispatch order.
//
//   s_e = softmax(l)_e or 1 / (1 + exp(-l_e)),   key_e = s_e + b_e   (without a bias: rank by l_e)
//   group score = sum of the group_top largest keys of the group; the top_groups best groups are kept
//   e_1..e_k = the experts of the kept groups ranked first by (key descending, index ascending)
//   gate_i = scale * s_{e_i} [/ sum_j s_{e_j}]         (the bias decides who is chosen, not the weight)
//   rows: expert segments in order, ascending tokens inside each: row_of, token_of_row, counts, offsets
// An expert whose logit or bias is -inf or NaN is masked: never chosen.  A token with fewer than k
// experts left gets index -1, gate 0 and row -1 in its last slots.
//
// The choice is that of the keys in 64 bits: scores are fp32, with a bound on their error beside them;
// where a choice is not decided by more than the bounds (about one token in two thousand on normal
// logits), the warp ranks that token again with 64-bit keys.  So which experts serve a token does not
// hang on the rounding of one exp.  Two slots that hold the same logit and bias are equal, not close:
// the lower index is right without a second look.
//
// One warp a token, runs of experts over its lanes (expert = lane * slots + slot, so that groups are
// neighbouring lanes and a lane's logits one or two 16-byte loads).  The k-th largest of the lanes' best
// keys leaves a few more than k candidates, which are ranked by counting.  Ranks inside a chunk of 32
// tokens come from one 32-bit token mask per expert.
//
// Measured on one GB300: one token of 256 experts in 8 groups 6 us on the device (the latency of one
// kernel); 8192 tokens 34 to 38 us a call (three kernels: about 25, 4 and 5 us, of the first about 13 us once for
// the few close calls of such a batch), against 1.4 us of bytes: bound by instruction issue (about 1200 a token,
// 0.56 of the slots) and by the 64-bit unit.  Gradient, 8192 x 64: 6 us on the device.
#include <algorithm>

#include "ops_common.cuh"

namespace colibri {
namespace {

constexpr int kRouteMaxE = 512, kRouteMaxK = 32, kRouteMaxGroups = 32;
constexpr int kRouteTokens = 32;  // tokens of a chunk: the bits of an expert's token mask
constexpr int kRouteWarps = 16;
constexpr int64_t kNoKey = INT64_MIN;  // below every ordered double

struct RouteManyArgs {
  const void* logits;
  int64_t ld;
  const float* bias;
  int T, E, k, groups, per_group, top_groups, group_top, softmax, renorm;
  int lanes_per_group;  // where every group is a run of 1, 2, 4 .. 32 whole lanes, else 0
  int aligned;          // logits rows start on 16 bytes
  float scale;
  int32_t *idx, *counts, *offsets, *row_of, *token_of_row;
  float* gate;
  int32_t* hist;  // [E][chunks]: a chunk's tokens per expert, then the tokens of earlier chunks
  int chunks;
};

// Floats as unsigned numbers in the same order (no NaN).
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);  // -0 becomes +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ float warp_max(float v) { return unordered(__reduce_max_sync(~0u, ordered(v))); }
__device__ __forceinline__ float warp_min(float v) { return unordered(__reduce_min_sync(~0u, ordered(v))); }

template <typename T>
__device__ __forceinline__ bool before(T va, int ia, T vb, int ib) {
  return va > vb || (va == vb && ia < ib);
}

// Doubles (no NaN) as integers in the same order: comparisons run at the integer rate, not the 64-bit one.
__device__ __forceinline__ int64_t ordered(double v) {
  const int64_t u = __double_as_longlong(v + 0.0);
  return u ^ ((u >> 63) & 0x7fffffffffffffffll);
}
// Best (value, index) of the warp, in every lane.
__device__ __forceinline__ void warp_best(int64_t& v, int& i) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const int64_t w = __shfl_xor_sync(~0u, v, o);
    const int j = __shfl_xor_sync(~0u, i, o);
    if (before(w, j, v, i)) v = w, i = j;
  }
}

// What of the experts does not change from token to token, in shared memory (registers are what bounds the
// warps at work): biases (-inf: masked, a NaN too; 0 without) and group numbers.
template <int NS>
struct Experts {
  float bias[NS * 32];
  uint8_t group[NS * 32];
  __device__ __forceinline__ void fill(const RouteManyArgs& a) {
    for (int e = threadIdx.x; e < NS * 32; e += blockDim.x) {
      float b = 0.f;
      if (a.bias && e < a.E) b = a.bias[e] > -INFINITY ? a.bias[e] : -INFINITY;
      bias[e] = b;
      group[e] = a.groups > 1 && e < a.E ? e / a.per_group : 0;
    }
  }
};

// A lane's logits as fp32; a NaN, and what lies past E, is -inf.
template <typename L, int NS>
__device__ __forceinline__ void load_logits(const RouteManyArgs& a, int t, int e0, float (&l)[NS]) {
  const L* row = static_cast<const L*>(a.logits) + t * a.ld;
  if constexpr (NS >= 8) {
    if (a.aligned && e0 + NS <= a.E) {
#pragma unroll
      for (int j = 0; j < NS; j += 8) {
        float v[8];
        load8(row + e0 + j, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) l[j + i] = v[i] > -INFINITY ? v[i] : -INFINITY;
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    l[j] = e0 + j < a.E ? to_float(row[e0 + j]) : -INFINITY;
    if (!(l[j] > -INFINITY)) l[j] = -INFINITY;
  }
}

// 1 / the softmax's sum in 64 bits over the row's logits, m their maximum (all lanes).
template <typename L>
__device__ __forceinline__ double softmax_scale(const RouteManyArgs& a, const L* row, float m) {
  double sum = 0.0;
  for (int e = threadIdx.x & 31; e < a.E; e += 32) {
    const float l = to_float(row[e]);
    if (l == m)
      sum += 1.0;
    else if (l > -INFINITY)
      sum += exp((double)l - (double)m);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  return sum;
}
// The biased score of an admissible logit in 64 bits.
__device__ __forceinline__ double exact_key(const RouteManyArgs& a, float l, float m, double sum, int e) {
  const double s = a.softmax ? (l == m ? 1.0 : exp((double)l - (double)m)) / sum : 1.0 / (1.0 + exp(-(double)l));
  return a.bias ? s + (double)a.bias[e] : s;
}

// Ranks the listed experts (at most 32, those that can be among the k best) by their 64-bit keys; the list
// becomes the ranking.  One evaluation a lane.
template <typename L>
__device__ __noinline__ void rank_candidates(const RouteManyArgs& a, int t, float m, int16_t* list, int count) {
  const int lane = threadIdx.x & 31;
  const L* row = static_cast<const L*>(a.logits) + t * a.ld;
  const double sum = a.softmax ? softmax_scale(a, row, m) : 1.0;
  const int e = lane < count ? list[lane] : 0;
  const int64_t key = lane < count ? ordered(exact_key(a, to_float(row[e]), m, sum, e)) : kNoKey;
  int rank = 0;
  for (int i = 0; i < count; ++i) rank += before(__shfl_sync(~0u, key, i), __shfl_sync(~0u, e, i), key, e);
  __syncwarp();
  if (lane < count) list[rank] = e;
  __syncwarp();
}

// The whole selection, groups and experts, by 64-bit keys: returns lane i's (i < k) expert, or -1.
template <typename L, int NS>
__device__ __noinline__ int select_exact(const RouteManyArgs& a, const Experts<NS>& ex, int t, float m) {
  const int lane = threadIdx.x & 31;
  const L* row = static_cast<const L*>(a.logits) + t * a.ld;
  const int e0 = lane * NS;
  const double sum = a.softmax ? softmax_scale(a, row, m) : 1.0;
  double key[NS];  // what groups are ranked by
  int64_t rank_by[NS];
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    const int e = e0 + j;
    const float l = e < a.E ? to_float(row[e]) : -INFINITY;
    const bool live = l > -INFINITY && ex.bias[e] > -INFINITY;
    key[j] = live ? exact_key(a, l, m, sum, e) : 0.0;
    rank_by[j] = live ? ordered(a.bias ? key[j] : (double)l) : kNoKey;
  }
  uint32_t kept = ~0u;
  if (a.groups > 1) {
    int64_t mine = kNoKey;
    for (int g = 0; g < a.groups; ++g) {
      double total = 0.0;
      int64_t worth = kNoKey;
      int first = -1;
      for (int n = 0; n < a.group_top; ++n) {
        int64_t v = kNoKey;
        int i = kRouteMaxE;
        double mine_d = 0.0;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          if (ex.group[e0 + j] != g || e0 + j == first || rank_by[j] == kNoKey) continue;
          // one expert a group and no bias: the logits rank the groups, as they rank the experts
          const int64_t r = a.group_top == 1 ? rank_by[j] : ordered(key[j]);
          if (before(r, e0 + j, v, i)) v = r, i = e0 + j, mine_d = key[j];
        }
        const int own = i;
        warp_best(v, i);
        if (i == kRouteMaxE) break;
        if (a.group_top == 1) {
          worth = v;
        } else {
          total += __shfl_sync(~0u, mine_d, __ffs(__ballot_sync(~0u, own == i)) - 1);
          worth = ordered(total);
        }
        first = i;
      }
      if (lane == g) mine = worth;
    }
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) rank += before(__shfl_sync(~0u, mine, g), g, mine, lane);
    kept = __ballot_sync(~0u, lane < a.groups && rank < a.top_groups);
  }
#pragma unroll
  for (int j = 0; j < NS; ++j)
    if (e0 + j >= a.E || !(kept >> ex.group[e0 + j] & 1)) rank_by[j] = kNoKey;
  int sel = -1;
  for (int n = 0; n < a.k; ++n) {
    int64_t v = kNoKey;
    int i = kRouteMaxE;
#pragma unroll
    for (int j = 0; j < NS; ++j)
      if (rank_by[j] != kNoKey && before(rank_by[j], e0 + j, v, i)) v = rank_by[j], i = e0 + j;
    warp_best(v, i);
    if (i == kRouteMaxE) break;
#pragma unroll
    for (int j = 0; j < NS; ++j)
      if (e0 + j == i) rank_by[j] = kNoKey;
    if (lane == n) sel = i;
  }
  return sel;
}

// The two larger of (a1 >= a2) and (b1 >= b2).
__device__ __forceinline__ void merge_top2(float& a1, float& a2, float b1, float b2) {
  const float lo = fminf(a1, b1);
  a1 = fmaxf(a1, b1);
  a2 = fmaxf(lo, fmaxf(a2, b2));
}

// Which groups compete (a bit each), by the sums of their best keys; `unsure` if the error bounds do not
// decide it.
template <int NS>
__device__ __forceinline__ uint32_t keep_groups(const RouteManyArgs& a, const Experts<NS>& ex, const float (&key)[NS],
                                                float err, bool& unsure) {
  const int lane = threadIdx.x & 31;
  const bool by_logit = a.group_top == 1 && !a.bias;  // keys are logits: exact
  float best = -INFINITY, second = -INFINITY, off = 0.f;  // of group `lane`, in its lane
  if (a.lanes_per_group) {
    // groups are runs of 1, 2, 4 .. 32 lanes: all of them at once, by exchanges inside the runs
    float v = -INFINITY, v2 = -INFINITY, o = err;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      v2 = fmaxf(v2, fminf(v, key[j]));
      v = fmaxf(v, key[j]);
    }
    for (int d = 1; d < a.lanes_per_group; d <<= 1) {
      merge_top2(v, v2, __shfl_xor_sync(~0u, v, d), __shfl_xor_sync(~0u, v2, d));
      o = fmaxf(o, __shfl_xor_sync(~0u, o, d));
    }
    const int from = (lane * a.lanes_per_group) & 31;
    best = __shfl_sync(~0u, v, from), second = __shfl_sync(~0u, v2, from), off = __shfl_sync(~0u, o, from);
  } else {
    for (int g = 0; g < a.groups; ++g) {
      float v = -INFINITY, v2 = -INFINITY, o = 0.f;
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        if (ex.group[lane * NS + j] != g || key[j] == -INFINITY) continue;
        o = err;
        v2 = fmaxf(v2, fminf(v, key[j]));
        v = fmaxf(v, key[j]);
      }
      const float b = warp_max(v);
      // the second best: the lane that gave the best (the first of equals) offers its next one
      const uint32_t who = __ballot_sync(~0u, v == b);
      const float b2 = a.group_top == 2 ? warp_max(lane == __ffs(who) - 1 ? v2 : v) : -INFINITY;
      o = warp_max(o);
      if (lane == g) best = b, second = b2, off = o;
    }
  }
  float total = best;
  if (a.group_top == 2 && second > -INFINITY) total += second;
  off = by_logit ? 0.f : 2.f * off + fabsf(total > -INFINITY ? total : 0.f) * 0x1p-23f;
  int rank = 0;
  for (int g = 0; g < a.groups; ++g) rank += before(__shfl_sync(~0u, total, g), g, total, lane);
  const bool in = lane < a.groups && rank < a.top_groups;
  if (!by_logit && a.top_groups < a.groups) {
    const float lowest = warp_min(in ? total - off : INFINITY);
    const float highest = warp_max(lane < a.groups && !in ? total + off : -INFINITY);
    unsure = !(lowest > highest) && highest > -INFINITY;
  }
  return __ballot_sync(~0u, in);
}

// A bound on the error of the fp32 key of a logit, besides 2^-120 (what is lost below the normal range): the
// score's and half an ulp of its sum with the bias.  Softmax: v - m is rounded to 2^-24 of itself, exp to 2
// ulp, the sum (at most 16 + 5 additions) and the product with 1 / sum to less than 2^-18.5 together.
// Sigmoid by the fast exp (2 + 1.173 |v| ulp) and the fast quotient (2 ulp).
__device__ __forceinline__ float key_error(const RouteManyArgs& a, float v, float m, float score, float key) {
  const float rel = a.softmax ? 0x1p-18f + 0x1p-22f * fminf(m - v, 200.f) : 0x1p-21f + 0x1.4p-23f * fabsf(v);
  return score * rel + fabsf(key) * 0x1p-23f;
}

struct RouteScratch {
  float key[kRouteMaxK];    // a token's candidates
  int16_t expert[kRouteMaxK];
};

// Routes token t with one warp: lane i (i < k) returns its expert (-1: none) and its score; m, the softmax's
// largest logit (0 for sigmoids).
template <typename L, int NS>
__device__ __forceinline__ void route_token(const RouteManyArgs& a, const Experts<NS>& ex, int t,
                                            RouteScratch& scratch, int& sel, float& s_sel, float& m) {
  const int lane = threadIdx.x & 31;
  const int e0 = lane * NS;
  float key[NS];
  load_logits<L, NS>(a, t, e0, key);
  float inv = 0.f;
  m = 0.f;
  auto raw_score = [&](float v) { return v == -INFINITY ? 0.f : (v == m ? 1.f : expf(v - m)); };
  if (a.softmax) {
    m = -INFINITY;
#pragma unroll
    for (int j = 0; j < NS; ++j) m = fmaxf(m, key[j]);
    m = warp_max(m);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NS; ++j) sum += raw_score(key[j]);
    sum = warp_sum(sum);
    inv = sum > 0.f ? 1.f / sum : 0.f;
  }
  float err = 0.f;  // the largest of this lane's keys
  if (a.bias || (a.groups > 1 && a.group_top == 2)) {  // else the logits are the keys
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const float l = key[j], b = ex.bias[e0 + j];
      const float s = a.softmax ? raw_score(l) * inv : __fdividef(1.f, 1.f + __expf(-l));
      const bool live = l > -INFINITY && b > -INFINITY;
      key[j] = live ? s + b : -INFINITY;
      if (live) err = fmaxf(err, key_error(a, l, m, s, key[j]));
    }
    err += 0x1p-120f;
  }
  bool unsure_groups = false, unsure = false;
  // the experts that are left, by (key, index)
  if (a.groups > 1) {
    const uint32_t kept = keep_groups<NS>(a, ex, key, err, unsure_groups);
    if (!a.bias && a.group_top == 2) load_logits<L, NS>(a, t, e0, key);
#pragma unroll
    for (int j = 0; j < NS; ++j)
      if (!(kept >> ex.group[e0 + j] & 1)) key[j] = -INFINITY;
  }
  float best = -INFINITY;
#pragma unroll
  for (int j = 0; j < NS; ++j) best = fmaxf(best, key[j]);
  // k lanes have a key at or above the k-th largest of the lanes' best, so the k best keys are among those at
  // or above it: the candidates, usually a few more than k
  uint32_t sorted = ordered(best);
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int d = size >> 1; d > 0; d >>= 1) {  // bitonic, descending
      const uint32_t other = __shfl_xor_sync(~0u, sorted, d);
      const bool up = ((lane & d) == 0) == ((lane & size) == 0);
      sorted = up ? max(sorted, other) : min(sorted, other);
    }
  const float least = unordered(__shfl_sync(~0u, sorted, a.k - 1));
  int n = 0;
#pragma unroll
  for (int j = 0; j < NS; ++j) n += key[j] > -INFINITY && key[j] >= least;
  auto exclusive = [&](int v, int& total) {
    int to = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int w = __shfl_up_sync(~0u, to, o);
      if (lane >= o) to += w;
    }
    total = __shfl_sync(~0u, to, 31);
    return to - v;
  };
  int count, to = exclusive(n, count);
  float mine = -INFINITY;
  sel = -1;
  if (count <= kRouteMaxK) {
#pragma unroll
    for (int j = 0; j < NS; ++j)
      if (key[j] > -INFINITY && key[j] >= least) scratch.key[to] = key[j], scratch.expert[to] = e0 + j, ++to;
    __syncwarp();
    // the list is in the order of the experts: equal keys rank by their places
    const float my = lane < count ? scratch.key[lane] : -INFINITY;
    const int e = scratch.expert[lane];
    int rank = 0;
    for (int i = 0; i < count; ++i) {
      const float o = scratch.key[i];
      rank += o > my || (o == my && i < lane);
    }
    __syncwarp();
    if (lane < count) scratch.key[rank] = my, scratch.expert[rank] = e;
    __syncwarp();
    if (lane < min(count, a.k)) sel = scratch.expert[lane], mine = scratch.key[lane];
    __syncwarp();
  } else {  // many equal or few lanes: one at a time
    uint32_t taken = 0;
    for (int i = 0; i < a.k; ++i) {
      float v = -INFINITY;
      int at = 0;
#pragma unroll
      for (int j = NS - 1; j >= 0; --j)
        if (!(taken >> j & 1) && key[j] >= v) v = key[j], at = j;
      const uint32_t o = ordered(v), top = __reduce_max_sync(~0u, o);
      if (top == ordered(-INFINITY)) break;
      const int owner = __ffs(__ballot_sync(~0u, o == top)) - 1;  // lanes in the order of their experts
      const int e = __shfl_sync(~0u, e0 + at, owner);
      if (lane == i) sel = e, mine = unordered(top);
      if (lane == owner) taken |= 1u << at;
    }
  }
  const L* row = static_cast<const L*>(a.logits) + t * a.ld;
  auto score_of = [&](float v) { return a.softmax ? raw_score(v) * inv : 1.f / (1.f + expf(-v)); };
  float ml = sel >= 0 ? to_float(row[sel]) : -INFINITY;
  s_sel = sel >= 0 ? score_of(ml) : 0.f;
  if (a.bias) {
    const int found = __popc(__ballot_sync(~0u, sel >= 0));
    const float off = sel >= 0 ? key_error(a, ml, m, s_sel * (1.f + 0x1p-18f), mine) + 0x1p-120f : 0.f;
    // neighbours in the ranking; equal logits with equal biases are no close call
    const float nv = __shfl_down_sync(~0u, mine, 1), no = __shfl_down_sync(~0u, off, 1), nl = __shfl_down_sync(~0u, ml, 1);
    const float mb = sel >= 0 ? a.bias[sel] : 0.f, nb = __shfl_down_sync(~0u, mb, 1);
    unsure = lane + 1 < found && !(mine - off > nv + no) && !(ml == nl && mb == nb);
    // the least that any chosen one can be, against everything that was not chosen
    const float lo = warp_min(sel >= 0 ? mine - off : INFINITY);
    int reach = 0;
#pragma unroll
    for (int j = 0; j < NS; ++j) reach += key[j] > -INFINITY && !(key[j] + err < lo);
    if (found == a.k && __reduce_add_sync(~0u, reach) > found) {
      const float ll = __shfl_sync(~0u, ml, a.k - 1), lb = __shfl_sync(~0u, mb, a.k - 1);
      const float lk = __shfl_sync(~0u, mine, a.k - 1);
      const int le = __shfl_sync(~0u, sel, a.k - 1);
      float l[NS];
      load_logits<L, NS>(a, t, e0, l);
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        const bool chosen = key[j] > lk || (key[j] == lk && e0 + j <= le);
        if (key[j] > -INFINITY && !chosen && !(key[j] + err < lo) && !(l[j] == ll && ex.bias[e0 + j] == lb)) unsure = true;
      }
    }
    unsure = __any_sync(~0u, unsure);
    if (unsure && !unsure_groups) {  // everything that may be among the best
      to = exclusive(reach, count);
      if (count <= kRouteMaxK) {
#pragma unroll
        for (int j = 0; j < NS; ++j)
          if (key[j] > -INFINITY && !(key[j] + err < lo)) scratch.expert[to++] = e0 + j;
        __syncwarp();
        rank_candidates<L>(a, t, m, scratch.expert, count);
        sel = lane < min(count, a.k) ? scratch.expert[lane] : -1;
        __syncwarp();
      }
    }
  }
  if (unsure_groups || (unsure && count > kRouteMaxK)) sel = select_exact<L, NS>(a, ex, t, m);
  if (unsure_groups || unsure) {
    ml = sel >= 0 ? to_float(row[sel]) : -INFINITY;
    s_sel = sel >= 0 ? score_of(ml) : 0.f;
  }
}

// Gates that divide by the chosen scores' sum hang on the scores' ratios alone, which stay what they are where
// fp32 loses the scores themselves (a sigmoid below a logit of about -88, a softmax of experts that far below
// the row's largest).  A token with a chosen score below kTinyScore takes its scores less a factor that is
// common to all of them: softmax, e^largest of the chosen over the row's sum; sigmoid, where s = e^l / (1 + e^l),
// e^largest if that is below one (else the largest score is a half or more, and what is lost is below 2^-125).
// Scores that 64 bits lose too, below e^-700, are zero: a logit of the type's lowest value is as good as masked.
// base: the softmax's largest logit, 0 for sigmoids.
constexpr float kTinyScore = 0x1p-100f;
__device__ __forceinline__ float relative_score(bool live, float l, float base, bool softmax) {
  if (l - base < -700.f) live = false;
  const float top = warp_max(live ? l : -INFINITY);
  if (!live) return 0.f;
  if (softmax) return l == top ? 1.f : expf(l - top);
  return top < 0.f ? expf(l - top) / (1.f + expf(l)) : 1.f / (1.f + expf(-l));
}

// offsets[e] = rows before expert e, from counts in shared memory, by one warp; returns nothing past it.
__device__ __forceinline__ void scan_counts(const int* counts, int* offsets, int E) {
  const int lane = threadIdx.x & 31;
  const int per = (E + 31) / 32;
  int sum = 0;
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i;
    if (e < E) sum += counts[e];
  }
  int before_me = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(~0u, before_me, o);
    if (lane >= o) before_me += v;
  }
  if (lane == 31) offsets[E] = before_me;
  before_me -= sum;
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i;
    if (e < E) {
      offsets[e] = before_me;
      before_me += counts[e];
    }
  }
}

// One chunk of 32 tokens a block.  With a single chunk the whole dispatch is done here; else row_of
// holds ranks inside the chunk and hist the chunk's counts.
template <typename L, int NS>
__global__ void __launch_bounds__(32 * kRouteWarps, NS <= 8 ? 2 : 1)
    route_tokens_kernel(const __grid_constant__ RouteManyArgs a) {
  __shared__ uint32_t mask[NS * 32];
  __shared__ int count[NS * 32], offset[NS * 32 + 1];
  __shared__ int16_t chosen[kRouteTokens][kRouteMaxK];
  __shared__ RouteScratch scratch[kRouteWarps];
  __shared__ __align__(16) Experts<NS> ex;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  for (int e = threadIdx.x; e < NS * 32; e += blockDim.x) mask[e] = 0;
  pdl_wait();
  const int t0 = blockIdx.x * kRouteTokens, n = min(kRouteTokens, a.T - t0);
  ex.fill(a);
  __syncthreads();
  for (int i = warp; i < n; i += warps) {
    int sel;
    float s, base;
    route_token<L, NS>(a, ex, t0 + i, scratch[warp], sel, s, base);
    if (a.renorm && __any_sync(~0u, sel >= 0 && s < kTinyScore)) {
      const L* row = static_cast<const L*>(a.logits) + (t0 + i) * a.ld;
      s = relative_score(sel >= 0, sel >= 0 ? to_float(row[sel]) : 0.f, base, a.softmax);
    }
    const float sum = warp_sum(lane < a.k ? s : 0.f);
    if (lane < a.k) {
      const int64_t o = (int64_t)(t0 + i) * a.k + lane;
      a.idx[o] = sel;
      a.gate[o] = a.renorm ? (sum > 0.f ? a.scale * (s / sum) : 0.f) : a.scale * s;
      chosen[i][lane] = sel;
      if (sel >= 0) atomicOr(&mask[sel], 1u << i);  // bits of different tokens: any order gives the same
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    count[e] = __popc(mask[e]);
    if (a.chunks > 1) a.hist[(int64_t)e * a.chunks + blockIdx.x] = count[e];
  }
  if (a.chunks == 1) {
    __syncthreads();
    if (warp == 0) scan_counts(count, offset, a.E);
    __syncthreads();
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) {
      a.offsets[e] = offset[e];
      if (e < a.E) a.counts[e] = count[e];
    }
    for (int i = offset[a.E] + threadIdx.x; i < a.T * a.k; i += blockDim.x) a.token_of_row[i] = -1;
  }
  for (int i = threadIdx.x; i < n * a.k; i += blockDim.x) {
    const int tok = i / a.k, e = chosen[tok][i % a.k];
    int r = -1;
    if (e >= 0) {
      r = __popc(mask[e] & ((1u << tok) - 1));
      if (a.chunks == 1) {
        r += offset[e];
        a.token_of_row[r] = tok;
      }
    }
    a.row_of[(int64_t)t0 * a.k + i] = r;
  }
}

// hist[e][c] becomes the tokens of e in chunks before c; counts[e] their total.  One warp an expert.
__global__ void __launch_bounds__(256) route_scan_kernel(RouteManyArgs a) {
  const int e = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  pdl_wait();
  if (e >= a.E) return;
  int32_t* h = a.hist + (int64_t)e * a.chunks;
  int carry = 0;
  for (int c0 = 0; c0 < a.chunks; c0 += 32) {
    const int v = c0 + lane < a.chunks ? h[c0 + lane] : 0;
    int run = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int w = __shfl_up_sync(~0u, run, o);
      if (lane >= o) run += w;
    }
    if (c0 + lane < a.chunks) h[c0 + lane] = carry + run - v;
    carry += __shfl_sync(~0u, run, 31);
  }
  if (lane == 0) a.counts[e] = carry;
}

// Ranks inside the chunks become rows.
__global__ void __launch_bounds__(256) route_rows_many_kernel(RouteManyArgs a) {
  __shared__ int count[kRouteMaxE], offset[kRouteMaxE + 1];
  pdl_wait();
  for (int e = threadIdx.x; e < a.E; e += 256) count[e] = a.counts[e];
  __syncthreads();
  if (threadIdx.x < 32) scan_counts(count, offset, a.E);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= a.E; e += 256) a.offsets[e] = offset[e];
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, n = (int64_t)a.T * a.k;
  if (i >= n) return;
  const int e = a.idx[i];
  if (e >= 0) {
    const int t = (int)(i / a.k);
    const int r = a.row_of[i] + a.hist[(int64_t)e * a.chunks + t / kRouteTokens] + offset[e];
    a.row_of[i] = r;
    a.token_of_row[r] = t;
  }
  if (i >= offset[a.E]) a.token_of_row[i] = -1;
}

struct RouteBackArgs {
  const void* logits;
  int64_t ld, ldd;
  const int32_t* idx;
  const float* d_gate;
  void* d_logits;
  int T, E, k, softmax, renorm;
  float scale;
};

// d_logits of one token a warp.  With q_i = s_i / sum_j s_j over the chosen experts:
//   renormalised: softmax  d_l = scale q_i (g_i - sum q g)           (the softmax's own sum drops out)
//                 sigmoid  d_l = scale q_i (g_i - sum q g) (1 - s_i)
//   else:         softmax  d_l = scale s_e (g_e - sum s g), g_e = 0 where e was not chosen
//                 sigmoid  d_l = scale g_i s_i (1 - s_i)
template <typename L, int NS>
__global__ void __launch_bounds__(256) route_backward_kernel(RouteBackArgs a) {
  __shared__ float dense[8][NS * 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* mine = dense[warp];
  pdl_wait();
  for (int t = blockIdx.x * 8 + warp; t < a.T; t += gridDim.x * 8) {
    const L* row = static_cast<const L*>(a.logits) + t * a.ld;
    int e = -1;
    float g = 0.f, l = -INFINITY;
    if (lane < a.k) {
      e = a.idx[(int64_t)t * a.k + lane];
      if (e < 0 || e >= a.E) e = -1;
      if (e >= 0) {
        g = a.d_gate[(int64_t)t * a.k + lane];
        l = to_float(row[e]);
        if (!(l > -INFINITY)) e = -1, g = 0.f;  // masked: its score is 0 and stays it
      }
    }
    for (int i = lane; i < NS * 32; i += 32) mine[i] = 0.f;
    __syncwarp();
    float v[NS], common = 0.f;
    if (a.softmax) {
      float m = -INFINITY;
      if (a.renorm) {
        m = warp_max(e >= 0 ? l : -INFINITY);
        if (m < -350.f) {  // the row's largest may be 700 above (a row with logits above 350 is not looked for)
          float top = -INFINITY;
#pragma unroll 1
          for (int i = lane; i < a.E; i += 32) top = fmaxf(top, to_float(row[i]));
          if (l - warp_max(top) < -700.f) e = -1, g = 0.f;  // a score of zero, as the forward pass has it
        }
      } else {
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          v[j] = lane + 32 * j < a.E ? to_float(row[lane + 32 * j]) : -INFINITY;
          if (!(v[j] > -INFINITY)) v[j] = -INFINITY;
          m = fmaxf(m, v[j]);
        }
        m = warp_max(m);
      }
      float sum = 0.f;
      float s = e < 0 ? 0.f : (l == m ? 1.f : expf(l - m));
      if (a.renorm) {
        sum = s;
      } else {
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          v[j] = v[j] == -INFINITY ? 0.f : (v[j] == m ? 1.f : expf(v[j] - m));
          sum += v[j];
        }
      }
      sum = warp_sum(sum);
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      s *= inv;
      common = warp_sum(s * g);
      if (a.renorm) {
        if (e >= 0) mine[e] = a.scale * s * (g - common);
      } else {
        if (e >= 0) mine[e] = g;
#pragma unroll
        for (int j = 0; j < NS; ++j) v[j] *= inv;
      }
    } else if (e >= 0) {
      // s (1 - s) from exp(-|l|): no cancellation where s is near 1
      const float x = expf(-fabsf(l)), inv = 1.f / (1.f + x);
      const float small = x * inv, big = inv;  // the smaller and the larger of s and 1 - s
      v[0] = l >= 0.f ? big : small;           // s
      common = l >= 0.f ? small : big;         // 1 - s
    }
    if (!a.softmax) {
      if (a.renorm) {
        float s = e >= 0 ? v[0] : 0.f;
        if (__any_sync(~0u, e >= 0 && s < kTinyScore)) s = relative_score(e >= 0, l, 0.f, false);
        const float sum = warp_sum(s), q = sum > 0.f ? s / sum : 0.f;
        const float mean = warp_sum(q * g);
        if (e >= 0) mine[e] = a.scale * q * (g - mean) * common;
      } else if (e >= 0) {
        mine[e] = a.scale * g * v[0] * common;
      }
    }
    __syncwarp();
    const bool full = a.softmax && !a.renorm;
    L* out = static_cast<L*>(a.d_logits) + t * a.ldd;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const int i = lane + 32 * j;
      if (i < a.E) out[i] = from_float<L>(full ? a.scale * v[j] * (mine[i] - common) : mine[i]);
    }
    __syncwarp();
  }
}

// f(L{}, slots as a constant) by the logits' type and the experts' number.
template <typename F>
cudaError_t by_experts(int dtype, int E, F f) {
  auto with = [&](auto l) {
    if (E <= 32) return f(l, std::integral_constant<int, 1>{});
    if (E <= 64) return f(l, std::integral_constant<int, 2>{});
    if (E <= 128) return f(l, std::integral_constant<int, 4>{});
    if (E <= 256) return f(l, std::integral_constant<int, 8>{});
    return f(l, std::integral_constant<int, 16>{});
  };
  return dtype == COLIBRI_DTYPE_F32 ? with(float{}) : with(__nv_bfloat16{});
}

int check_route_config(const colibri_moe_route_config_t* c, int32_t T, int64_t ld) {
  if (!c || T < 0) return COLIBRI_ERR_INVALID_ARG;
  if (c->num_experts < 1 || c->top_k < 1 || c->top_k > c->num_experts || !ops_dtype(c->logits_dtype) ||
      (c->score != COLIBRI_SCORE_SOFTMAX && c->score != COLIBRI_SCORE_SIGMOID) || (c->renormalize & ~1) ||
      (c->trusted_pointers & ~1))
    return COLIBRI_ERR_INVALID_ARG;
  if (c->groups < 1 || c->num_experts % c->groups || c->top_groups < 1 || c->top_groups > c->groups ||
      c->group_top < 1 || c->group_top > 2 || c->top_k > c->top_groups * (c->num_experts / c->groups))
    return COLIBRI_ERR_INVALID_ARG;
  if (c->num_experts > kRouteMaxE || c->top_k > kRouteMaxK || c->groups > kRouteMaxGroups) return COLIBRI_ERR_UNSUPPORTED;
  if (ld < c->num_experts) return COLIBRI_ERR_INVALID_ARG;
  if ((int64_t)T * c->top_k > INT32_MAX) return COLIBRI_ERR_INVALID_ARG;
  if (T > kOpsMaxRows) return COLIBRI_ERR_UNSUPPORTED;
  return COLIBRI_OK;
}

int route_chunks(int T) { return (T + kRouteTokens - 1) / kRouteTokens; }

}  // namespace
}  // namespace colibri

using namespace colibri;

extern "C" int colibri_moe_route_experts_workspace(const colibri_moe_route_config_t* cfg, int32_t T, size_t* bytes) {
  if (!bytes) return COLIBRI_ERR_INVALID_ARG;
  const int rc = check_route_config(cfg, T, cfg ? cfg->num_experts : 0);
  if (rc) return rc;
  const int chunks = route_chunks(T);
  *bytes = chunks > 1 ? (size_t)chunks * cfg->num_experts * sizeof(int32_t) : 0;
  return COLIBRI_OK;
}

extern "C" int colibri_moe_route_experts(const colibri_moe_route_config_t* cfg, const void* logits, int64_t ld,
                                         const float* bias, int32_t T, int32_t* idx, float* gate, int32_t* counts,
                                         int32_t* offsets, int32_t* row_of, int32_t* token_of_row, void* workspace,
                                         size_t workspace_bytes, void* stream) {
  const int rc = check_route_config(cfg, T, ld);
  if (rc) return rc;
  if (!counts || !offsets || (T > 0 && (!logits || !idx || !gate || !row_of || !token_of_row)))
    return COLIBRI_ERR_INVALID_ARG;
  const int chunks = route_chunks(T);
  if (chunks > 1 && (!workspace || workspace_bytes < (size_t)chunks * cfg->num_experts * sizeof(int32_t)))
    return COLIBRI_ERR_INVALID_ARG;
  int device = 0, sms = 0;
  if (!ops_device(&device, &sms)) return COLIBRI_ERR_CUDA;
  for (const void* p : {logits, (const void*)bias, (const void*)idx, (const void*)gate, (const void*)counts,
                        (const void*)offsets, (const void*)row_of, (const void*)token_of_row,
                        (const void*)(chunks > 1 ? workspace : nullptr)})
    if (p && !cfg->trusted_pointers && !ops_on_device(p, device)) return COLIBRI_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int E = cfg->num_experts;
  if (T == 0) {
    if (cudaMemsetAsync(counts, 0, E * sizeof(int32_t), s) != cudaSuccess ||
        cudaMemsetAsync(offsets, 0, (E + 1) * sizeof(int32_t), s) != cudaSuccess) {
      cudaGetLastError();
      return COLIBRI_ERR_CUDA;
    }
    return COLIBRI_OK;
  }
  RouteManyArgs a = {};
  a.logits = logits, a.ld = ld, a.bias = bias, a.T = T, a.E = E, a.k = cfg->top_k, a.groups = cfg->groups;
  a.per_group = E / cfg->groups, a.top_groups = cfg->top_groups;
  a.group_top = std::min(cfg->group_top, a.per_group), a.softmax = cfg->score == COLIBRI_SCORE_SOFTMAX;
  a.renorm = cfg->renormalize, a.scale = cfg->scale, a.idx = idx, a.gate = gate, a.counts = counts;
  a.offsets = offsets, a.row_of = row_of, a.token_of_row = token_of_row, a.hist = static_cast<int32_t*>(workspace);
  a.chunks = chunks;
  a.aligned = ops_aligned16(logits) && ld * ops_elem(cfg->logits_dtype) % 16 == 0;
  cudaError_t e = by_experts(cfg->logits_dtype, E, [&](auto l, auto ns) {
    constexpr int NS = decltype(ns)::value;
    const int lanes = a.per_group / NS;
    a.lanes_per_group = a.per_group % NS == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
    return pdl_launch(route_tokens_kernel<decltype(l), decltype(ns)::value>, dim3(chunks),
                      dim3(32 * std::min(kRouteWarps, T)), 0, s, a);
  });
  if (e != cudaSuccess) return COLIBRI_ERR_CUDA;
  if (chunks > 1) {
    e = pdl_launch(route_scan_kernel, dim3((E + 7) / 8), dim3(256), 0, s, a);
    if (e != cudaSuccess) return COLIBRI_ERR_CUDA;
    e = pdl_launch(route_rows_many_kernel, dim3((unsigned)(((int64_t)T * a.k + 255) / 256)), dim3(256), 0, s, a);
    if (e != cudaSuccess) return COLIBRI_ERR_CUDA;
  }
  return COLIBRI_OK;
}

extern "C" int colibri_moe_route_experts_backward(const colibri_moe_route_config_t* cfg, const void* logits, int64_t ld,
                                                  const int32_t* idx, const float* d_gate, int32_t T, void* d_logits,
                                                  int64_t ld_d, void* stream) {
  const int rc = check_route_config(cfg, T, ld);
  if (rc) return rc;
  if (T == 0) return COLIBRI_OK;
  if (!logits || !idx || !d_gate || !d_logits || ld_d < cfg->num_experts) return COLIBRI_ERR_INVALID_ARG;
  int device = 0, sms = 0;
  if (!ops_device(&device, &sms)) return COLIBRI_ERR_CUDA;
  for (const void* p : {logits, (const void*)idx, (const void*)d_gate, (const void*)d_logits})
    if (!cfg->trusted_pointers && !ops_on_device(p, device)) return COLIBRI_ERR_INVALID_ARG;
  RouteBackArgs a = {logits, ld, ld_d, idx, d_gate, d_logits, T, cfg->num_experts, cfg->top_k,
                     cfg->score == COLIBRI_SCORE_SOFTMAX, cfg->renormalize, cfg->scale};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = by_experts(cfg->logits_dtype, cfg->num_experts, [&](auto l, auto ns) {
    return pdl_launch(route_backward_kernel<decltype(l), decltype(ns)::value>, dim3(std::min((T + 7) / 8, sms * 8)),
                      dim3(256), 0, s, a);
  });
  return e == cudaSuccess ? COLIBRI_OK : COLIBRI_ERR_CUDA;
}
