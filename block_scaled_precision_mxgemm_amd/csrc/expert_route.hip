// expert_route.hip - routing of tokens to experts: scores, choice of k
// experts and their weights, the gradient of the weights, and the plan that
// sorts the (token, choice) slots by expert.
#include "mxg_internal.h"
#include "mxg_rows.h"

namespace mxg {
namespace {

constexpr int kRouteWaves = 4;  // per workgroup
constexpr double kInf = __builtin_inf();
constexpr double kMaxKey = 1.7976931348623157e308;
// Selection key of a NaN score: below every number, above the experts that
// cannot be chosen (-inf, and -kMaxKey once the keys are packed).
constexpr double kNanKey = -0x1p1023;

// L lanes work on a token, each on VPL experts in a row: a wave takes 4 tokens
// with up to 256 experts, one with more.  Most of the work is instructions on
// whole waves (the logits are few bytes), and with a token per wave each
// reduction would take the same instructions for a quarter of the tokens.
//
// Selection keys are doubles that carry the expert's number in their last 10
// bits, so that one v_max_f64 a step finds the largest score and, among equal
// ones, the lowest expert.  Scores whose first 42 bits agree count as equal.
// Without bias and group sums the key is the logit itself, of which both
// scores are increasing functions (an fp32 value leaves those bits free, so
// its order is exact); else it is formed in 64 bits: in 32 bits, scores that
// differ would tie.
__device__ __forceinline__ double pack_key(double x, int e) {
  x = fmin(x + 0.0, kMaxKey);  // one zero, no infinity
  const uint64_t u = (uint64_t)__double_as_longlong(x) & ~(uint64_t)1023;
  return __longlong_as_double((long long)(u | (uint64_t)((int64_t)u < 0 ? e : 1023 - e)));
}
__device__ __forceinline__ int key_expert(double key) {
  const long long u = __double_as_longlong(key);
  const int e = (int)(u & 1023);
  return u < 0 ? e : 1023 - e;
}

// Value of lane i ^ D's, or another of the same L lanes, such that log2(L) such
// steps reach all of them: rotations by DPP within rows of 16, then shuffles.
template <int D>
__device__ __forceinline__ int lane_step(int x) {
  if constexpr (D <= 8)
    return __builtin_amdgcn_mov_dpp(x, 0x120 + D, 0xf, 0xf, true);  // row_ror:D
  else
    return __shfl_xor(x, D);
}
template <int D>
__device__ __forceinline__ float lane_step(float x) {
  return __int_as_float(lane_step<D>(__float_as_int(x)));
}
template <int D>
__device__ __forceinline__ double lane_step(double x) {
  return __hiloint2double(lane_step<D>(__double2hiint(x)), lane_step<D>(__double2loint(x)));
}
// fmax of values that are not NaN.  For doubles it is the instruction itself:
// fmax first quiets both operands, which triples its cost.  The s_nop is the
// wait of a DPP move that may read the result next.
__device__ __forceinline__ float larger(float x, float y) { return fmaxf(x, y); }
__device__ __forceinline__ double larger(double x, double y) {
  double r;
  asm("v_max_f64 %0, %1, %2\n\ts_nop 1" : "=v"(r) : "v"(x), "v"(y));
  return r;
}
template <int L, class V>
__device__ __forceinline__ V lanes_max(V x) {
  if constexpr (L > 32) x = larger(x, lane_step<32>(x));
  if constexpr (L > 16) x = larger(x, lane_step<16>(x));
  x = larger(x, lane_step<8>(x));
  x = larger(x, lane_step<4>(x));
  x = larger(x, lane_step<2>(x));
  return larger(x, lane_step<1>(x));
}
template <int L, class V>
__device__ __forceinline__ V lanes_sum(V x) {
  if constexpr (L > 32) x += lane_step<32>(x);
  if constexpr (L > 16) x += lane_step<16>(x);
  x += lane_step<8>(x);
  x += lane_step<4>(x);
  x += lane_step<2>(x);
  return x + lane_step<1>(x);
}

// The lane's VPL logits from expert e0 on; -inf past the last.  `vec`: rows
// are whole numbers of the pieces loaded, and aligned to them.
template <int IN, int VPL>
__device__ __forceinline__ void load_logits(const typename RowElem<IN>::type* row, int e0, int E, bool vec,
                                            float (&l)[VPL]) {
  using R = RowElem<IN>;
  constexpr int P = R::VEC < VPL ? R::VEC : VPL;  // elements of a piece: 8 or 16 bytes
  if (vec && e0 < E) {
#pragma unroll
    for (int v = 0; v < VPL; v += P) {
      typename R::type x[P];
      if constexpr (sizeof(x) == 16)
        *reinterpret_cast<v4i*>(x) = *reinterpret_cast<const v4i*>(row + e0 + v);
      else
        *reinterpret_cast<v2i*>(x) = *reinterpret_cast<const v2i*>(row + e0 + v);
#pragma unroll
      for (int i = 0; i < P; i++) l[v + i] = R::get(x[i]);
    }
  } else {
#pragma unroll
    for (int v = 0; v < VPL; v++) l[v] = e0 + v < E ? R::get(row[e0 + v]) : -__builtin_inff();
  }
}
template <int IN, int VPL>
bool vector_rows(const void* p, int E) {
  using R = RowElem<IN>;
  constexpr int piece = (R::VEC < VPL ? R::VEC : VPL) * (int)sizeof(typename R::type);
  return E % VPL == 0 && (uintptr_t)p % piece == 0 && E * sizeof(typename R::type) % piece == 0;
}

// exp(l) scaled so that ratios of chosen scores survive where the scores
// themselves underflow: softmax exp(l - m), sigmoid exp(-m) / (1 + exp(-l)),
// m the largest chosen logit (sigmoid: at most 0).
__device__ __forceinline__ double chosen_score(int score, double l, double m) {
  if (score == kScoreSoftmax) return exp(l - m);
  return l < 0.0 ? exp(l - m) / (1.0 + exp(l)) : exp(-m) / (1.0 + exp(-l));
}

// `first` and `second` become the two largest of themselves and c.
__device__ __forceinline__ void two_largest(double& first, double& second, double c) {
  second = fmax(second, fmin(first, c));
  first = fmax(first, c);
}

// 1 / x for 1 <= x <= 2^1020: the hardware's estimate and two Newton steps,
// good to a few units in the last place.
__device__ __forceinline__ double reciprocal(double x) {
  double r = __builtin_amdgcn_rcp(x);
  r = fma(fma(-x, r, 1.0), r, r);
  return fma(fma(-x, r, 1.0), r, r);
}

// The same in fp32, for the weights (each exponential is off by a few roundings
// and one for each unit of its argument).
__device__ __forceinline__ float chosen_score32(int score, float l, float m) {
  if (score == kScoreSoftmax) return __expf(l - m);
  return l < 0.0f ? __expf(l - m) / (1.0f + __expf(l)) : __expf(-m) / (1.0f + __expf(-l));
}

// Choices of a token, L a round.
template <int L>
constexpr int kRounds = (64 + L - 1) / L;

template <int IN, int L, int VPL>
__global__ __launch_bounds__(kRouteWaves * 64) void route_kernel(RouteArgs a, bool vec) {
  constexpr int TPW = 64 / L;
  __shared__ double keys[kRouteWaves * TPW][L * VPL];
  __shared__ double group_key[kRouteWaves * TPW][64];
  __shared__ int chosen[kRouteWaves * TPW][64];
  const int lane = threadIdx.x & (L - 1), tok = threadIdx.x / L;
  const int64_t t0 = (int64_t)blockIdx.x * kRouteWaves * TPW + tok;
  const bool live = t0 < a.T;
  const int64_t t = live ? t0 : a.T - 1;  // lanes without a token repeat the last
  const auto* row = reinterpret_cast<const typename RowElem<IN>::type*>(a.logits) + t * a.E;
  const int e0 = lane * VPL;
  const bool softmax = a.score == kScoreSoftmax;
  float l[VPL];
  load_logits<IN, VPL>(row, e0, a.E, vec, l);
  float m = -__builtin_inff();
  float bad = 0.0f;
#pragma unroll
  for (int v = 0; v < VPL; v++) {
    m = fmaxf(m, l[v]);
    if (l[v] != l[v]) bad = 1.0f;
  }
  m = lanes_max<L>(m);
  // a softmax with a NaN, or with an infinite largest logit, is NaN throughout
  const bool nan_row = softmax && (lanes_max<L>(bad) > 0.0f || m == __builtin_inff());
  const bool by_logit = a.bias == nullptr && (a.group_top == 1 || a.groups == 1);
  double key[VPL];
  double sum = 1.0;
  if (by_logit) {
    if (softmax && !a.renormalize) {
      // the weights alone need the sum: in fp32, off by a rounding for each of
      // a lane's terms and a few for each exponential
      float f = 0.0f;
#pragma unroll
      for (int v = 0; v < VPL; v++) f += l[v] > -__builtin_inff() ? __expf(l[v] - m) : 0.0f;
      sum = (double)lanes_sum<L>(f);
    }
#pragma unroll
    for (int v = 0; v < VPL; v++) key[v] = (double)l[v];
  } else if (softmax) {
    sum = 0.0;
#pragma unroll
    for (int v = 0; v < VPL; v++) {
      key[v] = l[v] > -__builtin_inff() ? exp((double)l[v] - (double)m) : 0.0;
      sum += key[v];
    }
    sum = lanes_sum<L>(sum);
    const double inv = 1.0 / sum;
#pragma unroll
    for (int v = 0; v < VPL; v++) key[v] *= inv;
  } else {
#pragma unroll
    for (int v = 0; v < VPL; v++) {
      // below l = -707 all scores are taken as 2^-1020 (which a double has no
      // room to tell apart much further)
      key[v] = reciprocal(1.0 + fmin(exp(-(double)l[v]), 0x1p1020));
    }
  }
#pragma unroll
  for (int v = 0; v < VPL; v++) {
    if (a.bias != nullptr && e0 + v < a.E) key[v] += (double)a.bias[e0 + v];
    if (nan_row || l[v] != l[v] || key[v] != key[v]) key[v] = kNanKey;
    if (l[v] == -__builtin_inff()) key[v] = -kInf;
  }
  if (a.groups > 1) {
    // group scores: the sum of the group_top largest keys of each group, a
    // lane for each; then the rank of each group among all
    const int per = a.E / a.groups;
    const bool whole = per % VPL == 0;  // a lane's experts are of one group
    if (whole) {
      // the two largest of each lane, then of the group's lanes
      double first = -kInf, second = -kInf;
#pragma unroll
      for (int v = 0; v < VPL; v++) two_largest(first, second, key[v]);
      keys[tok][2 * lane] = first;
      keys[tok][2 * lane + 1] = second;
    } else {
#pragma unroll
      for (int v = 0; v < VPL; v++) keys[tok][e0 + v] = key[v];
    }
    wave_sync();
    const int n = whole ? per / VPL * 2 : per;
    for (int i = lane; i < a.groups; i += L) {
      double first = -kInf, second = -kInf;
      for (int e = i * n; e < (i + 1) * n; e++) two_largest(first, second, keys[tok][e]);
      group_key[tok][i] = a.group_top == 2 && second > -kInf ? fmax(first + second, -kMaxKey) : first;
    }
    wave_sync();
    int i = e0 / per, in = e0 - i * per;  // group of expert e0 + v, and its place there
    bool out = false;
#pragma unroll
    for (int v = 0; v < VPL; v++) {
      if (e0 + v < a.E && (v == 0 || in == 0)) {
        const double mine = group_key[tok][i];
        int rank = 0;
        for (int o = 0; o < a.groups; o++) {
          const double other = group_key[tok][o];
          rank += (other > mine || (other == mine && o < i)) ? 1 : 0;
        }
        out = rank >= a.top_groups;
      }
      if (out) key[v] = -kInf;
      if (++in == per) {
        in = 0;
        i++;
      }
    }
  }
#pragma unroll
  for (int v = 0; v < VPL; v++) key[v] = key[v] > -kInf ? pack_key(key[v], e0 + v) : -kMaxKey;
  // k rounds: the best left of each lane, then of all; its owner drops it (the
  // high word alone makes it less than every key)
  for (int j = 0; j < a.k; j++) {
    double best = key[0];
#pragma unroll
    for (int v = 1; v < VPL; v++) best = larger(best, key[v]);
    best = lanes_max<L>(best);
    const int e = best > -0x1.8p1023 ? key_expert(best) : -1;
    if (lane == 0) chosen[tok][j] = e;
#pragma unroll
    for (int v = 0; v < VPL; v++) {
      const int hi = __double2hiint(key[v]);
      key[v] = __hiloint2double(e == e0 + v ? (int)0xFFEFFFFF : hi, __double2loint(key[v]));
    }
  }
  wave_sync();
  // weights: a lane takes choices lane, lane + L, ...
  float p[kRounds<L>], total = 0.0f;
  int id[kRounds<L>];
  float lc[kRounds<L>], mc = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < kRounds<L>; i++) {
    const int j = lane + i * L;
    id[i] = j < a.k ? chosen[tok][j] : -1;
    lc[i] = id[i] >= 0 ? RowElem<IN>::get(row[id[i]]) : -__builtin_inff();
    mc = fmaxf(mc, lc[i]);
  }
  mc = a.renormalize ? lanes_max<L>(mc) : softmax ? m : 0.0f;
  if (!softmax) mc = fminf(mc, 0.0f);
#pragma unroll
  for (int i = 0; i < kRounds<L>; i++) {
    p[i] = 0.0f;
    if (i * L < a.k && id[i] >= 0) {
      p[i] = chosen_score32(a.score, lc[i], mc);
      total += p[i];
    }
  }
  const float f = a.scale / (a.renormalize ? lanes_sum<L>(total) : softmax ? (float)sum : 1.0f);
#pragma unroll
  for (int i = 0; i < kRounds<L>; i++) {
    const int j = lane + i * L;
    if (live && j < a.k) {
      a.ids[t * a.k + j] = id[i];
      a.weights[t * a.k + j] = id[i] >= 0 ? (nan_row ? __builtin_nanf("") : p[i] * f) : 0.0f;
    }
  }
}

// Gradient of the logits from that of the weights.  With c the chosen
// experts, p their scores and w = p / sum p where they are renormalized:
//   softmax, renormalized:  dl_c = scale w_c (dw_c - sum w dw)
//   sigmoid, renormalized:  dl_c = scale w_c (dw_c - sum w dw) (1 - p_c)
//   softmax:                dl_e = scale s_e (D_e - sum_f s_f D_f), D_e the sum of e's dw
//   sigmoid:                dl_c = scale dw_c p_c (1 - p_c)
// and zero elsewhere.  The softmax's own sum cancels in w, so that only the
// third reads more than the chosen logits.  The few chosen terms are formed in
// 64 bits, the third's row in 32.  In the sums all dw (D) are taken less that of
// the largest logit, which changes nothing, as the weights add up to one.  Where
// that choice has nearly all of the sum its dw would cancel against the sum's,
// and no type's digits hold the rest for every lead; so its own difference
// is zero, and the sum holds what the other choices add (a single choice has a
// constant weight: its gradient is exactly zero).
template <int IN, int L, int VPL>
__global__ __launch_bounds__(kRouteWaves * 64) void route_backward_kernel(RouteArgs a, const float* __restrict__ d_w,
                                                                          void* __restrict__ d_logits, bool vec) {
  constexpr int TPW = 64 / L;
  using R = RowElem<IN>;
  __shared__ int chosen[kRouteWaves * TPW][64];
  __shared__ float grad[kRouteWaves * TPW][64];
  const int lane = threadIdx.x & (L - 1), tok = threadIdx.x / L;
  const int64_t t0 = (int64_t)blockIdx.x * kRouteWaves * TPW + tok;
  const bool live = t0 < a.T;
  const int64_t t = live ? t0 : a.T - 1;
  const auto* row = reinterpret_cast<const typename R::type*>(a.logits) + t * a.E;
  const int e0 = lane * VPL;
  const bool softmax = a.score == kScoreSoftmax;
  int id[kRounds<L>];
  float lc[kRounds<L>], given[kRounds<L>], mc = -__builtin_inff();
  double g[kRounds<L>];
#pragma unroll
  for (int i = 0; i < kRounds<L>; i++) {
    const int j = lane + i * L;
    id[i] = j < a.k ? a.ids[t * a.k + j] : -1;
    if (id[i] >= a.E) id[i] = -1;
    const bool mine = id[i] >= 0;
    lc[i] = mine ? R::get(row[id[i]]) : -__builtin_inff();
    given[i] = mine ? d_w[t * a.k + j] : 0.0f;
    mc = fmaxf(mc, lc[i]);
  }
  float s[VPL];
  float sum = 1.0f;
  double dot = 0.0, total = 0.0;
  if (a.renormalize) {
    mc = lanes_max<L>(mc);
    float top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < kRounds<L>; i++) top = id[i] >= 0 && lc[i] == mc ? fmaxf(top, given[i]) : top;
    top = lanes_max<L>(top);
    if (!softmax) mc = fminf(mc, 0.0f);
    double w[kRounds<L>], dw[kRounds<L>];
#pragma unroll
    for (int i = 0; i < kRounds<L>; i++) {
      w[i] = 0.0;
      if (i * L < a.k && id[i] >= 0) {
        w[i] = chosen_score(a.score, (double)lc[i], (double)mc);
        dw[i] = (double)a.scale * ((double)given[i] - (double)top);
        total += w[i];
        dot += w[i] * dw[i];
      }
    }
    total = lanes_sum<L>(total);
    dot = lanes_sum<L>(dot);
    const double inv = 1.0 / total;
    dot *= inv;
#pragma unroll
    for (int i = 0; i < kRounds<L>; i++) {
      g[i] = 0.0;
      if (i * L < a.k && id[i] >= 0) {
        g[i] = w[i] * inv * (dw[i] - dot);
        if (!softmax) g[i] *= 1.0 / (1.0 + exp((double)lc[i]));
      }
    }
  } else if (softmax) {
    load_logits<IN, VPL>(row, e0, a.E, vec, s);
    float m = -__builtin_inff();
#pragma unroll
    for (int v = 0; v < VPL; v++) m = fmaxf(m, s[v]);
    m = lanes_max<L>(m);
    sum = 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; v++) {
      s[v] = s[v] == -__builtin_inff() ? 0.0f : __expf(s[v] - m);
      sum += s[v];
    }
    sum = lanes_sum<L>(sum);
#pragma unroll
    for (int i = 0; i < kRounds<L>; i++) g[i] = (double)given[i];  // the scale comes last
  } else {
#pragma unroll
    for (int i = 0; i < kRounds<L>; i++)
      g[i] = i * L < a.k && id[i] >= 0
                 ? (double)a.scale * (double)given[i] / ((1.0 + exp(-(double)lc[i])) * (1.0 + exp((double)lc[i])))
                 : 0.0;
  }
#pragma unroll
  for (int i = 0; i < kRounds<L>; i++) {
    const int j = lane + i * L;
    if (j < a.k) {
      chosen[tok][j] = id[i];
      grad[tok][j] = (float)g[i];
    }
  }
  wave_sync();
  float acc[VPL] = {};
  for (int j = 0; j < a.k; j++) {
    const int at = chosen[tok][j] - e0;
    const float gj = grad[tok][j];
#pragma unroll
    for (int v = 0; v < VPL; v++)
      if (at == v) acc[v] += gj;
  }
  if (!a.renormalize && softmax) {
    // the D of a largest logit (exp(0) is one; of equal logits any will do)
    float top = -__builtin_inff(), rest = 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; v++) top = s[v] == 1.0f ? fmaxf(top, acc[v]) : top;
    top = lanes_max<L>(top);
#pragma unroll
    for (int v = 0; v < VPL; v++) rest = fmaf(s[v], acc[v] - top, rest);
    const float inv = 1.0f / sum, f = a.scale * inv;
    rest = lanes_sum<L>(rest) * inv;
    // a NaN among the logits is one in every term (the sum is NaN), but experts
    // without a score have no gradient
#pragma unroll
    for (int v = 0; v < VPL; v++)
      acc[v] = s[v] == 0.0f ? 0.0f : s[v] * f * ((acc[v] - top) - rest);
  }
  if (!live) return;
  auto* out = reinterpret_cast<typename R::type*>(d_logits) + t * a.E;
  constexpr int P = R::VEC < VPL ? R::VEC : VPL;
  if (vec && e0 < a.E) {
#pragma unroll
    for (int v = 0; v < VPL; v += P) {
      typename R::type x[P];
#pragma unroll
      for (int i = 0; i < P; i++) x[i] = R::put(acc[v + i]);
      if constexpr (sizeof(x) == 16)
        *reinterpret_cast<v4i*>(out + e0 + v) = *reinterpret_cast<v4i*>(x);
      else
        *reinterpret_cast<v2i*>(out + e0 + v) = *reinterpret_cast<v2i*>(x);
    }
  } else {
#pragma unroll
    for (int v = 0; v < VPL; v++)
      if (e0 + v < a.E) out[e0 + v] = R::put(acc[v]);
  }
}

// ---- plan -------------------------------------------------------------------
//
// A stable counting sort of the slots by expert.  Up to kPlanRun slots one
// workgroup does it; above, runs of slots (at most kPlanRuns of them) have one
// each, and a first kernel leaves every run's counts in the workspace, from
// which each workgroup of the second adds up its first rows.  In a workgroup
// each wave counts the experts of its part of the run, the counts become first
// rows by a scan over experts and waves, and each wave then places its slots 64
// at a time; within the 64 the lanes of one expert find each other by ballots
// over the bits of the expert's number.  Slots without an expert (id outside
// 0 .. E-1) count as expert E: they get position -1, and the entries of `order`
// behind the last expert's rows are -1.
constexpr int kPlanWaves = 16;
constexpr int kPlanThreads = kPlanWaves * 64;
constexpr int kMaxExperts = 1024;
// One workgroup alone takes 7.4 us for 4096 slots of 128 experts and 1.1 us for
// each 1000 more (131072: 150); the two kernels 7 us for 6000, 10.3 for
// 131072 and 22 for 2^20.
constexpr int64_t kPlanRun = 4096;
constexpr int64_t kPlanRuns = 256;

__device__ __forceinline__ int plan_expert(int id, int E) { return (id < 0 || id >= E) ? E : id; }

// slots of a run: whole groups of 64 for every wave
inline int64_t plan_run(int64_t n) {
  if (n <= kPlanRun) return kPlanRun;
  const int64_t run = (n + kPlanRuns - 1) / kPlanRuns;
  return run < 2048 ? 2048 : (run + kPlanThreads - 1) / kPlanThreads * kPlanThreads;
}

__global__ __launch_bounds__(kPlanThreads) void plan_count_kernel(const int32_t* __restrict__ ids, int64_t n, int E,
                                                                  int64_t run, int* __restrict__ counts) {
  __shared__ int count[kMaxExperts + 1];
  for (int e = threadIdx.x; e <= E; e += kPlanThreads) count[e] = 0;
  __syncthreads();
  const int64_t lo = run * blockIdx.x, hi = lo + run < n ? lo + run : n;
  for (int64_t i = lo + threadIdx.x; i < hi; i += kPlanThreads) atomicAdd(&count[plan_expert(ids[i], E)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += kPlanThreads) counts[(int64_t)blockIdx.x * (E + 1) + e] = count[e];
}

__global__ __launch_bounds__(kPlanThreads) void plan_kernel(const int32_t* __restrict__ ids, int64_t n, int E,
                                                            int64_t run, const int* __restrict__ counts,
                                                            int32_t* __restrict__ offsets, int32_t* __restrict__ order,
                                                            int32_t* __restrict__ position) {
  __shared__ int count[kPlanWaves * (kMaxExperts + 1)];
  __shared__ int total[kMaxExperts + 1], before[kMaxExperts + 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int E1 = E + 1, runs = gridDim.x;
  for (int i = tid; i < kPlanWaves * E1; i += kPlanThreads) count[i] = 0;
  for (int e = tid; e < E1; e += kPlanThreads) total[e] = before[e] = 0;
  __syncthreads();
  const int64_t first = run * blockIdx.x, last = first + run < n ? first + run : n;
  const int64_t part = run / kPlanWaves;  // a multiple of 64
  const int64_t lo = first + part * wave < last ? first + part * wave : last;
  const int64_t hi = lo + part < last ? lo + part : last;
  int* mine = count + wave * E1;
  for (int64_t i = lo + lane; i < hi; i += 64) atomicAdd(&mine[plan_expert(ids[i], E)], 1);
  if (runs > 1) {
    // all runs' counts, and those of the runs before this one
    const int groups = kPlanThreads / E1 > 0 ? kPlanThreads / E1 : 1;
    for (int i = tid; i < groups * E1; i += kPlanThreads) {
      const int e = i % E1;
      // 8 runs' counts are loaded at a time
      int all = 0, ahead = 0;
      for (int b0 = i / E1; b0 < runs; b0 += 8 * groups) {
        int c[8];
#pragma unroll
        for (int u = 0; u < 8; u++) {
          const int b = b0 + u * groups;
          c[u] = b < runs ? counts[(int64_t)b * E1 + e] : 0;
        }
#pragma unroll
        for (int u = 0; u < 8; u++) {
          all += c[u];
          ahead += b0 + u * groups < (int)blockIdx.x ? c[u] : 0;
        }
      }
      atomicAdd(&total[e], all);
      atomicAdd(&before[e], ahead);
    }
  }
  __syncthreads();
  for (int e = tid; e < E1; e += kPlanThreads) {
    int s = 0;
    for (int w = 0; w < kPlanWaves; w++) {
      const int c = count[w * E1 + e];
      count[w * E1 + e] = s;
      s += c;
    }
    if (runs == 1) total[e] = s;
  }
  __syncthreads();
  if (wave == 0) {
    const int per = (E1 + 63) / 64;
    int s = 0;
    for (int i = 0; i < per; i++)
      if (lane * per + i < E1) s += total[lane * per + i];
    int at = wave_scan<false>(s);
    at -= s;
    for (int i = 0; i < per; i++) {
      const int e = lane * per + i;
      if (e >= E1) break;
      const int c = total[e];
      if (blockIdx.x == 0) offsets[e] = at;  // offsets[E]: the slots with an expert
      before[e] += at;
      at += c;
    }
  }
  __syncthreads();
  const int bits = 32 - __clz(E);
  for (int64_t i0 = lo; i0 < hi; i0 += 64) {
    const int64_t i = i0 + lane;
    const bool live = i < hi;
    const int e = live ? plan_expert(ids[i], E) : 0;
    uint64_t same = __ballot(live);
    for (int b = 0; b < bits; b++) {
      const uint64_t set = __ballot((e >> b) & 1);
      same &= ((e >> b) & 1) ? set : ~set;
    }
    if (live) {
      const int rank = __popcll(same & (((uint64_t)1 << lane) - 1));
      const int p = before[e] + mine[e] + rank;
      order[p] = e < E ? (int32_t)i : -1;
      position[i] = e < E ? p : -1;
    }
    wave_sync();
    if (live && (same >> lane) == 1) mine[e] += __popcll(same);
    wave_sync();
  }
}

template <int IN, int L, int VPL>
void route_lanes(const RouteArgs& a, const float* d_w, void* d_logits, hipStream_t stream) {
  constexpr int per = kRouteWaves * (64 / L);  // tokens of a workgroup
  const dim3 grid((unsigned)((a.T + per - 1) / per)), block(kRouteWaves * 64);
  const bool vec = vector_rows<IN, VPL>(a.logits, a.E) && (d_logits == nullptr || vector_rows<IN, VPL>(d_logits, a.E));
  if (d_logits != nullptr)
    hipLaunchKernelGGL((route_backward_kernel<IN, L, VPL>), grid, block, 0, stream, a, d_w, d_logits, vec);
  else
    hipLaunchKernelGGL((route_kernel<IN, L, VPL>), grid, block, 0, stream, a, vec);
}

template <int IN>
void route_in(const RouteArgs& a, const float* d_w, void* d_logits, hipStream_t stream) {
  if (a.E <= 64)
    route_lanes<IN, 16, 4>(a, d_w, d_logits, stream);
  else if (a.E <= 128)
    route_lanes<IN, 16, 8>(a, d_w, d_logits, stream);
  else if (a.E <= 256)
    route_lanes<IN, 16, 16>(a, d_w, d_logits, stream);
  else if (a.E <= 512)
    route_lanes<IN, 64, 8>(a, d_w, d_logits, stream);
  else
    route_lanes<IN, 64, 16>(a, d_w, d_logits, stream);
}

hipError_t route_type(const RouteArgs& a, int in_type, const float* d_w, void* d_logits, hipStream_t stream) {
  switch (in_type) {
    case kOutF32:
      route_in<kOutF32>(a, d_w, d_logits, stream);
      break;
    case kOutBF16:
      route_in<kOutBF16>(a, d_w, d_logits, stream);
      break;
    default:
      route_in<kOutF16>(a, d_w, d_logits, stream);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, int in_type, hipStream_t stream) {
  return route_type(a, in_type, nullptr, nullptr, stream);
}

hipError_t launch_route_backward(const RouteArgs& a, int in_type, const float* d_w, void* d_logits,
                                 hipStream_t stream) {
  return route_type(a, in_type, d_w, d_logits, stream);
}

int64_t plan_workspace(int64_t n, int E) {
  const int64_t run = plan_run(n);
  return n <= run ? 0 : (n + run - 1) / run * (E + 1) * (int64_t)sizeof(int);
}

hipError_t launch_plan(const int32_t* ids, int64_t n, int E, int32_t* offsets, int32_t* order, int32_t* position,
                       void* workspace, hipStream_t stream) {
  const int64_t run = plan_run(n);
  const dim3 grid((unsigned)((n + run - 1) / run)), block(kPlanThreads);
  int* counts = (int*)workspace;
  if (grid.x > 1) hipLaunchKernelGGL(plan_count_kernel, grid, block, 0, stream, ids, n, E, run, counts);
  hipLaunchKernelGGL(plan_kernel, grid, block, 0, stream, ids, n, E, run, counts, offsets, order, position);
  return hipGetLastError();
}

}  // namespace mxg
