// expert_route.hip - routing of tokens to experts: scores, choice of k
// experts and their weights, the gradient of the weights, and the plan that
// sorts the (token, choice) slots by expert.
#include "mxg_internal.h"
#include "mxg_rows.h"

namespace mxg {
namespace {

constexpr int kRouteWaves = 4;  // tokens per workgroup
constexpr double kInf = __builtin_inf();
// Selection key of a NaN score: below every number, above the experts that
// cannot be chosen (-inf).
constexpr double kNanKey = -1.7976931348623157e308;

// Selection keys are formed in 64 bits: the order of two experts is the order
// of their scores also where those are closer than 32 bits resolve.  Without
// bias and group sums the key is the logit itself, of which both scores are
// increasing functions.
//
// Largest of the wave, lowest index among equals.
__device__ __forceinline__ void wave_best(double& key, int& idx) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const double ok = __shfl_xor(key, d);
    const int oi = __shfl_xor(idx, d);
    if (ok > key || (ok == key && oi < idx)) {
      key = ok;
      idx = oi;
    }
  }
}

// exp(l) scaled so that ratios of chosen scores survive where the scores
// themselves underflow: softmax exp(l - m), sigmoid exp(-m) / (1 + exp(-l)),
// m the largest chosen logit (sigmoid: at most 0).
__device__ __forceinline__ double chosen_score(int score, double l, double m) {
  if (score == kScoreSoftmax) return exp(l - m);
  return l < 0.0 ? exp(l - m) / (1.0 + exp(l)) : exp(-m) / (1.0 + exp(-l));
}

template <int IN, int VPL>
__global__ __launch_bounds__(kRouteWaves * 64) void route_kernel(RouteArgs a) {
  __shared__ double keys[kRouteWaves][VPL * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
  if (t >= a.T) return;
  const auto* row = reinterpret_cast<const typename RowElem<IN>::type*>(a.logits) + t * a.E;
  double key[VPL];
  float l[VPL];
  float m = -__builtin_inff();
  bool nan = false;
#pragma unroll
  for (int v = 0; v < VPL; v++) {
    const int e = v * 64 + lane;
    l[v] = e < a.E ? RowElem<IN>::get(row[e]) : -__builtin_inff();
    m = fmaxf(m, l[v]);
    nan |= l[v] != l[v];
  }
  m = wave_max(m);
  // a softmax with a NaN, or with an infinite largest logit, is NaN throughout
  const bool nan_row = a.score == kScoreSoftmax && (__any(nan) || m == __builtin_inff());
  double sum = 1.0;
  if (a.score == kScoreSoftmax && !nan_row) {
    sum = 0.0;
#pragma unroll
    for (int v = 0; v < VPL; v++)
      if (l[v] > -__builtin_inff()) sum += exp((double)l[v] - (double)m);
    sum = wave_sum(sum);
  }
  const bool by_logit = a.bias == nullptr && a.group_top == 1;
#pragma unroll
  for (int v = 0; v < VPL; v++) {
    const int e = v * 64 + lane;
    double c = (double)l[v];
    if (!by_logit) {
      c = a.score == kScoreSoftmax ? exp((double)l[v] - (double)m) / sum : 1.0 / (1.0 + exp(-(double)l[v]));
      if (a.bias != nullptr && e < a.E) c += (double)a.bias[e];
    }
    if (nan_row || c != c) c = kNanKey;
    if (l[v] == -__builtin_inff() || e >= a.E) c = -kInf;
    key[v] = c;
  }
  if (a.groups > 1) {
    // group scores: the sum of the group_top largest keys of each group, by
    // one lane per group; then the rank of each group among all
#pragma unroll
    for (int v = 0; v < VPL; v++) keys[wave][v * 64 + lane] = key[v];
    __builtin_amdgcn_wave_barrier();
    const int per = a.E / a.groups;
    double s = -kInf;
    if (lane < a.groups) {
      double first = -kInf, second = -kInf;
      for (int i = 0; i < per; i++) {
        const double c = keys[wave][lane * per + i];
        if (c > first) {
          second = first;
          first = c;
        } else if (c > second) {
          second = c;
        }
      }
      s = first;
      if (a.group_top == 2 && second > -kInf) s = fmax(first + second, kNanKey);
    }
    int rank = 0;
    for (int o = 0; o < a.groups; o++) {
      const double so = __shfl(s, o);
      rank += (so > s || (so == s && o < lane)) ? 1 : 0;
    }
    const uint64_t kept = __ballot(lane < a.groups && rank < a.top_groups);
#pragma unroll
    for (int v = 0; v < VPL; v++) {
      const int e = v * 64 + lane;
      if (e < a.E && !((kept >> (e / per)) & 1)) key[v] = -kInf;
    }
  }
  // k rounds: the best left of each lane, then of the wave; its owner drops it
  int my_id = -1;
  float my_l = 0.0f;
  for (int j = 0; j < a.k; j++) {
    double best = -kInf;
    int idx = 0x7fffffff;
#pragma unroll
    for (int v = 0; v < VPL; v++)
      if (key[v] > best) {
        best = key[v];
        idx = v * 64 + lane;
      }
    wave_best(best, idx);
    if (best == -kInf) break;  // wave-uniform: no expert is left
    float lj = 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; v++)
      if (idx == v * 64 + lane) {
        key[v] = -kInf;
        lj = l[v];
      }
    lj = __shfl(lj, idx & 63);
    if (lane == j) {
      my_id = idx;
      my_l = lj;
    }
  }
  // weights: lane j holds choice j
  const bool mine = my_id >= 0;
  double p = 0.0;
  if (a.renormalize) {
    float mc = wave_max(mine ? my_l : -__builtin_inff());
    if (a.score == kScoreSigmoid) mc = fminf(mc, 0.0f);
    if (mine) p = chosen_score(a.score, (double)my_l, (double)mc);
    p /= wave_sum(p);
  } else if (mine) {
    p = a.score == kScoreSoftmax ? exp((double)my_l - (double)m) / sum : 1.0 / (1.0 + exp(-(double)my_l));
  }
  if (lane < a.k) {
    a.ids[t * a.k + lane] = my_id;
    a.weights[t * a.k + lane] = mine ? (nan_row ? __builtin_nanf("") : (float)(p * (double)a.scale)) : 0.0f;
  }
}

// Gradient of the logits from that of the weights.  With c the chosen
// experts, p their scores and w = p / sum p where they are renormalized:
//   softmax, renormalized:  dl_c = scale w_c (dw_c - sum w dw)
//   sigmoid, renormalized:  dl_c = scale w_c (dw_c - sum w dw) (1 - p_c)
//   softmax:                dl_e = s_e (scale dw_e [chosen] - scale sum_c dw_c s_c)
//   sigmoid:                dl_c = scale dw_c p_c (1 - p_c)
// and zero elsewhere.  (The softmax's own sum cancels in w, so that case reads
// no more than the chosen logits.)
template <int IN, int VPL>
__global__ __launch_bounds__(kRouteWaves * 64) void route_backward_kernel(RouteArgs a, const float* __restrict__ d_w,
                                                                          void* __restrict__ d_logits) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
  if (t >= a.T) return;
  using E = RowElem<IN>;
  const auto* row = reinterpret_cast<const typename E::type*>(a.logits) + t * a.E;
  auto* out = reinterpret_cast<typename E::type*>(d_logits) + t * a.E;
  int id = lane < a.k ? a.ids[t * a.k + lane] : -1;
  if (id >= a.E) id = -1;
  const bool mine = id >= 0;
  const float lc = mine ? E::get(row[id]) : -__builtin_inff();
  const double dw = mine ? (double)a.scale * (double)d_w[t * a.k + lane] : 0.0;
  const bool softmax = a.score == kScoreSoftmax;
  double g = 0.0;  // what the chosen expert's logit gets of its own
  double dot = 0.0, sum = 1.0;
  float m = 0.0f;
  float l[VPL];
  if (a.renormalize) {
    float mc = wave_max(lc);
    if (!softmax) mc = fminf(mc, 0.0f);
    double w = mine ? chosen_score(a.score, (double)lc, (double)mc) : 0.0;
    const double total = wave_sum(w);
    if (mine) w /= total;
    g = w * (dw - wave_sum(w * dw));
    if (!softmax && mine) g *= 1.0 / (1.0 + exp((double)lc));
  } else if (softmax) {
    m = -__builtin_inff();
#pragma unroll
    for (int v = 0; v < VPL; v++) {
      const int e = v * 64 + lane;
      l[v] = e < a.E ? E::get(row[e]) : -__builtin_inff();
      m = fmaxf(m, l[v]);
    }
    m = wave_max(m);
    sum = 0.0;
#pragma unroll
    for (int v = 0; v < VPL; v++)
      if (!(l[v] == -__builtin_inff())) sum += exp((double)l[v] - (double)m);
    sum = wave_sum(sum);
    g = mine ? exp((double)lc - (double)m) / sum * dw : 0.0;
    dot = wave_sum(g);
  } else if (mine) {
    g = dw / ((1.0 + exp(-(double)lc)) * (1.0 + exp((double)lc)));
  }
  double acc[VPL];
#pragma unroll
  for (int v = 0; v < VPL; v++) {
    acc[v] = 0.0;
    if (!a.renormalize && softmax && !(l[v] == -__builtin_inff())) acc[v] = -dot * (exp((double)l[v] - (double)m) / sum);
  }
  for (int j = 0; j < a.k; j++) {
    const int idj = __shfl(id, j);
    const double gj = __shfl(g, j);
#pragma unroll
    for (int v = 0; v < VPL; v++)
      if (idj == v * 64 + lane) acc[v] += gj;
  }
#pragma unroll
  for (int v = 0; v < VPL; v++) {
    const int e = v * 64 + lane;
    if (e < a.E) out[e] = E::put((float)acc[v]);
  }
}

// ---- plan -------------------------------------------------------------------
//
// A stable counting sort of the slots by expert in one workgroup: each wave
// counts the experts of its own run of slots, the counts become first rows by
// a scan over experts and waves, and each wave then places its slots 64 at a
// time; within the 64 the lanes of one expert find each other by ballots over
// the bits of the expert's number.  Slots without an expert (id outside
// 0 .. E-1) count as expert E: they get position -1, and the entries of
// `order` behind the last expert's rows are -1.
constexpr int kPlanWaves = 16;
constexpr int kMaxExperts = 1024;

__device__ __forceinline__ int plan_expert(int id, int E) { return (id < 0 || id >= E) ? E : id; }

__global__ __launch_bounds__(kPlanWaves * 64) void plan_kernel(const int32_t* __restrict__ ids, int64_t n, int E,
                                                               int32_t* __restrict__ offsets,
                                                               int32_t* __restrict__ order,
                                                               int32_t* __restrict__ position) {
  __shared__ int count[kPlanWaves][kMaxExperts + 1];
  __shared__ int total[kMaxExperts + 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i < kPlanWaves * (kMaxExperts + 1); i += kPlanWaves * 64) (&count[0][0])[i] = 0;
  __syncthreads();
  const int64_t run = (((n + kPlanWaves - 1) / kPlanWaves) + 63) / 64 * 64;
  const int64_t lo = run * wave < n ? run * wave : n;
  const int64_t hi = lo + run < n ? lo + run : n;
  for (int64_t i = lo + lane; i < hi; i += 64) atomicAdd(&count[wave][plan_expert(ids[i], E)], 1);
  __syncthreads();
  for (int e = tid; e <= E; e += kPlanWaves * 64) {
    int s = 0;
    for (int w = 0; w < kPlanWaves; w++) {
      const int c = count[w][e];
      count[w][e] = s;
      s += c;
    }
    total[e] = s;
  }
  __syncthreads();
  if (wave == 0) {
    const int per = (E + 1 + 63) / 64;
    int s = 0;
    for (int i = 0; i < per; i++)
      if (lane * per + i <= E) s += total[lane * per + i];
    int before = s;
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(before, d);
      if (lane >= d) before += o;
    }
    before -= s;
    for (int i = 0; i < per; i++) {
      const int e = lane * per + i;
      if (e > E) break;
      const int c = total[e];
      total[e] = before;
      offsets[e] = before;  // offsets[E]: the slots with an expert
      before += c;
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
      const int p = total[e] + count[wave][e] + rank;
      order[p] = e < E ? (int32_t)i : -1;
      position[i] = e < E ? p : -1;
    }
    __builtin_amdgcn_wave_barrier();
    if (live && (same >> lane) == 1) count[wave][e] += __popcll(same);
    __builtin_amdgcn_wave_barrier();
  }
}

template <int IN, int VPL>
void route_vpl(const RouteArgs& a, const float* d_w, void* d_logits, hipStream_t stream) {
  const dim3 grid((unsigned)((a.T + kRouteWaves - 1) / kRouteWaves)), block(kRouteWaves * 64);
  if (d_logits != nullptr)
    hipLaunchKernelGGL((route_backward_kernel<IN, VPL>), grid, block, 0, stream, a, d_w, d_logits);
  else
    hipLaunchKernelGGL((route_kernel<IN, VPL>), grid, block, 0, stream, a);
}

template <int IN>
void route_in(const RouteArgs& a, const float* d_w, void* d_logits, hipStream_t stream) {
  if (a.E <= 64)
    route_vpl<IN, 1>(a, d_w, d_logits, stream);
  else if (a.E <= 128)
    route_vpl<IN, 2>(a, d_w, d_logits, stream);
  else if (a.E <= 256)
    route_vpl<IN, 4>(a, d_w, d_logits, stream);
  else if (a.E <= 512)
    route_vpl<IN, 8>(a, d_w, d_logits, stream);
  else
    route_vpl<IN, 16>(a, d_w, d_logits, stream);
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
  (void)n;
  (void)E;
  return 0;
}

hipError_t launch_plan(const int32_t* ids, int64_t n, int E, int32_t* offsets, int32_t* order, int32_t* position,
                       void* workspace, hipStream_t stream) {
  (void)workspace;
  hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(kPlanWaves * 64), 0, stream, ids, n, E, offsets, order, position);
  return hipGetLastError();
}

}  // namespace mxg
