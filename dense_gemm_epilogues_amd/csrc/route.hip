// Routing of tokens to experts: each token's best experts by its router logits, and their weights, with gradients.
//
//   score s = softmax or sigmoid of a token's logits; key = the logit, or with a bias or groups s + bias in double;
//   groups: the topk_groups groups with the greatest sum of their group_top highest keys stay;
//   ids = the topk highest keys in falling order, the lowest index first among equal ones;
//   weights = scale s_id (renormalised: scale s_id / sum of the chosen s).
//
// Keys are in double because they decide between neighbours: a fp32 sigmoid gives different logits equal keys.  A logit
// of -infinity or NaN, or such a key, takes its expert out; a token with fewer than topk left has ids of -1 with weight 0.
//
// A wave takes a token, a lane VPL neighbouring experts, which stay in registers; a choice is one maximum over the
// wave's lanes, whose best ones stand ready.
#include "block_ops.hpp"
#include "fp8_device.hpp"

namespace ep {
namespace {

constexpr int kWaves = 4;  // tokens a workgroup

__device__ __forceinline__ double inf64() { return __builtin_inf(); }

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v = __builtin_fmax(v, __shfl_xor(v, d));
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
template <class T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  return v;
}

// A lane's logits (experts lane VPL .. + VPL - 1); -infinity for NaN and past the last expert.
template <int E, int VPL>
__device__ __forceinline__ void load_logits(const void* base, int64_t at, int first, int experts, float* l) {
  const char* p = (const char*)base + (at + first) * elt_size(E);
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    l[i] = first + i < experts ? load_elt<E>(p + i * elt_size(E)) : -__builtin_inff();
    if (l[i] != l[i]) l[i] = -__builtin_inff();
  }
}

// e^(l - m), 1 where both are the same infinity
__device__ __forceinline__ double exp_below(float l, float m) { return l == m ? 1.0 : exp((double)l - (double)m); }

// 1 / (1 + e^-l)
__device__ __forceinline__ double sigmoid64(float l) { return 1.0 / (1.0 + exp(-(double)l)); }

// The wave's greatest key, and which lane has it first; keys are a lane's best ones.
template <class K>
__device__ __forceinline__ int first_best(K mine, K& best) {
  best = wave_max(mine);
  return __builtin_ctzll(__ballot(mine == best));
}

template <int VPL, class K>
__device__ __forceinline__ void lane_best(const K (&key)[VPL], K& mine, int& at) {
  mine = key[0];
  at = 0;
#pragma unroll
  for (int i = 1; i < VPL; ++i)
    if (key[i] > mine) {
      mine = key[i];
      at = i;
    }
}

// The topk best of the wave's keys: lane j gets the j-th one's expert (-1: none) and logit.
template <int VPL, class K>
__device__ __forceinline__ void choose(K (&key)[VPL], const float (&l)[VPL], int topk, int& id, float& logit) {
  const K none = -(K)__builtin_inf();
  const int lane = lane_id();
  id = -1;
  logit = 0.0f;
  K mine;
  int at;
  lane_best<VPL>(key, mine, at);
  for (int j = 0; j < topk; ++j) {
    K best;
    const int from = first_best(mine, best);
    if (!(best > none)) break;
    float v = l[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) v = at == i ? l[i] : v;
    const int e = __shfl(lane * VPL + at, from);
    const float lv = __shfl(v, from);
    if (lane == j) {
      id = e;
      logit = lv;
    }
    if (lane == from) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i == at) key[i] = none;
      lane_best<VPL>(key, mine, at);
    }
  }
}

// Takes the keys of all but the best groups out.  The sums of the groups' highest keys are found group by group (their
// experts need not lie in whole lanes).
template <int VPL>
__device__ __forceinline__ void keep_groups(const RouteArgs& p, double (&key)[VPL], int first) {
  const int size = p.experts / p.groups, lane = lane_id();
  double mine = -inf64();  // lane g: group g's score
  for (int g = 0; g < p.groups; ++g) {
    double k1 = -inf64(), k2 = -inf64();
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = first + i;
      const double k = e >= g * size && e < (g + 1) * size ? key[i] : -inf64();
      k2 = __builtin_fmax(k2, __builtin_fmin(k1, k));
      k1 = __builtin_fmax(k1, k);
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const double o1 = __shfl_xor(k1, d), o2 = __shfl_xor(k2, d);
      k2 = __builtin_fmax(__builtin_fmin(k1, o1), __builtin_fmax(k2, o2));
      k1 = __builtin_fmax(k1, o1);
    }
    const double sum = p.group_top == 2 && k2 > -inf64() ? k1 + k2 : k1;
    if (lane == g) mine = sum;
  }
  uint64_t kept = 0;
  for (int j = 0; j < p.topk_groups; ++j) {
    double best;
    const int from = first_best(mine, best);
    if (!(best > -inf64())) break;
    kept |= 1ull << from;
    if (lane == from) mine = -inf64();
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (!(kept >> min((first + i) / size, 63) & 1)) key[i] = -inf64();
}

template <int E, int VPL>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(RouteArgs p) {
  const int64_t token = (int64_t)blockIdx.x * kWaves + wave_id();
  if (token >= p.tokens) return;
  const int lane = lane_id(), first = lane * VPL;
  float l[VPL];
  load_logits<E, VPL>(p.logits, token * p.ld, first, p.experts, l);
  float top = l[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) top = fmaxf(top, l[i]);
  top = wave_max(top);
  const bool keyed = p.bias || p.groups > 1;
  double total = 1.0;
  double s[VPL];
  if (p.score == SC_SOFTMAX && (keyed || !p.renormalize)) {
    total = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      s[i] = l[i] > -__builtin_inff() ? exp_below(l[i], top) : 0.0;
      total += s[i];
    }
    total = wave_sum(total);
  }
  int id;
  float logit;
  if (keyed) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if (p.score == SC_SOFTMAX) s[i] = s[i] / total;
      else s[i] = sigmoid64(l[i]);
      const double k = p.bias && first + i < p.experts ? s[i] + (double)p.bias[first + i] : s[i];
      s[i] = l[i] > -__builtin_inff() && k == k ? k : -inf64();
    }
    if (p.groups > 1) keep_groups<VPL>(p, s, first);
    choose<VPL>(s, l, p.topk, id, logit);
  } else {
    float key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = l[i];
    choose<VPL>(key, l, p.topk, id, logit);
  }
  // the chosen ones' scores, one a lane
  double w = id < 0 ? 0.0 : p.score == SC_SIGMOID ? sigmoid64(logit) : exp_below(logit, top);
  if (p.renormalize) total = wave_sum(w);
  w = total > 0.0 ? w / total * p.scale : 0.0;
  if (lane < p.topk) {
    p.ids[token * p.topk + lane] = id;
    p.weights[token * p.topk + lane] = (float)w;
  }
}

// ------------------------------------------------------------------------------------- gradients
// With chosen c, S = sum of the chosen s, n = scale and G = sum over c of dw_c s_c:
//   ds_c = n dw_c, or renormalised n (dw_c - G / S) / S; ds = 0 elsewhere
//   sigmoid: dl = ds s (1 - s); softmax: dl = s (ds - sum ds s), whose sum is 0 where renormalised
// An expert chosen twice gets both.
template <int E, int VPL>
__global__ __launch_bounds__(64 * kWaves) void route_back_kernel(RouteBackArgs p) {
  const int64_t token = (int64_t)blockIdx.x * kWaves + wave_id();
  if (token >= p.tokens) return;
  const int lane = lane_id(), first = lane * VPL;
  float l[VPL];
  load_logits<E, VPL>(p.logits, token * p.ld, first, p.experts, l);
  // lane j: choice j
  int id = -1;
  float dw = 0.0f, logit = -__builtin_inff();
  if (lane < p.topk) {
    id = p.ids[token * p.topk + lane];
    if (id < 0 || id >= p.experts) id = -1;
    if (id >= 0) {
      dw = p.dweights[token * p.ld_dw + lane];
      logit = load_elt<E>((const char*)p.logits + (token * p.ld + id) * elt_size(E));
      if (!(logit > -__builtin_inff())) id = -1;
    }
  }
  float top = l[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) top = fmaxf(top, l[i]);
  top = wave_max(top);
  double s[VPL], total = 0.0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    s[i] = !(l[i] > -__builtin_inff()) ? 0.0 : p.score == SC_SIGMOID ? sigmoid64(l[i]) : exp_below(l[i], top);
    total += s[i];
  }
  double sc = id < 0 ? 0.0 : p.score == SC_SIGMOID ? sigmoid64(logit) : exp_below(logit, top);
  if (p.score == SC_SOFTMAX) {
    total = wave_sum(total);
    total = total > 0.0 ? 1.0 / total : 0.0;
    sc *= total;
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] *= total;
  }
  double ds = id < 0 ? 0.0 : (double)dw * p.scale;
  if (p.renormalize) {
    const double chosen = wave_sum(sc), along = wave_sum(ds * sc);
    ds = id >= 0 && chosen > 0.0 ? (ds - along / chosen) / chosen : 0.0;
  }
  const double mean = p.score == SC_SOFTMAX && !p.renormalize ? wave_sum(ds * sc) : 0.0;
  double d[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) d[i] = 0.0;
  for (int j = 0; j < p.topk; ++j) {
    const int e = __shfl(id, j);
    const double g = __shfl(ds, j);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (e == first + i) d[i] += g;
  }
  char* o = (char*)p.dlogits + (token * p.ld_out + first) * elt_size(E);
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const double v = p.score == SC_SIGMOID ? d[i] * s[i] * (1.0 - s[i]) : s[i] * (d[i] - mean);
    if (first + i < p.experts) store_elt<E>(o + i * elt_size(E), (float)v);
  }
}

template <int E>
hipError_t launch_route_e(const RouteArgs& p, hipStream_t s) {
  const unsigned grid = (unsigned)((p.tokens + kWaves - 1) / kWaves);
  if (p.experts <= 64) route_kernel<E, 1><<<grid, 64 * kWaves, 0, s>>>(p);
  else if (p.experts <= 128) route_kernel<E, 2><<<grid, 64 * kWaves, 0, s>>>(p);
  else if (p.experts <= 256) route_kernel<E, 4><<<grid, 64 * kWaves, 0, s>>>(p);
  else if (p.experts <= 512) route_kernel<E, 8><<<grid, 64 * kWaves, 0, s>>>(p);
  else route_kernel<E, 16><<<grid, 64 * kWaves, 0, s>>>(p);
  return hipGetLastError();
}

template <int E>
hipError_t launch_back_e(const RouteBackArgs& p, hipStream_t s) {
  const unsigned grid = (unsigned)((p.tokens + kWaves - 1) / kWaves);
  if (p.experts <= 64) route_back_kernel<E, 1><<<grid, 64 * kWaves, 0, s>>>(p);
  else if (p.experts <= 128) route_back_kernel<E, 2><<<grid, 64 * kWaves, 0, s>>>(p);
  else if (p.experts <= 256) route_back_kernel<E, 4><<<grid, 64 * kWaves, 0, s>>>(p);
  else if (p.experts <= 512) route_back_kernel<E, 8><<<grid, 64 * kWaves, 0, s>>>(p);
  else route_back_kernel<E, 16><<<grid, 64 * kWaves, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(int elt, const RouteArgs& p, hipStream_t s) {
  if (elt == EL_F16) return launch_route_e<EL_F16>(p, s);
  if (elt == EL_BF16) return launch_route_e<EL_BF16>(p, s);
  return launch_route_e<EL_F32>(p, s);
}

hipError_t launch_route_backward(int elt, const RouteBackArgs& p, hipStream_t s) {
  if (elt == EL_F16) return launch_back_e<EL_F16>(p, s);
  if (elt == EL_BF16) return launch_back_e<EL_BF16>(p, s);
  return launch_back_e<EL_F32>(p, s);
}

}  // namespace ep
