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
// A wave takes a token; its lanes are dealt out to the groups (a power of two to each), a lane takes VPL neighbouring
// experts of its group, which stay in registers, sorted, as whole numbers in the order of their keys: a choice is one maximum over
// the lanes' best and takes about 30 instructions.  Instructions are what bounds it: 100 of them for each of 8192 tokens take
// 1.3 us.  So keys are first made in fp32, which holds the order wherever neighbours are further apart than its error, and that
// is checked for the groups and choices that came out; a token that fails (about one in a thousand with random logits; those with equal scores at the
// border) is done again in double.
#include "block_ops.hpp"
#include "fp8_device.hpp"
#include "wave_ops.hpp"

namespace ep {
namespace {

constexpr int kWaves = 4;  // tokens a workgroup

__device__ __forceinline__ double inf64() { return __builtin_inf(); }
__device__ __forceinline__ float inf32() { return __builtin_inff(); }

struct Add {
  template <class T>
  __device__ T operator()(T a, T b) const { return a + b; }
};
struct Max {
  __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// A constant as a scalar operand (as a vector one it takes two instructions at each use), where there are registers for it
template <bool S>
__device__ __forceinline__ double scalar(double c) {
  if constexpr (S) asm("" : "+s"(c));
  return c;
}

// e^x to about 2^-52 of it, for x from -745 to 709: x = n ln 2 + r, |r| <= ln 2 / 2, and 14 terms of e^r's series (the next
// is below 2^-57).  A third of the library function's instructions.
template <bool S>
__device__ __forceinline__ double exp64(double x) {
  const double n = __builtin_rint(x * scalar<S>(1.4426950408889634));
  const double r = __builtin_fma(n, scalar<S>(-2.3190468138462996e-17), __builtin_fma(n, scalar<S>(-0.69314718055994531), x));
  constexpr double c[12] = {1.0 / 479001600.0, 1.0 / 39916800.0, 1.0 / 3628800.0, 1.0 / 362880.0, 1.0 / 40320.0, 1.0 / 5040.0,
                            1.0 / 720.0, 1.0 / 120.0, 1.0 / 24.0, 1.0 / 6.0, 0.5, 1.0};
  double p = __builtin_fma(r, 1.0 / 6227020800.0, scalar<S>(c[0]));
#pragma unroll
  for (int i = 1; i < 12; ++i) p = __builtin_fma(p, r, scalar<S>(c[i]));
  return __builtin_amdgcn_ldexp(__builtin_fma(p, r, 1.0), (int)n);
}

// e^(l - m) for l <= m, 1 where both are the same infinity, 0 where the double has no place for it
template <bool S = true>
__device__ __forceinline__ double exp_below(float l, float m) {
  const double x = (double)l - (double)m;
  return l == m ? 1.0 : x > -745.0 ? exp64<S>(x) : 0.0;
}

// 1 / (1 + e^-l): the hardware's reciprocal and two steps of Newton's method
template <bool S = true>
__device__ __forceinline__ double sigmoid64(float l) {
  const double d = 1.0 + exp64<S>(__builtin_fmin(__builtin_fmax(-(double)l, -745.0), 709.0));
  double y = __builtin_amdgcn_rcp(d);
  y = __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
  y = __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
  return l < -709.0f ? 0.0 : y;
}

// VPL neighbouring values of a row from p, -infinity past the n-th and for NaN
template <int E, int VPL>
__device__ __forceinline__ void load_logits(const char* p, int n, float* l) {
  if constexpr (VPL >= 8) {
#pragma unroll
    for (int i = 0; i < VPL; i += 8) load8<E>(p + i * elt_size(E), n - i, l + i);
  } else {
    constexpr int BYTES = VPL * elt_size(E), WORDS = (BYTES + 3) / 4;
    typedef uint32_t words __attribute__((ext_vector_type(WORDS < 2 ? 2 : WORDS), aligned(1)));
    if (BYTES >= 8 && n >= VPL) {
      const words w = *(const words*)p;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        l[i] = E == EL_F32 ? elt_f32<E>(w[i]) : elt_f32<E>(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu);
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) l[i] = i < n ? load_elt<E>(p + i * elt_size(E)) : 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) l[i] = i < n && l[i] == l[i] ? l[i] : -inf32();
}

template <int VPL>
__device__ __forceinline__ float max_of(const float* l) {
  float top = l[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) top = fmaxf(top, l[i]);
  return top;
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

// The topk best of the wave's keys: lane j gets the j-th one's expert (-1: none).
template <int VPL, class K>
__device__ __forceinline__ void choose(K (&key)[VPL], int first, int topk, int& id) {
  const int lane = lane_id();
  id = -1;
  K mine;
  int at;
  lane_best<VPL>(key, mine, at);
  for (int j = 0; j < topk; ++j) {
    const float mine32 = (float)mine, best32 = wave_reduce(mine32, Max());
    if (!(best32 > -inf32())) break;
    uint64_t same = __ballot(mine32 == best32);
    int from = __builtin_ctzll(same);
    if constexpr (sizeof(K) == 8) {
      if (same &= same - 1) {  // equal in fp32
        K best = read_lane(mine, from);
        for (; same; same &= same - 1) {
          const int other = __builtin_ctzll(same);
          const K k = read_lane(mine, other);
          if (k > best) {
            best = k;
            from = other;
          }
        }
      }
    }
    const int e = read_lane(first + at, from);
    id = lane == j ? e : id;
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = lane == from && i == at ? -(K)__builtin_inf() : key[i];
    lane_best<VPL>(key, mine, at);
  }
}

// Takes the keys of all but the best groups out.  A group's lanes (1 << shift) find its two highest keys together.
template <int VPL>
__device__ __forceinline__ void keep_groups(const RouteArgs& p, double (&key)[VPL]) {
  double k1 = key[0], k2 = -inf64();
#pragma unroll
  for (int i = 1; i < VPL; ++i) {
    k2 = __builtin_fmax(k2, __builtin_fmin(k1, key[i]));
    k1 = __builtin_fmax(k1, key[i]);
  }
  auto merge = [&](double o1, double o2) __attribute__((always_inline)) {
    k2 = __builtin_fmax(__builtin_fmin(k1, o1), __builtin_fmax(k2, o2));
    k1 = __builtin_fmax(k1, o1);
  };
  if (p.shift > 0) merge(lane_xor<1>(k1), lane_xor<1>(k2));
  if (p.shift > 1) merge(lane_xor<2>(k1), lane_xor<2>(k2));
  if (p.shift > 2) merge(lane_xor<4>(k1), lane_xor<4>(k2));
  if (p.shift > 3) merge(lane_xor<8>(k1), lane_xor<8>(k2));
  if (p.shift > 4) merge(lane_xor<16>(k1), lane_xor<16>(k2));
  const double mine = p.group_top == 2 && k2 > -inf64() ? k1 + k2 : k1;
  const int g = lane_id() >> p.shift;
  int better = 0;  // groups that come before this lane's
  for (int i = 0; i < p.groups; ++i) {
    const double other = read_lane(mine, i << p.shift);
    better += other > mine || (other == mine && i < g) ? 1 : 0;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) key[i] = better < p.topk_groups ? key[i] : -inf64();
}

// ---- in fp32
// A whole number in the order of v's values (0 and -0 alike), above 0
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __builtin_bit_cast(float, u ^ ((uint32_t)((int)~u >> 31) | 0x80000000u));
}

struct MaxU {
  __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return max(a, b); }
};

// A lane's keys in falling order, equal ones by rising place, and their places, 4 bits each
template <int VPL>
__device__ __forceinline__ uint32_t sort_lane(uint32_t (&key)[VPL]) {
  uint32_t at[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) at[i] = i;
  // neighbours in odd and even pairs by turns: stable, and short enough for up to 8
#pragma unroll
  for (int r = 0; r < VPL; ++r)
#pragma unroll
    for (int i = r & 1; i + 1 < VPL; i += 2) {
      const bool swap = key[i + 1] > key[i];
      const uint32_t k = max(key[i], key[i + 1]), l = min(key[i], key[i + 1]), a = swap ? at[i + 1] : at[i], b = swap ? at[i] : at[i + 1];
      key[i] = k;
      key[i + 1] = l;
      at[i] = a;
      at[i + 1] = b;
    }
  uint32_t places = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) places |= at[i] << (4 * i);
  return places;
}

// The topk best keys: lane j gets the j-th one's expert, and its key (0: none); `next` is the best key that is left, 0 if there is none.
template <int VPL>
__device__ __forceinline__ void choose_sorted(uint32_t (&key)[VPL], int first, int topk, int& id, uint32_t& chosen, uint32_t& next) {
  const int lane = lane_id();
  uint32_t places = sort_lane<VPL>(key);
  id = -1;
  chosen = 0;
  for (int j = 0;; ++j) {
    next = wave_reduce(key[0], MaxU());
    if (j == topk || next == 0) break;
    const uint64_t same = __ballot(key[0] == next);
    const int from = __builtin_ctzll(same);
    const int e = read_lane(first + (int)(places & 15), from);
    const bool own = lane == from;
    id = lane == j ? e : id;
    chosen = lane == j ? next : chosen;
#pragma unroll
    for (int i = 0; i + 1 < VPL; ++i) key[i] = own ? key[i + 1] : key[i];
    key[VPL - 1] = own ? 0u : key[VPL - 1];
    places = own ? places >> 4 : places;
  }
}

// Groups by their keys in fp32; false if the keys' error, at most `off` each, could change which.
template <int VPL>
__device__ __forceinline__ bool keep_groups32(const RouteArgs& p, float (&key)[VPL], float off) {
  float k1 = key[0], k2 = -inf32();
#pragma unroll
  for (int i = 1; i < VPL; ++i) {
    k2 = fmaxf(k2, fminf(k1, key[i]));
    k1 = fmaxf(k1, key[i]);
  }
  auto merge = [&](float o1, float o2) __attribute__((always_inline)) {
    k2 = fmaxf(fminf(k1, o1), fmaxf(k2, o2));
    k1 = fmaxf(k1, o1);
  };
  if (p.shift > 0) merge(lane_xor<1>(k1), lane_xor<1>(k2));
  if (p.shift > 1) merge(lane_xor<2>(k1), lane_xor<2>(k2));
  if (p.shift > 2) merge(lane_xor<4>(k1), lane_xor<4>(k2));
  if (p.shift > 3) merge(lane_xor<8>(k1), lane_xor<8>(k2));
  if (p.shift > 4) merge(lane_xor<16>(k1), lane_xor<16>(k2));
  const float mine = p.group_top == 2 && k2 > -inf32() ? k1 + k2 : k1;
  // groups that may and that must come before this lane's, itself among the first: two sums of two keys are off by 4 errors and
  // two roundings, which are below the keys' own
  const float low = mine - 7.0f * off, high = mine + 7.0f * off;
  int may = 0, must = 0;
  for (int i = 0; i < p.groups; ++i) {
    const float other = read_lane(mine, i << p.shift);
    may += other >= low ? 1 : 0;
    must += other > high ? 1 : 0;
  }
  const bool on = must < p.topk_groups;
  const bool sure = !(mine > -inf32()) || (may <= p.topk_groups) == on;
#pragma unroll
  for (int i = 0; i < VPL; ++i) key[i] = on ? key[i] : -inf32();
  return __ballot(!sure) == 0;
}

// What fp32's scores are off at most, as parts of the greatest score.  Sigmoid: e^-l by its argument's rounding, |l| 2^-24, and the
// hardware's exp2, 2^-23, which s (1 - s) brings below 0.23 2^-24 + 0.25 2^-23; the sum's rounding and the reciprocal, 2^-24 and 2^-23 of s:
// together below 2.8e-7.  Softmax: e^-x, x = top - l: x's rounding and its product's, 2 x 2^-24 with x e^-x <= 0.37, exp2, the sum over up to
// 512 experts (8 additions in a lane, 6 more, each 2^-24), the quotient's two roundings: below 1.7e-6 of the greatest.
constexpr float kOffSigmoid = 4e-7f, kOffSoftmax = 2e-6f;

// The choice by keys in fp32; false where it is not certain.
template <int VPL>
__device__ __forceinline__ bool route32(const RouteArgs& p, const float (&l)[VPL], float top, int first, int n, int& id) {
  float key[VPL], off;
  if (p.score == SC_SOFTMAX) {
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      key[i] = __builtin_amdgcn_exp2f((l[i] - top) * 1.44269504088896341f);
      total += key[i];
    }
    const float over = 1.0f / wave_reduce(total, Add());  // the greatest score
    if (!(over > 0.0f)) return false;                     // (infinite logits, or none at all)
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] *= over;
    off = kOffSoftmax * over;
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(l[i] * -1.44269504088896341f));
    off = kOffSigmoid;
  }
  float size = 0.0f;
  if (p.bias) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      key[i] += i < n ? p.bias[first + i] : 0.0f;
      size = fmaxf(size, l[i] > -inf32() && key[i] == key[i] ? __builtin_fabsf(key[i]) : 0.0f);
    }
    off += wave_reduce(size, Max()) * 0x1p-23f;  // the sum's rounding
    if (!(off < inf32())) return false;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) key[i] = l[i] > -inf32() && key[i] > -inf32() ? key[i] : -inf32();
  if (p.groups > 1 && !keep_groups32<VPL>(p, key, off)) return false;
  uint32_t u[VPL], chosen, next;
#pragma unroll
  for (int i = 0; i < VPL; ++i) u[i] = key[i] > -inf32() ? ordered(key[i]) : 0u;
  choose_sorted<VPL>(u, first, p.topk, id, chosen, next);
  // each further than both errors from the next (which lane j + 1 holds, or `next`)
  const int lane = lane_id();
  uint32_t after = (uint32_t)__shfl_down((int)chosen, 1);
  if (lane == p.topk - 1) after = next;
  const bool sure = lane >= p.topk || chosen == 0 || after == 0 || unordered(chosen) - unordered(after) > 2.5f * off;
  return __ballot(!sure) == 0;
}

// (32 experts a lane stay in registers only where the compiler counts on few waves)
template <int E, int VPL>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(1, VPL > 16 ? 2 : 8))) void route_kernel(RouteArgs p) {
  const int64_t token = (int64_t)blockIdx.x * kWaves + wave_id();
  if (token >= p.tokens) return;
  const int lane = lane_id(), g = lane >> p.shift, size = p.experts / p.groups;
  const int at = (lane & ((1 << p.shift) - 1)) * VPL, first = g * size + at, n = g < p.groups ? size - at : 0;
  float l[VPL];
  load_logits<E, VPL>((const char*)p.logits + (token * p.ld + first) * elt_size(E), n, l);
  const float top = p.score == SC_SOFTMAX ? wave_reduce(max_of<VPL>(l), Max()) : 0.0f;
  const bool keyed = p.bias || p.groups > 1;
  double total = 1.0;  // what the scores are over
  int id;
  bool sure = false;
  if constexpr (VPL <= 8) {
    if (keyed) {
      sure = route32<VPL>(p, l, top, first, n, id);
    } else {
      uint32_t u[VPL], chosen, next;
#pragma unroll
      for (int i = 0; i < VPL; ++i) u[i] = l[i] > -inf32() ? ordered(l[i]) : 0u;
      choose_sorted<VPL>(u, first, p.topk, id, chosen, next);
      sure = true;
    }
  }
  const bool summed = p.score == SC_SOFTMAX && ((keyed && !sure) || !p.renormalize);
  constexpr bool S = VPL <= 16;
  double s[VPL];
  if (summed) {
    total = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      s[i] = l[i] > -inf32() ? exp_below<S>(l[i], top) : 0.0;
      total += s[i];
    }
    total = wave_reduce(total, Add());
  }
  if (!sure) {
    if (keyed) {
      const double over = 1.0 / total;
      int left = n;
      if (VPL > 16) asm("" : "+v"(left));  // (compared again: 32 answers kept take the scalar registers)
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        s[i] = p.score == SC_SOFTMAX ? s[i] * over : sigmoid64<S>(l[i]);
        const double k = p.bias && i < left ? s[i] + (double)p.bias[first + i] : s[i];
        s[i] = l[i] > -inf32() && k == k ? k : -inf64();
      }
      if (p.groups > 1) keep_groups<VPL>(p, s);
      choose<VPL>(s, first, p.topk, id);
    } else {
      float key[VPL];
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = l[i];
      choose<VPL>(key, first, p.topk, id);
    }
  }
  const float logit = id < 0 ? 0.0f : load_elt<E>((const char*)p.logits + (token * p.ld + id) * elt_size(E));
  // the chosen ones' scores, one a lane
  double w = id < 0 ? 0.0 : p.score == SC_SIGMOID ? sigmoid64<S>(logit) : exp_below<S>(logit, top);
  if (p.renormalize) total = wave_reduce(w, Add());
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
// So only the chosen logits are read, but for softmax that is not renormalised.  An expert chosen twice gets both.
template <int E, int VPL>
__global__ __launch_bounds__(64 * kWaves) void route_back_kernel(RouteBackArgs p) {
  const int64_t token = (int64_t)blockIdx.x * kWaves + wave_id();
  if (token >= p.tokens) return;
  const int lane = lane_id(), first = lane * VPL, n = p.experts - first;
  const char* row = (const char*)p.logits + token * p.ld * elt_size(E);
  // lane j: choice j
  int id = -1;
  float dw = 0.0f, logit = -inf32();
  if (lane < p.topk) {
    id = p.ids[token * p.topk + lane];
    if (id < 0 || id >= p.experts) id = -1;
    if (id >= 0) {
      dw = p.dweights[token * p.ld_dw + lane];
      logit = load_elt<E>(row + id * elt_size(E));
      if (!(logit > -inf32())) id = -1;
    }
  }
  if (id < 0) logit = -inf32();
  const bool dense = p.score == SC_SOFTMAX && !p.renormalize;
  float l[VPL], top, out[VPL];
  double s[VPL], over = 1.0;
  if (dense) {
    load_logits<E, VPL>(row + first * elt_size(E), n, l);
    top = wave_reduce(max_of<VPL>(l), Max());
    double total = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      s[i] = l[i] > -inf32() ? exp_below(l[i], top) : 0.0;
      total += s[i];
    }
    total = wave_reduce(total, Add());
    over = total > 0.0 ? 1.0 / total : 0.0;
  } else {
    top = wave_reduce(logit, Max());
  }
  const double sc = id < 0 ? 0.0 : p.score == SC_SIGMOID ? sigmoid64(logit) : exp_below(logit, top) * over;
  double ds = id < 0 ? 0.0 : (double)dw * p.scale;
  if (p.renormalize) {
    const double chosen = wave_reduce(sc, Add()), along = wave_reduce(ds * sc, Add());
    ds = id >= 0 && chosen > 0.0 ? (ds - along / chosen) / chosen : 0.0;
  }
  const float mine = (float)(p.score == SC_SIGMOID ? ds * sc * (1.0 - sc) : ds * sc);
  if (dense) {
    const double mean = wave_reduce(ds * sc, Add()) * over;
#pragma unroll
    for (int i = 0; i < VPL; ++i) out[i] = (float)(-s[i] * mean);
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) out[i] = 0.0f;
  }
  for (int j = 0; j < p.topk; ++j) {
    const int e = read_lane(id, j);
    const float v = read_lane(mine, j);
#pragma unroll
    for (int i = 0; i < VPL; ++i) out[i] += e == first + i ? v : 0.0f;
  }
  char* o = (char*)p.dlogits + (token * p.ld_out + first) * elt_size(E);
  if constexpr (VPL >= 8) {
#pragma unroll
    for (int i = 0; i < VPL; i += 8) store8<E>(o + i * elt_size(E), n - i, out + i);
  } else {
    constexpr int BYTES = VPL * elt_size(E), WORDS = (BYTES + 3) / 4;
    typedef uint32_t words __attribute__((ext_vector_type(WORDS < 2 ? 2 : WORDS), aligned(1)));
    if (BYTES >= 8 && n >= VPL) {
      words w;
#pragma unroll
      for (int i = 0; i < WORDS; ++i) {
        if constexpr (E == EL_F32) w[i] = __builtin_bit_cast(uint32_t, out[i]);
        else w[i] = pack2_elt<E>(out[(2 * i) % VPL], out[(2 * i + 1) % VPL]);
      }
      *(words*)o = w;
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i < n) store_elt<E>(o + i * elt_size(E), out[i]);
    }
  }
}

// Lanes that a group's experts take with so many each, a power of two
int lanes_of(int size, int each) {
  int lanes = 1;
  while (lanes * each < size) lanes *= 2;
  return lanes;
}

// The fewest experts a lane with which the groups fit the wave (32 always do, with 1024 experts in up to 64 groups)
int each_of(int size, int groups) {
  int each = 1;
  while (lanes_of(size, each) * groups > 64) each *= 2;
  return each;
}

template <int E>
hipError_t launch_route_e(RouteArgs p, hipStream_t s) {
  const unsigned grid = (unsigned)((p.tokens + kWaves - 1) / kWaves);
  const int size = p.experts / p.groups, each = each_of(size, p.groups);
  p.shift = __builtin_ctz((unsigned)lanes_of(size, each));
  if (each == 1) route_kernel<E, 1><<<grid, 64 * kWaves, 0, s>>>(p);
  else if (each == 2) route_kernel<E, 2><<<grid, 64 * kWaves, 0, s>>>(p);
  else if (each == 4) route_kernel<E, 4><<<grid, 64 * kWaves, 0, s>>>(p);
  else if (each == 8) route_kernel<E, 8><<<grid, 64 * kWaves, 0, s>>>(p);
  else if (each == 16) route_kernel<E, 16><<<grid, 64 * kWaves, 0, s>>>(p);
  else route_kernel<E, 32><<<grid, 64 * kWaves, 0, s>>>(p);
  return hipGetLastError();
}

template <int E>
hipError_t launch_back_e(const RouteBackArgs& p, hipStream_t s) {
  const unsigned grid = (unsigned)((p.tokens + kWaves - 1) / kWaves);
  const int each = each_of(p.experts, 1);
  if (each == 1) route_back_kernel<E, 1><<<grid, 64 * kWaves, 0, s>>>(p);
  else if (each == 2) route_back_kernel<E, 2><<<grid, 64 * kWaves, 0, s>>>(p);
  else if (each == 4) route_back_kernel<E, 4><<<grid, 64 * kWaves, 0, s>>>(p);
  else if (each == 8) route_back_kernel<E, 8><<<grid, 64 * kWaves, 0, s>>>(p);
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
