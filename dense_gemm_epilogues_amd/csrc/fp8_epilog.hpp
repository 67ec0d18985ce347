// The 8-bit products' epilogue, P = a b^T + bias, D = act(P) + residual: activations and their derivatives, in fp32.
//
// What it costs beside 8192 x 17408 x 5120 (608 us without): a bias 9 us (the accumulators start from it), ReLU 10, SiLU 23, GELU 52
// (21 instructions a value, nothing to hide behind: both waves of a SIMD are at their tile's end), the saved P 44 (285 MB), the residual 60
// (as many); passes over D of their own would read and write it, 114 us, for each.
#pragma once
#include "fp8_device.hpp"
#include "normal_dist.hpp"

namespace ep {

// 1 / (1 + e^-t) on the hardware's exp2 and reciprocal (1 ulp each); 0 and 1 at the ends
__device__ __forceinline__ float logistic(float t) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t * -1.44269504088896341f));
}

__device__ __forceinline__ float activate(int act, float v) {
  if (act == ACT_RELU) return v > 0.0f ? v : 0.0f;
  if (act == ACT_GELU) return gelu_f(v);
  if (act == ACT_SILU) return v * logistic(v);
  return v;
}

// d act'(v)
template <int ACT>
__device__ __forceinline__ float back_through(float d, float v) {
  if constexpr (ACT == ACT_RELU) return v > 0.0f ? d : 0.0f;  // (whatever d is)
  else if constexpr (ACT == ACT_GELU) return d * gelu_grad_f(v);
  else if constexpr (ACT == ACT_SILU) {
    const float s = logistic(v);
    return d * (s + v * s * (1.0f - s));
  } else return d;
}

// The bias of 8 columns from n on, `left` of them inside the matrix
template <int OT>
__device__ __forceinline__ void load_bias8(const Fp8Epilog& e, int n, int left, float* f) {
  if (!e.bias) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 0.0f;
  } else if (e.bias32) {
    load8<EL_F32>((const char*)e.bias + (int64_t)n * 4, left, f);
  } else {
    load8<OT>((const char*)e.bias + (int64_t)n * elt_size(OT), left, f);
  }
}

__device__ __forceinline__ void activate8(int act, float* f) {
  if (act == ACT_RELU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = activate(ACT_RELU, f[i]);
  } else if (act == ACT_GELU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = activate(ACT_GELU, f[i]);
  } else if (act == ACT_SILU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = activate(ACT_SILU, f[i]);
  }
}

// D of 8 columns of a row from their P in f
template <int OT>
__device__ __forceinline__ void finish8(const Fp8Epilog& e, int64_t row, int n, int left, float* f) {
  activate8(e.act, f);
  if (e.res) {
    float r[8];
    load8<OT>((const char*)e.res + (row * e.ld_res + n) * elt_size(OT), left, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] += r[i];
  }
}

// One value of P from its product, P stored, and D
template <int OT>
__device__ __forceinline__ float finish1(const Fp8Epilog& e, int64_t row, int n, float v) {
  if (e.bias) v += e.bias32 ? ((const float*)e.bias)[n] : load_elt<OT>((const char*)e.bias + (int64_t)n * elt_size(OT));
  if (e.pre) store_elt<OT>((char*)e.pre + (row * e.ld_pre + n) * elt_size(OT), v);
  v = activate(e.act, v);
  if (e.res) v += load_elt<OT>((const char*)e.res + (row * e.ld_res + n) * elt_size(OT));
  return v;
}

}  // namespace ep
