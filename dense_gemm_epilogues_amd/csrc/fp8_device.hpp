// Device helpers shared by the 8-bit and expert kernels: element access at any alignment, rounding
// to e4m3, block scales.
#pragma once
#include "fp8_ops.hpp"

namespace ep {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
// the same at any byte address: gfx950 global memory instructions take unaligned addresses, so rows
// of odd length keep 16-byte accesses
typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_u __attribute__((ext_vector_type(2), aligned(1)));

template <int E>
__device__ __forceinline__ float elt_f32(uint32_t bits) {
  if constexpr (E == EL_F16) return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
  else if constexpr (E == EL_BF16) return __builtin_bit_cast(float, bits << 16);
  else return __builtin_bit_cast(float, bits);
}

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bhalf2_t __attribute__((ext_vector_type(2)));

// two floats rounded to nearest even in one word, the first in the low half
template <int E>
__device__ __forceinline__ uint32_t pack2_elt(float lo, float hi) {
  if constexpr (E == EL_F16) {
    const half2_t v = {(_Float16)lo, (_Float16)hi};
    return __builtin_bit_cast(uint32_t, v);
  } else {
    const bhalf2_t v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
  }
}

template <int E>
__device__ __forceinline__ void store_elt(char* p, float v) {
  if constexpr (E == EL_F32) *(float*)p = v;
  else *(uint16_t*)p = (uint16_t)pack2_elt<E>(v, v);
}

template <int E>
__device__ __forceinline__ float load_elt(const char* p) {
  if constexpr (E == EL_F32) return *(const float*)p;
  else return elt_f32<E>(*(const uint16_t*)p);
}

// fewer than 8 elements from p, the others as zeros (one branch: an element past the end loads the last one and is dropped)
template <int E>
__device__ __forceinline__ void load_tail(const char* p, int n, float* f) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = 0.0f;
  if (n > 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = i < n ? i : n - 1;
      const float v = load_elt<E>(p + at * elt_size(E));
      f[i] = i < n ? v : 0.0f;
    }
  }
}

// 16 bytes from and to p; NT: past the caches' replacement (non-temporal)
template <bool NT>
__device__ __forceinline__ u32x4 get16(const char* p) {
  if constexpr (NT) return __builtin_nontemporal_load((const u32x4_u*)p);
  else return *(const u32x4_u*)p;
}
template <bool NT>
__device__ __forceinline__ void put16(char* p, u32x4 w) {
  if constexpr (NT) __builtin_nontemporal_store(w, (u32x4_u*)p);
  else *(u32x4_u*)p = w;
}

// 8 elements from p, those at or past `n` as zeros
template <int E, bool NT = false>
__device__ __forceinline__ void load8(const char* p, int n, float* f) {
  if constexpr (E == EL_F32) {
    if (n >= 8) {
      const u32x4 a = get16<NT>(p), b = get16<NT>(p + 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = elt_f32<E>(a[i]);
        f[4 + i] = elt_f32<E>(b[i]);
      }
    } else {
      load_tail<E>(p, n, f);
    }
  } else {
    if (n >= 8) {
      const u32x4 a = get16<NT>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = elt_f32<E>(a[i] & 0xffffu);
        f[2 * i + 1] = elt_f32<E>(a[i] >> 16);
      }
    } else {
      load_tail<E>(p, n, f);
    }
  }
}

// 8 elements to p, those at or past `n` left alone
template <int E, bool NT = false>
__device__ __forceinline__ void store8(char* p, int n, const float* f) {
  if constexpr (E == EL_F32) {
    if (n >= 8) {
      put16<NT>(p, __builtin_bit_cast(u32x4, f32x4{f[0], f[1], f[2], f[3]}));
      put16<NT>(p + 16, __builtin_bit_cast(u32x4, f32x4{f[4], f[5], f[6], f[7]}));
      return;
    }
  } else {
    if (n >= 8) {
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = pack2_elt<E>(f[2 * i], f[2 * i + 1]);
      put16<NT>(p, w);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) store_elt<E>(p + i * elt_size(E), f[i]);
}

// 8 neighbouring values of a row of `len` >= 8 at column n, wherever the row ends: near its end the last 8 are loaded and
// moved down, without branches.  What lies at or past the end is undefined.
template <int N>
__device__ __forceinline__ void move_down(uint32_t (&w)[N], int by) {  // by whole words, up to N - 1
#pragma unroll
  for (int d = 1; d < N; d *= 2) {
    uint32_t on = by & d ? ~0u : 0u;
    asm("" : "+v"(on));  // (bits, not a condition: those are short of scalar registers)
#pragma unroll
    for (int i = 0; i + d < N; ++i) w[i] = (w[i + d] & on) | (w[i] & ~on);
  }
}
__device__ __forceinline__ u32x4 window8_16(const char* row, int n, int len) {  // of 16-bit values, as they are
  const int at = min(n, len - 8);
  const u32x4 v = *(const u32x4_u*)(row + (uint32_t)at * 2u);
  if (len % 8 == 0) return v;
  const int by = n - at;
  uint32_t w[4] = {v[0], v[1], v[2], v[3]};
  move_down<4>(w, by >> 1);
  if (len & 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = by & 1 ? (w[i] >> 16) | (i < 3 ? w[i + 1] << 16 : 0u) : w[i];
  }
  return u32x4{w[0], w[1], w[2], w[3]};
}
template <int E>
__device__ __forceinline__ void window8(const char* row, int n, int len, float* f) {
  if constexpr (E == EL_F32) {
    const int at = min(n, len - 8);
    const u32x4 a = *(const u32x4_u*)(row + (int64_t)at * 4), b = *(const u32x4_u*)(row + (int64_t)at * 4 + 16);
    uint32_t w[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    if (len % 8) move_down<8>(w, n - at);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = elt_f32<E>(w[i]);
  } else {
    const u32x4 w = window8_16(row, n, len);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = elt_f32<E>(w[i] & 0xffffu);
      f[2 * i + 1] = elt_f32<E>(w[i] >> 16);
    }
  }
}

// |v| of a finite value, 0 of an infinity or NaN
__device__ __forceinline__ float finite_abs(float v) {
  const float a = __builtin_fabsf(v);
  return a < __builtin_inff() ? a : 0.0f;
}

// A block's scale is amax / 448, its values are multiplied by fp32(448 / amax): both divisions are
// correctly rounded, so a value's error is one rounding of the factor, one of the product and one to
// e4m3.  amax is kept at or above 2^-90, so neither quotient leaves the normal range.
__device__ __forceinline__ float scale_inv(float amax) { return kF8Max / amax; }
__device__ __forceinline__ float scale_of(float amax) { return amax / kF8Max; }

// four values times their factors as e4m3, lowest byte first.  The factors keep finite values at or
// below 448; what is above the type's range, so infinities, and NaN convert to NaN.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)); }
__device__ __forceinline__ int lane_id() { return (int)(threadIdx.x & 63); }

}  // namespace ep
