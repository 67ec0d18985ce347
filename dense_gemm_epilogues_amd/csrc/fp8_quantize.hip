// Quantisation to e4m3 with one fp32 scale for each block of 1 x 128 or 128 x 128 values, of a matrix
// or of its transpose.
//
// For a block with finite maximum amax (at least 2^-90): scale = amax / 448 and
// q = e4m3(fp32(v * fp32(448 / amax))), rounded to nearest even; infinities and NaN become NaN and do
// not count for amax.  One pass: each value is read once, kept in registers as fp32 while its block's
// maximum is found, and written once, so the kernels are bound by HBM: 8192 x 5120 bf16 in 25 us (5.1 TB/s, the rate
// of a large device copy), its transpose in 128 x 128 blocks in 29 (4.3 TB/s).  (Non-temporal loads: 31 and 35 us
// for an input that was just written.)
#include "fp8_device.hpp"

namespace ep {
namespace {

constexpr int kThreads = 256;

// 16 values of one row; those at or past n read as zeros
template <int E>
__device__ __forceinline__ void load16(const char* p, int n, float* f) {
  load8<E>(p, n, f);
  load8<E>(p + 8 * elt_size(E), n - 8, f + 8);
}

__device__ __forceinline__ u32x4 quant16(const float* f, float inv) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = to_e4m3x4(f[4 * i] * inv, f[4 * i + 1] * inv, f[4 * i + 2] * inv, f[4 * i + 3] * inv);
  return w;
}

__device__ __forceinline__ void put_bytes(uint8_t* q, int n, u32x4 w) {
  if (n >= 16) {
    *(u32x4_u*)q = w;
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) q[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
}

// 1 x 128 blocks along the rows: 8 lanes of 16 values per block; a workgroup takes 8 rows by 4
// blocks, so that the features-outermost scales leave in runs of 8.
template <int E>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(QuantArgs p, int kb_groups) {
  const int sub = (int)threadIdx.x & 7, g = (int)threadIdx.x >> 3;
  const int kb = ((int)blockIdx.x % kb_groups) * 4 + (g & 3);
  const int64_t row = (int64_t)((int)blockIdx.x / kb_groups) * 8 + (g >> 2);
  const int col = kb * kScaleBlock + sub * 16;
  const bool on = row < p.m && kb * kScaleBlock < p.k;
  const int n = on ? p.k - col : 0;
  float f[16];
  load16<E>((const char*)p.x + (row * p.ldx + col) * elt_size(E), n, f);
  float amax = kAmaxMin;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, finite_abs(f[i]));
#pragma unroll
  for (int d = 1; d < 8; d *= 2) amax = fmaxf(amax, __shfl_xor(amax, d));
  if (!on) return;
  const u32x4 w = quant16(f, scale_inv(amax));
  if (n > 0) put_bytes(p.q + row * p.ldq + col, n, w);
  if (sub == 0) p.scale[(int64_t)kb * p.m + row] = scale_of(amax);
}

// One 128 x 128 tile of x per workgroup; thread t holds 16 features of rows 32 i + t / 8.
// ROWS 128: one scale for the tile; ROWS 1 (TRANS only): one for each feature.  TRANS: the e4m3 tile
// goes through LDS, where each thread picks up 4 features of 16 rows as 16 words and transposes them
// as 4 x 4 bytes, so that both sides move 16 bytes per lane in whole 128-byte lines.
template <int E, int ROWS, bool TRANS>
__global__ __launch_bounds__(kThreads) void quantize_tile_kernel(QuantArgs p, int tiles_k) {
  __shared__ float red[4][kScaleBlock];
  __shared__ __align__(16) uint8_t tile[TRANS ? kScaleBlock * kScaleBlock : 16];
  const int tm = (int)blockIdx.x / tiles_k, tk = (int)blockIdx.x % tiles_k;
  const int m0 = tm * kScaleBlock, k0 = tk * kScaleBlock;
  const int t = (int)threadIdx.x, sub = t & 7, rg = t >> 3, lane = lane_id(), wave = wave_id();
  const int col = k0 + sub * 16;
  float f[4][16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = m0 + 32 * i + rg;
    load16<E>((const char*)p.x + ((int64_t)row * p.ldx + col) * elt_size(E), row < p.m ? p.k - col : 0, f[i]);
  }
  float amax[ROWS == 1 ? 16 : 1];
  if constexpr (ROWS == 1) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      amax[j] = kAmaxMin;
#pragma unroll
      for (int i = 0; i < 4; ++i) amax[j] = fmaxf(amax[j], finite_abs(f[i][j]));
#pragma unroll
      for (int d = 8; d < 64; d *= 2) amax[j] = fmaxf(amax[j], __shfl_xor(amax[j], d));
    }
    if (lane < 8) {
#pragma unroll
      for (int j = 0; j < 16; ++j) red[wave][lane * 16 + j] = amax[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int c = sub * 16 + j;
      amax[j] = fmaxf(fmaxf(red[0][c], red[1][c]), fmaxf(red[2][c], red[3][c]));
    }
    if (rg == 0) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (col + j < p.k) p.scale[(int64_t)tm * p.k + col + j] = scale_of(amax[j]);
    }
  } else {
    float a = kAmaxMin;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) a = fmaxf(a, finite_abs(f[i][j]));
#pragma unroll
    for (int d = 1; d < 64; d *= 2) a = fmaxf(a, __shfl_xor(a, d));
    if (lane == 0) red[0][wave] = a;
    __syncthreads();
    a = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    amax[0] = a;
    if (t == 0) {
      const int64_t at = TRANS ? (int64_t)tk * ((p.m + kScaleBlock - 1) / kScaleBlock) + tm : (int64_t)tm * tiles_k + tk;
      p.scale[at] = scale_of(a);
    }
  }
  float inv[ROWS == 1 ? 16 : 1];
#pragma unroll
  for (int j = 0; j < (ROWS == 1 ? 16 : 1); ++j) inv[j] = scale_inv(amax[j]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    u32x4 w;
    if constexpr (ROWS == 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = to_e4m3x4(f[i][4 * j] * inv[4 * j], f[i][4 * j + 1] * inv[4 * j + 1],
                         f[i][4 * j + 2] * inv[4 * j + 2], f[i][4 * j + 3] * inv[4 * j + 3]);
      }
    } else {
      w = quant16(f[i], inv[0]);
    }
    const int r = 32 * i + rg;
    if constexpr (TRANS) {
      // word kd of row r at kd ^ 8 (r / 16 % 4): the 16-byte pieces stay whole and the reads below
      // spread over the banks
      const int pos = (sub * 4) ^ (((r >> 4) & 3) << 3);
      *(u32x4*)(tile + r * kScaleBlock + pos * 4) = w;
    } else if (m0 + r < p.m && col < p.k) {
      put_bytes(p.q + (int64_t)(m0 + r) * p.ldq + col, p.k - col, w);
    }
  }
  if constexpr (TRANS) {
    __syncthreads();
    const int mg = t & 7, kd = t >> 3;  // rows 16 mg .. + 15, features 4 kd .. + 3
    const int pos = kd ^ ((mg & 3) << 3);
    u32x4 out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = *(const uint32_t*)(tile + (mg * 16 + 4 * j + e) * kScaleBlock + pos * 4);
      // bytes b of v0..v3 into word b: two rounds of byte pairs
      const uint32_t lo01 = __builtin_amdgcn_perm(v[1], v[0], 0x05010400u);  // v0.0 v1.0 v0.1 v1.1
      const uint32_t hi01 = __builtin_amdgcn_perm(v[1], v[0], 0x07030602u);  // v0.2 v1.2 v0.3 v1.3
      const uint32_t lo23 = __builtin_amdgcn_perm(v[3], v[2], 0x05010400u);
      const uint32_t hi23 = __builtin_amdgcn_perm(v[3], v[2], 0x07030602u);
      out[0][j] = __builtin_amdgcn_perm(lo23, lo01, 0x05040100u);
      out[1][j] = __builtin_amdgcn_perm(lo23, lo01, 0x07060302u);
      out[2][j] = __builtin_amdgcn_perm(hi23, hi01, 0x05040100u);
      out[3][j] = __builtin_amdgcn_perm(hi23, hi01, 0x07060302u);
    }
    const int mm = m0 + mg * 16;
    if (mm < p.m) {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int k = k0 + 4 * kd + b;
        if (k < p.k) put_bytes(p.q + (int64_t)k * p.ldq + mm, p.m - mm, out[b]);
      }
    }
  }
}

template <int E>
hipError_t launch_e(int rows, bool transpose, const QuantArgs& p, hipStream_t s) {
  const int tk = (p.k + kScaleBlock - 1) / kScaleBlock;
  const unsigned blocks = (unsigned)quantize_blocks(rows, transpose, p.m, p.k);
  if (rows == 1 && !transpose) quantize_rows_kernel<E><<<blocks, kThreads, 0, s>>>(p, (tk + 3) / 4);
  else if (rows == 1) quantize_tile_kernel<E, 1, true><<<blocks, kThreads, 0, s>>>(p, tk);
  else if (transpose) quantize_tile_kernel<E, 128, true><<<blocks, kThreads, 0, s>>>(p, tk);
  else quantize_tile_kernel<E, 128, false><<<blocks, kThreads, 0, s>>>(p, tk);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize(int elt, int rows, bool transpose, const QuantArgs& p, hipStream_t s) {
  if (elt == EL_F16) return launch_e<EL_F16>(rows, transpose, p, s);
  if (elt == EL_BF16) return launch_e<EL_BF16>(rows, transpose, p, s);
  return launch_e<EL_F32>(rows, transpose, p, s);
}

}  // namespace ep
