// The gradient of the 8-bit products' epilogue, as the operands of the two products that follow it.
//
//   g = dout act'(P) (fp32);  q = e4m3 rows of g with scales of 1 x 128, an operand of dA = g B;
//   qt = the same of its transpose, an operand of dB = g^T A;  dbias = sum over rows of g
//
// One pass: a workgroup holds a 128 x 128 tile of g in registers, finds the maxima along both directions and its column
// sums, and writes both quantisations, the transposed one through LDS.  Bound by HBM and, with an activation, nearly by
// the arithmetic (46 instructions a value at the copy's rate).
#include "block_ops.hpp"
#include "fp8_epilog.hpp"

namespace ep {
namespace {

constexpr int kThreads = 256;

template <int E>
__device__ __forceinline__ void load16(const char* p, int n, float* f) {
  load8<E>(p, n, f);
  load8<E>(p + 8 * elt_size(E), n - 8, f + 8);
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

// Thread t holds 16 columns, 16 (t % 8) .. + 15, of rows 32 i + t / 8.
template <int E, int ACT>
__global__ __launch_bounds__(kThreads) void epilogue_back_kernel(EpilogBackArgs p, int tiles_n) {
  __shared__ float red[2][4][kScaleBlock];
  __shared__ __align__(16) uint8_t tile[kScaleBlock * kScaleBlock];
  const int tm = (int)(blockIdx.x / (unsigned)tiles_n), tn = (int)(blockIdx.x % (unsigned)tiles_n);
  const int m0 = tm * kScaleBlock, n0 = tn * kScaleBlock;
  const int t = (int)threadIdx.x, sub = t & 7, rg = t >> 3, lane = lane_id(), wave = wave_id();
  const int col = n0 + sub * 16;
  float f[4][16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = m0 + 32 * i + rg;
    const int n = row < p.m ? p.n - col : 0;
    load16<E>((const char*)p.dout + (row * p.ld + col) * elt_size(E), n, f[i]);
    if constexpr (ACT != ACT_NONE) {
      float v[16];
      load16<E>((const char*)p.pre + (row * p.ldp + col) * elt_size(E), n, v);
#pragma unroll
      for (int j = 0; j < 16; ++j) f[i][j] = back_through<ACT>(f[i][j], v[j]);
    }
  }
  // rows: 8 lanes a block
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float amax = kAmaxMin;
#pragma unroll
    for (int j = 0; j < 16; ++j) amax = fmaxf(amax, finite_abs(f[i][j]));
#pragma unroll
    for (int d = 1; d < 8; d *= 2) amax = fmaxf(amax, __shfl_xor(amax, d));
    const float inv = scale_inv(amax);
    const int64_t row = m0 + 32 * i + rg;
    if (row < p.m && col < p.n) {
      u32x4 w;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = to_e4m3x4(f[i][4 * j] * inv, f[i][4 * j + 1] * inv, f[i][4 * j + 2] * inv, f[i][4 * j + 3] * inv);
      put_bytes(p.q + row * p.ldq + col, p.n - col, w);
      if (sub == 0) p.scale[(int64_t)tn * p.m + row] = scale_of(amax);
    }
  }
  // columns: maxima and sums over the thread's rows, the wave's and the four waves'
  float amax[16], sum[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    amax[j] = kAmaxMin;
    sum[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      amax[j] = fmaxf(amax[j], finite_abs(f[i][j]));
      sum[j] += f[i][j];
    }
#pragma unroll
    for (int d = 8; d < 64; d *= 2) {
      amax[j] = fmaxf(amax[j], __shfl_xor(amax[j], d));
      sum[j] += __shfl_xor(sum[j], d);
    }
  }
  if (lane < 8) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      red[0][wave][lane * 16 + j] = amax[j];
      red[1][wave][lane * 16 + j] = sum[j];
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const int c = sub * 16 + j;
    amax[j] = fmaxf(fmaxf(red[0][0][c], red[0][1][c]), fmaxf(red[0][2][c], red[0][3][c]));
  }
  if (t < kScaleBlock && n0 + t < p.n)
    p.part[(int64_t)tm * p.n + n0 + t] = (red[1][0][t] + red[1][1][t]) + (red[1][2][t] + red[1][3][t]);
  if (rg == 0) {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (col + j < p.n) p.scale_t[(int64_t)tm * p.n + col + j] = scale_of(amax[j]);
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) amax[j] = scale_inv(amax[j]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = to_e4m3x4(f[i][4 * j] * amax[4 * j], f[i][4 * j + 1] * amax[4 * j + 1], f[i][4 * j + 2] * amax[4 * j + 2],
                       f[i][4 * j + 3] * amax[4 * j + 3]);
    }
    // word kd of row r at kd ^ 8 (r / 16 % 4): the 16-byte pieces stay whole and the reads below spread over the banks
    const int r = 32 * i + rg, pos = (sub * 4) ^ (((r >> 4) & 3) << 3);
    *(u32x4*)(tile + r * kScaleBlock + pos * 4) = w;
  }
  __syncthreads();
  // 16 rows (of g) of 4 columns a thread: 16 words, transposed as 4 x 4 bytes
  const int mg = t & 7, kd = t >> 3, pos = kd ^ ((mg & 3) << 3);
  u32x4 out[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = *(const uint32_t*)(tile + (mg * 16 + 4 * j + e) * kScaleBlock + pos * 4);
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
      const int n = n0 + 4 * kd + b;
      if (n < p.n) put_bytes(p.qt + (int64_t)n * p.ldqt + mm, p.m - mm, out[b]);
    }
  }
}

template <int E>
hipError_t launch_e(const EpilogBackArgs& p, hipStream_t s) {
  const int tiles_n = (p.n + kScaleBlock - 1) / kScaleBlock;
  const unsigned grid = (unsigned)((int64_t)((p.m + kScaleBlock - 1) / kScaleBlock) * tiles_n);
  if (p.act == ACT_RELU) epilogue_back_kernel<E, ACT_RELU><<<grid, kThreads, 0, s>>>(p, tiles_n);
  else if (p.act == ACT_GELU) epilogue_back_kernel<E, ACT_GELU><<<grid, kThreads, 0, s>>>(p, tiles_n);
  else if (p.act == ACT_SILU) epilogue_back_kernel<E, ACT_SILU><<<grid, kThreads, 0, s>>>(p, tiles_n);
  else epilogue_back_kernel<E, ACT_NONE><<<grid, kThreads, 0, s>>>(p, tiles_n);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_epilogue_backward(int elt, const EpilogBackArgs& p, hipStream_t s) {
  if (elt == EL_F16) return launch_e<EL_F16>(p, s);
  if (elt == EL_BF16) return launch_e<EL_BF16>(p, s);
  return launch_e<EL_F32>(p, s);
}

}  // namespace ep
