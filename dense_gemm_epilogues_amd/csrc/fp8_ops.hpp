// Interface between the C ABI of the 8-bit and expert operators (fp8_api.cpp) and their kernels
// (fp8_gemm.hip, fp8_quantize.hip, experts.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ep {

// element types of activations and outputs (0 and 1 as DType of ep_internal.hpp)
enum Elt : int { EL_F16 = 0, EL_BF16 = 1, EL_F32 = 2 };
constexpr int elt_size(int e) { return e == EL_F32 ? 4 : 2; }

constexpr int kScaleBlock = 128;       // k-values per scale
constexpr float kF8Max = 448.0f;       // largest finite e4m3 value
constexpr float kAmaxMin = 0x1p-90f;   // smallest block maximum a scale is made from

// D[m][n] = sum over k-blocks of sa[m][kb] sb[n / 128][kb] sum_{k in kb} a[m][k] b[n][k]
struct Fp8Gemm {
  const uint8_t* a;
  const uint8_t* b;
  const float* sa;
  const float* sb;
  void* d;
  int64_t lda, ldb, ldd;             // elements (bytes for a and b)
  int64_t sa_m, sa_k, sb_n, sb_k;    // scale strides, elements
  int64_t b_e, sb_e;                 // grouped: strides between experts
  const int* offsets;                // grouped, weight gradient: [experts + 1]
  int experts;
  int M, N, K;                       // grouped: M = all rows; weight gradient: K = all rows
  int tiles_m, tiles_n;
  int splits, kb_per_split;          // matmul: K ranges, each into its own part of `part`
  float* part;                       // [splits][M][N]
  int cus;                           // of the device
};

// what follows a product: P = a b^T + bias, D = act(P) + residual
enum Activation : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_SILU = 3 };
struct Fp8Epilog {
  const void* bias;                  // [N], or null
  const void* res;                   // [M][N] of D's type, or null
  void* pre;                         // [M][N] of D's type: P, or null
  int64_t ld_res, ld_pre;
  int act;
  int bias32;                        // bias is fp32, else of D's type
};
struct Fp8GemmEpilog : Fp8Gemm {
  Fp8Epilog e;
};

enum GemmMode : int { GM_MATMUL = 0, GM_GROUPED = 1, GM_WGRAD = 2 };

hipError_t launch_fp8_tiles(int mode, int out, Fp8Gemm& p, hipStream_t s);
// few rows: b streams past them
hipError_t launch_fp8_rows(int mode, int out, Fp8Gemm& p, hipStream_t s);
int fp8_splits(int m, int n, int k);
// the same of a plain product with an epilogue; few: a few rows
hipError_t launch_fp8_epilog(int out, bool few, Fp8GemmEpilog& p, hipStream_t s);

struct QuantArgs {
  const void* x;
  int64_t ldx;                       // elements
  int m, k;                          // of x
  uint8_t* q;
  int64_t ldq;
  float* scale;                      // rows 1: [ceil][rows], features outermost; rows 128: [blocks][blocks]
};
// workgroups of a quantisation (m x k as given): 8 rows by 4 blocks of 1 x 128 each, or a tile of 128 x 128
constexpr int64_t quantize_blocks(int rows, bool transpose, int64_t m, int64_t k) {
  const int64_t kb = (k + kScaleBlock - 1) / kScaleBlock;
  return rows == 1 && !transpose ? (kb + 3) / 4 * ((m + 7) / 8) : kb * ((m + kScaleBlock - 1) / kScaleBlock);
}
hipError_t launch_quantize(int elt, int rows, bool transpose, const QuantArgs& p, hipStream_t s);

struct OrderArgs {
  const void* ids;                   // [slots] int32 or int64
  int id_bytes;
  int slots, experts, align, capacity;
  int* pos;                          // [slots]
  int* src;                          // [capacity]
  int* offsets;                      // [experts + 1]
  int* hist;                         // workspace [blocks][experts]
};
int order_blocks(int slots);
hipError_t launch_order(const OrderArgs& p, hipStream_t s);

struct ExpertRows {
  const void* x;                     // dispatch: tokens [T][h]; combine: expert rows [rows][h]
  int64_t ldx;
  const void* dout;                  // combine backward: [T][h]
  int64_t ld_dout;
  void* out;                         // dispatch: rows; combine: tokens; backward: dy rows
  int64_t ldo;
  const int* pos;                    // [T][topk]
  const int* src;                    // [rows]
  const float* w;                    // [T][topk], or null: ones
  int64_t ldw;
  float* dw;                         // backward: [T][topk]
  float* scale;                      // dispatch with quantisation: [ceil(h/128)][rows]
  int tokens, topk, rows, h;
};
hipError_t launch_dispatch(int elt, bool quantize, const ExpertRows& p, hipStream_t s);
hipError_t launch_combine(int elt, const ExpertRows& p, hipStream_t s);
hipError_t launch_combine_backward(int elt, const ExpertRows& p, hipStream_t s);

}  // namespace ep
