// Mixture-of-experts row movement: the order of (token, choice) slots by expert, tokens copied (or
// quantised) into that order, their weighted return, and the gradients of the return.
//
// Every kernel but the order is bound by HBM: it is one pass over the expert rows, walked by token, so
// that a token's row is read (or written) once whatever the number of its choices.  8192 tokens, 8 of 64 experts,
// 5120 bf16 features: combined in 132 us (5.5 TB/s), their gradients in 297 (4.7), ordered and dispatched in 159
// (the order 14 of them); a large device copy reaches 5.1 TB/s, a fill 6.9.
#include "fp8_device.hpp"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kOrderThreads = 512;
constexpr int kOrderWaves = kOrderThreads / 64;
constexpr int kMaxExperts = 1024;
constexpr int kOrderSlots = 1024;   // slots a workgroup of the order takes, at least
constexpr int kOrderBlocksMax = 128;

// --------------------------------------------------------------------------------- order
// Stable counting sort by expert in two launches: each workgroup counts its run of slots, then every
// workgroup sums the counts before its own (at most 128 x experts words, from L2), places its slots in
// order and writes the padding of some experts.  A run of at most 1024 slots needs one workgroup and
// one launch.
__device__ __forceinline__ int slot_expert(const OrderArgs& p, int i) {
  int64_t e = p.id_bytes == 8 ? ((const int64_t*)p.ids)[i] : (int64_t)((const int*)p.ids)[i];
  return e >= 0 && e < p.experts ? (int)e : -1;
}

__device__ __forceinline__ int run_length(const OrderArgs& p, int blocks) {
  const int run = (p.slots + blocks - 1) / blocks;
  return (run + kOrderThreads - 1) / kOrderThreads * kOrderThreads;
}

__global__ __launch_bounds__(kOrderThreads) void order_count_kernel(OrderArgs p) {
  __shared__ int cnt[kMaxExperts];
  for (int e = threadIdx.x; e < p.experts; e += kOrderThreads) cnt[e] = 0;
  __syncthreads();
  const int run = run_length(p, (int)gridDim.x);
  const int64_t i0 = (int64_t)blockIdx.x * run;
  const int64_t i1 = i0 + run < p.slots ? i0 + run : p.slots;
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kOrderThreads) {
    const int e = slot_expert(p, (int)i);
    if (e >= 0) atomicAdd(&cnt[e], 1);  // (whole numbers: the order of additions does not matter)
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.experts; e += kOrderThreads) p.hist[(int64_t)blockIdx.x * p.experts + e] = cnt[e];
}

template <bool ONE>
__global__ __launch_bounds__(kOrderThreads) void order_place_kernel(OrderArgs p) {
  __shared__ int total[kMaxExperts];           // slots of each expert
  __shared__ int next[kMaxExperts];            // rows this workgroup's next slots of each expert take
  __shared__ int cnt[kOrderWaves][kMaxExperts];
  __shared__ int part[kOrderWaves];
  const int t = threadIdx.x, lane = lane_id(), wave = wave_id(), E = p.experts;
  const int run = ONE ? (p.slots + kOrderThreads - 1) / kOrderThreads * kOrderThreads : run_length(p, (int)gridDim.x);
  const int64_t i0 = (int64_t)blockIdx.x * run;
  const int64_t i1 = i0 + run < p.slots ? i0 + run : p.slots;
  if constexpr (ONE) {
    for (int e = t; e < E; e += kOrderThreads) total[e] = 0;
    __syncthreads();
    for (int64_t i = t; i < i1; i += kOrderThreads) {
      const int e = slot_expert(p, (int)i);
      if (e >= 0) atomicAdd(&total[e], 1);
    }
    for (int e = t; e < E; e += kOrderThreads) next[e] = 0;
    __syncthreads();
  } else {
    for (int e = t; e < E; e += kOrderThreads) total[e] = next[e] = 0;
    __syncthreads();
    // every thread takes words of the whole table, 8 loads at a time (whole numbers: the order of additions
    // does not matter)
    const int words = (int)gridDim.x * E, mine = (int)blockIdx.x * E;
    for (int k0 = t; k0 < words; k0 += 8 * kOrderThreads) {
      int v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = k0 + u * kOrderThreads < words ? p.hist[k0 + u * kOrderThreads] : 0;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int k = k0 + u * kOrderThreads;
        if (v[u]) {
          atomicAdd(&total[k % E], v[u]);
          if (k < mine) atomicAdd(&next[k % E], v[u]);
        }
      }
    }
    __syncthreads();
  }
  // exclusive sums of the padded counts, kOrderThreads experts at a time
  int base = 0;
  for (int e0 = 0; e0 < E; e0 += kOrderThreads) {
    const int e = e0 + t;
    const int c = e < E ? total[e] : 0;
    const int padded = (c + p.align - 1) / p.align * p.align;
    int sum = padded;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(sum, d);
      if (lane >= d) sum += v;
    }
    if (lane == 63) part[wave] = sum;
    __syncthreads();
    int before = base, whole = 0;
#pragma unroll
    for (int w = 0; w < kOrderWaves; ++w) {
      before += w < wave ? part[w] : 0;
      whole += part[w];
    }
    const int first = before + sum - padded;
    if (e < E) {
      next[e] += first;
      if (blockIdx.x == 0) {
        p.offsets[e] = first;
        if (e == E - 1) p.offsets[E] = first + padded;
      }
      // padding rows, the experts dealt out to the workgroups
      if (e % (int)gridDim.x == (int)blockIdx.x)
        for (int r = first + c; r < first + padded; ++r) p.src[r] = -1;
    }
    base += whole;
    __syncthreads();
  }
  for (int64_t r = base + (int64_t)blockIdx.x * kOrderThreads + t; r < p.capacity; r += (int64_t)gridDim.x * kOrderThreads)
    p.src[r] = -1;
  // kOrderThreads slots at a time: a slot's place is its expert's next row, plus the same expert's slots in the
  // waves before and in the lanes before
  int bits = 0;
  while ((1 << bits) < E) ++bits;
  for (int64_t i = i0; i < i1; i += kOrderThreads) {
    const int64_t slot = i + t;
    const int e = slot < i1 ? slot_expert(p, (int)slot) : -1;
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t on = __ballot((e >> b) & 1);
      same &= ((e >> b) & 1) ? on : ~on;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    for (int k = t; k < E * kOrderWaves; k += kOrderThreads) cnt[k / E][k % E] = 0;
    __syncthreads();
    if (e >= 0 && rank == 0) cnt[wave][e] = __popcll(same);
    __syncthreads();
    int row = -1;
    if (e >= 0) {
      row = next[e] + rank;
      for (int w = 0; w < wave; ++w) row += cnt[w][e];
    }
    if (slot < i1) {
      p.pos[slot] = row;
      if (row >= 0 && row < p.capacity) p.src[row] = (int)slot;
    }
    __syncthreads();
    for (int k = t; k < E; k += kOrderThreads) {
      int add = 0;
#pragma unroll
      for (int w = 0; w < kOrderWaves; ++w) add += cnt[w][k];
      next[k] += add;
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------------------ row kernels
// A workgroup takes one token and up to kSpan features; further features go to blockIdx.y.  Behind the
// tokens' workgroups come those of the padding rows, 64 rows each.
constexpr int kSpan = kThreads * 8;
constexpr int kPadRows = 64;

// Expert rows that no cache holds (the Infinity Cache is 256 MB) pass non-temporally: 8192 tokens to 64 experts,
// 8 choices, 5120 features, ordered and dispatched in 159 us (180 without), combined in 132 (150), the gradients in
// 297 (317).
// Smaller ones are likely in a cache when the next kernel reads them.
constexpr int64_t kStreamBytes = (int64_t)256 << 20;
bool streams(int elt, const ExpertRows& p) { return (int64_t)p.rows * p.h * elt_size(elt) > kStreamBytes; }

// zeros in the padding rows (src < 0) among rows r0 .. r0 + 63, and the scale of an empty block
template <int E, bool Q, bool NT>
__device__ void pad_rows(const ExpertRows& p, int64_t r0) {
  const int es = Q ? 1 : elt_size(E);
  for (int64_t r = r0 + wave_id(); r < r0 + kPadRows && r < p.rows; r += kThreads / 64) {
    if (__builtin_amdgcn_readfirstlane(p.src[r]) >= 0) continue;
    char* o = (char*)p.out + r * p.ldo * es;
    const int64_t bytes = (int64_t)p.h * es;
    for (int64_t c = lane_id() * 16; c < bytes; c += 64 * 16) {
      if (c + 16 <= bytes) put16<NT>(o + c, u32x4{0, 0, 0, 0});
      else
        for (int64_t b = c; b < bytes; ++b) o[b] = 0;
    }
    if constexpr (Q) {
      for (int kb = lane_id(); kb * kScaleBlock < p.h; kb += 64) p.scale[(int64_t)kb * p.rows + r] = scale_of(kAmaxMin);
    }
  }
}

template <int E, bool Q, bool NT>
__global__ __launch_bounds__(kThreads) void dispatch_kernel(ExpertRows p, int token_blocks) {
  const int bx = (int)blockIdx.x;
  if (bx >= token_blocks) {
    if (blockIdx.y == 0) pad_rows<E, Q, NT>(p, (int64_t)(bx - token_blocks) * kPadRows);
    return;
  }
  const int c = (int)blockIdx.y * kSpan + (int)threadIdx.x * 8;
  const int n = p.h - c;
  const int64_t token = bx;
  float f[8];
  if constexpr (Q) {
    load8<E>((const char*)p.x + (token * p.ldx + c) * elt_size(E), n, f);
    float amax = kAmaxMin;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, finite_abs(f[i]));
#pragma unroll
    for (int d = 1; d < 16; d *= 2) amax = fmaxf(amax, __shfl_xor(amax, d));
    const float inv = scale_inv(amax);
    const u32x2 w = {to_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                     to_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv)};
    for (int j = 0; j < p.topk; ++j) {
      const int r = p.pos[token * p.topk + j];
      if (r < 0 || r >= p.rows || n <= 0) continue;
      uint8_t* o = (uint8_t*)p.out + (int64_t)r * p.ldo + c;
      if (n >= 8) {
        *(u32x2_u*)o = w;
      } else {
        for (int i = 0; i < n; ++i) o[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
      }
      if ((threadIdx.x & 15) == 0) p.scale[(int64_t)(c / kScaleBlock) * p.rows + r] = scale_of(amax);
    }
  } else {
    if (n <= 0) return;
    // (copied as bits: NaN payloads and subnormals pass unchanged)
    const char* x = (const char*)p.x + (token * p.ldx + c) * 2;
    if (n >= 8) {
      const u32x4 w = *(const u32x4_u*)x;
      for (int j = 0; j < p.topk; ++j) {
        const int r = p.pos[token * p.topk + j];
        if (r >= 0 && r < p.rows) put16<NT>((char*)p.out + ((int64_t)r * p.ldo + c) * 2, w);
      }
    } else {
      for (int j = 0; j < p.topk; ++j) {
        const int r = p.pos[token * p.topk + j];
        if (r < 0 || r >= p.rows) continue;
        uint16_t* o = (uint16_t*)p.out + (int64_t)r * p.ldo + c;
        for (int i = 0; i < n; ++i) o[i] = ((const uint16_t*)x)[i];
      }
    }
  }
}

// out[t] = sum over a token's kept choices of w * y[row], in choice order, summed in fp32
template <int E, bool NT>
__global__ __launch_bounds__(kThreads) void combine_kernel(ExpertRows p) {
  const int c = (int)blockIdx.y * kSpan + (int)threadIdx.x * 8;
  const int n = p.h - c;
  if (n <= 0) return;
  const int64_t token = blockIdx.x;
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
  for (int j = 0; j < p.topk; ++j) {
    const int r = p.pos[token * p.topk + j];
    if (r < 0 || r >= p.rows) continue;
    const float w = p.w ? p.w[token * p.ldw + j] : 1.0f;
    float f[8];
    load8<E, NT>((const char*)p.x + ((int64_t)r * p.ldx + c) * elt_size(E), n, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += w * f[i];
  }
  store8<E, NT>((char*)p.out + (token * p.ldo + c) * elt_size(E), n, acc);
}

// dy[row] = w * dout[t]; dw[t][j] = sum over the features of y[row] * dout[t].  One workgroup walks a
// token's whole row, so dw needs no second pass; padding rows' dy are zeros.
// choices whose sums are held at once (fp32: 8 take more scalar registers than there are)
template <int E>
constexpr int kChoicesOf = E == EL_F32 ? 4 : 8;
template <int E, bool NT>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(ExpertRows p, int token_blocks) {
  constexpr int kChoices = kChoicesOf<E>;
  __shared__ float red[kThreads / 64][kChoices];
  const int bx = (int)blockIdx.x;
  if (bx >= token_blocks) {
    pad_rows<E, false, NT>(p, (int64_t)(bx - token_blocks) * kPadRows);
    return;
  }
  const int64_t token = bx;
  for (int j0 = 0; j0 < p.topk; j0 += kChoices) {
    int row[kChoices];
    float w[kChoices], dot[kChoices];
#pragma unroll
    for (int j = 0; j < kChoices; ++j) {
      const bool in = j0 + j < p.topk;
      const int r = in ? p.pos[token * p.topk + j0 + j] : -1;
      row[j] = r >= 0 && r < p.rows ? r : -1;
      w[j] = in ? (p.w ? p.w[token * p.ldw + j0 + j] : 1.0f) : 0.0f;
      asm("" : "+v"(w[j]));  // (uniform, but the scalar registers are short)
      dot[j] = 0.0f;
    }
    const int h8 = p.h & ~7;
    for (int c = (int)threadIdx.x * 8; c < h8; c += kSpan) {
      float g[8];
      load8<E>((const char*)p.dout + (token * p.ld_dout + c) * elt_size(E), 8, g);
#pragma unroll
      for (int j = 0; j < kChoices; ++j) {
        if (row[j] < 0) continue;
        float y[8], o[8];
        load8<E, NT>((const char*)p.x + ((int64_t)row[j] * p.ldx + c) * elt_size(E), 8, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dot[j] += y[i] * g[i];
          o[i] = w[j] * g[i];
        }
        store8<E, NT>((char*)p.out + ((int64_t)row[j] * p.ldo + c) * elt_size(E), 8, o);
      }
    }
    const int c = h8 + (int)threadIdx.x;  // the last features, one a thread
    if (c < p.h) {
      const float g = load_elt<E>((const char*)p.dout + (token * p.ld_dout + c) * elt_size(E));
#pragma unroll
      for (int j = 0; j < kChoices; ++j) {
        if (row[j] < 0) continue;
        dot[j] += load_elt<E>((const char*)p.x + ((int64_t)row[j] * p.ldx + c) * elt_size(E)) * g;
        store_elt<E>((char*)p.out + ((int64_t)row[j] * p.ldo + c) * elt_size(E), w[j] * g);
      }
    }
#pragma unroll
    for (int j = 0; j < kChoices; ++j) {
#pragma unroll
      for (int d = 1; d < 64; d *= 2) dot[j] += __shfl_xor(dot[j], d);
      if (lane_id() == 0) red[wave_id()][j] = dot[j];
    }
    __syncthreads();
    const int j = (int)threadIdx.x;
    if (j < kChoices && j0 + j < p.topk)
      p.dw[token * p.topk + j0 + j] = (red[0][j] + red[1][j]) + (red[2][j] + red[3][j]);
    __syncthreads();
  }
}

unsigned pad_blocks(const ExpertRows& p) { return (unsigned)((p.rows + kPadRows - 1) / kPadRows); }
unsigned spans(const ExpertRows& p) { return (unsigned)((p.h + kSpan - 1) / kSpan); }

}  // namespace

int order_blocks(int slots) {
  const int b = (slots + kOrderSlots - 1) / kOrderSlots;
  return b < kOrderBlocksMax ? b : kOrderBlocksMax;
}

hipError_t launch_order(const OrderArgs& p, hipStream_t s) {
  const int blocks = order_blocks(p.slots);
  if (blocks <= 1) {
    order_place_kernel<true><<<1, kOrderThreads, 0, s>>>(p);
  } else {
    order_count_kernel<<<blocks, kOrderThreads, 0, s>>>(p);
    order_place_kernel<false><<<blocks, kOrderThreads, 0, s>>>(p);
  }
  return hipGetLastError();
}

namespace {

template <int E, bool Q>
void start_dispatch(bool nt, const ExpertRows& p, hipStream_t s) {
  const dim3 grid((unsigned)p.tokens + pad_blocks(p), spans(p));
  if (nt) dispatch_kernel<E, Q, true><<<grid, kThreads, 0, s>>>(p, p.tokens);
  else dispatch_kernel<E, Q, false><<<grid, kThreads, 0, s>>>(p, p.tokens);
}

template <int E>
void start_combine(const ExpertRows& p, hipStream_t s) {
  const dim3 grid((unsigned)p.tokens, spans(p));
  if (streams(E, p)) combine_kernel<E, true><<<grid, kThreads, 0, s>>>(p);
  else combine_kernel<E, false><<<grid, kThreads, 0, s>>>(p);
}

template <int E>
void start_combine_backward(const ExpertRows& p, hipStream_t s) {
  const unsigned grid = (unsigned)p.tokens + pad_blocks(p);
  if (streams(E, p)) combine_backward_kernel<E, true><<<grid, kThreads, 0, s>>>(p, p.tokens);
  else combine_backward_kernel<E, false><<<grid, kThreads, 0, s>>>(p, p.tokens);
}

}  // namespace

hipError_t launch_dispatch(int elt, bool quantize, const ExpertRows& p, hipStream_t s) {
  if (!quantize) {
    ExpertRows q = p;  // (moved as 16-bit pieces, whatever the type)
    if (elt == EL_F32) {
      q.h *= 2;
      q.ldx *= 2;
      q.ldo *= 2;
    }
    start_dispatch<EL_F16, false>(streams(elt, p), q, s);
  } else if (elt == EL_F32) start_dispatch<EL_F32, true>(false, p, s);
  else if (elt == EL_F16) start_dispatch<EL_F16, true>(false, p, s);
  else start_dispatch<EL_BF16, true>(false, p, s);
  return hipGetLastError();
}

hipError_t launch_combine(int elt, const ExpertRows& p, hipStream_t s) {
  if (elt == EL_F16) start_combine<EL_F16>(p, s);
  else if (elt == EL_BF16) start_combine<EL_BF16>(p, s);
  else start_combine<EL_F32>(p, s);
  return hipGetLastError();
}

hipError_t launch_combine_backward(int elt, const ExpertRows& p, hipStream_t s) {
  if (elt == EL_F16) start_combine_backward<EL_F16>(p, s);
  else if (elt == EL_BF16) start_combine_backward<EL_BF16>(p, s);
  else start_combine_backward<EL_F32>(p, s);
  return hipGetLastError();
}

}  // namespace ep
