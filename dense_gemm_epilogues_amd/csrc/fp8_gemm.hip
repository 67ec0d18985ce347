// e4m3 matrix products with block scales, on v_mfma_f32_16x16x128_f8f6f4: plain, grouped by expert,
// and the experts' weight gradients.
//
//   D[m][n] = sum over blocks kb of 128 k-values of sa[m][kb] sb[n / 128][kb] P_kb[m][n],
//   P_kb[m][n] = sum_{k in kb} a[m][k] b[n][k].
//
// One such MFMA spans exactly one scale block (K = 128), so P_kb of a 16 x 16 block is the result of
// one instruction started from zero, and D gains it by one fp32 multiply-add per value with the factor
// t = sa sb.  The operands go in swapped (b's rows first): a lane then holds 4 neighbouring n of ONE
// row m = lane % 16, so t is one register per 16 rows of a.
//
// How exact the sums are.  That instruction (as every e4m3 MFMA of gfx950) adds the products of 8
// neighbouring k in fixed point, 14 bits below the largest of them, before its fp32 accumulator:
// measured, normal operands give sums off by 1.5e-5 of the result's norm per block (fp32 sums: 1e-8).
// Next to a bf16 or fp16 output's rounding (1.7e-3, 2.1e-4 of the norm) that is nothing, and it is the
// unit's only way to its full rate.  Where it would show or buys nothing the operands are widened to
// fp16 first, which holds every e4m3 value, and multiplied by v_mfma_f32_16x16x32_f16, whose sums are
// fp32 throughout (WIDE): fp32 outputs, sums of at most 256 values (bound by the output's bytes), and
// the few-row kernel (bound by the weights').
#include "fp8_device.hpp"

namespace ep {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr uint32_t kOOB = 0x80000000u;  // a buffer offset past every extent

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* base, int64_t bytes) {
  const uint32_t n = bytes <= 0 ? 0u : (bytes >= 0x7fffffffLL ? 0x7fffffffu : (uint32_t)bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)n, 0x00020000);
}

__device__ __forceinline__ f32x4 mfma128(i32x8 x, i32x8 y) {
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  // formats e4m3 (0, 0) and no block exponents: the plain v_mfma_f32_16x16x128_f8f6f4
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, zero, 0, 0, 0, 0, 0, 0);
}

// 32 e4m3 values as fp16, 8 at a time
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
struct Wide {
  f16x8 v[4];
};
__device__ __forceinline__ Wide widen(i32x8 x) {
  Wide w;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const half2_t lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x[2 * g + h], 1.0f, false);
      const half2_t hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x[2 * g + h], 1.0f, true);
      w.v[g][4 * h] = lo[0];
      w.v[g][4 * h + 1] = lo[1];
      w.v[g][4 * h + 2] = hi[0];
      w.v[g][4 * h + 3] = hi[1];
    }
  }
  return w;
}
__device__ __forceinline__ f32x4 mfma128(const Wide& x, const Wide& y) {
  f32x4 c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int g = 0; g < 4; ++g) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(x.v[g], y.v[g], c, 0, 0, 0);
  return c;
}
template <bool WIDE>
struct FragOf {
  typedef i32x8 type;
  static __device__ __forceinline__ i32x8 of(i32x8 x) { return x; }
};
template <>
struct FragOf<true> {
  typedef Wide type;
  static __device__ __forceinline__ Wide of(i32x8 x) { return widen(x); }
};

__device__ __forceinline__ i32x8 join8(u32x4 a, u32x4 b) {
  return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// Workgroups go round-robin over the 8 XCDs: place `bid` of `n` in an order whose contiguous eighths
// run on one XCD each, so that neighbouring tiles share an L2.
__device__ __forceinline__ int xcd_order(int bid, int n) {
  const int x = bid & 7, l = bid >> 3, q = n >> 3, r = n & 7;
  return x < r ? x * (q + 1) + l : r * (q + 1) + (x - r) * q + l;
}

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return min(max(v, lo), hi); }

// rows of group e, kept inside [0, rows] whatever the offsets hold
__device__ __forceinline__ void group_rows(const int* offsets, int e, int rows, int& r0, int& r1) {
  r0 = clampi(offsets[e], 0, rows);
  r1 = clampi(offsets[e + 1], r0, rows);
}

__device__ __forceinline__ int wave_scan(int v) {  // inclusive sum over the lanes
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int u = __shfl_up(v, d);
    if (lane_id() >= d) v += u;
  }
  return v;
}

template <int OT>
__device__ __forceinline__ void store_row8(char* d, int n, f32x4 lo, f32x4 hi) {
  const float f[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  store8<OT>(d, n, f);
}

// ---------------------------------------------------------------------------------------- tiles
constexpr int kGroupM = 8;

// BM x BN tiles of D, WGM x WGN waves; both operands go through LDS in a ring of two stages of one
// scale block (128 bytes a row: one cache line, 8 lanes of 16 bytes), filled by buffer loads that
// write LDS while the stage before is computed.  16-byte piece c of row r is kept at piece c ^ (r & 7),
// which the fragment reads (16 rows at one piece per 16 lanes) take without bank conflicts.  Within
// each 32 rows of b, LDS row 16 u + 4 q + i holds n = 8 q + 4 u + i, so that a lane's values of two
// neighbouring blocks are 8 neighbouring n: a 16-byte store.
template <int MODE, int OT, int BM, int BN, int WGM, int WGN, bool WIDE>
__global__ __launch_bounds__(64 * WGM * WGN) __attribute__((amdgpu_waves_per_eu(2)))
void fp8_tile_kernel(Fp8Gemm p) {
  constexpr int WAVES = WGM * WGN, WTM = BM / WGM, WTN = BN / WGN, MT = WTM / 16, NT = WTN / 16;
  constexpr int SLOTS = (BM + BN) / 8, PER_WAVE = SLOTS / WAVES, STAGE = (BM + BN) * 128;
  static_assert(SLOTS % WAVES == 0 && (BM / 8) % PER_WAVE == 0 && NT % 2 == 0 && WTN <= 128 && 128 % WTN == 0, "tile");
  __shared__ __align__(128) char lds[2 * STAGE];
  const int lane = lane_id(), wave = wave_id();
  const int wm = wave / WGN, wn = wave % WGN;

  // ---- which tile
  int m0, mv, n0, kb0, kb1, klen;  // rows from m0, mv of them; columns from n0; scale blocks kb0 .. kb1
  const uint8_t *a = p.a, *b = p.b;
  const float *sa = p.sa, *sb = p.sb;
  char* d = (char*)p.d;
  bool zero_only = false, poison = false;
  if constexpr (MODE == GM_MATMUL) {
    const int tiles = p.tiles_m * p.tiles_n;
    const int split = (int)blockIdx.x / tiles;
    const int t = xcd_order((int)blockIdx.x - split * tiles, tiles);
    const int group = kGroupM * p.tiles_n, g = t / group, first = g * kGroupM;
    const int gm = min(p.tiles_m - first, kGroupM), w = t - g * group;
    m0 = (first + w % gm) * BM;
    n0 = (w / gm) * BN;
    mv = min(BM, p.M - m0);
    kb0 = split * p.kb_per_split;
    kb1 = min(kb0 + p.kb_per_split, (p.K + kScaleBlock - 1) / kScaleBlock);
    klen = p.K;
    if (p.splits > 1) d = (char*)(p.part + (int64_t)split * p.M * p.N);
  } else if constexpr (MODE == GM_GROUPED) {
    // tiles of the groups in order, then those of the rows behind the last group, which are zeroed
    int base = 0, total = 0;
    const int last = clampi(p.offsets[p.experts], 0, p.M);
    const int tail = (p.M - last + BM - 1) / BM;
    for (int e0 = 0; e0 < p.experts; e0 += 64) {
      int r0 = 0, r1 = 0;
      if (e0 + lane < p.experts) group_rows(p.offsets, e0 + lane, p.M, r0, r1);
      total += __shfl(wave_scan((r1 - r0 + BM - 1) / BM), 63);
    }
    const int tiles = (total + tail) * p.tiles_n;
    if ((int)blockIdx.x >= tiles) return;
    const int t = xcd_order((int)blockIdx.x, tiles);
    int e = p.experts, first = total, cnt = tail, r0 = last, r1 = p.M;
    for (int e0 = 0; e0 < p.experts; e0 += 64) {
      int q0 = 0, q1 = 0;
      if (e0 + lane < p.experts) group_rows(p.offsets, e0 + lane, p.M, q0, q1);
      const int c = (q1 - q0 + BM - 1) / BM;
      const int ends = base + wave_scan(c);
      const uint64_t past = __ballot(ends * p.tiles_n > t);
      if (past) {
        const int l = __builtin_ctzll(past);
        e = e0 + l;
        cnt = __shfl(c, l);
        first = __shfl(ends, l) - cnt;
        r0 = __shfl(q0, l);
        r1 = __shfl(q1, l);
        break;
      }
      base = __shfl(ends, 63);
    }
    e = __builtin_amdgcn_readfirstlane(e);
    cnt = __builtin_amdgcn_readfirstlane(cnt);
    first = __builtin_amdgcn_readfirstlane(first);
    r0 = __builtin_amdgcn_readfirstlane(r0);
    r1 = __builtin_amdgcn_readfirstlane(r1);
    const int w = t - first * p.tiles_n;
    m0 = r0 + (w % cnt) * BM;
    n0 = (w / cnt) * BN;
    mv = min(BM, r1 - m0);
    zero_only = e == p.experts;
    if (!zero_only) {
      b += (int64_t)e * p.b_e;
      sb += (int64_t)e * p.sb_e;
    }
    kb0 = 0;
    kb1 = zero_only ? 0 : (p.K + kScaleBlock - 1) / kScaleBlock;
    klen = p.K;
  } else {
    const int tiles = p.tiles_m * p.tiles_n;
    const int u = xcd_order((int)blockIdx.x, tiles * p.experts);
    const int e = u / tiles, t = u - e * tiles;
    const int group = kGroupM * p.tiles_n, g = t / group, first = g * kGroupM;
    const int gm = min(p.tiles_m - first, kGroupM), w = t - g * group;
    m0 = (first + w % gm) * BM;
    n0 = (w / gm) * BN;
    mv = min(BM, p.M - m0);
    int r0, r1;
    group_rows(p.offsets, e, p.K, r0, r1);
    r0 = __builtin_amdgcn_readfirstlane(r0);
    r1 = __builtin_amdgcn_readfirstlane(r1);
    // a group that does not start and end on scale blocks has no scales of its own: NaN
    poison = (r0 | r1) % kScaleBlock != 0;
    kb0 = r0 / kScaleBlock;
    kb1 = poison ? kb0 : r1 / kScaleBlock;
    klen = r1;
    d += (int64_t)e * p.M * p.ldd * elt_size(OT);
  }
  const int nv = min(BN, p.N - n0);
  a += (int64_t)m0 * p.lda + (int64_t)kb0 * kScaleBlock;
  b += (int64_t)n0 * p.ldb + (int64_t)kb0 * kScaleBlock;
  klen -= kb0 * kScaleBlock;
  const int nkb = kb1 - kb0;

  // ---- loads: slot s of a stage is 8 rows; a wave's slots are neighbours and all of one operand
  const bool a_side = wave * PER_WAVE < BM / 8;
  const int64_t ld = a_side ? p.lda : p.ldb;
  const int rows = a_side ? mv : nv;
  const __amdgpu_buffer_rsrc_t rs = rsrc_of(a_side ? a : b, (int64_t)(rows - 1) * ld + klen);
  const int piece = (lane & 7) ^ (lane >> 3);
  uint32_t voff[PER_WAVE];
#pragma unroll
  for (int s = 0; s < PER_WAVE; ++s) {
    int r = (wave * PER_WAVE + s) * 8 + (lane >> 3);
    if (!a_side) {
      r -= BM;
      const int u = (r >> 4) & 1, q = (r >> 2) & 3, i = r & 3;
      r = (r & ~31) + 8 * q + 4 * u + i;
    }
    voff[s] = r < rows ? (uint32_t)(r * ld) + piece * 16 : kOOB;
    asm("" : "+v"(voff[s]));  // (computed once, not again in every step)
  }
  auto issue = [&](int kb, int stage) __attribute__((always_inline)) {
    const int k0 = kb * kScaleBlock;
    const bool in = k0 + piece * 16 < klen;  // (k is a multiple of 16: pieces are whole or absent)
    char* dst = lds + stage * STAGE + wave * PER_WAVE * 1024;
#pragma unroll
    for (int s = 0; s < PER_WAVE; ++s)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(dst + s * 1024), 16,
                                               (int)(in ? voff[s] : kOOB), k0, 0, 0);
  };
  // ---- scales of this wave's rows and its 128 columns
  const float* sap = sa + (int64_t)m0 * p.sa_m + (int64_t)kb0 * p.sa_k;
  const float* sbp = sb + (int64_t)((n0 + wn * WTN) / kScaleBlock) * p.sb_n + (int64_t)kb0 * p.sb_k;
  const bool n_on = n0 + wn * WTN < p.N;
  uint32_t soff[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) soff[i] = (uint32_t)(min(wm * WTM + i * 16 + (lane & 15), mv - 1) * p.sa_m);
  float sn[MT], sbn = 0.0f;
  auto scales = [&](int kb) __attribute__((always_inline)) {
    const float* q = sap + (int64_t)kb * p.sa_k;
#pragma unroll
    for (int i = 0; i < MT; ++i) sn[i] = q[soff[i]];
    sbn = n_on ? sbp[(int64_t)kb * p.sb_k] : 0.0f;
  };

  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const bool active = wm * WTM < mv && n_on;  // (the other waves only load)

  const int frow = (lane & 15) * 128, fpiece = ((lane >> 4) ^ (lane & 7)) * 16;
  auto frag = [&](const char* base, int block) __attribute__((always_inline)) {
    const char* r = base + block * 2048 + frow;
    return FragOf<WIDE>::of(join8(*(const u32x4*)(r + fpiece), *(const u32x4*)(r + (fpiece ^ 64))));
  };
  if (nkb > 0) {
    scales(0);
    issue(0, 0);
  }
  for (int kb = 0; kb < nkb; ++kb) {
    // this wave's loads of the stage have landed; behind the barrier everyone's have, and everyone
    // has read the stage that is loaded next
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0), visible to the compiler's own wait counting
    asm volatile("s_barrier" ::: "memory");
    float t[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) t[i] = sn[i] * sbn;
    if (kb + 1 < nkb) {
      scales(kb + 1);
      issue(kb + 1, (kb + 1) & 1);
    }
    if (active) {
      const char* As = lds + (kb & 1) * STAGE + wm * WTM * 128;
      const char* Bs = lds + (kb & 1) * STAGE + BM * 128 + wn * WTN * 128;
      // one column block of MT MFMAs at a time, the multiply-adds of the block before in their shadow
      typename FragOf<WIDE>::type fa[MT], fb[2];
      f32x4 pr[2][MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) fa[i] = frag(As, i);
      fb[0] = frag(Bs, 0);
      fb[1] = frag(Bs, 1);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          pr[j & 1][i] = mfma128(fb[j & 1], fa[i]);
          __builtin_amdgcn_sched_barrier(0);
          if (j > 0) acc[i][j - 1] += pr[(j - 1) & 1][i] * t[i];
          __builtin_amdgcn_sched_barrier(0);
        }
        if (j + 2 < NT) fb[j & 1] = frag(Bs, j + 2);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[i][NT - 1] += pr[(NT - 1) & 1][i] * t[i];
    }
  }

  // ---- store
  if (!(wm * WTM < mv && n_on)) return;
  if (poison) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = acc[i][j] + __builtin_nanf("");
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = wm * WTM + i * 16 + (lane & 15);
    if (m >= mv) continue;
#pragma unroll
    for (int j = 0; j < NT; j += 2) {
      const int n = wn * WTN + j * 16 + 8 * (lane >> 4);
      if (n >= nv) continue;
      if (MODE == GM_MATMUL && p.splits > 1)
        store_row8<EL_F32>(d + ((int64_t)(m0 + m) * p.N + n0 + n) * 4, nv - n, acc[i][j], acc[i][j + 1]);
      else
        store_row8<OT>(d + ((int64_t)(m0 + m) * p.ldd + n0 + n) * elt_size(OT), nv - n, acc[i][j], acc[i][j + 1]);
    }
  }
}

// D = sum of the K ranges' parts, in their order
template <int OT>
__global__ __launch_bounds__(256) void fp8_join_kernel(Fp8Gemm p) {
  const int64_t mn = (int64_t)p.M * p.N;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < mn; i += (int64_t)gridDim.x * 256 * 8) {
    float f[8], g[8];
    const int n = (int)min((int64_t)8, mn - i);
    load8<EL_F32>((const char*)(p.part + i), n, f);
    for (int s = 1; s < p.splits; ++s) {
      load8<EL_F32>((const char*)(p.part + (int64_t)s * mn + i), n, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] += g[j];
    }
    const int64_t row = i / p.N, col = i - row * p.N;
    char* d = (char*)p.d;
    if (n == 8 && col + 8 <= p.N) {
      store8<OT>(d + (row * p.ldd + col) * elt_size(OT), 8, f);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j >= n) continue;
        const int64_t r = (i + j) / p.N, c = i + j - r * p.N;
        store_elt<OT>(d + (r * p.ldd + c) * elt_size(OT), f[j]);
      }
    }
  }
}

// ----------------------------------------------------------------------------------------- rows
// Few rows of a: bound by reading b once.  A workgroup takes 16 rows of b (columns of D); its waves
// deal out the scale blocks, stream them from memory into registers and join their sums in LDS.
// Rows of a come from the caches, MT x 16 at a time.
template <int MODE, int OT, int MT, int NW>
__global__ __launch_bounds__(64 * NW) void fp8_rows_kernel(Fp8Gemm p) {
  constexpr int U = MT == 1 ? 4 : 2;  // scale blocks in flight per wave
  __shared__ f32x4 red[NW][MT][64];
  const int lane = lane_id(), wave = wave_id();
  const int n0 = (int)blockIdx.x * 16;
  const uint8_t* b = p.b;
  const float* sb = p.sb;
  int r0, r1;
  if constexpr (MODE == GM_GROUPED) {
    // the blockIdx.y-th group that has rows; behind the last one the rows that no group has
    int seen = 0, found = -1;
    for (int e0 = 0; e0 < p.experts && found < 0; e0 += 64) {
      int q0 = 0, q1 = 0;
      if (e0 + lane < p.experts) group_rows(p.offsets, e0 + lane, p.M, q0, q1);
      const int c = wave_scan(q1 > q0 ? 1 : 0);
      const uint64_t hit = __ballot(q1 > q0 && seen + c == (int)blockIdx.y + 1);
      if (hit) {
        const int l = __builtin_ctzll(hit);
        found = e0 + l;
        r0 = __shfl(q0, l);
        r1 = __shfl(q1, l);
      }
      seen += __shfl(c, 63);
    }
    found = __builtin_amdgcn_readfirstlane(found);
    if (found < 0) {
      if (seen != (int)blockIdx.y) return;
      r0 = clampi(p.offsets[p.experts], 0, p.M);
      for (int i = threadIdx.x; i < (p.M - r0) * 16; i += 64 * NW) {
        const int n = n0 + (i & 15);
        if (n < p.N) store_elt<OT>((char*)p.d + ((int64_t)(r0 + (i >> 4)) * p.ldd + n) * elt_size(OT), 0.0f);
      }
      return;
    }
    r0 = __builtin_amdgcn_readfirstlane(r0);
    r1 = __builtin_amdgcn_readfirstlane(r1);
    b += (int64_t)found * p.b_e;
    sb += (int64_t)found * p.sb_e;
  } else {
    r0 = (int)blockIdx.y * (16 * MT);
    r1 = min(r0 + 16 * MT, p.M);
  }
  const int nkb = (p.K + kScaleBlock - 1) / kScaleBlock;
  const int nv = min(16, p.N - n0);
  const __amdgpu_buffer_rsrc_t rb = rsrc_of(b + (int64_t)n0 * p.ldb, (int64_t)(nv - 1) * p.ldb + p.K);
  const float* sbp = sb + (int64_t)(n0 / kScaleBlock) * p.sb_n;
  const int piece = lane >> 4, frow = lane & 15;
  const uint32_t boff = frow < nv ? (uint32_t)(frow * p.ldb) + piece * 16 : kOOB;
  for (int m0 = r0; m0 < r1; m0 += 16 * MT) {
    const int mv = min(16 * MT, r1 - m0);
    const __amdgpu_buffer_rsrc_t ra = rsrc_of(p.a + (int64_t)m0 * p.lda, (int64_t)(mv - 1) * p.lda + p.K);
    const float* sap = p.sa + (int64_t)m0 * p.sa_m;
    uint32_t aoff[MT], soff[MT];
    f32x4 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int m = i * 16 + frow;
      aoff[i] = m < mv ? (uint32_t)(m * p.lda) + piece * 16 : kOOB;
      soff[i] = (uint32_t)(min(m, mv - 1) * p.sa_m);
      acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    u32x4 fb[2][U][2], fa[2][U][MT][2];
    float s[2][U][MT], sw[2][U];
    auto load = [&](int kb, int x) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = kb + u * NW;
        const int kc = min(k, nkb - 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool in = k * kScaleBlock + piece * 16 + h * 64 < p.K;
          const uint32_t at = (uint32_t)(k * kScaleBlock + h * 64);
          fb[x][u][h] = __builtin_amdgcn_raw_buffer_load_b128(rb, in ? boff + (boff == kOOB ? 0 : at) : kOOB, 0, 0);
#pragma unroll
          for (int i = 0; i < MT; ++i)
            fa[x][u][i][h] = __builtin_amdgcn_raw_buffer_load_b128(ra, in ? aoff[i] + (aoff[i] == kOOB ? 0 : at) : kOOB, 0, 0);
        }
        const float* q = sap + (int64_t)kc * p.sa_k;
#pragma unroll
        for (int i = 0; i < MT; ++i) s[x][u][i] = q[soff[i]];
        sw[x][u] = sbp[(int64_t)kc * p.sb_k];
      }
    };
    auto compute = [&](int kb, int x) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (kb + u * NW < nkb) {  // (uniform)
          const Wide vb = widen(join8(fb[x][u][0], fb[x][u][1]));
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            const f32x4 pr = mfma128(vb, widen(join8(fa[x][u][i][0], fa[x][u][i][1])));
            acc[i] += pr * (s[x][u][i] * sw[x][u]);
          }
        }
      }
    };
    if (wave < nkb) load(wave, 0);
    for (int kb = wave; kb < nkb; kb += 2 * U * NW) {
      if (kb + U * NW < nkb) load(kb + U * NW, 1);
      compute(kb, 0);
      if (kb + 2 * U * NW < nkb) load(kb + 2 * U * NW, 0);
      if (kb + U * NW < nkb) compute(kb + U * NW, 1);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) red[wave][i][lane] = acc[i];
    __syncthreads();
    for (int o = threadIdx.x; o < 256 * MT; o += 64 * NW) {
      const int i = o >> 8, m = i * 16 + ((o >> 4) & 15), n = o & 15;  // n = 4 q + r of lane 16 q + m
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) v += ((const float*)&red[w][i][(n >> 2) * 16 + (m & 15)])[n & 3];
      if (m < mv && n < nv) store_elt<OT>((char*)p.d + ((int64_t)(m0 + m) * p.ldd + n0 + n) * elt_size(OT), v);
    }
    __syncthreads();
  }
}

template <int MODE, int OT, int BM, int BN, int WGM, int WGN, bool WIDE>
hipError_t launch_tile(Fp8Gemm& p, hipStream_t s) {
  p.tiles_n = (p.N + BN - 1) / BN;
  p.tiles_m = (p.M + BM - 1) / BM;
  if (MODE == GM_GROUPED) p.tiles_m += (p.experts < p.M ? p.experts : p.M) + 1;  // (at most)
  const int64_t blocks = (int64_t)p.tiles_m * p.tiles_n * (MODE == GM_WGRAD ? p.experts : p.splits);
  if (blocks >= 0x7fffffffLL / (64 * WGM * WGN)) return hipErrorInvalidConfiguration;
  fp8_tile_kernel<MODE, OT, BM, BN, WGM, WGN, WIDE><<<(unsigned)blocks, 64 * WGM * WGN, 0, s>>>(p);
  return hipGetLastError();
}

template <int MODE, int OT>
hipError_t launch_tiles(Fp8Gemm& p, hipStream_t s) {
  if constexpr (OT != EL_F32) {
    if (MODE == GM_WGRAD || p.K > 2 * kScaleBlock) {
      const hipError_t e = launch_tile<MODE, OT, 256, 256, 4, 2, false>(p, s);
      if (e != hipSuccess || p.splits == 1) return e;
      const int64_t b = ((int64_t)p.M * p.N + 2047) / 2048;
      fp8_join_kernel<OT><<<(unsigned)(b < 4096 ? b : 4096), 256, 0, s>>>(p);
      return hipGetLastError();
    }
  }
  return launch_tile<MODE, OT, 128, 128, 2, 2, true>(p, s);
}

template <int MODE, int OT, int MT>
hipError_t launch_rows_mt(Fp8Gemm& p, hipStream_t s) {
  const unsigned gy = MODE == GM_GROUPED ? (unsigned)((p.experts < p.M ? p.experts : p.M) + 1)
                                         : (unsigned)((p.M + 16 * MT - 1) / (16 * MT));
  const dim3 grid((unsigned)((p.N + 15) / 16), gy);
  if (p.K >= 64 * kScaleBlock) fp8_rows_kernel<MODE, OT, MT, 8><<<grid, 512, 0, s>>>(p);
  else fp8_rows_kernel<MODE, OT, MT, 4><<<grid, 256, 0, s>>>(p);
  return hipGetLastError();
}

template <int MODE, int OT>
hipError_t launch_rows(Fp8Gemm& p, int rows_at_once, hipStream_t s) {
  if (rows_at_once == 16) return launch_rows_mt<MODE, OT, 1>(p, s);
  return launch_rows_mt<MODE, OT, 2>(p, s);
}

}  // namespace

int fp8_splits(int m, int n, int k) { return 1; }

hipError_t launch_fp8_tiles(int mode, int out, Fp8Gemm& p, hipStream_t s) {
#define EP_CASE(M_, O_) \
  if (mode == M_ && out == O_) return launch_tiles<M_, O_>(p, s);
  EP_CASE(GM_MATMUL, EL_F16) EP_CASE(GM_MATMUL, EL_BF16) EP_CASE(GM_MATMUL, EL_F32)
  EP_CASE(GM_GROUPED, EL_F16) EP_CASE(GM_GROUPED, EL_BF16) EP_CASE(GM_GROUPED, EL_F32)
  EP_CASE(GM_WGRAD, EL_F16) EP_CASE(GM_WGRAD, EL_BF16) EP_CASE(GM_WGRAD, EL_F32)
#undef EP_CASE
  return hipErrorInvalidValue;
}

hipError_t launch_fp8_rows(int mode, int out, Fp8Gemm& p, int rows_at_once, hipStream_t s) {
#define EP_CASE(M_, O_) \
  if (mode == M_ && out == O_) return launch_rows<M_, O_>(p, rows_at_once, s);
  EP_CASE(GM_MATMUL, EL_F16) EP_CASE(GM_MATMUL, EL_BF16) EP_CASE(GM_MATMUL, EL_F32)
  EP_CASE(GM_GROUPED, EL_F16) EP_CASE(GM_GROUPED, EL_BF16) EP_CASE(GM_GROUPED, EL_F32)
#undef EP_CASE
  return hipErrorInvalidValue;
}

}  // namespace ep
