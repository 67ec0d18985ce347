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
// How exact the sums are.  That instruction adds the products of 8 neighbouring k in fixed point before its
// fp32 accumulator.  With 2^E the largest product of the 8 pairs' powers of two (a subnormal operand's counting as
// 2^-6), a product is cut off, towards zero, to a multiple of 2^(E - 13): each of the other 7 loses less than 2^-13
// of the largest, where that has normal operands.  Measured next to 64 bits, of the result's norm: 1.5e-5 with
// normally distributed operands, 2.2e-5 with one feature in a hundred 12 times larger, 4.1e-5 with sizes spread over
// the whole type (fp32 sums: 1e-8).  Next to a bf16 or fp16 output's rounding (1.7e-3, 2.1e-4) that is little, and
// it is the unit's only way to its full rate; but two large products that cancel among the 8 take what is smaller than
// that with them.  Where it would show or buys nothing the operands are widened to fp16 first, which holds every
// e4m3 value, and multiplied by v_mfma_f32_16x16x32_f16, whose sums are fp32 throughout: fp32 outputs and, but for
// weight gradients, sums of at most 256 values (fp8_wide_kernel; the latter bound by the output's bytes), and the
// few-row kernel (bound by the weights').
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

// v, computed here and not kept in registers from before the loop around it
__device__ __forceinline__ int here(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// v, made once and held in one register: what it is made of is hidden
__device__ __forceinline__ int keep(int v) {
  asm("" : "+v"(v));
  return v;
}

__device__ __forceinline__ int wave_scan(int v) {  // inclusive sum over the lanes
  const int lane = here(lane_id());
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int u = __shfl_up(v, d);
    if (lane >= d) v += u;
  }
  return v;
}

__device__ __forceinline__ int wave_max_scan(int v) {  // inclusive maximum over the lanes
  const int lane = here(lane_id());
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int u = __shfl_up(v, d);
    if (lane >= d) v = max(v, u);
  }
  return v;
}

// Rows of the 64 groups from e0 on, one a lane (past the last group: none), kept inside [0, rows] and apart
// from each other whatever the offsets hold: one below an earlier one counts as that one.  So there are never
// more tiles than the launch counted on, which the walk over the tiles needs, and no row has two groups.
// `top` is the greatest offset before group e0, and afterwards before group e0 + 64.
__device__ __forceinline__ void groups_at(const int* offsets, int experts, int e0, int rows, int& top, int& r0, int& r1) {
  const int e = e0 + lane_id();
  r0 = r1 = 0;
  if (e < experts) {
    r0 = clampi(offsets[e], 0, rows);
    r1 = clampi(offsets[e + 1], 0, rows);
  }
  if (__ballot(e < experts && r1 < r0)) r0 = wave_max_scan(r0);
  r0 = max(r0, top);
  r1 = max(r0, r1);
  top = __builtin_amdgcn_readfirstlane(__shfl(r1, min(63, experts - 1 - e0)));
}

template <int OT>
__device__ __forceinline__ void store_row8(char* d, int n, f32x4 lo, f32x4 hi) {
  const float f[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  store8<OT>(d, n, f);
}

// ---------------------------------------------------------------------------------------- tiles
constexpr int kGroupM = 8;
constexpr int kTilesAtOnce = 512;

template <class T>
__device__ __forceinline__ T* global_ptr(T* p) {
  return (T*)(__attribute__((address_space(1))) T*)(uint64_t)p;
}

// A kernel's only argument, read from its segment here and not kept in registers from before a loop.
__device__ __forceinline__ Fp8Gemm args_here() {
  typedef const __attribute__((address_space(4))) uint32_t* Words;
  const uint64_t at = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
  uint32_t lo = (uint32_t)at, hi = (uint32_t)(at >> 32);
  asm volatile("" : "+s"(lo), "+s"(hi));
  const Words k = (Words)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)hi) << 32 |
                          (uint32_t)__builtin_amdgcn_readfirstlane((int)lo));
  uint32_t w[sizeof(Fp8Gemm) / 4];
#pragma unroll
  for (size_t i = 0; i < sizeof(Fp8Gemm) / 4; ++i) w[i] = k[i];
  Fp8Gemm p = __builtin_bit_cast(Fp8Gemm, w);
  // (global, which the compiler can no longer see; flat accesses would count as LDS accesses too, and with
  // those pending it waits for all fragment reads at once)
  p.sa = global_ptr(p.sa);
  p.sb = global_ptr(p.sb);
  p.d = global_ptr(p.d);
  p.offsets = global_ptr(p.offsets);
  return p;
}

// One BM x BN tile of D and the scale blocks that go into it.
struct Tile {
  int m0, mv, n0, nv;      // rows from m0, mv of them; columns from n0, nv of them
  int kb0, nkb, klen;      // scale blocks from kb0, nkb of them (0: the tile is `fill`); k-values end at klen
  int part;                // expert, or K range
  float fill;
};

// The tiles of a product in the order they are worked on: bands of kGroupM tile rows, column by column,
// so that neighbours share operand panels; grouped: expert by expert, then the rows behind the last group.
template <int MODE, int BM, int BN>
struct Tiles {
  int count;               // tiles there are
  int e0 = 0, base = 0, top = 0;  // grouped: a group to go on from, tile rows and the greatest offset before it

  __device__ __forceinline__ explicit Tiles(const Fp8Gemm& p) {
    if constexpr (MODE == GM_GROUPED) {
      int total = 0, end = 0;
      for (int e = 0; e < p.experts; e += 64) {
        int r0, r1;
        groups_at(p.offsets, p.experts, e, p.M, end, r0, r1);
        total += __shfl(wave_scan((r1 - r0 + BM - 1) / BM), 63);
      }
      total += (p.M - end + BM - 1) / BM;
      count = __builtin_amdgcn_readfirstlane(total) * p.tiles_n;
    } else {
      count = p.tiles_m * p.tiles_n * (MODE == GM_WGRAD ? p.experts : p.splits);
    }
  }

  static __device__ __forceinline__ void place(int tiles_n, int w, int rows, int& tm, int& tn) {
    const int group = kGroupM * tiles_n, g = w / group, first = g * kGroupM;
    const int gm = min(rows - first, kGroupM), v = w - g * group;
    tm = first + v % gm;
    tn = v / gm;
  }

  // tile u; for the groups u must not fall from one call to the next
  __device__ __forceinline__ Tile at(const Fp8Gemm& p, int u) {
    Tile t;
    t.part = t.kb0 = 0;
    t.klen = p.K;
    t.fill = 0.0f;
    int tm, tn;
    if constexpr (MODE == GM_MATMUL) {
      const int tiles = p.tiles_m * p.tiles_n;
      t.part = u / tiles;
      place(p.tiles_n, u - t.part * tiles, p.tiles_m, tm, tn);
      t.m0 = tm * BM;
      t.mv = min(BM, p.M - t.m0);
      t.kb0 = t.part * p.kb_per_split;
      t.nkb = min(p.kb_per_split, (p.K + kScaleBlock - 1) / kScaleBlock - t.kb0);
    } else if constexpr (MODE == GM_GROUPED) {
      int e = -1, first = 0, r0 = 0, r1 = 0;
      for (; e0 < p.experts; e0 += 64) {
        int q0, q1, end = top;
        groups_at(p.offsets, p.experts, e0, p.M, end, q0, q1);
        const int c = (q1 - q0 + BM - 1) / BM;
        const int ends = base + wave_scan(c);
        const uint64_t past = __ballot(ends * p.tiles_n > u);
        if (past) {
          const int l = __builtin_ctzll(past);
          e = e0 + l;
          first = __shfl(ends - c, l);
          r0 = __shfl(q0, l);
          r1 = __shfl(q1, l);
          break;
        }
        base = __builtin_amdgcn_readfirstlane(__shfl(ends, 63));
        top = end;
      }
      if (e < 0) {
        e = p.experts;
        first = base;
        r0 = top;
        r1 = p.M;
      }
      t.part = __builtin_amdgcn_readfirstlane(e);
      first = __builtin_amdgcn_readfirstlane(first);
      r0 = __builtin_amdgcn_readfirstlane(r0);
      r1 = __builtin_amdgcn_readfirstlane(r1);
      place(p.tiles_n, u - first * p.tiles_n, (r1 - r0 + BM - 1) / BM, tm, tn);
      t.m0 = r0 + tm * BM;
      t.mv = min(BM, r1 - t.m0);
      t.nkb = t.part == p.experts ? 0 : (p.K + kScaleBlock - 1) / kScaleBlock;
    } else {
      const int tiles = p.tiles_m * p.tiles_n;
      t.part = u / tiles;
      place(p.tiles_n, u - t.part * tiles, p.tiles_m, tm, tn);
      t.m0 = tm * BM;
      t.mv = min(BM, p.M - t.m0);
      const int r0 = __builtin_amdgcn_readfirstlane(clampi(p.offsets[t.part], 0, p.K));
      const int r1 = __builtin_amdgcn_readfirstlane(clampi(p.offsets[t.part + 1], r0, p.K));
      t.kb0 = r0 / kScaleBlock;
      t.nkb = r1 / kScaleBlock - t.kb0;
      t.klen = r1;
      if (r0 < r1 && (r0 | r1) % kScaleBlock) {  // such a group has no scales of its own
        t.nkb = 0;
        t.fill = __builtin_nanf("");
      }
    }
    t.n0 = tn * BN;
    t.nv = min(BN, p.N - t.n0);
    return t;
  }

};

template <int MODE>
__device__ __forceinline__ const uint8_t* tile_a(const Fp8Gemm& p, const Tile& t) {
  return p.a + (int64_t)t.m0 * p.lda + (int64_t)t.kb0 * kScaleBlock;
}
template <int MODE>
__device__ __forceinline__ const uint8_t* tile_b(const Fp8Gemm& p, const Tile& t) {
  return p.b + (MODE == GM_GROUPED ? (int64_t)t.part * p.b_e : 0) + (int64_t)t.n0 * p.ldb + (int64_t)t.kb0 * kScaleBlock;
}
template <int MODE>
__device__ __forceinline__ const float* tile_sa(const Fp8Gemm& p, const Tile& t) {
  return p.sa + (int64_t)t.m0 * p.sa_m + (int64_t)t.kb0 * p.sa_k;
}
template <int MODE>
__device__ __forceinline__ const float* tile_sb(const Fp8Gemm& p, const Tile& t, int n) {  // of column n0 + n
  return p.sb + (MODE == GM_GROUPED ? (int64_t)t.part * p.sb_e : 0) + (int64_t)((t.n0 + n) / kScaleBlock) * p.sb_n + (int64_t)t.kb0 * p.sb_k;
}
// element (0, 0) of the tile; experts' gradients and K ranges' parts lie one behind another
template <int MODE, int OT>
__device__ __forceinline__ char* tile_d(const Fp8Gemm& p, const Tile& t) {
  const int64_t row = (int64_t)(MODE == GM_GROUPED ? 0 : t.part) * p.M + t.m0;
  return (char*)p.d + (row * p.ldd + t.n0) * elt_size(OT);
}

// a tile without products
template <int MODE, int OT, int BN>
__device__ __forceinline__ void fill_tile(const Fp8Gemm& p, const Tile& t) {
  const f32x4 v = {t.fill, t.fill, t.fill, t.fill};
  char* d = tile_d<MODE, OT>(p, t);
  for (int i = here((int)threadIdx.x); i < t.mv * (BN / 8); i += (int)blockDim.x) {
    const int m = i / (BN / 8), n = i % (BN / 8) * 8;
    if (n < t.nv) store_row8<OT>(d + (m * p.ldd + n) * elt_size(OT), t.nv - n, v, v);
  }
}

// Row of a 16-row block that lane l (of 16) holds: LDS row 16 u + 4 q + i of each 32 holds row 8 q + 4 u + i,
// so that a lane's values of two neighbouring blocks along n are 8 neighbouring ones.
__device__ __forceinline__ int row_in(int block, int l) {
  return (block >> 1) * 32 + (l >> 2) * 8 + (block & 1) * 4 + (l & 3);
}

// a wave's accumulators to D: in a lane one row of each 16 (in row_in's order, or lane by lane) and 8
// neighbouring columns
template <int MODE, int OT, bool PERM, int MT, int NT>
__device__ __forceinline__ void store_tile(const Fp8Gemm& p, const Tile& t, int m_at, int n_at, f32x4 (&acc)[MT][NT]) {
  const int lane = here(lane_id());
  char* d = tile_d<MODE, OT>(p, t) + (m_at * p.ldd + n_at) * elt_size(OT);
  const int n0 = 8 * (lane >> 4);
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = PERM ? row_in(i, lane & 15) : i * 16 + (lane & 15);
    if (m >= t.mv - m_at) continue;
    char* row = d + (m * p.ldd + n0) * elt_size(OT);
#pragma unroll
    for (int j = 0; j < NT; j += 2) {
      const int left = t.nv - n_at - n0 - j * 16;
      if (left > 0) store_row8<OT>(row + j * 16 * elt_size(OT), left, acc[i][j], acc[i][j + 1]);
    }
  }
}

// The same for 16-bit outputs and rows in row_in's order: neighbouring lanes, which hold neighbouring rows,
// first trade halves of 64 columns, so that a store instruction writes whole 128-byte lines, which leave the
// caches to the operands (non-temporal).  The experts' weight gradients, 2.7 GB of stores: 1518 us with half
// lines, 1345 with whole ones, 1220 non-temporal.
template <int MODE, int OT, int MT, int NT>
__device__ __forceinline__ void store_lines(const Fp8Gemm& p, const Tile& t, int m_at, int n_at, f32x4 (&acc)[MT][NT]) {
  const int lane = here(lane_id());
  const bool odd = lane & 1;
  char* d = tile_d<MODE, OT>(p, t) + (m_at * p.ldd + n_at) * 2;
  const int n0 = 8 * (lane >> 4) + (odd ? 32 : 0);
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = row_in(i, lane & 14);
    char* row = d + (m * p.ldd + n0) * 2;
    const int rows = t.mv - m_at - m;
#pragma unroll
    for (int j = 0; j < NT; j += 4) {
      u32x4 a, b, x, y;  // the row's first and second 32 columns' pieces; traded
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        a[h] = pack2_elt<OT>(acc[i][j + h / 2][2 * (h & 1)], acc[i][j + h / 2][2 * (h & 1) + 1]);
        b[h] = pack2_elt<OT>(acc[i][j + 2 + h / 2][2 * (h & 1)], acc[i][j + 2 + h / 2][2 * (h & 1) + 1]);
        const uint32_t got = (uint32_t)__builtin_amdgcn_mov_dpp((int)(odd ? a[h] : b[h]), 0xb1, 0xf, 0xf, true);
        x[h] = odd ? got : a[h];
        y[h] = odd ? b[h] : got;
      }
      const int left = t.nv - n_at - n0 - j * 16;
      if (left >= 8) {
        if (rows > 0) __builtin_nontemporal_store(x, (u32x4_u*)(row + j * 32));
        if (rows > 1) __builtin_nontemporal_store(y, (u32x4_u*)(row + p.ldd * 2 + j * 32));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (e >= left) continue;
          if (rows > 0) *(uint16_t*)(row + j * 32 + e * 2) = (uint16_t)(x[e >> 1] >> (16 * (e & 1)));
          if (rows > 1) *(uint16_t*)(row + p.ldd * 2 + j * 32 + e * 2) = (uint16_t)(y[e >> 1] >> (16 * (e & 1)));
        }
      }
    }
  }
}

// ---- the e4m3 tiles
// Which of three or four register slots column block j's fragment of b takes, and when it is read: the two
// last blocks and the next step's first one are held at the same time, a slot is free once its block's MFMAs
// are issued.
template <int NT>
__device__ constexpr int slot_of(int j) {
  constexpr int eight[8] = {2, 0, 1, 0, 1, 2, 0, 1};
  return NT == 8 ? eight[j] : j;
}
template <int NT>
__device__ constexpr int read_after(int j) {  // the column block behind whose MFMAs block j is read, -1: the step's start
  int r = -1;
  for (int i = 0; i < j; ++i)
    if (slot_of<NT>(i) == slot_of<NT>(j)) r = i;
  return r;
}

template <int NT>
__device__ constexpr bool read_first(int j) {
  return read_after<NT>(j) < 0 || read_after<NT>(j) >= NT - 2;
}

// BM x BN tiles of D, WGM x WGN waves, as many workgroups as fit the chip, each walking its share of the
// tiles.  Both operands and their scales go through LDS in a ring of S stages of one scale block (128 bytes
// a row: one cache line, 8 lanes of 16 bytes), filled by loads that write LDS themselves.  16-byte piece c of
// row r is kept at piece c ^ (r & 7), which the fragment reads (16 rows at one piece per 16 lanes) take
// without bank conflicts; the rows of each 32 are in row_in's order.
//
// Two barriers a step.  Behind the first, after the first column block, every wave holds its fragments of a:
// the stage's part of a is free, and the loads of the step S ahead go into it.  Behind the second, before the
// last two blocks, every wave holds what it reads of b as well: the loads of b follow, and the next stage has
// landed.  The last two blocks' MFMAs go row block by row block, each row block's fragment of a followed by the
// next step's, and a step's last product is added behind the next step's first MFMA, so that the matrix unit
// waits little between steps.  The steps run on from tile to tile: the next tile's operands land while this
// one's last steps are multiplied.
//
// Measured on one MI355X: 8192 x 17408 x 5120 in 602 us, 2426 TFLOP/s (596 to 705 from run to run, by the clock;
// one tile a workgroup, all loads at a step's start: 667).  What bounds it is power: the card runs it at 1.7 GHz of 2.4, the matrix unit is busy for 60 % of
// the cycles.  From registers alone the same MFMAs with random operands reach 3863 TFLOP/s, 3484 with their
// multiply-adds; without the loads (operands left in LDS) a step takes 12 % fewer cycles, without the multiply-adds 15 %.
template <int MODE, int OT, int BM, int BN, int WGM, int WGN, int S>
__global__ __launch_bounds__(64 * WGM * WGN) __attribute__((amdgpu_waves_per_eu(2)))
void fp8_tile_kernel(Fp8Gemm p) {
#ifdef __HIP_DEVICE_COMPILE__  // (the host's pass drops a body with register constraints it does not know)
  constexpr int WAVES = WGM * WGN, WTM = BM / WGM, WTN = BN / WGN, MT = WTM / 16, NT = WTN / 16;
  constexpr int OPS = (BM + BN) * 128, STAGE = OPS + WAVES * 256;
  constexpr int N = MT * NT, R = NT == 8 ? 3 : 4;  // a step's MFMAs; results in flight: the multiply-adds follow 2 MFMAs behind
  static_assert(BM == 32 * WAVES && BN == 32 * WAVES && WTN <= 128 && 128 % WTN == 0 && BM / 64 < WAVES, "tile");
  static_assert((NT == 8 || NT == 4) && MT == 4, "schedule");
  __shared__ __align__(128) char lds[S * STAGE];
  const int lane = lane_id(), wave = wave_id();
  const int wm = wave / WGN, wn = wave % WGN;
  Tiles<MODE, BM, BN> tiles(p);
  int bid = (int)blockIdx.x;
  const int blocks = (int)gridDim.x;

  // the next tile with products, the others filled on the way
  auto next = [&](Tile& t) __attribute__((always_inline)) {
    const Fp8Gemm q = args_here();
    t.nkb = 0;
    while (bid < tiles.count && t.nkb == 0) {
      t = tiles.at(q, xcd_order(bid, tiles.count));
      bid += blocks;
      if (t.nkb == 0) fill_tile<MODE, OT, BN>(q, t);
    }
    return t.nkb > 0;
  };

  // ---- the loads' side: a wave's 32 rows of a and of b, 8 of them a piece, and 64 scales: rows' in the first
  // BM / 64 waves, the columns' in the next one (the others load some rows' into places of their own)
  const int piece16 = ((lane & 7) ^ (lane >> 3)) * 16;
  const bool sb_wave = wave == BM / 64;
  // a lane's row of piece 0 (pieces are 8 LDS rows, see row_in); the others are row_of(s) behind it.  Rows past
  // the tile's are past the descriptor's range, which the hardware checks without the scalar offset
  auto row_of = [](int s) __attribute__((always_inline)) { return 16 * (s & 1) + 4 * (s >> 1); };
  const int row0 = 8 * (lane >> 5) + ((lane >> 3) & 3);
  __amdgpu_buffer_rsrc_t ra, rb;
  int lda = 0, ldb = 0;
  uint32_t aoff, boff, ak = 0, bk = 0;
  int lk = 0, lklen = 0, ls_left = 0;  // k of the next step, where k ends, steps of scales to come
  const float* lsp;
  int64_t ls_step = 0;
  uint32_t lsoff;
  auto load_tile = [&](const Tile& t) __attribute__((always_inline)) {
    const Fp8Gemm q = args_here();
    lda = (int)q.lda;
    ldb = (int)q.ldb;
    const int rows_a = t.mv - wave * 32, rows_b = t.nv - wave * 32;  // (at most 0: the wave loads zeros)
    lk = 0;
    lklen = min(t.klen - t.kb0 * kScaleBlock, t.nkb * kScaleBlock);
    ra = rsrc_of(tile_a<MODE>(q, t) + (int64_t)(wave * 32) * lda, rows_a > 0 ? (int64_t)(rows_a - 1) * lda + lklen : 0);
    rb = rsrc_of(tile_b<MODE>(q, t) + (int64_t)(wave * 32) * ldb, rows_b > 0 ? (int64_t)(rows_b - 1) * ldb + lklen : 0);
    aoff = (uint32_t)(row0 * lda + piece16);
    boff = (uint32_t)(row0 * ldb + piece16);
    lsp = sb_wave ? tile_sb<MODE>(q, t, 0) : tile_sa<MODE>(q, t);
    lsoff = (uint32_t)(sb_wave ? min(lane, (t.nv - 1) / kScaleBlock) * (int)q.sb_n
                               : min(wave % (BM / 64) * 64 + lane, t.mv - 1) * (int)q.sa_m) * 4;
    ls_step = sb_wave ? q.sb_k : q.sa_k;
    ls_left = t.nkb;
  };
  auto load_k = [&]() __attribute__((always_inline)) {  // (k is a multiple of 16: pieces are whole or absent)
    const bool in = lk + piece16 < lklen;
    ak = in ? aoff : kOOB;
    bk = in ? boff : kOOB;
  };
  auto load_a = [&](int stage, int s) __attribute__((always_inline)) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        ra, (__attribute__((address_space(3))) void*)(lds + stage * STAGE + (wave * 4 + s) * 1024), 16,
        (int)(ak + row_of(s) * lda), lk, 0, 0);
  };
  auto load_b = [&](int stage, int s) __attribute__((always_inline)) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rb, (__attribute__((address_space(3))) void*)(lds + stage * STAGE + BM * 128 + (wave * 4 + s) * 1024), 16,
        (int)(bk + row_of(s) * ldb), lk, 0, 0);
  };
  auto load_scales = [&](int stage) __attribute__((always_inline)) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rsrc_of(lsp, 0x7fffffff), (__attribute__((address_space(3))) void*)(lds + stage * STAGE + OPS + wave * 256), 4, (int)lsoff, 0, 0, 0);
  };
  auto load_done = [&]() __attribute__((always_inline)) {
    lk += kScaleBlock;
    if (--ls_left > 0) lsp += ls_step;
  };

  // ---- the products' side
  const int frow = (lane & 15) * 128 + ((lane >> 4) ^ (lane & 7)) * 16;
  const int va = keep(wm * WTM * 128 + frow), vb = keep(BM * 128 + wn * WTN * 128 + frow);
  const int vt = keep(OPS + (wm * WTM + row_in(0, lane & 15)) * 4);
  // block's fragment of the operand whose lane offset in this stage is `at`
  auto frag = [&](int at, int block) __attribute__((always_inline)) {
    return join8(*(const u32x4*)(lds + at + block * 2048), *(const u32x4*)(lds + (at ^ 64) + block * 2048));
  };
  f32x4 acc[MT][NT], pr[R];
  i32x8 fa[MT], fb[NT == 8 ? 3 : 4];
  float t[MT], tn[MT], tb = 0.0f, t_last = 0.0f;
  auto read_scales = [&](int at) __attribute__((always_inline)) {
    const char* q = lds + at + vt;
#pragma unroll
    for (int i = 0; i < MT; ++i) tn[i] = *(const float*)(q + row_in(i, 0) * 4);
    tb = *(const float*)(lds + at + OPS + (BM + wn * WTN / kScaleBlock) * 4);
  };
  // the step's MFMAs in order: column blocks, the last two of them row block by row block
  auto mfma = [&](int x) __attribute__((always_inline)) {
    constexpr int H = MT * (NT - 2);
    const int i = x < H ? x % MT : (x - H) / 2, j = x < H ? x / MT : NT - 2 + (x - H) % 2;
    pr[x % R] = mfma128(fb[slot_of<NT>(j)], fa[i]);
  };
  auto add = [&](int x) __attribute__((always_inline)) {
    constexpr int H = MT * (NT - 2);
    const int i = x < H ? x % MT : (x - H) / 2, j = x < H ? x / MT : NT - 2 + (x - H) % 2;
    acc[i][j] += pr[x % R] * t[i];
  };
  // a step's last product is added behind the next step's first MFMA
  auto add_last = [&]() __attribute__((always_inline)) { acc[MT - 1][NT - 1] += pr[(N - 1) % R] * t_last; };
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    pr[(N - 1) % R] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    t_last = 0.0f;
  };

  Tile cur, ahead;
  if (!next(cur)) return;
  clear();
  load_tile(cur);
#pragma unroll
  for (int s = 0; s < S; ++s) {
    load_scales(s);
    load_k();
#pragma unroll
    for (int x = 0; x < 4; ++x) load_a(s, x);
#pragma unroll
    for (int x = 0; x < 4; ++x) load_b(s, x);
    load_done();
  }
  constexpr int WAIT0 = (S - 1) * 9, WAIT = (S - 2) * 9 + 5;
  __builtin_amdgcn_s_waitcnt((WAIT0 & 15) | ((WAIT0 >> 4) << 14) | 0x0f70);
  asm volatile("s_barrier" ::: "memory");
  // what a step finds in registers, or on its way: all of a, the first block of b, the scales' products
  read_scales(0);
#pragma unroll
  for (int i = 0; i < MT; ++i) fa[i] = frag(va, i);
  fb[slot_of<NT>(0)] = frag(vb, 0);
#pragma unroll
  for (int i = 0; i < MT; ++i) t[i] = tn[i] * tb;

  bool more = false, done = false;
  int step = 0, steps = max(cur.nkb, S), stage = 0;  // (a tile of fewer steps than stages gets empty ones)
  auto steps_on = [&]() __attribute__((always_inline)) {  // (the other waves only load)
    return (wm * WTM < cur.mv) & (wn * WTN < cur.nv) ? cur.nkb : 0;
  };
  int on = steps_on();
  while (!done) {
    const int stage1 = stage + 1 == S ? 0 : stage + 1;
    if (__builtin_expect(step + S == steps, 0)) {  // the loads go on to the next tile, or to nothing
      more = next(ahead);
      if (more) load_tile(ahead);
      else lklen = 0;
      __builtin_amdgcn_s_waitcnt(0xc07f);  // (lgkmcnt: with scalar loads pending the compiler could not count fragment reads)
    }
    load_k();
    // second barrier: this wave's loads of the next stage have landed, and it holds all it reads of this one
    // (a wait visible to the compiler's own counting); behind it that holds for everyone
    auto barrier = [&]() __attribute__((always_inline)) {
      __builtin_amdgcn_s_waitcnt((WAIT & 15) | ((WAIT >> 4) << 14) | 0x0070);
      asm volatile("s_barrier" ::: "memory");
    };
    if (__builtin_expect(step < on, 1)) {
      const int b_at = keep(vb + stage * STAGE);
#pragma unroll
      for (int j = 1; j < NT; ++j)
        if (read_first<NT>(j)) fb[slot_of<NT>(j)] = frag(b_at, j);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < NT - 2; ++j) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const int x = j * MT + i;
          mfma(x);
          __builtin_amdgcn_sched_barrier(0);
          if (x == 0) add_last();
          if (x >= 2) add(x - 2);
          __builtin_amdgcn_sched_barrier(0);
          // the loads of a, over the blocks left before the last two
          if (j > 0 && (NT == 4 || i == 1)) {
            if (NT == 4 ? i == 0 : j == 1) load_scales(stage);
            if (NT == 4) load_a(stage, i);
            else if (j > 1) load_a(stage, j - 2);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
#pragma unroll
        for (int n = j + 1; n < NT; ++n)
          if (read_after<NT>(n) == j && !read_first<NT>(n)) fb[slot_of<NT>(n)] = frag(b_at, n);
        __builtin_amdgcn_sched_barrier(0);
        if (j == 0) asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
      }
      barrier();
      read_scales(stage1 * STAGE);
      const int a_next = keep(va + stage1 * STAGE);
      fb[slot_of<NT>(0)] = frag(vb + stage1 * STAGE, 0);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int x = MT * (NT - 2) + 2 * i + h;
          mfma(x);
          __builtin_amdgcn_sched_barrier(0);
          add(x - 2);
          __builtin_amdgcn_sched_barrier(0);
          if (h == 0) load_b(stage, i);
          __builtin_amdgcn_sched_barrier(0);
        }
        fa[i] = frag(a_next, i);
        __builtin_amdgcn_sched_barrier(0);
      }
      add(N - 2);
      t_last = t[MT - 1];
#pragma unroll
      for (int i = 0; i < MT; ++i) t[i] = tn[i] * tb;
    } else {
      __builtin_amdgcn_s_waitcnt(0xc07f);
      asm volatile("s_barrier" ::: "memory");
      load_scales(stage);
#pragma unroll
      for (int x = 0; x < 4; ++x) load_a(stage, x);
      barrier();
      read_scales(stage1 * STAGE);
      fb[slot_of<NT>(0)] = frag(vb + stage1 * STAGE, 0);
#pragma unroll
      for (int x = 0; x < 4; ++x) load_b(stage, x);
      const int a_next = keep(va + stage1 * STAGE);
#pragma unroll
      for (int i = 0; i < MT; ++i) fa[i] = frag(a_next, i);
#pragma unroll
      for (int i = 0; i < MT; ++i) t[i] = tn[i] * tb;
    }
    load_done();
    stage = stage1;
    if (__builtin_expect(++step == steps, 0)) {
      // (the last loads write LDS too: not after the workgroup has left it)
      if (!more) __builtin_amdgcn_s_waitcnt(0x0070);
      add_last();
      if constexpr (OT == EL_F32) store_tile<MODE, OT, true>(args_here(), cur, wm * WTM, wn * WTN, acc);
      else store_lines<MODE, OT>(args_here(), cur, wm * WTM, wn * WTN, acc);
      done = !more;
      clear();
      cur = ahead;
      step = 0;
      steps = max(cur.nkb, S);
      on = steps_on();
    }
  }
#endif
}

// ---- the same with operands widened to fp16: one tile a workgroup, 128 x 128 so that two of them share a
// compute unit and one's loads pass behind the other's products.
template <int MODE, int OT, int BM, int BN, int WGM, int WGN>
__global__ __launch_bounds__(64 * WGM * WGN) __attribute__((amdgpu_waves_per_eu(2)))
void fp8_wide_kernel(Fp8Gemm p) {
  constexpr int WAVES = WGM * WGN, WTM = BM / WGM, WTN = BN / WGN, MT = WTM / 16, NT = WTN / 16;
  constexpr int SLOTS = (BM + BN) / 8, PER_WAVE = SLOTS / WAVES, STAGE = (BM + BN) * 128;
  static_assert(SLOTS % WAVES == 0 && (BM / 8) % PER_WAVE == 0 && NT % 2 == 0 && WTN <= 128 && 128 % WTN == 0, "tile");
  __shared__ __align__(128) char lds[2 * STAGE];
  const int lane = lane_id(), wave = wave_id();
  const int wm = wave / WGN, wn = wave % WGN;
  Tiles<MODE, BM, BN> tiles(p);
  if ((int)blockIdx.x >= tiles.count) return;
  const Tile tile = tiles.at(p, xcd_order((int)blockIdx.x, tiles.count));
  if (tile.nkb <= 0) {
    fill_tile<MODE, OT, BN>(p, tile);
    return;
  }
  const int mv = tile.mv, nv = tile.nv, nkb = tile.nkb;
  const int klen = tile.klen - tile.kb0 * kScaleBlock;

  // ---- loads: slot s of a stage is 8 rows; a wave's slots are neighbours and all of one operand
  const bool a_side = wave * PER_WAVE < BM / 8;
  const int64_t ld = a_side ? p.lda : p.ldb;
  const int rows = a_side ? mv : nv;
  const __amdgpu_buffer_rsrc_t rs = rsrc_of(a_side ? tile_a<MODE>(p, tile) : tile_b<MODE>(p, tile), (int64_t)(rows - 1) * ld + klen);
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
  const float* sap = tile_sa<MODE>(p, tile);
  const bool n_on = wn * WTN < nv;
  const float* sbp = tile_sb<MODE>(p, tile, n_on ? wn * WTN : 0);
  uint32_t soff[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) soff[i] = (uint32_t)(min(wm * WTM + i * 16 + (lane & 15), mv - 1) * p.sa_m);
  float sn[MT], sbn = 0.0f;
  auto scales = [&](int kb) __attribute__((always_inline)) {
    const float* q = sap + (int64_t)kb * p.sa_k;
#pragma unroll
    for (int i = 0; i < MT; ++i) sn[i] = q[soff[i]];
    sbn = sbp[(int64_t)kb * p.sb_k];
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
    return widen(join8(*(const u32x4*)(r + fpiece), *(const u32x4*)(r + (fpiece ^ 64))));
  };
  scales(0);
  issue(0, 0);
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
      Wide fa[MT], fb[2];
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

  if (active) store_tile<MODE, OT, false>(p, tile, wm * WTM, wn * WTN, acc);
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
// Few rows: bound by reading b once.  A workgroup takes 16 rows of b
// (columns of D) by 8 of a; its waves deal out the scale blocks and join their sums in LDS.  Each wave has a ring
// of its own in LDS, filled by loads that write it themselves and ordered by the wave's load count alone: what
// is in flight (6 KB of b a wave, 16 waves a compute unit) takes no registers.  One token's 8
// experts, n 4096, k 5120, in 30 us (5.5 TB/s, the inputs changing from pass to pass); the first form through LDS took
// 32, through registers 40, with 8 waves a workgroup 35.
constexpr int kRowsWaves = 4;
template <int MODE, int OT>
__global__ __launch_bounds__(64 * kRowsWaves) void fp8_rows_kernel(Fp8Gemm p) {
  constexpr int NW = kRowsWaves, D = 3, AT_A = 2048, AT_S = AT_A + 1024, SLOT = AT_S + 256;  // 16 rows of b, 8 of a, 9 scales
  __shared__ __align__(128) char ring[NW * D * SLOT];  // (39 KB: four workgroups a compute unit)
  const int lane = lane_id(), wave = wave_id();
  const int n0 = (int)blockIdx.x * 16;
  const uint8_t* b = p.b;
  const float* sb = p.sb;
  int r0, r1;
  if constexpr (MODE == GM_GROUPED) {
    // the blockIdx.y-th group that has rows; behind the last one the rows that no group has
    int seen = 0, found = -1, top = 0;
    for (int e0 = 0; e0 < p.experts && found < 0; e0 += 64) {
      int q0, q1;
      groups_at(p.offsets, p.experts, e0, p.M, top, q0, q1);
      uint64_t some = __ballot(q1 > q0);
      const int n = __builtin_popcountll(some), skip = (int)blockIdx.y - seen;
      if (skip < n) {
        for (int k = 0; k < skip; ++k) some &= some - 1;
        const int l = __builtin_ctzll(some);
        found = e0 + l;
        r0 = __builtin_amdgcn_readfirstlane(__shfl(q0, l));
        r1 = __builtin_amdgcn_readfirstlane(__shfl(q1, l));
      }
      seen += n;
    }
    if (found < 0) {
      if (seen != (int)blockIdx.y) return;
      r0 = top;
      for (int i = threadIdx.x; i < (p.M - r0) * 16; i += 64 * NW) {
        const int n = n0 + (i & 15);
        if (n < p.N) store_elt<OT>((char*)p.d + ((int64_t)(r0 + (i >> 4)) * p.ldd + n) * elt_size(OT), 0.0f);
      }
      return;
    }
    b += (int64_t)found * p.b_e;
    sb += (int64_t)found * p.sb_e;
  } else {
    r0 = 0;
    r1 = p.M;
  }
  const int nkb = (p.K + kScaleBlock - 1) / kScaleBlock;
  const int nv = min(16, p.N - n0);
  const __amdgpu_buffer_rsrc_t rb = rsrc_of(b + (int64_t)n0 * p.ldb, (int64_t)(nv - 1) * p.ldb + p.K);
  const float* sbp = sb + (int64_t)(n0 / kScaleBlock) * p.sb_n;
  const int ldb = (int)p.ldb, n_mine = (nkb - wave + NW - 1) / NW;
  // as in the tiles, piece c of row r is kept at piece c ^ (r & 7); rows past nv or mv are past the descriptors' ranges
  const int row = lane >> 3, piece16 = ((lane & 7) ^ row) * 16;
  const uint32_t boff = (uint32_t)(row * ldb + piece16), aoff = (uint32_t)(row * (int)p.lda + piece16);
  const int bread = (lane & 15) * 128 + ((lane >> 4) ^ (lane & 7)) * 16;
  const int aread = AT_A + (lane & 7) * 128 + ((lane >> 4) ^ (lane & 7)) * 16;
  char* const mine = ring + wave * (D * SLOT);
  for (int m0 = r0; m0 < r1; m0 += 8) {
    const int mv = min(8, r1 - m0);
    const __amdgpu_buffer_rsrc_t ra = rsrc_of(p.a + (int64_t)m0 * p.lda, (int64_t)(mv - 1) * p.lda + p.K);
    const float* sap = p.sa + (int64_t)m0 * p.sa_m;
    const float* sp = (lane < 8 ? sap + min(lane, mv - 1) * p.sa_m + wave * p.sa_k : sbp + wave * p.sb_k);
    const int64_t s_step = NW * (lane < 8 ? p.sa_k : p.sb_k);
    if (n_mine <= 0) sp = sbp;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    typedef __attribute__((address_space(3))) void* Lds;
    auto load = [&](int i, char* slot) __attribute__((always_inline)) {  // the wave's i-th block; nothing past its last
      const int kb = wave + i * NW, k = min(kb, nkb - 1) * kScaleBlock;
      const bool in = kb < nkb && k + piece16 < p.K;
      const uint32_t bo = in ? boff : kOOB, ao = in ? aoff : kOOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (Lds)slot, 16, (int)bo, k, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (Lds)(slot + 1024), 16, (int)(bo + 8 * ldb), k, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (Lds)(slot + AT_A), 16, (int)ao, k, 0, 0);
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)sp, (Lds)(slot + AT_S), 4, 0, 0);
      if (kb + NW < nkb) sp += s_step;
    };
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, mine + d * SLOT);
    char* slot = mine;
    for (int i = 0; i < n_mine; ++i) {
      constexpr int kWait = (D - 1) * 4;
      __builtin_amdgcn_s_waitcnt((kWait & 15) | ((kWait >> 4) << 14) | 0x0f70);  // the block has landed
      asm volatile("" ::: "memory");
      const i32x8 vb = join8(*(const u32x4*)(slot + bread), *(const u32x4*)(slot + (bread ^ 64)));
      const i32x8 va = join8(*(const u32x4*)(slot + aread), *(const u32x4*)(slot + (aread ^ 64)));
      const float t = *(const float*)(slot + AT_S + (lane & 7) * 4) * *(const float*)(slot + AT_S + 32);
      __builtin_amdgcn_s_waitcnt(0xc07f);  // and is in registers: its place is free
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      load(i + D, slot);
      acc += mfma128(widen(vb), widen(va)) * t;
      slot = slot == mine + (D - 1) * SLOT ? mine : slot + SLOT;
    }
    __builtin_amdgcn_s_waitcnt(0x0f70);  // (the loads past the end write LDS too: not into the next rows' blocks)
    __syncthreads();
    f32x4* const red = (f32x4*)ring;
    red[wave * 64 + lane] = acc;
    __syncthreads();
    for (int o = threadIdx.x; o < 128; o += 64 * NW) {
      const int m = o >> 4, n = o & 15;  // n = 4 q + r of lane 16 q + m
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) v += ((const float*)&red[w * 64 + (n >> 2) * 16 + m])[n & 3];
      if (m < mv && n < nv) store_elt<OT>((char*)p.d + ((int64_t)(m0 + m) * p.ldd + n0 + n) * elt_size(OT), v);
    }
    __syncthreads();
  }
}

// (fewer than 2^24, which the C ABI has checked)
template <int MODE, int BM, int BN>
int64_t count_tiles(Fp8Gemm& p) {
  p.tiles_n = (p.N + BN - 1) / BN;
  p.tiles_m = (p.M + BM - 1) / BM;
  if (MODE == GM_GROUPED) p.tiles_m += (p.experts < p.M ? p.experts : p.M) + 1;  // (at most)
  return (int64_t)p.tiles_m * p.tiles_n * (MODE == GM_WGRAD ? p.experts : p.splits);
}

// As many workgroups as run at once (a multiple of 8: a workgroup's tiles are all of one XCD's share).
template <int MODE, int OT, int BM, int BN, int WGM, int WGN, int PER_CU>
hipError_t launch_tile(Fp8Gemm& p, hipStream_t s) {
  const int64_t tiles = count_tiles<MODE, BM, BN>(p);
  const int whole = (p.cus >= 8 ? p.cus & ~7 : 8) * PER_CU;
  fp8_tile_kernel<MODE, OT, BM, BN, WGM, WGN, 2><<<(unsigned)(tiles < whole ? tiles : whole), 64 * WGM * WGN, 0, s>>>(p);
  return hipGetLastError();
}

template <int MODE, int OT>
hipError_t launch_wide(Fp8Gemm& p, hipStream_t s) {
  const int64_t tiles = count_tiles<MODE, 128, 128>(p);
  fp8_wide_kernel<MODE, OT, 128, 128, 2, 2><<<(unsigned)tiles, 256, 0, s>>>(p);
  return hipGetLastError();
}

template <int MODE, int OT>
hipError_t launch_tiles(Fp8Gemm& p, hipStream_t s) {
  if constexpr (MODE == GM_MATMUL) {
    if (p.splits > 1) {
      Fp8Gemm q = p;
      q.d = p.part;
      q.ldd = p.N;
      const hipError_t e = OT == EL_F32 ? launch_wide<MODE, EL_F32>(q, s) : launch_tile<MODE, EL_F32, 128, 128, 2, 2, 2>(q, s);
      if (e != hipSuccess) return e;
      const int64_t b = ((int64_t)p.M * p.N + 2047) / 2048;
      fp8_join_kernel<OT><<<(unsigned)(b < 4096 ? b : 4096), 256, 0, s>>>(p);
      return hipGetLastError();
    }
  }
  if constexpr (OT != EL_F32) {
    if (MODE == GM_WGRAD || p.K > 2 * kScaleBlock) {
      // fewer 256 x 256 tiles than compute units: 128 x 128 ones, two workgroups a unit (777 x 5003 x 4112: 36 us
      // with operands that no cache holds, 59 with 80 large tiles); with more the large ones, which read half as much
      // through the caches (8192 x 17408 x 5120: 602 us, 744 with small ones)
      const int64_t big = (int64_t)((p.M + 255) / 256) * ((p.N + 255) / 256) * (MODE == GM_WGRAD ? p.experts : 1);
      // so with few rows an expert: 64 experts of 64 rows, n 4096, k 5120: 244 us, 267 with large tiles (of 128: 282, 281)
      if (big < p.cus || (MODE == GM_GROUPED && p.M <= 96 * (int64_t)p.experts)) return launch_tile<MODE, OT, 128, 128, 2, 2, 2>(p, s);
      return launch_tile<MODE, OT, 256, 256, 4, 2, 1>(p, s);
    }
  }
  return launch_wide<MODE, OT>(p, s);
}

template <int MODE, int OT>
hipError_t launch_rows(Fp8Gemm& p, hipStream_t s) {
  const unsigned groups = MODE == GM_GROUPED ? (unsigned)((p.experts < p.M ? p.experts : p.M) + 1) : 1u;
  const dim3 grid((unsigned)((p.N + 15) / 16), groups);
  fp8_rows_kernel<MODE, OT><<<grid, 64 * kRowsWaves, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

// K ranges of a product with few tiles.  A step of 128 x 128 tiles takes 0.6 us with two of them on every compute
// unit; ranges cost a launch (5 us) and their parts' way through memory, written and read at about 4 TB/s.  By
// this model 64 x 5120 x 5120 takes 5 ranges (17 us, unsplit 35), 128 x 5120 x 17408 takes 8 (39 us, unsplit 110),
// 1024 x 4096 x 5120 none (36 us, 40 with 2); operands that no cache holds.
int fp8_splits(int m, int n, int k) {
  const int64_t tiles = (int64_t)((m + 127) / 128) * ((n + 127) / 128);
  const int blocks = (k + kScaleBlock - 1) / kScaleBlock;
  int best = 1;
  double least = blocks * 0.6;
  for (int s = 2; s * tiles <= kTilesAtOnce && s <= blocks / 4; ++s) {
    const int each = (blocks + s - 1) / s, parts = (blocks + each - 1) / each;
    const double us = each * 0.6 + 5.0 + 8.0 * parts * m * n / 4e6;
    if (us < least) {
      least = us;
      best = parts;
    }
  }
  return best;
}

hipError_t launch_fp8_tiles(int mode, int out, Fp8Gemm& p, hipStream_t s) {
#define EP_CASE(M_, O_) \
  if (mode == M_ && out == O_) return launch_tiles<M_, O_>(p, s);
  EP_CASE(GM_MATMUL, EL_F16) EP_CASE(GM_MATMUL, EL_BF16) EP_CASE(GM_MATMUL, EL_F32)
  EP_CASE(GM_GROUPED, EL_F16) EP_CASE(GM_GROUPED, EL_BF16) EP_CASE(GM_GROUPED, EL_F32)
  EP_CASE(GM_WGRAD, EL_F16) EP_CASE(GM_WGRAD, EL_BF16) EP_CASE(GM_WGRAD, EL_F32)
#undef EP_CASE
  return hipErrorInvalidValue;
}

hipError_t launch_fp8_rows(int mode, int out, Fp8Gemm& p, hipStream_t s) {
#define EP_CASE(M_, O_) \
  if (mode == M_ && out == O_) return launch_rows<M_, O_>(p, s);
  EP_CASE(GM_MATMUL, EL_F16) EP_CASE(GM_MATMUL, EL_BF16) EP_CASE(GM_MATMUL, EL_F32)
  EP_CASE(GM_GROUPED, EL_F16) EP_CASE(GM_GROUPED, EL_BF16) EP_CASE(GM_GROUPED, EL_F32)
#undef EP_CASE
  return hipErrorInvalidValue;
}

}  // namespace ep
