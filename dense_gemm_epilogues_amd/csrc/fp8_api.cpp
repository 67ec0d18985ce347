// C ABI of the 8-bit block-scaled products and the expert operators: validation and dispatch.  Every
// call only enqueues kernels; workspaces are the caller's.
#include "ep.h"
#include "api_shared.hpp"
#include "fp8_ops.hpp"

using namespace ep;

namespace {

constexpr int64_t kMaxLd8 = (int64_t)1 << 23;  // 256 rows stay inside one 2^31-byte buffer window
constexpr int64_t kMaxCount = ((int64_t)1 << 31) - 4096;
constexpr int64_t kMaxScaleStride = (int64_t)1 << 21;  // as are 256 rows' scales

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
ep_status done(hipError_t e, const char* what) {
  if (e != hipSuccess) return (ep_status)api_fail(EP_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return EP_OK;
}
#define EP_REQUIRE(cond, status, ...) \
  do {                                \
    if (!(cond)) return (ep_status)api_fail(status, __VA_ARGS__); \
  } while (0)

ep_status check_elt(int elt) {
  EP_REQUIRE(elt == EP_ELT_F16 || elt == EP_ELT_BF16 || elt == EP_ELT_F32, EP_ERR_UNSUPPORTED, "unknown element type %d", elt);
  return EP_OK;
}

// what the three products check alike; `rows_a` and `rows_b` are the operands' row counts, k their length
ep_status check_product(int64_t rows_a, int64_t rows_b, int64_t k, const void* a, int64_t lda, const float* sa,
                        int64_t sa_m, int64_t sa_k, const void* b, int64_t ldb, const float* sb, int64_t sb_n,
                        int64_t sb_k, const void* d, int64_t ldd, int64_t n, int out) {
  EP_REQUIRE(rows_a >= 1 && rows_b >= 1 && k >= 1, EP_ERR_INVALID_ARG, "sizes must be at least 1");
  EP_REQUIRE(rows_a < kMaxCount && rows_b < kMaxCount, EP_ERR_UNSUPPORTED, "sizes must be below 2^31 - 4096");
  EP_REQUIRE(k % 16 == 0, EP_ERR_UNSUPPORTED, "the contracted length (%lld) must be a multiple of 16", (long long)k);
  EP_REQUIRE(a && sa && b && sb && d, EP_ERR_INVALID_ARG, "null operand, scale or output pointer");
  EP_REQUIRE(aligned(a, 16) && aligned(b, 16), EP_ERR_INVALID_ARG, "operands must be 16-byte aligned");
  EP_REQUIRE(lda >= k && ldb >= k && lda % 16 == 0 && ldb % 16 == 0, EP_ERR_INVALID_ARG,
             "operand row strides must be multiples of 16 and at least the contracted length");
  EP_REQUIRE(lda < kMaxLd8 && ldb < kMaxLd8, EP_ERR_UNSUPPORTED, "operand row strides must be below 2^23");
  EP_REQUIRE(aligned(sa, 4) && aligned(sb, 4), EP_ERR_INVALID_ARG, "scales must be 4-byte aligned");
  EP_REQUIRE(sa_m >= 0 && sa_k >= 0 && sb_n >= 0 && sb_k >= 0, EP_ERR_INVALID_ARG, "negative scale stride");
  EP_REQUIRE(sa_m < kMaxScaleStride, EP_ERR_UNSUPPORTED, "the row stride of a's scales must be below 2^21");
  // (a tile's second scale ends inside a window of 2^31 - 1 bytes)
  EP_REQUIRE(sb_n < ((int64_t)1 << 29) - 1, EP_ERR_UNSUPPORTED, "the row stride of b's scales must be below 2^29 - 1");
  EP_REQUIRE(ldd >= n, EP_ERR_INVALID_ARG, "output row stride below the row length");
  const ep_status st = check_elt(out);
  if (st != EP_OK) return st;
  EP_REQUIRE(aligned(d, elt_size(out)), EP_ERR_INVALID_ARG, "misaligned output");
  return EP_OK;
}

// 128 x 128 tiles of 256 threads, one a workgroup, in a launch of fewer than 2^32 threads.  (The kernels that walk
// larger tiles have fewer.)
ep_status check_tiles(int64_t tiles_m, int64_t tiles_n, int64_t parts) {
  constexpr int64_t kMost = ((int64_t)1 << 24) - 1;
  EP_REQUIRE(tiles_m * tiles_n <= kMost && tiles_m * tiles_n * parts <= kMost, EP_ERR_UNSUPPORTED,
             "the output has too many tiles for one launch");
  return EP_OK;
}
int64_t tiles_of(int64_t n) { return (n + 127) / 128; }

// Products that stream b past a few rows, without tiles: matmuls of up to 8 rows (8 x 17408 x 5120 in 19.5 us, 25 in
// tiles with K ranges; 16 rows 32, 25.5 in tiles; operands that no cache holds) and up to 4 rows an expert on average (64
// experts, n 4096, k 5120: 8 rows in 27 us, 33 in tiles, 32 rows in 107 and 117, 256 in 216 and 228, 384 even).  The
// offsets are on the device, so the largest group is not known here: 256 rows, all of one expert, take 137 us (28.5 in
// tiles), half of them as long as in tiles (251).  A workgroup of 256 threads takes 16 columns, so from 2^28 columns
// on, where a launch would pass 2^32 threads, tiles take these too.
constexpr int64_t kRowsPath = 8;
constexpr int64_t kRowsColumns = ((int64_t)1 << 28) - 16;
bool few_rows(int64_t rows, int64_t n, int64_t experts) { return rows <= 4 * experts && n <= kRowsColumns; }
bool few_rows(int64_t rows, int64_t n) { return rows <= kRowsPath && n <= kRowsColumns; }

}  // namespace

extern "C" {

ep_status ep_quantize_fp8(const void* x, int64_t m, int64_t k, int64_t ldx, int elt, int block_rows, int transpose,
                          void* q, int64_t ldq, float* scale, void* stream) {
  api_clear();
  EP_REQUIRE(m >= 1 && k >= 1, EP_ERR_INVALID_ARG, "sizes must be at least 1");
  EP_REQUIRE(m < kMaxCount && k < kMaxCount, EP_ERR_UNSUPPORTED, "sizes must be below 2^31 - 4096");
  EP_REQUIRE(x && q && scale, EP_ERR_INVALID_ARG, "null pointer");
  ep_status st = check_elt(elt);
  if (st != EP_OK) return st;
  EP_REQUIRE(block_rows == 1 || block_rows == 128, EP_ERR_UNSUPPORTED, "scale blocks are 1 x 128 or 128 x 128");
  EP_REQUIRE(aligned(x, elt_size(elt)) && aligned(scale, 4), EP_ERR_INVALID_ARG, "misaligned pointer");
  EP_REQUIRE(ldx >= k && ldq >= (transpose ? m : k), EP_ERR_INVALID_ARG, "row stride below the row length");
  EP_REQUIRE(quantize_blocks(block_rows, transpose != 0, m, k) < ((int64_t)1 << 24), EP_ERR_UNSUPPORTED,
             "the matrix has too many blocks for one launch");  // (workgroups of 256 threads, fewer than 2^32 of those)
  if ((st = (ep_status)api_stream(stream)) != EP_OK) return st;
  QuantArgs p{x, ldx, (int)m, (int)k, (uint8_t*)q, ldq, scale};
  return done(launch_quantize(elt, block_rows, transpose != 0, p, (hipStream_t)stream), "quantize_fp8");
}

ep_status ep_matmul_fp8_workspace(int64_t m, int64_t n, int64_t k, size_t* bytes) {
  api_clear();
  EP_REQUIRE(bytes, EP_ERR_INVALID_ARG, "null pointer");
  *bytes = 0;
  if (m < 1 || n < 1 || k < 1 || m >= kMaxCount || n >= kMaxCount || k >= kMaxLd8 || few_rows(m, n)) return EP_OK;
  const int s = fp8_splits((int)m, (int)n, (int)k);
  if (s > 1) *bytes = (size_t)s * m * n * 4;
  return EP_OK;
}

ep_status ep_matmul_fp8(int64_t m, int64_t n, int64_t k, const void* a, int64_t lda, const float* sa, int64_t sa_m,
                        int64_t sa_k, const void* b, int64_t ldb, const float* sb, int64_t sb_n, int64_t sb_k, void* d,
                        int64_t ldd, int out, void* workspace, size_t workspace_bytes, void* stream) {
  api_clear();
  ep_status st = check_product(m, n, k, a, lda, sa, sa_m, sa_k, b, ldb, sb, sb_n, sb_k, d, ldd, n, out);
  if (st != EP_OK) return st;
  Fp8Gemm p{};
  p.a = (const uint8_t*)a; p.b = (const uint8_t*)b; p.sa = sa; p.sb = sb; p.d = d;
  p.lda = lda; p.ldb = ldb; p.ldd = ldd;
  p.sa_m = sa_m; p.sa_k = sa_k; p.sb_n = sb_n; p.sb_k = sb_k;
  p.M = (int)m; p.N = (int)n; p.K = (int)k;
  p.splits = 1;
  p.kb_per_split = (int)((k + 127) / 128);
  const bool rows = few_rows(m, n);
  if (!rows) {
    if ((st = check_tiles(tiles_of(m), tiles_of(n), 1)) != EP_OK) return st;
    p.splits = fp8_splits(p.M, p.N, p.K);
    if (p.splits > 1) {
      EP_REQUIRE(workspace && workspace_bytes >= (size_t)p.splits * m * n * 4, EP_ERR_INVALID_ARG,
                 "the workspace is smaller than ep_matmul_fp8_workspace says");
      EP_REQUIRE(aligned(workspace, 16), EP_ERR_INVALID_ARG, "the workspace must be 16-byte aligned");
      p.kb_per_split = (p.kb_per_split + p.splits - 1) / p.splits;
      p.part = (float*)workspace;
    }
  }
  if ((st = (ep_status)api_stream(stream, &p.cus)) != EP_OK) return st;
  if (rows) return done(launch_fp8_rows(GM_MATMUL, out, p, (hipStream_t)stream), "matmul_fp8");
  return done(launch_fp8_tiles(GM_MATMUL, out, p, (hipStream_t)stream), "matmul_fp8");
}

ep_status ep_grouped_matmul_fp8(int64_t rows, int64_t n, int64_t k, int64_t experts, const int32_t* offsets, const void* a,
                                int64_t lda, const float* sa, int64_t sa_m, int64_t sa_k, const void* b, int64_t b_e,
                                int64_t ldb, const float* sb, int64_t sb_e, int64_t sb_n, int64_t sb_k, void* d, int64_t ldd,
                                int out, void* stream) {
  api_clear();
  ep_status st = check_product(rows, n, k, a, lda, sa, sa_m, sa_k, b, ldb, sb, sb_n, sb_k, d, ldd, n, out);
  if (st != EP_OK) return st;
  EP_REQUIRE(experts >= 1 && offsets, EP_ERR_INVALID_ARG, "at least one expert and its offsets are needed");
  EP_REQUIRE(experts < 65535, EP_ERR_UNSUPPORTED, "at most 65534 experts");
  EP_REQUIRE(aligned(offsets, 4), EP_ERR_INVALID_ARG, "misaligned offsets");
  EP_REQUIRE(b_e >= 0 && sb_e >= 0 && b_e % 16 == 0, EP_ERR_INVALID_ARG, "the expert stride of b must be a multiple of 16");
  const bool few = few_rows(rows, n, experts);
  if (!few && (st = check_tiles(tiles_of(rows) + (experts < rows ? experts : rows) + 1, tiles_of(n), 1)) != EP_OK) return st;
  Fp8Gemm p{};
  if ((st = (ep_status)api_stream(stream, &p.cus)) != EP_OK) return st;
  p.a = (const uint8_t*)a; p.b = (const uint8_t*)b; p.sa = sa; p.sb = sb; p.d = d;
  p.lda = lda; p.ldb = ldb; p.ldd = ldd;
  p.sa_m = sa_m; p.sa_k = sa_k; p.sb_n = sb_n; p.sb_k = sb_k;
  p.b_e = b_e; p.sb_e = sb_e;
  p.offsets = offsets; p.experts = (int)experts;
  p.M = (int)rows; p.N = (int)n; p.K = (int)k;
  p.splits = 1;
  if (few)
    return done(launch_fp8_rows(GM_GROUPED, out, p, (hipStream_t)stream), "grouped_matmul_fp8");
  return done(launch_fp8_tiles(GM_GROUPED, out, p, (hipStream_t)stream), "grouped_matmul_fp8");
}

ep_status ep_grouped_wgrad_fp8(int64_t m, int64_t n, int64_t rows, int64_t experts, const int32_t* offsets, const void* a,
                               int64_t lda, const float* sa, int64_t sa_m, int64_t sa_k, const void* b, int64_t ldb,
                               const float* sb, int64_t sb_n, int64_t sb_k, void* d, int64_t ldd, int out, void* stream) {
  api_clear();
  ep_status st = check_product(m, n, rows, a, lda, sa, sa_m, sa_k, b, ldb, sb, sb_n, sb_k, d, ldd, n, out);
  if (st != EP_OK) return st;
  EP_REQUIRE(experts >= 1 && offsets, EP_ERR_INVALID_ARG, "at least one expert and its offsets are needed");
  EP_REQUIRE(experts < 65535, EP_ERR_UNSUPPORTED, "at most 65534 experts");
  EP_REQUIRE(aligned(offsets, 4), EP_ERR_INVALID_ARG, "misaligned offsets");
  if ((st = check_tiles(tiles_of(m), tiles_of(n), experts)) != EP_OK) return st;
  Fp8Gemm p{};
  if ((st = (ep_status)api_stream(stream, &p.cus)) != EP_OK) return st;
  p.a = (const uint8_t*)a; p.b = (const uint8_t*)b; p.sa = sa; p.sb = sb; p.d = d;
  p.lda = lda; p.ldb = ldb; p.ldd = ldd;
  p.sa_m = sa_m; p.sa_k = sa_k; p.sb_n = sb_n; p.sb_k = sb_k;
  p.offsets = offsets; p.experts = (int)experts;
  p.M = (int)m; p.N = (int)n; p.K = (int)rows;
  p.splits = 1;
  return done(launch_fp8_tiles(GM_WGRAD, out, p, (hipStream_t)stream), "grouped_wgrad_fp8");
}

ep_status ep_expert_order_sizes(int64_t slots, int64_t experts, int64_t align, int64_t* capacity, size_t* workspace_bytes) {
  api_clear();
  EP_REQUIRE(capacity && workspace_bytes, EP_ERR_INVALID_ARG, "null pointer");
  EP_REQUIRE(slots >= 0 && experts >= 1 && align >= 1, EP_ERR_INVALID_ARG, "sizes must be at least 1 (slots: 0)");
  EP_REQUIRE(experts <= 1024 && align <= 4096 && slots < kMaxCount, EP_ERR_UNSUPPORTED,
             "at most 1024 experts, rows aligned to at most 4096, below 2^31 - 4096 slots");
  const int64_t padded = slots + (experts < slots ? experts : slots) * (align - 1);
  *capacity = (padded + align - 1) / align * align;
  EP_REQUIRE(*capacity < kMaxCount, EP_ERR_UNSUPPORTED, "the ordered rows pass 2^31 - 4096");
  const int blocks = order_blocks((int)slots);
  *workspace_bytes = blocks > 1 ? (size_t)blocks * experts * 4 : 0;
  return EP_OK;
}

ep_status ep_expert_order(const void* ids, int id_bytes, int64_t slots, int64_t experts, int64_t align, int32_t* pos,
                          int32_t* src, int32_t* offsets, void* workspace, size_t workspace_bytes, void* stream) {
  int64_t capacity = 0;
  size_t need = 0;
  ep_status st = ep_expert_order_sizes(slots, experts, align, &capacity, &need);
  if (st != EP_OK) return st;
  EP_REQUIRE(id_bytes == 4 || id_bytes == 8, EP_ERR_UNSUPPORTED, "expert ids are 32 or 64 bits");
  EP_REQUIRE(offsets && (slots == 0 || (ids && pos && src)), EP_ERR_INVALID_ARG, "null pointer");
  EP_REQUIRE(aligned(ids, id_bytes) && aligned(pos, 4) && aligned(src, 4) && aligned(offsets, 4), EP_ERR_INVALID_ARG,
             "misaligned pointer");
  EP_REQUIRE(need == 0 || (workspace && workspace_bytes >= need && aligned(workspace, 4)), EP_ERR_INVALID_ARG,
             "the workspace is smaller than ep_expert_order_sizes says");
  if ((st = (ep_status)api_stream(stream)) != EP_OK) return st;
  OrderArgs p{ids, id_bytes, (int)slots, (int)experts, (int)align, (int)capacity, pos, src, offsets, (int*)workspace};
  return done(launch_order(p, (hipStream_t)stream), "expert_order");
}

ep_status ep_expert_dispatch(const void* x, int64_t tokens, int64_t h, int64_t ldx, int elt, const int32_t* pos, int64_t topk,
                             const int32_t* src, int64_t rows, void* out, int64_t ldo, float* scale, void* stream) {
  api_clear();
  EP_REQUIRE(tokens >= 0 && h >= 1 && topk >= 1 && rows >= 1, EP_ERR_INVALID_ARG, "sizes must be at least 1 (tokens: 0)");
  EP_REQUIRE(h < ((int64_t)1 << 26) && rows < kMaxCount && tokens < kMaxCount && topk <= 65536, EP_ERR_UNSUPPORTED, "sizes out of range");
  ep_status st = check_elt(elt);
  if (st != EP_OK) return st;
  EP_REQUIRE(src && out && (tokens == 0 || (x && pos)), EP_ERR_INVALID_ARG, "null pointer");
  EP_REQUIRE(aligned(x, elt_size(elt)) && aligned(out, scale ? 1 : elt_size(elt)) && aligned(pos, 4) && aligned(src, 4) &&
                 aligned(scale, 4), EP_ERR_INVALID_ARG, "misaligned pointer");
  EP_REQUIRE(ldx >= h && ldo >= h, EP_ERR_INVALID_ARG, "row stride below the row length");
  EP_REQUIRE(tokens + (rows + 63) / 64 < ((int64_t)1 << 23), EP_ERR_UNSUPPORTED, "too many tokens for one launch");
  // (copied as 16-bit pieces, 2048 of them to each of at most 65535 workgroups)
  EP_REQUIRE(scale || elt != EP_ELT_F32 || h <= (int64_t)65535 * 1024, EP_ERR_UNSUPPORTED, "rows of fp32 values have at most 65535 * 1024");
  if ((st = (ep_status)api_stream(stream)) != EP_OK) return st;
  ExpertRows p{};
  p.x = x; p.ldx = ldx; p.out = out; p.ldo = ldo; p.pos = pos; p.src = src; p.scale = scale;
  p.tokens = (int)tokens; p.topk = (int)topk; p.rows = (int)rows; p.h = (int)h;
  return done(launch_dispatch(elt, scale != nullptr, p, (hipStream_t)stream), "expert_dispatch");
}

ep_status ep_expert_combine(const void* y, int64_t rows, int64_t h, int64_t ldy, int elt, const int32_t* pos, int64_t tokens,
                            int64_t topk, const float* w, int64_t ldw, void* out, int64_t ldo, void* stream) {
  api_clear();
  EP_REQUIRE(tokens >= 1 && h >= 1 && topk >= 1 && rows >= 0, EP_ERR_INVALID_ARG, "sizes must be at least 1 (rows: 0)");
  EP_REQUIRE(h < ((int64_t)1 << 26) && rows < kMaxCount && topk <= 65536, EP_ERR_UNSUPPORTED, "sizes out of range");
  ep_status st = check_elt(elt);
  if (st != EP_OK) return st;
  EP_REQUIRE(pos && out && (rows == 0 || y), EP_ERR_INVALID_ARG, "null pointer");
  EP_REQUIRE(aligned(y, elt_size(elt)) && aligned(out, elt_size(elt)) && aligned(pos, 4) && aligned(w, 4), EP_ERR_INVALID_ARG,
             "misaligned pointer");
  EP_REQUIRE(ldy >= h && ldo >= h && (!w || ldw >= topk), EP_ERR_INVALID_ARG, "row stride below the row length");
  EP_REQUIRE(tokens < ((int64_t)1 << 23), EP_ERR_UNSUPPORTED, "too many tokens for one launch");
  if ((st = (ep_status)api_stream(stream)) != EP_OK) return st;
  ExpertRows p{};
  p.x = y; p.ldx = ldy; p.out = out; p.ldo = ldo; p.pos = pos; p.w = w; p.ldw = ldw;
  p.tokens = (int)tokens; p.topk = (int)topk; p.rows = (int)rows; p.h = (int)h;
  return done(launch_combine(elt, p, (hipStream_t)stream), "expert_combine");
}

ep_status ep_expert_combine_backward(const void* dout, int64_t tokens, int64_t h, int64_t ld_dout, int elt, const void* y,
                                     int64_t rows, int64_t ldy, const int32_t* pos, int64_t topk, const int32_t* src,
                                     const float* w, int64_t ldw, void* dy, int64_t ld_dy, float* dw, void* stream) {
  api_clear();
  EP_REQUIRE(tokens >= 0 && h >= 1 && topk >= 1 && rows >= 0, EP_ERR_INVALID_ARG, "sizes must be at least 1 (tokens, rows: 0)");
  EP_REQUIRE(h < ((int64_t)1 << 26) && rows < kMaxCount && topk <= 65536, EP_ERR_UNSUPPORTED, "sizes out of range");
  ep_status st = check_elt(elt);
  if (st != EP_OK) return st;
  EP_REQUIRE((tokens == 0 || (dout && pos && dw)) && (rows == 0 || (y && dy && src)), EP_ERR_INVALID_ARG, "null pointer");
  EP_REQUIRE(aligned(y, elt_size(elt)) && aligned(dout, elt_size(elt)) && aligned(dy, elt_size(elt)) && aligned(pos, 4) &&
                 aligned(src, 4) && aligned(w, 4) && aligned(dw, 4), EP_ERR_INVALID_ARG, "misaligned pointer");
  EP_REQUIRE(ldy >= h && ld_dout >= h && ld_dy >= h && (!w || ldw >= topk), EP_ERR_INVALID_ARG, "row stride below the row length");
  EP_REQUIRE(tokens + (rows + 63) / 64 < ((int64_t)1 << 23), EP_ERR_UNSUPPORTED, "too many tokens for one launch");
  if (tokens == 0 && rows == 0) return EP_OK;
  if ((st = (ep_status)api_stream(stream)) != EP_OK) return st;
  ExpertRows p{};
  p.x = y; p.ldx = ldy; p.dout = dout; p.ld_dout = ld_dout; p.out = dy; p.ldo = ld_dy; p.pos = pos; p.src = src;
  p.w = w; p.ldw = ldw; p.dw = dw;
  p.tokens = (int)tokens; p.topk = (int)topk; p.rows = (int)rows; p.h = (int)h;
  return done(launch_combine_backward(elt, p, (hipStream_t)stream), "expert_combine_backward");
}

}  // extern "C"
