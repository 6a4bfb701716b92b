// Kernel launchers of libnf4lora (implemented in the .hip files).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "nf4_host.hpp"

namespace nf4k {

enum { MODE_FWD = 0, MODE_DX = 1 };

// codes2/absmax2/dqs2: the residual (second-stage) tensor, or NULL for one stage.
hipError_t launch_quantize(const float* W, int64_t nblocks, bool dq, uint8_t* codes, void* absmax, float* dqs,
                           uint8_t* codes2, void* absmax2, float* dqs2, const NF4Enc& e, const NF4Consts& c,
                           hipStream_t st);
hipError_t launch_dequantize(const uint8_t* codes, const void* absmax, const float* dqs, const uint8_t* codes2,
                             const void* absmax2, const float* dqs2, int64_t nweights, bool dq, bool bf16, void* out,
                             const NF4Consts& c, hipStream_t st);
// nf4 quantize of one stage plus the reconstruction error of W (as launch_error
// computes it) from the same read of W; err_dq: error with the double-quantized
// scales (requires dq) rather than the plain block absmax.
hipError_t launch_quantize_error(const float* W, int64_t nblocks, bool dq, uint8_t* codes, void* absmax, float* dqs,
                                 bool err_dq, double* part, double* err, const NF4Enc& e, const NF4Consts& c,
                                 hipStream_t st);
hipError_t launch_error(const float* W, int64_t nblocks, bool dq, double* part, double* err, const NF4Enc& c,
                        hipStream_t st);
// launch_error for n linears (W[i], rows[i] x cols[i]) in batches of up to 64:
// err[i] as launch_error writes it for linear i, bit for bit; part holds one
// (D, Wn) pair per group of every linear, linear after linear.
hipError_t launch_error_batch(const float* const* W, const int64_t* rows, const int64_t* cols, int32_t n, bool dq,
                              double* part, double* err, const NF4Enc& c, hipStream_t st);
hipError_t launch_topk(const double* e, int n, int k, int* idx, hipStream_t st);
// Workspace of the allocation-free forward: one device array of this size per
// GPU (scratch.hip).  noalloc_scratch gives its address on the current device.
constexpr size_t kNoAllocScratchBytes = (size_t)16 << 20;
hipError_t noalloc_scratch(void** ptr);

// MFMA-only probe: `workgroups` x 512 threads, each wave `iters` rounds of 8
// v_mfma_f32_32x32x16_bf16; out gets one float per thread.
hipError_t launch_mfma_peak(int iters, int workgroups, float* out, hipStream_t st);
// *flag_dev = 1 if any of W[0 .. count) is an infinity or a NaN, else 0.
hipError_t launch_check_finite(const float* W, int64_t count, int* flag_dev, hipStream_t st);

// The passes over W (quantize, error) run one 256-thread workgroup per group of
// 256 blocks; a launch holds at most kMaxLaunchGroups groups, so its work-item
// count (groups * 256) stays below 2^32.  Up to kErrBatch linears share one
// launch of the batched error pass.
constexpr int64_t kMaxLaunchGroups = ((int64_t)1 << 24) - 1;
constexpr int kErrBatch = 64;
inline int64_t error_groups(int64_t rows, int64_t cols) { return (rows * cols / 64 + 255) / 256; }
// The next launch of a batched error pass over n linears starts at linear c0
// and takes the k linears c0 .. c0 + k - 1 (the return value): as many as fit in
// kErrBatch linears and kMaxLaunchGroups groups.  g0[i] is the first group of
// linear c0 + i within the launch and g0[k] the launch's group count (g0 has
// kErrBatch + 1 entries).  Returns 0 when linear c0 alone has more than
// kMaxLaunchGroups groups.
int error_batch_chunk(const int64_t* rows, const int64_t* cols, int32_t n, int32_t c0, int64_t* g0);

// Weight source of the fused GEMM: NF4 with fp32 absmax, NF4 with 8-bit
// double-quantized scales, or a bf16 weight (no quantization).
enum { kSrcNF4 = 0, kSrcNF4DQ = 1, kSrcBF16 = 2 };
// Tail B2: [N][R] (b2kn == 0), or k-major [R][N] with rows b2kn .. R-1 absent (read as zero).
hipError_t launch_nf4_gemm(int mode, int src, const uint16_t* A, const uint16_t* Wb, const uint8_t* codes,
                           const void* absmax, const float* dqs, const uint8_t* codes2, const void* absmax2,
                           const float* dqs2, const uint16_t* A2, const uint16_t* B2, int R, int b2kn, uint16_t* C,
                           int64_t M, int N, int K, const NF4Consts& c, hipStream_t st);

// W' = base + s (L1 L2)^T into fp32 or bf16; base 0: fp32 W, 1: NF4, 2: NF4 with 8-bit scales.
hipError_t launch_merge(int base, const float* W, const uint8_t* codes, const void* absmax, const float* dqs,
                        const uint8_t* codes2, const void* absmax2, const float* dqs2, const uint16_t* L1,
                        const uint16_t* L2, int r, float s, int64_t rows, int64_t cols, bool out_bf16, void* out,
                        const NF4Consts& c, hipStream_t st);

// One launch of k_prep: up to kPrepPads layout copies and kPrepZeros clears.
// Unused jobs have orows * ocols == 0 / n == 0.
constexpr int kPrepPads = 3;
constexpr int kPrepZeros = 2;
struct PadJob {  // out[i][j] = (i < irows && j < jcols) ? in[i*si + j*sj] : 0, out is [orows][ocols]
  const uint16_t* in;
  uint16_t* out;
  int64_t si, sj, irows, jcols, orows, ocols;
};
struct ZeroJob {
  uint32_t* p;
  int64_t n;  // 32-bit words
};
struct PrepArgs {
  PadJob pad[kPrepPads];
  ZeroJob zero[kPrepZeros];
};
hipError_t launch_prep(const PrepArgs& a, hipStream_t st);

// NT skinny product with its split reduction: out = alpha * A[M][K] B[RP][K]^T.
struct NtArgs {
  const uint16_t* A;
  const uint16_t* B;
  int64_t M;
  int K;
  int ksplit, krange;
  float* part;      // [ksplit][M][RP] fp32 (unused if ksplit == 1)
  unsigned* cnt;    // [ceil(M/64)] zeroed counters
  int r;
  float alpha1;
  uint16_t* out1;   // [M][ld1], columns < r, or NULL
  int ld1;
  float alpha2;
  uint16_t* out2;   // [M][RP], or NULL
  int bkn;          // 0: B is [RP][K]; > 0: B is k-major [K][bkn] (its first r columns used;
                    // whole-K kernel only, bkn % 8 == 0)
};
// TN skinny product with its split reduction: out = alpha * P[M][:r]^T Q[M][N].
struct TnArgs {
  const uint16_t* P;  // [M][ldp], 16-byte aligned, ldp % 8 == 0, columns r .. ceil8(r)-1 zero
  int ldp, r;
  const uint16_t* Q;
  int64_t M;
  int N;
  int msplit;
  int64_t mrange;
  float* part;      // [msplit][RP][N] fp32 (unused if msplit == 1)
  unsigned* cnt;    // [ceil(N/64)] zeroed counters
  float alpha;
  int trans;        // 0: out [r][N]; 1: out [N][r]
  float* out;
};
void plan_nt(int64_t M, int K, int* ksplit, int* krange);
void plan_tn(int64_t M, int N, int* msplit, int64_t* mrange);
hipError_t launch_skinny_nt(const NtArgs& a, int RP, hipStream_t st);
hipError_t launch_skinny_tn(const TnArgs& a, int RP, hipStream_t st);
// two TN products over the same tokens in one launch when possible (b may be NULL)
hipError_t launch_skinny_tn2(const TnArgs& a, const TnArgs* b, int RP, hipStream_t st);
// true when the launchers above use the unsplit kernels (whole K / all tokens
// per workgroup), which need neither the partial buffers nor the counters
bool skinny_nt_whole(int64_t M, int RP);
bool skinny_tn_whole(int64_t M, int RP);
// the kernel one NT product takes (its contraction K; bkn: k-major B)
bool skinny_nt_use_whole(int64_t M, int K, int RP, bool bkn);
// column band of the all-token TN kernel for products of N0 and N1 columns
// (N1 = 0: one product): 64 (whole 128-byte lines of Q per load) when that
// still gives 192 workgroups or more, else 32
int skinny_tn_band(int N0, int N1);
// row panels per group of the fused GEMM's tile order for a contraction of K:
// 2 while 16 panels of 256 rows (the 8 XCDs' working set) stay within the
// Infinity Cache, i.e. K <= 16384, else 1
int gemm_group_m(int K);
// A launch holds at most 2^32 - 1 work-items.  Rows per launch of an NT
// product over M token rows: M itself up to kNtLaunchRows, else equal
// consecutive ranges, each a multiple of 64 rows and at least 2^22 rows (so
// that each range takes the kernel the full product would).
constexpr int64_t kNtLaunchRows = (int64_t)1 << 24;
int64_t nt_launch_rows(int64_t M);
// 256-row panels per launch of the fused GEMM with tiles_n column tiles
// (512 work-items per tile)
int64_t gemm_launch_panels(int64_t tiles_n);

// ---- the 8-bit operators and the norm ----
// Weak: a host-only build of the ABI layer (argument checks without kernels)
// links without these definitions; api.cpp then reports NF4_ERR_HIP for a call
// that would launch one.
#define NF4K_WEAK __attribute__((weak))

// block_rows: 1 (a scale per row and 128 columns) or 128 (per 128 x 128 block)
NF4K_WEAK hipError_t launch_fp8_quantize(const void* X, bool bf16, int64_t rows, int64_t cols, bool e5m2,
                                         int block_rows, uint8_t* codes, float* scales, hipStream_t st);
NF4K_WEAK hipError_t launch_fp8_dequantize(const uint8_t* codes, const float* scales, int64_t rows, int64_t cols,
                                           bool e5m2, int block_rows, bool bf16, void* out, hipStream_t st);

// threads of a workgroup of the norm for rows of width H, and the rows it holds
int rmsnorm_threads(int H);
int rmsnorm_teams(int H);
// workgroups of the norm's gradient, each with a partial dw [H]
int rmsnorm_parts(int64_t M, int H);
constexpr int kMaxNormWidth = 32768;  // 1024 threads, 4 chunks of 8 columns
NF4K_WEAK hipError_t launch_rmsnorm_fwd(const uint16_t* X, const uint16_t* R, const uint16_t* w, int64_t M, int H,
                                        float eps, uint16_t* Hout, uint16_t* Y, uint8_t* codes, float* scales,
                                        float* rstd, hipStream_t st);
NF4K_WEAK hipError_t launch_rmsnorm_bwd(const uint16_t* dY, const uint16_t* Hs, const uint16_t* w, const float* rstd,
                                        const uint16_t* dH, int64_t M, int H, uint16_t* dX, float* dw, float* part,
                                        hipStream_t st);

// Layer norm; `part` of its gradient is rmsnorm_parts(M, H) rows of H for dw, and as many for db.
NF4K_WEAK hipError_t launch_layernorm_fwd(const uint16_t* X, const uint16_t* R, const uint16_t* w, const uint16_t* b,
                                          int64_t M, int H, float eps, uint16_t* Hout, uint16_t* Y, uint8_t* codes,
                                          float* scales, float* mean, float* rstd, hipStream_t st);
NF4K_WEAK hipError_t launch_layernorm_bwd(const uint16_t* dY, const uint16_t* Hs, const uint16_t* w, const float* mean,
                                          const float* rstd, const uint16_t* dH, int64_t M, int H, uint16_t* dX,
                                          float* dw, float* db, float* part, hipStream_t st);

// ---- rows sorted by id, and the adapters of many requests ----
constexpr int kMaxIds = 4096;
constexpr int64_t kMaxRoutedRows = (int64_t)1 << 30;
// The rows of a wave's run, and the runs of one workgroup that takes them all (true), or the workgroups of 4.
bool plan_route(int64_t M, int n, int* runs, int64_t* run);
// ints of the counts that several workgroups share (0: one workgroup takes all rows)
int64_t route_counts(int64_t M, int n);
NF4K_WEAK hipError_t launch_route(const int32_t* ids, int64_t M, int n, int32_t* order, int32_t* offsets, int* counts,
                                  hipStream_t st);

// The adapters of many requests (adapters.hip).  Their rows: adapter a's are
// order[offsets[a] .. offsets[a + 1]), or these numbers themselves without an order.
struct AdapterRows {
  const int32_t* offsets;
  const int32_t* order;  // or NULL
  int n;
  int64_t M;
};
struct AdapterCall {
  AdapterRows rows;
  const uint16_t* L1;  // [n][h][r]
  const uint16_t* L2;  // [n][r][o]
  const float* s;      // [n]
  int64_t o, h;
  int r;
};
// T or G as three bf16 parts, for the products over rows
constexpr int kZeroBytes = 512;
struct Split3 {
  const float* from;  // [M][r]
  uint16_t* to;       // [M][nz][3][rp], or NULL
  void* zero;         // kZeroBytes to be cleared
  int nz, rp;
};
struct AdapterNarrow {
  AdapterRows rows;
  const uint16_t* A;  // [M][K]
  const uint16_t* L;
  int64_t K;
  int r;
  int64_t krange;
  float* part;  // [splits][M][r]
  unsigned tiles;  // workgroups past them split T
  Split3 split;
};
struct AdapterWide {
  AdapterRows rows;
  const float* part;  // [splits][M][r]
  int splits;
  const uint16_t* L;
  int64_t N;
  int r;
  const float* s;
  const uint16_t* base;  // or NULL
  uint16_t* out;
  float* T_out;  // the joined parts, or NULL
  int blocks;    // blocks of 128 columns a workgroup goes over
  Split3 split;  // the joined parts in this form too, where `to` is set
};
struct AdapterFew {
  AdapterRows rows;
  const uint16_t* X;
  const uint16_t* L1;
  int64_t K;
  const uint16_t* L2;
  int64_t N;
  int r;
  const float* s;
  const uint16_t* base;  // or NULL
  uint16_t* out;
  float* T_out;  // or NULL
};
struct AdapterGrad {
  const void* Q;          // [M][N], bf16 or codes
  const float* q_scales;  // of codes
  int64_t N;
  const float* P;      // [M][r], beside codes
  const uint16_t* P3;  // in three parts, beside bf16
  int r;
  const float* s;
  int item;       // rows an item, a multiple of 64
  int64_t items;  // at most
  int64_t parts;  // items of adapters that have several, at most
  int single;     // every adapter's rows are one item, and the products clear what has none
  int trans;      // out [n][N][r], else [n][r][N]
  float* part;    // [parts][r * N]
  float* out;
  const void* zero;  // kZeroBytes of zeros
};
constexpr int kMaxAdapterItem = 4096;
constexpr int64_t kMaxAdapterRows = (int64_t)1 << 26;  // tiles of 16 rows stay one launch
// Tiles of rows of the products of one row, and the splits of a contraction over K
// (`lines`: by L2's rows, for G; else by L1's columns, for T).
struct AdapterPlan {
  int bm;         // rows a tile: 16, 64 or 128
  int64_t tiles;  // at most
  int splits;
  int64_t krange;
};
AdapterPlan plan_adapters_rows(int64_t M, int n, int64_t K, bool lines);
// Workgroups of a tile of 16 rows where one launch makes T and Y (rank up to 16; 0: two launches).
int plan_adapters_few(int64_t M, int n, int64_t h, int64_t o, int r);
// Tiles of rows of the products over the rank.
struct AdapterWidePlan {
  int bm;         // rows a tile: 16 (4 blocks of 128 columns a workgroup, one a wave) or 64
  int64_t tiles;  // at most
  int blocks;     // blocks of 128 columns that a workgroup of 64 rows goes over
};
AdapterWidePlan plan_adapters_wide(int64_t M, int n, int64_t N, int r);
// Whether their workgroups add up the splits by themselves, or a launch before them does.
bool plan_adapters_fold(int64_t M, int r, int splits, const AdapterWidePlan& w, int64_t N);
// Rows of an item of the adapters' gradients, the items there are at most, and those of adapters
// that have several, whose sums need a place of their own.
struct AdapterItems {
  int item;
  int64_t items;
  int single;  // no adapter has two, and no join is launched
  int64_t parts;
};
AdapterItems plan_adapters_items(int64_t M, int n, int64_t h, int64_t o, int r);
// Byte offsets of the parts of the backward pass's workspace; the zeros come first.  `total` has
// room for every item's sums.
struct AdapterGradSpace {
  size_t gparts, g, g3, t3, parts, total;
};
AdapterGradSpace plan_adapters_space(int64_t M, int n, int64_t h, int64_t o, int r);
// Its bytes: without the room of items that are all of their adapter's and go straight to the results.
size_t plan_adapters_bwd_bytes(int64_t M, int n, int64_t h, int64_t o, int r);
NF4K_WEAK hipError_t launch_adapters_fwd(const AdapterCall& c, const uint16_t* X, const uint16_t* base, uint16_t* Y,
                                         float* T_out, void* ws, hipStream_t st);
// x8: 0 X is bf16, 1 e4m3, 2 e5m2
NF4K_WEAK hipError_t launch_adapters_bwd(const AdapterCall& c, const void* X, int x8, const float* x_scales,
                                         const uint16_t* dY, const float* T, const uint16_t* base, uint16_t* dX,
                                         float* dL1, float* dL2, void* ws, hipStream_t st);

// C [M][N] = A W^T (or A W) in 8 bits, scaled by block, plus A2 B2^T; with
// `offsets` grouped by expert (rows offsets[e] .. offsets[e + 1] by W[e], B2[e])
struct Fp8Gemm {
  const uint8_t* A;
  bool a_e5m2;
  const float* a_scales;
  int64_t M;
  const uint8_t* W;
  const float* w_scales;
  int64_t rows, cols;
  bool transpose;
  int experts;  // 0: one weight, no offsets
  const int32_t* offsets;
  const uint16_t* A2;
  const uint16_t* B2;
  int R;
  uint16_t* C;
  float* part;  // fp8_split_bytes of it, or NULL: no contraction is split
};
// The product's tile kinds (rows bm by columns bn a workgroup of `threads`), and
// what one costs; plan_fp8 picks the kind, or two for two ranges of rows, that
// the costs say takes the least time.  Returns the number of parts (their rows
// add up to M).  experts > 0: one kind for all.
enum {
  kFp8Wide8, kFp8Wide4, kFp8Wide2, kFp8Ring22, kFp8Ring21, kFp8Rows11, kFp8Rows12, kFp8Rows22, kFp8Rows42, kFp8Rows44,
  kFp8Rows14T, kFp8Rows24T, kFp8Rows44T, kFp8Kinds
};
struct Fp8Kind {
  int bm, bn, threads;
  double start, u0, u1;
};
struct Fp8Part {
  int kind;
  int64_t rows;
  int splits;  // workgroups that share a tile's contraction: 1, 2, 3, 4, 6 or 8
};
const Fp8Kind* fp8_kinds();
// A grouped product is one launch: its workgroups (every expert's last tile may be
// partly filled), and whether their work-items stay below 2^32.  plan_fp8 needs
// the largest kind, kFp8Wide8, to fit.
int64_t fp8_grouped_tiles(int kind, int64_t M, int N, int experts);
bool fp8_grouped_fits(int kind, int64_t M, int N, int experts);
int plan_fp8(int64_t M, int N, int K, bool transpose, int experts, bool may_split, Fp8Part parts[2]);
// bytes of the fp32 parts that plan_fp8 with may_split wants (0: it splits nothing)
int64_t fp8_split_bytes(int64_t M, int N, int K, bool transpose, int experts);
NF4K_WEAK hipError_t launch_fp8_gemm(const Fp8Gemm& g, hipStream_t st);

}  // namespace nf4k
