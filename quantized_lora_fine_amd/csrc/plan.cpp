// Launch planning of libnf4lora: how the skinny adapter products split their
// contraction, and how the batched error pass groups linears into launches.
// Host code only (no kernels), so the C ABI layer and its CPU-only tests
// link it without a GPU.
#include "launch.hpp"

namespace nf4k {

// split-K factor for an NT skinny product over M rows (64 rows per
// workgroup): about 512 workgroups, each K range a multiple of 128.
void plan_nt(int64_t M, int K, int* ksplit, int* krange) {
  const int64_t mblocks = (M + 63) / 64;
  int64_t ks = (512 + mblocks - 1) / (mblocks > 0 ? mblocks : 1);
  const int64_t kmax = (K + 127) / 128;
  if (ks > kmax) ks = kmax;
  if (ks < 1) ks = 1;
  int kr = (int)(((K + ks - 1) / ks + 127) / 128 * 128);
  ks = (K + kr - 1) / kr;
  *ksplit = (int)ks;
  *krange = kr;
}

// split-M factor for a TN skinny product with N output columns (64 per
// workgroup): about 512 workgroups, token ranges a multiple of 256 (a whole
// number of chunks for every rank).
void plan_tn(int64_t M, int N, int* msplit, int64_t* mrange) {
  const int64_t nblocks = (N + 63) / 64;
  int64_t ms = (512 + nblocks - 1) / nblocks;
  const int64_t mmax = (M + 255) / 256;
  if (ms > mmax) ms = mmax;
  if (ms < 1) ms = 1;
  int64_t mr = ((M + ms - 1) / ms + 255) / 256 * 256;
  if (mr < 256) mr = 256;
  ms = (M + mr - 1) / mr;
  if (ms < 1) ms = 1;
  *msplit = (int)ms;
  *mrange = mr;
}


// whole-K workgroups when the rank is small and there are rows enough for them
bool skinny_nt_whole(int64_t M, int RP) {
  if (RP > 64) return false;
  const int rw = RP <= 16 ? 8 : (RP <= 32 ? 16 : 32);
  return (M + rw - 1) / rw >= 64;
}

// The whole-K kernel for one NT product, given its contraction K and B layout.
// A k-major B takes it always.  A rank-64 product with a long contraction over
// many rows (G at 8192+ tokens against 8192+ outputs) takes the split kernel
// instead: a whole-K workgroup of 32 rows reads the entire 64 x K operand from
// L2, a split workgroup of 64 rows half of that per row.
bool skinny_nt_use_whole(int64_t M, int K, int RP, bool bkn) {
  if (!skinny_nt_whole(M, RP)) return false;
  if (bkn) return true;
  return !(RP == 64 && M >= 8192 && K >= 8192);
}

// all tokens per workgroup when the rank is small and the token count is not tiny
bool skinny_tn_whole(int64_t M, int RP) { return RP <= 64 && M >= 512; }

int skinny_tn_band(int N0, int N1) {
  const int64_t wide = ((int64_t)N0 + 63) / 64 + ((int64_t)N1 + 63) / 64;
  return wide >= 192 ? 64 : 32;
}

int gemm_group_m(int K) { return K <= 16384 ? 2 : 1; }

int64_t nt_launch_rows(int64_t M) {
  if (M <= kNtLaunchRows) return M;
  const int64_t n = (M + kNtLaunchRows - 1) / kNtLaunchRows;
  return ((M + n - 1) / n + 63) / 64 * 64;
}

int64_t gemm_launch_panels(int64_t tiles_n) {
  const int64_t per = ((int64_t)0xFFFFFFFF / 512) / (tiles_n > 0 ? tiles_n : 1);
  return per > 0 ? per : 1;
}

int rmsnorm_teams(int H) { return H <= 128 ? 16 : H <= 2048 ? 4 : 1; }

int rmsnorm_threads(int H) {
  if (H <= 2048) return 256;
  const int chunks = H <= 8192 ? 1 : H <= 16384 ? 2 : 4;
  return (H + 512 * chunks - 1) / (512 * chunks) * 64;  // 8 columns a thread and chunk
}

int rmsnorm_parts(int64_t M, int H) {
  const int teams = rmsnorm_teams(H);
  const int64_t groups = (M + teams - 1) / teams;
  // one workgroup a compute unit where it holds a whole row (16384 x 8192 with dH:
  // 193 us against 198 and 203 for 512 and 1024, whose parts of dw are more, without dH
  // 151 against 154 and 156; 1999 x 5120 with dH: 18.6 against 21.3 and 25.4; by replayed
  // graphs), two where its waves hold several
  const int64_t most = teams > 1 ? 512 : 256;
  return (int)(groups < most ? groups : most);
}

// Tiles of the block-scaled product, with what one takes on an MI355X: `start`
// microseconds around its loop, and u0 to u1 microseconds for every 128 of the
// contraction, u0 when few compute units have a tile and u1 when all do.  Fitted
// to the times of every kind for 1 to 8192 rows by 12 weights of 560 x 1200 to
// 28672 x 8192, each way; the kind that these costs choose is 1 % slower than the
// fastest one in the mean, 23 % at worst (160 rows by 9104 x 5888).  Unsplit, nothing
// stands for the weight's own stream: with the weight in the caches the times hold (64
// rows by 28672 x 8192: 43 us predicted, 43 measured), from memory it takes longer (66).
const Fp8Kind* fp8_kinds() {
  static const Fp8Kind kinds[kFp8Kinds] = {
      {256, 256, 512, 4.6, 1.11, 1.66},   // kFp8Wide8
      {128, 256, 512, 2.3, 0.81, 1.04},   // kFp8Wide4
      {64, 256, 512, 1.1, 0.69, 0.78},    // kFp8Wide2
      {128, 128, 512, 1.3, 0.54, 0.71},   // kFp8Ring22
      {128, 64, 512, 1.2, 0.33, 0.47},    // kFp8Ring21
      {16, 16, 256, 0.4, 0.040, 0.053},   // kFp8Rows11
      {16, 32, 256, 0.3, 0.070, 0.080},   // kFp8Rows12
      {32, 32, 512, 0.3, 0.083, 0.144},   // kFp8Rows22
      {64, 32, 256, 1.2, 0.133, 0.197},   // kFp8Rows42
      {64, 64, 256, 1.8, 0.234, 0.291},   // kFp8Rows44
      {16, 64, 256, 0.8, 0.220, 0.259},   // kFp8Rows14T
      {32, 64, 256, 1.3, 0.259, 0.320},   // kFp8Rows24T
      {64, 64, 256, 2.0, 0.349, 0.420},   // kFp8Rows44T
  };
  return kinds;
}

int64_t fp8_grouped_tiles(int kind, int64_t M, int N, int experts) {
  const Fp8Kind& k = fp8_kinds()[kind];
  return (M / k.bm + (M < experts ? M : experts)) * ((N + k.bn - 1) / k.bn);
}

bool fp8_grouped_fits(int kind, int64_t M, int N, int experts) {
  return fp8_grouped_tiles(kind, M, N, experts) <= (int64_t)0xFFFFFFFF / fp8_kinds()[kind].threads;
}

namespace {

constexpr int kCUs = 256;
constexpr double kFp8Launch = 3.0;  // microseconds

constexpr double kFp8Join = 2.5, kFp8JoinRate = 4e6;  // the join's launch, and bytes a microsecond of it
constexpr int64_t kFp8SplitBytes = (int64_t)1 << 26;

// the launch and every set of tiles that the compute units hold at once
double fp8_time(int kind, int64_t tiles_m, int N, int K, int splits) {
  const Fp8Kind& k = fp8_kinds()[kind];
  const int64_t tiles = tiles_m * ((N + k.bn - 1) / k.bn) * splits;
  const double fill = tiles >= kCUs ? 1.0 : (double)tiles / kCUs;
  const int64_t steps = ((K + 127) / 128 + splits - 1) / splits;
  return kFp8Launch + (double)((tiles + kCUs - 1) / kCUs) * (k.start + steps * (k.u0 + (k.u1 - k.u0) * fill));
}

// The kind, and over how many workgroups a tile's contraction is split: where
// there are fewer tiles than compute units, as long as each part has 4 blocks, the
// parts fit 64 MB, and a tenth is gained by the costs: no split beats the weights'
// own stream, and the join is a launch more (3 rows by 11008 x 4096 transposed, by
// replayed graphs: 25 -> 14.4 us with the weight in the caches, 39 -> 20.2 from memory;
// 900 rows by 6144 x 1328 transposed 47 -> 28 and 61 -> 30).
int fp8_best(int64_t M, int N, int K, bool transpose, int experts, bool may_split, double* time, int* splits) {
  int best = -1;
  double least = 0;
  *splits = 1;
  const double stream = (double)(experts ? std::min<int64_t>(M, experts) : 1) * N * K / 5.5e6;  // the weights, once
  for (int i = 0; i < kFp8Kinds; ++i) {
    const bool wide = i <= kFp8Wide2, t = i >= kFp8Rows14T;
    if (!wide && t != transpose) continue;
    // Bound by the weight's stream, not by the tiles' own time: the kinds that put
    // two workgroups on a compute unit, whose starts hide behind each other.  Up
    // to 8 rows of one weight the narrowest (28672 x 8192, 1 row: 42 us against 45
    // and 51 for 32 columns by 16 and by 32 rows), few rows of many experts the next
    // one (64 experts of 1536 x 4096, 48 rows: 34 us against 39 and 43).
    if (!transpose && !experts && M <= 8 && i != kFp8Rows11) continue;
    if (!transpose && experts && M <= 4 * (int64_t)experts && i != kFp8Rows12 &&
        fp8_grouped_fits(kFp8Rows12, M, N, experts))
      continue;
    const int64_t bm = fp8_kinds()[i].bm;
    int64_t tiles_m = (M + bm - 1) / bm;
    if (experts) {
      // the rows' tiles, half a tile more for every expert that can have rows, and a
      // tenth: the counts are not known, and one tile past a set costs a set (32
      // experts of 2048 x 4096, 4096 rows: 90 us against 115 without it)
      const int64_t used = M < experts ? M : experts;
      tiles_m = (M / bm + used / 2) * 11 / 10;
      if (tiles_m < used) tiles_m = used;
      if (!fp8_grouped_fits(i, M, N, experts)) continue;
    }
    const int64_t tiles = tiles_m * ((N + fp8_kinds()[i].bn - 1) / fp8_kinds()[i].bn);
    for (int s : {1, 2, 3, 4, 6, 8}) {
      if (s > 1 && (!may_split || s > K / 512 || s * tiles > 2 * kCUs || s * M * N * 4 > kFp8SplitBytes)) break;
      double x = fp8_time(i, tiles_m, N, K, s);
      if (s > 1)
        x = 1.1 * (std::max(x, kFp8Launch + stream) + kFp8Join + (double)(M * N * (8 * s + 2)) / kFp8JoinRate);
      if (best < 0 || x < least) {
        least = x;
        best = i;
        *splits = s;
      }
    }
  }
  *time = least;
  return best;
}

}  // namespace

int plan_fp8(int64_t M, int N, int K, bool transpose, int experts, bool may_split, Fp8Part parts[2]) {
  double least;
  parts[0].kind = fp8_best(M, N, K, transpose, experts, may_split, &least, &parts[0].splits);
  parts[0].rows = M;
  int n = 1;
  if (experts) return n;
  // or whole sets of wide tiles, and the rows that are left by themselves: a few
  // rows past a set would hold every compute unit for another whole one
  for (int i = kFp8Wide8; i <= kFp8Wide2; ++i) {
    const Fp8Kind& k = fp8_kinds()[i];
    const int64_t tiles_n = (N + k.bn - 1) / k.bn;
    const int64_t sets = (M / k.bm) * tiles_n / kCUs;
    const int64_t rows = sets * kCUs / tiles_n * k.bm;
    if (rows <= 0 || rows >= M) continue;
    double rest;
    int splits;
    const int kind = fp8_best(M - rows, N, K, transpose, 0, may_split, &rest, &splits);
    const double x = fp8_time(i, rows / k.bm, N, K, 1) + rest;
    if (x < 0.95 * least) {  // a second launch has to be worth it
      least = x;
      n = 2;
      parts[0].kind = i;
      parts[0].rows = rows;
      parts[0].splits = 1;
      parts[1].kind = kind;
      parts[1].rows = M - rows;
      parts[1].splits = splits;
    }
  }
  return n;
}

int64_t fp8_split_bytes(int64_t M, int N, int K, bool transpose, int experts) {
  Fp8Part parts[2];
  const int n = plan_fp8(M, N, K, transpose, experts, true, parts);
  int64_t most = 0;
  for (int i = 0; i < n; ++i)
    if (parts[i].splits > 1 && parts[i].splits * parts[i].rows * N * 4 > most)
      most = parts[i].splits * parts[i].rows * N * 4;
  return most;
}

int error_batch_chunk(const int64_t* rows, const int64_t* cols, int32_t n, int32_t c0, int64_t* g0) {
  int k = 0;
  g0[0] = 0;
  while (k < kErrBatch && c0 + k < n) {
    const int64_t end = g0[k] + error_groups(rows[c0 + k], cols[c0 + k]);
    if (end > kMaxLaunchGroups) break;
    g0[k + 1] = end;
    ++k;
  }
  return k;
}

}  // namespace nf4k
