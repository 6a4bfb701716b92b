// Unit checks of the 8-bit product's and the norm's launch planning (host only).
#include <cstdio>
#include <cstdlib>

#include "launch.hpp"

using namespace nf4k;

static int failures = 0;
#define CHECK(c)                                                  \
  do {                                                            \
    if (!(c)) {                                                   \
      std::printf("line %d: %s\n", __LINE__, #c);                 \
      ++failures;                                                 \
    }                                                             \
  } while (0)

static uint64_t state = 1;
static int64_t pick(int64_t lo, int64_t hi) {
  state = state * 6364136223846793005ull + 1442695040888963407ull;
  return lo + (int64_t)((state >> 20) % (uint64_t)(hi - lo + 1));
}

static bool transposed(int kind) { return kind >= kFp8Rows14T; }
static bool wide(int kind) { return kind <= kFp8Wide2; }

int main() {
  bool reached[kFp8Kinds] = {};
  bool split = false, joined = false;
  // what the parts have to be for any product
  for (int n = 0; n < 200000; ++n) {
    const int64_t M = pick(0, 1) ? pick(1, 600) : pick(1, (int64_t)1 << pick(1, 31));
    const int N = 16 * (int)pick(1, pick(0, 3) ? 1024 : 262144), K = 16 * (int)pick(1, pick(0, 3) ? 1024 : 262144);
    const bool t = pick(0, 1);
    const int experts = pick(0, 2) ? 0 : (int)pick(1, 4096);
    if (experts && !fp8_grouped_fits(kFp8Wide8, M, N, experts)) continue;  // refused before
    const bool may_split = pick(0, 1);
    Fp8Part parts[2];
    const int c = plan_fp8(M, N, K, t, experts, may_split, parts);
    CHECK(c == 1 || (c == 2 && !experts));
    int64_t rows = 0;
    for (int i = 0; i < c; ++i) {
      CHECK(parts[i].rows > 0 && parts[i].kind >= 0 && parts[i].kind < kFp8Kinds);
      CHECK(wide(parts[i].kind) || transposed(parts[i].kind) == t);
      CHECK(!experts || fp8_grouped_fits(parts[i].kind, M, N, experts));
      const int k = parts[i].splits;
      CHECK(k == 1 || k == 2 || k == 3 || k == 4 || k == 6 || k == 8);  // the join's kinds
      CHECK((may_split || parts[i].splits == 1));
      if (parts[i].splits > 1) {
        joined = true;
        // no part of the contraction is empty, and the workspace holds the sums
        CHECK(parts[i].splits <= (K + 127) / 128);
        CHECK(parts[i].splits * parts[i].rows * N * 4 <= fp8_split_bytes(M, N, K, t, experts));
        CHECK(fp8_split_bytes(M, N, K, t, experts) <= (int64_t)1 << 26);
      } else if (c == 1 && may_split) {
        CHECK(fp8_split_bytes(M, N, K, t, experts) == 0);
      }
      rows += parts[i].rows;
      reached[parts[i].kind] = true;
    }
    CHECK(rows == M);
    if (c == 2) {
      split = true;
      CHECK(wide(parts[0].kind) && parts[0].rows % fp8_kinds()[parts[0].kind].bm == 0);
    }
  }
  for (int i = 0; i < kFp8Kinds; ++i) {
    if (!reached[i]) std::printf("kind %d is never chosen\n", i);
    CHECK(reached[i]);
    CHECK(fp8_kinds()[i].threads % 64 == 0 && fp8_kinds()[i].bm % 16 == 0 && fp8_kinds()[i].bn % 16 == 0);
  }
  CHECK(split && joined);
  Fp8Part p[2];
  // one token takes the narrowest tiles; a few rows over many experts the next ones
  CHECK(plan_fp8(1, 28672, 8192, false, 0, false, p) == 1 && p[0].kind == kFp8Rows11);
  CHECK(plan_fp8(48, 1536, 4096, false, 64, false, p) == 1 && p[0].kind == kFp8Rows12);
  // 16384 x 28672: 7168 large tiles are 28 whole sets of 256
  CHECK(plan_fp8(16384, 28672, 8192, false, 0, false, p) == 1 && p[0].kind == kFp8Wide8);
  // a grouped product of narrow rows and many of them takes the kinds that one launch holds
  CHECK(!fp8_grouped_fits(kFp8Rows11, (int64_t)1 << 30, 16, 1) && fp8_grouped_fits(kFp8Wide8, (int64_t)1 << 30, 16, 4096));
  for (bool t : {false, true})
    CHECK(plan_fp8((int64_t)1 << 30, 16, 16, t, 4096, false, p) == 1 && fp8_grouped_fits(p[0].kind, (int64_t)1 << 30, 16, 4096));
  CHECK(plan_fp8(16384, 1 << 22, 16, false, 4096, false, p) == 1 || !fp8_grouped_fits(kFp8Wide8, 16384, 1 << 22, 4096));
  // three rows past a whole set of 256-row tiles go by themselves
  CHECK(plan_fp8(4099, 4096, 11008, true, 0, false, p) == 2 && p[0].rows == 4096 && p[0].kind == kFp8Wide8 &&
        transposed(p[1].kind));

  // the norm: every width has threads for its columns in at most 4 chunks of 8
  for (int H = 16; H <= kMaxNormWidth; H += 16) {
    const int nt = rmsnorm_threads(H), teams = rmsnorm_teams(H);
    CHECK(nt % 64 == 0 && nt <= 1024 && nt % teams == 0);
    CHECK((int64_t)nt / teams * 8 * 4 >= H);
    CHECK(rmsnorm_parts(0, H) == 0 && rmsnorm_parts(1, H) == 1);
    const int most = rmsnorm_parts((int64_t)1 << 31, H);
    CHECK(most == 256 || most == 512);
    for (int64_t M : {5, 100, 1000, 100000}) CHECK(rmsnorm_parts(M, H) <= (M + teams - 1) / teams);
  }
  if (failures) {
    std::printf("%d failures\n", failures);
    return 1;
  }
  std::printf("fp8 plan units: ok\n");
  return 0;
}
