// Unit checks of the launch planning of the rows' sorting and of the adapters (host only).
#include <algorithm>
#include <cstdio>
#include <vector>

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
// a size of any magnitude up to 2^bits
static int64_t any(int bits) { return std::max<int64_t>(1, pick(1, (int64_t)1 << pick(0, bits))); }

static void route_plan(int64_t M, int n, bool* ones) {
  int runs = 0;
  int64_t run = 0;
  const bool one = plan_route(M, n, &runs, &run);
  ones[one] = true;
  CHECK(run >= 64 && run % 64 == 0 && runs >= 1);
  if (one) {
    CHECK(runs <= 16 && runs * run >= M);                       // waves of one workgroup
    CHECK((int64_t)runs * (n + 1) * 4 <= 65536);                // its counts in LDS
    CHECK(route_counts(M, n) == 0);
  } else {
    CHECK(4 * run * runs >= M && 4 * run * (runs - 1) < M);     // no workgroup without rows
    CHECK(runs <= 256);
    CHECK(route_counts(M, n) == (int64_t)runs * (n + 1));
    CHECK(4 * (n + 1) * 4 + 16 <= 160 * 1024);                  // LDS of a workgroup
  }
}

// tiles of bm rows for the adapters' counts
static int64_t tiles_of(const std::vector<int64_t>& counts, int64_t bm) {
  int64_t t = 0;
  for (int64_t c : counts) t += (c + bm - 1) / bm;
  return t;
}

int main() {
  bool ones[2] = {};
  for (int64_t M : {0, 1, 63, 64, 65, 8191, 8192, 8193, 1 << 20, 1 << 30})
    for (int n : {1, 63, 64, 1023, 1024, 4096}) route_plan(M, n, ones);
  for (int i = 0; i < 100000; ++i) route_plan(pick(0, 9) ? any(30) : 0, (int)any(12), ones);
  CHECK(ones[0] && ones[1]);

  bool bm16 = false, bm64 = false, bm128 = false, few = false, fold = false, sum = false, single = false, wide16 = false, wide64 = false, several = false;
  for (int i = 0; i < 200000; ++i) {
    const int64_t M = any(26), h = 16 * any(18), o = 16 * any(18);
    const int n = (int)any(12), r = 8 * (int)pick(1, 32);
    for (bool lines : {false, true}) {
      const int64_t K = lines ? o : h;
      const AdapterPlan p = plan_adapters_rows(M, n, K, lines);
      CHECK(p.bm == 16 || p.bm == 64 || p.bm == 128);
      bm16 |= p.bm == 16, bm64 |= p.bm == 64, bm128 |= p.bm == 128;
      // the splits cover the contraction, and none is empty
      CHECK(p.krange % 256 == 0 && p.splits >= 1 && p.splits * p.krange >= K && (p.splits - 1) * p.krange < K);
      CHECK(p.splits <= 65535 && p.tiles >= 1);
      // work-items of a launch, with those that split T
      CHECK((p.tiles + (M + 63) / 64) * 256 < (int64_t)1 << 32);
    }
    const AdapterPlan p = plan_adapters_rows(M, n, h, false);
    const AdapterWidePlan w = plan_adapters_wide(M, n, o, r);
    CHECK((w.bm == 16 || w.bm == 64) && w.blocks >= 1 && w.tiles * 256 < (int64_t)1 << 32);
    CHECK(((o + 127) / 128 + w.blocks - 1) / w.blocks <= 65535);
    wide16 |= w.bm == 16, wide64 |= w.bm == 64;
    if (const int groups = plan_adapters_few(M, n, h, o, r)) {
      few = true;
      CHECK(p.bm == 16 && r <= 16 && groups <= 65535 && p.tiles <= 16);  // one launch of the tiles planned here
    }
    const AdapterItems it = plan_adapters_items(M, n, h, o, r);
    CHECK(it.item % 64 == 0 && it.item >= 64 && it.item <= kMaxAdapterItem && it.items >= 1);
    CHECK(it.items + (it.single ? n : 0) <= 65535);
    if (it.single) CHECK(it.item >= M);
    single |= it.single != 0;
    several |= !it.single && it.item < M;
    const AdapterGradSpace s = plan_adapters_space(M, n, h, o, r);
    const int64_t splits = plan_adapters_rows(M, n, o, true).splits;
    CHECK(s.gparts >= kZeroBytes && s.g - s.gparts >= (size_t)(splits * M * r * 4) && s.g3 - s.g >= (size_t)M * r * 4);
    CHECK(s.gparts % 16 == 0 && s.g % 16 == 0 && s.g3 % 16 == 0 && s.t3 % 16 == 0 && s.parts % 16 == 0);
    CHECK(s.t3 - s.g3 >= (size_t)M * r * 6 && s.parts - s.t3 >= (size_t)M * r * 6);
    CHECK(s.total - s.parts >= (it.single ? 0 : (size_t)it.items * r * (h + o) * 4));
    (plan_adapters_fold(M, r, (int)splits, plan_adapters_wide(M, n, h, r), h) ? fold : sum) = true;
    CHECK(plan_adapters_fold(M, r, 1, w, o));
    // whatever the rows' counts are, the launches hold their tiles and items
    if (M <= 1 << 16 && i % 8 == 0) {
      std::vector<int64_t> counts((size_t)n, 0);
      int64_t left = M;
      const bool thin = pick(0, 1);
      for (int a = 0; a < n && left; ++a) {
        const int64_t most = a + 1 == n ? left : thin ? std::min<int64_t>(left, 2 * M / n + 1) : left;
        counts[(size_t)a] = a + 1 == n ? left : pick(0, most);
        left -= counts[(size_t)a];
      }
      for (bool lines : {false, true}) {
        const AdapterPlan q = plan_adapters_rows(M, n, lines ? o : h, lines);
        CHECK(tiles_of(counts, q.bm) <= q.tiles);
      }
      CHECK(tiles_of(counts, w.bm) <= w.tiles);
      CHECK(tiles_of(counts, it.item) <= it.items);
    }
  }
  CHECK(bm16 && bm64 && bm128 && few && wide16 && wide64 && fold && sum && single && several);
  if (failures) {
    std::printf("%d failures\n", failures);
    return 1;
  }
  std::printf("adapter plan units: ok\n");
  return 0;
}
