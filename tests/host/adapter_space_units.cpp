// Unit checks of the backward pass's workspace for the adapters: room for the sums of every item of an adapter that has
// several, and for no others (host only).
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

static uint64_t state = 7;
static int64_t pick(int64_t lo, int64_t hi) {
  state = state * 6364136223846793005ull + 1442695040888963407ull;
  return lo + (int64_t)((state >> 20) % (uint64_t)(hi - lo + 1));
}
static int64_t any(int bits) { return std::max<int64_t>(1, pick(1, (int64_t)1 << pick(0, bits))); }

// items of the adapters that have more than one
static int64_t parts_of(const std::vector<int64_t>& counts, int64_t item) {
  int64_t t = 0;
  for (int64_t c : counts) t += c > item ? (c + item - 1) / item : 0;
  return t;
}

int main() {
  int64_t most = 0, fewer = 0;
  for (int i = 0; i < 100000; ++i) {
    const int64_t M = any(i % 8 ? 26 : 15), h = 16 * any(18), o = 16 * any(18);
    const int n = (int)any(12), r = 8 * (int)pick(1, 32);
    const AdapterItems it = plan_adapters_items(M, n, h, o, r);
    const AdapterGradSpace s = plan_adapters_space(M, n, h, o, r);
    const size_t bytes = plan_adapters_bwd_bytes(M, n, h, o, r), each = (size_t)r * (h + o) * 4;
    CHECK(it.parts >= 0 && it.parts <= it.items && it.parts * it.item <= 2 * M);
    CHECK(bytes == s.parts + (size_t)it.parts * each);
    if (it.item >= M) CHECK(it.parts == 0);
    if (!it.single && it.parts < it.items) ++fewer;
    if (i % 8) continue;
    // as many adapters as can be of just over an item, of just over two, and of any rows
    for (int64_t rows : {(int64_t)it.item + 1, (int64_t)2 * it.item + 1, (int64_t)0}) {
      std::vector<int64_t> counts;
      int64_t left = M;
      for (int a = 0; a < n && left; ++a) {
        counts.push_back(rows ? std::min(left, rows) : pick(0, left));
        left -= counts.back();
      }
      CHECK(parts_of(counts, it.item) <= it.parts);
      most = std::max(most, parts_of(counts, it.item));
    }
  }
  CHECK(most > 8 && fewer > 0);
  if (failures) {
    std::printf("%d failures\n", failures);
    return 1;
  }
  std::printf("adapter space units: ok\n");
  return 0;
}
