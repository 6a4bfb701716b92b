// The tiles of the adapters' products at sizes measured with both kinds: each gets the kind that was faster (host only).
#include <cstdio>

#include "launch.hpp"

using namespace nf4k;

static int failures = 0;
static void check(bool ok, const char* what, int64_t M, int n, int64_t N, int r, int bm) {
  if (ok) return;
  std::printf("%s of %lld rows, %d adapters, %lld columns, rank %d: tiles of %d\n", what, (long long)M, n, (long long)N, r,
              bm);
  ++failures;
}

int main() {
  struct Case {
    int64_t M;
    int n;
    int64_t K;
    int r;
    bool few;  // tiles of 16 are faster
  };
  const Case t[] = {{256, 1, 4096, 16, true},    {1024, 1, 4096, 16, true},   {1024, 1, 11008, 16, true},
                    {1024, 1, 11008, 64, true},  {700, 1, 28672, 64, true},   {1024, 2, 11008, 64, true},
                    {4096, 1, 4096, 64, true},   {1536, 1, 11008, 128, true}, {2048, 8, 4096, 64, true},
                    {1024, 1, 28672, 64, false}, {4096, 1, 11008, 64, false}, {1024, 16, 11008, 64, false},
                    {1024, 8, 28672, 64, false}, {2048, 1, 28672, 16, false}, {1536, 16, 11008, 32, false}};
  for (const Case& c : t) {
    const int bm = plan_adapters_rows(c.M, c.n, c.K, false).bm;
    check((bm == 16) == c.few, "T", c.M, c.n, c.K, c.r, bm);
  }
  const Case g[] = {{256, 1, 4096, 16, true}, {256, 32, 28672, 16, true}, {1024, 1, 4096, 64, false}, {512, 32, 28672, 32, false}};
  for (const Case& c : g) {
    const int bm = plan_adapters_rows(c.M, c.n, c.K, true).bm;
    // (1024 rows of rank 64 are level, and take the larger ones)
    check((bm == 16) == c.few, "G", c.M, c.n, c.K, c.r, bm);
  }
  const Case y[] = {{64, 16, 11008, 16, true},   {640, 1, 28672, 16, true},   {1024, 1, 4096, 64, true},
                    {512, 1, 28672, 64, true},   {496, 2, 28672, 64, true},   {3800, 1, 4096, 64, true},
                    {512, 1, 28672, 128, true},  {32, 32, 28672, 64, true},   {220, 220, 4096, 128, true},
                    {1024, 1, 28672, 16, false}, {2048, 1, 28672, 16, false}, {4096, 1, 4096, 64, false},
                    {1024, 1, 28672, 64, false}, {448, 8, 28672, 64, false},  {1536, 1, 11008, 128, false}};
  for (const Case& c : y) {
    const int bm = plan_adapters_wide(c.M, c.n, c.K, c.r).bm;
    check((bm == 16) == c.few, "Y", c.M, c.n, c.K, c.r, bm);
  }
  if (failures) {
    std::printf("%d failures\n", failures);
    return 1;
  }
  std::printf("adapter rule units: ok\n");
  return 0;
}
