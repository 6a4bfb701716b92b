// Rows sorted by id (gfx950): a stable counting sort, so that the rows of each id, an
// adapter's or an expert's, stand together in their own order.
//
// A wave takes a run of consecutive rows.  It counts its ids in LDS, the counts are
// turned into first places (ids ascending, runs ascending within an id), and it goes
// through its rows again, 64 at a time: lanes of the same id find each other by one
// ballot for each bit of the id, take the id's next place plus their number among them,
// and the lowest of them moves that place on.  No order depends on timing: the counts
// are integers, and every place has one writer.
// Rows whose id is outside [0, n) count as id n and come last.
//
// Bound by latencies that follow one another, not by bytes (131072 rows: 1 MB).  Up to some
// 8192 rows one workgroup does everything: 64 rows of 48 ids 3.5 us, a launch with its two
// trips to memory.  131072 rows of 256 ids take 3.4 and 10.6 us in two launches; with a third
// between them for the counts' sums it was 17.6 a call, and is 13.2.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"

namespace nf4k {

namespace {

constexpr int kAhead = 8;  // rows of a lane whose ids are loaded at once

// the lane's next kAhead keys from row m on, 64 rows apart; -1 past m1
__device__ __forceinline__ void load_keys(const int32_t* ids, int64_t m, int64_t m1, int n, int (&key)[kAhead]) {
#pragma unroll
  for (int u = 0; u < kAhead; ++u) key[u] = m + 64 * u < m1 ? ids[m + 64 * u] : 0;
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    key[u] = (unsigned)key[u] < (unsigned)n ? key[u] : n;
    if (m + 64 * u >= m1) key[u] = -1;
  }
}

// counts[key] += 1 for the wave's rows [m0, m1), of which the first are in `keys`
__device__ __forceinline__ void count_run(const int32_t* ids, int64_t m0, int64_t m1, int n, int* counts,
                                          const int (&keys)[kAhead]) {
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (keys[u] >= 0) atomicAdd(counts + keys[u], 1);
  for (int64_t m = m0 + (threadIdx.x & 63) + 64 * kAhead; m < m1; m += 64 * kAhead) {
    int key[kAhead];
    load_keys(ids, m, m1, n, key);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (key[u] >= 0) atomicAdd(counts + key[u], 1);
  }
}

// order[next[key]++] = m for the wave's rows [m0, m1), in their order.  `next` is the
// wave's own; the LDS operations of one wave stay in order, and the fences keep the
// compiler from moving them.  `keys` are the first ones, loaded already.
__device__ __forceinline__ void place_run(const int32_t* ids, int64_t m0, int64_t m1, int n, int bits, int* next,
                                          int32_t* order, int64_t rows, int (&keys)[kAhead]) {
  const int lane = threadIdx.x & 63;
  for (int64_t b = m0; b < m1; b += 64 * kAhead) {  // the same for every lane: ballots see the whole wave
    if (b > m0) load_keys(ids, b + lane, m1, n, keys);
    // the lanes of the same key, for all the rows at once: a ballot waits for the vector unit
    uint64_t same[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) same[u] = __ballot(keys[u] >= 0);
    for (int i = 0; i < bits; ++i) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const bool bit = (keys[u] >> i) & 1;
        const uint64_t one = __ballot(bit);
        same[u] &= bit ? one : ~one;
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int key = keys[u];
      const bool in = key >= 0;
      const int rank = __popcll(same[u] & (((uint64_t)1 << lane) - 1));
      const int at = in ? next[key] : 0;
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      __builtin_amdgcn_wave_barrier();
      if (in && rank == 0) next[key] = at + __popcll(same[u]);
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      __builtin_amdgcn_wave_barrier();
      // ids that change while this runs could move a place past the end
      if (in && (uint64_t)(int64_t)(at + rank) < (uint64_t)rows) order[at + rank] = (int32_t)(b + 64 * u + lane);
    }
  }
}

__device__ __forceinline__ int wave_incl(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Everything by one workgroup of `blockDim.x / 64` runs, whose counts fit in LDS.
__global__ __launch_bounds__(1024) void k_route_one(const int32_t* __restrict__ ids, int64_t M, int n, int bits,
                                                    int64_t run, int32_t* __restrict__ order,
                                                    int32_t* __restrict__ offsets) {
  extern __shared__ int counts[];  // [runs][n + 1]
  __shared__ int red[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, runs = blockDim.x >> 6;
  const int64_t m0 = min(wave * run, M), m1 = min(m0 + run, M);
  int keys[kAhead];
  load_keys(ids, m0 + lane, m1, n, keys);
  for (int i = threadIdx.x; i < runs * (n + 1); i += blockDim.x) counts[i] = 0;
  __syncthreads();
  count_run(ids, m0, m1, n, counts + wave * (n + 1), keys);
  __syncthreads();
  int base = 0;
  for (int k0 = 0; k0 <= n; k0 += blockDim.x) {
    const int key = k0 + threadIdx.x;
    int sum = 0;
    if (key <= n)
      for (int r = 0; r < runs; ++r) sum += counts[r * (n + 1) + key];
    const int incl = wave_incl(sum);
    if (lane == 63) red[wave] = incl;
    __syncthreads();
    int at = base + incl - sum;
    for (int w = 0; w < runs; ++w) {
      if (w < wave) at += red[w];
      base += red[w];
    }
    __syncthreads();
    if (key <= n) {
      offsets[key] = at;
      for (int r = 0; r < runs; ++r) {
        const int c = counts[r * (n + 1) + key];
        counts[r * (n + 1) + key] = at;
        at += c;
      }
    }
  }
  __syncthreads();
  place_run(ids, m0, m1, n, bits, counts + wave * (n + 1), order, M, keys);
}

// The same in two launches, for many rows: a workgroup of 4 waves has a run for each; the
// first launch counts the workgroups' ids, counts [workgroups][n + 1].
__global__ __launch_bounds__(256) void k_route_count(const int32_t* __restrict__ ids, int64_t M, int n, int64_t run,
                                                     int* __restrict__ counts) {
  extern __shared__ int mine[];
  const int64_t m0 = min((blockIdx.x * 4 + (threadIdx.x >> 6)) * run, M), m1 = min(m0 + run, M);
  int keys[kAhead];
  load_keys(ids, m0 + (threadIdx.x & 63), m1, n, keys);
  for (int i = threadIdx.x; i <= n; i += 256) mine[i] = 0;
  __syncthreads();
  count_run(ids, m0, m1, n, mine, keys);
  __syncthreads();
  for (int i = threadIdx.x; i <= n; i += 256) counts[(int64_t)blockIdx.x * (n + 1) + i] = mine[i];
}
// The second adds up, key by key, the counts of the workgroups before and of all; its waves
// count their own runs once more.
__global__ __launch_bounds__(256) void k_route_place(const int32_t* __restrict__ ids, int64_t M, int n, int bits,
                                                     int64_t run, const int* __restrict__ counts,
                                                     int32_t* __restrict__ order, int32_t* __restrict__ offsets) {
  extern __shared__ int next[];  // [4][n + 1]
  __shared__ int red[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, groups = gridDim.x;
  const int64_t m0 = min((blockIdx.x * 4 + wave) * run, M), m1 = min(m0 + run, M);
  int keys[kAhead];
  load_keys(ids, m0 + lane, m1, n, keys);
  // the counts of 64 workgroups for the thread's two keys; the first are on their way while
  // the ids are counted
  int v[2][64];
  auto load_counts = [&](int key, int g0) {
    const int last = key < n;  // the second key is there
#pragma unroll
    for (int u = 0; u < 64; ++u) {
      const int* const c = counts + (int64_t)min(g0 + u, groups - 1) * (n + 1) + min(key, n);
      v[0][u] = c[0];
      v[1][u] = c[last];
    }
  };
  load_counts(2 * tid, 0);
  for (int i = tid; i < 4 * (n + 1); i += 256) next[i] = 0;
  __syncthreads();
  count_run(ids, m0, m1, n, next + wave * (n + 1), keys);
  __syncthreads();
  int base = 0;
  for (int k0 = 0; k0 <= n; k0 += 512) {  // two neighbouring keys a thread
    const int key = k0 + 2 * tid;
    int before[2] = {0, 0}, all[2] = {0, 0};
    for (int g0 = 0; g0 < groups; g0 += 64) {
      if (k0 + g0 > 0) load_counts(key, g0);
#pragma unroll
      for (int u = 0; u < 64; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (g0 + u < (int)blockIdx.x) before[i] += v[i][u];
          if (g0 + u < groups) all[i] += v[i][u];
        }
    }
    if (key > n) all[0] = 0;
    if (key >= n) all[1] = 0;
    const int incl = wave_incl(all[0] + all[1]);
    if (lane == 63) red[wave] = incl;
    __syncthreads();
    int at = base + incl - all[0] - all[1];
    for (int w = 0; w < 4; ++w) {
      if (w < wave) at += red[w];
      base += red[w];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (key + i <= n) {
        if (blockIdx.x == 0) offsets[key + i] = at;
        int to = at + before[i];
        for (int w = 0; w < 4; ++w) {
          const int c = next[w * (n + 1) + key + i];
          next[w * (n + 1) + key + i] = to;
          to += c;
        }
      }
      at += all[i];
    }
  }
  __syncthreads();
  place_run(ids, m0, m1, n, bits, next + wave * (n + 1), order, M, keys);
}

}  // namespace

hipError_t launch_route(const int32_t* ids, int64_t M, int n, int32_t* order, int32_t* offsets, int* counts,
                        hipStream_t st) {
  int runs;
  int64_t run;
  const bool one = plan_route(M, n, &runs, &run);
  int bits = 1;
  while ((n >> bits) != 0) ++bits;  // keys 0 .. n
  const size_t lds = (size_t)(n + 1) * 4;
  if (one) {
    hipLaunchKernelGGL(k_route_one, dim3(1), dim3(64 * runs), lds * runs, st, ids, M, n, bits, run, order, offsets);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(k_route_count, dim3(runs), dim3(256), lds, st, ids, M, n, run, counts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_route_place, dim3(runs), dim3(256), 4 * lds, st, ids, M, n, bits, run, counts, order, offsets);
  return hipGetLastError();
}

}  // namespace nf4k
