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

// counts[key] += 1 for the wave's rows [m0, m1)
__device__ __forceinline__ void count_run(const int32_t* ids, int64_t m0, int64_t m1, int n, int* counts) {
  for (int64_t m = m0 + (threadIdx.x & 63); m < m1; m += 64 * kAhead) {
    int key[kAhead];
    load_keys(ids, m, m1, n, key);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (key[u] >= 0) atomicAdd(counts + key[u], 1);
  }
}

// order[next[key]++] = m for the wave's rows [m0, m1), in their order.  `next` is the
// wave's own; the LDS operations of one wave stay in order, and the fences keep the
// compiler from moving them.
__device__ __forceinline__ void place_run(const int32_t* ids, int64_t m0, int64_t m1, int n, int bits, int* next,
                                          int32_t* order, int64_t rows) {
  const int lane = threadIdx.x & 63;
  for (int64_t b = m0; b < m1; b += 64 * kAhead) {  // the same for every lane: ballots see the whole wave
    int keys[kAhead];
    load_keys(ids, b + lane, m1, n, keys);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int key = keys[u];
      const bool in = key >= 0;
      uint64_t same = __ballot(in);
      for (int i = 0; i < bits; ++i) {
        const uint64_t one = __ballot((key >> i) & 1);
        same &= (key >> i) & 1 ? one : ~one;
      }
      const int rank = __popcll(same & (((uint64_t)1 << lane) - 1));
      const int at = in ? next[key] : 0;
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      __builtin_amdgcn_wave_barrier();
      if (in && rank == 0) next[key] = at + __popcll(same);
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
  for (int i = threadIdx.x; i < runs * (n + 1); i += blockDim.x) counts[i] = 0;
  __syncthreads();
  const int64_t m0 = min(wave * run, M), m1 = min(m0 + run, M);
  count_run(ids, m0, m1, n, counts + wave * (n + 1));
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
  place_run(ids, m0, m1, n, bits, counts + wave * (n + 1), order, M);
}

// The same in three launches, a workgroup of one wave a run; counts [n + 1][runs].
__global__ __launch_bounds__(64) void k_route_count(const int32_t* __restrict__ ids, int64_t M, int n, int64_t run,
                                                    int* __restrict__ counts) {
  extern __shared__ int mine[];
  for (int i = threadIdx.x; i <= n; i += 64) mine[i] = 0;
  __syncthreads();
  const int64_t m0 = blockIdx.x * run;
  count_run(ids, m0, min(m0 + run, M), n, mine);
  __syncthreads();
  for (int i = threadIdx.x; i <= n; i += 64) counts[(int64_t)i * gridDim.x + blockIdx.x] = mine[i];
}
// A wave turns one key's counts into the places before each run, and totals[key] into their sum.
__global__ __launch_bounds__(256) void k_route_scan(int* __restrict__ counts, int runs, int n,
                                                    int* __restrict__ totals) {
  const int key = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (key > n) return;
  int* c = counts + (int64_t)key * runs;
  int base = 0;
  for (int r0 = 0; r0 < runs; r0 += 256) {
    int v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = r0 + 64 * u + lane < runs ? c[r0 + 64 * u + lane] : 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int incl = wave_incl(v[u]);
      if (r0 + 64 * u + lane < runs) c[r0 + 64 * u + lane] = base + incl - v[u];
      base += __shfl(incl, 63);
    }
  }
  if (lane == 0) totals[key] = base;
}
__global__ __launch_bounds__(64) void k_route_place(const int32_t* __restrict__ ids, int64_t M, int n, int bits,
                                                    int64_t run, const int* __restrict__ counts,
                                                    const int* __restrict__ totals, int32_t* __restrict__ order,
                                                    int32_t* __restrict__ offsets) {
  extern __shared__ int next[];
  const int lane = threadIdx.x;
  int base = 0;
  for (int k0 = 0; k0 <= n; k0 += 64) {
    const int key = k0 + lane;
    const int v = key <= n ? totals[key] : 0;
    const int incl = wave_incl(v);
    if (key <= n) {
      next[key] = base + incl - v + counts[(int64_t)key * gridDim.x + blockIdx.x];
      if (blockIdx.x == 0) offsets[key] = base + incl - v;
    }
    base += __shfl(incl, 63);
  }
  __syncthreads();
  const int64_t m0 = blockIdx.x * run;
  place_run(ids, m0, min(m0 + run, M), n, bits, next, order, M);
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
  int* totals = counts + (int64_t)(n + 1) * runs;
  hipLaunchKernelGGL(k_route_count, dim3(runs), dim3(64), lds, st, ids, M, n, run, counts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_route_scan, dim3(n / 4 + 1), dim3(256), 0, st, counts, runs, n, totals);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_route_place, dim3(runs), dim3(64), lds, st, ids, M, n, bits, run, counts, totals, order,
                     offsets);
  return hipGetLastError();
}

}  // namespace nf4k
