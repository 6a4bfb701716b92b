// What the norms' kernels share: how a row is held, its sums, and the kernel for a
// width.
#pragma once

#include <type_traits>

#include "fp8.hpp"
#include "launch.hpp"

namespace nf4k {

namespace {

__device__ __forceinline__ void widen8(u32x4 r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __builtin_bit_cast(float, r[i] << 16);
    v[2 * i + 1] = __builtin_bit_cast(float, r[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ u32x4 narrow8(const float (&v)[8]) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  return r;
}

// How a row is held: TPR = 16 or 64 threads of a wave (several rows a workgroup,
// no barrier), or TPR = 0: the whole workgroup, of as many waves as the row needs.
// Every thread has NC chunks of 8 neighbouring columns, a row's width apart.
template <int TPR>
__device__ __forceinline__ int row_threads() { return TPR ? TPR : (int)blockDim.x; }

// Sum over 16 lanes or the wave; every lane gets it.  Lane exchanges in the vector
// unit, not LDS permutes (1.5 % less at 16384 x 8192, forward).
template <int N, class F>
__device__ __forceinline__ F wave_add(F x) {
  constexpr int W = sizeof(F) / 4;
  struct Words {
    int w[W];
  };
  auto dpp = [&](auto ctrl) {
    Words v = __builtin_bit_cast(Words, x);
#pragma unroll
    for (int i = 0; i < W; ++i) v.w[i] = __builtin_amdgcn_mov_dpp(v.w[i], decltype(ctrl)::value, 0xF, 0xF, true);
    x += __builtin_bit_cast(F, v);
  };
  dpp(std::integral_constant<int, 0xB1>{});   // quad_perm [1,0,3,2]
  dpp(std::integral_constant<int, 0x4E>{});   // quad_perm [2,3,0,1]
  dpp(std::integral_constant<int, 0x141>{});  // row_half_mirror
  dpp(std::integral_constant<int, 0x140>{});  // row_mirror
  if constexpr (N == 64) {
    Words a = __builtin_bit_cast(Words, x), b = a;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const auto r = __builtin_amdgcn_permlane16_swap(a.w[i], a.w[i], false, false);
      a.w[i] = r[0];
      b.w[i] = r[1];
    }
    x = __builtin_bit_cast(F, a) + __builtin_bit_cast(F, b);
    a = __builtin_bit_cast(Words, x);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const auto r = __builtin_amdgcn_permlane32_swap(a.w[i], a.w[i], false, false);
      a.w[i] = r[0];
      b.w[i] = r[1];
    }
    x = __builtin_bit_cast(F, a) + __builtin_bit_cast(F, b);
  }
  return x;
}

// Sum over the threads of a row, in a fixed order; every thread gets it.  `red`
// (TPR = 0: a value for each of up to 16 waves, the unused ones zero) must not be
// the one of the previous call.
template <int TPR, class F>
__device__ __forceinline__ F row_sum(F x, F (&red)[16]) {
  x = wave_add<TPR == 16 ? 16 : 64>(x);
  if constexpr (TPR == 0) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0;
#pragma unroll
    for (int i = 0; i < 16; i += 4) x += (red[i] + red[i + 1]) + (red[i + 2] + red[i + 3]);
  }
  return x;
}
template <int TPR, class F>
__device__ __forceinline__ void row_sum_init(F (&red)[16]) {
  // waves that the workgroup does not have count as zero; the barrier in row_sum orders this
  if (TPR == 0 && threadIdx.x < 16 && threadIdx.x >= (blockDim.x >> 6)) red[threadIdx.x] = 0;
}

}  // namespace

}  // namespace nf4k

// the kernel for a width: rows by 16 or 64 threads of a wave up to 2048 columns, by
// the workgroup beyond, with at most 1024 threads
#define NF4K_NORM_SHAPES(CALL)         \
  do {                                 \
    if (H <= 128) CALL(16, 1);         \
    else if (H <= 512) CALL(64, 1);    \
    else if (H <= 1024) CALL(64, 2);   \
    else if (H <= 2048) CALL(64, 4);   \
    else if (H <= 8192) CALL(0, 1);    \
    else if (H <= 16384) CALL(0, 2);   \
    else CALL(0, 4);                   \
  } while (0)
