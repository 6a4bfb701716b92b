// 8-bit storage in blocks of 128 (gfx950): quantization and dequantization.
//
// A block is 128 columns of one row (activations) or of 128 rows (a weight);
// the blocks at the right and lower edge are shorter.  With F the format's
// largest value,
//     amax = max(max |x| over the block, 2^-100),  scale = amax / F,
//     code = rne8(x * (F * (1 / amax))),
// each quotient and product rounded to fp32.
#include <algorithm>
#include <type_traits>

#include "fp8.hpp"
#include "launch.hpp"

namespace nf4k {

namespace {

// 16 bytes of input: 8 bf16 or 4 fp32 values
template <bool BF16>
struct In;
template <>
struct In<true> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void widen(u32x4 r, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __builtin_bit_cast(float, r[i] << 16);
      v[2 * i + 1] = __builtin_bit_cast(float, r[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct In<false> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void widen(u32x4 r, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = r[i];  // a value: a bit cast of the element itself takes the vector's first one
      v[i] = __builtin_bit_cast(float, w);
    }
  }
};

// One scale per row and 128 columns: 16 lanes hold a block, 8 values each, and
// find its largest magnitude in four DPP steps.  Bound by memory: 16384 x 8192 bf16
// 75 us, 5.4 TB/s; 1 x 4096 2 us beside the launch.
template <bool BF16, bool E5M2>
__global__ __launch_bounds__(256) void k_fp8_quant_rows(const void* __restrict__ X, uint32_t blocks, int cols,
                                                        uint32_t kb, uint8_t* __restrict__ codes,
                                                        float* __restrict__ scales) {
  const uint32_t b = blockIdx.x * 16 + (threadIdx.x >> 4);
  const int l = threadIdx.x & 15;
  if (b >= blocks) return;
  const uint32_t row = b / kb;
  const int col = (int)(b - row * kb) * 128 + l * 8;
  const bool in = col < cols;  // cols is a multiple of 16: a lane's 8 values are all in or all out
  const int64_t at = (int64_t)row * cols + col;
  float v[8] = {};
  if (in) {
    if constexpr (BF16) {
      In<true>::widen(*(const u32x4*)((const uint16_t*)X + at), v);
    } else {
      In<false>::widen(*(const u32x4*)((const float*)X + at), v);
      In<false>::widen(*(const u32x4*)((const float*)X + at + 4), v + 4);
    }
  }
  const float amax = row16_max(fmaxf(abs_max4(v[0], v[1], v[2], v[3]), abs_max4(v[4], v[5], v[6], v[7])));
  float scale, mul;
  fp8_scale<E5M2>(amax, scale, mul);
  if (in) {
    uint2 o;
    o.x = pack_fp8x4<E5M2>(v[0] * mul, v[1] * mul, v[2] * mul, v[3] * mul);
    o.y = pack_fp8x4<E5M2>(v[4] * mul, v[5] * mul, v[6] * mul, v[7] * mul);
    *(uint2*)(codes + at) = o;
  }
  if (l == 0) scales[b] = scale;
}

// One scale per 128 x 128 block: a workgroup holds the block in registers, so
// the weight is read once.  Bound by memory; a weight is not used again soon, so
// both sides go past the caches (28672 x 8192 fp32: 191 us, 6.2 TB/s, against 208
// with ordinary loads and stores).
template <bool BF16, bool E5M2>
__global__ __launch_bounds__(256) void k_fp8_quant_tiles(const void* __restrict__ X, int64_t rows, int cols, int kb,
                                                         uint8_t* __restrict__ codes, float* __restrict__ scales) {
  constexpr int N = In<BF16>::N;
  constexpr int LPR = 128 / N;    // lanes per row
  constexpr int RPI = 256 / LPR;  // rows per load of the workgroup
  constexpr int IT = 128 / RPI;
  const uint32_t rb = blockIdx.x / (uint32_t)kb;
  const int cb = (int)(blockIdx.x - rb * kb);
  const int r = threadIdx.x / LPR;
  const int col = cb * 128 + (threadIdx.x % LPR) * N;
  const int64_t row0 = (int64_t)rb * 128 + r;
  const bool incol = col < cols;
  u32x4 raw[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int64_t row = row0 + i * RPI;
    raw[i] = u32x4{0u, 0u, 0u, 0u};
    if (incol && row < rows)
      raw[i] = __builtin_nontemporal_load((const u32x4*)((const uint8_t*)X + (row * cols + col) * (BF16 ? 2 : 4)));
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    float v[N];
    In<BF16>::widen(raw[i], v);
#pragma unroll
    for (int j = 0; j < N; j += 4) amax = fmaxf(amax, abs_max4(v[j], v[j + 1], v[j + 2], v[j + 3]));
  }
  amax = row16_max(amax);
  amax = fmaxf(amax, __shfl_xor(amax, 16));
  amax = fmaxf(amax, __shfl_xor(amax, 32));
  __shared__ float red[4];
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = amax;
  __syncthreads();
  amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  float scale, mul;
  fp8_scale<E5M2>(amax, scale, mul);
  if (threadIdx.x == 0) scales[blockIdx.x] = scale;
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int64_t row = row0 + i * RPI;
    if (!incol || row >= rows) continue;
    float v[N];
    In<BF16>::widen(raw[i], v);
    uint32_t o[N / 4];
#pragma unroll
    for (int j = 0; j < N; j += 4)
      o[j / 4] = pack_fp8x4<E5M2>(v[j] * mul, v[j + 1] * mul, v[j + 2] * mul, v[j + 3] * mul);
    uint8_t* dst = codes + row * cols + col;
    if constexpr (N == 8) __builtin_nontemporal_store((uint64_t)o[1] << 32 | o[0], (uint64_t*)dst);
    else __builtin_nontemporal_store(o[0], (uint32_t*)dst);
  }
}

// 16 bytes of output a lane and store, so that a wave writes whole lines; four of
// them on the way.  Bound by memory: 28672 x 8192 to fp32 197 us, 6.0 TB/s (16 codes
// a lane, whose stores are 64 bytes apart: 356 us), to bf16 128 us, 5.5 TB/s.
template <bool E5M2, bool OUT16>
__global__ __launch_bounds__(256) void k_fp8_dequant(const uint8_t* __restrict__ codes,
                                                     const float* __restrict__ scales, uint32_t n, uint32_t per_row,
                                                     int kb, int row_shift, void* __restrict__ out) {
  constexpr int V = OUT16 ? 8 : 4;  // values of 16 bytes; per_row of them in a row, n in all
  const uint32_t i0 = blockIdx.x * 1024 + threadIdx.x;
  uint32_t c[4][V / 4];
  float s[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint32_t i = min(i0 + u * 256, n - 1);
    const uint32_t row = i / per_row;
    const uint32_t* src = (const uint32_t*)(codes + (int64_t)i * V);
#pragma unroll
    for (int k = 0; k < V / 4; ++k) c[u][k] = src[k];
    s[u] = scales[(int64_t)(row >> row_shift) * kb + ((i - row * per_row) * V >> 7)];
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint32_t i = i0 + u * 256;
    if (i >= n) break;
    float v[V];
#pragma unroll
    for (int k = 0; k < V / 4; ++k) {
      float t[4];
      unpack_fp8x4<E5M2>(c[u][k], t);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * k + j] = t[j] * s[u];
    }
    if constexpr (OUT16) {
      u32x4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
      ((u32x4*)out)[i] = o;
    } else {
      ((floatx4*)out)[i] = floatx4{v[0], v[1], v[2], v[3]};
    }
  }
}

}  // namespace

hipError_t launch_fp8_quantize(const void* X, bool bf16, int64_t rows, int64_t cols, bool e5m2, int block_rows,
                               uint8_t* codes, float* scales, hipStream_t st) {
  const int kb = (int)((cols + 127) / 128);
#define NF4K_BY_TYPE(CALL)                                                        \
  do {                                                                            \
    if (bf16) { if (e5m2) { CALL(true, true); } else { CALL(true, false); } }     \
    else { if (e5m2) { CALL(false, true); } else { CALL(false, false); } }        \
  } while (0)
  // at most 2^23 workgroups of 256 a launch: its work-items stay below 2^32
  constexpr int64_t kMost = (int64_t)1 << 23;
  if (block_rows == 1) {
    const int64_t step = kMost * 16 / kb;  // rows a launch
    for (int64_t r0 = 0; r0 < rows; r0 += step) {
      const int64_t blocks = std::min(step, rows - r0) * kb;
      const uint8_t* in = (const uint8_t*)X + r0 * cols * (bf16 ? 2 : 4);
#define NF4K_CALL(B, E)                                                                                          \
  hipLaunchKernelGGL((k_fp8_quant_rows<B, E>), dim3((unsigned)((blocks + 15) / 16)), dim3(256), 0, st, (const void*)in, \
                     (uint32_t)blocks, (int)cols, (uint32_t)kb, codes + r0 * cols, scales + r0 * kb)
      NF4K_BY_TYPE(NF4K_CALL);
#undef NF4K_CALL
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  const int64_t step = kMost / kb * 128;
  for (int64_t r0 = 0; r0 < rows; r0 += step) {
    const int64_t nr = std::min(step, rows - r0);
    const int64_t blocks = (nr + 127) / 128 * kb;
    const uint8_t* in = (const uint8_t*)X + r0 * cols * (bf16 ? 2 : 4);
#define NF4K_CALL(B, E)                                                                                          \
  hipLaunchKernelGGL((k_fp8_quant_tiles<B, E>), dim3((unsigned)blocks), dim3(256), 0, st, (const void*)in, nr, (int)cols, \
                     kb, codes + r0 * cols, scales + r0 / 128 * kb)
    NF4K_BY_TYPE(NF4K_CALL);
#undef NF4K_CALL
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_fp8_dequantize(const uint8_t* codes, const float* scales, int64_t rows, int64_t cols, bool e5m2,
                                 int block_rows, bool bf16, void* out, hipStream_t st) {
  const int kb = (int)((cols + 127) / 128);
  const int64_t per_row = cols / (bf16 ? 8 : 4);
  // whole blocks of rows a launch, its values of 16 bytes below 2^31
  const int64_t step = std::max<int64_t>(1, ((int64_t)1 << 31) / per_row / 128) * 128;
  for (int64_t r0 = 0; r0 < rows; r0 += step) {
    const int64_t n = std::min(step, rows - r0) * per_row;
    const dim3 gr((unsigned)((n + 1023) / 1024)), bl(256);
    uint8_t* const to = (uint8_t*)out + r0 * cols * (bf16 ? 2 : 4);
#define NF4K_CALL(B, E)                                                                                       \
  hipLaunchKernelGGL((k_fp8_dequant<E, B>), gr, bl, 0, st, codes + r0 * cols, scales + r0 / block_rows * kb,  \
                     (uint32_t)n, (uint32_t)per_row, kb, block_rows == 1 ? 0 : 7, (void*)to)
    NF4K_BY_TYPE(NF4K_CALL);
#undef NF4K_CALL
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace nf4k
