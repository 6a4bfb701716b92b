// Root-mean-square norm with the residual's addition, an 8-bit output, and its
// gradient (gfx950).
//
// Forward, per row of width H:
//     h = bf16(x + res)  (h = x without a residual),
//     rstd = 1 / sqrt(mean(h^2) + eps),   y = h * rstd * w;
// y leaves as bf16, as 8-bit codes with a scale per 128 columns (quantized from
// the fp32 y, not from its bf16 rounding), or both.
// Gradient, with xhat = h * rstd and u = dy * w:
//     dx = rstd * (u - xhat * mean(u * xhat)) + dh,   dw = sum over rows dy * xhat.
// Statistics, sums and y are fp32.
#include <algorithm>
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

// Sum over the TPR threads of a row, in a fixed order; every thread gets it.
// TPR of 16 and 64 stay inside a wave; a larger TPR is the whole workgroup, and
// `red` (one float per wave) must not be the one of the previous call.
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float* red) {
#pragma unroll
  for (int o = 1; o < (TPR < 64 ? TPR : 64); o <<= 1) x += __shfl_xor(x, o);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    x = red[0];
#pragma unroll
    for (int i = 1; i < W; ++i) x += red[i];
  }
  return x;
}

struct NormArgs {
  const uint16_t* X;
  const uint16_t* R;  // residual, or NULL
  const uint16_t* w;
  int64_t rows;
  int H;
  float eps;
  uint16_t* Hout;  // with a residual
  uint16_t* Y;     // or NULL
  uint8_t* codes;  // or NULL
  float* scales;
  float* rstd;  // or NULL
};

// TPR threads hold a row in registers, NC chunks of 8 columns each; 16
// neighbouring threads hold one block of the 8-bit output.
template <int TPR, int NC>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_rmsnorm(NormArgs p) {
  constexpr int NT = TPR < 256 ? 256 : TPR;
  __shared__ float red[TPR / 64 + 1];
  const int64_t row = (int64_t)blockIdx.x * (NT / TPR) + threadIdx.x / TPR;
  const int t = threadIdx.x % TPR;
  if (row >= p.rows) return;  // whole rows of threads; with TPR > 64 the whole workgroup
  const int64_t base = row * p.H;
  u32x4 hb[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int col = (c * TPR + t) * 8;
    hb[c] = u32x4{0u, 0u, 0u, 0u};
    if (col < p.H) hb[c] = *(const u32x4*)(p.X + base + col);
  }
  if (p.R) {
    u32x4 rb[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * TPR + t) * 8;
      rb[c] = u32x4{0u, 0u, 0u, 0u};
      if (col < p.H) rb[c] = *(const u32x4*)(p.R + base + col);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float a[8], b[8];
      widen8(hb[c], a);
      widen8(rb[c], b);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] += b[j];
      hb[c] = narrow8(a);
      const int col = (c * TPR + t) * 8;
      if (col < p.H) *(u32x4*)(p.Hout + base + col) = hb[c];
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float a[8];
    widen8(hb[c], a);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(a[j], a[j], ss);
  }
  ss = row_sum<TPR>(ss, red);
  const float rstd = 1.f / sqrtf(ss / (float)p.H + p.eps);
  if (p.rstd && t == 0) p.rstd[row] = rstd;
  const int64_t kb = (p.H + 127) / 128;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int col = (c * TPR + t) * 8;
    const bool in = col < p.H;
    float a[8], w[8];
    widen8(hb[c], a);
    u32x4 wb = {0u, 0u, 0u, 0u};
    if (in) wb = *(const u32x4*)(p.w + col);
    widen8(wb, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = a[j] * rstd * w[j];
    if (p.Y && in) *(u32x4*)(p.Y + base + col) = narrow8(a);
    if (p.codes) {
      // 0 * inf of a row without any magnitude and eps = 0 stays out of the block's padding
      const float m = in ? fmaxf(abs_max4(a[0], a[1], a[2], a[3]), abs_max4(a[4], a[5], a[6], a[7])) : 0.f;
      float scale, mul;
      fp8_scale<false>(row16_max(m), scale, mul);
      if (in) {
        uint2 o;
        o.x = pack_fp8x4<false>(a[0] * mul, a[1] * mul, a[2] * mul, a[3] * mul);
        o.y = pack_fp8x4<false>(a[4] * mul, a[5] * mul, a[6] * mul, a[7] * mul);
        *(uint2*)(p.codes + base + col) = o;
        if ((t & 15) == 0) p.scales[row * kb + (col >> 7)] = scale;
      }
    }
  }
}

struct NormGradArgs {
  const uint16_t* dY;
  const uint16_t* Hs;
  const uint16_t* w;
  const float* rstd;
  const uint16_t* dH;  // or NULL
  int64_t rows;
  int H;
  uint16_t* dX;
  float* part;  // [gridDim.x][H]
};

// A workgroup takes every gridDim.x-th group of NT / TPR rows; each thread
// keeps its columns' share of dw in registers over all of them.
template <int TPR, int NC>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_rmsnorm_grad(NormGradArgs p) {
  constexpr int NT = TPR < 256 ? 256 : TPR;
  constexpr int TEAMS = NT / TPR;
  __shared__ float red[2][TPR / 64 + 1];
  const int team = threadIdx.x / TPR;
  const int t = threadIdx.x % TPR;
  float dw[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[c][j] = 0.f;
  const float invH = 1.f / (float)p.H;
  int flip = 0;
  for (int64_t row = (int64_t)blockIdx.x * TEAMS + team; row < p.rows; row += (int64_t)gridDim.x * TEAMS) {
    const int64_t base = row * p.H;
    const float rstd = p.rstd[row];
    u32x4 gb[NC], hb[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * TPR + t) * 8;
      gb[c] = hb[c] = u32x4{0u, 0u, 0u, 0u};
      if (col < p.H) {
        gb[c] = *(const u32x4*)(p.dY + base + col);
        hb[c] = *(const u32x4*)(p.Hs + base + col);
      }
    }
    float dot = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * TPR + t) * 8;
      float g[8], h[8], w[8];
      u32x4 wb = {0u, 0u, 0u, 0u};
      if (col < p.H) wb = *(const u32x4*)(p.w + col);
      widen8(gb[c], g);
      widen8(hb[c], h);
      widen8(wb, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xhat = h[j] * rstd;
        dot = __builtin_fmaf(g[j] * w[j], xhat, dot);
        dw[c][j] = __builtin_fmaf(g[j], xhat, dw[c][j]);
      }
    }
    dot = row_sum<TPR>(dot, red[flip]) * invH;
    flip ^= 1;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * TPR + t) * 8;
      if (col >= p.H) continue;
      float g[8], h[8], w[8], d[8] = {};
      widen8(gb[c], g);
      widen8(hb[c], h);
      widen8(*(const u32x4*)(p.w + col), w);
      if (p.dH) widen8(*(const u32x4*)(p.dH + base + col), d);
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = __builtin_fmaf(rstd, g[j] * w[j] - h[j] * rstd * dot, d[j]);
      *(u32x4*)(p.dX + base + col) = narrow8(d);
    }
  }
  if constexpr (TEAMS > 1) {
    __shared__ float sum[TEAMS][TPR * NC * 8];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[team][(c * TPR + t) * 8 + j] = dw[c][j];
    __syncthreads();
    for (int col = threadIdx.x; col < p.H; col += NT) {
      float s = sum[0][col];
      for (int k = 1; k < TEAMS; ++k) s += sum[k][col];
      p.part[(int64_t)blockIdx.x * p.H + col] = s;
    }
  } else {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * TPR + t) * 8;
      if (col >= p.H) continue;
      floatx4* dst = (floatx4*)(p.part + (int64_t)blockIdx.x * p.H + col);
      dst[0] = floatx4{dw[c][0], dw[c][1], dw[c][2], dw[c][3]};
      dst[1] = floatx4{dw[c][4], dw[c][5], dw[c][6], dw[c][7]};
    }
  }
}

// dw[col] = sum of the parts in a fixed order: 16 waves, each every 16th part
__global__ __launch_bounds__(1024) void k_rmsnorm_dw(const float* __restrict__ part, int n, int H,
                                                     float* __restrict__ dw) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane;
  float s = 0.f;
  if (col < H)
    for (int i = wave; i < n; i += 16) s += part[(int64_t)i * H + col];
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && col < H) {
    for (int i = 1; i < 16; ++i) s += red[i][lane];
    dw[col] = s;
  }
}

}  // namespace

// the kernels' (threads per row, chunks) by width; see rmsnorm_threads
#define NF4K_NORM_SHAPES(CALL)                         \
  do {                                                 \
    if (tpr == 16) CALL(16, 1);                        \
    else if (tpr == 64) { if (H <= 512) CALL(64, 1); else CALL(64, 4); } \
    else if (tpr == 256) { if (H <= 4096) CALL(256, 2); else CALL(256, 4); } \
    else if (tpr == 512) CALL(512, 4);                 \
    else CALL(1024, 4);                                \
  } while (0)

hipError_t launch_rmsnorm_fwd(const uint16_t* X, const uint16_t* R, const uint16_t* w, int64_t M, int H, float eps,
                              uint16_t* Hout, uint16_t* Y, uint8_t* codes, float* scales, float* rstd,
                              hipStream_t st) {
  const int tpr = rmsnorm_threads(H), nt = std::max(tpr, 256), teams = nt / tpr;
  const int64_t kb = (H + 127) / 128;
  constexpr int64_t kMost = (int64_t)1 << 21;  // workgroups a launch: its work-items stay below 2^32
  for (int64_t r0 = 0; r0 < M; r0 += kMost * teams) {
    NormArgs a{X + r0 * H, R ? R + r0 * H : nullptr, w, std::min(kMost * teams, M - r0), H, eps,
               Hout ? Hout + r0 * H : nullptr, Y ? Y + r0 * H : nullptr, codes ? codes + r0 * H : nullptr,
               scales ? scales + r0 * kb : nullptr, rstd ? rstd + r0 : nullptr};
    const dim3 gr((unsigned)((a.rows + teams - 1) / teams)), bl(nt);
#define NF4K_CALL(T, N) hipLaunchKernelGGL((k_rmsnorm<T, N>), gr, bl, 0, st, a)
    NF4K_NORM_SHAPES(NF4K_CALL);
#undef NF4K_CALL
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_rmsnorm_bwd(const uint16_t* dY, const uint16_t* Hs, const uint16_t* w, const float* rstd,
                              const uint16_t* dH, int64_t M, int H, uint16_t* dX, float* dw, float* part,
                              hipStream_t st) {
  const int tpr = rmsnorm_threads(H), nt = std::max(tpr, 256);
  const int parts = rmsnorm_parts(M, H);
  NormGradArgs a{dY, Hs, w, rstd, dH, M, H, dX, part};
  const dim3 gr((unsigned)parts), bl(nt);
#define NF4K_CALL(T, N) hipLaunchKernelGGL((k_rmsnorm_grad<T, N>), gr, bl, 0, st, a)
  NF4K_NORM_SHAPES(NF4K_CALL);
#undef NF4K_CALL
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_rmsnorm_dw, dim3((unsigned)((H + 63) / 64)), dim3(1024), 0, st, part, parts, H, dw);
  return hipGetLastError();
}

}  // namespace nf4k
