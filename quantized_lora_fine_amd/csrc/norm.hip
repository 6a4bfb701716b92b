// Root-mean-square norm with the residual's addition, an 8-bit output, and its
// gradient (gfx950).
//
// Forward, per row of width H:
//     h = bf16(x + res)  (h = x without a residual),
//     rstd = 1 / sqrt(mean(h^2) + eps),   y = h * rstd * w;
// y leaves as bf16, as 8-bit codes with a scale per 128 columns (quantized from
// y, not from its bf16 rounding), or both.  A product h * w of bf16 values is exact
// in fp32; the sum of squares is fp64, and rstd = 2^-k (hi + lo) with two fp32 values,
// so that fma(hw, hi, hw * lo) is y rounded once, to fp32; bf16 values, codes and
// scales are rounded from there.  Of 600 rows of 4096, 5 have a code that y in 64 bits
// puts on the other side of a tie, and 178 with fp32 throughout.  By replayed graphs at
// 16384 x 8192 with a residual and both outputs: 209 us with fp32 throughout, 211 so,
// 217 with y and the root in fp64; at 16384 x 4096 with the 8-bit output alone 83.5, 89
// and 95.  The factor 2^-k goes with the pair, or, for rows far from 1, with h (for all
// rows that would take 1 % more time).
// Gradient, with xhat = h * rstd and u = dy * w:
//     dx = rstd * (u - xhat * mean(u * xhat)) + dh,   dw = sum over rows dy * xhat.
// The gradient's sums are fp32.
#include <algorithm>

#include "norm.hpp"

namespace nf4k {

namespace {

struct NormArgs {
  const uint16_t* X;
  const uint16_t* R;  // residual, or NULL
  const uint16_t* w;
  int64_t rows;
  int H;
  double inv_H;
  float eps;
  uint16_t* Hout;  // with a residual
  uint16_t* Y;     // or NULL
  uint8_t* codes;  // or NULL
  float* scales;
  float* rstd;  // or NULL
};

// The row stays in registers, so each byte moves once; 16 neighbouring threads hold
// one block of the 8-bit output.  Bound by memory: 16384 x 8192 with a residual and
// both outputs 211 us, 5.8 TB/s; one row of 4096 3.1 us by replayed graphs, the launch
// and three waits.
template <int TPR, int NC>
__global__ __launch_bounds__(TPR ? 256 : 1024) void k_rmsnorm(NormArgs p) {
  __shared__ __align__(16) double red[16];
  row_sum_init<TPR>(red);
  const int T = row_threads<TPR>();
  const int64_t row = TPR ? (int64_t)blockIdx.x * (256 / (TPR ? TPR : 1)) + threadIdx.x / (TPR ? TPR : 1) : blockIdx.x;
  const int t = TPR ? threadIdx.x % (TPR ? TPR : 1) : threadIdx.x;
  if (row >= p.rows) return;  // whole rows of threads (TPR = 0: no workgroup)
  const int64_t base = row * p.H;
  u32x4 hb[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int col = (c * T + t) * 8;
    hb[c] = u32x4{0u, 0u, 0u, 0u};
    if (col < p.H) hb[c] = *(const u32x4*)(p.X + base + col);
  }
  if (p.R) {
    u32x4 rb[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * T + t) * 8;
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
      const int col = (c * T + t) * 8;
      if (col < p.H) *(u32x4*)(p.Hout + base + col) = hb[c];
    }
  }
  double ss = 0;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float a[8];
    widen8(hb[c], a);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = __builtin_fma((double)a[j], (double)a[j], ss);
  }
  ss = row_sum<TPR>(ss, red);
  // one step of Newton's from the fp32 root of mean / 4^k, which is 1/4 or more and
  // below 1; a root of 0 or infinity stands as it is.  Far from 1, rstd may lie past
  // fp32's range (a row of bf16's subnormals), and so may its product with a block's
  // multiplier (up to 448 * 2^100, for a block of zeros) or h * w: there h is multiplied
  // by 2^-k and the products take the root, from 1 to 2, alone.  Up to 2^17 rstd's
  // product with a multiplier is below 2^126, and the factor stays with it.
  double mean = __builtin_fma(ss, p.inv_H, (double)p.eps);
  const int k = (__builtin_amdgcn_frexp_exp(mean) + 1) >> 1;
  mean = __builtin_amdgcn_ldexp(mean, -2 * k);
  const float root = 1.f / sqrtf((float)mean);
  const float e = (float)__builtin_fma(-mean, (double)root * (double)root, 1.);
  const float rest = fabsf(e) < 1.f ? 0.5f * root * e : 0.f;
  if (p.rstd && t == 0) p.rstd[row] = ldexpf(root + rest, -k);
  const int far = (unsigned)(k + 16) <= 32u ? 0 : k;
  const float hi = ldexpf(root, far - k), lo = ldexpf(rest, far - k);
  const int64_t kb = (p.H + 127) / 128;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int col = (c * T + t) * 8;
    const bool in = col < p.H;
    float a[8], w[8];
    widen8(hb[c], a);
    u32x4 wb = {0u, 0u, 0u, 0u};
    if (in) wb = *(const u32x4*)(p.w + col);
    widen8(wb, w);
    if (far) {
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = ldexpf(a[j], -far);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j] *= a[j];
      a[j] = __builtin_fmaf(w[j], hi, w[j] * lo);
    }
    if (p.Y && in) *(u32x4*)(p.Y + base + col) = narrow8(a);
    if (p.codes) {
      // 0 * inf of a row without any magnitude and eps = 0 stays out of the block's padding
      const float m = in ? fmaxf(abs_max4(a[0], a[1], a[2], a[3]), abs_max4(a[4], a[5], a[6], a[7])) : 0.f;
      float scale, mul;
      fp8_scale<false>(row16_max(m), scale, mul);
      if (in) {
        uint2 o;
        const float mhi = hi * mul, mlo = __builtin_fmaf(hi, mul, -mhi) + lo * mul;
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = __builtin_fmaf(w[j], mhi, w[j] * mlo);
        o.x = pack_fp8x4<false>(a[0], a[1], a[2], a[3]);
        o.y = pack_fp8x4<false>(a[4], a[5], a[6], a[7]);
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

// A workgroup takes every gridDim.x-th row (TPR > 0: group of 256 / TPR rows), the
// next one's loads under way while it works on one; each thread keeps its
// columns' share of dw in registers over all of them.  Bound by memory: 16384 x 8192
// with dH 193 to 196 us, 5.5 TB/s, without 151; 1999 x 5120 with dH 17 to 19 us (256
// workgroups have 7 or 8 rows each: the first row's wait and the parts' join are a
// third of it).
template <int TPR, int NC>
__global__ __launch_bounds__(TPR ? 256 : 1024) void k_rmsnorm_grad(NormGradArgs p) {
  constexpr int TEAMS = TPR ? 256 / (TPR ? TPR : 1) : 1;
  __shared__ __align__(16) float red[2][16];
  row_sum_init<TPR>(red[0]);
  row_sum_init<TPR>(red[1]);
  const int T = row_threads<TPR>();
  const int team = TPR ? threadIdx.x / (TPR ? TPR : 1) : 0;
  const int t = TPR ? threadIdx.x % (TPR ? TPR : 1) : threadIdx.x;
  constexpr bool kAhead = NC == 1;  // wider rows fill the registers as they are
  float dw[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[c][j] = 0.f;
  // w stays in registers, or (NC = 4) comes from the caches for every row; a load
  // in the loop waits for the next row's, which are older
  u32x4 wb[NC];
  auto load_weight = [&](int c) {
    const int col = (c * T + t) * 8;
    wb[c] = u32x4{0u, 0u, 0u, 0u};
    if (col < p.H) wb[c] = *(const u32x4*)(p.w + col);
  };
#pragma unroll
  for (int c = 0; c < NC; ++c) load_weight(c);
  auto weight = [&](int c, float (&w)[8]) {
    if constexpr (NC == 4) load_weight(c);
    widen8(wb[c], w);
  };
  const float invH = 1.f / (float)p.H;
  const int64_t stride = (int64_t)gridDim.x * TEAMS;
  struct Row {
    u32x4 g[NC], h[NC], d[NC];
    float rstd;
  };
  auto load = [&](int64_t row, Row& r) {
    const int64_t base = row * p.H;
    r.rstd = p.rstd[row];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * T + t) * 8;
      r.g[c] = r.h[c] = r.d[c] = u32x4{0u, 0u, 0u, 0u};
      if (col < p.H) {
        r.g[c] = *(const u32x4*)(p.dY + base + col);
        r.h[c] = *(const u32x4*)(p.Hs + base + col);
        if (p.dH) r.d[c] = *(const u32x4*)(p.dH + base + col);
      }
    }
  };
  int flip = 0;
  int64_t row = (int64_t)blockIdx.x * TEAMS + team;
  Row cur;
  if (kAhead && row < p.rows) load(row, cur);
  for (; row < p.rows; row += stride) {
    Row next;  // past the last row: that one again, so that no branch keeps the loads back
    if constexpr (kAhead) load(min(row + stride, p.rows - 1), next);
    else load(row, cur);
    float dot = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float g[8], h[8], w[8];
      widen8(cur.g[c], g);
      widen8(cur.h[c], h);
      weight(c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xhat = h[j] * cur.rstd;
        dot = __builtin_fmaf(g[j] * w[j], xhat, dot);
        dw[c][j] = __builtin_fmaf(g[j], xhat, dw[c][j]);
      }
    }
    dot = row_sum<TPR>(dot, red[flip]) * invH;
    flip ^= 1;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * T + t) * 8;
      if (col >= p.H) continue;
      float g[8], h[8], d[8], w[8];
      widen8(cur.g[c], g);
      widen8(cur.h[c], h);
      widen8(cur.d[c], d);
      weight(c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = __builtin_fmaf(cur.rstd, g[j] * w[j] - h[j] * cur.rstd * dot, d[j]);
      *(u32x4*)(p.dX + row * p.H + col) = narrow8(d);
    }
    if constexpr (kAhead) cur = next;
  }
  if constexpr (TEAMS > 1) {
    __shared__ float sum[TEAMS][TPR * NC * 8];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[team][(c * TPR + t) * 8 + j] = dw[c][j];
    __syncthreads();
    for (int col = threadIdx.x; col < p.H; col += 256) {
      float x = sum[0][col];
      for (int k = 1; k < TEAMS; ++k) x += sum[k][col];
      p.part[(int64_t)blockIdx.x * p.H + col] = x;
    }
  } else {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * T + t) * 8;
      if (col >= p.H) continue;
      floatx4* dst = (floatx4*)(p.part + (int64_t)blockIdx.x * p.H + col);
      dst[0] = floatx4{dw[c][0], dw[c][1], dw[c][2], dw[c][3]};
      dst[1] = floatx4{dw[c][4], dw[c][5], dw[c][6], dw[c][7]};
    }
  }
}

// dw[col] = sum of the n parts in a fixed order.  32 columns a workgroup, so that a
// width of 4096 has 128 of them; 32 runs of lanes each take every 32nd part, 8
// loads at a time (256 parts of 8192 columns: 4.9 us).
__global__ __launch_bounds__(1024) void k_rmsnorm_dw(const float* __restrict__ part, int n, int H,
                                                     float* __restrict__ dw) {
  __shared__ float red[32][33];
  const int l = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + l;
  float s = 0.f;
  if (col < H) {
    for (int i0 = run; i0 < n; i0 += 32 * 8) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = i0 + 32 * u < n ? part[(int64_t)(i0 + 32 * u) * H + col] : 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) s += v[u];
    }
  }
  red[run][l] = s;
  __syncthreads();
  // run r of the workgroup joins column r: lane l has its share l
  float x = red[l][run];
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor(x, o);
  if (l == 0 && blockIdx.x * 32 + run < H) dw[blockIdx.x * 32 + run] = x;
}

}  // namespace

hipError_t launch_rmsnorm_fwd(const uint16_t* X, const uint16_t* R, const uint16_t* w, int64_t M, int H, float eps,
                              uint16_t* Hout, uint16_t* Y, uint8_t* codes, float* scales, float* rstd,
                              hipStream_t st) {
  const int nt = rmsnorm_threads(H), teams = rmsnorm_teams(H);
  const int64_t kb = (H + 127) / 128;
  constexpr int64_t kMost = (int64_t)1 << 21;  // workgroups a launch: its work-items stay below 2^32
  for (int64_t r0 = 0; r0 < M; r0 += kMost * teams) {
    NormArgs a{X + r0 * H, R ? R + r0 * H : nullptr, w, std::min(kMost * teams, M - r0), H, 1. / H, eps,
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
  const int nt = rmsnorm_threads(H);
  const int parts = rmsnorm_parts(M, H);
  NormGradArgs a{dY, Hs, w, rstd, dH, M, H, dX, part};
  const dim3 gr((unsigned)parts), bl(nt);
#define NF4K_CALL(T, N) hipLaunchKernelGGL((k_rmsnorm_grad<T, N>), gr, bl, 0, st, a)
  NF4K_NORM_SHAPES(NF4K_CALL);
#undef NF4K_CALL
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_rmsnorm_dw, dim3((unsigned)((H + 31) / 32)), dim3(1024), 0, st, part, parts, H, dw);
  return hipGetLastError();
}

}  // namespace nf4k
