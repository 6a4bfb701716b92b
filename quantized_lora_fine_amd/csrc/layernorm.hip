// Layer norm with the residual's addition, an 8-bit output, and its gradient (gfx950).
//
// Forward, per row of width H:
//     h = bf16(x + res)  (h = x without a residual),
//     mean = sum(h) / H,   rstd = 1 / sqrt(sum((h - mean)^2) / H + eps),
//     y = (h - mean) * rstd * w + b;
// y is computed in fp64 and rounded once to fp32, from where it is narrowed to bf16,
// to 8-bit codes with a scale per 128 columns, or both.  The two sums are fp64: the
// row stays in registers, so the second pass over it moves no byte, and a row far from
// zero loses nothing to the difference of two large sums.
// Gradient, with xhat = (h - mean) * rstd and u = dy * w:
//     dx = rstd * (u - mean(u) - xhat * mean(u * xhat)) + dh,
//     dw = sum over rows dy * xhat,   db = sum over rows dy.
// The gradient's sums are fp32.
//
// Both go once over their rows and are bound by memory: 16384 rows of 8192 with a residual
// and both outputs (1.21 GB) 220 us, 5.5 TB/s, the copy's rate in spite of the fp64
// arithmetic; the gradient with dh (1.07 GB) 191 us, 5.6 TB/s, and 5 for the joining of dw
// and db.  1999 rows of 5120: 16.8 and 4.  One row: 3.0.
#include <algorithm>

#include "norm.hpp"

namespace nf4k {

namespace {

struct LayerNormArgs {
  const uint16_t* X;
  const uint16_t* R;  // residual, or NULL
  const uint16_t* w;
  const uint16_t* b;  // or NULL
  int64_t rows;
  int H;
  double inv_H;
  float eps;
  uint16_t* Hout;  // with a residual
  uint16_t* Y;     // or NULL
  uint8_t* codes;  // or NULL
  float* scales;
  float* mean;  // or NULL
  float* rstd;  // or NULL
};

// How a row is held is the root-mean-square norm's (norm.hpp).
template <int TPR, int NC>
__global__ __launch_bounds__(TPR ? 256 : 1024) void k_layernorm(LayerNormArgs p) {
  __shared__ __align__(16) double red[2][16];
  row_sum_init<TPR>(red[0]);
  row_sum_init<TPR>(red[1]);
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
  double s = 0;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float a[8];
    widen8(hb[c], a);
#pragma unroll
    for (int j = 0; j < 8; ++j) s += (double)a[j];
  }
  s = row_sum<TPR>(s, red[0]);
  // the quotient rounded once: a row of equal values has exactly their mean
  double mean = s * p.inv_H;
  mean = __builtin_fma(__builtin_fma(-mean, (double)p.H, s), p.inv_H, mean);
  double ss = 0;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float a[8];
    widen8(hb[c], a);
    if ((c * T + t) * 8 < p.H) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double d = (double)a[j] - mean;
        ss = __builtin_fma(d, d, ss);
      }
    }
  }
  ss = row_sum<TPR>(ss, red[1]);
  // One step of Newton's from the fp32 root of var / 4^k, which is 1/4 or more and below
  // 1, so no magnitude is out of range; 2^-45 from the root.  var = 0 (a constant row and
  // eps = 0) gives a NaN.
  double var = __builtin_fma(ss, p.inv_H, (double)p.eps);
  const int k = (__builtin_amdgcn_frexp_exp(var) + 1) >> 1;
  var = __builtin_amdgcn_ldexp(var, -2 * k);
  double rstd = (double)__builtin_amdgcn_rsqf((float)var);
  const double e = __builtin_fma(-var * rstd, rstd, 1.);
  rstd = __builtin_amdgcn_ldexp(__builtin_fma(0.5 * rstd, e, rstd), -k);
  if (t == 0) {
    if (p.mean) p.mean[row] = (float)mean;
    if (p.rstd) p.rstd[row] = (float)rstd;
  }
  const int64_t kb = (p.H + 127) / 128;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int col = (c * T + t) * 8;
    const bool in = col < p.H;
    float a[8], w[8], b[8];
    widen8(hb[c], a);
    u32x4 wb = {0u, 0u, 0u, 0u}, bb = {0u, 0u, 0u, 0u};
    if (in) {
      wb = *(const u32x4*)(p.w + col);
      if (p.b) bb = *(const u32x4*)(p.b + col);
    }
    widen8(wb, w);
    widen8(bb, b);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      a[j] = (float)__builtin_fma(((double)a[j] - mean) * rstd, (double)w[j], (double)b[j]);
    if (p.Y && in) *(u32x4*)(p.Y + base + col) = narrow8(a);
    if (p.codes) {
      const float m = in ? fmaxf(abs_max4(a[0], a[1], a[2], a[3]), abs_max4(a[4], a[5], a[6], a[7])) : 0.f;
      float scale, mul;
      fp8_scale<false>(row16_max(m), scale, mul);
      if (in) {
        uint2 o;
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] *= mul;
        o.x = pack_fp8x4<false>(a[0], a[1], a[2], a[3]);
        o.y = pack_fp8x4<false>(a[4], a[5], a[6], a[7]);
        *(uint2*)(p.codes + base + col) = o;
        if ((t & 15) == 0) p.scales[row * kb + (col >> 7)] = scale;
      }
    }
  }
}

// two sums of a row at once
struct Pair {
  float a, b;
  Pair() = default;
  __device__ __forceinline__ Pair(int) : a(0.f), b(0.f) {}
  __device__ __forceinline__ Pair(float x, float y) : a(x), b(y) {}
  __device__ __forceinline__ Pair operator+(const Pair& o) const { return Pair(a + o.a, b + o.b); }
  __device__ __forceinline__ Pair& operator+=(const Pair& o) {
    a += o.a;
    b += o.b;
    return *this;
  }
};

struct LayerNormGradArgs {
  const uint16_t* dY;
  const uint16_t* Hs;
  const uint16_t* w;
  const float* mean;
  const float* rstd;
  const uint16_t* dH;  // or NULL
  int64_t rows;
  int H;
  uint16_t* dX;
  float* part;   // [gridDim.x][H]: dw's
  float* partb;  // [gridDim.x][H]: db's, or NULL
};

// The layout of the work is the root-mean-square norm's gradient's: a workgroup takes
// every gridDim.x-th row (TPR > 0: group of 256 / TPR rows), the next one's loads under
// way, and each thread keeps its columns' share of dw and db in registers.
template <int TPR, int NC>
__global__ __launch_bounds__(TPR ? 256 : 1024) void k_layernorm_grad(LayerNormGradArgs p) {
  constexpr int TEAMS = TPR ? 256 / (TPR ? TPR : 1) : 1;
  __shared__ __align__(16) Pair red[2][16];
  row_sum_init<TPR>(red[0]);
  row_sum_init<TPR>(red[1]);
  const int T = row_threads<TPR>();
  const int team = TPR ? threadIdx.x / (TPR ? TPR : 1) : 0;
  const int t = TPR ? threadIdx.x % (TPR ? TPR : 1) : threadIdx.x;
  constexpr bool kAhead = NC == 1;  // wider rows fill the registers as they are
  float dw[NC][8], db[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[c][j] = db[c][j] = 0.f;
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
    float mean, rstd;
  };
  auto load = [&](int64_t row, Row& r) {
    const int64_t base = row * p.H;
    r.mean = p.mean[row];
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
    // columns past the row's end have dy = w = 0 and add nothing
    Pair dot(0);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float g[8], h[8], w[8];
      widen8(cur.g[c], g);
      widen8(cur.h[c], h);
      weight(c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xhat = (h[j] - cur.mean) * cur.rstd, u = g[j] * w[j];
        dot.a += u;
        dot.b = __builtin_fmaf(u, xhat, dot.b);
        dw[c][j] = __builtin_fmaf(g[j], xhat, dw[c][j]);
        db[c][j] += g[j];
      }
    }
    dot = row_sum<TPR>(dot, red[flip]);
    flip ^= 1;
    const float m1 = dot.a * invH, m2 = dot.b * invH;
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
      for (int j = 0; j < 8; ++j) {
        const float xhat = (h[j] - cur.mean) * cur.rstd;
        d[j] = __builtin_fmaf(cur.rstd, __builtin_fmaf(g[j], w[j], -m1) - xhat * m2, d[j]);
      }
      *(u32x4*)(p.dX + row * p.H + col) = narrow8(d);
    }
    if constexpr (kAhead) cur = next;
  }
  auto out = [&](float* part, float (&v)[NC][8]) {
    if constexpr (TEAMS > 1) {
      __shared__ float sum[TEAMS][TPR * NC * 8];
      __syncthreads();  // the other output's reads are done
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[team][(c * TPR + t) * 8 + j] = v[c][j];
      __syncthreads();
      for (int col = threadIdx.x; col < p.H; col += 256) {
        float x = sum[0][col];
        for (int k = 1; k < TEAMS; ++k) x += sum[k][col];
        part[(int64_t)blockIdx.x * p.H + col] = x;
      }
    } else {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int col = (c * T + t) * 8;
        if (col >= p.H) continue;
        floatx4* dst = (floatx4*)(part + (int64_t)blockIdx.x * p.H + col);
        dst[0] = floatx4{v[c][0], v[c][1], v[c][2], v[c][3]};
        dst[1] = floatx4{v[c][4], v[c][5], v[c][6], v[c][7]};
      }
    }
  };
  out(p.part, dw);
  if (p.partb) out(p.partb, db);
}

// dw[col] (blockIdx.y = 1: db[col]) = sum of the n parts in a fixed order: 32 columns a
// workgroup, 32 runs of lanes that each take every 32nd part, 8 loads at a time.
__global__ __launch_bounds__(1024) void k_layernorm_join(const float* __restrict__ part,
                                                         const float* __restrict__ partb, int n, int H,
                                                         float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float red[32][33];
  const float* from = blockIdx.y ? partb : part;
  float* to = blockIdx.y ? db : dw;
  const int l = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + l;
  float s = 0.f;
  if (col < H) {
    for (int i0 = run; i0 < n; i0 += 32 * 8) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = i0 + 32 * u < n ? from[(int64_t)(i0 + 32 * u) * H + col] : 0.f;
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
  if (l == 0 && blockIdx.x * 32 + run < H) to[blockIdx.x * 32 + run] = x;
}

}  // namespace

hipError_t launch_layernorm_fwd(const uint16_t* X, const uint16_t* R, const uint16_t* w, const uint16_t* b, int64_t M,
                                int H, float eps, uint16_t* Hout, uint16_t* Y, uint8_t* codes, float* scales,
                                float* mean, float* rstd, hipStream_t st) {
  const int nt = rmsnorm_threads(H), teams = rmsnorm_teams(H);
  const int64_t kb = (H + 127) / 128;
  constexpr int64_t kMost = (int64_t)1 << 21;  // workgroups a launch: its work-items stay below 2^32
  for (int64_t r0 = 0; r0 < M; r0 += kMost * teams) {
    LayerNormArgs a{X + r0 * H, R ? R + r0 * H : nullptr, w, b, std::min(kMost * teams, M - r0), H, 1. / H, eps,
                    Hout ? Hout + r0 * H : nullptr, Y ? Y + r0 * H : nullptr, codes ? codes + r0 * H : nullptr,
                    scales ? scales + r0 * kb : nullptr, mean ? mean + r0 : nullptr, rstd ? rstd + r0 : nullptr};
    const dim3 gr((unsigned)((a.rows + teams - 1) / teams)), bl(nt);
#define NF4K_CALL(T, N) hipLaunchKernelGGL((k_layernorm<T, N>), gr, bl, 0, st, a)
    NF4K_NORM_SHAPES(NF4K_CALL);
#undef NF4K_CALL
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_layernorm_bwd(const uint16_t* dY, const uint16_t* Hs, const uint16_t* w, const float* mean,
                                const float* rstd, const uint16_t* dH, int64_t M, int H, uint16_t* dX, float* dw,
                                float* db, float* part, hipStream_t st) {
  const int nt = rmsnorm_threads(H);
  const int parts = rmsnorm_parts(M, H);
  float* partb = db ? part + (int64_t)parts * H : nullptr;
  LayerNormGradArgs a{dY, Hs, w, mean, rstd, dH, M, H, dX, part, partb};
  const dim3 gr((unsigned)parts), bl(nt);
#define NF4K_CALL(T, N) hipLaunchKernelGGL((k_layernorm_grad<T, N>), gr, bl, 0, st, a)
  NF4K_NORM_SHAPES(NF4K_CALL);
#undef NF4K_CALL
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_layernorm_join, dim3((unsigned)((H + 31) / 32), db ? 2 : 1), dim3(1024), 0, st, part, partb,
                     parts, H, dw, db);
  return hipGetLastError();
}

}  // namespace nf4k
