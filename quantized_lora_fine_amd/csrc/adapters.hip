// Low-rank adapters of many requests beside a shared projection, and their gradients
// (gfx950).
//
// A row m with adapter a has
//     T[m] = X[m] L1[a],            Y[m] = base[m] + s[a] T[m] L2[a],
// and from dY, with G[m] = dY[m] L2[a]^T,
//     dL2[a] = s[a] sum_m T[m]^T dY[m],   dL1[a] = s[a] sum_m X[m]^T G[m],
//     dX[m] = base[m] + s[a] G[m] L1[a]^T.
// Three kinds of product: k_adapters_narrow contracts a row over the layer's width (T,
// G), k_adapters_wide contracts the rank (Y, dX), k_adapters_grad contracts the rows of an
// adapter (dL1, dL2).  All run on v_mfma_f32_16x16x32_bf16.  X, dY, L1 and L2 are bf16 as
// they are; T and G are fp32 and enter a product as a sum of bf16 values: two where the
// result is bf16 (they leave 2^-17 of a value), three where it is fp32 (which leave nothing
// of its 24 bits; two would leave 2e-6 of a sum, ten times an fp32 sum's own error).  That
// is MFMAs in products that are bound by memory.  8-bit codes are bf16 values exactly, and
// their scale, one for a row and 128 columns, goes to that row of G.
//
// Rows are named by (order, offsets): adapter a's are order[offsets[a]] to
// order[offsets[a + 1] - 1] (without an order: the rows of these numbers).  A workgroup takes
// a tile of one adapter's rows and finds it from the offsets by itself, so nothing waits
// for the host.  Whatever the offsets and the order hold, no row outside the buffers is
// touched.
#include <algorithm>

#include "fp8.hpp"
#include "launch.hpp"

namespace nf4k {

namespace {

constexpr int kAhead = 2;  // steps of 32 columns whose loads are under way in k_adapters_narrow

// Tile t of `bm` rows: its adapter, positions [p0, p1), and whether they are all of the
// adapter's.  Every wave scans the tile counts of 64 adapters at a time.
struct Tile {
  int a;
  int p0, p1;
  bool whole;
};
__device__ __forceinline__ bool find_tile(const AdapterRows& R, int bm, uint32_t t, Tile& tile) {
  const int lane = threadIdx.x & 63;
  const int M = (int)R.M;
  uint32_t base = 0;  // (counts may wrap where offsets do not ascend; the rows stay inside all the same)
  for (int a0 = 0; a0 < R.n; a0 += 64) {
    const int i = a0 + lane;
    int lo = 0, cnt = 0;
    if (i < R.n) {
      lo = min(max(R.offsets[i], 0), M);
      cnt = max(min(max(R.offsets[i + 1], 0), M) - lo, 0);  // lo + cnt <= M
    }
    const uint32_t tiles = (uint32_t)(((int64_t)cnt + bm - 1) / bm);
    uint32_t incl = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t v = __shfl_up(incl, o);
      if (lane >= o) incl += v;
    }
    const uint64_t hit = __ballot(base + incl > t);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      const uint32_t first = base + (uint32_t)__builtin_amdgcn_readlane((int)(incl - tiles), l);
      const int l0 = __builtin_amdgcn_readlane(lo, l), ln = __builtin_amdgcn_readlane(cnt, l);
      const int64_t p0 = (int64_t)l0 + (int64_t)(t - first) * bm;
      tile.a = a0 + l;
      tile.p0 = (int)min(p0, (int64_t)l0 + ln);
      tile.p1 = (int)min(p0 + bm, (int64_t)l0 + ln);
      tile.whole = ln <= bm;
      return tile.p0 < tile.p1;
    }
    base += (uint32_t)__builtin_amdgcn_readlane((int)incl, 63);
  }
  return false;
}

// the row at a position of the tile, -1 past its end and where the order holds none
__device__ __forceinline__ int64_t row_at(const AdapterRows& R, const Tile& t, int p) {
  if (p >= t.p1) return -1;
  const int64_t row = R.order ? (int64_t)R.order[p] : p;
  return (uint64_t)row < (uint64_t)R.M ? row : -1;
}

// Four neighbouring fp32 values as W bf16 ones each, from the largest on; one that is no
// number stands in the first alone.
template <int W>
__device__ __forceinline__ void split4(floatx4 x, uint2 (&part)[W]) {
#pragma unroll
  for (int w = 0; w < W; ++w) {
    part[w] = uint2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
    if (w + 1 == W) break;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t word = i < 2 ? part[w].x : part[w].y;
      const float h = __builtin_bit_cast(float, i & 1 ? word & 0xFFFF0000u : word << 16);
      x[i] = fabsf(h) < INFINITY ? x[i] - h : 0.f;
    }
  }
}

// ---------------------------------------------------------------------------
// part[split][m][j] = sum over the split's k of A[m][k] L[a][k][j] (KMAJOR: L1
// [n][K][r]) or A[m][k] L[a][j][k] (L2 [n][r][K]).  A workgroup has 16 NM rows,
// 16 NJ columns of the rank (blockIdx.z: which 64) and a range of k (blockIdx.y).  Its 4
// waves take every fourth step of 32 k, kAhead steps' loads under way, and their sums are
// added in LDS in wave order.  A's rows are the MFMA's second operand, so a lane ends with
// 4 neighbouring columns of one row; a row or column past the end repeats a valid one and
// is not written.  L1 goes through LDS for transposing reads, each wave's own part.
// ---------------------------------------------------------------------------
template <bool KMAJOR, int NJ, int NM>
__global__ __launch_bounds__(256) void k_adapters_narrow(AdapterNarrow p) {
  constexpr int RP = 16 * NJ, BM = 16 * NM;
  constexpr int ROW = RP * 2 + (NJ == 1 ? 0 : 16);                      // LDS bytes of a k row of L1
  constexpr int STAGE = KMAJOR ? 32 * ROW * kAhead : 0;                 // a wave's
  constexpr int SMEM = 4 * STAGE > 4 * BM * RP * 4 ? 4 * STAGE : 4 * BM * RP * 4;
  __shared__ __align__(16) uint8_t smem[SMEM];
  Tile tile;
  if (!find_tile(p.rows, BM, blockIdx.x, tile)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, g = lane >> 4;
  const int j0 = blockIdx.z * 64;
  const int64_t K = p.K;
  const int64_t k0 = (int64_t)blockIdx.y * p.krange, k1 = min(k0 + p.krange, K);
  const uint16_t* arow[NM];
#pragma unroll
  for (int i = 0; i < NM; ++i) {
    const int64_t row = row_at(p.rows, tile, tile.p0 + 16 * i + li);
    arow[i] = p.A + max(row, (int64_t)0) * K + 8 * g;
  }
  const uint16_t* L = p.L + (int64_t)tile.a * K * p.r;
  uint8_t* stage = smem + wave * STAGE;
  floatx4 acc[NJ][NM];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int i = 0; i < NM; ++i) acc[j][i] = floatx4{0.f, 0.f, 0.f, 0.f};
  constexpr u32x4 kZero = {0u, 0u, 0u, 0u};
  // L1's pieces of 8 columns: 2 NJ a k row
  constexpr int PPR = 2 * NJ, KPL = 64 / PPR, NL = 32 / KPL;
  for (int64_t s0 = k0 + 32 * wave; s0 < k1; s0 += 128 * kAhead) {
    u32x4 x[kAhead][NM], l[kAhead][KMAJOR ? NL : NJ];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t k = s0 + 128 * u;
      const bool in = k + 8 * g < k1;
#pragma unroll
      for (int i = 0; i < NM; ++i) x[u][i] = in ? *(const u32x4*)(arow[i] + k) : kZero;
      if constexpr (KMAJOR) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
          const int64_t kr = k + KPL * i + lane / PPR;
          const int j = j0 + 8 * (lane % PPR);
          l[u][i] = kr < k1 && j < p.r ? *(const u32x4*)(L + kr * p.r + j) : kZero;
        }
      } else {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          l[u][j] = in ? *(const u32x4*)(L + (int64_t)min(j0 + 16 * j + li, p.r - 1) * K + k + 8 * g) : kZero;
      }
    }
    if constexpr (KMAJOR) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int i = 0; i < NL; ++i)
          *(u32x4*)(stage + (32 * u + KPL * i + lane / PPR) * ROW + 16 * (lane % PPR)) = l[u][i];
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        bf16x8 f;
        if constexpr (KMAJOR)
          f = lds_tr8(stage + (32 * u + 8 * g + (li >> 2)) * ROW + 2 * (16 * j + 4 * (li & 3)), ROW);
        else f = __builtin_bit_cast(bf16x8, l[u][j]);
#pragma unroll
        for (int i = 0; i < NM; ++i)
          acc[j][i] =
              __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, __builtin_bit_cast(bf16x8, x[u][i]), acc[j][i], 0, 0, 0);
      }
    }
  }
  __syncthreads();
  float* red = (float*)smem;  // [4][BM][RP]
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int i = 0; i < NM; ++i) *(floatx4*)(red + (wave * BM + 16 * i + li) * RP + 16 * j + 4 * g) = acc[j][i];
  __syncthreads();
  for (int e = threadIdx.x; e < BM * RP / 4; e += 256) {
    const int m = e / (RP / 4), j = 4 * (e % (RP / 4));
    const int64_t row = row_at(p.rows, tile, tile.p0 + m);
    if (row < 0 || j0 + j >= p.r) continue;
    floatx4 s = *(const floatx4*)(red + m * RP + j);
#pragma unroll
    for (int w = 1; w < 4; ++w) s += *(const floatx4*)(red + (w * BM + m) * RP + j);
    *(floatx4*)(p.part + ((int64_t)blockIdx.y * p.rows.M + row) * p.r + j0 + j) = s;
  }
}

// sum of a value's splits, in their order
__device__ __forceinline__ floatx4 join4(const float* part, int64_t stride, int splits) {
  floatx4 s = *(const floatx4*)part;
  for (int q = 1; q < splits; ++q) s += *(const floatx4*)(part + q * stride);
  return s;
}

// ---------------------------------------------------------------------------
// out[m][c] = bf16(base[m][c] + s[a] sum_j P[m][j] L[a][j][c]) (JMAJOR: L2 [n][r][N])
// or with L[a][c][j] (L1 [n][N][r]).  A workgroup has 16 NM rows and 256 columns, 64 a
// wave.  P (its splits joined) is split into hi and lo in LDS, 16 of the rank a step: the
// MFMA's 32 products are hi's 16 and lo's, against the same 16 of L.  L is the first
// operand with its columns so dealt that a lane ends with 16 neighbouring ones of a row.
// ---------------------------------------------------------------------------
template <bool JMAJOR, int NM, int RMAX>
__global__ __launch_bounds__(256) void k_adapters_wide(AdapterWide p) {
  constexpr int BM = 16 * NM;
  constexpr int LROW = 64 * 2 + 16;  // LDS bytes of a rank row of L2: 64 columns
  __shared__ __align__(16) uint8_t smem[BM * (RMAX * 4 + 16) + (JMAJOR ? 4 * 16 * LROW : 0)];
  Tile tile;
  if (!find_tile(p.rows, BM, blockIdx.x, tile)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, g = lane >> 4;
  const int r = p.r, r16 = (r + 15) / 16 * 16;
  const int64_t N = p.N;
  const int prow = r16 * 4 + 16;  // LDS bytes of a row of P: for each 16 of the rank hi, then lo
  for (int e = threadIdx.x; e < BM * r16 / 4; e += 256) {
    const int m = e / (r16 / 4), j = 4 * (e % (r16 / 4));
    const int64_t row = row_at(p.rows, tile, tile.p0 + m);
    floatx4 v = {0.f, 0.f, 0.f, 0.f};
    if (row >= 0 && j < r) {
      v = join4(p.part + row * r + j, p.rows.M * r, p.splits);
      if (p.T_out && blockIdx.y == 0) *(floatx4*)(p.T_out + row * r + j) = v;
    }
    uint2 part[2];
    split4(v, part);
    uint8_t* to = smem + m * prow + (j / 16) * 64 + (j % 16) * 2;
    *(uint2*)to = part[0];
    *(uint2*)(to + 32) = part[1];
  }
  __syncthreads();
  const int64_t c0 = (int64_t)blockIdx.y * 256 + 64 * wave;
  if (c0 >= N) return;
  uint8_t* stage = smem + BM * prow + wave * 16 * LROW;
  const int64_t c = c0 + 16 * g;  // this lane's 16 columns of the result
  int64_t at[NM];
  u32x4 b[NM][2];
#pragma unroll
  for (int i = 0; i < NM; ++i) {
    const int64_t row = row_at(p.rows, tile, tile.p0 + 16 * i + li);
    at[i] = row < 0 || c >= N ? -1 : row * N + c;
    b[i][0] = b[i][1] = u32x4{0u, 0u, 0u, 0u};
    if (p.base && at[i] >= 0) {
      b[i][0] = *(const u32x4*)(p.base + at[i]);
      b[i][1] = *(const u32x4*)(p.base + at[i] + 8);
    }
  }
  const uint16_t* L = p.L + (int64_t)tile.a * N * r;
  floatx4 acc[4][NM];
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int i = 0; i < NM; ++i) acc[q][i] = floatx4{0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < r16; j0 += 16) {
    bf16x8 f[4];
    if constexpr (JMAJOR) {
      u32x4 v[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = j0 + 8 * i + lane / 8;
        const int64_t cc = c0 + 8 * (lane % 8);
        v[i] = j < r && cc < N ? *(const u32x4*)(L + j * N + cc) : u32x4{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) *(u32x4*)(stage + (8 * i + lane / 8) * LROW + 16 * (lane % 8)) = v[i];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        f[q] = lds_tr8(stage + (8 * (g & 1) + (li >> 2)) * LROW + 2 * (16 * (li & 3) + 4 * q), LROW);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t cc = min(c0 + 16 * (li >> 2) + 4 * q + (li & 3), N - 1);
        const int j = j0 + 8 * (g & 1);
        f[q] = __builtin_bit_cast(bf16x8, j < r ? *(const u32x4*)(L + cc * r + j) : u32x4{0u, 0u, 0u, 0u});
      }
    }
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      const bf16x8 t = *(const bf16x8*)(smem + (16 * i + li) * prow + (j0 / 16) * 64 + (g >> 1) * 32 + (g & 1) * 16);
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[q][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[q], t, acc[q][i], 0, 0, 0);
    }
  }
  const float s = p.s[tile.a];
#pragma unroll
  for (int i = 0; i < NM; ++i) {
    if (at[i] < 0) continue;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      u32x4 o;
#pragma unroll
      for (int w = 0; w < 4; ++w) {  // columns 8 hf + 2 w and the next, from acc[2 hf + w / 2]
        const floatx4 v = acc[2 * hf + w / 2][i];
        const float lo = __builtin_fmaf(s, v[2 * (w & 1)], __builtin_bit_cast(float, b[i][hf][w] << 16));
        const float up = __builtin_fmaf(s, v[2 * (w & 1) + 1], __builtin_bit_cast(float, b[i][hf][w] & 0xFFFF0000u));
        o[w] = pack_bf16x2(lo, up);
      }
      *(u32x4*)(p.out + at[i] + 8 * hf) = o;
    }
  }
}

// ---------------------------------------------------------------------------
// dL[a][j][c] (or [c][j]) = s[a] sum over a's rows of P[m][j] Q[m][c]: a workgroup has
// 128 columns of Q, 16 NJ of the rank (blockIdx.z: which 64) and up to p.item rows of an
// adapter, 64 at a time through LDS, the next 64 under way in registers.  Rows past the
// tile are zero in both.  An adapter whose rows are all here is written out, otherwise the
// item's sums go to a part of their own, which k_adapters_join adds in order.  Q in 8 bits
// (X8 1: e4m3, 2: e5m2) becomes bf16 on its way into LDS, and P is multiplied by the scale
// of its row and this block of 128 columns.
// ---------------------------------------------------------------------------
template <int X8, int NJ>
__device__ __forceinline__ void grad_tile(const AdapterRows& rows, const AdapterGrad& p, uint8_t* smem) {
  constexpr int KR = 64, RP = 16 * NJ;
  constexpr int QROW = 128 * 2 + 16, PROW = RP * 2 + 16;
  constexpr int JW = NJ == 4 ? 2 : 1, CW = 4 / JW;      // waves over the rank and over the columns
  constexpr int FJ = NJ / JW, FC = 8 / CW;              // a wave's fragments
  constexpr int QL = X8 ? 2 : 4;                        // 16-byte loads of Q a thread
  constexpr int PL = (KR * RP / 4 + 255) / 256;         // 4-value pieces of P a thread
  uint8_t* qs = smem;
  uint8_t* ps = smem + KR * QROW;  // [3][KR] rows
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, li = lane & 15, g = lane >> 4;
  Tile tile;
  if (!find_tile(rows, p.item, blockIdx.x, tile)) return;
  const int64_t N = p.N, c0 = (int64_t)blockIdx.y * 128;
  const int r = p.r, j0 = blockIdx.z * 64;
  const int64_t kb = (N + 127) / 128;
  u32x4 q[QL];
  floatx4 v[PL];
  constexpr int CP = X8 ? 8 : 16;  // pieces of a row
  auto load = [&](int p0) {
#pragma unroll
    for (int i = 0; i < QL; ++i) {
      const int e = 256 * i + tid;
      const int64_t row = row_at(rows, tile, p0 + e / CP);
      const int64_t c = c0 + (e % CP) * (128 / CP);
      q[i] = u32x4{0u, 0u, 0u, 0u};
      if (row >= 0 && c < N) q[i] = *(const u32x4*)((const uint8_t*)p.Q + (row * N + c) * (X8 ? 1 : 2));
    }
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = 256 * i + tid, m = e / (RP / 4), j = j0 + 4 * (e % (RP / 4));
      v[i] = floatx4{0.f, 0.f, 0.f, 0.f};
      if (m >= KR) continue;
      const int64_t row = row_at(rows, tile, p0 + m);
      if (row < 0 || j >= r) continue;
      v[i] = join4(p.P + row * r + j, rows.M * r, p.splits);
      if (X8) v[i] *= p.q_scales[row * kb + blockIdx.y];
    }
  };
  auto store = [&]() {
#pragma unroll
    for (int i = 0; i < QL; ++i) {
      const int e = 256 * i + tid;
      uint8_t* to = qs + (e / CP) * QROW + (e % CP) * (256 / CP);
      if constexpr (X8 == 0) {
        *(u32x4*)to = q[i];
      } else {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float a[4], b[4];
          unpack_fp8x4<X8 == 2>(q[i][2 * hf], a);
          unpack_fp8x4<X8 == 2>(q[i][2 * hf + 1], b);
          *(u32x4*)(to + 16 * hf) = u32x4{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(b[0], b[1]),
                                          pack_bf16x2(b[2], b[3])};
        }
      }
    }
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = 256 * i + tid, m = e / (RP / 4), j = 4 * (e % (RP / 4));
      if (m >= KR) continue;
      uint2 part[3];
      split4(v[i], part);
#pragma unroll
      for (int w = 0; w < 3; ++w) *(uint2*)(ps + (w * KR + m) * PROW + 2 * j) = part[w];
    }
  };
  const int wj = wave / CW, wc = wave % CW;
  floatx4 acc[FJ][FC];
#pragma unroll
  for (int j = 0; j < FJ; ++j)
#pragma unroll
    for (int c = 0; c < FC; ++c) acc[j][c] = floatx4{0.f, 0.f, 0.f, 0.f};
  load(tile.p0);
  for (int p0 = tile.p0; p0 < tile.p1; p0 += KR) {
    __syncthreads();
    store();
    if (p0 + KR < tile.p1) load(p0 + KR);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KR; k += 32) {
      const int tr = k + 8 * g + (li >> 2), tc = 4 * (li & 3);
      bf16x8 fp[FJ][3];
#pragma unroll
      for (int j = 0; j < FJ; ++j)
#pragma unroll
        for (int w = 0; w < 3; ++w)
          fp[j][w] = lds_tr8(ps + (w * KR + tr) * PROW + 2 * (16 * (wj * FJ + j) + tc), PROW);
#pragma unroll
      for (int c = 0; c < FC; ++c) {
        const bf16x8 fq = lds_tr8(qs + tr * QROW + 2 * (16 * (wc * FC + c) + tc), QROW);
#pragma unroll
        for (int w = 2; w >= 0; --w)
#pragma unroll
          for (int j = 0; j < FJ; ++j)
            acc[j][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp[j][w], fq, acc[j][c], 0, 0, 0);
      }
    }
  }
  const float s = tile.whole ? p.s[tile.a] : 1.f;
  float* out = tile.whole ? p.out + (int64_t)tile.a * r * N : p.part + (int64_t)blockIdx.x * r * N;
#pragma unroll
  for (int j = 0; j < FJ; ++j)
#pragma unroll
    for (int c = 0; c < FC; ++c) {
      const int jj = j0 + 16 * (wj * FJ + j) + 4 * g;
      const int64_t cc = c0 + 16 * (wc * FC + c) + li;
      if (jj >= r || cc >= N) continue;  // r % 4 == 0
      const floatx4 o = acc[j][c] * s;
      if (p.trans) {
        *(floatx4*)(out + cc * r + jj) = o;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) out[(jj + i) * N + cc] = o[i];
      }
    }
}

template <int X8, int NJ>
__global__ __launch_bounds__(256) void k_adapters_grad(AdapterRows rows, AdapterGrad p) {
  constexpr int SMEM = 64 * (128 * 2 + 16) + 3 * 64 * (16 * NJ * 2 + 16);
  __shared__ __align__(16) uint8_t smem[SMEM];
  grad_tile<X8, NJ>(rows, p, smem);
}

// Outputs of adapters with several items: their parts' sums in order; with none: zeros.
__global__ __launch_bounds__(256) void k_adapters_join(AdapterRows rows, AdapterGrad p0, AdapterGrad p1) {
  const AdapterGrad& p = blockIdx.z ? p1 : p0;
  const int a = blockIdx.y, lane = threadIdx.x & 63;
  const int M = (int)rows.M;
  // items before a's, and a's own
  uint32_t first = 0, own = 0;
  for (int a0 = 0; a0 <= a; a0 += 64) {
    const int i = a0 + lane;
    uint32_t items = 0;
    if (i <= a) {
      const int lo = min(max(rows.offsets[i], 0), M);
      const int cnt = max(min(max(rows.offsets[i + 1], 0), M) - lo, 0);
      items = (uint32_t)(((int64_t)cnt + p.item - 1) / p.item);
    }
    const uint64_t me = __ballot(i == a);
    if (me) own = (uint32_t)__builtin_amdgcn_readlane((int)items, __builtin_ctzll(me));
    uint32_t sum = i < a ? items : 0;
#pragma unroll
    for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
    first += sum;
  }
  if (own == 1) return;
  const int64_t size = (int64_t)p.r * p.N;
  const float s = p.s[a];
  // items past the launch (offsets that do not ascend) have no part
  const uint32_t end = min(first + own, (uint32_t)p.items);
  for (int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; e < size; e += (int64_t)gridDim.x * 1024) {
    floatx4 v = {0.f, 0.f, 0.f, 0.f};
    for (uint32_t i = first; i < end; ++i) v += *(const floatx4*)(p.part + i * size + e);
    *(floatx4*)(p.out + a * size + e) = own ? v * s : v;
  }
}

template <bool KMAJOR, int NM>
hipError_t narrow_of(const AdapterNarrow& p, dim3 gr, hipStream_t st) {
  if (p.r <= 16) hipLaunchKernelGGL((k_adapters_narrow<KMAJOR, 1, NM>), gr, dim3(256), 0, st, p);
  else if (p.r <= 32) hipLaunchKernelGGL((k_adapters_narrow<KMAJOR, 2, NM>), gr, dim3(256), 0, st, p);
  else hipLaunchKernelGGL((k_adapters_narrow<KMAJOR, 4, NM>), gr, dim3(256), 0, st, p);
  return hipGetLastError();
}

hipError_t narrow(const AdapterCall& c, const AdapterPlan& pl, const uint16_t* A, int64_t K, const uint16_t* L,
                  bool kmajor, float* part, hipStream_t st) {
  AdapterNarrow p{c.rows, A, L, K, c.r, pl.krange, part};
  const dim3 gr((unsigned)pl.tiles, (unsigned)pl.splits, (unsigned)((c.r + 63) / 64));
  if (pl.bm == 16) return kmajor ? narrow_of<true, 1>(p, gr, st) : narrow_of<false, 1>(p, gr, st);
  return kmajor ? narrow_of<true, 4>(p, gr, st) : narrow_of<false, 4>(p, gr, st);
}

template <bool JMAJOR, int NM>
hipError_t wide_of(const AdapterWide& p, dim3 gr, hipStream_t st) {
  if (p.r <= 64) hipLaunchKernelGGL((k_adapters_wide<JMAJOR, NM, 64>), gr, dim3(256), 0, st, p);
  else hipLaunchKernelGGL((k_adapters_wide<JMAJOR, NM, 256>), gr, dim3(256), 0, st, p);
  return hipGetLastError();
}

hipError_t wide(const AdapterCall& c, const AdapterPlan& pl, const float* part, const uint16_t* L, bool jmajor,
                int64_t N, const uint16_t* base, uint16_t* out, float* T_out, hipStream_t st) {
  AdapterWide p{c.rows, part, pl.splits, L, N, c.r, c.s, base, out, T_out};
  const dim3 gr((unsigned)pl.tiles, (unsigned)((N + 255) / 256));
  if (pl.bm == 16) return jmajor ? wide_of<true, 1>(p, gr, st) : wide_of<false, 1>(p, gr, st);
  return jmajor ? wide_of<true, 4>(p, gr, st) : wide_of<false, 4>(p, gr, st);
}

template <int X8>
hipError_t grad_of(const AdapterRows& rows, const AdapterGrad& p, hipStream_t st) {
  const dim3 gr((unsigned)p.items, (unsigned)((p.N + 127) / 128), (unsigned)((p.r + 63) / 64));
  if (p.r <= 16) hipLaunchKernelGGL((k_adapters_grad<X8, 1>), gr, dim3(256), 0, st, rows, p);
  else if (p.r <= 32) hipLaunchKernelGGL((k_adapters_grad<X8, 2>), gr, dim3(256), 0, st, rows, p);
  else hipLaunchKernelGGL((k_adapters_grad<X8, 4>), gr, dim3(256), 0, st, rows, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adapters_fwd(const AdapterCall& c, const uint16_t* X, const uint16_t* base, uint16_t* Y, float* T_out,
                               void* ws, hipStream_t st) {
  const AdapterPlan pl = plan_adapters_rows(c.rows.M, c.rows.n, c.h);
  hipError_t e = narrow(c, pl, X, c.h, c.L1, true, (float*)ws, st);
  if (e != hipSuccess) return e;
  return wide(c, pl, (const float*)ws, c.L2, true, c.o, base, Y, T_out, st);
}

hipError_t launch_adapters_bwd(const AdapterCall& c, const void* X, int x8, const float* x_scales, const uint16_t* dY,
                               const float* T, const uint16_t* base, uint16_t* dX, float* dL1, float* dL2, void* ws,
                               hipStream_t st) {
  const AdapterPlan pl = plan_adapters_rows(c.rows.M, c.rows.n, c.o);
  const AdapterItems it = plan_adapters_items(c.rows.M, c.rows.n, c.h, c.o, c.r);
  float* G = (float*)ws;
  float* parts = G + pl.splits * c.rows.M * c.r;
  hipError_t e = narrow(c, pl, dY, c.o, c.L2, false, G, st);
  if (e != hipSuccess) return e;
  const AdapterGrad g1{X, x_scales, c.h, G, pl.splits, c.r, c.s, it.item, it.items, 1, parts, dL1};
  const AdapterGrad g2{dY, nullptr, c.o, T, 1, c.r, c.s, it.item, it.items, 0, parts + it.items * c.r * c.h, dL2};
  e = x8 == 0 ? grad_of<0>(c.rows, g1, st) : x8 == 1 ? grad_of<1>(c.rows, g1, st) : grad_of<2>(c.rows, g1, st);
  if (e != hipSuccess) return e;
  e = grad_of<0>(c.rows, g2, st);
  if (e != hipSuccess) return e;
  const int64_t most = std::max(c.h, c.o) * c.r;
  const dim3 gr((unsigned)std::min<int64_t>((most + 1023) / 1024, 1024), (unsigned)c.rows.n, 2);
  hipLaunchKernelGGL(k_adapters_join, gr, dim3(256), 0, st, c.rows, g1, g2);
  e = hipGetLastError();
  if (e != hipSuccess || !dX) return e;
  return wide(c, pl, G, c.L1, false, c.h, base, dX, nullptr, st);
}

}  // namespace nf4k
