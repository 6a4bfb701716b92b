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
// of its 24 bits; two would leave 2e-6 of a sum, ten times an fp32 sum's own error).  The
// matrix cores have room for it: three parts at rank 64 are their highest load, 32 % of the
// cycles.  8-bit codes are bf16 values exactly, and their scale, one for a row and 128
// columns, goes to that row of G, whose product with it is rounded to fp32 once.
//
// All of it is bound by memory where there are many rows (X and dY are read, base and Y or dX
// read and written), by launches and latencies that follow one another where there are few.
// Times below are of one MI355X by kernel trace; a large copy there reaches 5.4 TB/s.
//
// Rows are named by (order, offsets): adapter a's are order[offsets[a]] to
// order[offsets[a + 1] - 1] (without an order: the rows of these numbers).  A workgroup takes
// a tile of one adapter's rows and finds it from the offsets by itself, so nothing waits
// for the host.  Whatever the offsets and the order hold, no row outside the buffers is
// touched.
#include <algorithm>
#include <type_traits>

#include "fp8.hpp"
#include "launch.hpp"

namespace nf4k {

namespace {

// Tile t of `bm` rows: its adapter, positions [p0, p1), whether they are all of the adapter's,
// and, where they are not, its number among the tiles of adapters that have several.  Every wave
// scans the tile counts of 64 adapters at a time.
struct Tile {
  int a;
  int p0, p1;
  bool whole;
  uint32_t part;
};
__device__ __forceinline__ bool find_tile(const AdapterRows& R, int bm, uint32_t t, Tile& tile) {
  const int lane = threadIdx.x & 63;
  const int M = (int)R.M;
  uint32_t base = 0;  // (counts may wrap where offsets do not ascend; the rows stay inside all the same)
  uint32_t alone = 0;  // tiles that are all of their adapter's
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
    const uint64_t hit = __ballot(base + incl > t), single = __ballot(tiles == 1);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      const uint32_t first = base + (uint32_t)__builtin_amdgcn_readlane((int)(incl - tiles), l);
      const int l0 = __builtin_amdgcn_readlane(lo, l), ln = __builtin_amdgcn_readlane(cnt, l);
      const int64_t p0 = (int64_t)l0 + (int64_t)(t - first) * bm;
      tile.a = a0 + l;
      tile.p0 = (int)min(p0, (int64_t)l0 + ln);
      tile.p1 = (int)min(p0 + bm, (int64_t)l0 + ln);
      tile.whole = ln <= bm;
      tile.part = t - alone - (uint32_t)__popcll(single & (((uint64_t)1 << l) - 1));
      return tile.p0 < tile.p1;
    }
    base += (uint32_t)__builtin_amdgcn_readlane((int)incl, 63);
    alone += (uint32_t)__popcll(single);
  }
  return false;
}

// the row at a position of the tile, -1 past its end and where the order holds none
__device__ __forceinline__ int64_t row_at(const AdapterRows& R, const Tile& t, int p) {
  if (p >= t.p1) return -1;
  const int64_t row = R.order ? (int64_t)R.order[p] : p;
  return (uint64_t)row < (uint64_t)R.M ? row : -1;
}

// Four neighbouring fp32 values as two bf16 ones each.  The first is at most the largest bf16
// value, which fp32's last ones would round past to an infinity; what lies beyond stands in the
// second, and so does an infinity or a NaN.
__device__ __forceinline__ void split4(floatx4 x, uint2 (&part)[2]) {
  constexpr float kTop = 0x1.FEp127f;
  float c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = __builtin_amdgcn_fmed3f(x[i], -kTop, kTop);
  part[0] = uint2{pack_bf16x2(c[0], c[1]), pack_bf16x2(c[2], c[3])};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t word = i < 2 ? part[0].x : part[0].y;
    x[i] -= __builtin_bit_cast(float, i & 1 ? word & 0xFFFF0000u : word << 16);
  }
  part[1] = uint2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
}

// As three bf16 ones each, whose sum they are: 8 bits at a time are cut off the top, and what
// is left has 16 and then 8.  (An infinity leaves a NaN.)
__device__ __forceinline__ void split4(floatx4 x, uint2 (&part)[3]) {
#pragma unroll
  for (int w = 0; w < 3; ++w) {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v = x[i];
      b[i] = __builtin_bit_cast(uint32_t, v);
    }
    // the upper halves of two words
    part[w] = uint2{__builtin_amdgcn_perm(b[1], b[0], 0x07060302u), __builtin_amdgcn_perm(b[3], b[2], 0x07060302u)};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] -= __builtin_bit_cast(float, b[i] & 0xFFFF0000u);
  }
}

// A row of P as the products over rows take it: [nz][3][rp] bf16, the three parts of 64
// columns of the rank (rp of them where there are fewer) after one another.
__device__ __forceinline__ void store3(const Split3& o, int64_t row, int j, const uint2 (&part)[3]) {
  uint16_t* const to = o.to + ((row * o.nz + j / 64) * 3) * o.rp + j % 64;
#pragma unroll
  for (int w = 0; w < 3; ++w) *(uint2*)(to + w * o.rp) = part[w];
}

// Rows 64 `block` and on of T in that form, and (block 0) zeros for rows that are not there.
__device__ __forceinline__ void split_rows(const Split3& o, int64_t block, int64_t M, int r) {
  if (block == 0 && threadIdx.x < kZeroBytes / 16) ((u32x4*)o.zero)[threadIdx.x] = u32x4{0u, 0u, 0u, 0u};
  const int64_t e1 = min(64 * (block + 1), M) * r / 4;
  for (int64_t e = 16 * block * r + threadIdx.x; e < e1; e += 256) {
    const int64_t row = e / (r / 4);
    uint2 part[3];
    split4(*(const floatx4*)(o.from + 4 * e), part);
    store3(o, row, (int)(4 * (e - row * (r / 4))), part);
  }
}

// ---------------------------------------------------------------------------
// part[split][m][j] = sum over the split's k of A[m][k] L[a][k][j] (KMAJOR: L1
// [n][K][r]) or A[m][k] L[a][j][k] (L2 [n][r][K]), for tiles of 16 rows.  A workgroup has
// 16 NJ columns of the rank (blockIdx.z: which 64) and a range of k (blockIdx.y).  Its 4
// waves take every fourth step of 32 k, kAhead steps' loads under way, and their sums are
// added in LDS in wave order.  A's rows are the MFMA's second operand, so a lane ends with
// 4 neighbouring columns of one row; a row or column past the end repeats a valid one and
// is not written.  L1 goes through LDS for transposing reads, each wave's own part.
// For tiles most of whose rows are not there: no barrier in the loop, whose few steps are
// latencies one behind the other.  64 rows of 4096 by 48 adapters of rank 32 (12 MB) 6.0 us.
// Workgroups past the tiles split T for the products over rows (in a backward pass).
// ---------------------------------------------------------------------------
template <bool KMAJOR, int NJ>
__global__ __launch_bounds__(256) void k_adapters_narrow_few(AdapterNarrow p) {
  constexpr int NM = 1, kAhead = NJ == 4 ? 2 : 4;
  constexpr int RP = 16 * NJ, BM = 16 * NM;
  constexpr int ROW = RP * 2 + (NJ == 1 ? 0 : 16);                      // LDS bytes of a k row of L1
  constexpr int STAGE = KMAJOR ? 32 * ROW * kAhead : 0;                 // a wave's
  constexpr int SMEM = 4 * STAGE > 4 * BM * RP * 4 ? 4 * STAGE : 4 * BM * RP * 4;
  __shared__ __align__(16) uint8_t smem[SMEM];
  if (blockIdx.x >= p.tiles) {
    if (blockIdx.y == 0 && blockIdx.z == 0) split_rows(p.split, blockIdx.x - p.tiles, p.rows.M, p.r);
    return;
  }
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

// ---------------------------------------------------------------------------
// The same for tiles of BM = 64 MW rows: both operands are copied straight into LDS, 64 of
// k a step through a ring of ST buffers, ST - 1 steps under way.  A wave owns 16 MW rows,
// so nothing is joined.  16-byte pieces of a row of 128 bytes stand XORed by the row, so
// that fragments of 16 rows fall on different banks; rows of L1 are as long as the rank,
// and only those of 128 bytes need that.  A step past K repeats valid memory, and its
// fragments are zeroed.
// 16384 rows of 28672 at rank 64: 179 us, 5.3 TB/s, the copy's rate.  8192 rows of 4096 at
// rank 64: 29 us, 7977 at rank 16: 26, about twice their bytes' time, since 8 to 16 steps a
// workgroup do not hide its start.
// ---------------------------------------------------------------------------
constexpr int kWaitLds = 15 | (3 << 14) | (0x7 << 4);  // lgkmcnt(0), vmcnt as it is
constexpr int wait_vm(int n) { return (n & 15) | ((n >> 4) << 14) | (0x7 << 4) | (0xF << 8); }
typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef __attribute__((address_space(1))) const void* global_ptr_t;

// Reads of a buffer of LDS while copies are on their way into others: the compiler cannot
// tell a transposing read from the copies' destinations and would wait for all copies
// before each.  The reads and their wait are one block of assembly.  Transposing reads make
// fragments of 8 rows (k) of a column, as lds_tr8: `at` is the byte address of the lane's 4
// columns in row 8 g + e, ROW the bytes of a row.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t lds_at(const uint8_t* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)p;
}
__device__ __forceinline__ bf16x8 halves(u32x2 a, u32x2 b) {
  return __builtin_bit_cast(bf16x8, u32x4{a[0], a[1], b[0], b[1]});
}
template <int ROW>
__device__ __forceinline__ void tr_read2(const uint32_t (&at)[2], bf16x8 (&f)[2]) {
  u32x2 v[4];
  asm volatile(
      "ds_read_b64_tr_b16 %0, %4\n"
      "ds_read_b64_tr_b16 %1, %4 offset:%6\n"
      "ds_read_b64_tr_b16 %2, %5\n"
      "ds_read_b64_tr_b16 %3, %5 offset:%6\n"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
      : "v"(at[0]), "v"(at[1]), "n"(4 * ROW));
  f[0] = halves(v[0], v[1]);
  f[1] = halves(v[2], v[3]);
}
template <int ROW>
__device__ __forceinline__ void tr_read4(const uint32_t (&at)[4], bf16x8 (&f)[4]) {
  u32x2 v[8];
  asm volatile(
      "ds_read_b64_tr_b16 %0, %8\n"
      "ds_read_b64_tr_b16 %1, %8 offset:%12\n"
      "ds_read_b64_tr_b16 %2, %9\n"
      "ds_read_b64_tr_b16 %3, %9 offset:%12\n"
      "ds_read_b64_tr_b16 %4, %10\n"
      "ds_read_b64_tr_b16 %5, %10 offset:%12\n"
      "ds_read_b64_tr_b16 %6, %11\n"
      "ds_read_b64_tr_b16 %7, %11 offset:%12\n"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]), "=&v"(v[7])
      : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(4 * ROW));
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = halves(v[2 * i], v[2 * i + 1]);
}
// fragments that lie as they are read, 2048 bytes (16 rows of 128) apart
template <int N>
__device__ __forceinline__ void b128_read(uint32_t at, bf16x8 (&f)[N]) {
  u32x4 v[N];
  if constexpr (N == 1) {
    asm volatile("ds_read_b128 %0, %1\n"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(v[0])
                 : "v"(at));
  } else if constexpr (N == 2) {
    asm volatile("ds_read_b128 %0, %2\n"
                 "ds_read_b128 %1, %2 offset:2048\n"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(v[0]), "=&v"(v[1])
                 : "v"(at));
  } else {
    static_assert(N == 4, "1, 2 or 4 fragments");
    asm volatile("ds_read_b128 %0, %4\n"
                 "ds_read_b128 %1, %4 offset:2048\n"
                 "ds_read_b128 %2, %4 offset:4096\n"
                 "ds_read_b128 %3, %4 offset:6144\n"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
                 : "v"(at));
  }
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = __builtin_bit_cast(bf16x8, v[i]);
}
// the same by transposing reads, with an address for each half
template <int N>
__device__ __forceinline__ void tr_read_rows(const uint32_t (&at)[2 * N], bf16x8 (&f)[N]) {
  u32x2 v[2 * N];
  if constexpr (N == 1) {
    asm volatile(
        "ds_read_b64_tr_b16 %0, %2\n"
        "ds_read_b64_tr_b16 %1, %3\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1])
        : "v"(at[0]), "v"(at[1]));
  } else if constexpr (N == 2) {
    asm volatile(
        "ds_read_b64_tr_b16 %0, %4\n"
        "ds_read_b64_tr_b16 %1, %5\n"
        "ds_read_b64_tr_b16 %2, %6\n"
        "ds_read_b64_tr_b16 %3, %7\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
        : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]));
  } else {
    asm volatile(
        "ds_read_b64_tr_b16 %0, %8\n"
        "ds_read_b64_tr_b16 %1, %9\n"
        "ds_read_b64_tr_b16 %2, %10\n"
        "ds_read_b64_tr_b16 %3, %11\n"
        "ds_read_b64_tr_b16 %4, %12\n"
        "ds_read_b64_tr_b16 %5, %13\n"
        "ds_read_b64_tr_b16 %6, %14\n"
        "ds_read_b64_tr_b16 %7, %15\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]), "=&v"(v[7])
        : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "v"(at[4]), "v"(at[5]), "v"(at[6]), "v"(at[7]));
  }
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = halves(v[2 * i], v[2 * i + 1]);
}
// 8 rows of a column of codes, as bf16; `at`: the lane's 8 columns in row 8 g + (lane & 15) / 2
typedef float floatx2 __attribute__((ext_vector_type(2)));
template <bool E5M2>
__device__ __forceinline__ bf16x8 codes8(u32x2 v) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (E5M2) {
      o[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(v[i], 1.f, false));
      o[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(v[i], 1.f, true));
    } else {
      o[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], 1.f, false));
      o[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], 1.f, true));
    }
  }
  return __builtin_bit_cast(bf16x8, o);
}
template <bool E5M2, int N>
__device__ __forceinline__ void tr_read8(const uint32_t (&at)[N], bf16x8 (&f)[N]) {
  u32x2 v[N];
  if constexpr (N == 2) {
    asm volatile(
        "ds_read_b64_tr_b8 %0, %2\n"
        "ds_read_b64_tr_b8 %1, %3\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1])
        : "v"(at[0]), "v"(at[1]));
  } else {
    static_assert(N == 4, "2 or 4 fragments");
    asm volatile(
        "ds_read_b64_tr_b8 %0, %4\n"
        "ds_read_b64_tr_b8 %1, %5\n"
        "ds_read_b64_tr_b8 %2, %6\n"
        "ds_read_b64_tr_b8 %3, %7\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
        : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]));
  }
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = codes8<E5M2>(v[i]);
}
// the three parts of a fragment, PART bytes apart
template <int ROW, int PART>
__device__ __forceinline__ void tr_read3(uint32_t at, bf16x8 (&f)[3]) {
  u32x2 v[6];
  asm volatile(
      "ds_read_b64_tr_b16 %0, %6\n"
      "ds_read_b64_tr_b16 %1, %6 offset:%7\n"
      "ds_read_b64_tr_b16 %2, %6 offset:%8\n"
      "ds_read_b64_tr_b16 %3, %6 offset:%9\n"
      "ds_read_b64_tr_b16 %4, %6 offset:%10\n"
      "ds_read_b64_tr_b16 %5, %6 offset:%11\n"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5])
      : "v"(at), "n"(4 * ROW), "n"(PART), "n"(PART + 4 * ROW), "n"(2 * PART), "n"(2 * PART + 4 * ROW));
#pragma unroll
  for (int i = 0; i < 3; ++i) f[i] = halves(v[2 * i], v[2 * i + 1]);
}
// two such fragments
template <int ROW, int PART>
__device__ __forceinline__ void tr_read6(const uint32_t (&at)[2], bf16x8 (&f)[2][3]) {
  u32x2 v[12];
  asm volatile(
      "ds_read_b64_tr_b16 %0, %12\n"
      "ds_read_b64_tr_b16 %1, %12 offset:%14\n"
      "ds_read_b64_tr_b16 %2, %12 offset:%15\n"
      "ds_read_b64_tr_b16 %3, %12 offset:%16\n"
      "ds_read_b64_tr_b16 %4, %12 offset:%17\n"
      "ds_read_b64_tr_b16 %5, %12 offset:%18\n"
      "ds_read_b64_tr_b16 %6, %13\n"
      "ds_read_b64_tr_b16 %7, %13 offset:%14\n"
      "ds_read_b64_tr_b16 %8, %13 offset:%15\n"
      "ds_read_b64_tr_b16 %9, %13 offset:%16\n"
      "ds_read_b64_tr_b16 %10, %13 offset:%17\n"
      "ds_read_b64_tr_b16 %11, %13 offset:%18\n"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]), "=&v"(v[7]),
        "=&v"(v[8]), "=&v"(v[9]), "=&v"(v[10]), "=&v"(v[11])
      : "v"(at[0]), "v"(at[1]), "n"(4 * ROW), "n"(PART), "n"(PART + 4 * ROW), "n"(2 * PART), "n"(2 * PART + 4 * ROW));
#pragma unroll
  for (int i = 0; i < 6; ++i) f[i / 3][i % 3] = halves(v[2 * i], v[2 * i + 1]);
}

template <bool KMAJOR, int NJ, int MW>
__global__ __launch_bounds__(256) void k_adapters_narrow(AdapterNarrow p) {
  constexpr int RP = 16 * NJ, BM = 64 * MW;
  constexpr int XB = BM * 128, SB = XB + RP * 128 + 128;
  constexpr int XI = 2 * MW, LI = NJ == 1 ? 1 : NJ / 2;  // copies of a wave and step
  constexpr int ST = NJ == 4 && MW == 2 ? 3 : 4;         // two workgroups a compute unit, or more
  __shared__ __attribute__((aligned(1024))) uint8_t S0[SB];
  __shared__ __attribute__((aligned(1024))) uint8_t S1[SB];
  __shared__ __attribute__((aligned(1024))) uint8_t S2[SB];
  __shared__ __attribute__((aligned(1024))) uint8_t S3[ST > 3 ? SB : 16];
  auto buf = [&](int b) -> uint8_t* { return b == 0 ? S0 : b == 1 ? S1 : b == 2 ? S2 : S3; };
  if (blockIdx.x >= p.tiles) {
    if (blockIdx.y == 0 && blockIdx.z == 0) split_rows(p.split, blockIdx.x - p.tiles, p.rows.M, p.r);
    return;
  }
  Tile tile;
  if (!find_tile(p.rows, BM, blockIdx.x, tile)) return;
  const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int j0 = blockIdx.z * 64, r = p.r, rw = min(r - j0, 64);  // columns of the rank here
  const int64_t K = p.K;
  const int64_t k0 = (int64_t)blockIdx.y * p.krange, k1 = min(k0 + p.krange, K);
  const int steps = (int)((k1 - k0 + 63) / 64);
  // X: copy i has rows 32 i + tid / 8
  const uint16_t* xp[XI];
  const int xc = 8 * ((tid & 7) ^ ((tid >> 3) & 7));
#pragma unroll
  for (int i = 0; i < XI; ++i)
    xp[i] = p.A + max(row_at(p.rows, tile, tile.p0 + 32 * i + (tid >> 3)), (int64_t)0) * K + k0;
  const uint16_t* L = p.L + (int64_t)tile.a * K * r;
  const uint16_t* lp[LI];
  int lk[LI];  // KMAJOR: the row of k within a step
#pragma unroll
  for (int i = 0; i < LI; ++i) {
    int e = NJ == 1 ? tid & 127 : 256 * i + tid;
    if constexpr (KMAJOR) {
      e = min(e, 8 * rw - 1);
      const int per = rw / 8;
      lk[i] = e / per;
      int c = e - lk[i] * per;
      if (rw == 64) c ^= ((lk[i] >> 1) & 1) << 1;
      lp[i] = L + k0 * r + j0 + 8 * c;
    } else {
      lp[i] = L + (int64_t)(j0 + min(e >> 3, rw - 1)) * K + k0;
    }
  }
  // Where the width is a power of two, tiles begin at different steps: all workgroups would
  // otherwise read from the same few memory channels at a time (16000 rows of 8192: 80 us
  // against 90; whole calls of 8192 rows of 16384 at rank 64 82 against 119, of 8192 level).
  // Elsewhere the tiles' common steps share L (16384 rows of 28672 at rank 64: 178 us, and 196
  // with steps of their own).  Multiples of 4096 that are no power of two need neither: calls of
  // 8192 rows of 12288 and 24576 are level.  Of 11008, at rank 64, apart would be 69 against 72.
  const int first = (K & (K - 1)) == 0 ? (int)(blockIdx.x * 5u % (unsigned)steps) : 0;
  auto place = [&](int t) -> int { return t + first < steps ? t + first : t + first - steps; };
  auto copy = [&](int t, int b) {
    t = place(min(t, steps - 1));  // a step behind the last copies it once more, and is not used
    uint8_t* const to = buf(b);
    const int64_t k = 64 * (int64_t)t, left = K - k0 - k;  // from here to the row's end
    const int64_t x = k + (xc < left ? xc : 0);
#pragma unroll
    for (int i = 0; i < XI; ++i)
      __builtin_amdgcn_global_load_lds((global_ptr_t)(xp[i] + x), (lds_ptr_t)(to + (4 * i + wave) * 1024), 16, 0, 0);
#pragma unroll
    for (int i = 0; i < LI; ++i) {
      const uint16_t* from = KMAJOR ? lp[i] + (k + min((int64_t)lk[i], left - 1)) * r : lp[i] + x;
      __builtin_amdgcn_global_load_lds((global_ptr_t)from,
                                       (lds_ptr_t)(to + XB + (NJ == 1 ? wave & 1 : 4 * i + wave) * 1024), 16, 0, 0);
    }
  };
  floatx4 acc[NJ][MW];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int i = 0; i < MW; ++i) acc[j][i] = floatx4{0.f, 0.f, 0.f, 0.f};
  const int rb = KMAJOR ? 2 * rw : 128;
  const int e = li >> 2, q = li & 3, swz = rw == 64 && e >= 2 ? 2 : 0;
  auto compute = [&](int t, int b) {
    uint8_t* const at = buf(b);
    const int64_t left = k1 - k0 - 64 * (int64_t)place(t);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const bool in = 32 * ks + 8 * g < left;
      const int piece = ((4 * ks + g) ^ (li & 7)) << 4;
      bf16x8 fx[MW];
      b128_read<MW>(lds_at(at) + (wave * 16 * MW + li) * 128 + piece, fx);
      if (!in) {
#pragma unroll
        for (int i = 0; i < MW; ++i) fx[i] = __builtin_bit_cast(bf16x8, u32x4{0u, 0u, 0u, 0u});
      }
      bf16x8 fl[NJ];
      if constexpr (KMAJOR) {
        // rows of the rank's own length: the second half of a fragment has its own address
        uint32_t at2[2 * NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          at2[2 * j] = lds_at(at + XB) + (32 * ks + 8 * g + e) * rb + (((2 * j + (q >> 1)) ^ swz) << 4) + ((q & 1) << 3);
          at2[2 * j + 1] = at2[2 * j] + 4 * rb;
        }
        tr_read_rows<NJ>(at2, fl);
      } else {
        b128_read<NJ>(lds_at(at + XB) + li * 128 + piece, fl);
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        u32x4 v = __builtin_bit_cast(u32x4, fl[j]);
        if (!in) v = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < MW; ++i)
          acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, v), fx[i], acc[j][i], 0, 0, 0);
      }
    }
  };
  auto step = [&](int t, int b) {
    // this step's copies are there, everybody's, and the reads of the step before are done
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(wait_vm((ST - 2) * (XI + LI)) & kWaitLds);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    copy(t + ST - 1, (b + ST - 1) % ST);
    __builtin_amdgcn_sched_barrier(0);
    compute(t, b);
  };
#pragma unroll
  for (int b = 0; b < ST - 1; ++b) copy(b, b);
  for (int t = 0; t < steps; t += ST) {
    step(t, 0);
#pragma unroll
    for (int b = 1; b < ST; ++b)
      if (t + b < steps) step(t + b, b);
  }
#pragma unroll
  for (int i = 0; i < MW; ++i) {
    const int64_t row = row_at(p.rows, tile, tile.p0 + wave * 16 * MW + 16 * i + li);
    if (row < 0) continue;
    float* to = p.part + ((int64_t)blockIdx.y * p.rows.M + row) * r + j0;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (16 * j + 4 * g < rw) *(floatx4*)(to + 16 * j + 4 * g) = acc[j][i];
  }
  __builtin_amdgcn_s_waitcnt(0);  // no copy is on its way into LDS that is no longer this workgroup's
}

// sum of a value's splits, in their order, 4 loads at a time
__device__ __forceinline__ floatx4 join4(const float* part, int64_t stride, int splits) {
  floatx4 s = *(const floatx4*)part;
  for (int q = 1; q < splits; q += 4) {
    floatx4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = *(const floatx4*)(part + min(q + u, splits - 1) * stride);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (q + u < splits) s += v[u];
  }
  return s;
}

// ---------------------------------------------------------------------------
// out[m][c] = bf16(base[m][c] + s[a] sum_j P[m][j] L[a][j][c]) (JMAJOR: L2 [n][r][N])
// or with L[a][c][j] (L1 [n][N][r]).  A workgroup has 16 RW rows and goes over `blocks`
// blocks of 128 columns, the next block's base and L under way; RW = 1: each wave has a
// block of its own.  P (its splits joined) is split into hi and lo in LDS, 16 of the rank
// a step: the MFMA's 32 products are hi's 16 and lo's, against the same 16 of L.  P is the
// first operand and column i of L's fragment f is 8 i + f, so a lane ends with 8
// neighbouring columns of 4 rows, and 16 lanes read and write 256 bytes of a row.  For that
// a panel of L stands in LDS with column 8 i + f at place 16 f + i.  A rank above 16 NJ is
// taken in runs of 16 NJ.
// Bound by reading base and writing the output: 7977 rows by 11008 of rank 16 79 us (4.4 TB/s),
// 8192 by 11008 of rank 64 92 (3.9), 16384 by 8192 of rank 64 119 (4.5), where a copy of such a
// size reaches 5.4; the rest are the starts of 1024 workgroups, with the joining of P in each.
// 64 rows by 11008 of rank 32: 9.9 us.
// ---------------------------------------------------------------------------
template <bool JMAJOR, int NJ, int RW, int RMAX>
__global__ __launch_bounds__(256, RW == 1 && NJ < 4 ? 4 : 1) void k_adapters_wide(AdapterWide p) {
  constexpr int BM = 16 * RW, RC = 16 * NJ;
  constexpr int NB = RW == 4 ? 2 : 1, G = 4 / RW, TG = 64 * RW;  // panel buffers; groups of waves, their threads
  constexpr int LROW = JMAJOR ? 128 * 2 + 32 : RC * 2;           // LDS bytes of a row of the panel
  constexpr int PB = JMAJOR ? RC * LROW : 128 * LROW;
  constexpr int PL = 128 * RC / 8 / TG;                          // 16-byte pieces of a panel a thread
  constexpr int PROW = RMAX * 4 + 16;                            // of a row of P: for each 16 of the rank hi, then lo
  __shared__ __align__(16) uint8_t ps[BM * PROW];
  __shared__ __align__(16) uint8_t panel[G][NB][PB];
  Tile tile;
  if (!find_tile(p.rows, BM, blockIdx.x, tile)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, li = lane & 15, g = lane >> 4;
  const int grp = wave / RW, tg = tid % TG;
  const int r = p.r, r16 = (r + 15) / 16 * 16;
  const int64_t N = p.N;
  const int nblocks = (int)((N + 127) / 128);
  // RW = 1: a block past the columns' end goes through the same barriers and writes nothing
  const int cb0 = RW == 4 ? blockIdx.y * p.blocks : blockIdx.y * 4 + grp;
  const int cb1 = RW == 4 ? min(cb0 + p.blocks, nblocks) : cb0 + 1;
  const int runs = RMAX == RC ? 1 : (r16 + RC - 1) / RC;
  const uint16_t* L = p.L + (int64_t)tile.a * N * r;
  int64_t at[4];  // this lane's 4 rows, or -1
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int64_t row = row_at(p.rows, tile, tile.p0 + (RW == 4 ? 16 * wave : 0) + 4 * g + v);
    at[v] = row < 0 ? -1 : row * N;
  }
  // base: of rows that are not there a valid one's; without a base one piece for all, not used
  const uint16_t* const from = p.base ? p.base : p.L;
  const int64_t some = p.base ? -1 : 0;
  const uint32_t keep = p.base ? 0xFFFFFFFFu : 0u;
  auto load_base = [&](int cb, u32x4 (&b)[4]) __attribute__((always_inline)) {
    const int64_t c = min((int64_t)cb * 128 + 8 * li, N - 8);
#pragma unroll
    for (int v = 0; v < 4; ++v) b[v] = *(const u32x4*)(from + ((max(at[v], (int64_t)0) + c) & some));
  };
  // pieces of the panel: JMAJOR 16 a row of the rank, else RC / 8 a column
  auto load_panel = [&](int cb, int run, u32x4 (&l)[PL]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = TG * i + tg;
      const int j = run * RC + (JMAJOR ? e / 16 : 8 * (e % (RC / 8)));
      const int64_t c = (int64_t)cb * 128 + (JMAJOR ? 8 * (e % 16) : e / (RC / 8));
      const int64_t o = JMAJOR ? (int64_t)min(j, r - 1) * N + min(c, N - 8) : min(c, N - 1) * r + min(j, r - 8);
      l[i] = *(const u32x4*)(L + o);
      if (j >= r) l[i] = u32x4{0u, 0u, 0u, 0u};  // P's zeros there are multiplied by it
    }
  };
  // Pieces of 16 bytes of a row of L1's panel stand XORed by this, so that the 16 lanes that
  // LDS serves at once (0-3, 12-15 and 20-27, and so on) read from different banks.
  auto place = [](int row) -> int {
    const int k = row >> 2 & 3;
    return NJ == 4 ? row & 7 : NJ == 2 ? (k & 1) << 1 ^ (k >> 1) * 3 : 0;
  };
  auto store_panel = [&](uint8_t* to, const u32x4 (&l)[PL]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = TG * i + tg;
      if constexpr (JMAJOR) {
        uint8_t* const at = to + e / 16 * LROW + 2 * (e % 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          *(uint16_t*)(at + 64 * k) = (uint16_t)l[i][k];
          *(uint16_t*)(at + 64 * k + 32) = (uint16_t)(l[i][k] >> 16);
        }
      } else {
        const int c = e / (RC / 8), row = (c & 7) * 16 + (c >> 3);
        *(u32x4*)(to + row * LROW + ((e % (RC / 8) ^ place(row)) << 4)) = l[i];
      }
    }
  };
  // The panels are numbered through the blocks and their runs of the rank; the one after the
  // next is loaded while one is multiplied.
  const int panels = (cb1 - cb0) * runs;
  auto load_panel_no = [&](int i, u32x4 (&l)[PL]) __attribute__((always_inline)) {
    i = min(i, panels - 1);
    load_panel(runs == 1 ? cb0 + i : cb0 + i / runs, runs == 1 ? 0 : i % runs, l);
  };
  u32x4 b0[4], b1[4], l0[PL], l1[PL];
  load_panel_no(0, l0);
  load_base(cb0, b0);
  if constexpr (NB == 2) load_panel_no(1, l1);
  constexpr int PT = (BM * RMAX / 4 + 255) / 256;  // 4-value pieces of P a thread, up to 4 of them at once
#pragma unroll 1
  for (int i0 = 0; i0 < PT; i0 += 4) {
    floatx4 v[PT < 4 ? PT : 4];
    int64_t o[PT < 4 ? PT : 4];
#pragma unroll
    for (int i = 0; i < (PT < 4 ? PT : 4); ++i) {
      const int e = 256 * (i0 + i) + tid, m = e / (r16 / 4), j = 4 * (e % (r16 / 4));
      const int64_t row = m < BM && j < r ? row_at(p.rows, tile, tile.p0 + m) : -1;
      o[i] = row < 0 ? -1 : row * r + j;
      v[i] = floatx4{0.f, 0.f, 0.f, 0.f};
    }
    constexpr int QU = RW == 1 && NJ < 4 ? 8 : 4;  // splits at once
    for (int q0 = 0; q0 < p.splits; q0 += QU) {
      floatx4 x[PT < 4 ? PT : 4][QU];
#pragma unroll
      for (int i = 0; i < (PT < 4 ? PT : 4); ++i)
#pragma unroll
        for (int u = 0; u < QU; ++u)
          x[i][u] = *(const floatx4*)(p.part + min(q0 + u, p.splits - 1) * (p.rows.M * r) + max(o[i], (int64_t)0));
#pragma unroll
      for (int i = 0; i < (PT < 4 ? PT : 4); ++i)
#pragma unroll
        for (int u = 0; u < QU; ++u)
          if (q0 + u < p.splits) v[i] += x[i][u];
    }
#pragma unroll
    for (int i = 0; i < (PT < 4 ? PT : 4); ++i) {
      const int e = 256 * (i0 + i) + tid, m = e / (r16 / 4), j = 4 * (e % (r16 / 4));
      if (m >= BM) continue;
      if (o[i] < 0) v[i] = floatx4{0.f, 0.f, 0.f, 0.f};
      else if (blockIdx.y == 0) {
        if (p.T_out) *(floatx4*)(p.T_out + o[i]) = v[i];
        if (p.split.to) {
          uint2 three[3];
          split4(v[i], three);
          store3(p.split, (o[i] - j) / r, j, three);
        }
      }
      uint2 part[2];
      split4(v[i], part);
      uint8_t* to = ps + m * PROW + (j / 16) * 64 + (j % 16) * 2;
      *(uint2*)to = part[0];
      *(uint2*)(to + 32) = part[1];
    }
  }
  store_panel(panel[grp][0], l0);
  __syncthreads();
  const float s = p.s[tile.a];
  const uint8_t* pa = ps + (RW == 4 ? 16 * wave + li : li) * PROW + (g >> 1) * 32 + (g & 1) * 16;
  floatx4 acc[8];
  auto multiply = [&](const uint8_t* lp, int run) __attribute__((always_inline)) {
#pragma unroll
    for (int st = 0; st < NJ; ++st) {
      if (NJ > 1 && run * RC + 16 * st >= r16) break;  // the same for all; P's places past r16 hold nothing
      const bf16x8 a = *(const bf16x8*)(pa + (run * NJ + st) * 64);
#pragma unroll
      for (int f = 0; f < 8; ++f) {
        bf16x8 w;
        if constexpr (JMAJOR)
          w = lds_tr8(const_cast<uint8_t*>(lp) + (16 * st + 8 * (g & 1) + (li >> 2)) * LROW + 2 * (16 * f + 4 * (li & 3)),
                      LROW);
        else w = *(const bf16x8*)(lp + (16 * f + li) * LROW + (((2 * st + (g & 1)) ^ place(li)) << 4));
        acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, w, acc[f], 0, 0, 0);
      }
    }
  };
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int f = 0; f < 8; ++f) acc[f] = floatx4{0.f, 0.f, 0.f, 0.f};
  };
  auto write = [&](int cb, const u32x4 (&b)[4], auto all) __attribute__((always_inline)) {
    const int64_t c = (int64_t)cb * 128 + 8 * li;
    u32x4 o[4];
#pragma unroll
    for (int v = 0; v < 4; ++v)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t w = b[v][k] & keep;
        o[v][k] = pack_bf16x2(__builtin_fmaf(s, acc[2 * k][v], __builtin_bit_cast(float, w << 16)),
                              __builtin_fmaf(s, acc[2 * k + 1][v], __builtin_bit_cast(float, w & 0xFFFF0000u)));
      }
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (decltype(all)::value || (at[v] >= 0 && c < N)) *(u32x4*)(p.out + at[v] + c) = o[v];
  };
  if constexpr (NB == 1) {
    // one block a wave
    clear();
    for (int run = 0; run < runs; ++run) {
      if (run + 1 < runs) load_panel_no(run + 1, l0);
      multiply(panel[grp][0], run);
      if (run + 1 < runs) {
        __syncthreads();  // the panel's reads are done
        store_panel(panel[grp][0], l0);
        __syncthreads();
      }
    }
    write(cb0, b0, std::false_type{});
  } else {
    // Block cb, from panel i on, of which the next one's pieces are in `l` (the other set
    // takes the one after that).  Whole tiles have a loop of their own, whose writes stand
    // under no condition: the compiler then knows how many are on their way, and waits for
    // no more of them than it has to.
    auto one = [&](int i, int run, const u32x4 (&l)[PL], u32x4 (&after)[PL]) __attribute__((always_inline)) {
      load_panel_no(i + 2, after);
      multiply(panel[0][i & 1], run);
      store_panel(panel[0][(i + 1) & 1], l);
    };
    auto go = [&](auto all) __attribute__((always_inline)) {
      if constexpr (RMAX == RC) {
        auto block = [&](int cb, const u32x4 (&b)[4], u32x4 (&nb)[4], const u32x4 (&l)[PL], u32x4 (&after)[PL]) __attribute__((always_inline)) {
          load_base(min(cb + 1, cb1 - 1), nb);
          clear();
          one(cb - cb0, 0, l, after);
          write(cb, b, all);
          __syncthreads();
        };
        int cb = cb0;
        for (; cb + 1 < cb1; cb += 2) {
          block(cb, b0, b1, l1, l0);
          block(cb + 1, b1, b0, l0, l1);
        }
        if (cb < cb1) block(cb, b0, b1, l1, l0);
      } else {
        for (int cb = cb0, i = 0; cb < cb1; ++cb) {
          load_base(cb, b0);
          clear();
          for (int run = 0; run < runs; ++run, ++i) {
            one(i, run, l1, l0);
#pragma unroll
            for (int k = 0; k < PL; ++k) l1[k] = l0[k];
            __syncthreads();
          }
          write(cb, b0, all);
        }
      }
    };
    bool all = (int64_t)cb1 * 128 <= N;
#pragma unroll
    for (int v = 0; v < 4; ++v) all = all && at[v] >= 0;
    if (__all(all)) go(std::true_type{});
    else go(std::false_type{});
  }
}

// ---------------------------------------------------------------------------
// The forward pass of a tile of 16 rows in one launch, for ranks up to 16: every workgroup
// of a tile makes the whole T, its 16 waves taking every 16th step of 32 columns of X, and
// then its part of the columns of Y, a block of 128 a wave at a time.  Making T again in
// each of a tile's workgroups reads L1[a] from the caches.  An eager call of a few rows in two
// launches is bound by the host, for which each is 3.7 us; in one it is bound by this kernel's
// chain of loads: offsets, order, two rounds of X and L1, the join, Y (one token, rank 16,
// 4096 x 4096: 11.4 us a call that allocates its results and 8.5 one that is given them, against 15.2
// and 13.0 with two launches; by replayed graphs 8.4 against 8.1).
// The products are those of k_adapters_narrow_few and k_adapters_wide.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(1024) void k_adapters_few(AdapterFew p) {
  constexpr int WV = 16, RP = 16;
  constexpr int AHEAD = 4;                                // steps whose loads are under way
  constexpr int ROW = RP * 2;                             // LDS bytes of a k row of L1
  constexpr int STAGE = 32 * ROW * AHEAD;                 // a wave's
  constexpr int LROW = 128 * 2 + 32, PB = RP * LROW;      // a row of L2's panel, and a wave's panel
  constexpr int PL = 128 * RP / 8 / 64, PROW = RP * 4 + 16;
  constexpr int AREA = STAGE > PB ? STAGE : PB;
  constexpr int RED = WV * 16 * RP * 4;
  __shared__ __align__(16) uint8_t smem[WV * AREA > RED ? WV * AREA : RED];
  __shared__ __align__(16) uint8_t ps[16 * PROW];
  Tile tile;
  if (!find_tile(p.rows, 16, blockIdx.x, tile)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, li = lane & 15, g = lane >> 4;
  const int r = p.r;
  const int64_t K = p.K, N = p.N;
  const int nblocks = (int)((N + 127) / 128), stride = WV * (int)gridDim.y;
  const uint16_t* L2 = p.L2 + (int64_t)tile.a * N * r;
  int64_t at[4];  // this lane's 4 rows of Y, or -1
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int64_t row = row_at(p.rows, tile, tile.p0 + 4 * g + v);
    at[v] = row < 0 ? -1 : row * N;
  }
  const uint16_t* const from = p.base ? p.base : p.L2;  // without a base one piece for all, not used
  const int64_t some = p.base ? -1 : 0;
  const uint32_t keep = p.base ? 0xFFFFFFFFu : 0u;
  auto load_block = [&](int cb, u32x4 (&l)[PL], u32x4 (&b)[4]) {
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int j = 4 * i + lane / 16;
      const int64_t c = min((int64_t)cb * 128 + 8 * (lane % 16), N - 8);
      l[i] = *(const u32x4*)(L2 + (int64_t)min(j, r - 1) * N + c);
      if (j >= r) l[i] = u32x4{0u, 0u, 0u, 0u};
    }
    const int64_t c = min((int64_t)cb * 128 + 8 * li, N - 8);
#pragma unroll
    for (int v = 0; v < 4; ++v) b[v] = *(const u32x4*)(from + ((max(at[v], (int64_t)0) + c) & some));
  };
  int cb = blockIdx.y * WV + wave;
  u32x4 l[PL], b[4];
  load_block(min(cb, nblocks - 1), l, b);  // ahead of T's

  // T
  const int64_t trow = row_at(p.rows, tile, tile.p0 + tid / (RP / 4));
  const int tj = 4 * (tid % (RP / 4));
  floatx4 t = {0.f, 0.f, 0.f, 0.f};
  {
    const uint16_t* const x = p.X + max(row_at(p.rows, tile, tile.p0 + li), (int64_t)0) * K + 8 * g;
    const uint16_t* const L1 = p.L1 + (int64_t)tile.a * K * r;
    uint8_t* const stage = smem + wave * AREA;
    floatx4 acc = {0.f, 0.f, 0.f, 0.f};
    constexpr u32x4 kZero = {0u, 0u, 0u, 0u};
    for (int64_t s0 = 32 * wave; s0 < K; s0 += 32 * WV * AHEAD) {
      u32x4 fx[AHEAD], fl[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int64_t k = s0 + 32 * WV * u, kr = k + lane / 2;
        const int j = 8 * (lane & 1);
        fx[u] = k + 8 * g < K ? *(const u32x4*)(x + k) : kZero;
        fl[u] = kr < K && j < r ? *(const u32x4*)(L1 + kr * r + j) : kZero;
      }
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) *(u32x4*)(stage + u * 32 * ROW + lane * 16) = fl[u];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            lds_tr8(stage + (32 * u + 8 * g + (li >> 2)) * ROW + 8 * (li & 3), ROW),
            __builtin_bit_cast(bf16x8, fx[u]), acc, 0, 0, 0);
    }
    __syncthreads();
    float* const red = (float*)smem;  // [WV][16][RP]
    *(floatx4*)(red + (wave * 16 + li) * RP + 4 * g) = acc;
    __syncthreads();
    if (tid < 16 * RP / 4) {
      const float* const from = red + tid / (RP / 4) * RP + tj;
      t = *(const floatx4*)from;
#pragma unroll
      for (int w = 1; w < WV; ++w) t += *(const floatx4*)(from + w * 16 * RP);
    }
  }
  if (tid < 16 * RP / 4) {
    // a row past the tile has another row's sums, or nothing of the rank's, and is not written
    if (trow < 0 || tj >= r) t = floatx4{0.f, 0.f, 0.f, 0.f};
    else if (p.T_out && blockIdx.y == 0) *(floatx4*)(p.T_out + trow * r + tj) = t;
    uint2 part[2];
    split4(t, part);
    uint8_t* to = ps + tid / (RP / 4) * PROW + (tj / 16) * 64 + (tj % 16) * 2;
    *(uint2*)to = part[0];
    *(uint2*)(to + 32) = part[1];
  }
  __syncthreads();

  // Y
  const float s = p.s[tile.a];
  const uint8_t* const pa = ps + li * PROW + (g >> 1) * 32 + (g & 1) * 16;
  uint8_t* const panel = smem + wave * AREA;  // the wave's own: no barrier from here on
  for (; cb < nblocks; cb += stride) {
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      uint8_t* const to = panel + (4 * i + lane / 16) * LROW + 2 * (lane % 16);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        *(uint16_t*)(to + 64 * k) = (uint16_t)l[i][k];
        *(uint16_t*)(to + 64 * k + 32) = (uint16_t)(l[i][k] >> 16);
      }
    }
    u32x4 base[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) base[v] = b[v];
    load_block(min(cb + stride, nblocks - 1), l, b);
    floatx4 acc[8];
#pragma unroll
    for (int f = 0; f < 8; ++f) acc[f] = floatx4{0.f, 0.f, 0.f, 0.f};
    const bf16x8 a = *(const bf16x8*)pa;
#pragma unroll
    for (int f = 0; f < 8; ++f)
      acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
          a, lds_tr8(panel + (8 * (g & 1) + (li >> 2)) * LROW + 2 * (16 * f + 4 * (li & 3)), LROW), acc[f], 0, 0, 0);
    const int64_t c = (int64_t)cb * 128 + 8 * li;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      u32x4 o;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t w = base[v][k] & keep;
        o[k] = pack_bf16x2(__builtin_fmaf(s, acc[2 * k][v], __builtin_bit_cast(float, w << 16)),
                           __builtin_fmaf(s, acc[2 * k + 1][v], __builtin_bit_cast(float, w & 0xFFFF0000u)));
      }
      if (at[v] >= 0 && c < N) *(u32x4*)(p.out + at[v] + c) = o;
    }
  }
}

// ---------------------------------------------------------------------------
// dL[a][j][c] (or [c][j]) = s[a] sum over a's rows of P[m][j] Q[m][c]: a workgroup has
// 256 columns of Q, 16 NJ of the rank (blockIdx.z: which 64) and up to p.item rows of an
// adapter (blockIdx.y).  Both operands are copied straight into LDS, 32 rows a step through
// a ring of ST buffers, and read with transposing reads: the products contract the rows.
// Rows past the tile come from zeros.  16-byte pieces stand XORed by the row, so that the
// lanes that LDS serves at once fall on different banks.  An adapter whose rows are all here
// is written out, otherwise the item's sums go to a part of their own, which
// k_adapters_join adds in order.
//
// bf16 (X8 0): P comes as three bf16 parts, made once for all columns.
// 8 bits (X8 1: e4m3, 2: e5m2): the codes are read transposed and become bf16 in registers;
// P comes in fp32 and is multiplied by the scales of its row, one for each 128 columns (rounded
// to fp32), and split a step ahead into tiles beside the ring.
//
// The two waves of a SIMD take turns: the lower four read a step and multiply it (and split
// before), the upper four multiply the step before and read (and split last).
//
// A step takes 0.78 us at rank 16, the copy's rate, and 0.97 at rank 64, whose parts of P are
// 12 KB beside Q's 16 and whose MFMAs are four times as many (busy 32 % of the cycles, LDS
// 18 %, no conflicts); a workgroup's start and end are 7 us.  8192 rows by 11008 and 4096
// columns, 8 adapters of rank 64: 85 us; 16384 rows by 8192 columns of codes and 28672 of dY at
// rank 64: 341 (3.2 TB/s).  Measured beside it: tiles of 512 columns, 316 us for the latter but
// 89 for the former; two workgroups a compute unit with rings of two steps, 8 % slower; rings of
// 5 to 7 steps, level.
// ---------------------------------------------------------------------------
template <int X8, int NJ>
struct GradTile {
  static constexpr int KR = 32, RP = 16 * NJ, ST = X8 ? 5 : 4;
  static constexpr int PROW = 3 * RP * 2;                         // LDS bytes of a row of P's parts
  static constexpr int QROW = X8 ? 256 : 512, QB = KR * QROW;     // of Q
  static constexpr int PB = X8 ? KR * RP * 4 : KR * PROW;         // of P as it is copied
  static constexpr int SB = QB + PB + (X8 ? 256 : 0);             // a buffer, with the scales
  // behind the ring P's parts for two blocks of columns, of two steps
  static constexpr int SMEM = ST * SB + (X8 ? 4 * KR * PROW : 0);
  static constexpr int LIST = kMaxAdapterItem + (ST + 1) * KR;
};

// Zeros for an adapter without rows, where no other kernel writes them: its columns c0 to
// c0 + 255 and the workgroup's 64 of the rank.
__device__ __forceinline__ void clear_empty(const AdapterRows& rows, const AdapterGrad& p, int a, int64_t c0) {
  const int M = (int)rows.M;
  if (min(max(rows.offsets[a + 1], 0), M) > min(max(rows.offsets[a], 0), M)) return;
  const int j0 = blockIdx.z * 64, rw = min(p.r - j0, 64);
  const int64_t cols = min(p.N - c0, (int64_t)256);
  float* const out = p.out + (int64_t)a * p.r * p.N;
  constexpr floatx4 kZero = {0.f, 0.f, 0.f, 0.f};
  for (int e = 4 * threadIdx.x; e < cols * rw; e += 4 * blockDim.x) {
    if (p.trans) *(floatx4*)(out + (c0 + e / rw) * p.r + j0 + e % rw) = kZero;
    else *(floatx4*)(out + (j0 + e / cols) * p.N + c0 + e % cols) = kZero;
  }
}

template <int X8, int NJ>
__device__ __forceinline__ void grad_tile(const AdapterRows& rows, const AdapterGrad& p, int cblock, uint8_t* ring,
                                          int* list) {
  using G = GradTile<X8, NJ>;
  constexpr int KR = G::KR, RP = G::RP, ST = G::ST, PROW = G::PROW, QB = G::QB, SB = G::SB;
  constexpr int JW = NJ == 4 ? 2 : 1, CW = 8 / JW;      // waves over the rank and over the columns
  constexpr int FJ = NJ / JW, FC = 16 / CW;             // a wave's fragments
  constexpr int QI = X8 ? 1 : 2;                        // 1 KB copies of Q a wave and step
  constexpr int NP = G::PB / 1024;                      // of P a step
  constexpr int PI = NP > 8 ? 2 : 1;                    // and a wave
  constexpr int C = QI + PI + (X8 ? 1 : 0);             // copies of a wave and step
  const uint32_t split = lds_at(ring) + ST * SB;
  const int64_t N = p.N, c0 = (int64_t)cblock * 256;
  if (blockIdx.y >= p.items) {
    clear_empty(rows, p, blockIdx.y - (int)p.items, c0);
    return;
  }
  Tile tile;
  if (!find_tile(rows, p.item, blockIdx.y, tile)) return;
  const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = p.r, j0 = blockIdx.z * 64;
  const int steps = (tile.p1 - tile.p0 + KR - 1) / KR;
  // the rows of every step, -1 where there is none
  const int count = tile.p1 - tile.p0;
  for (int i = tid; i < (steps + ST) * KR; i += 512) {
    int row = tile.p0 + i;
    if (rows.order) row = rows.order[min(row, tile.p1 - 1)];
    list[i] = i < count && (uint32_t)row < (uint32_t)rows.M ? row : -1;
  }
  __syncthreads();

  // where this lane's pieces come from; Q: rows 2 (8 i + wave) and the next (X8: 4 wave to + 3)
  const int qm = X8 ? 4 * wave + (lane >> 4) : 2 * wave + (lane >> 5);
  int64_t qc = X8 ? c0 + 16 * ((lane & 15) ^ (qm & 15)) : c0 + 8 * ((lane & 31) ^ ((qm & 3) << 1 | (qm & 8)));
  qc = qc < N ? qc : 0;
  const uint8_t* const qbase = (const uint8_t*)p.Q + (X8 ? 1 : 2) * qc;
  const uint32_t qstride = (uint32_t)N * (X8 ? 1 : 2);
  constexpr int CPR = X8 ? RP / 4 : PROW / 16;  // pieces of a row of P
  const uint8_t* pbase[PI];
  int pm[PI];
#pragma unroll
  for (int i = 0; i < PI; ++i) {
    const int e = 64 * ((8 * i + wave) % NP) + lane;
    pm[i] = e / CPR;
    int c = e % CPR;
    if constexpr (X8 != 0) {
      pbase[i] = j0 + 4 * c < r ? (const uint8_t*)(p.P + j0 + 4 * c) : nullptr;
    } else {
      if (NJ == 4) c ^= (pm[i] & 2) | (pm[i] & 8) >> 1;
      pbase[i] = (const uint8_t*)p.P3 + (blockIdx.z * CPR + c) * 16;
    }
  }
  const uint32_t pstride = X8 ? (uint32_t)r * 4 : gridDim.z * PROW;
  const int kb = (int)((N + 127) / 128);
  const float* const sbase = X8 ? p.q_scales + min(2 * cblock + (lane & 1), kb - 1) : nullptr;
  int rq[QI], rp[PI], rs = 0;  // rows of the next copies
  auto next_rows = [&](int t) {
#pragma unroll
    for (int i = 0; i < QI; ++i) rq[i] = list[KR * t + 16 * i + qm];
#pragma unroll
    for (int i = 0; i < PI; ++i) rp[i] = list[KR * t + pm[i]];
    if constexpr (X8 != 0) rs = list[KR * t + (lane >> 1)];
  };
  auto copy = [&](int b) {
    uint8_t* const to = ring + b * SB;  // (a step past the last is all zeros, and not used)
#pragma unroll
    for (int i = 0; i < QI; ++i) {
      const void* there = qbase + (uint64_t)(uint32_t)rq[i] * qstride;
      __builtin_amdgcn_global_load_lds((global_ptr_t)(rq[i] < 0 ? p.zero : there),
                                       (lds_ptr_t)(to + (8 * i + wave) * 1024), 16, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < PI; ++i) {
      const void* there = pbase[i] + (uint64_t)(uint32_t)rp[i] * pstride;
      __builtin_amdgcn_global_load_lds((global_ptr_t)(rp[i] < 0 || (X8 && !pbase[i]) ? p.zero : there),
                                       (lds_ptr_t)(to + QB + (8 * i + wave) % NP * 1024), 16, 0, 0);
    }
    if constexpr (X8 != 0) {  // every wave copies the same scales
      const void* there = sbase + (uint64_t)(uint32_t)rs * (uint32_t)kb;
      __builtin_amdgcn_global_load_lds((global_ptr_t)(rs < 0 ? p.zero : there), (lds_ptr_t)(to + QB + G::PB), 4, 0, 0);
    }
  };

  const int wj = wave / CW, wc = wave % CW;
  const int e = li >> 2, q = li & 3;
  floatx4 acc[FJ][FC];
#pragma unroll
  for (int j = 0; j < FJ; ++j)
#pragma unroll
    for (int c = 0; c < FC; ++c) acc[j][c] = floatx4{0.f, 0.f, 0.f, 0.f};
  // a lane's addresses within a buffer, and within a tile of P's parts
  uint32_t pa[FJ], qa[FC];
#pragma unroll
  for (int j = 0; j < FJ; ++j)
    pa[j] = (8 * g + e) * PROW +
            (((2 * (wj * FJ + j) + (q >> 1)) ^ (NJ == 4 ? (e & 2) | (g & 1) << 2 : 0)) << 4) + ((q & 1) << 3);
#pragma unroll
  for (int c = 0; c < FC; ++c) {
    const int f = wc * FC + c;
    if constexpr (X8 != 0) qa[c] = (8 * g + (li >> 1)) * 256 + ((f ^ ((g & 1) << 3 | li >> 1)) << 4) + ((li & 1) << 3);
    else qa[c] = (8 * g + e) * 512 + (((2 * f + (q >> 1)) ^ (e << 1 | (g & 1) << 3)) << 4) + ((q & 1) << 3);
  }
  bf16x8 fp[FJ][3], fq[FC];
  auto read = [&](int t, int b) {
    const uint32_t at = lds_at(ring) + b * SB;
    const uint32_t parts =
        X8 ? split + ((t & 1) * 2 + (wc * FC >> 3)) * (KR * PROW) : at + QB;
    uint32_t pt[FJ], qt[FC];
#pragma unroll
    for (int j = 0; j < FJ; ++j) pt[j] = parts + pa[j];
#pragma unroll
    for (int c = 0; c < FC; ++c) qt[c] = at + qa[c];
    if constexpr (X8 != 0) tr_read8<X8 == 2, FC>(qt, fq);
    else if constexpr (FC == 4) tr_read4<512>(qt, fq);
    else tr_read2<512>(qt, fq);
    if constexpr (FJ == 2) tr_read6<PROW, 2 * RP>(pt, fp);
    else tr_read3<PROW, 2 * RP>(pt[0], fp[0]);
  };
  auto multiply = [&]() {
#pragma unroll
    for (int w = 2; w >= 0; --w)
#pragma unroll
      for (int c = 0; c < FC; ++c)
#pragma unroll
        for (int j = 0; j < FJ; ++j)
          acc[j][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp[j][w], fq[c], acc[j][c], 0, 0, 0);
  };
  // P's parts of step t, from buffer b, for both blocks of columns: a thread has 4 values
  auto make_parts = [&](int t, int b) {
    if (tid >= KR * RP / 4) return;
    const int m = tid / (RP / 4), j = 4 * (tid % (RP / 4));
    const uint32_t at = lds_at(ring) + b * SB + QB;
    floatx4 v;
    floatx2 sc;
    asm volatile("ds_read_b128 %0, %2\n"
                 "ds_read_b64 %1, %3\n"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(v), "=&v"(sc)
                 : "v"(at + 16 * tid), "v"(at + G::PB + 8 * m));
    const int piece = (j >> 3) ^ (NJ == 4 ? (m & 2) | (m & 8) >> 1 : 0);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint2 part[3];
      split4(v * sc[k], part);
      // (in assembly for the same reason as the reads; the barrier's wait counts them)
      asm volatile("ds_write_b64 %0, %1\n"
                   "ds_write_b64 %0, %2 offset:%4\n"
                   "ds_write_b64 %0, %3 offset:%5"
                   :
                   : "v"(split + ((t & 1) * 2 + k) * (KR * PROW) + m * PROW + (piece << 4) + (j & 4) * 2),
                     "v"(u32x2{part[0].x, part[0].y}), "v"(u32x2{part[1].x, part[1].y}),
                     "v"(u32x2{part[2].x, part[2].y}), "n"(2 * RP), "n"(4 * RP)
                   : "memory");
    }
  };
  const bool early = wave < 4;
  // X8: the parts of the next step are made in this one, so its copies have to be there
  constexpr int kFly = X8 ? ST - 3 : ST - 2;
  auto arrive = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(wait_vm(kFly * C) & kWaitLds);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  auto step = [&](int t, int b) {
    arrive();  // the copies are there, everybody's, and the reads of the step before are done
    copy((b + ST - 1) % ST);
    next_rows(t + ST);
    __builtin_amdgcn_sched_barrier(0);
    if (early) {
      if constexpr (X8 != 0) make_parts(t + 1, (b + 1) % ST);
      read(t, b);
      multiply();
    } else {
      if (t > 0) multiply();
      read(t, b);
      if constexpr (X8 != 0) make_parts(t + 1, (b + 1) % ST);
    }
  };
#pragma unroll
  for (int b = 0; b < ST - 1; ++b) {
    next_rows(b);
    copy(b);
  }
  next_rows(ST - 1);
  if constexpr (X8 != 0) {
    arrive();
    make_parts(0, 0);
  }
  for (int t = 0; t < steps; t += ST) {
    step(t, 0);
#pragma unroll
    for (int b = 1; b < ST; ++b)
      if (t + b < steps) step(t + b, b);
  }
  if (!early) multiply();
  const float s = tile.whole ? p.s[tile.a] : 1.f;
  const bool room = tile.whole || tile.part < (uint32_t)p.parts;  // else offsets that do not ascend
  float* out = tile.whole ? p.out + (int64_t)tile.a * r * N : p.part + (int64_t)tile.part * r * N;
#pragma unroll
  for (int j = 0; j < FJ; ++j)
#pragma unroll
    for (int c = 0; c < FC; ++c) {
      const int jj = j0 + 16 * (wj * FJ + j) + 4 * g;
      const int64_t cc = c0 + 16 * (wc * FC + c) + li;
      if (jj >= r || cc >= N || !room) continue;  // r % 4 == 0
      const floatx4 o = acc[j][c] * s;
      if (p.trans) {
        *(floatx4*)(out + cc * r + jj) = o;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) out[(jj + i) * N + cc] = o[i];
      }
    }
  __builtin_amdgcn_s_waitcnt(0);  // no copy is on its way into LDS that is no longer this workgroup's
}

// dL1's columns, then dL2's.
template <int X8, int NJ>
__global__ __launch_bounds__(512) void k_adapters_grad(AdapterRows rows, AdapterGrad p1, AdapterGrad p2) {
  using G = GradTile<X8, NJ>;
  using G0 = GradTile<0, NJ>;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[G::SMEM > G0::SMEM ? G::SMEM : G0::SMEM];
  __shared__ int list[G::LIST];
  const int n1 = (int)((p1.N + 255) / 256), cb = blockIdx.x;
  if (cb < n1) grad_tile<X8, NJ>(rows, p1, cb, ring, list);
  else grad_tile<0, NJ>(rows, p2, cb - n1, ring, list);
}

// Outputs of adapters with several items: their parts' sums in order; with none: zeros.
// Bound by the parts' bytes: 7 of 64 x 36864 and their sum, 76 MB, 15 us.
__global__ __launch_bounds__(256) void k_adapters_join(AdapterRows rows, AdapterGrad p0, AdapterGrad p1) {
  const AdapterGrad& p = blockIdx.z ? p1 : p0;
  const int a = blockIdx.y, lane = threadIdx.x & 63;
  const int M = (int)rows.M;
  // the parts before a's (an adapter of one item has none), and a's own items
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
    uint32_t sum = i < a && items > 1 ? items : 0;
#pragma unroll
    for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
    first += sum;
  }
  if (own == 1) return;
  const int64_t size = (int64_t)p.r * p.N;
  const float s = p.s[a];
  // (offsets that do not ascend: some items have no part)
  const uint32_t end = min(first + own, (uint32_t)p.parts);
  for (int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; e < size; e += (int64_t)gridDim.x * 1024) {
    floatx4 v = {0.f, 0.f, 0.f, 0.f};
    for (uint32_t i = first; i < end; ++i) v += *(const floatx4*)(p.part + i * size + e);
    *(floatx4*)(p.out + a * size + e) = own ? v * s : v;
  }
}

template <bool KMAJOR, int NJ>
hipError_t narrow_of(const AdapterNarrow& p, int bm, dim3 gr, hipStream_t st) {
  if (bm == 16) hipLaunchKernelGGL((k_adapters_narrow_few<KMAJOR, NJ>), gr, dim3(256), 0, st, p);
  else if (bm == 64) hipLaunchKernelGGL((k_adapters_narrow<KMAJOR, NJ, 1>), gr, dim3(256), 0, st, p);
  else hipLaunchKernelGGL((k_adapters_narrow<KMAJOR, NJ, 2>), gr, dim3(256), 0, st, p);
  return hipGetLastError();
}

hipError_t narrow(const AdapterCall& c, const AdapterPlan& pl, const uint16_t* A, int64_t K, const uint16_t* L,
                  bool kmajor, float* part, const Split3& split, hipStream_t st) {
  AdapterNarrow p{c.rows, A, L, K, c.r, pl.krange, part, (unsigned)pl.tiles, split};
  const int64_t more = split.to ? (c.rows.M + 63) / 64 : 0;
  const dim3 gr((unsigned)(pl.tiles + more), (unsigned)pl.splits, (unsigned)((c.r + 63) / 64));
  if (kmajor)
    return c.r <= 16   ? narrow_of<true, 1>(p, pl.bm, gr, st)
           : c.r <= 32 ? narrow_of<true, 2>(p, pl.bm, gr, st)
                       : narrow_of<true, 4>(p, pl.bm, gr, st);
  return c.r <= 16   ? narrow_of<false, 1>(p, pl.bm, gr, st)
         : c.r <= 32 ? narrow_of<false, 2>(p, pl.bm, gr, st)
                     : narrow_of<false, 4>(p, pl.bm, gr, st);
}

template <bool JMAJOR, int RW>
hipError_t wide_of(const AdapterWide& p, dim3 gr, hipStream_t st) {
  if (p.r <= 16) hipLaunchKernelGGL((k_adapters_wide<JMAJOR, 1, RW, 16>), gr, dim3(256), 0, st, p);
  else if (p.r <= 32) hipLaunchKernelGGL((k_adapters_wide<JMAJOR, 2, RW, 32>), gr, dim3(256), 0, st, p);
  else if (p.r <= 64) hipLaunchKernelGGL((k_adapters_wide<JMAJOR, 4, RW, 64>), gr, dim3(256), 0, st, p);
  // (with panels of 64 of L2's rows for each wave a compute unit would hold one workgroup: 1024
  // rows by 4096 of rank 128 26 us against 20)
  else if (p.r <= 128)
    hipLaunchKernelGGL((k_adapters_wide<JMAJOR, RW == 1 && JMAJOR ? 2 : 4, RW, 128>), gr, dim3(256), 0, st, p);
  else hipLaunchKernelGGL((k_adapters_wide<JMAJOR, 4, RW, 256>), gr, dim3(256), 0, st, p);
  return hipGetLastError();
}

hipError_t wide(const AdapterCall& c, const AdapterWidePlan& pl, const float* part, int splits, const uint16_t* L,
                bool jmajor, int64_t N, const uint16_t* base, uint16_t* out, float* T_out, const Split3& split,
                hipStream_t st) {
  AdapterWide p{c.rows, part, splits, L, N, c.r, c.s, base, out, T_out, pl.blocks, split};
  const int64_t nb = (N + 127) / 128;
  const dim3 gr((unsigned)pl.tiles, (unsigned)(pl.bm == 16 ? (nb + 3) / 4 : (nb + pl.blocks - 1) / pl.blocks));
  if (pl.bm == 16) return jmajor ? wide_of<true, 1>(p, gr, st) : wide_of<false, 1>(p, gr, st);
  return jmajor ? wide_of<true, 4>(p, gr, st) : wide_of<false, 4>(p, gr, st);
}

// The splits' sum, as it is, in three parts, or both: 4 splits of 16384 rows of rank 64 5.4 us.
// Where there are few values every workgroup of the next product adds the splits up by itself
// instead, which saves a launch.  `out` may be `part`.
__global__ __launch_bounds__(256) void k_adapters_sum(const float* part, int64_t size, int splits, int r, float* out,
                                                      Split3 split) {
  for (int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; e < size; e += (int64_t)gridDim.x * 1024) {
    const floatx4 v = join4(part + e, size, splits);
    if (out) *(floatx4*)(out + e) = v;
    if (!split.to) continue;
    uint2 three[3];
    split4(v, three);
    store3(split, e / r, (int)(e % r), three);
  }
}

hipError_t sum(const float* part, int64_t size, int splits, int r, float* out, const Split3& split, hipStream_t st) {
  // (2^20 workgroups at most: a launch's work-items stay below 2^32)
  const int64_t groups = std::min<int64_t>((size + 1023) / 1024, 1 << 20);
  hipLaunchKernelGGL(k_adapters_sum, dim3((unsigned)groups), dim3(256), 0, st, part, size, splits, r, out, split);
  return hipGetLastError();
}

template <int X8>
hipError_t grad_of(const AdapterRows& rows, const AdapterGrad& p1, const AdapterGrad& p2, hipStream_t st) {
  const dim3 gr((unsigned)((p1.N + 255) / 256 + (p2.N + 255) / 256), (unsigned)(p2.items + (p2.single ? rows.n : 0)),
                (unsigned)((p2.r + 63) / 64));
  if (p2.r <= 16) hipLaunchKernelGGL((k_adapters_grad<X8, 1>), gr, dim3(512), 0, st, rows, p1, p2);
  else if (p2.r <= 32) hipLaunchKernelGGL((k_adapters_grad<X8, 2>), gr, dim3(512), 0, st, rows, p1, p2);
  else hipLaunchKernelGGL((k_adapters_grad<X8, 4>), gr, dim3(512), 0, st, rows, p1, p2);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adapters_fwd(const AdapterCall& c, const uint16_t* X, const uint16_t* base, uint16_t* Y, float* T_out,
                               void* ws, hipStream_t st) {
  const AdapterPlan pl = plan_adapters_rows(c.rows.M, c.rows.n, c.h, false);
  if (const int groups = plan_adapters_few(c.rows.M, c.rows.n, c.h, c.o, c.r)) {
    const AdapterFew p{c.rows, X, c.L1, c.h, c.L2, c.o, c.r, c.s, base, Y, T_out};
    const dim3 gr((unsigned)pl.tiles, (unsigned)groups);  // (these tiles are of 16 rows: M <= 16 n)
    hipLaunchKernelGGL(k_adapters_few, gr, dim3(1024), 0, st, p);
    return hipGetLastError();
  }
  hipError_t e = narrow(c, pl, X, c.h, c.L1, true, (float*)ws, Split3{}, st);
  if (e != hipSuccess) return e;
  const AdapterWidePlan wp = plan_adapters_wide(c.rows.M, c.rows.n, c.o, c.r);
  float* const T = (float*)ws;
  const bool fold = plan_adapters_fold(c.rows.M, c.r, pl.splits, wp, c.o);
  if (!fold) e = sum(T, c.rows.M * c.r, pl.splits, c.r, T, Split3{}, st);
  if (e != hipSuccess) return e;
  return wide(c, wp, T, fold ? pl.splits : 1, c.L2, true, c.o, base, Y, T_out, Split3{}, st);
}

hipError_t launch_adapters_bwd(const AdapterCall& c, const void* X, int x8, const float* x_scales, const uint16_t* dY,
                               const float* T, const uint16_t* base, uint16_t* dX, float* dL1, float* dL2, void* ws,
                               hipStream_t st) {
  const AdapterPlan pl = plan_adapters_rows(c.rows.M, c.rows.n, c.o, true);
  const AdapterItems it = plan_adapters_items(c.rows.M, c.rows.n, c.h, c.o, c.r);
  const AdapterGradSpace sp = plan_adapters_space(c.rows.M, c.rows.n, c.h, c.o, c.r);
  uint8_t* const w = (uint8_t*)ws;
  float* const gparts = (float*)(w + sp.gparts);
  float* const parts = (float*)(w + sp.parts);
  const int nz = (c.r + 63) / 64, rp = c.r <= 16 ? 16 : c.r <= 32 ? 32 : 64;
  const Split3 t3{T, (uint16_t*)(w + sp.t3), w, nz, rp};
  // G for the products over rows: three parts, or fp32 beside 8-bit codes
  const Split3 g3{nullptr, x8 ? nullptr : (uint16_t*)(w + sp.g3), nullptr, nz, rp};
  float* const G = pl.splits > 1 ? (float*)(w + sp.g) : gparts;
  float* const G_out = pl.splits > 1 ? G : nullptr;
  hipError_t e = narrow(c, pl, dY, c.o, c.L2, false, gparts, t3, st);
  if (e != hipSuccess) return e;
  // G's splits are joined by a kernel of their own, or by dX's
  const AdapterWidePlan wp = plan_adapters_wide(c.rows.M, c.rows.n, c.h, c.r);
  if (dX && plan_adapters_fold(c.rows.M, c.r, pl.splits, wp, c.h)) {
    e = wide(c, wp, gparts, pl.splits, c.L1, false, c.h, base, dX, x8 ? G_out : nullptr, g3, st);
  } else {
    if (G_out || g3.to) e = sum(gparts, c.rows.M * c.r, pl.splits, c.r, G_out, g3, st);
    if (e != hipSuccess) return e;
    if (dX) e = wide(c, wp, G, 1, c.L1, false, c.h, base, dX, nullptr, Split3{}, st);
  }
  if (e != hipSuccess) return e;
  const AdapterGrad g1{X, x_scales, c.h, G, g3.to, c.r, c.s, it.item, it.items, it.parts, it.single, 1, parts, dL1, w};
  const AdapterGrad g2{dY, nullptr, c.o, nullptr, t3.to, c.r, c.s, it.item, it.items, it.parts, it.single, 0,
                       parts + it.parts * c.r * c.h, dL2, w};
  e = x8 == 0   ? grad_of<0>(c.rows, g1, g2, st)
      : x8 == 1 ? grad_of<1>(c.rows, g1, g2, st)
                : grad_of<2>(c.rows, g1, g2, st);
  if (e != hipSuccess || it.single) return e;
  const int64_t most = std::max(c.h, c.o) * c.r;
  const dim3 gr((unsigned)std::min<int64_t>((most + 1023) / 1024, 1024), (unsigned)c.rows.n, 2);
  hipLaunchKernelGGL(k_adapters_join, gr, dim3(256), 0, st, c.rows, g1, g2);
  return hipGetLastError();
}

}  // namespace nf4k
