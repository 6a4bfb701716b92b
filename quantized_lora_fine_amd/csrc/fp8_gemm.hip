// Block-scaled 8-bit matrix product on MFMA (gfx950), dense or grouped by expert.
//
//   C[m][n] = sum over blocks g of 128 k:  As[m][g] * Ws(n, g) * sum_{k in g} A[m][k] B[n][k]
//             + sum_j A2[m][j] B2[n][j]
//
// A is e4m3 or e5m2 with a scale per row and 128 k; B is the e4m3 weight
// [rows][cols] with a scale per 128 x 128 block, as stored (N = rows, K = cols)
// or, for the input gradient, contracted over its rows (N = cols, K = rows).
// A block's 128 products are one v_mfma_f32_16x16x128_f8f6f4 from a zero
// accumulator, so each block's fp32 sum is multiplied by its own scale when it
// is added to the fp32 result.  The weight's fragment is the first operand: a
// lane then holds one row m and four neighbouring n, its A scale is one
// register, and the W scale is one value per wave and step.
//
// Precision.  The instruction aligns the products of 8 neighbouring k to the
// largest of them, p, cuts each off below 2^-13 p, and adds these groups in fp32.
// That loss (2^-13 of a product, a few 2^-13 of a group at worst) is the price of
// the 8-bit rate and lies well below the codes' own rounding of 2^-4.
#include <algorithm>
#include <type_traits>

#include "fp8.hpp"
#include "launch.hpp"

namespace nf4k {

namespace {

constexpr uint32_t kRsrcFlags = 0x00020000u;  // raw buffer, gfx9-family dword3
constexpr uint32_t kOOB = 0x80000000u;        // an offset past every buffer's range

typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2* lds_i32x2_ptr;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, (int)kRsrcFlags);
}

struct Args {
  const uint8_t* A;
  const float* as;
  const uint8_t* W;
  const float* ws;
  const int32_t* offsets;
  const uint16_t* A2;
  const uint16_t* B2;
  uint16_t* C;
  int64_t M;
  int N, K, R;
  int experts;
  int tiles_n;
  float* part;  // [gridDim.y][M][N], where the contraction is split over gridDim.y workgroups
};

// This workgroup's blocks of the contraction: kb of them from kb0 on.
__device__ __forceinline__ void k_range(int blocks, int& kb0, int& kb) {
  kb0 = 0;
  kb = blocks;
  if (gridDim.y == 1) return;
  const uint32_t y = blockIdx.y;
  kb0 = (int)(blocks * y / gridDim.y);
  kb = (int)(blocks * (y + 1) / gridDim.y) - kb0;
}

// Tile `t` of a product grouped by expert: its expert and rows [m0, m1).  Every
// wave finds it by itself: 64 experts at a time, a scan of their tile counts.
// Offsets outside [0, M] are clamped, so no row outside the buffers is touched
// whatever they hold.
__device__ __forceinline__ bool find_tile(const Args& p, int bm, int t, int& e, int64_t& m0, int64_t& m1) {
  const int lane = threadIdx.x & 63;
  const int M = (int)p.M;
  uint32_t base = 0;  // (counts may wrap where offsets do not ascend; the rows stay inside all the same)
  for (int e0 = 0; e0 < p.experts; e0 += 64) {
    const int i = e0 + lane;
    int lo = 0, n = 0;
    if (i < p.experts) {
      lo = min(max(p.offsets[i], 0), M);
      n = max(min(max(p.offsets[i + 1], 0), M) - lo, 0);  // lo + n <= M
    }
    const uint32_t tiles = (uint32_t)(((int64_t)n + bm - 1) / bm);
    uint32_t incl = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t v = __shfl_up(incl, o);
      if (lane >= o) incl += v;
    }
    const uint64_t hit = __ballot(base + incl > (uint32_t)t);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      const uint32_t first = base + (uint32_t)__builtin_amdgcn_readlane((int)(incl - tiles), l);
      const int l0 = __builtin_amdgcn_readlane(lo, l), ln = __builtin_amdgcn_readlane(n, l);
      e = e0 + l;
      m0 = (int64_t)l0 + (int64_t)((uint32_t)t - first) * bm;
      m1 = min(m0 + bm, (int64_t)l0 + ln);
      return m0 < m1;
    }
    base += (uint32_t)__builtin_amdgcn_readlane((int)incl, 63);
  }
  return false;
}

// four neighbouring sums of a split contraction
__device__ __forceinline__ void store_part(const Args& p, int64_t m0, int mrows, int row, int n, floatx4 s) {
  if (row < mrows && n < p.N) *(floatx4*)(p.part + (blockIdx.y * p.M + m0 + row) * p.N + n) = s;
}

constexpr int kWaitLds = 15 | (3 << 14) | (0x7 << 4);  // lgkmcnt(0), vmcnt as it is
constexpr int wait_vm(int n) { return (n & 15) | ((n >> 4) << 14) | (0x7 << 4) | (0xF << 8); }

// The tile of this workgroup.  Workgroups are dealt to the 8 XCDs round-robin;
// ids are renumbered so that an XCD's run of 32 (as many as it holds at once)
// covers 4 row panels by 8 column tiles, which share those 12 panels in its L2.
// A grouped product does not use the last of its tiles, so there the runs of 32
// go to the XCDs in turn; a dense one gives each XCD one stretch.
__device__ __forceinline__ void tile_of(bool grouped, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int G = 4, U = 32;
  const int nwg = tiles_m * tiles_n;
  int id = blockIdx.x;
  if (grouped) {
    if (id < nwg / (8 * U) * (8 * U)) id = ((id >> 3) / U * 8 + (id & 7)) * U + (id >> 3) % U;
  } else if ((nwg & 7) == 0) {
    id = (id & 7) * (nwg >> 3) + (id >> 3);
  }
  const int grp = id / (G * tiles_n);
  const int gm = min(G, tiles_m - G * grp);
  const int gi = id - G * grp * tiles_n;
  tm = G * grp + gi % gm;
  tn = gi / gm;
}

// Tiles of 256, 128 or 64 rows by 256 columns (NI = 8, 4, 2) for products with enough
// of them: 8 waves, each 64 rows by 16 NI columns.  A step is one block of 128 k.
// Its fragments take LDS 16 (4 + NI) KB, its copies 4 (NI + 8) KB, its MFMAs 256 NI
// cycles: the 256 x 256 tile is the largest whose accumulators (128 registers) and
// two steps of operands (132 KB) fit, and the one that LDS holds up least.
// 16384 rows by 28672 x 8192: 3.3 ms, 2.35 PFLOP/s.  The chip runs at 1.6 GHz there
// (the power limit) with the matrix cores busy 63 % of the cycles; copies of the
// kernel without the multiply-adds of the scales are 17 % faster, without the copies
// of the operands 22 %, without the barriers 2 %.  The library's 8-bit product with
// one scale for a whole matrix takes 2.5 ms.
// 2048 rows by 4096 x 4096 (128 x 256 tiles, one a compute unit): 39 us with the weight
// in the caches, 41 from memory, 1.7 PFLOP/s.  No unit is full there: the matrix cores
// are busy 35 % of the cycles, LDS 21 %; of the waves' cycles a third go to
// instructions, 30 % to waits for copies, LDS and barriers, and in the rest a wave
// could go on but for the issue.
// Transposed, W's fragments are 8-byte transposing reads at half the rate of the
// 16-byte ones: 4096 rows by 11008 x 4096: 163 to 169 us, 2.2 PFLOP/s, the matrix cores
// busy 57 % of the cycles, LDS 38 % with 14 % of conflicts.
template <int NI, bool TR, bool E5M2, bool GROUPED>
__global__ __launch_bounds__(512, 2) void k_fp8_wide(Args p) {
  constexpr int WGM = NI / 2, NW = 8;  // 16 / NI waves beside each other
  constexpr int BM = 64 * WGM, BN = 256;
  constexpr int MI = 4;
  constexpr int WN = 16 * NI;  // columns of a wave
  constexpr int HW = WN / 2;   // and of a half of them
  constexpr int AI = BM / 64;  // 1 KB copies of A per wave
  // operand buffers: three where a step is short, so that copies run two steps
  // ahead; two 256 x 256 steps are all that fits.  W<step><half>
  constexpr int NB3 = NI == 8 ? 2 : 3;
  constexpr int X2 = NB3 == 3 ? 1 : 0;
  __shared__ __attribute__((aligned(1024))) uint8_t A0[BM * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t A1[BM * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t A2[X2 ? BM * 128 : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t W00[BN * 64];
  __shared__ __attribute__((aligned(1024))) uint8_t W01[BN * 64];
  __shared__ __attribute__((aligned(1024))) uint8_t W10[BN * 64];
  __shared__ __attribute__((aligned(1024))) uint8_t W11[BN * 64];
  __shared__ __attribute__((aligned(1024))) uint8_t W20[X2 ? BN * 64 : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t W21[X2 ? BN * 64 : 16];
  __shared__ __attribute__((aligned(1024))) float S0[NW * 64];
  __shared__ __attribute__((aligned(1024))) float S1[NW * 64];
  __shared__ __attribute__((aligned(1024))) float S2[X2 ? NW * 64 : 16];
  auto abuf = [&](int b) -> uint8_t* { return b == 0 ? A0 : b == 1 ? A1 : A2; };
  auto wbuf = [&](int b, int h) -> uint8_t* {
    return h == 0 ? (b == 0 ? W00 : b == 1 ? W10 : W20) : (b == 0 ? W01 : b == 1 ? W11 : W21);
  };
  auto sbuf = [&](int b) -> float* { return b == 0 ? S0 : b == 1 ? S1 : S2; };
  constexpr int SR = BM / NW;  // A scales a wave copies

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WGM, wn = wave / WGM;
  const int g = lane >> 4, l16 = lane & 15;

  const int tiles_m = (int)gridDim.x / p.tiles_n;
  int tm, tn;
  tile_of(GROUPED, tiles_m, p.tiles_n, tm, tn);
  const int n0 = tn * BN;
  const int N = p.N, K = p.K;
  const int KS = (K + 127) / 128;
  int kb0, KB;
  k_range(KS, kb0, KB);
  const int KL = K - kb0 * 128;  // columns from this workgroup's first on
  const int NB = (N + 127) / 128;
  int e = 0;
  int64_t m0, m1;
  if constexpr (GROUPED) {
    if (!find_tile(p, BM, tm, e, m0, m1)) return;
  } else {
    m0 = (int64_t)tm * BM;
    m1 = min(m0 + BM, p.M);
  }
  const int mrows = (int)(m1 - m0);
  const uint8_t* W = p.W + (GROUPED ? (int64_t)e * N * K : 0) + (TR ? (int64_t)kb0 * 128 * N : kb0 * 128);
  const float* ws = p.ws + (GROUPED ? (int64_t)e * NB * KS : 0) + (TR ? (int64_t)kb0 * NB : kb0);

  const __amdgpu_buffer_rsrc_t ar = make_rsrc(p.A + m0 * K + kb0 * 128, (uint32_t)((int64_t)mrows * K - kb0 * 128));
  const __amdgpu_buffer_rsrc_t sr = make_rsrc(p.as + m0 * KS + kb0, (uint32_t)(((int64_t)mrows * KS - kb0) * 4));
  const int nrows = min(BN, N - n0);
  // The buffer range covers the rows that exist, and its check takes the scalar
  // offset in, so one lane offset serves all of a wave's copies.
  const int c_row = wave * 8 + (lane >> 3);          // of copy i: plus i * 64
  const int c_chunk = (lane & 7) ^ (c_row & 7);      // the 16-byte chunk that goes to this lane's place
  const uint32_t a_off = (uint32_t)(c_row * K + c_chunk * 16);
  // half h of a W tile holds columns wn * WN + h * HW .. + HW - 1 of every wave
  // column, 128 in all
  uint32_t w_off;
  int col0 = 0;
  constexpr int CH = HW / 16;  // chunks of a wave column's half (TR)
  if constexpr (TR) {
    col0 = n0 + (c_chunk / CH) * WN + (c_chunk % CH) * 16;  // + h * HW
    w_off = (uint32_t)(c_row * N + col0);
  } else {
    w_off = (uint32_t)(((c_row / HW) * WN + c_row % HW) * K + c_chunk * 16);  // copy 1: + 128 rows
  }
  const uint32_t s_off = lane < SR ? (uint32_t)((wave * SR + lane) * KS * 4) : kOOB;
  // Steps behind the last one load its tile once more, so the loop has no
  // branches and every wait counts the same loads.
  auto copy_a = [&](int kt, int b, int i) {
    kt = min(kt, KB - 1);
    const uint32_t off = kt * 128 + c_chunk * 16 < KL ? a_off : kOOB;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(ar, (lds_ptr_t)(abuf(b) + (i * NW + wave) * 1024), 16, off,
                                             kt * 128 + i * 64 * K, 0, 0);
  };
  auto copy_s = [&](int kt, int b) {
    kt = min(kt, KB - 1);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(sr, (lds_ptr_t)(sbuf(b) + wave * 64), 4, s_off, kt * 4, 0, 0);
  };
  auto copy_w = [&](int kt, int b, int h, int i) {
    kt = min(kt, KB - 1);
    const lds_ptr_t to = (lds_ptr_t)(wbuf(b, h) + (i * NW + wave) * 1024);
    if constexpr (TR) {
      const __amdgpu_buffer_rsrc_t wr =
          make_rsrc(W + (int64_t)kt * 128 * N, (uint32_t)(min(128, KL - kt * 128) * (int64_t)N));
      const uint32_t off = col0 + h * HW < N ? w_off : kOOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, to, 16, off, h * HW + i * 64 * N, 0, 0);
    } else {
      const __amdgpu_buffer_rsrc_t wr = make_rsrc(W + (int64_t)n0 * K, (uint32_t)((int64_t)nrows * K - kb0 * 128));
      const uint32_t off = kt * 128 + c_chunk * 16 < KL ? w_off : kOOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, to, 16, off, kt * 128 + (i * 128 + h * HW) * K, 0, 0);
    }
  };
  const int nb = min((n0 + wn * WN) >> 7, NB - 1);
  auto load_ws = [&](int kt) -> float {
    const int k = min(kt + lane, KB - 1);
    return TR ? ws[(int64_t)k * NB + nb] : ws[(int64_t)nb * KS + k];
  };

  // LDS places of this lane's fragment pieces; subtile i adds 2 KB, or (TR) flips
  // the slot bits
  uint32_t f_lo, f_hi;
  if constexpr (TR) {
    const int x = l16 >> 1;
    f_lo = (uint32_t)((16 * g + x) * 128 + (((wn * CH) ^ x) << 4) + (l16 & 1) * 8);
    f_hi = f_lo + 8 * 128;
  } else {
    f_lo = (uint32_t)((wn * HW + l16) * 128 + ((g ^ (l16 & 7)) << 4));
    f_hi = f_lo ^ 64;
  }
  auto frag_w = [&](uint8_t* Wb, int i) -> i32x8 {  // i: 0 .. NI / 2 - 1 of the half
    if constexpr (TR) {
      i32x8 f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const i32x2 v = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (lds_i32x2_ptr)(Wb + (f_lo ^ (uint32_t)(i << 4)) + (q & 1) * 8 * 128 + (q >> 1) * 64 * 128));
        f[2 * q] = v.x;
        f[2 * q + 1] = v.y;
      }
      return f;
    } else {
      const u32x4 lo = *(const u32x4*)(Wb + f_lo + i * 2048);
      const u32x4 hi = *(const u32x4*)(Wb + f_hi + i * 2048);
      return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
    }
  };
  const uint32_t fa_lo = (uint32_t)((wm * 64 + l16) * 128 + ((g ^ (l16 & 7)) << 4));
  const uint32_t fa_hi = fa_lo ^ 64;
  auto frag_a = [&](const uint8_t* Ab, int i) -> i32x8 {
    const u32x4 lo = *(const u32x4*)(Ab + fa_lo + i * 2048);
    const u32x4 hi = *(const u32x4*)(Ab + fa_hi + i * 2048);
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  };
  // A scale of row r of the tile: copied by wave r / SR, lane r % SR
  auto read_s = [&](const float* Sb, float (&s)[MI]) {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int r = wm * 64 + i * 16 + l16;
      s[i] = Sb[(r / SR) * 64 + r % SR];
    }
  };

  floatx4 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};

  // A step is NI groups of 4 MFMAs, one group per 16 columns, in two halves with a
  // barrier before each.  The group's W fragment is read during the group before
  // it; the next step's A fragments replace this step's as the last group is done
  // with them; the multiply-adds of a group run beside the next one's MFMAs.
  // Copies, B the number of buffers:
  //   before the 1st half of step kt: the 2nd half of W (kt + B - 1),
  //   before the 2nd half:            A, its scales and the 1st half of W (kt + B),
  // each into memory whose readers that barrier has seen through, and B - 1 steps
  // before the barrier that waits for it.
  auto barrier = [&](auto outstanding) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(wait_vm(decltype(outstanding)::value));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  constexpr int C0 = 2, C1 = 3 + AI;  // copies issued before a 1st and a 2nd half
  constexpr std::integral_constant<int, (NB3 - 1) * C1 + (NB3 - 2) * C0> kHalf1{};  // may be under way at a 1st half
  constexpr std::integral_constant<int, (NB3 - 1) * C0 + (NB3 - 2) * C1> kHalf0{};  // and at a 2nd half
  i32x8 fa[MI], fw[2];
  floatx4 d[2][MI];
  float s[MI], sc[MI];
  float wsr = load_ws(0);
  auto fold = [&](int j, floatx4 (&dd)[MI]) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[i][j][v] = __builtin_fmaf(dd[i][v], sc[i], acc[i][j][v]);
  };
  auto step = [&](int kt, int b) {  // b = kt % NB3, a constant in every copy of the step
    uint8_t* const An = abuf((b + 1) % NB3);
    uint8_t* const Wc0 = wbuf(b, 0);
    uint8_t* const Wc1 = wbuf(b, 1);
    uint8_t* const Wn0 = wbuf((b + 1) % NB3, 0);
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      if (j == 0) barrier(kHalf1);
      if (j == NI / 2) barrier(kHalf0);
      __builtin_amdgcn_sched_barrier(0);
      fw[(j + 1) & 1] = j + 1 < NI / 2 ? frag_w(Wc0, j + 1) : j + 1 < NI ? frag_w(Wc1, j + 1 - NI / 2) : frag_w(Wn0, 0);
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        d[j & 1][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw[j & 1], fa[i], floatx4{0.f, 0.f, 0.f, 0.f}, 0,
                                                                       E5M2 ? 1 : 0, 0, 0, 0, 0);
        if (j == NI - 1) fa[i] = frag_a(An, i);
      }
      // the group before this one (of the step before: its scales are still in sc)
      fold((j + NI - 1) % NI, d[(j + 1) & 1]);
      if (j == 0) {
        const float w = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wsr), kt & 63));
#pragma unroll
        for (int i = 0; i < MI; ++i) sc[i] = s[i] * w;
      }
      if (j == NI - 1) read_s(sbuf((b + 1) % NB3), s);
#pragma unroll
      for (int i = 0; i < MI; ++i) asm volatile("" : "+v"(acc[i][(j + NI - 1) % NI]));
      __builtin_amdgcn_sched_group_barrier(0x100, TR ? 4 : 2, 0);
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
      // this half's copies, spread over its groups: a burst would hold up every wave
      constexpr int H = NI / 2;
      if (j < H) {
#pragma unroll
        for (int c = j * C0 / H; c < (j + 1) * C0 / H; ++c) copy_w(kt + NB3 - 1, (b + NB3 - 1) % NB3, 1, c);
      } else {
#pragma unroll
        for (int c = (j - H) * C1 / H; c < (j - H + 1) * C1 / H; ++c) {
          if (c < 2) copy_w(kt + NB3, b, 0, c);
          else if (c < 2 + AI) copy_a(kt + NB3, b, c - 2);
          else copy_s(kt + NB3, b);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (((kt + 1) & 63) == 0) {
      wsr = load_ws(kt + 1);
      // waited for here, or every step's use would wait for the copies under way
      __builtin_amdgcn_s_waitcnt(wait_vm(0));
    }
  };
  // in the order that the loop would have issued them
  auto first = [&](int b) {
#pragma unroll
    for (int c = 0; c < 2; ++c) copy_w(b, b, 0, c);
#pragma unroll
    for (int c = 0; c < AI; ++c) copy_a(b, b, c);
    copy_s(b, b);
  };
  first(0);
#pragma unroll
  for (int b = 1; b < NB3; ++b) {
#pragma unroll
    for (int c = 0; c < 2; ++c) copy_w(b - 1, b - 1, 1, c);
    first(b);
  }
  barrier(kHalf1);
  fw[0] = frag_w(W00, 0);
#pragma unroll
  for (int i = 0; i < MI; ++i) fa[i] = frag_a(A0, i);
  read_s(S0, s);
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    sc[i] = 0.f;
    d[1][i] = floatx4{0.f, 0.f, 0.f, 0.f};
  }
  int kt = 0;
  for (; kt + NB3 <= KB; kt += NB3) {
#pragma unroll
    for (int b = 0; b < NB3; ++b) step(kt + b, b);
  }
  if (kt < KB) step(kt, 0);
  if (NB3 == 3 && kt + 1 < KB) step(kt + 1, 1);
  fold(NI - 1, d[(NI - 1) & 1]);
  __builtin_amdgcn_s_waitcnt(wait_vm(0));

  if (p.R && blockIdx.y == 0) {
    const __amdgpu_buffer_rsrc_t a2 = make_rsrc(p.A2 + m0 * p.R, (uint32_t)((int64_t)mrows * p.R * 2));
    const __amdgpu_buffer_rsrc_t b2 =
        make_rsrc(p.B2 + ((GROUPED ? (int64_t)e * N : 0) + n0) * p.R, (uint32_t)((int64_t)nrows * p.R * 2));
    for (int k0 = 0; k0 < p.R; k0 += 32) {
      const int k = k0 + 8 * g;
      bf16x8 fa[MI];
#pragma unroll
      for (int i = 0; i < MI; ++i)
        fa[i] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(
            a2, k < p.R ? (uint32_t)(((wm * 64 + i * 16 + l16) * p.R + k) * 2) : kOOB, 0, 0));
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const bf16x8 fbb = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(
            b2, k < p.R ? (uint32_t)(((wn * WN + j * 16 + l16) * p.R + k) * 2) : kOOB, 0, 0));
#pragma unroll
        for (int i = 0; i < MI; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fbb, fa[i], acc[i][j], 0, 0, 0);
      }
    }
  }

  if (gridDim.y > 1) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
        store_part(p, m0, mrows, wm * 64 + i * 16 + l16, n0 + wn * WN + j * 16 + 4 * g, acc[i][j]);
    return;
  }
  __syncthreads();
  // the result tile of a wave in its own part of the operand buffers
  constexpr int WB = 64 * WN * 2, PA = BM * 128 / WB, PW = 16384 / WB;
  static_assert(2 * PA + 4 * PW >= NW, "the result tile fits");
  uint8_t* st;
  if (wave < PA) st = A0 + wave * WB;
  else if (wave < 2 * PA) st = A1 + (wave - PA) * WB;
  else {
    const int q = wave - 2 * PA;
    st = (q / PW == 0 ? W00 : q / PW == 1 ? W01 : q / PW == 2 ? W10 : W11) + (q % PW) * WB;
  }
  constexpr int PC = WN / 8;  // 16-byte pieces of a row
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int r = i * 16 + l16;
      const int piece = j * 2 + (g >> 1);
      uint2 o;
      o.x = pack_bf16x2(acc[i][j][0], acc[i][j][1]);
      o.y = pack_bf16x2(acc[i][j][2], acc[i][j][3]);
      *(uint2*)(st + r * (WN * 2) + ((piece ^ (r & (PC - 1))) << 4) + (g & 1) * 8) = o;
    }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < PC; ++q) {
    const int o = q * 64 + lane;
    const int r = o / PC, piece = o % PC;
    const int row = wm * 64 + r;
    const int n = n0 + wn * WN + piece * 8;
    if (row < mrows && n < N)
      *(u32x4*)(p.C + (m0 + row) * N + n) = *(const u32x4*)(st + r * (WN * 2) + ((piece ^ (r & (PC - 1))) << 4));
  }
}

// Few rows, or few tiles.  A workgroup makes a tile of 16 MT rows by 16 NT columns;
// its NWV waves take every NWV-th block of the contraction and join their sums
// through LDS in a fixed order at the end.  A wave stages its own operands: rows
// of 128 bytes (TR: k rows of 64 bytes) copied straight into its part of LDS, ST
// rounds in flight, so the loop has no barrier.  (Fragments loaded from memory
// into registers take four times as long: the address path joins neighbouring
// lanes only, and a fragment's neighbouring lanes are different rows.)
// One row by 28672 x 8192: 40 to 42 us with the weight out of the caches, 5.6 TB/s,
// what a copy reaches; by 4096 x 4096 5.4 to 5.6 us, of which the launch and the first
// loads are 3.  Transposed a workgroup's time goes with its k rows (1.5 ns each, whatever
// it takes of a row's 128-byte line), so few rows are slower there: 3 rows by
// 11008 x 4096 39 us with the weight out of the caches, 20 with the contraction split
// over 3.  32 or 128 bytes of each k row instead of 64 are within 10 % of it either way,
// and copies issued before a round's products instead of after are no faster.
template <int MT, int NT, int NWV, int ST, bool TR, bool SPLIT, bool E5M2, bool GROUPED>
__global__ __launch_bounds__(NWV * 64) void k_fp8_rows(Args p) {
  static_assert(!TR || NT == 4, "64 bytes of each k row");
  constexpr int BM = 16 * MT, BN = 16 * NT;
  constexpr int WB = (MT + NT) * 2048 + 256;  // a wave's bytes of one round: A, W, A scales
  constexpr int WOFF = MT * 2048, SOFF = (MT + NT) * 2048;
  __shared__ __attribute__((aligned(1024))) uint8_t L0[NWV * WB];
  __shared__ __attribute__((aligned(1024))) uint8_t L1[NWV * WB];
  __shared__ __attribute__((aligned(1024))) uint8_t L2[ST > 2 ? NWV * WB : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t L3[ST > 3 ? NWV * WB : 16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, l16 = lane & 15;
  const int tiles_m = (int)gridDim.x / p.tiles_n;
  int id = blockIdx.x;
  if constexpr (GROUPED) {
    // runs of 8 column tiles to the XCDs in turn: the last tiles may have no rows, so
    // one stretch for each XCD would leave some without work (64 experts of
    // 1536 x 4096, 48 rows: 34 us against 42; 1 row of room for 200: 10 against 23)
    constexpr int U = 8;
    if (id < (int)gridDim.x / (8 * U) * (8 * U)) id = ((id >> 3) / U * 8 + (id & 7)) * U + (id >> 3) % U;
  } else if ((gridDim.x & 7) == 0) {
    id = (id & 7) * (gridDim.x >> 3) + (id >> 3);
  }
  const int tm = GROUPED ? id / p.tiles_n : id % tiles_m;
  const int n0 = (GROUPED ? id % p.tiles_n : id / tiles_m) * BN;
  const int N = p.N, K = p.K;
  const int KS = (K + 127) / 128;
  int kb0 = 0, KB = KS;
  if constexpr (SPLIT) k_range(KS, kb0, KB);
  const int KL = K - kb0 * 128;  // columns from this workgroup's first on
  const int NB = (N + 127) / 128;
  int e = 0;
  int64_t m0, m1;
  if constexpr (GROUPED) {
    if (!find_tile(p, BM, tm, e, m0, m1)) return;
  } else {
    m0 = (int64_t)tm * BM;
    m1 = min(m0 + BM, p.M);
  }
  const int mrows = (int)(m1 - m0);
  const int nrows = min(BN, N - n0);
  const uint8_t* W = p.W + (GROUPED ? (int64_t)e * N * K : 0) + (TR ? (int64_t)kb0 * 128 * N : kb0 * 128);
  const float* ws = p.ws + (GROUPED ? (int64_t)e * NB * KS : 0) + (TR ? (int64_t)kb0 * NB : kb0);
  const __amdgpu_buffer_rsrc_t ar = make_rsrc(p.A + m0 * K + kb0 * 128, (uint32_t)((int64_t)mrows * K - kb0 * 128));
  const __amdgpu_buffer_rsrc_t sr = make_rsrc(p.as + m0 * KS + kb0, (uint32_t)(((int64_t)mrows * KS - kb0) * 4));

  // copies: 8 lanes a row, chunks XORed with the row's low bits (see k_fp8_wide)
  const int c_row = lane >> 3, c_k = ((lane & 7) ^ c_row) * 16;
  const uint32_t a_off = (uint32_t)(c_row * K + c_k);
  // TR: 4 lanes a k row, chunk c of row r at place c ^ (r / 4 % 4)
  const int t_row = lane >> 2;
  const int t_col = n0 + ((lane & 3) ^ ((t_row >> 2) & 3)) * 16;
  const uint32_t t_off = t_col < N ? (uint32_t)(t_row * N + t_col) : kOOB;
  // (a branch around the other lanes would make the compiler's own waits count this
  // load as one that may not be there)
  const uint32_t s_off = lane < BM ? (uint32_t)(lane * KS * 4) : kOOB;
  auto lbuf = [&](int b) -> uint8_t* { return (b == 0 ? L0 : b == 1 ? L1 : b == 2 ? L2 : L3) + wave * WB; };
  constexpr int LOADS = 2 * MT + 2 * NT + 1;
  auto copy = [&](int kt, int b) {
    kt = min(kt, KB - 1);  // a round behind the last copies it once more, and is not used
    uint8_t* const to = lbuf(b);
    const bool in = kt * 128 + c_k < KL;
    const uint32_t off = in ? a_off : kOOB;
    if constexpr (TR) {
      const __amdgpu_buffer_rsrc_t wr =
          make_rsrc(W + (int64_t)kt * 128 * N, (uint32_t)(min(128, KL - kt * 128) * (int64_t)N));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, (lds_ptr_t)(to + WOFF + i * 1024), 16, t_off, i * 16 * N, 0, 0);
    } else {
      const __amdgpu_buffer_rsrc_t wr = make_rsrc(W + (int64_t)n0 * K, (uint32_t)((int64_t)nrows * K - kb0 * 128));
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, (lds_ptr_t)(to + WOFF + i * 1024), 16, off, kt * 128 + i * 8 * K,
                                                 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ar, (lds_ptr_t)(to + i * 1024), 16, off, kt * 128 + i * 8 * K, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(sr, (lds_ptr_t)(to + SOFF), 4, s_off, kt * 4, 0, 0);
  };
  // W scales of this wave's rounds, one a lane
  const int nb = n0 >> 7;
  auto load_ws = [&](int r) -> float {
    const int k = min((r + lane) * NWV + wave, KB - 1);
    return TR ? ws[(int64_t)k * NB + nb] : ws[(int64_t)nb * KS + k];
  };

  floatx4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  const uint32_t f_lo = (uint32_t)(l16 * 128 + ((g ^ (l16 & 7)) << 4));
  auto frag = [&](const uint8_t* at) -> i32x8 {
    const u32x4 lo = *(const u32x4*)(at + f_lo);
    const u32x4 hi = *(const u32x4*)(at + (f_lo ^ 64));
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  };
  auto frag_t = [&](uint8_t* at, int j) -> i32x8 {  // k rows of 64 bytes
    i32x8 f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = (q >> 1) * 64 + 16 * g + (q & 1) * 8 + (l16 >> 1);
      const i32x2 v = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
          (lds_i32x2_ptr)(at + r * 64 + ((j ^ ((r >> 2) & 3)) << 4) + (l16 & 1) * 8));
      f[2 * q] = v.x;
      f[2 * q + 1] = v.y;
    }
    return f;
  };

  const int rounds = (KB - wave + NWV - 1) / NWV;  // of this wave; 0 when it has none
  float wsr = load_ws(0);
#pragma unroll
  for (int b = 0; b < ST - 1; ++b) copy(b * NWV + wave, b);
  auto round = [&](int r, int b) {
    copy((r + ST - 1) * NWV + wave, (b + ST - 1) % ST);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(wait_vm((ST - 1) * LOADS));  // all but the rounds ahead
    asm volatile("" ::: "memory");
    uint8_t* const at = lbuf(b);
    const float w = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wsr), r & 63));
    i32x8 fw[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) fw[j] = TR ? frag_t(at + WOFF, j) : frag(at + WOFF + j * 2048);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const i32x8 fa = frag(at + i * 2048);
      const float s = *(const float*)(at + SOFF + (i * 16 + l16) * 4) * w;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const floatx4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw[j], fa, floatx4{0.f, 0.f, 0.f, 0.f}, 0,
                                                                           E5M2 ? 1 : 0, 0, 0, 0, 0);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][j][v] = __builtin_fmaf(d[v], s, acc[i][j][v]);
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) asm volatile("" : "+v"(acc[i][j]));
    // the reads of this round are done before its memory is copied to again
    __builtin_amdgcn_s_waitcnt(kWaitLds);
    if (((r + 1) & 63) == 0) {
      wsr = load_ws(r + 1);
      __builtin_amdgcn_s_waitcnt(wait_vm(0));
    }
  };
  int r = 0;
  for (; r + ST <= rounds; r += ST) {
#pragma unroll
    for (int b = 0; b < ST; ++b) round(r + b, b);
  }
#pragma unroll
  for (int b = 0; b < ST - 1; ++b)
    if (r + b < rounds) round(r + b, b);
  __builtin_amdgcn_s_waitcnt(wait_vm(0));

  // the low-rank term: runs of 32 of its columns, dealt to the waves
  for (int k0 = wave * 32; k0 < (SPLIT && blockIdx.y ? 0 : p.R); k0 += NWV * 32) {
    const __amdgpu_buffer_rsrc_t a2 = make_rsrc(p.A2 + m0 * p.R, (uint32_t)((int64_t)mrows * p.R * 2));
    const __amdgpu_buffer_rsrc_t b2 =
        make_rsrc(p.B2 + ((GROUPED ? (int64_t)e * N : 0) + n0) * p.R, (uint32_t)((int64_t)nrows * p.R * 2));
    const int k = k0 + 8 * g;
    const uint32_t o = k < p.R ? (uint32_t)((l16 * p.R + k) * 2) : kOOB;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const bf16x8 fb = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(b2, o, j * 16 * p.R * 2, 0));
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const bf16x8 fa = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(a2, o, i * 16 * p.R * 2, 0));
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb, fa, acc[i][j], 0, 0, 0);
      }
    }
  }

  __syncthreads();  // every wave is done with its rounds: their memory holds the sums
  static_assert(MT * NT * 1024 <= WB, "a wave's sums fit its part");
  floatx4* const part = (floatx4*)L0;
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) part[(wave * MT * NT + i * NT + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  for (int q = threadIdx.x; q < MT * NT * 64; q += NWV * 64) {
    const int t = q >> 6, l = q & 63;
    floatx4 s = part[q];
#pragma unroll
    for (int w = 1; w < NWV; ++w) s += part[w * MT * NT * 64 + q];
    const int row = t / NT * 16 + (l & 15);
    const int n = n0 + t % NT * 16 + 4 * (l >> 4);
    if constexpr (SPLIT) store_part(p, m0, mrows, row, n, s);
    else if (row < mrows && n < N)
      *(uint2*)(p.C + (m0 + row) * N + n) = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
  }
}

// Tiles of 128 x 128 and 128 x 64, not transposed, for products whose 256-column
// tiles would leave compute units without one.  8 waves share the operands of a
// step, which go through a ring of ST buffers, ST - 1 steps under way.  A step has
// one barrier; its fragments were read during the step before it.  Bound by LDS: a
// step of a 128 x 64 tile takes 0.33 us, of which 64 KB of fragments and 24 KB of
// copies are 0.3.  (4 waves with tiles twice as large read less, but wait for
// themselves: 0.53 us.  64 x 64 tiles, 0.20 us, are no better than k_fp8_rows';
// transposed, the 8-byte reads of W make a step 0.75 us, more than k_fp8_rows
// needs.)  With the weight out of the caches 128 rows by 9104 x 5888 take 33 us, 415
// TFLOP/s, against 39 for the best of the other tiles; with it in them 512 rows by
// 4096 x 4096 18 us against 23.
template <int BM, int BN, int ST, bool E5M2, bool GROUPED>
__global__ __launch_bounds__(512) void k_fp8_ring(Args p) {
  constexpr int NW = 8;
  constexpr int WR = BN == 64 ? 4 : 2, WC = NW / WR;  // waves below and beside each other
  constexpr int MI = BM / WR / 16, NI = BN / WC / 16;
  constexpr int AI = BM / 64, WI = BN / 64;  // 1 KB copies of a wave and step
  constexpr int SR = BM / NW;                // A scales a wave copies
  constexpr int WOFF = BM * 128, SOFF = WOFF + BN * 128, SB = SOFF + NW * 256;
  static_assert(ST % 2 == 0, "the fragments' registers alternate with the buffers");
  __shared__ __attribute__((aligned(1024))) uint8_t L0[SB];
  __shared__ __attribute__((aligned(1024))) uint8_t L1[SB];
  __shared__ __attribute__((aligned(1024))) uint8_t L2[SB];
  __shared__ __attribute__((aligned(1024))) uint8_t L3[SB];
  __shared__ __attribute__((aligned(1024))) uint8_t L4[ST > 4 ? SB : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t L5[ST > 4 ? SB : 16];
  auto lbuf = [&](int b) -> uint8_t* {
    return b == 0 ? L0 : b == 1 ? L1 : b == 2 ? L2 : b == 3 ? L3 : b == 4 ? L4 : L5;
  };
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WR, wn = wave / WR;
  const int g = lane >> 4, l16 = lane & 15;
  const int tiles_m = (int)gridDim.x / p.tiles_n;
  int tm, tn;
  tile_of(GROUPED, tiles_m, p.tiles_n, tm, tn);
  const int n0 = tn * BN;
  const int N = p.N, K = p.K;
  const int KS = (K + 127) / 128;
  int kb0, KB;
  k_range(KS, kb0, KB);
  const int KL = K - kb0 * 128;  // columns from this workgroup's first on
  const int NB = (N + 127) / 128;
  int e = 0;
  int64_t m0, m1;
  if constexpr (GROUPED) {
    if (!find_tile(p, BM, tm, e, m0, m1)) return;
  } else {
    m0 = (int64_t)tm * BM;
    m1 = min(m0 + BM, p.M);
  }
  const int mrows = (int)(m1 - m0);
  const int nrows = min(BN, N - n0);
  const uint8_t* W = p.W + (GROUPED ? (int64_t)e * N * K : 0) + kb0 * 128;
  const float* ws = p.ws + (GROUPED ? (int64_t)e * NB * KS : 0) + kb0;
  const __amdgpu_buffer_rsrc_t ar = make_rsrc(p.A + m0 * K + kb0 * 128, (uint32_t)((int64_t)mrows * K - kb0 * 128));
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(W + (int64_t)n0 * K, (uint32_t)((int64_t)nrows * K - kb0 * 128));
  const __amdgpu_buffer_rsrc_t sr = make_rsrc(p.as + m0 * KS + kb0, (uint32_t)(((int64_t)mrows * KS - kb0) * 4));

  // copies and fragments as in k_fp8_wide
  const int c_row = wave * 8 + (lane >> 3);  // of copy i: plus i * 64
  const int c_chunk = (lane & 7) ^ (c_row & 7);
  const uint32_t c_off = (uint32_t)(c_row * K + c_chunk * 16);
  const uint32_t s_off = lane < SR ? (uint32_t)((wave * SR + lane) * KS * 4) : kOOB;
  constexpr int C = AI + WI + 1;  // loads a step
  auto copy = [&](int kt, int b) {
    kt = min(kt, KB - 1);  // a step behind the last copies it once more, and is not used
    uint8_t* const to = lbuf(b);
    const uint32_t off = kt * 128 + c_chunk * 16 < KL ? c_off : kOOB;
#pragma unroll
    for (int i = 0; i < AI; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ar, (lds_ptr_t)(to + (i * NW + wave) * 1024), 16, off,
                                               kt * 128 + i * 64 * K, 0, 0);
#pragma unroll
    for (int i = 0; i < WI; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, (lds_ptr_t)(to + WOFF + (i * NW + wave) * 1024), 16, off,
                                               kt * 128 + i * 64 * K, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(sr, (lds_ptr_t)(to + SOFF + wave * 256), 4, s_off, kt * 4, 0, 0);
  };
  const int nb = n0 >> 7;
  auto load_ws = [&](int kt) -> float {
    return ws[(int64_t)nb * KS + min(kt + lane, KB - 1)];
  };

  constexpr int WN = BN / WC;  // columns of a wave
  const uint32_t fa_at = (uint32_t)((wm * MI * 16 + l16) * 128 + ((g ^ (l16 & 7)) << 4));
  const uint32_t fw_at = (uint32_t)((wn * WN + l16) * 128 + ((g ^ (l16 & 7)) << 4));
  auto frag = [&](const uint8_t* at, uint32_t o, int i) -> i32x8 {
    const u32x4 lo = *(const u32x4*)(at + o + i * 2048);
    const u32x4 hi = *(const u32x4*)(at + (o ^ 64) + i * 2048);
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  };
  floatx4 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  i32x8 fa[2][MI], fw[2][NI];
  float s[2][MI];
  auto read = [&](int b, int x) {
    uint8_t* const at = lbuf(b);
#pragma unroll
    for (int j = 0; j < NI; ++j) fw[x][j] = frag(at + WOFF, fw_at, j);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      fa[x][i] = frag(at, fa_at, i);
      const int r = (wm * MI + i) * 16 + l16;
      s[x][i] = *(const float*)(at + SOFF + r / SR * 256 + r % SR * 4);
    }
  };
  // every wave's copies but those of the `ahead` newest steps are there, and every
  // wave's reads so far are done
  auto barrier = [&](auto ahead) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(wait_vm(decltype(ahead)::value * C) & kWaitLds);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  float wsr = load_ws(0);
#pragma unroll
  for (int b = 0; b < ST; ++b) copy(b, b);
  barrier(std::integral_constant<int, ST - 1>{});
  read(0, 0);
  auto step = [&](int kt, int b) {
    const int x = b & 1;
    __builtin_amdgcn_sched_barrier(0);
    barrier(std::integral_constant<int, ST - 2>{});  // step kt + 1 is there, the reads of step kt are done
    copy(kt + ST, b);
    __builtin_amdgcn_sched_barrier(0);
    read((b + 1) % ST, x ^ 1);
    const float w = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wsr), kt & 63));
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const float sc = s[x][i] * w;
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const floatx4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            fw[x][j], fa[x][i], floatx4{0.f, 0.f, 0.f, 0.f}, 0, E5M2 ? 1 : 0, 0, 0, 0, 0);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][j][v] = __builtin_fmaf(d[v], sc, acc[i][j][v]);
      }
    }
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) asm volatile("" : "+v"(acc[i][j]));
    if (((kt + 1) & 63) == 0) {
      wsr = load_ws(kt + 1);
      __builtin_amdgcn_s_waitcnt(wait_vm(0));
    }
  };
  int kt = 0;
  for (; kt + ST <= KB; kt += ST) {
#pragma unroll
    for (int b = 0; b < ST; ++b) step(kt + b, b);
  }
#pragma unroll
  for (int b = 0; b < ST - 1; ++b)
    if (kt + b < KB) step(kt + b, b);
  __builtin_amdgcn_s_waitcnt(wait_vm(0));

  if (p.R && blockIdx.y == 0) {
    const __amdgpu_buffer_rsrc_t a2 = make_rsrc(p.A2 + m0 * p.R, (uint32_t)((int64_t)mrows * p.R * 2));
    const __amdgpu_buffer_rsrc_t b2 =
        make_rsrc(p.B2 + ((GROUPED ? (int64_t)e * N : 0) + n0) * p.R, (uint32_t)((int64_t)nrows * p.R * 2));
    for (int k0 = 0; k0 < p.R; k0 += 32) {
      const int k = k0 + 8 * g;
      bf16x8 fb[NI];
#pragma unroll
      for (int j = 0; j < NI; ++j)
        fb[j] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(
            b2, k < p.R ? (uint32_t)(((wn * WN + j * 16 + l16) * p.R + k) * 2) : kOOB, 0, 0));
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const bf16x8 f = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(
            a2, k < p.R ? (uint32_t)((((wm * MI + i) * 16 + l16) * p.R + k) * 2) : kOOB, 0, 0));
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], f, acc[i][j], 0, 0, 0);
      }
    }
  }

  if (gridDim.y > 1) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
        store_part(p, m0, mrows, (wm * MI + i) * 16 + l16, n0 + wn * WN + j * 16 + 4 * g, acc[i][j]);
    return;
  }
  __syncthreads();  // every wave is done with the buffers: the result tile goes through the first
  constexpr int PC = BN / 8;  // 16-byte pieces of a row
  static_assert(BM * BN * 2 <= SB, "the result tile fits");
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int r = (wm * MI + i) * 16 + l16;
      const int piece = wn * (WN / 8) + j * 2 + (g >> 1);
      uint2 o;
      o.x = pack_bf16x2(acc[i][j][0], acc[i][j][1]);
      o.y = pack_bf16x2(acc[i][j][2], acc[i][j][3]);
      *(uint2*)(L0 + r * (BN * 2) + ((piece ^ (r & (PC - 1))) << 4) + (g & 1) * 8) = o;
    }
  __syncthreads();
#pragma unroll
  for (int q = threadIdx.x; q < BM * PC; q += 512) {
    const int r = q / PC, piece = q % PC;
    const int n = n0 + piece * 8;
    if (r < mrows && n < N)
      *(u32x4*)(p.C + (m0 + r) * N + n) = *(const u32x4*)(L0 + r * (BN * 2) + ((piece ^ (r & (PC - 1))) << 4));
  }
}

// C = bf16(sum of the parts), in their order; of a grouped product the experts' rows
// alone.  8 values a lane, whose parts are all loaded at once (512 columns by 11008
// transposed, one row: 8.9 us with the product, against 10.4 for a loop over them).
template <int SPLITS>
__global__ __launch_bounds__(256) void k_fp8_join(const float* __restrict__ part, int64_t M, int N,
                                                  const int32_t* __restrict__ offsets, int experts,
                                                  uint16_t* __restrict__ C) {
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;  // M * N / 8 < 2^31
  const uint32_t per_row = (uint32_t)N / 8;
  if (i >= (uint32_t)M * per_row) return;
  if (offsets) {
    const int row = (int)(i / per_row);
    if (row < offsets[0] || row >= offsets[experts]) return;
  }
  floatx4 v[SPLITS][2];
#pragma unroll
  for (int k = 0; k < SPLITS; ++k) {
    const floatx4* at = (const floatx4*)(part + k * M * N + (int64_t)i * 8);
    v[k][0] = at[0];
    v[k][1] = at[1];
  }
  floatx4 lo = v[0][0], hi = v[0][1];
#pragma unroll
  for (int k = 1; k < SPLITS; ++k) {
    lo += v[k][0];
    hi += v[k][1];
  }
  *(u32x4*)(C + (int64_t)i * 8) = u32x4{pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]), pack_bf16x2(hi[0], hi[1]),
                                        pack_bf16x2(hi[2], hi[3])};
}

// one launch of tile kind `kind` over all of p's rows
hipError_t launch_part(const Fp8Gemm& q, Args p, int kind, int splits, hipStream_t st) {
  const Fp8Kind& k = fp8_kinds()[kind];
  p.tiles_n = (p.N + k.bn - 1) / k.bn;
  const int64_t tiles =
      q.experts ? fp8_grouped_tiles(kind, p.M, p.N, q.experts) : (p.M + k.bm - 1) / k.bm * p.tiles_n;
  const dim3 gr((unsigned)tiles, (unsigned)splits), bl((unsigned)k.threads);
#define NF4K_LAUNCH(...) hipLaunchKernelGGL((__VA_ARGS__), gr, bl, 0, st, p)
#define NF4K_FLAGS(KERNEL, ...)                                                     \
  do {                                                                              \
    if (q.experts) {                                                                \
      if (q.a_e5m2) NF4K_LAUNCH(KERNEL<__VA_ARGS__, true, true>);                   \
      else NF4K_LAUNCH(KERNEL<__VA_ARGS__, false, true>);                           \
    } else {                                                                        \
      if (q.a_e5m2) NF4K_LAUNCH(KERNEL<__VA_ARGS__, true, false>);                  \
      else NF4K_LAUNCH(KERNEL<__VA_ARGS__, false, false>);                          \
    }                                                                               \
  } while (0)
#define NF4K_WIDE(NI)                                       \
  do {                                                      \
    if (q.transpose) NF4K_FLAGS(k_fp8_wide, NI, true);      \
    else NF4K_FLAGS(k_fp8_wide, NI, false);                 \
  } while (0)
// (without the split's few instructions one row by 4096 x 4096 is 4 % faster)
#define NF4K_ROWS(...)                                              \
  do {                                                              \
    if (splits > 1) NF4K_FLAGS(k_fp8_rows, __VA_ARGS__, true);      \
    else NF4K_FLAGS(k_fp8_rows, __VA_ARGS__, false);                \
  } while (0)
  switch (kind) {
    case kFp8Wide8: NF4K_WIDE(8); break;
    case kFp8Wide4: NF4K_WIDE(4); break;
    case kFp8Wide2: NF4K_WIDE(2); break;
    case kFp8Ring22: NF4K_FLAGS(k_fp8_ring, 128, 128, 4); break;
    case kFp8Ring21: NF4K_FLAGS(k_fp8_ring, 128, 64, 6); break;
    case kFp8Rows11: NF4K_ROWS(1, 1, 4, 4, false); break;
    case kFp8Rows12: NF4K_ROWS(1, 2, 4, 3, false); break;
    case kFp8Rows22: NF4K_ROWS(2, 2, 8, 2, false); break;
    case kFp8Rows42: NF4K_ROWS(4, 2, 4, 3, false); break;
    case kFp8Rows44: NF4K_ROWS(4, 4, 4, 2, false); break;
    case kFp8Rows14T: NF4K_ROWS(1, 4, 4, 3, true); break;
    case kFp8Rows24T: NF4K_ROWS(2, 4, 4, 3, true); break;
    default: NF4K_ROWS(4, 4, 4, 2, true); break;
  }
#undef NF4K_ROWS
#undef NF4K_WIDE
#undef NF4K_FLAGS
#undef NF4K_LAUNCH
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
#define NF4K_JOIN(S)                                                                                               \
  hipLaunchKernelGGL(k_fp8_join<S>, dim3((unsigned)((p.M * (p.N / 8) + 255) / 256)), dim3(256), 0, st, p.part, p.M, \
                     p.N, q.experts ? q.offsets : nullptr, q.experts, p.C)
  switch (splits) {
    case 2: NF4K_JOIN(2); break;
    case 3: NF4K_JOIN(3); break;
    case 4: NF4K_JOIN(4); break;
    case 6: NF4K_JOIN(6); break;
    default: NF4K_JOIN(8); break;
  }
#undef NF4K_JOIN
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_gemm(const Fp8Gemm& q, hipStream_t st) {
  Args p{};
  p.W = q.W;
  p.ws = q.w_scales;
  p.offsets = q.offsets;
  p.B2 = q.B2;
  p.N = (int)(q.transpose ? q.cols : q.rows);
  p.K = (int)(q.transpose ? q.rows : q.cols);
  p.R = q.R;
  p.experts = q.experts;
  const int KB = (p.K + 127) / 128;
  Fp8Part parts[2];
  p.part = q.part;
  const int n = plan_fp8(q.M, p.N, p.K, q.transpose, q.experts, q.part != nullptr, parts);
  int64_t r0 = 0;
  for (int i = 0; i < n; ++i) {
    // a launch holds at most 2^32 - 1 work-items: more tiles run as ranges of rows
    const Fp8Kind& k = fp8_kinds()[parts[i].kind];
    const int64_t tiles_n = (p.N + k.bn - 1) / k.bn;
    const int64_t most = q.experts ? q.M : std::max<int64_t>(1, (int64_t)0xFFFFFFFF / k.threads / tiles_n) * k.bm;
    for (const int64_t end = r0 + parts[i].rows; r0 < end;) {
      const int64_t rows = std::min(most, end - r0);
      p.A = q.A + r0 * p.K;
      p.as = q.a_scales + r0 * KB;
      p.A2 = q.A2 ? q.A2 + r0 * q.R : nullptr;
      p.C = q.C + r0 * p.N;
      p.M = rows;
      const hipError_t e = launch_part(q, p, parts[i].kind, parts[i].splits, st);
      if (e != hipSuccess) return e;
      r0 += rows;
    }
  }
  return hipSuccess;
}

}  // namespace nf4k
