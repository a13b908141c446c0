// Linear layers with 4-bit weights and group scales (gfx950).
//
//   y_ij = round( sum_g s_jg sum_{k in group g} x_ik (q_jk - z_jg)  + b_j )
//
// q in 0..15, groups of 32, 64 or 128 consecutive K, one scale (the type of x)
// and one zero point per output and group.
//
// The sum of a group is taken on the matrix cores over the integers q, which
// fp16 and bf16 hold exactly: P = sum x q and X = sum x (the same step with a
// right operand of ones), both fp32 chains of the 16x16x32 step in ascending K
// from +0.  Then, in fp32,
//   acc = fma(s, fma(-z, X, P), acc), groups in ascending order from +0,
// and one rounding of acc + b.  Nothing but x and s is ever rounded to 16 bits:
// the product is as exact as one with fp32 weights.  (Rounding s (q - z) to 16
// bits first, as a 16-bit weight would be, costs a bf16 result half its
// accuracy.)
//
// Batch invariance.  That order of operations is a function of (K, group)
// alone.  Every kernel below follows it, however it spreads rows, columns and
// groups over waves, so a row's bits do not depend on M.
//
// Packed weights.  A block of 16 outputs x 128 K is 1 KB: lane l's 16 bytes at
// 16 l hold output l % 16, dword t the K elements 32 t + 8 (l / 16) .. + 7 of the
// block, which is what lane l feeds step t.  Nibble order within a dword: bytes
// 0..3 carry k 0..3 in their low and k 4..7 in their high halves, so that a
// mask (and a shift) leaves four bytes q.  As e4m3 such a byte is q 2^-9 (0..7
// subnormal, 8..15 the first binade), and the conversion with scale 2^9 turns
// two of them into two 16-bit integers: 7 instructions for 8 weights.
// Behind the blocks, one dword per (group, output): the scale's 16 bits and the
// zero point above them.
#include "kernel_common.h"
#include "layer_internal.h"

namespace imm {
namespace {
using namespace dev;

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// The eight integers of a packed dword as one 16x16x32 operand.
template <int IN>
__device__ __forceinline__ i32x4 decode8(unsigned w) {
  typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const unsigned lo = w & 0x0f0f0f0fu, hi = (w >> 4) & 0x0f0f0f0fu;
  i32x4 r;
  if constexpr (IN == GEMM_F16) {
    r[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.0f, false));
    r[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.0f, true));
    r[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.0f, false));
    r[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.0f, true));
  } else {
    r[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false));
    r[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true));
    r[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false));
    r[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true));
  }
  return r;
}

// The right operand of X = sum x: eight ones.
template <int IN>
__device__ __forceinline__ i32x4 ones8() {
  constexpr int one = IN == GEMM_F16 ? 0x3c003c00 : 0x3f803f80;
  return i32x4{one, one, one, one};
}

template <int IN>
__device__ __forceinline__ float scale_of(unsigned sz) {
  if constexpr (IN == GEMM_F16)
    return (float)__builtin_bit_cast(_Float16, (unsigned short)(sz & 0xffffu));
  else
    return __uint_as_float(sz << 16);
}
__device__ __forceinline__ float zero_of(unsigned sz) { return (float)(sz >> 16); }

// ---- packing ---------------------------------------------------------------

// One thread per packed dword.  q [N, K / 2]: byte j of a row holds element 2 j
// in its low and 2 j + 1 in its high half.
__global__ __launch_bounds__(256) void w4_pack_kernel(const unsigned char* q, unsigned* packed,
                                                      int64_t N, int64_t K, int64_t kblocks,
                                                      int64_t dwords) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= dwords) return;
  const int t = (int)(i & 3), lane = (int)(i >> 2) & 63;
  const int64_t blk = i >> 8, kb = blk % kblocks, nb = blk / kblocks;
  const int64_t n = nb * 16 + lane % 16, k = kb * 128 + 32 * t + 8 * (lane / 16);
  unsigned r = 0;
  if (n < N && k < K) {
    // K is a multiple of 32, so the eight elements lie in the row
    const unsigned char* p = q + (n * K + k) / 2;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const unsigned v = (p[e >> 1] >> (4 * (e & 1))) & 15u;
      r |= v << (8 * (e & 3) + 4 * (e >> 2));
    }
  }
  packed[i] = r;
}

// One thread per (group, output): the scale's bits and the zero point (8
// without zero points); padding outputs get zeros.
__global__ __launch_bounds__(256) void w4_pack_scales_kernel(const unsigned short* scales,
                                                             const unsigned char* zeros,
                                                             unsigned* sz, int64_t N, int64_t np,
                                                             int64_t groups) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= groups * np) return;
  const int64_t n = i % np, gr = i / np;
  unsigned r = 0;
  if (n < N) {
    const int64_t at = n * groups + gr;
    r = scales[at] | ((zeros ? (unsigned)zeros[at] : 8u) << 16);
  }
  sz[i] = r;
}

// ---- few rows ----------------------------------------------------------------

// A workgroup of 8 waves owns RB x CB blocks of 16 x 16 outputs.  The waves
// share K: wave w takes the 128-K blocks w, w + 8, ...; each leaves P - z X of
// its groups in LDS, and after a barrier one thread per output adds the round's
// groups in ascending order.  So all of a workgroup's weight loads are in
// flight at once (U KB a wave and round, the next round's issued before this
// one's arithmetic), while the order of the sum stays the one above.
template <int IN, int G, int RB, int CB>
struct SkinnyShape {
  static constexpr int W = 8;
  static constexpr int NG = 128 / G;                  // groups per 128-K block
  static constexpr int GKB = RB * CB;                 // KB of LDS per group
  // blocks per wave and round: up to 4, within 32 KB of sums (two buffers)
  static constexpr int U0 = 32 / (W * NG * GKB);
  static constexpr int U = U0 < 1 ? 1 : U0 > 4 ? 4 : U0;
  static constexpr int GPR = W * U * NG;              // groups per round
  static constexpr int ELEMS = 256 * RB * CB;
  static constexpr int PER = (ELEMS + 511) / 512;     // outputs per thread
  static constexpr int LDS = 2 * GPR * (ELEMS + 16 * CB) * 4;
};

template <int IN, int G, int RB, int CB>
__global__ __launch_bounds__(512) void w4_skinny_kernel(W4Args g) {
  using S = SkinnyShape<IN, G, RB, CB>;
  constexpr int W = S::W, NG = S::NG, U = S::U, GPR = S::GPR, ELEMS = S::ELEMS, PER = S::PER;
  static_assert(S::LDS <= 160 * 1024, "LDS");
  __shared__ __attribute__((aligned(16))) float part[2][GPR][ELEMS];
  __shared__ float scl[2][GPR][16 * CB];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane % 16, hq = lane / 16;
  const int64_t cgroups = (g.nblocks + CB - 1) / CB;
  const int64_t cg = blockIdx.x % cgroups, rg = blockIdx.x / cgroups;
  const int64_t m0 = rg * (16 * RB), nb0 = cg * CB;
  const int kblocks = (int)g.kblocks;
  const int ksteps = (int)(g.K / 32);

  // rows past M and column blocks past N read the last one there is and are
  // never stored
  const char* xrow[RB];
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    const int64_t row = m0 + 16 * i + lr;
    xrow[i] = static_cast<const char*>(g.x) + ((row < g.M ? row : g.M - 1) * g.K + 8 * hq) * 2;
  }
  const u32x4* wblk[CB];
  const unsigned* szp[CB];
#pragma unroll
  for (int j = 0; j < CB; ++j) {
    const int64_t nb = nb0 + j < g.nblocks ? nb0 + j : g.nblocks - 1;
    wblk[j] = reinterpret_cast<const u32x4*>(g.packed) + nb * g.kblocks * 64 + lane;
    szp[j] = g.sz + nb * 16 + lr;
  }
  const int64_t np = g.nblocks * 16;

  float acc[PER];
#pragma unroll
  for (int p = 0; p < PER; ++p) acc[p] = 0.0f;

  const int rounds = (kblocks + W * U - 1) / (W * U);
  u32x4 wn[U][CB];
  auto load_w = [&](int r) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = (r * U + u) * W + w;
#pragma unroll
      for (int j = 0; j < CB; ++j) {
        wn[u][j] = u32x4{};
        if (kb < kblocks) wn[u][j] = wblk[j][(int64_t)kb * 64];
      }
    }
  };
  load_w(0);
  for (int r = 0; r < rounds; ++r) {
    const int buf = r & 1;
    // this round's rows of x and scales, then the next round's weights
    i32x4 a[U][4][RB];
    unsigned sz[U][NG][CB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = (r * U + u) * W + w;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < RB; ++i) {
          a[u][t][i] = i32x4{};
          if (kb * 4 + t < ksteps)
            a[u][t][i] = *reinterpret_cast<const i32x4*>(xrow[i] + (int64_t)(kb * 4 + t) * 64);
        }
#pragma unroll
      for (int s = 0; s < NG; ++s)
#pragma unroll
        for (int j = 0; j < CB; ++j) {
          sz[u][s][j] = 0;
          if ((int64_t)kb * NG + s < g.groups) sz[u][s][j] = szp[j][((int64_t)kb * NG + s) * np];
        }
    }
    u32x4 wc[U][CB];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < CB; ++j) wc[u][j] = wn[u][j];
    if (r + 1 < rounds) load_w(r + 1);
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int s = 0; s < NG; ++s) {
        f32x4 P[RB][CB], X[RB];
#pragma unroll
        for (int i = 0; i < RB; ++i) {
          X[i] = f32x4{};
#pragma unroll
          for (int j = 0; j < CB; ++j) P[i][j] = f32x4{};
        }
#pragma unroll
        for (int t = s * (G / 32); t < (s + 1) * (G / 32); ++t) {
          i32x4 b[CB];
#pragma unroll
          for (int j = 0; j < CB; ++j) b[j] = decode8<IN>(wc[u][j][t]);
#pragma unroll
          for (int i = 0; i < RB; ++i) {
            X[i] = mfma16_v<IN>(a[u][t][i], ones8<IN>(), X[i]);
#pragma unroll
            for (int j = 0; j < CB; ++j) P[i][j] = mfma16_v<IN>(a[u][t][i], b[j], P[i][j]);
          }
        }
        const int gr = (u * W + w) * NG + s;
#pragma unroll
        for (int j = 0; j < CB; ++j) {
          const float z = zero_of(sz[u][s][j]);
          if (hq == 0) scl[buf][gr][16 * j + lr] = scale_of<IN>(sz[u][s][j]);
#pragma unroll
          for (int i = 0; i < RB; ++i) {
            f32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = fmaf(-z, X[i][e], P[i][j][e]);
            *reinterpret_cast<f32x4*>(&part[buf][gr][((i * CB + j) * 64 + lane) * 4]) = v;
          }
        }
      }
    }
    // One barrier a round: the buffer filled two rounds on was read before the
    // next round's barrier.
    __syncthreads();
    const int64_t left = g.groups - (int64_t)r * GPR;
    const int ng = left < GPR ? (int)left : GPR;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const int e = tid + 512 * p;
      if (e < ELEMS) {
        const int col = 16 * ((e / 256) % CB) + (e / 4) % 16;
#pragma unroll 8
        for (int k = 0; k < ng; ++k) acc[p] = fmaf(scl[buf][k][col], part[buf][k][e], acc[p]);
      }
    }
  }
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int e = tid + 512 * p;
    if (e < ELEMS) {
      // element e: block e / 256, lane (e / 4) % 64, register e % 4 of its accumulators
      const int blk = e / 256, ln = (e / 4) % 64;
      const int64_t row = m0 + 16 * (blk / CB) + 4 * (ln / 16) + e % 4;
      const int64_t col = (nb0 + blk % CB) * 16 + ln % 16;
      if (row < g.M && col < g.N)
        store_out<IN>(g.y, row * g.N + col, g.bias ? acc[p] + g.bias[col] : acc[p]);
    }
  }
}

// ---- many rows ---------------------------------------------------------------

// X = sum x of every (row, group), fp32 [groups, m_pad], by the chain of the
// few-rows kernel: one wave per 16 rows and group.  The tile kernel reads it
// instead of spending a fifth of its matrix steps on it (each column of waves
// would repeat them).  Rows past M repeat the last row.
template <int IN, int G>
__global__ __launch_bounds__(256) void w4_group_sums_kernel(W4Args g) {
  const int lane = threadIdx.x & 63;
  const int64_t task = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t gr = task % g.groups, m0 = task / g.groups * 16;
  if (m0 >= g.m_pad) return;
  const int64_t row = m0 + lane % 16;
  const char* p = static_cast<const char*>(g.x) +
                  ((row < g.M ? row : g.M - 1) * g.K + gr * G + 8 * (lane / 16)) * 2;
  i32x4 a[G / 32];
#pragma unroll
  for (int t = 0; t < G / 32; ++t) a[t] = *reinterpret_cast<const i32x4*>(p + 64 * t);
  f32x4 X{};
#pragma unroll
  for (int t = 0; t < G / 32; ++t) X = mfma16_v<IN>(a[t], ones8<IN>(), X);
  if (lane % 16 == 0)
    *reinterpret_cast<f32x4*>(g.sums + gr * g.m_pad + m0 + 4 * (lane / 16)) = X;
}

constexpr unsigned OOB = 0x80000000u;  // an offset past every buffer: zeros

// 16 bytes per lane from base + off to LDS (lane l at dst + 16 l).  (The
// host pass, which knows no 16-byte transfers, would drop the kernel's stub.)
__device__ __forceinline__ void dma16(const void* base, char* dst, unsigned off) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, 0x7fffffff, 0x00020000),
      IMM_LDS(dst), 16, off, 0, 0, 0);
#endif
}

template <int OFF>
__device__ __forceinline__ unsigned ds_read_b32_at(unsigned addr) {
  static_assert(OFF >= 0 && OFF < 65536, "ds_read offset field");
  unsigned v;
  asm volatile("ds_read_b32 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "n"(OFF));
  return v;
}

// A workgroup of WM x WN waves owns a tile of TM x TN outputs, each wave FM x FN
// blocks of 16 x 16.  K is walked in stages of one 128-K block.  A ring of NS
// LDS stages (x rows of 256 bytes, packed weight blocks as they lie in memory;
// beside it scale words and group sums) is filled by buffer->LDS DMA.  A wave decodes its
// own weight blocks from LDS to registers, sums a group into P on the matrix
// cores and folds P into acc with two fused multiply-adds an element.  The
// matrix steps and the vector work (decode 28 instructions a block and stage,
// fold 8 a block pair and group) take about the same time, so two waves share
// a SIMD and fill each other's gaps.
//
// LDS reads are inline assembly with explicit waits (the compiler would make
// each wait for every DMA in flight).  The stage change sits before the last
// k-step: all of the wave's reads of stage t have landed, its DMA of stage t + 1
// too, and after one barrier the slot of stage t is refilled and the first
// fragments of stage t + 1 are read under that k-step's arithmetic.  Scale
// words and sums are read after that barrier, when a group ends, so their ring
// has one slot more: a refill overwrites those of the stage before.
//
// 16-byte chunk c of an x row r lies at slot c ^ (r & 15): the 16 rows that a
// quarter of a wave reads at one chunk fall on different banks.
template <int G, int FM, int FN, int WM, int WN, int NS>
struct TileShape {
  static constexpr int TM = 16 * FM * WM, TN = 16 * FN * WN, WAVES = WM * WN;
  static constexpr int NG = 128 / G;
  static constexpr int A_STAGE = TM * 256, B_STAGE = TN * 64;
  static constexpr int RS = 1024 / (TN * 4), RX = 1024 / (TM * 4);  // rows per 1 KB transfer
  static constexpr int IS = (NG + RS - 1) / RS, IX = (NG + RX - 1) / RX;
  static constexpr int ITEMS = IS + IX;
  static constexpr int STAGE = A_STAGE + B_STAGE;
  static constexpr int META = ITEMS * 1024;      // scale words and sums of a stage
  static constexpr int LDS = NS * STAGE + (NS + 1) * META;
  static constexpr int DA = A_STAGE / 1024 / WAVES, DB = B_STAGE / 1024 / WAVES;
  static_assert(DA * WAVES * 1024 == A_STAGE && DB * WAVES * 1024 == B_STAGE, "DMA split");
  static_assert(ITEMS <= WAVES && RS >= 1 && RX >= 1, "one scale or sum transfer per wave");
  static_assert(LDS <= 160 * 1024, "LDS");
};

template <int IN, int G, int FM, int FN, int WM, int WN, int NS>
__global__ __launch_bounds__(WM * WN * 64, 2) void w4_tile_kernel(W4Args g) {
  using S = TileShape<G, FM, FN, WM, WN, NS>;
  constexpr int TM = S::TM, TN = S::TN, NG = S::NG, KPG = G / 32;
  __shared__ __attribute__((aligned(1024))) char lds[S::LDS];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w / WN, wn = w % WN;
  const int lb = lane % 16, hq = lane / 16;
  int64_t ksl, pm, pn;
  raster_tile(blockIdx.x, g.grid, g.tiles_m, g.tiles_n, 8, &ksl, &pm, &pn);
  const int64_t m0 = pm * TM, nb0 = pn * (TN / 16);
  const int nt = (int)g.kblocks;
  const int groups = (int)g.groups;
  const int64_t np = g.nblocks * 16;

  // ---- DMA: this lane's offsets from the stage's first byte
  unsigned a_off[S::DA], b_off[S::DB];
  int a_k[S::DA];  // first K element of the chunk within the stage
#pragma unroll
  for (int i = 0; i < S::DA; ++i) {
    const int row = 4 * (w * S::DA + i) + lane / 16;
    const int c = (lane % 16) ^ (row & 15);
    a_off[i] = m0 + row < g.M ? (unsigned)(row * g.K * 2 + c * 16) : OOB;
    a_k[i] = 8 * c;
  }
#pragma unroll
  for (int i = 0; i < S::DB; ++i) {
    const int j = w * S::DB + i;
    b_off[i] = nb0 + j < g.nblocks ? (unsigned)(j * g.kblocks * 1024 + lane * 16) : OOB;
  }
  auto dma_stage = [&](int t) {
    const int slot = (t % NS) * S::STAGE;
    // past the last stage every transfer is a zero fill, so that the counts of
    // transfers in flight never change
    const bool live = t < nt;
    const int64_t krem = g.K - (int64_t)t * 128;
    const char* pa = static_cast<const char*>(g.x) + (m0 * g.K + (int64_t)(live ? t : 0) * 128) * 2;
    const char* pb = static_cast<const char*>(g.packed) + (nb0 * g.kblocks + (live ? t : 0)) * 1024;
#pragma unroll
    for (int i = 0; i < S::DA; ++i)
      dma16(pa, lds + slot + (w * S::DA + i) * 1024, live && a_k[i] < krem ? a_off[i] : OOB);
#pragma unroll
    for (int i = 0; i < S::DB; ++i)
      dma16(pb, lds + slot + S::A_STAGE + (w * S::DB + i) * 1024,
            live ? b_off[i] : OOB);
    if (w < S::ITEMS) {
      // 1 KB of scale words (rows of TN) or of group sums (rows of TM)
      const bool sums = w >= S::IS;
      const int per = sums ? TM / 4 : TN / 4;                   // lanes per row
      const int item = sums ? w - S::IS : w;
      const int gi = t * NG + item * (sums ? S::RX : S::RS);    // first group of the item
      const int gl = item * (sums ? S::RX : S::RS) + lane / per;
      const int at = (lane % per) * 4;
      const int64_t pitch = sums ? g.m_pad : np;
      const char* base = sums ? reinterpret_cast<const char*>(g.sums) + m0 * 4
                              : reinterpret_cast<const char*>(g.sz) + nb0 * 64;
      const bool ok = live && gl < NG && t * NG + gl < groups && (sums || nb0 * 16 + at < np);
      const unsigned off = ok ? (unsigned)((lane / per) * pitch * 4 + at * 4) : OOB;
      dma16(base + (gi < groups ? gi : 0) * pitch * 4,
            lds + NS * S::STAGE + (t % (NS + 1)) * S::META + w * 1024, off);
    }
  };
  auto fence = [&]() { __builtin_amdgcn_sched_barrier(0); };
  auto lds_wait = [&]() {
    fence();
    __builtin_amdgcn_s_waitcnt(lgkmcnt_imm(0));
    fence();
  };
  // all transfers of stage t + 1 landed, NS - 2 later stages in flight
  auto dma_wait = [&]() {
    constexpr int D = S::DA + S::DB;
    fence();
    if (w < S::ITEMS)
      __builtin_amdgcn_s_waitcnt(vmcnt_imm((NS - 2) * (D + 1)));
    else
      __builtin_amdgcn_s_waitcnt(vmcnt_imm((NS - 2) * D));
    __builtin_amdgcn_s_barrier();
    fence();
  };

  // ---- LDS reads
  const unsigned lds0 = (unsigned)(uintptr_t)((__attribute__((address_space(3))) char*)lds);
  unsigned a_rd[4];
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
    a_rd[ks] = lds0 + (wm * FM * 16 + lb) * 256 + (((4 * ks + hq) ^ lb) << 4);
  const unsigned b_rd = lds0 + S::A_STAGE + wn * FN * 1024 + lane * 16;
  const unsigned s_rd = lds0 + NS * S::STAGE + (wn * FN * 16 + lb) * 4;
  const unsigned x_rd = lds0 + NS * S::STAGE + S::IS * 1024 + (wm * FM * 16 + 4 * hq) * 4;

  i32x4 A[2][FM], W[FN];
  f32x4 P[FM][FN], acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = P[i][j] = f32x4{};

  auto read_a = [&](auto KS, int slot, i32x4 (&F)[FM]) {
    constexpr int ks = decltype(KS)::value;
    static_for<0, FM>([&](auto I) { F[decltype(I)::value] = ds_read_b128_at<decltype(I)::value * 4096>(a_rd[ks] + slot); });
  };
  auto read_w = [&](int slot) {
    static_for<0, FN>([&](auto J) { W[decltype(J)::value] = ds_read_b128_at<decltype(J)::value * 1024>(b_rd + slot); });
  };
  for (int t = 0; t < NS; ++t) dma_stage(t);
  // stage 0 landed: NS - 1 later ones in flight
  fence();
  if (w < S::ITEMS)
    __builtin_amdgcn_s_waitcnt(vmcnt_imm((NS - 1) * (S::DA + S::DB + 1)));
  else
    __builtin_amdgcn_s_waitcnt(vmcnt_imm((NS - 1) * (S::DA + S::DB)));
  __builtin_amdgcn_s_barrier();
  fence();
  read_w(0);
  read_a(std::integral_constant<int, 0>{}, 0, A[0]);

  for (int t = 0; t < nt; ++t) {
    const int slot = (t % NS) * S::STAGE, next = ((t + 1) % NS) * S::STAGE;
    const int meta = (t % (NS + 1)) * S::META;
    static_for<0, 4>([&](auto KS) {
      constexpr int ks = decltype(KS)::value;
      constexpr bool ends = (ks + 1) % KPG == 0;  // this k-step ends a group
      constexpr int gi = ks / KPG;                // the group within the stage
      lds_wait();  // this k-step's fragments
      i32x4 b[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) b[j] = decode8<IN>((unsigned)W[j][ks]);
      fence();
      if constexpr (ks < 3) {
        read_a(std::integral_constant<int, ks + 1>{}, slot, A[(ks + 1) & 1]);
      } else {
        dma_wait();
        dma_stage(t + NS);
        read_w(next);
        read_a(std::integral_constant<int, 0>{}, next, A[0]);
      }
      fence();
      unsigned sz[FN];
      i32x4 X[FM];
      static_for<0, FM>([&](auto I) {
        constexpr int i = decltype(I)::value;
#pragma unroll
        for (int j = 0; j < FN; ++j)
          P[i][j] = mfma16_v<IN>(A[ks & 1][i], b[j], ks % KPG == 0 ? f32x4{} : P[i][j]);
        if constexpr (ends && i == FM - 2) {
          // the group's scale words and sums, under the rest of its matrix steps
          fence();
          static_for<0, FN>([&](auto J) {
            sz[decltype(J)::value] = ds_read_b32_at<gi * TN * 4 + decltype(J)::value * 64>(s_rd + meta);
          });
          static_for<0, FM>([&](auto R) {
            X[decltype(R)::value] = ds_read_b128_at<gi * TM * 4 + decltype(R)::value * 64>(x_rd + meta);
          });
          fence();
        }
      });
      if constexpr (ends) {
        lds_wait();
        if (t * NG + gi < groups) {
          float sc[FN], zn[FN];
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            sc[j] = scale_of<IN>(sz[j]);
            zn[j] = -zero_of(sz[j]);
          }
#pragma unroll
          for (int i = 0; i < FM; ++i) {
            const f32x4 xs = __builtin_bit_cast(f32x4, X[i]);
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                acc[i][j][e] = fmaf(sc[j], fmaf(zn[j], xs[e], P[i][j][e]), acc[i][j][e]);
          }
        }
      }
    });
  }
  // No transfer or read is in flight when the workgroup ends; the reads of the
  // stage past the last one keep their registers until they have landed.
  fence();
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
  __builtin_amdgcn_s_waitcnt(lgkmcnt_imm(0));
  fence();
#pragma unroll
  for (int i = 0; i < FM; ++i) keep_live<4>(A[0][i]);
#pragma unroll
  for (int j = 0; j < FN; ++j) keep_live<4>(W[j]);
  fence();
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int64_t col = (nb0 + wn * FN + j) * 16 + lb;
    if (col >= g.N) continue;
    const float bias = g.bias ? g.bias[col] : 0.0f;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t row = m0 + (wm * FM + i) * 16 + 4 * hq + e;
        if (row < g.M) store_out<IN>(g.y, row * g.N + col, g.bias ? acc[i][j][e] + bias : acc[i][j][e]);
      }
  }
}

template <int IN, int G, int FM, int FN, int WM, int WN, int NS>
hipError_t launch_tile(W4Args a, hipStream_t s) {
  using S = TileShape<G, FM, FN, WM, WN, NS>;
  const int64_t tasks = a.groups * (a.m_pad / 16);
  hipLaunchKernelGGL((w4_group_sums_kernel<IN, G>), dim3((unsigned)((tasks + 3) / 4)), dim3(256), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  a.tiles_m = (a.M + S::TM - 1) / S::TM;
  a.tiles_n = (a.N + S::TN - 1) / S::TN;
  a.grid = a.tiles_m * a.tiles_n;
  hipLaunchKernelGGL((w4_tile_kernel<IN, G, FM, FN, WM, WN, NS>), dim3((unsigned)a.grid),
                     dim3(WM * WN * 64), 0, s, a);
  return hipGetLastError();
}

template <int IN, int G, int RB, int CB>
hipError_t launch_skinny(const W4Args& a, hipStream_t s) {
  const int64_t cg = (a.nblocks + CB - 1) / CB, rg = (a.M + 16 * RB - 1) / (16 * RB);
  hipLaunchKernelGGL((w4_skinny_kernel<IN, G, RB, CB>), dim3((unsigned)(cg * rg)), dim3(512), 0, s, a);
  return hipGetLastError();
}

template <int IN, int G>
hipError_t launch_group(const W4Args& a, hipStream_t s) {
  if (a.sums) return launch_tile<IN, G, 4, 4, 2, 4, G == 32 ? 2 : 3>(a, s);
  if (a.M <= 16) return launch_skinny<IN, G, 1, 1>(a, s);
  return launch_skinny<IN, G, 2, 1>(a, s);
}

template <int IN>
hipError_t launch_in(const W4Args& a, hipStream_t s) {
  if (a.group == 128) return launch_group<IN, 128>(a, s);
  if (a.group == 64) return launch_group<IN, 64>(a, s);
  return launch_group<IN, 32>(a, s);
}

}  // namespace

hipError_t launch_w4_pack(int64_t N, int64_t K, int group, const void* q, const void* scales,
                          const void* zeros, void* packed, hipStream_t s) {
  const int64_t nblocks = (N + 15) / 16, kblocks = (K + 127) / 128, groups = K / group;
  const int64_t dwords = nblocks * kblocks * 256, pairs = groups * nblocks * 16;
  unsigned* const out = static_cast<unsigned*>(packed);
  hipLaunchKernelGGL(w4_pack_kernel, dim3((unsigned)((dwords + 255) / 256)), dim3(256), 0, s,
                     static_cast<const unsigned char*>(q), out, N, K, kblocks, dwords);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(w4_pack_scales_kernel, dim3((unsigned)((pairs + 255) / 256)), dim3(256), 0, s,
                     static_cast<const unsigned short*>(scales),
                     static_cast<const unsigned char*>(zeros), out + dwords, N, nblocks * 16, groups);
  return hipGetLastError();
}

bool w4_uses_tiles(int64_t M, int64_t K) {
  // the tile kernel's 32-bit offsets within 128 rows of x
  return M > 64 && K > 0 && 128 * K * 2 < ((int64_t)1 << 31);
}

hipError_t launch_w4(int in, const W4Args& a, hipStream_t s) {
  return in == GEMM_F16 ? launch_in<GEMM_F16>(a, s) : launch_in<GEMM_BF16>(a, s);
}

}  // namespace imm
