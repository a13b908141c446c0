// Linear layers with 4-bit weights and group scales (gfx950).
//
//   y_ij = round( sum_g s_jg sum_{k in group g} x_ik (q_jk - z_jg)  + b_j )
//
// q in 0..15, groups of 32, 64 or 128 consecutive K, one scale (the type of x)
// and one zero point per output and group.
//
// The sum of a group is taken on the matrix cores.  X = sum x comes first (the
// 16x16x32 step with an operand of ones), and is split into three bf16 pieces
// that add up to it exactly; P starts as their 16x16x32 bf16 step with -z, and
// the 16x16x32 steps over x and the integers q (exact in fp16 and bf16) follow
// in ascending K, all in one fp32 accumulator: P = -z X + sum x q.  Then, in fp32,
//   acc = fma(s, P, acc), groups in ascending order from +0,
// and one rounding of acc + b.  Nothing but x and s is ever rounded to 16 bits.
// (Rounding s (q - z) to 16 bits first, as a 16-bit weight would be, costs a bf16
// result half its accuracy.)  P is a difference of two sums, so its fp32 error goes
// with sum |x| (q + z), not with sum |x| |q - z| as that of fp32 weights would: x
// with q = z throughout need not give 0, and a group of bf16 x whose sum |x| (q + z)
// passes 2^128 overflows though its sum x (q - z) may not.  (z as a matrix step leaves
// the vector unit, whose work does not hide in the tile kernel, one multiply-add per
// element and group; a second one in place of that step was as fast within two per cent.)
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
// Behind the blocks, one dword per (group, output): the scale's 16 bits, and
// above them -z as bf16 (exact: eight bits).
#include <algorithm>

#include "buffer_access.h"
#include "kernel_common.h"
#include "layer_internal.h"

namespace imm {
namespace {
using namespace dev;

// Dword p (two integers) of the 16x16x32 operand in a packed dword.
template <int IN>
__device__ __forceinline__ int decode_pair(unsigned w, int p) {
  const unsigned v = (p < 2 ? w : w >> 4) & 0x0f0f0f0fu;
  if constexpr (IN == GEMM_F16)
    return __builtin_bit_cast(int, p % 2 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 512.0f, true)
                                         : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 512.0f, false));
  else
    return __builtin_bit_cast(int, p % 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 512.0f, true)
                                         : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 512.0f, false));
}

// The eight integers of a packed dword as one 16x16x32 operand.
template <int IN>
__device__ __forceinline__ i32x4 decode8(unsigned w) {
  i32x4 r;
#pragma unroll
  for (int p = 0; p < 4; ++p) r[p] = decode_pair<IN>(w, p);
  return r;
}

// The other operand of X = sum x: eight ones.  x is the right operand there, so
// every register of lane l holds the sum of row l % 16.
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

// x as three bf16 values whose sum is x: (first | second << 16, third).
__device__ __forceinline__ i32x2 split3(float x) {
  const float h = (float)(__bf16)x, r = x - h, m = (float)(__bf16)r;
  const unsigned short hb = f32_to_bf16(h), mb = f32_to_bf16(m), lb = f32_to_bf16(r - m);
  return i32x2{(int)(hb | ((unsigned)mb << 16)), (int)lb};
}
// -z against the three pieces of X, which take the first three of the step's 32
// K positions (`first` is all ones in lanes 0..15 and 0 elsewhere).
__device__ __forceinline__ i32x4 zero_operand(unsigned sz, unsigned first) {
  const unsigned z = (sz >> 16) & first;
  return i32x4{(int)(z | (z << 16)), (int)z, 0, 0};
}
// The start of P: -z X.  x holds the pieces in its first two dwords; the other
// two meet zeros.  Chained matrix steps of different opcodes (this one and the
// fp16 step) overlap in the pipeline without a dependency check between the
// first's result and the second's accumulator input, so callers hold the
// starts in place (hold) and leave at least 32 cycles before the next step.
__device__ __forceinline__ f32x4 start_of_sum(const i32x4& x, const i32x4& z) {
  return mfma16_v<GEMM_BF16>(x, z, f32x4{});
}
// An empty statement that needs v: what makes v stays before it.
__device__ __forceinline__ void hold(f32x4& v) { asm volatile("" : "+v"(v)); }

// ---- packing ---------------------------------------------------------------

// A thread per packed dword (or several, past the threads of a launch).
// q [N, K / 2]: byte j of a row holds element 2 j in its low and 2 j + 1 in its high
// half.
__global__ __launch_bounds__(256) void w4_pack_kernel(const unsigned char* q, unsigned* packed,
                                                      int64_t N, int64_t K, int64_t kblocks,
                                                      int64_t dwords) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < dwords; i += (int64_t)gridDim.x * 256) {
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
}

// A thread per (group, output), or several: the scale's bits and the zero point's
// negative (8 without zero points); padding outputs get zeros.
__global__ __launch_bounds__(256) void w4_pack_scales_kernel(const unsigned short* scales,
                                                             const unsigned char* zeros,
                                                             unsigned* sz, int64_t N, int64_t np,
                                                             int64_t groups) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < groups * np; i += (int64_t)gridDim.x * 256) {
    const int64_t n = i % np, gr = i / np;
    unsigned r = 0;
    if (n < N) {
      const int64_t at = n * groups + gr;
      r = scales[at] | (__float_as_uint(-(zeros ? (float)zeros[at] : 8.0f)) & 0xffff0000u);
    }
    sz[i] = r;
  }
}

// ---- few rows ----------------------------------------------------------------

// A workgroup makes a unit of RB x CB blocks of 16 x 16 outputs.  Four waves do
// nothing but move: rows of x, weight blocks and scale words go to a ring of NS
// LDS stages of SB 128-K blocks.  SB / U H waves multiply, each U blocks of the
// stage (for half of the unit's columns, or rows, where H is 2), and leave P of
// their groups in LDS; behind the next barrier every thread adds the stage's groups
// of its outputs in ascending order, which keeps the order of the sum the one
// above.  One barrier a stage publishes stage t (each moving wave has waited for
// its own transfers) and the sums of stage t - 1, and frees the slot of stage
// t - 1; where LDS holds the sums of one stage only, another lets them be added.
//
// 16-byte chunk c of row r of x lies at slot c ^ (r & 15) of the row: the 16 rows
// that a quarter of a wave reads at one chunk fall on different banks.  XR rows
// of x are kept: 16 RB, or 4 where M <= 4, so that the ring holds more weights.
//
// Measured at K = 4096, group 128 (in brackets what a kernel without the moving
// waves took, each wave loading its own rows and blocks to registers): 1 x 4096
// 5.3 us (5.7), 1 x 14336 9.9 (13.1; 3 TB/s), 1 x 131072 62 (64; 4.3 TB/s),
// 16 x 14336 11.3 (14.2), 64 x 4096 9.7 (12.3), 256 x 4096 24.6 (29.8).  Single
// units are bound by a stage's latency, LDS to sums; wide grids of few rows by the
// weights; more rows by LDS, which x passes once for every column group.  (A wave per block
// of outputs, over all of K and without exchanged sums, costs some 430 cycles for 128
// K: 29 x 4096, K = 14336, group 64 31.7 us against 23.9.)
template <int G, int RB, int CB, int XR, int SB, int U, int H>
struct RowsShape {
  static constexpr int MOVERS = 4, WAVES = SB / U * H, THREADS = 64 * (MOVERS + WAVES);
  static constexpr int RBW = H == 2 && CB == 1 ? RB / 2 : RB;  // blocks of a wave
  static constexpr int CBW = H == 2 && CB > 1 ? CB / 2 : CB;
  static constexpr int NG = 128 / G, GPS = SB * NG;            // groups per stage
  static constexpr int XROW = SB * 256, XBYTES = XR * XROW, WBYTES = CB * SB * 1024;
  static constexpr int SZ = (GPS * CB * 64 + 1023) / 1024;     // transfers of scale words
  static constexpr int STAGE = XBYTES + WBYTES + SZ * 1024;
  static constexpr int T = (XBYTES + WBYTES) / 1024 / MOVERS;  // transfers of each moving wave
  static_assert(T * MOVERS * 1024 == XBYTES + WBYTES, "transfers");
  static constexpr int LPB = XR == 4 ? 16 : 64;                // lanes whose outputs are kept
  static constexpr int ELEMS = 4 * LPB * RB * CB;
  static constexpr int V = ELEMS > 64 * WAVES ? ELEMS / (64 * WAVES) : 1;  // outputs of a thread
  static_assert(V <= 4, "outputs of a thread share a lane");
  static constexpr int SUMS = GPS * (ELEMS + 16 * CB) * 4, ALL = 160 * 1024;
  static constexpr int BUFS = 2 * SUMS + 2 * STAGE <= ALL ? 2 : 1;
  static constexpr int fit = (ALL - BUFS * SUMS) / STAGE, flight = 2 + 63 / (T + (SZ + MOVERS - 1) / MOVERS);
  static constexpr int least = fit < flight ? fit : flight;
  static constexpr int NS = least < 8 ? least : 8;
  static_assert(NS >= 2, "LDS");
};

template <int IN, int G, int RB, int CB, int XR, int SB, int U, int H>
__global__ __launch_bounds__((4 + SB / U * H) * 64) void w4_rows_kernel(W4Args g) {
  using S = RowsShape<G, RB, CB, XR, SB, U, H>;
  constexpr int NG = S::NG, GPS = S::GPS, NS = S::NS, RBW = S::RBW, CBW = S::CBW, V = S::V;
  __shared__ __attribute__((aligned(1024))) char ring[NS * S::STAGE];
  __shared__ __attribute__((aligned(16))) float part[S::BUFS][GPS][S::ELEMS];
  __shared__ float scl[S::BUFS][GPS][16 * CB];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const unsigned cgroups = (unsigned)((g.nblocks + CB - 1) / CB);
  const int64_t nb0 = (int64_t)(blockIdx.x % cgroups) * CB, m0 = (int64_t)(blockIdx.x / cgroups) * (16 * RB);
  const int K = (int)g.K, kblocks = (int)g.kblocks, nt = (kblocks + SB - 1) / SB;
  const int64_t np = g.nblocks * 16;
  auto barrier = [&]() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  };

  if (w >= S::WAVES) {
    // ---- the moving waves: kilobytes p, p + 4, ... of a stage (x, then weights), and
    // kilobytes p, p + 4, ... of its scale words
    constexpr int T = S::T, XT = S::XBYTES / 1024;
    const int p = w - S::WAVES;
    const auto xbuf = buffer_at(static_cast<const char*>(g.x) + m0 * K * 2);
    const auto wbuf = buffer_at(static_cast<const char*>(g.packed) + nb0 * kblocks * 1024);
    const int64_t sz_step = (int64_t)GPS * np * 4;
    const char* sz = reinterpret_cast<const char*>(g.sz) + nb0 * 64;
    auto move = [&](int t) {
      char* const slot = ring + t % NS * S::STAGE;
#pragma unroll
      for (int i = 0; i < T; ++i) {
        const int q = p + 4 * i;  // below XT for all four waves or for none
        if (4 * i < XT) {
          const int r = q / (SB / 4), c = q % (SB / 4) * 64 + ((lane & 48) | ((lane ^ r) & 15));
          const bool live = m0 + r < g.M && t * (SB * 128) + 8 * c < K;
          dma16(xbuf, slot + q * 1024, live ? (unsigned)(c * 16) : OOB, r * K * 2 + t * S::XROW);
        } else {
          const int j = (q - XT) / SB, kb = (q - XT) % SB;
          const bool live = nb0 + j < g.nblocks && t * SB + kb < kblocks;
          dma16(wbuf, slot + q * 1024, live ? (unsigned)lane * 16 : OOB, (j * kblocks + t * SB + kb) * 1024);
        }
      }
#pragma unroll
      for (int q = p; q < S::SZ; q += 4) {
        const int sg = (q * 64 + lane) / (4 * CB), sc = (q * 64 + lane) % (4 * CB);
        const bool live = sg < GPS && t * GPS + sg < g.groups && nb0 * 16 + 4 * sc < np;
        dma16(buffer_at(sz), slot + S::XBYTES + S::WBYTES + q * 1024,
              live ? (unsigned)(sg * np * 4 + sc * 16) : OOB, 0);
      }
      sz += sz_step;
    };
    // all transfers but those of the last n stages have landed
    auto wait = [&](int n) {
      auto upto = [&](auto ONE) {
        constexpr int each = T + S::SZ / 4 + decltype(ONE)::value;
        if (n >= NS - 2) __builtin_amdgcn_s_waitcnt(vmcnt_imm((NS - 2) * each));
#define IMM_LATER(k) else if (NS - 2 > k && n == k) __builtin_amdgcn_s_waitcnt(vmcnt_imm(k * each));
        IMM_LATER(5) IMM_LATER(4) IMM_LATER(3) IMM_LATER(2) IMM_LATER(1)
#undef IMM_LATER
        else __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
      };
      __builtin_amdgcn_sched_barrier(0);
      if (p < S::SZ % 4)
        upto(std::integral_constant<int, 1>{});
      else
        upto(std::integral_constant<int, 0>{});
      __builtin_amdgcn_sched_barrier(0);
    };
    for (int t = 0; t < NS - 1 && t < nt; ++t) move(t);
    for (int t = 0; t < nt; ++t) {
      wait(nt - 1 - t);
      __builtin_amdgcn_s_barrier();
      if (t + NS - 1 < nt) move(t + NS - 1);
      if (S::BUFS == 1) __builtin_amdgcn_s_barrier();
    }
    if (S::BUFS == 2) __builtin_amdgcn_s_barrier();
    return;
  }

  // ---- the multiplying waves
  const int tid = threadIdx.x, lr = lane % 16, hq = lane / 16;
  const unsigned first = hq == 0 ? ~0u : 0u;
  constexpr int KW = SB / U;
  const int kb0 = w % KW, half = w / KW;  // blocks kb0, kb0 + KW, ...
  const int i0 = CB == 1 ? half * RBW : 0, j0 = CB == 1 ? 0 : half * CBW;
  const int xr = lr % XR;  // (row blocks i of 16 rows follow each other)
  int x_at[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) x_at[t] = (i0 * 16 + xr) * S::XROW + kb0 * 256 + (((4 * t + hq) ^ xr) & 15) * 16;
  // this thread's outputs: V floats from e of the unit, registers e % 4 .. of a lane
  const int e = V * tid, eb = e / (4 * S::LPB), el = e / 4 % S::LPB;
  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.0f;
  auto add_sums = [&](int t) {
    const int buf = t % S::BUFS, left = (int)(g.groups - (int64_t)t * GPS);
    if (S::ELEMS < 64 * S::WAVES && e >= S::ELEMS) return;
    const int col = 16 * (eb % CB) + el % 16;
    constexpr int C = GPS < 16 ? GPS : 16;  // groups whose sums are read at once
#pragma unroll
    for (int k0 = 0; k0 < GPS; k0 += C) {
      float p[C][V], s[C];
#pragma unroll
      for (int k = 0; k < C; ++k) {
        s[k] = scl[buf][k0 + k][col];
#pragma unroll
        for (int v = 0; v < V; ++v) p[k][v] = part[buf][k0 + k][e + v];
      }
#pragma unroll
      for (int k = 0; k < C; ++k)
        if (k0 + k < left)
#pragma unroll
          for (int v = 0; v < V; ++v) acc[v] = fmaf(s[k], p[k][v], acc[v]);
    }
  };
  for (int t = 0; t < nt; ++t) {
    barrier();
    const char* const slot = ring + t % NS * S::STAGE;
    const int buf = t % S::BUFS;
    i32x4 a[U][4][RBW];
    u32x4 wt[U][CBW];
    unsigned sz[U][NG][CBW];
#pragma unroll
    for (int b = 0; b < U; ++b) {
#pragma unroll
      for (int i = 0; i < RBW; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          a[b][u][i] = *reinterpret_cast<const i32x4*>(slot + x_at[u] + b * (KW * 256) + i * 16 * S::XROW);
#pragma unroll
      for (int j = 0; j < CBW; ++j) {
        const int kb = kb0 + b * KW;
        wt[b][j] = *reinterpret_cast<const u32x4*>(slot + S::XBYTES + ((j0 + j) * SB + kb) * 1024 + lane * 16);
#pragma unroll
        for (int s = 0; s < NG; ++s)
          sz[b][s][j] = *reinterpret_cast<const unsigned*>(slot + S::XBYTES + S::WBYTES +
                                                           ((kb * NG + s) * CB + j0 + j) * 64 + lr * 4);
      }
    }
    // the chains of all the wave's groups side by side: first every start, ...
    f32x4 P[U][NG][RBW][CBW];
#pragma unroll
    for (int i = 0; i < RBW; ++i) {
      f32x4 X[U][NG];
#pragma unroll
      for (int u = 0; u < G / 32; ++u)
#pragma unroll
        for (int b = 0; b < U; ++b)
#pragma unroll
          for (int s = 0; s < NG; ++s)
            X[b][s] = mfma16_v<IN>(ones8<IN>(), a[b][s * (G / 32) + u][i], u == 0 ? f32x4{} : X[b][s]);
#pragma unroll
      for (int b = 0; b < U; ++b)
#pragma unroll
        for (int s = 0; s < NG; ++s) {
          const i32x2 x3 = split3(X[b][s][0]);
          const i32x4 xs{x3[0], x3[1], 0, 0};
#pragma unroll
          for (int j = 0; j < CBW; ++j) {
            P[b][s][i][j] = start_of_sum(xs, zero_operand(sz[b][s][j], first));
            hold(P[b][s][i][j]);
          }
        }
    }
    asm volatile("s_nop 15\n\ts_nop 15");
    __builtin_amdgcn_sched_barrier(0);
    // (the sums of the stage before under this one's matrix steps: 29 x 4096,
    // K = 14336, group 64 23.4 us, behind them 26.0)
    if (S::BUFS == 2 && t > 0) add_sums(t - 1);
    // ... then the steps over x and q
#pragma unroll
    for (int u = 0; u < G / 32; ++u)
#pragma unroll
      for (int b = 0; b < U; ++b)
#pragma unroll
        for (int s = 0; s < NG; ++s)
#pragma unroll
          for (int j = 0; j < CBW; ++j) {
            const i32x4 q = decode8<IN>(wt[b][j][s * (G / 32) + u]);
#pragma unroll
            for (int i = 0; i < RBW; ++i)
              P[b][s][i][j] = mfma16_v<IN>(a[b][s * (G / 32) + u][i], q, P[b][s][i][j]);
          }
#pragma unroll
    for (int b = 0; b < U; ++b)
#pragma unroll
      for (int s = 0; s < NG; ++s) {
        const int gr = (kb0 + b * KW) * NG + s;
#pragma unroll
        for (int j = 0; j < CBW; ++j) {
          if (hq == 0 && i0 == 0) scl[buf][gr][16 * (j0 + j) + lr] = scale_of<IN>(sz[b][s][j]);
#pragma unroll
          for (int i = 0; i < RBW; ++i)
            if (S::LPB == 64 || lane < S::LPB)
              *reinterpret_cast<f32x4*>(&part[buf][gr][(((i0 + i) * CB + j0 + j) * S::LPB + lane) * 4]) =
                  P[b][s][i][j];
        }
      }
    if constexpr (S::BUFS == 1) {
      barrier();
      add_sums(t);
    }
  }
  if constexpr (S::BUFS == 2) {
    barrier();
    if (nt > 0) add_sums(nt - 1);
  }
  if (S::ELEMS < 64 * S::WAVES && e >= S::ELEMS) return;
  const int64_t col = (nb0 + eb % CB) * 16 + el % 16;
  if (col >= g.N) return;
  const float bias = g.bias ? g.bias[col] : 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t row = m0 + 16 * (eb / CB) + 4 * (el / 16) + (e + v) % 4;
    if (row < g.M) store_out<IN>(g.y, row * g.N + col, g.bias ? acc[v] + bias : acc[v]);
  }
}

template <int IN, int G, int RB, int CB, int XR, int SB, int U, int H>
hipError_t launch_rows(const W4Args& a, hipStream_t s) {
  // at most 2^21 workgroups a launch (column groups stay below 2^19)
  const int64_t cgroups = (a.nblocks + CB - 1) / CB, most = ((int64_t)1 << 21) / cgroups * (16 * RB);
  for (int64_t m = 0; m < a.M; m += most) {
    W4Args b = a;
    b.M = a.M - m < most ? a.M - m : most;
    b.x = static_cast<const char*>(a.x) + m * a.K * 2;
    b.y = static_cast<char*>(a.y) + m * a.N * 2;
    const int64_t units = cgroups * ((b.M + 16 * RB - 1) / (16 * RB));
    hipLaunchKernelGGL((w4_rows_kernel<IN, G, RB, CB, XR, SB, U, H>), dim3((unsigned)units),
                       dim3(RowsShape<G, RB, CB, XR, SB, U, H>::THREADS), 0, s, b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// ---- many rows ---------------------------------------------------------------

// The three pieces of X = sum x for every (group, row), 8 bytes each,
// [groups, m_pad], by the chain of the few-rows kernel: one wave per 16 rows and
// group.  The tile kernel reads them instead of spending a fifth of its matrix
// steps on X (each column of waves would repeat them).  Rows past M repeat the
// last row.
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
  for (int t = 0; t < G / 32; ++t) X = mfma16_v<IN>(ones8<IN>(), a[t], X);
  if (lane < 16) static_cast<i32x2*>(g.sums)[gr * g.m_pad + row] = split3(X[0]);
}

// The same 8 bytes twice, as a 4-dword operand.
template <int OFF>
__device__ __forceinline__ i32x4 ds_read_b64_twice_at(unsigned addr) {
  static_assert(OFF % 8 == 0 && OFF >= 0 && OFF / 8 < 256, "ds_read2 offset field");
  i32x4 v;
  asm volatile("ds_read2_b64 %0, %1 offset0:%2 offset1:%2" : "=v"(v) : "v"(addr), "n"(OFF / 8));
  return v;
}
template <int OFF>
__device__ __forceinline__ unsigned ds_read_b32_at(unsigned addr) {
  static_assert(OFF >= 0 && OFF < 65536, "ds_read offset field");
  unsigned v;
  asm volatile("ds_read_b32 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "n"(OFF));
  return v;
}

// A copy in a register of its own (so that the next stage's weight blocks can
// land in the ones it came from).
__device__ __forceinline__ unsigned copied(unsigned v) {
  unsigned r;
  asm volatile("v_mov_b32 %0, %1" : "=v"(r) : "v"(v));
  return r;
}

// A workgroup of WM x WN waves owns a tile of TM x TN outputs, each wave FM x FN
// blocks of 16 x 16.  K is walked in stages of one 128-K block.  A ring of NS
// LDS stages (x rows of 256 bytes, packed weight blocks as they lie in memory,
// scale words and pieces of X) is filled by buffer->LDS DMA.  A wave decodes its
// own weight blocks from LDS to registers, sums a group into P on the matrix
// cores and folds P into acc with one fused multiply-add an element.  Every
// matrix step is followed by the vector work that fits under it: a quarter of
// the next block column's decoding and, in the last k-step of a group, the fold
// of the block column before.
//
// LDS reads are inline assembly with explicit waits (the compiler would make
// each wait for every DMA in flight), spread between the matrix steps: sixteen
// of them in a row, in all eight waves, held the steps up for 500 cycles.  The stage change sits before the last
// k-step: all of the wave's reads of stage t have landed, its DMA of stage t + 1
// too, and after one barrier the first fragments of stage t + 1 are read under
// that k-step's arithmetic.  The refill of stage t's slot is spread over the
// next four k-steps: the eight waves' transfers, issued at once, would stall
// each other's matrix steps behind them.
//
// 16-byte chunk c of an x row r lies at slot c ^ (r & 15): the 16 rows that a
// quarter of a wave reads at one chunk fall on different banks.
template <int G, int FM, int FN, int WM, int WN, int NS>
struct TileShape {
  static constexpr int TM = 16 * FM * WM, TN = 16 * FN * WN, WAVES = WM * WN;
  static constexpr int NG = 128 / G;
  static constexpr int A_STAGE = TM * 256, B_STAGE = TN * 64;
  static constexpr int RS = 1024 / (TN * 4), RX = 1024 / (TM * 8);  // rows per 1 KB transfer
  static constexpr int IS = (NG + RS - 1) / RS, IX = (NG + RX - 1) / RX;
  static constexpr int ITEMS = IS + IX;
  static constexpr int STAGE = A_STAGE + B_STAGE + ITEMS * 1024;
  static constexpr int LDS = NS * STAGE;
  // transfers of 1 KB: DA of x rows per wave, then the weight blocks and the
  // items dealt out to the waves in turn (REST of them, waves below MORE one more)
  static constexpr int DA = A_STAGE / 1024 / WAVES, NB = B_STAGE / 1024;
  static constexpr int REST = (NB + ITEMS) / WAVES, MORE = (NB + ITEMS) % WAVES;
  static constexpr int DMAS = DA + REST + (MORE ? 1 : 0);
  static_assert(DA * WAVES * 1024 == A_STAGE, "DMA split");
  static_assert(ITEMS <= WAVES && RS >= 1 && RX >= 1, "one scale or sum transfer per wave");
  static_assert(LDS <= 160 * 1024, "LDS");
  // where the scale words and the pieces of group gi lie behind the blocks
  static constexpr int sz_at(int gi) { return gi / RS * 1024 + gi % RS * (TN * 4); }
  static constexpr int x_at(int gi) { return (IS + gi / RX) * 1024 + gi % RX * (TM * 8); }
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

  // ---- DMA.  Transfer i of x of this wave fills rows 4 (w DA + i) .. + 3: lane l
  // brings chunk c of row l / 16, which belongs at slot l % 16.  What depends on
  // the lane alone is made once (a row past M reads out of range: zeros), what
  // the wave shares goes into the scalar offset, so that a transfer costs no
  // vector work.
  unsigned a_off[S::DA];
#pragma unroll
  for (int i = 0; i < S::DA; ++i) {
    const int row = 4 * (w * S::DA + i) + lane / 16, c = (lane % 16) ^ (row & 15);
    a_off[i] = m0 + row < g.M ? (unsigned)(lane / 16 * g.K * 2 + c * 16) : OOB;
  }
  const unsigned b_off = lane * 16;
  // the wave's item, if below ITEMS: 1 KB of scale words (rows of 4 TN bytes) or of
  // pieces of X (rows of 8 TM bytes), a row per group of the stage
  const int item = (w + S::WAVES - S::NB % S::WAVES) % S::WAVES;
  const bool sums = item >= S::IS;
  const int64_t mpitch = sums ? g.m_pad * 8 : np * 4;
  const int mrow = sums ? lane / (TM / 2) : lane / (TN / 4);
  const int mat = (sums ? lane % (TM / 2) : lane % (TN / 4)) * 16;
  const int mgroup = (sums ? (item - S::IS) * S::RX : item * S::RS) + mrow;  // this lane's group
  const unsigned m_off = mgroup < NG && mrow < (sums ? S::RX : S::RS) &&
                                 (sums || nb0 * 64 + mat < np * 4)
                             ? (unsigned)(mgroup * mpitch + mat)
                             : OOB;
  const auto abuf = buffer_at(static_cast<const char*>(g.x) + m0 * g.K * 2);
  const auto bbuf = buffer_at(static_cast<const char*>(g.packed) + nb0 * g.kblocks * 1024);
  const auto mbuf = buffer_at(sums ? static_cast<const char*>(g.sums) + m0 * 8
                                   : reinterpret_cast<const char*>(g.sz) + nb0 * 64);
  const int a_pitch = (int)(8 * g.K), b_pitch = (int)(g.kblocks * 1024), m_step = (int)(mpitch * NG);
  // Transfer x of this wave for stage t, into the slot at `slot`.
  constexpr int DMAS = S::DMAS;
  const int whole = (int)(g.K / 128);  // stages before a partial one
  auto dma_one = [&](int t, int slot, int x) {
    if (x < S::DA) {
      const int q = w * S::DA + x;
      unsigned off = a_off[x];
      if (t >= whole) {  // chunks past K: zeros
        const int c = (lane % 16) ^ ((4 * q + lane / 16) & 15);
        off = 8 * c < g.K - (int64_t)t * 128 ? off : OOB;
      }
      dma16(abuf, lds + slot + q * 1024, off, q * a_pitch + t * 256);
      return;
    }
    const int j = (x - S::DA) * S::WAVES + w;
    if ((x - S::DA + 1) * S::WAVES <= S::NB || j < S::NB)
      dma16(bbuf, lds + slot + S::A_STAGE + j * 1024, nb0 + j < g.nblocks ? b_off : OOB,
            j * b_pitch + t * 1024);
    else if (j - S::NB < S::ITEMS)
      dma16(mbuf, lds + slot + S::A_STAGE + S::B_STAGE + item * 1024,
            t * NG + mgroup < groups ? m_off : OOB, t * m_step);
  };
  auto fence = [&]() { __builtin_amdgcn_sched_barrier(0); };
  auto lds_wait = [&]() {
    fence();
    __builtin_amdgcn_s_waitcnt(lgkmcnt_imm(0));
    fence();
  };
  // All transfers of a stage landed, those of the `later` stages after it in
  // flight; then every wave's.
  auto dma_wait = [&](auto LATER) {
    constexpr int later = decltype(LATER)::value, D = S::DA + S::REST;
    fence();
    if (w < S::MORE)
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(later * (D + 1)));
    else
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(later * D));
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
  const unsigned s_rd = lds0 + S::A_STAGE + S::B_STAGE + (wn * FN * 16 + lb) * 4;
  const unsigned x_rd = lds0 + S::A_STAGE + S::B_STAGE + (wm * FM * 16 + lb) * 8;
  const unsigned first_lanes = hq == 0 ? ~0u : 0u;

  i32x4 A[2][FM], W[FN];
  i32x4 X[FM];        // pieces (twice) of the next group to start, and its scale words
  unsigned sz[FN];
  f32x4 P[FM][FN], acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = P[i][j] = f32x4{};

  // LDS read r of those that a k-step ks issues for the k-step after it, from the
  // slot at `from`: (after the last k-step of a stage) the weight blocks, the x
  // fragments and (where a group starts there) its scale words and pieces.
  auto read_next = [&](auto KS, auto R, int from) {
    constexpr int ks = (decltype(KS)::value + 1) % 4, nw = ks == 0 ? FN : 0, r = decltype(R)::value;
    constexpr int gi = ks / KPG;
    if constexpr (r < nw)
      W[r] = ds_read_b128_at<r * 1024>(b_rd + from);
    else if constexpr (r < nw + FM)
      A[ks & 1][r - nw] = ds_read_b128_at<(r - nw) * 4096>(a_rd[ks] + from);
    else if constexpr (r < nw + FM + FN)
      sz[r - nw - FM] = ds_read_b32_at<S::sz_at(gi) + (r - nw - FM) * 64>(s_rd + from);
    else
      X[r - nw - FM - FN] = ds_read_b64_twice_at<(r - nw - FM - FN) * 128>(x_rd + (from + S::x_at(gi)));
  };
  // how many there are
  auto reads_of = [](int ks) { return (ks == 3 ? FN : 0) + FM + ((ks + 1) % KPG == 0 ? FN + FM : 0); };

  for (int t = 0; t < NS && t < nt; ++t) {
#pragma unroll
    for (int x = 0; x < DMAS; ++x) dma_one(t, t * S::STAGE, x);
  }
  if (nt >= NS)
    dma_wait(std::integral_constant<int, NS - 1>{});
  else
    dma_wait(std::integral_constant<int, 0>{});
  static_for<0, 2 * (FM + FN)>([&](auto R) { read_next(std::integral_constant<int, 3>{}, R, 0); });
  lds_wait();

  float sc[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) sc[j] = 0.0f;
  int slot = 0, prev = 0;  // of stage t, of the stage before
  for (int t = 0; t < nt; ++t) {
    const int next = slot + S::STAGE < NS * S::STAGE ? slot + S::STAGE : 0;
    static_for<0, 4>([&](auto KS) {
      constexpr int ks = decltype(KS)::value;
      constexpr bool first = ks % KPG == 0;       // this k-step starts a group
      constexpr bool ends = (ks + 1) % KPG == 0;  // ... ends one
      if constexpr (ks > 0) lds_wait();  // this k-step's fragments
      unsigned wd[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) wd[j] = ks < 3 ? (unsigned)W[j][ks] : copied((unsigned)W[j][ks]);
      if constexpr (first) {
        // P starts as -z X.  A group past K gets the scale -0, whose fold (of a
        // sum of zeros) leaves every acc as it is.
        const bool exists = t * NG + ks / KPG < groups;
        static_for<0, FN>([&](auto J) {
          constexpr int j = decltype(J)::value;
          const i32x4 z = zero_operand(sz[j], first_lanes);
          sc[j] = exists ? scale_of<IN>(sz[j]) : -0.0f;
#pragma unroll
          for (int i = 0; i < FM; ++i) {
            P[i][j] = start_of_sum(X[i], z);
            hold(P[i][j]);
          }
        });
      }
      i32x4 b = decode8<IN>(wd[0]), bn{};
      fence();
      if constexpr (ks == 3) {
        if (t + NS <= nt)  // the stages t + 2 .. t + NS - 1 are in flight
          dma_wait(std::integral_constant<int, NS - 2>{});
        else
          dma_wait(std::integral_constant<int, 0>{});
      }
      auto fold = [&](int i, int j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(sc[j], P[i][j][e], acc[i][j][e]);
        // holds the fold at its place (instruction selection may otherwise sink
        // it past later k-steps, with P alive until there)
        hold(acc[i][j]);
      };
      static_for<0, FN>([&](auto J) {
        constexpr int j = decltype(J)::value;
        static_for<0, FM>([&](auto I) {
          constexpr int i = decltype(I)::value;
          P[i][j] = mfma16_v<IN>(A[ks & 1][i], b, P[i][j]);
          if constexpr (j + 1 < FN) {
#pragma unroll
            for (int p = i * 4 / FM; p < (i + 1) * 4 / FM; ++p) bn[p] = decode_pair<IN>(wd[j + 1], p);
          }
          if constexpr (ends && j > 0) fold(i, j - 1);
          // the next k-step's LDS reads, over the first three quarters
          constexpr int blk = j * FM + i, SPAN = FM * FN * 3 / 4, NR = reads_of(ks);
          static_for<(blk < SPAN ? blk * NR / SPAN : NR), (blk < SPAN ? (blk + 1) * NR / SPAN : NR)>(
              [&](auto R) { read_next(KS, R, ks == 3 ? next : slot); });
          // the refill of the slot that the last stage change freed
          constexpr int at = ((ks + 1) % 4 * FN + j) * FM + i, NB = 4 * FM * FN;
#pragma unroll
          for (int x = at * DMAS / NB; x < (at + 1) * DMAS / NB; ++x) {
            const int r = ks == 3 ? t + NS : t + NS - 1;
            if (r >= NS && r < nt) dma_one(r, ks == 3 ? slot : prev, x);
          }
          fence();
        });
        b = bn;
      });
      if constexpr (ends) {
#pragma unroll
        for (int i = 0; i < FM; ++i) fold(i, FN - 1);
      }
      if constexpr (ks == 3) lds_wait();  // before the loop's own register copies
    });
    prev = slot;
    slot = next;
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
#pragma unroll
  for (int i = 0; i < FM; ++i) keep_live<4>(X[i]);
#pragma unroll
  for (int j = 0; j < FN; ++j) asm volatile("" : : "v"(sz[j]));
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

// Which tile takes a grid: 64 x 128 (four waves of 64 x 32; three workgroups
// share a compute unit and fill each other's waits) or 128 x 256 (eight waves of
// 64 x 64, alone on its unit).  The large one shares its decoding among more
// rows and is 5 % faster on a full machine (4096 x 14336, K = 4096, group 128: 532
// against 558 us), the small one fills small and odd grids (256 x 6144: 49
// against 74 us, 2048 x 6144: 129 against 147, but 2048 x 4096, four workgroups a
// unit, 114 against 88).  Cost in us per K = 4096 on 256 units: 72 a round of large
// tiles; 60 for three small tiles on a unit, 36 and 46 for one or two left over.
// Other groups and K scale all of them: at ten grids (256 to 4096 rows, 4096 to 14336
// columns) in both types the rule's tile is the faster one, or within 4 %, for
// groups 64 (2048 x 6144: small 148, large 171 us; 2048 x 4096: 108, 96) and 32
// (203, 230; 142, 132) as for 128.  Bits do not depend on the tile.
bool large_tiles(int64_t M, int64_t N) {
  auto per_unit = [&](int64_t tm, int64_t tn) {
    return (((M + tm - 1) / tm) * ((N + tn - 1) / tn) + 255) / 256;
  };
  const int64_t n = per_unit(64, 128), left = n % 3;
  return 72 * per_unit(128, 256) < n / 3 * 60 + (left == 0 ? 0 : left == 1 ? 36 : 46);
}

// Blocks of 16 columns in a unit of the few-rows kernel: the fewest that leave at
// most one unit for each of 256 compute units, up to four (two for pairs of row
// blocks with groups below 128, whose sums fill the LDS).  Wide units read x once
// for more columns and share the chain's fixed costs, narrow ones fill the machine
// (us, one, two and four blocks, in the kernel's first form: 64 x 14336, K = 4096
// 55, 40, 31; 1 x 4096, K = 14336 12.5, 16.9, 26.3).
int few_rows_columns(int64_t M, int64_t N, int G) {
  const int64_t units = (N + 15) / 16 * (M <= 16 ? 1 : (M + 31) / 32);
  return units <= 256 ? 1 : units <= 512 || (G != 128 && M > 16) ? 2 : 4;
}

template <int IN, int G>
hipError_t launch_group(const W4Args& a, hipStream_t s) {
  if (a.sums)
    return large_tiles(a.M, a.N) ? launch_tile<IN, G, 4, 4, 2, 4, G == 32 ? 2 : 3>(a, s)
                                 : launch_tile<IN, G, 4, 2, 1, 4, 2>(a, s);
  const int cb = few_rows_columns(a.M, a.N, G);
  // Stages of eight blocks where a column block is all a unit has (at 16 rows; four
  // blocks: 16 x 4096, K = 14336 18.7 us against 13.8), of sixteen at 4 rows, two
  // blocks a wave (eight, one a wave: 1 x 4096, K = 14336 12.8 against 10.8); of four
  // where x or the sums take the LDS.  More waves beat more blocks a wave where both
  // fit (16 x 14336, K = 4096: 11.4 us, with two blocks on half the waves 13.1).
  constexpr bool FINE = G == 32;  // many sums: less of LDS is left for the stages
  if (a.M <= 4)
    return cb == 4   ? launch_rows<IN, G, 1, 4, 4, 8, 1, 1>(a, s)
           : cb == 2 ? launch_rows<IN, G, 1, 2, 4, FINE ? 8 : 16, FINE ? 1 : 2, 1>(a, s)
                     : launch_rows<IN, G, 1, 1, 4, FINE ? 8 : 16, FINE ? 1 : 2, 1>(a, s);
  // (more rows too, 16 to a unit, where those units still fit the machine: 64 x 1024,
  // K = 4096 5.9 us against 7.6 with 32, 48 x 512, K = 8192 7.9 against 11.6)
  if (a.M <= 16 || a.nblocks * ((a.M + 15) / 16) <= 256)
    return cb == 4   ? launch_rows<IN, G, 1, 4, 16, 4, 1, 2>(a, s)
           : cb == 2 ? launch_rows<IN, G, 1, 2, 16, FINE ? 4 : 8, 1, FINE ? 2 : 1>(a, s)
                     : launch_rows<IN, G, 1, 1, 16, 8, 1, 1>(a, s);
  if constexpr (G == 128)
    if (cb == 4) return launch_rows<IN, G, 2, 4, 32, 4, 1, 2>(a, s);
  return cb == 2 ? launch_rows<IN, G, 2, 2, 32, 4, 1, 2>(a, s) : launch_rows<IN, G, 2, 1, 32, 4, 1, 2>(a, s);
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
  // (a launch holds fewer than 2^32 threads)
  auto grid = [](int64_t items) { return dim3((unsigned)std::min((items + 255) / 256, (int64_t)1 << 20)); };
  hipLaunchKernelGGL(w4_pack_kernel, grid(dwords), dim3(256), 0, s, static_cast<const unsigned char*>(q),
                     out, N, K, kblocks, dwords);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(w4_pack_scales_kernel, grid(pairs), dim3(256), 0, s,
                     static_cast<const unsigned short*>(scales),
                     static_cast<const unsigned char*>(zeros), out + dwords, N, nblocks * 16, groups);
  return hipGetLastError();
}

// The tile kernel takes what would be many units of the few-rows kernel.  In us at
// K = 4096, few rows against tiles: group 128, 256 x 6144 (768 units) 36 and 49,
// 128 x 14336 (896) 47 and 50, 512 x 4096 (1024) 48 and 44; group 64, 256 x 4096 (1024)
// 43 and 49, 128 x 6144 (768) 33 and 55, 96 x 14336 (1344) 62 and 56; group 32,
// 128 x 4096 (512) 37 and 57, 256 x 4096 (1024) 71 and 57.  16 rows are bound by the
// weights in both, up to the widest: 16 x 131072 75 and 96 us, group 32 139 and 137.
bool w4_uses_tiles(int64_t M, int64_t N, int64_t K, int group) {
  const int64_t cb = few_rows_columns(M, N, group), cgroups = ((N + 15) / 16 + cb - 1) / cb;
  const int64_t most = group == 128 ? 960 : group == 64 ? 1024 : 512;
  if (M <= 16 || cgroups * ((M + 31) / 32) <= most) return false;
  // the tile kernel's 31-bit offsets: within 128 rows of x, within the scale
  // words and within the pieces of X
  const int64_t groups = K / group, wide = N + 16 > 2 * (M + kW4RowPad) ? N + 16 : 2 * (M + kW4RowPad);
  return K > 0 && 256 * K < kMaxOffset && groups * wide * 4 < kMaxOffset;
}

hipError_t launch_w4(int in, const W4Args& a, hipStream_t s) {
  return in == GEMM_F16 ? launch_in<GEMM_F16>(a, s) : launch_in<GEMM_BF16>(a, s);
}

}  // namespace imm
