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
// and one rounding of acc + b.  Nothing but x and s is ever rounded to 16 bits:
// the product is as exact as one with fp32 weights.  (Rounding s (q - z) to 16
// bits first, as a 16-bit weight would be, costs a bf16 result half its
// accuracy.  z as a matrix step leaves the vector unit, whose work does not
// hide in the tile kernel, one multiply-add per element and group; a second one
// in place of that step was as fast within two per cent.)
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

// One thread per (group, output): the scale's bits and the zero point's negative
// (8 without zero points); padding outputs get zeros.
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
    r = scales[at] | (__float_as_uint(-(zeros ? (float)zeros[at] : 8.0f)) & 0xffff0000u);
  }
  sz[i] = r;
}

// ---- few rows ----------------------------------------------------------------

// A workgroup of 8 waves makes a unit of RB x CB blocks of 16 x 16 outputs at a
// time.  The waves share K: in a round, wave w takes U of the 128-K blocks w,
// w + 8, ..., and leaves P of its groups in LDS; after a barrier every thread adds
// the round's groups of its outputs in ascending order, which keeps the order of
// the sum the one above.  The grid is kSkinnyGroups workgroups at most (two on a
// compute unit where registers allow: one's sums run under the other's matrix
// steps) and each walks its units (column groups of a row group) and their rounds
// as one sequence, with the weights of the next two rounds and the rows and scale
// words of the next one in flight.  Loads return in order: a round's rows are
// requested before the weights of the round after it, so waiting for them leaves
// those in flight.  Few rows and many columns are bound by the stream of the
// weights (1 x 131072, K = 4096: 65 us, 4.1 TB/s); small grids by the round, some
// 3 us of latencies (1 x 4096, K = 4096: 5.7 us; one round of four blocks a wave and
// one workgroup a unit: 6.9), more rows by the reads of x that every column
// group repeats (see skinny_columns).
template <int G, int RB, int CB>
struct SkinnyShape {
  static constexpr int W = 8;
  static constexpr int NG = 128 / G;                  // groups per 128-K block
  static constexpr int ELEMS = 256 * RB * CB;
  // blocks per wave and round: up to 2, within 32 fragments of x and 64 KB of sums
  static constexpr int UR = 2 / RB, UL = 64 / (W * NG * RB * CB);
  static constexpr int U = UL < 1 ? 1 : UL < UR ? UL : UR;
  static constexpr int GPR = W * U * NG;              // groups per round
  static constexpr int PER = (ELEMS + 511) / 512;     // outputs per thread
  // sums of two rounds where they fit; one, and a barrier more, where not
  static constexpr int ROUND = GPR * (ELEMS + 16 * CB) * 4;
  static constexpr int BUFS = 2 * ROUND <= 160 * 1024 ? 2 : 1;
  static constexpr int LDS = BUFS * ROUND;
};
constexpr int64_t kSkinnyGroups = 512;

template <int IN, int G, int RB, int CB>
__global__ __launch_bounds__(512, 2) void w4_skinny_kernel(W4Args g) {
  using S = SkinnyShape<G, RB, CB>;
  constexpr int W = S::W, NG = S::NG, U = S::U, GPR = S::GPR, ELEMS = S::ELEMS, PER = S::PER;
  static_assert(S::LDS <= 160 * 1024, "LDS");
  __shared__ __attribute__((aligned(16))) float part[S::BUFS][GPR][ELEMS];
  __shared__ float scl[S::BUFS][GPR][16 * CB];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane % 16, hq = lane / 16;
  const unsigned first = hq == 0 ? ~0u : 0u;
  const int64_t cgroups = (g.nblocks + CB - 1) / CB;
  const int64_t units = cgroups * ((g.M + 16 * RB - 1) / (16 * RB));
  const int kblocks = (int)g.kblocks, ksteps = (int)(g.K / 32);
  const int rounds = kblocks > 0 ? (kblocks + W * U - 1) / (W * U) : 1;
  const int64_t np = g.nblocks * 16;

  // A place in the sequence: round r of a unit, and the unit's first row and
  // column block.
  struct Place {
    unsigned unit, rg, cg;
    int r;
  };
  const unsigned nunits = (unsigned)units, ncg = (unsigned)cgroups;
  auto place_at = [&](unsigned unit) { return Place{unit, unit / ncg, unit % ncg, 0}; };
  auto advance = [&](Place& p) {
    if (++p.r == rounds) p = place_at(p.unit + gridDim.x);
  };
  // No load is predicated: what a round reads past the last row, column block,
  // K block or group is another row's or block's (or, past the end of its
  // matrix, zeros), goes into sums that nothing adds up, or into rows and columns
  // that are never stored.  Offsets: the lane's, made once, and the wave's.
  const unsigned x_off = (unsigned)(lr * g.K * 2 + 16 * hq), x_block = (unsigned)(32 * g.K);
  const unsigned w_off = lane * 16, w_block = (unsigned)(g.kblocks * 1024);
  const unsigned s_off = lr * 4, s_group = (unsigned)(np * 4);
  auto load_weights = [&](const Place& p, u32x4 (&wt)[U][CB]) {
    const int64_t at = ((int64_t)p.cg * CB * kblocks + (int64_t)p.r * U * W + w) * 1024;
    const int64_t end = g.nblocks * g.kblocks * 1024;
    const auto buf = buffer_at(static_cast<const char*>(g.packed) + (at < end ? at : 0),
                               p.unit < nunits && at < end ? end - at : 0);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < CB; ++j) wt[u][j] = load_b128(buf, w_off + (u * (W * 1024) + j * w_block));
  };
  auto load_rows = [&](const Place& p, i32x4 (&a)[U][4][RB], unsigned (&sz)[U][NG][CB]) {
    const int64_t m0 = (int64_t)p.rg * (16 * RB), k0 = ((int64_t)p.r * U * W + w) * 128;
    const int64_t xat = (m0 * g.K + k0) * 2, xend = g.M * g.K * 2;
    const auto xbuf = buffer_at(static_cast<const char*>(g.x) + (xat < xend ? xat : 0),
                                p.unit < nunits && xat < xend ? xend - xat : 0);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t)
          a[u][t][i] = __builtin_bit_cast(i32x4, load_b128(xbuf, x_off + (u * (W * 256) + t * 64 + i * x_block)));
    const int64_t sat = (k0 / G * np + (int64_t)p.cg * CB * 16) * 4, send = g.groups * np * 4;
    const auto sbuf = buffer_at(reinterpret_cast<const char*>(g.sz) + (sat < send ? sat : 0),
                                p.unit < nunits && sat < send ? send - sat : 0);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int s = 0; s < NG; ++s)
#pragma unroll
        for (int j = 0; j < CB; ++j)
          sz[u][s][j] = load_b32(sbuf, s_off + ((unsigned)(u * W * NG + s) * s_group + j * 64));
  };

  u32x4 wt[2][U][CB];
  i32x4 a[2][U][4][RB];
  unsigned sz[2][U][NG][CB];
  float acc[PER];
#pragma unroll
  for (int p = 0; p < PER; ++p) acc[p] = 0.0f;
  Place now = place_at(blockIdx.x), rows = now, weights = now;
  load_weights(weights, wt[0]);
  advance(weights);
  load_rows(rows, a[0], sz[0]);
  advance(rows);
  load_weights(weights, wt[1]);
  advance(weights);

  auto step = [&](auto BUF) {
    constexpr int buf = decltype(BUF)::value, sums = buf % S::BUFS;
    // element e of a unit: block e / 256, lane (e / 4) % 64, register e % 4 of its
    // accumulators
    auto column = [&](int e) {
      return ((int64_t)now.cg * CB + (e / 256) % CB) * 16 + (e / 4) % 16;
    };
    // (the bias before the loads that stay in flight past its use)
    float bias[PER];
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const int e = tid + 512 * p;
      bias[p] = 0.0f;
      if (g.bias && now.r == rounds - 1 && e < ELEMS && column(e) < g.N) bias[p] = g.bias[column(e)];
    }
    load_rows(rows, a[1 - buf], sz[1 - buf]);
    advance(rows);
    // the chains of all the wave's groups side by side: first every start, ...
    f32x4 P[U][NG][RB][CB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      f32x4 X[U][NG];
#pragma unroll
      for (int t = 0; t < G / 32; ++t)
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int s = 0; s < NG; ++s)
            X[u][s] = mfma16_v<IN>(ones8<IN>(), a[buf][u][s * (G / 32) + t][i], t == 0 ? f32x4{} : X[u][s]);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int s = 0; s < NG; ++s) {
          const i32x2 x3 = split3(X[u][s][0]);
          const i32x4 xs{x3[0], x3[1], 0, 0};
#pragma unroll
          for (int j = 0; j < CB; ++j) {
            P[u][s][i][j] = start_of_sum(xs, zero_operand(sz[buf][u][s][j], first));
            hold(P[u][s][i][j]);
          }
        }
    }
    asm volatile("s_nop 15\n\ts_nop 15");
    __builtin_amdgcn_sched_barrier(0);
    // ... then the steps over x and q
#pragma unroll
    for (int t = 0; t < G / 32; ++t)
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int s = 0; s < NG; ++s)
#pragma unroll
          for (int j = 0; j < CB; ++j) {
            const i32x4 b = decode8<IN>(wt[buf][u][j][s * (G / 32) + t]);
#pragma unroll
            for (int i = 0; i < RB; ++i)
              P[u][s][i][j] = mfma16_v<IN>(a[buf][u][s * (G / 32) + t][i], b, P[u][s][i][j]);
          }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int s = 0; s < NG; ++s) {
        const int gr = (u * W + w) * NG + s;
#pragma unroll
        for (int j = 0; j < CB; ++j) {
          if (hq == 0) scl[sums][gr][16 * j + lr] = scale_of<IN>(sz[buf][u][s][j]);
#pragma unroll
          for (int i = 0; i < RB; ++i)
            *reinterpret_cast<f32x4*>(&part[sums][gr][((i * CB + j) * 64 + lane) * 4]) = P[u][s][i][j];
        }
      }
    load_weights(weights, wt[buf]);
    advance(weights);
    // One barrier a round: the buffer filled two rounds on was read before the
    // next round's barrier.  (Fences of LDS alone: __syncthreads would wait for
    // the loads in flight.)
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    const int64_t left = g.groups - (int64_t)now.r * GPR;
    const int ng = left < GPR ? (int)left : GPR;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const int e = tid + 512 * p;
      if (e < ELEMS) {
        const int col = 16 * ((e / 256) % CB) + (e / 4) % 16;
        constexpr int C = GPR < 16 ? GPR : 16;  // groups whose sums are read at once
        static_assert(GPR % C == 0, "round");
        int k = 0;
        for (; k + C <= ng; k += C) {
          float v[C], sc[C];
#pragma unroll
          for (int c = 0; c < C; ++c) {
            v[c] = part[sums][k + c][e];
            sc[c] = scl[sums][k + c][col];
          }
#pragma unroll
          for (int c = 0; c < C; ++c) acc[p] = fmaf(sc[c], v[c], acc[p]);
        }
        for (; k < ng; ++k) acc[p] = fmaf(scl[sums][k][col], part[sums][k][e], acc[p]);
        if (now.r == rounds - 1) {
          const int64_t row = (int64_t)now.rg * (16 * RB) + 16 * (e / 256 / CB) + 4 * ((e / 4) % 64 / 16) + e % 4;
          const int64_t out = column(e);
          if (row < g.M && out < g.N) store_out<IN>(g.y, row * g.N + out, g.bias ? acc[p] + bias[p] : acc[p]);
          acc[p] = 0.0f;
        }
      }
    }
    if constexpr (S::BUFS == 1) {
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    }
    advance(now);
  };
  while (now.unit < nunits) {
    step(std::integral_constant<int, 0>{});
    if (now.unit >= nunits) break;
    step(std::integral_constant<int, 1>{});
  }
}

template <int IN, int G, int RB, int CB>
hipError_t launch_skinny(const W4Args& a, hipStream_t s) {
  const int64_t units = (a.nblocks + CB - 1) / CB * ((a.M + 16 * RB - 1) / (16 * RB));
  hipLaunchKernelGGL((w4_skinny_kernel<IN, G, RB, CB>),
                     dim3((unsigned)(units < kSkinnyGroups ? units : kSkinnyGroups)), dim3(512), 0, s, a);
  return hipGetLastError();
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
  const auto abuf = buffer_at(static_cast<const char*>(g.x) + m0 * g.K * 2, kMaxOffset * 2);
  const auto bbuf = buffer_at(static_cast<const char*>(g.packed) + nb0 * g.kblocks * 1024, kMaxOffset * 2);
  const auto mbuf = buffer_at(sums ? static_cast<const char*>(g.sums) + m0 * 8
                                   : reinterpret_cast<const char*>(g.sz) + nb0 * 64, kMaxOffset * 2);
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
// tiles; 60 for three small tiles on a unit, 36 and 46 for one or two left over
// (other groups and K scale all of them).  Bits do not depend on the tile.
bool large_tiles(int64_t M, int64_t N) {
  auto per_unit = [&](int64_t tm, int64_t tn) {
    return (((M + tm - 1) / tm) * ((N + tn - 1) / tn) + 255) / 256;
  };
  const int64_t n = per_unit(64, 128), left = n % 3;
  return 72 * per_unit(128, 256) < n / 3 * 60 + (left == 0 ? 0 : left == 1 ? 36 : 46);
}

// Blocks of 16 columns in a unit of the few-rows kernel: the fewest that leave at
// most one unit for each of 256 compute units, up to four (two for pairs of row
// blocks with groups of 32, whose sums fill the LDS).  Wide units read x once for
// more columns and share the chain's fixed costs (64 x 14336, K = 4096: one block
// 55 us, two 40, four 31; 16 x 14336: 20.6, 17.3, 14.1), narrow ones fill the machine
// (64 x 4096: two 12.4, four 15.7; 1 x 4096, K = 14336: one 12.5, two 16.9, four 26.3).
int skinny_columns(int64_t M, int64_t N, int G) {
  const int64_t units = (N + 15) / 16 * (M <= 16 ? 1 : (M + 31) / 32);
  return units <= 256 ? 1 : units <= 512 || (G == 32 && M > 16) ? 2 : 4;
}

template <int IN, int G>
hipError_t launch_group(const W4Args& a, hipStream_t s) {
  if (a.sums)
    return large_tiles(a.M, a.N) ? launch_tile<IN, G, 4, 4, 2, 4, G == 32 ? 2 : 3>(a, s)
                                 : launch_tile<IN, G, 4, 2, 1, 4, 2>(a, s);
  const int cb = skinny_columns(a.M, a.N, G);
  if (a.M <= 16)
    return cb == 4 ? launch_skinny<IN, G, 1, 4>(a, s)
                   : cb == 2 ? launch_skinny<IN, G, 1, 2>(a, s) : launch_skinny<IN, G, 1, 1>(a, s);
  if constexpr (G != 32)
    if (cb == 4) return launch_skinny<IN, G, 2, 4>(a, s);
  return cb == 2 ? launch_skinny<IN, G, 2, 2>(a, s) : launch_skinny<IN, G, 2, 1>(a, s);
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

// The tile kernel takes what the few-rows kernel would need more than three units
// on a compute unit for (two with shorter groups, which are dearer there).  In us at
// K = 4096, few rows against tiles: group 128, 256 x 6144 (three units) 42 and
// 49, 512 x 4096 (four) 54 and 45; group 64, 128 x 6144 (two) 41 and 55,
// 256 x 6144 (three) 59 and 55; group 32, 128 x 4096 (two) 38 and 57, 512 x 2048 at
// K = 8192 (eight) 167 and 111.  16 rows are bound by the weights in both, up to the
// widest: 16 x 131072 74 and 96 us, group 32 140 and 137.
bool w4_uses_tiles(int64_t M, int64_t N, int64_t K, int group) {
  const int64_t cb = skinny_columns(M, N, group), cgroups = ((N + 15) / 16 + cb - 1) / cb;
  if (M <= 16 || cgroups * ((M + 31) / 32) <= (group == 128 ? 3 : 2) * 256) return false;
  // the tile kernel's 31-bit offsets: within 128 rows of x, within the scale
  // words and within the pieces of X
  const int64_t groups = K / group, wide = N + 16 > 2 * (M + kW4RowPad) ? N + 16 : 2 * (M + kW4RowPad);
  return K > 0 && 256 * K < kMaxOffset && groups * wide * 4 < kMaxOffset;
}

hipError_t launch_w4(int in, const W4Args& a, hipStream_t s) {
  return in == GEMM_F16 ? launch_in<GEMM_F16>(a, s) : launch_in<GEMM_BF16>(a, s);
}

}  // namespace imm
