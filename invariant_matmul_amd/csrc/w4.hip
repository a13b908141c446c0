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

template <int IN, int G, int RB, int CB>
hipError_t launch_skinny(const W4Args& a, hipStream_t s) {
  const int64_t cg = (a.nblocks + CB - 1) / CB, rg = (a.M + 16 * RB - 1) / (16 * RB);
  hipLaunchKernelGGL((w4_skinny_kernel<IN, G, RB, CB>), dim3((unsigned)(cg * rg)), dim3(512), 0, s, a);
  return hipGetLastError();
}

template <int IN, int G>
hipError_t launch_group(const W4Args& a, hipStream_t s) {
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

hipError_t launch_w4(int in, const W4Args& a, hipStream_t s) {
  return in == GEMM_F16 ? launch_in<GEMM_F16>(a, s) : launch_in<GEMM_BF16>(a, s);
}

}  // namespace imm
