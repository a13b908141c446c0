// Row kernels beside the GEMM: root-mean-square norm with the residual's
// addition (16-bit or fp8 output with a scale per row), its backward pass, and
// the fp8 quantisation of rows.
//
//   h = round(x + r)                      (h = x without a residual)
//   rstd = 1 / sqrt(sum_k h_k^2 / cols + eps)
//   t_k = (h_k * rstd) * w_k              (t = x in the plain quantisation)
//   y_k = round(t_k), or q_k = round8(t_k / scale) with
//   scale = max(max_k |t_k| / FMAX, 2^-120), both quotients rounded in fp32
//
// All of it is one pass over memory: a row's 16-byte vectors stay in the
// registers of the threads that own the row between the sum of squares, the
// maximum and the store, so each input is read once and each output written
// once.  The bytes bound it: about 10 operations an element, against 4 bytes (16-bit;
// with a residual 8) in whose time the vector units could do 20.  Measured:
// 8191 x 8192 fp16 with a residual 97 to 99 us (5.4 TB/s), 4096 x 4096 bf16 backward 28 us
// (5 TB/s), 4099 x 14336 fp16 to e4m3 with a residual 93 us (4.4 TB/s), 32776 x 128
// without one 5.8 us (2.9 TB/s), one row of 4096 2.9 us: a launch and a round trip to
// memory.
//
// Batch invariance.  The threads of a row, the vectors each of them holds and
// the order of the sum (own elements in ascending order, lanes by halving
// distances, waves in ascending order) follow from cols alone, so a row's bits
// never depend on how many rows share the call.
//
// Range.  bf16 squares reach from 2^-266 to 2^256.  A row whose fp32 sum overflows, or
// is so small that its terms lost bits to the subnormals (with an eps that does not
// cover that), sums its values times a power of two once more, from the registers.  The
// branch that no common row takes costs 0.1 us of a bf16 row's 3.1 and 0.3 us of
// 32776 x 128's 5.3; 8191 x 8192 with a residual takes 97.9 us with it and 97.7 without.
//
// Rounding.  Sums, statistics and t are fp32.  The residual stream h is rounded
// to its own type before the norm reads it: the fused call then has the bits of
// the addition followed by the norm, and the backward pass recomputes from the
// stored stream exactly what the forward pass normalised.
#include "kernel_common.h"
#include "layer_internal.h"

namespace imm {
namespace {
using namespace dev;

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

constexpr float kMinRowScale = 0x1p-120f;

// Below these a row's sum of squares is taken again.  From 2^-100 up its terms lose
// nothing that counts below fp32's least value 2^-149: 32768 of them lose at most
// 2^-135, 2^-35 of the sum, and a mean that is off by 2^-149 is 2^-49 of an eps of 2^-100.
constexpr float kLeastSum = 0x1p-100f, kLeastEps = 0x1p-100f;
constexpr float kF32Max = 3.402823466e38f;

// Eight 16-bit values of one 16-byte vector, widened.
template <int IN>
__device__ __forceinline__ void widen8(const u32x4& v, float (&f)[8]) {
  if constexpr (IN == GEMM_F16) {
    const f16x8 h = __builtin_bit_cast(f16x8, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (float)h[e];
  } else {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      f[2 * d] = __uint_as_float(v[d] << 16);
      f[2 * d + 1] = __uint_as_float(v[d] & 0xffff0000u);
    }
  }
}

// ... and eight fp32 values rounded to nearest, ties to even.
template <int IN>
__device__ __forceinline__ u32x4 narrow8(const float (&f)[8]) {
  if constexpr (IN == GEMM_F16) {
    f16x8 h;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = (_Float16)f[e];
    return __builtin_bit_cast(u32x4, h);
  } else {
    bf16x8 h;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = (__bf16)f[e];
    return __builtin_bit_cast(u32x4, h);
  }
}

// Eight fp32 values rounded to fp8 (nearest, ties to even; NaN stays NaN).
template <int OUT>
__device__ __forceinline__ u32x2 narrow8_f8(const float (&f)[8]) {
  u32x2 r;
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    int v = 0;
    if constexpr (OUT == GEMM_F8_E4M3) {
      v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * d], f[4 * d + 1], v, false);
      v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * d + 2], f[4 * d + 3], v, true);
    } else {
      v = __builtin_amdgcn_cvt_pk_bf8_f32(f[4 * d], f[4 * d + 1], v, false);
      v = __builtin_amdgcn_cvt_pk_bf8_f32(f[4 * d + 2], f[4 * d + 3], v, true);
    }
    r[d] = (unsigned)v;
  }
  return r;
}

struct AddOp {
  __device__ __forceinline__ static float f(float a, float b) { return a + b; }
};
// Maximum of |t| as bit patterns: above every number lies infinity, above it
// the NaNs, so a NaN anywhere in the row reaches the scale.
struct MaxOp {
  __device__ __forceinline__ static unsigned f(unsigned a, unsigned b) { return a > b ? a : b; }
};

// One value per row from one value per thread of the row.  TPR <= 64: lanes
// of one wave.  Above: every wave's value through LDS, joined in ascending
// wave order by every thread; `slot` is a buffer that no other reduction of
// the same row pass uses, so one barrier per reduction is enough.
template <class OP, int TPR, class V>
__device__ __forceinline__ V row_reduce(V v, V* slot) {
#pragma unroll
  for (int d = (TPR < 64 ? TPR : 64) / 2; d > 0; d >>= 1) v = OP::f(v, __shfl_xor(v, d));
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slot[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v = OP::f(v, slot[w]);
  }
  return v;
}

__device__ __forceinline__ u32x4 load16(const void* base, int64_t vec) {
  return static_cast<const u32x4*>(base)[vec];
}
__device__ __forceinline__ void store16(void* base, int64_t vec, const u32x4& v) {
  static_cast<u32x4*>(base)[vec] = v;
}

// x / by rounded in fp32, from inv = 1 / by (rounded) and low = 1 / by - inv.  q comes from
// 1 / by to 2^-46 of itself and one rounding, so it is one of the two neighbours of the
// quotient; then the remainder x - q by is an fp32 number, and q + remainder inv rounds as
// the quotient does (P. Markstein, Computation of elementary functions on the IBM RISC
// System/6000 processor, IBM J. Res. Dev. 34, 1990).  The sign is that of x, for zeros too.
// A product with inv alone puts some 3 codes in 100000 on the other side of a tie.  In us,
// that product, this and the compiler's division: 4099 x 14336 bf16 with a residual 80.7,
// 82.0 and 84.0, 4096 x 4096 quantised alone 12.65, 12.95 and 13.4, 32 x 14336 alone 3.25,
// 3.5 and 4.3.
__device__ __forceinline__ float quotient(float x, float by, float inv, float low) {
  const float q = fmaf(x, inv, x * low);
  return copysignf(fmaf(fmaf(-q, by, x), inv, q), x);
}

// TPR threads own a row, each holding VPT vectors of 8 values (vector
// t + TPR * i of the row); RPB rows share a workgroup of TPR * RPB threads.
// OUT: IN (the norm in the input's type) or an fp8 type (with scales).
// NORM = false: t = x, the plain quantisation.
template <int IN, int OUT, bool NORM, int TPR, int VPT, int RPB>
__global__ __launch_bounds__(TPR * RPB) void rms_norm_kernel(RmsNormArgs g) {
  static_assert(TPR <= 64 || RPB == 1, "rows that share a workgroup lie inside a wave");
  constexpr bool F8 = OUT == GEMM_F8_E4M3 || OUT == GEMM_F8_E5M2;
  __shared__ float sum_slot[TPR > 64 ? TPR / 64 : 1];
  __shared__ unsigned max_slot[TPR > 64 ? TPR / 64 : 1];
  __shared__ float again_slot[TPR > 64 ? TPR / 64 : 1];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  const bool live = row < g.rows;
  const int nv = (int)(g.cols / 8);  // 0: only row_scale (2^-120) and rstd (0 / 0) are written
  const int64_t base = row * nv;

  u32x4 h[VPT], w[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = t + TPR * i;
    h[i] = u32x4{};
    w[i] = u32x4{};
    if (live && v < nv) {
      h[i] = load16(g.x, base + v);
      if (NORM && g.weight) w[i] = load16(g.weight, v);
    }
  }
  if (NORM && g.residual) {
    u32x4 r[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = t + TPR * i;
      r[i] = u32x4{};
      if (live && v < nv) r[i] = load16(g.residual, base + v);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = t + TPR * i;
      float a[8], b[8];
      widen8<IN>(h[i], a);
      widen8<IN>(r[i], b);
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] += b[e];
      h[i] = narrow8<IN>(a);
      if (live && v < nv) store16(g.residual_out, base + v, h[i]);
    }
  }
  float rstd = 1.0f;
  if constexpr (NORM) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float a[8];
      widen8<IN>(h[i], a);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(a[e], a[e], ss);
    }
    ss = row_reduce<AddOp, TPR>(ss, sum_slot);
    // bf16 squares reach from 2^-266 to 2^256.  A row whose sum leaves fp32 (all of its
    // threads see it) sums h f once more, f a power of two: a function of the row alone.
    float f = 1.0f;
    if constexpr (IN == GEMM_BF16) {
      // (h under a new name: what follows widens it anew, and the 32 fp32 values of
      // before need not live through the branch)
#pragma unroll
      for (int i = 0; i < VPT; ++i) asm volatile("" : "+v"(h[i]));
      if (!(ss <= kF32Max) || (ss < kLeastSum && g.eps < kLeastEps)) {
        f = ss < 1.0f ? 0x1p100f : 0x1p-100f;
        ss = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          float a[8];
          widen8<IN>(h[i], a);
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(a[e] * f, a[e] * f, ss);
        }
        ss = row_reduce<AddOp, TPR>(ss, again_slot);
      }
    }
    const float r = 1.0f / sqrtf(ss / (float)g.cols + g.eps * f * f), kept = r * f;
    rstd = kept;
    if constexpr (IN == GEMM_BF16) {
      if (kept > kF32Max && ss > 0.0f) {
        // subnormal rows without eps: rstd is no fp32 value, h rstd is.  h times 2^32
        // (exact), rstd over it
        rstd = r * (f * 0x1p-32f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          float a[8];
          widen8<IN>(h[i], a);
#pragma unroll
          for (int e = 0; e < 8; ++e) a[e] *= 0x1p32f;
          h[i] = narrow8<IN>(a);
        }
      }
    }
    if (g.rstd && live && t == 0) g.rstd[row] = kept;
  }
  auto scaled = [&](int i, float (&a)[8]) {
    widen8<IN>(h[i], a);
    if constexpr (NORM) {
      if (g.weight) {
        float b[8];
        widen8<IN>(w[i], b);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] = a[e] * rstd * b[e];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] = a[e] * rstd;
      }
    }
  };
  if constexpr (!F8) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = t + TPR * i;
      float a[8];
      scaled(i, a);
      if (live && v < nv) store16(g.out, base + v, narrow8<IN>(a));
    }
  } else {
    constexpr float FMAX = OUT == GEMM_F8_E4M3 ? 448.0f : 57344.0f;
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      // vectors past the row hold zeros, and zero * rstd * zero may be a NaN
      // of their own: they stay out of the maximum
      if (t + TPR * i < nv) {
        float a[8];
        scaled(i, a);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = MaxOp::f(m, __float_as_uint(a[e]) & 0x7fffffffu);
      }
    }
    m = row_reduce<MaxOp, TPR>(m, max_slot);
    const float amax = __uint_as_float(m);
    // comparison that keeps a NaN
    float scale = amax / FMAX;
    scale = scale < kMinRowScale ? kMinRowScale : scale;
    // the quotients by a small scale are those of t and scale times 2^60, whose
    // remainders are no subnormals; an infinite or NaN maximum makes the whole row NaN
    // (its true values have no fp8 form)
    const float lift = scale < 0x1p-60f ? 0x1p60f : 1.0f, by = scale * lift;
    const float inv = amax <= kF32Max ? 1.0f / by : __builtin_nanf("");
    const float low = fmaf(-by, inv, 1.0f) * inv;
    if (live && t == 0) g.row_scale[row] = scale;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = t + TPR * i;
      float a[8];
      scaled(i, a);
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] = quotient(a[e] * lift, by, inv, low);
      if (live && v < nv) static_cast<u32x2*>(g.out)[base + v] = narrow8_f8<OUT>(a);
    }
  }
}

// Backward of the norm.  With n_k = h_k rstd and g_k = w_k dy_k:
//   dx_k = rstd (g_k - n_k sum_j(g_j n_j) / cols) + dh_k,
//   dw_k = sum over rows of dy_k n_k.
// dh is the gradient that reaches the residual stream by its other way; dx is
// the gradient of x and of the residual alike.  A workgroup takes the rows
// blockIdx, blockIdx + gridDim, ... and keeps its part of dw in registers (rows
// that share a workgroup add theirs in LDS at the end, in ascending order); the
// parts go to a workspace [parts, cols] and a second kernel adds them in a fixed
// order, so the result is a function of the inputs alone (no atomics).
template <int IN, int TPR, int VPT, int RPB>
__global__ __launch_bounds__(TPR * RPB) void rms_norm_backward_kernel(RmsNormBwdArgs g) {
  static_assert(TPR <= 64 || RPB == 1, "rows that share a workgroup lie inside a wave");
  // two slots, used in turn: a wave may be a row ahead of the slowest reader
  __shared__ float slot[2][TPR > 64 ? TPR / 64 : 1];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int nv = (int)(g.cols / 8);
  const float inv_cols = 1.0f / (float)g.cols;
  u32x4 w[VPT];
  float dw[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = t + TPR * i;
    w[i] = u32x4{};
    if (g.weight && v < nv) w[i] = load16(g.weight, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.0f;
  }
  int turn = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < g.rows; row0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = row0 + sub;
    const bool live = row < g.rows;
    const int64_t base = row * nv;
    u32x4 h[VPT], dy[VPT], dh[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = t + TPR * i;
      h[i] = dy[i] = dh[i] = u32x4{};
      if (live && v < nv) {
        h[i] = load16(g.h, base + v);
        dy[i] = load16(g.dy, base + v);
        if (g.dh) dh[i] = load16(g.dh, base + v);
      }
    }
    const float rstd = live ? g.rstd[row] : 0.0f;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float a[8], b[8], c[8];
      widen8<IN>(h[i], a);
      widen8<IN>(dy[i], b);
      widen8<IN>(w[i], c);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = a[e] * rstd;
        dw[i][e] = fmaf(b[e], n, dw[i][e]);
        dot = fmaf(g.weight ? b[e] * c[e] : b[e], n, dot);
      }
    }
    dot = row_reduce<AddOp, TPR>(dot, slot[turn]) * inv_cols;
    turn ^= 1;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = t + TPR * i;
      float a[8], b[8], c[8], d[8];
      widen8<IN>(h[i], a);
      widen8<IN>(dy[i], b);
      widen8<IN>(w[i], c);
      widen8<IN>(dh[i], d);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        a[e] = fmaf(rstd, (g.weight ? b[e] * c[e] : b[e]) - a[e] * rstd * dot, d[e]);
      if (live && v < nv) store16(g.dx, base + v, narrow8<IN>(a));
    }
  }
  if (g.parts) {
    f32x4* const out = reinterpret_cast<f32x4*>(g.parts + (int64_t)blockIdx.x * g.cols);
    __shared__ f32x4 mine[RPB > 1 ? RPB : 1][RPB > 1 ? 2 * TPR * VPT : 1];
    f32x4* const to = RPB > 1 ? mine[sub] : out;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = t + TPR * i;
      if (v < nv) {
        to[2 * v] = f32x4{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
        to[2 * v + 1] = f32x4{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
      }
    }
    if constexpr (RPB > 1) {
      __syncthreads();
      for (int c = threadIdx.x; c < 2 * nv; c += TPR * RPB) {
        f32x4 a = mine[0][c];
#pragma unroll
        for (int r = 1; r < RPB; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) a[e] += mine[r][c][e];
        out[c] = a;
      }
    }
  }
}

// dw = sum of the parts.  A workgroup owns 16 columns: 4 threads across (four
// columns each) and 64 down, thread row s adding the parts s, s + 64, ... in
// ascending order, eight loads at a time; then the 16 rows of a wave by halving
// distances and the waves in ascending order.  Latency bounds it, so few loads
// follow each other: with 32 columns a workgroup, 32 rows down and a load at a time
// the backward pass of 2048 x 1040 took 31 us (and left four times the parts),
// now 8.8, that of 777 x 1040 15.5, now 6.9.
template <int IN>
__global__ __launch_bounds__(256) void rms_norm_dweight_kernel(const float* parts, int64_t nparts,
                                                               int64_t cols, void* out) {
  __shared__ f32x4 sums[4][4];
  const int c = threadIdx.x % 4, s = threadIdx.x / 4;
  const int64_t c4 = (int64_t)blockIdx.x * 4 + c, n4 = cols / 4;
  const f32x4* const p = reinterpret_cast<const f32x4*>(parts) + c4;
  f32x4 a{};
  for (int64_t r0 = s; r0 < nparts; r0 += 512) {
    f32x4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int64_t r = r0 + 64 * u;
      v[u] = f32x4{};
      if (c4 < n4 && r < nparts) v[u] = p[r * n4];
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) a[e] += v[u][e];
  }
#pragma unroll
  for (int d = 32; d >= 4; d >>= 1)
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] += __shfl_xor(a[e], d);
  if (threadIdx.x % 64 < 4) sums[threadIdx.x / 64][c] = a;
  __syncthreads();
  if (threadIdx.x < 4 && c4 < n4) {
#pragma unroll
    for (int w = 1; w < 4; ++w)
#pragma unroll
      for (int e = 0; e < 4; ++e) a[e] += sums[w][c][e];
#pragma unroll
    for (int e = 0; e < 4; ++e) store_out<IN>(out, c4 * 4 + e, a[e]);
  }
}

// Calls f with the (TPR, VPT, RPB) of a row of `cols` elements.  One wave and
// no barrier up to 2048 columns (four rows a workgroup), parts of a wave for
// the short rows of a head, several waves above.  Twice the threads with half the
// vectors each: one row of 2048 to 16384 columns 2.4 to 3.7 us against 2.9 to 3.9,
// but 16384 x 2048 backward 48 us against 37, 4096 x 4096 to e4m3 23.6 against 22.4,
// and 8192 x 8192 91 against 94; half the threads: one row of 4096 3.3 us against
// 2.8, 4096 x 8192 to e4m3 44.6 against 37.5, 8192 x 4096 backward 47 against 42.
template <int TPR_, int VPT_, int RPB_>
struct RowShape {
  static constexpr int TPR = TPR_, VPT = VPT_, RPB = RPB_;
};
template <class F>
void with_row_shape(int64_t cols, F&& f) {
  const int64_t nv = cols / 8;
  if (nv <= 16) f(RowShape<16, 1, 16>{});
  else if (nv <= 32) f(RowShape<32, 1, 8>{});
  else if (nv <= 64) f(RowShape<64, 1, 4>{});
  else if (nv <= 128) f(RowShape<64, 2, 4>{});
  else if (nv <= 256) f(RowShape<64, 4, 4>{});
  else if (nv <= 512) f(RowShape<256, 2, 1>{});
  else if (nv <= 1024) f(RowShape<256, 4, 1>{});
  else if (nv <= 2048) f(RowShape<512, 4, 1>{});
  else f(RowShape<1024, 4, 1>{});
}

template <int IN, int OUT, bool NORM>
hipError_t launch_rows(const RmsNormArgs& a, hipStream_t s) {
  hipError_t e = hipSuccess;
  with_row_shape(a.cols, [&](auto shape) {
    using S = decltype(shape);
    // (a launch holds fewer than 2^32 threads)
    constexpr int64_t most = ((int64_t)1 << 31) / S::TPR;
    constexpr int out_bytes = OUT == IN ? 2 : 1;
    auto at = [&](const void* p, int64_t bytes) { return p ? static_cast<const char*>(p) + bytes : nullptr; };
    for (int64_t r = 0; r < a.rows && e == hipSuccess; r += most) {
      RmsNormArgs b = a;
      b.rows = a.rows - r < most ? a.rows - r : most;
      b.x = at(a.x, r * a.cols * 2);
      b.residual = at(a.residual, r * a.cols * 2);
      b.residual_out = const_cast<char*>(at(a.residual_out, r * a.cols * 2));
      b.out = const_cast<char*>(at(a.out, r * a.cols * out_bytes));
      b.row_scale = a.row_scale ? a.row_scale + r : nullptr;
      b.rstd = a.rstd ? a.rstd + r : nullptr;
      const dim3 grid((unsigned)((b.rows + S::RPB - 1) / S::RPB)), block(S::TPR * S::RPB);
      hipLaunchKernelGGL((rms_norm_kernel<IN, OUT, NORM, S::TPR, S::VPT, S::RPB>), grid, block, 0, s, b);
      e = hipGetLastError();
    }
  });
  return e;
}

template <int IN>
hipError_t launch_rows_in(int out, bool norm, const RmsNormArgs& a, hipStream_t s) {
  if (norm) {
    if (out == GEMM_F8_E4M3) return launch_rows<IN, GEMM_F8_E4M3, true>(a, s);
    if (out == GEMM_F8_E5M2) return launch_rows<IN, GEMM_F8_E5M2, true>(a, s);
    return launch_rows<IN, IN, true>(a, s);
  }
  if (out == GEMM_F8_E4M3) return launch_rows<IN, GEMM_F8_E4M3, false>(a, s);
  return launch_rows<IN, GEMM_F8_E5M2, false>(a, s);
}

template <int IN>
hipError_t launch_backward_in(const RmsNormBwdArgs& a, void* dweight, hipStream_t s) {
  if (a.rows > 0) {
    with_row_shape(a.cols, [&](auto shape) {
      using S = decltype(shape);
      const dim3 grid((unsigned)rms_norm_backward_groups(a.rows, a.cols)), block(S::TPR * S::RPB);
      hipLaunchKernelGGL((rms_norm_backward_kernel<IN, S::TPR, S::VPT, S::RPB>), grid, block, 0, s, a);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!dweight) return hipSuccess;  // (no rows: dw is the sum of no parts, zero)
  hipLaunchKernelGGL(rms_norm_dweight_kernel<IN>, dim3((unsigned)((a.cols + 15) / 16)), dim3(256), 0,
                     s, a.parts, rms_norm_backward_groups(a.rows, a.cols), a.cols, dweight);
  return hipGetLastError();
}

int rows_per_group(int64_t cols) {
  int r = 1;
  with_row_shape(cols, [&](auto shape) { r = decltype(shape)::RPB; });
  return r;
}

}  // namespace

int64_t rms_norm_backward_groups(int64_t rows, int64_t cols) {
  const int64_t rpb = rows_per_group(cols), all = (rows + rpb - 1) / rpb;
  return all < kRmsNormBwdGroups ? all : kRmsNormBwdGroups;
}

hipError_t launch_rms_norm(int in, int out, bool norm, const RmsNormArgs& a, hipStream_t s) {
  return in == GEMM_F16 ? launch_rows_in<GEMM_F16>(out, norm, a, s)
                        : launch_rows_in<GEMM_BF16>(out, norm, a, s);
}

hipError_t launch_rms_norm_backward(int in, const RmsNormBwdArgs& a, void* dweight, hipStream_t s) {
  return in == GEMM_F16 ? launch_backward_in<GEMM_F16>(a, dweight, s)
                        : launch_backward_in<GEMM_BF16>(a, dweight, s);
}

}  // namespace imm
