// The norm of every query and key head with the rotation of its position, and
// the backward pass.
//
//   n = x / sqrt(mean_d x_d^2 + eps), y_d = n_d w_d      (y = x without the norm)
//   angle_i = position[axis(i)] inv_freq_i, i < rot / 2, in fp64
//   (z_a, z_b) = (y_a cos - y_b sin, y_b cos + y_a sin) for the pairs
//     (a, b) = (i, i + rot / 2), or (2 i, 2 i + 1) interleaved
//   z_d = y_d for d >= rot, out = round(z)
//
// The angle of a far position needs more than fp32: at position 10^6 its
// rounding alone would be 0.06 of a radian.  Here the turns position inv_freq / (2 pi) are fp64, lose their
// whole part there, and the fraction (below 1/2 in magnitude) goes to fp32: an
// angle is off by 2^-24 of itself.
//
// A workgroup takes a few tokens: it makes their sines and cosines once, in
// LDS, for all heads; then LPH lanes own a head, 8 elements each, and the head
// is read once and written once.  The bytes bound it.
//
// A head's bits follow from its own values, its position, the weight and the
// sizes alone.  Sums and statistics are fp32, with one rounding at the end.
#include "decoder_internal.h"
#include "kernel_common.h"
#include "rows16.h"

namespace imm {
namespace {
using namespace dev;

constexpr float kF32Max = 3.402823466e38f;
constexpr float kLeastSum = 0x1p-100f, kLeastEps = 0x1p-100f;
constexpr int kThreads = 256;
constexpr int kMaxAngles = 1024;  // of a workgroup's tokens

template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int d = LPH / 2; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// cos and sin of every token of the workgroup, [token][rot / 2].
__device__ __forceinline__ void make_angles(const HeadRopeArgs& g, int64_t t0, int nt,
                                            float2* angles) {
  const int half = g.rot / 2;
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int t = i / half, f = i - t * half;
    int axis = 0;
#pragma unroll
    for (int a = 0; a < kRopeMaxAxes - 1; ++a) axis += a + 1 < g.axes && f >= g.section_end[a];
    const double pos = (double)g.positions[(int64_t)axis * g.tokens + t0 + t];
    double turns = pos * g.inv_freq[f] * 0.15915494309189533577;
    turns -= rint(turns);
    float s, c;
    sincospif(2.0f * (float)turns, &s, &c);
    angles[i] = float2{c, s};
  }
}

// 1 / rms of a head from its 8 elements in each of LPH lanes: n = (x f) r, f a
// power of two that is 1 unless the fp32 sum of squares left fp32's range (bf16 squares
// reach from 2^-266 to 2^256; a function of the head alone).
template <int IN, int LPH>
__device__ __forceinline__ float head_rstd(const float (&x)[8], int dim, float eps, float* f) {
  float ss = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
  ss = head_sum<LPH>(ss);
  *f = 1.0f;
  if constexpr (IN == GEMM_BF16) {
    if (!(ss <= kF32Max) || (ss < kLeastSum && eps < kLeastEps)) {
      *f = ss < 1.0f ? 0x1p100f : 0x1p-100f;
      ss = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e] * *f, x[e] * *f, ss);
      ss = head_sum<LPH>(ss);
    }
  }
  return 1.0f / sqrtf(ss / (float)dim + eps * *f * *f);
}

// The rotation of the 8 elements from column c of a head, by the angle (sign 1)
// or against it (-1).  Partner values of the split form come from the lane
// rot / 16 further on.
__device__ __forceinline__ void rotate(float (&y)[8], int c, int rot, bool interleaved, float sign,
                                       const float2* angles) {
  if (interleaved) {
    if (c < rot) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 cs = angles[(c + e) / 2];
        const float sn = sign * cs.y, a = y[e], b = y[e + 1];
        y[e] = fmaf(a, cs.x, -(b * sn));
        y[e + 1] = fmaf(b, cs.x, a * sn);
      }
    }
    return;
  }
  const int half = rot / 2;
  const bool low = c < half;
  const int lane = threadIdx.x & 63;
  const int partner = c < rot ? (low ? lane + rot / 16 : lane - rot / 16) : lane;
  float other[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) other[e] = __shfl(y[e], partner);
  if (c < rot) {
    const float2* const a = angles + (low ? c : c - half);
    const float to = low ? -sign : sign;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = fmaf(y[e], a[e].x, other[e] * (to * a[e].y));
  }
}

template <int IN, int LPH, bool BACKWARD>
__global__ __launch_bounds__(kThreads) void head_rope_kernel(HeadRopeArgs g) {
  constexpr int HEADS = kThreads / LPH;  // at a time
  __shared__ float2 angles[kMaxAngles];
  const int sub = threadIdx.x / LPH, c = (threadIdx.x % LPH) * 8;
  const bool in = c < g.dim;
  const int all = g.heads[0] + g.heads[1], half = g.rot / 2;
  const bool norm = g.norm;
  float w[2][8], dw[2][8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    u32x4_t v{};
    if (norm && g.weight[i] && in) v = *reinterpret_cast<const u32x4_t*>(static_cast<const char*>(g.weight[i]) + 2 * c);
    widen8<IN>(v, w[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (!g.weight[i]) w[i][e] = 1.0f;
      dw[i][e] = 0.0f;
    }
  }
  const int64_t step = (int64_t)gridDim.x * g.tokens_per_group;
  for (int64_t t0 = (int64_t)blockIdx.x * g.tokens_per_group; t0 < g.tokens; t0 += step) {
    const int nt = (int)(g.tokens - t0 < g.tokens_per_group ? g.tokens - t0 : g.tokens_per_group);
    __syncthreads();  // the last round's angles have been read
    make_angles(g, t0, nt, angles);
    __syncthreads();
    for (int i0 = 0; i0 < nt * all; i0 += HEADS) {
      const int item = i0 + sub;
      const bool live = item < nt * all && in;
      const int t = item < nt * all ? item / all : 0;
      int h = item < nt * all ? item - t * all : 0;
      const int which = h >= g.heads[0];
      h -= which ? g.heads[0] : 0;
      const int64_t at = (t0 + t) * g.token_stride[which] + h * g.head_stride[which] + c;
      const int64_t to = ((t0 + t) * g.heads[which] + h) * g.dim + c;
      u32x4_t xv{}, dv{};
      if (live && (!BACKWARD || norm)) xv = *reinterpret_cast<const u32x4_t*>(static_cast<const char*>(g.x[which]) + 2 * at);
      if (BACKWARD && live) dv = *reinterpret_cast<const u32x4_t*>(static_cast<const char*>(g.dy[which]) + 2 * to);
      float x[8];
      widen8<IN>(xv, x);
      float f = 1.0f, r = 1.0f;
      if (norm) {
        r = head_rstd<IN, LPH>(x, g.dim, g.eps, &f);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (x[e] * f) * r;
      }
      const float2* const a = angles + t * half;
      if constexpr (!BACKWARD) {
        if (norm) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= which ? w[1][e] : w[0][e];
        }
        rotate(x, c, g.rot, g.interleaved, 1.0f, a);
        if (live) *reinterpret_cast<u32x4_t*>(static_cast<char*>(g.out[which]) + 2 * to) = narrow8<IN>(x);
      } else {
        float d[8];
        widen8<IN>(dv, d);
        rotate(d, c, g.rot, g.interleaved, -1.0f, a);
        if (norm) {
          float dot = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            // (lanes past the head's end or past the last head hold zeros: 0 r may be a NaN)
            const float dn = live ? d[e] * x[e] : 0.0f;
            dw[0][e] += which ? 0.0f : dn;
            dw[1][e] += which ? dn : 0.0f;
            d[e] *= which ? w[1][e] : w[0][e];
            dot += live ? d[e] * x[e] : 0.0f;
          }
          dot = head_sum<LPH>(dot) / (float)g.dim;
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] = (d[e] - x[e] * dot) * r * f;
        }
        if (live) *reinterpret_cast<u32x4_t*>(static_cast<char*>(g.out[which]) + 2 * to) = narrow8<IN>(d);
      }
    }
  }
  if constexpr (BACKWARD) {
    if (g.parts) {
      // the HEADS lanes of a column, in ascending order
      __shared__ float mine[HEADS][2][LPH * 8];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) mine[sub][i][c + e] = dw[i][e];
      __syncthreads();
      for (int i = threadIdx.x; i < 2 * g.dim; i += kThreads) {
        const int which = i >= g.dim, d = i - which * g.dim;
        float s = mine[0][which][d];
        for (int k = 1; k < HEADS; ++k) s += mine[k][which][d];
        g.parts[(int64_t)blockIdx.x * 2 * g.dim + i] = s;
      }
    }
  }
}

// The weights' gradients: the sum of the parts.  A workgroup owns 16 columns,
// 16 threads down each; a thread adds every 16th part in ascending order, and the
// 16 sums are added in ascending order.
template <int IN>
__global__ __launch_bounds__(kThreads) void head_rope_dweight_kernel(const float* parts, int groups,
                                                                     int dim, void* dq, void* dk) {
  __shared__ float sums[16][16];
  const int c = threadIdx.x % 16, s = threadIdx.x / 16;
  const int col = blockIdx.x * 16 + c;
  float a = 0.0f;
  if (col < 2 * dim) {
    for (int r = s; r < groups; r += 16) a += parts[(int64_t)r * 2 * dim + col];
  }
  sums[s][c] = a;
  __syncthreads();
  if (s == 0 && col < 2 * dim) {
    for (int k = 1; k < 16; ++k) a += sums[k][c];
    void* const to = col < dim ? dq : dk;
    if (to) store_out<IN>(to, col < dim ? col : col - dim, a);
  }
}

// Tokens of a workgroup: about 8 rounds of heads, so that the angles' time is
// hidden by other workgroups' rounds, and never more angles than LDS holds.
int tokens_per_group(int64_t tokens, int heads, int dim, int rot) {
  const int lph = dim <= 64 ? 8 : dim <= 128 ? 16 : dim <= 256 ? 32 : 64;
  const int at_a_time = kThreads / lph;
  int n = heads > 0 ? 8 * at_a_time / heads : 1;
  if (rot > 0 && n > kMaxAngles / (rot / 2)) n = kMaxAngles / (rot / 2);
  if (n > (tokens + 1023) / 1024) n = (int)((tokens + 1023) / 1024);
  return n < 1 ? 1 : n;
}

template <bool BACKWARD>
hipError_t launch(int in, const HeadRopeArgs& a, unsigned grid, hipStream_t s) {
  auto go = [&](auto dt, auto lanes) {
    hipLaunchKernelGGL((head_rope_kernel<decltype(dt)::value, decltype(lanes)::value, BACKWARD>),
                       dim3(grid), dim3(kThreads), 0, s, a);
  };
  auto by_dim = [&](auto dt) {
    if (a.dim <= 64) go(dt, std::integral_constant<int, 8>{});
    else if (a.dim <= 128) go(dt, std::integral_constant<int, 16>{});
    else if (a.dim <= 256) go(dt, std::integral_constant<int, 32>{});
    else go(dt, std::integral_constant<int, 64>{});
  };
  if (in == GEMM_F16) by_dim(std::integral_constant<int, GEMM_F16>{});
  else by_dim(std::integral_constant<int, GEMM_BF16>{});
  return hipGetLastError();
}

}  // namespace

int64_t head_rope_groups(int64_t tokens, int heads, int dim) {
  const int64_t per = tokens_per_group(tokens, heads, dim, dim), all = (tokens + per - 1) / per;
  return all < kRopeBwdGroups ? all : kRopeBwdGroups;
}

hipError_t launch_head_rope(int in, HeadRopeArgs a, hipStream_t s) {
  a.tokens_per_group = tokens_per_group(a.tokens, a.heads[0] + a.heads[1], a.dim, a.rot);
  // (a grid of fewer than 2^24 workgroups; the kernel walks on in its steps)
  int64_t grid = (a.tokens + a.tokens_per_group - 1) / a.tokens_per_group;
  if (grid > 1 << 20) grid = 1 << 20;
  return launch<false>(in, a, (unsigned)grid, s);
}

hipError_t launch_head_rope_backward(int in, HeadRopeArgs a, void* const* dweight, hipStream_t s) {
  const int heads = a.heads[0] + a.heads[1];
  a.tokens_per_group = tokens_per_group(a.tokens, heads, a.dim, a.dim);
  const int64_t groups = head_rope_groups(a.tokens, heads, a.dim);
  if (a.tokens > 0 && heads > 0) {
    const hipError_t e = launch<true>(in, a, (unsigned)groups, s);
    if (e != hipSuccess) return e;
  }
  if (!dweight[0] && !dweight[1]) return hipSuccess;
  const int n = a.tokens > 0 && heads > 0 ? (int)groups : 0;  // (no heads: no parts, zero)
  const dim3 grid((unsigned)((2 * a.dim + 15) / 16));
  if (in == GEMM_F16)
    hipLaunchKernelGGL(head_rope_dweight_kernel<GEMM_F16>, grid, dim3(kThreads), 0, s, a.parts, n,
                       a.dim, dweight[0], dweight[1]);
  else
    hipLaunchKernelGGL(head_rope_dweight_kernel<GEMM_BF16>, grid, dim3(kThreads), 0, s, a.parts, n,
                       a.dim, dweight[0], dweight[1]);
  return hipGetLastError();
}

}  // namespace imm
