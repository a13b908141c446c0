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
// A wave takes a token: a lane makes the sine and cosine of a frequency (through LDS to the
// lanes that need them, once for all heads); then LPH lanes own a head, 8 elements each,
// four heads' loads in flight at a time, and every head is read once and written once.  Where there are
// few tokens, several waves share one.  The bytes bound it from a few thousand tokens on: 8191
// tokens of 32 + 8 heads of 128 take 39 us (4.3 TB/s; the same tensors again and again, from
// the last-level cache, 32), 4096 of 16 + 8 heads forward and backward 15 + 25 and the weights'
// sums 4, one token 3.5.  (Factors in LDS and half as many loads in flight: 39 us instead
// of 32.)
//
// A head's bits follow from its own values, its position, the weight and the
// sizes alone.  Sums and statistics are fp32, with one rounding at the end.
#include "decoder_internal.h"
#include "kernel_common.h"
#include "lanes.h"
#include "rows16.h"

namespace imm {
namespace {
using namespace dev;

constexpr float kF32Max = 3.402823466e38f;
constexpr float kLeastSum = 0x1p-100f, kLeastEps = 0x1p-100f;
constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kDeep = 4;  // vectors of a lane in flight

template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
  each_down<LPH / 2>([&](auto d) { v += lane_xor<decltype(d)::value>(v); });
  return v;
}

// A lane's factors: out_e = y_e own[e] + partner_e other[e].
struct Turn {
  float own[8], other[8];
};

// The factors of token t for the 8 elements from column c, turned by the angle (sign 1) or
// against it (-1).  `angles`: the wave's LDS.
__device__ __forceinline__ Turn make_turn(const HeadRopeArgs& g, int64_t t, int c, float sign, float2* angles) {
  const int half = g.rot / 2;
  for (int f = threadIdx.x & 63; f < half; f += 64) {
    int axis = 0;
#pragma unroll
    for (int a = 0; a < kRopeMaxAxes - 1; ++a) axis += a + 1 < g.axes && f >= g.section_end[a];
    const double pos = (double)g.positions[(int64_t)axis * g.tokens + t];
    double turns = pos * g.inv_freq[f] * 0.15915494309189533577;
    turns -= rint(turns);
    float s, k;
    sincospif(2.0f * (float)turns, &s, &k);
    angles[f] = float2{k, sign * s};
  }
  __builtin_amdgcn_wave_barrier();  // (a wave's LDS operations are in order)
  Turn r;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    r.own[e] = 1.0f;
    r.other[e] = 0.0f;
    if (c < g.rot) {
      const bool first = g.interleaved ? e % 2 == 0 : c < half;
      const float2 a = angles[g.interleaved ? (c + e) / 2 : (c < half ? c : c - half) + e];
      r.own[e] = a.x;
      r.other[e] = first ? -a.y : a.y;
    }
  }
  __builtin_amdgcn_wave_barrier();
  return r;
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

// Partner values: the neighbour's (interleaved), or those rot / 2 further on, in the
// lane rot / 16 from here.  FULL: whole heads of 8 LPH elements turn, so the partner's lane is half
// a head away and the exchange stays in the vector unit.
template <int LPH, bool FULL>
__device__ __forceinline__ void rotate(float (&y)[8], const HeadRopeArgs& g, int c, const Turn& turn) {
  float other[8];
  if (g.interleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) other[e] = y[e ^ 1];
  } else if constexpr (FULL) {
#pragma unroll
    for (int e = 0; e < 8; ++e) other[e] = lane_xor<LPH / 2>(y[e]);
  } else {
    const int lane = threadIdx.x & 63;
    const int partner = c < g.rot ? (c < g.rot / 2 ? lane + g.rot / 16 : lane - g.rot / 16) : lane;
#pragma unroll
    for (int e = 0; e < 8; ++e) other[e] = __shfl(y[e], partner);
  }
  // (elements that do not turn stay as they are, infinities and the partner's among them)
  if (c < g.rot) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = fmaf(y[e], turn.own[e], other[e] * turn.other[e]);
  }
}

template <int IN, int LPH, bool FULL, bool BACKWARD>
__global__ __launch_bounds__(kThreads) void head_rope_kernel(HeadRopeArgs g) {
  constexpr int HEADS = 64 / LPH;  // of a wave at a time
  __shared__ float2 angles[kWaves][kRopeMaxDim / 2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
  const int sub = lane / LPH, c = (lane % LPH) * 8;
  const bool in = c < g.dim;
  const int all = g.heads[0] + g.heads[1];
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
  const int64_t units = g.tokens << g.share, step = (int64_t)gridDim.x * kWaves;
  for (int64_t u = (int64_t)blockIdx.x * kWaves + wave; u < units; u += step) {
    const int64_t t = u >> g.share;
    const int part = (int)(u - (t << g.share)), stride = HEADS << g.share;
    Turn turn;
    for (int h0 = part * HEADS; h0 < all; h0 += kDeep * stride) {
      u32x4_t xv[kDeep], dv[kDeep];
      int which[kDeep];
      int64_t to[kDeep];
      bool live[kDeep];
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        int h = h0 + i * stride + sub;
        live[i] = in && h < all;
        h = h < all ? h : 0;
        which[i] = h >= g.heads[0];
        h -= which[i] ? g.heads[0] : 0;
        const int64_t at = t * (which[i] ? g.token_stride[1] : g.token_stride[0]) +
                           h * (which[i] ? g.head_stride[1] : g.head_stride[0]) + c;
        to[i] = (t * (which[i] ? g.heads[1] : g.heads[0]) + h) * g.dim + c;
        xv[i] = dv[i] = u32x4_t{};
        const void* const x = which[i] ? g.x[1] : g.x[0];
        const void* const dy = which[i] ? g.dy[1] : g.dy[0];
        if (live[i] && (!BACKWARD || norm)) xv[i] = *reinterpret_cast<const u32x4_t*>(static_cast<const char*>(x) + 2 * at);
        if (BACKWARD && live[i]) dv[i] = *reinterpret_cast<const u32x4_t*>(static_cast<const char*>(dy) + 2 * to[i]);
      }
      if (h0 == part * HEADS) turn = make_turn(g, t, c, BACKWARD ? -1.0f : 1.0f, angles[wave]);
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        if (h0 + i * stride >= all) break;
        float x[8];
        widen8<IN>(xv[i], x);
        float f = 1.0f, r = 1.0f;
        if (norm) {
          r = head_rstd<IN, LPH>(x, g.dim, g.eps, &f);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = (x[e] * f) * r;
        }
        void* const out = which[i] ? g.out[1] : g.out[0];
        if constexpr (!BACKWARD) {
          if (norm) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= which[i] ? w[1][e] : w[0][e];
          }
          rotate<LPH, FULL>(x, g, c, turn);
          if (live[i]) *reinterpret_cast<u32x4_t*>(static_cast<char*>(out) + 2 * to[i]) = narrow8<IN>(x);
        } else {
          float d[8];
          widen8<IN>(dv[i], d);
          rotate<LPH, FULL>(d, g, c, turn);
          if (norm) {
            float dot = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              // (lanes past the head's end or past the last head hold zeros: 0 r may be a NaN)
              const float dn = live[i] ? d[e] * x[e] : 0.0f;
              dw[0][e] += which[i] ? 0.0f : dn;
              dw[1][e] += which[i] ? dn : 0.0f;
              d[e] *= which[i] ? w[1][e] : w[0][e];
              dot += live[i] ? d[e] * x[e] : 0.0f;
            }
            dot = head_sum<LPH>(dot) / (float)g.dim;
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = (d[e] - x[e] * dot) * r * f;
          }
          if (live[i]) *reinterpret_cast<u32x4_t*>(static_cast<char*>(out) + 2 * to[i]) = narrow8<IN>(d);
        }
      }
    }
  }
  if constexpr (BACKWARD) {
    if (g.parts) {
      // the lanes of a column, in ascending order
      __shared__ float mine[kWaves * HEADS][2][LPH * 8];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) mine[wave * HEADS + sub][i][c + e] = dw[i][e];
      __syncthreads();
      for (int i = threadIdx.x; i < 2 * g.dim; i += kThreads) {
        const int which = i >= g.dim, d = i - which * g.dim;
        float s = mine[0][which][d];
        for (int k = 1; k < kWaves * HEADS; ++k) s += mine[k][which][d];
        g.parts[(int64_t)blockIdx.x * 2 * g.dim + i] = s;
      }
    }
  }
}

// The weights' gradients: the sum of the parts.  A workgroup owns 16 columns,
// 64 threads down each; a thread adds every 64th part in ascending order, 8 loads at a time,
// and the 64 sums are added in ascending order.
constexpr int kDown = 64;
template <int IN>
__global__ __launch_bounds__(16 * kDown) void head_rope_dweight_kernel(const float* parts, int groups,
                                                                       int dim, void* dq, void* dk) {
  __shared__ float sums[kDown][16];
  const int c = threadIdx.x % 16, s = threadIdx.x / 16;
  const int col = blockIdx.x * 16 + c;
  float a = 0.0f;
  if (col < 2 * dim) {
    for (int r0 = s; r0 < groups; r0 += 8 * kDown) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = r0 + i * kDown < groups ? parts[(int64_t)(r0 + i * kDown) * 2 * dim + col] : 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) a += v[i];
    }
  }
  sums[s][c] = a;
  __syncthreads();
  if (s == 0 && col < 2 * dim) {
    for (int k = 1; k < kDown; ++k) a += sums[k][c];
    void* const to = col < dim ? dq : dk;
    if (to) store_out<IN>(to, col < dim ? col : col - dim, a);
  }
}

int lanes_per_head(int dim) { return dim <= 64 ? 8 : dim <= 128 ? 16 : dim <= 256 ? 32 : 64; }
// Waves that share a token, as a power of two: one, or as many as make 2048 waves of few tokens
// while each still has heads.
int share_of(int64_t tokens, int heads, int dim) {
  const int rounds = (heads * lanes_per_head(dim) + 63) / 64;
  int share = 0;
  while ((tokens << share) < 2048 && (1 << share) < rounds) ++share;
  return share;
}

template <bool BACKWARD>
hipError_t launch(int in, const HeadRopeArgs& a, unsigned grid, hipStream_t s) {
  auto go = [&](auto dt, auto lanes) {
    constexpr int IN = decltype(dt)::value, LPH = decltype(lanes)::value;
    const auto kernel = a.rot == 8 * LPH ? head_rope_kernel<IN, LPH, true, BACKWARD> : head_rope_kernel<IN, LPH, false, BACKWARD>;
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(kThreads), 0, s, a);
  };
  auto by_dim = [&](auto dt) {
    switch (lanes_per_head(a.dim)) {
      case 8: return go(dt, std::integral_constant<int, 8>{});
      case 16: return go(dt, std::integral_constant<int, 16>{});
      case 32: return go(dt, std::integral_constant<int, 32>{});
      default: return go(dt, std::integral_constant<int, 64>{});
    }
  };
  if (in == GEMM_F16) by_dim(std::integral_constant<int, GEMM_F16>{});
  else by_dim(std::integral_constant<int, GEMM_BF16>{});
  return hipGetLastError();
}

// Workgroups of all tokens.
int64_t groups_of(int64_t tokens, int heads, int dim) {
  return ((tokens << share_of(tokens, heads, dim)) + kWaves - 1) / kWaves;
}

}  // namespace

int64_t head_rope_groups(int64_t tokens, int heads, int dim) {
  const int64_t all = groups_of(tokens, heads, dim);
  return all < kRopeBwdGroups ? all : kRopeBwdGroups;
}

hipError_t launch_head_rope(int in, HeadRopeArgs a, hipStream_t s) {
  const int heads = a.heads[0] + a.heads[1];
  a.share = share_of(a.tokens, heads, a.dim);
  // (a launch of fewer than 2^32 threads; the kernel walks on in its steps)
  int64_t grid = groups_of(a.tokens, heads, a.dim);
  if (grid > 1 << 20) grid = 1 << 20;
  return launch<false>(in, a, (unsigned)grid, s);
}

hipError_t launch_head_rope_backward(int in, HeadRopeArgs a, void* const* dweight, hipStream_t s) {
  const int heads = a.heads[0] + a.heads[1];
  a.share = share_of(a.tokens, heads, a.dim);
  int64_t groups = head_rope_groups(a.tokens, heads, a.dim);
  if (!a.parts) groups = groups_of(a.tokens, heads, a.dim);  // nothing of a workgroup's own is kept
  if (groups > 1 << 20) groups = 1 << 20;
  if (a.tokens > 0 && heads > 0) {
    const hipError_t e = launch<true>(in, a, (unsigned)groups, s);
    if (e != hipSuccess) return e;
  }
  if (!dweight[0] && !dweight[1]) return hipSuccess;
  const int n = a.tokens > 0 && heads > 0 ? (int)groups : 0;  // (no heads: no parts, zero)
  const dim3 grid((unsigned)((2 * a.dim + 15) / 16)), block(16 * kDown);
  if (in == GEMM_F16)
    hipLaunchKernelGGL(head_rope_dweight_kernel<GEMM_F16>, grid, block, 0, s, a.parts, n, a.dim,
                       dweight[0], dweight[1]);
  else
    hipLaunchKernelGGL(head_rope_dweight_kernel<GEMM_BF16>, grid, block, 0, s, a.parts, n, a.dim,
                       dweight[0], dweight[1]);
  return hipGetLastError();
}

}  // namespace imm
