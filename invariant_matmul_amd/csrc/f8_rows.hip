// Few fp8 rows with row and column scales (gfx950): the product of decoding and
// small batches, C = ((A B^T) row_scale) col_scale + bias with A [M, K], B [N, K].
//
// The bits are those of the tile kernels: every output is one chain of
// 16x16x128 steps in ascending K from +0, with zeros past the end of K in the
// last step.  The chain is no bound here (a step every 40 cycles: 2 us at
// K = 14336); the time is the stream of the weights, which one chain per output
// leaves to few workgroups (N / 16 columns' chains on 256 compute units), so each
// has to keep many bytes in flight.  A workgroup owns 16 CB columns and 16 RB rows.
// Four waves do nothing but move the columns' weights to a ring of NS LDS stages of
// 1024 K each, a whole kilobyte of a row per transfer; RB waves multiply, one
// block of 16 rows each, with their rows' next stage on its way to registers.
// One barrier a stage: it publishes stage t (each moving wave has waited for
// its own transfers) and frees the slot of stage t - 1.
//
// 16-byte chunk c of column n's kilobyte lies at slot c ^ (n & 15), the low four
// bits: the 16 columns that a quarter of a wave reads at one chunk fall on
// different banks.
#include "buffer_access.h"
#include "kernel_common.h"
#include "layer_internal.h"

namespace imm {
namespace {
using namespace dev;

constexpr int kStageK = 1024, kMovers = 4;

template <int IN, int OUT, int RB, int CB, int NS>
__global__ __launch_bounds__((kMovers + RB) * 64) void f8_rows_kernel(ScaledArgs g) {
  constexpr int STAGE = 16 * CB * kStageK, T = 16 * CB / kMovers;
  static_assert(NS * STAGE <= 160 * 1024 && NS >= 2 && (NS - 2) * T < 64, "ring");
  __shared__ __attribute__((aligned(1024))) char ring[NS * STAGE];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * (16 * CB), m0 = (int64_t)blockIdx.y * (16 * RB);
  const int K = (int)g.K, nt = (K + kStageK - 1) / kStageK;

  if (w >= RB) {
    // ---- the moving waves: rows p, p + 4, ... of the columns' weights
    const int p = w - RB;
    const auto buf = buffer_at(static_cast<const char*>(g.B) + n0 * K, kMaxOffset * 2);
    unsigned chunk[T];
#pragma unroll
    for (int i = 0; i < T; ++i) {
      const int r = p + kMovers * i;
      chunk[i] = n0 + r < g.N ? (unsigned)((lane & 48) | ((lane ^ r) & 15)) * 16 : OOB;
    }
    auto move = [&](int t) {
      char* const slot = ring + t % NS * STAGE;
      const bool partial = (t + 1) * kStageK > K;
#pragma unroll
      for (int i = 0; i < T; ++i) {
        const int r = p + kMovers * i;
        const unsigned off = partial && chunk[i] + t * kStageK >= (unsigned)K ? OOB : chunk[i];
        dma16(buf, slot + r * kStageK, off, r * K + t * kStageK);
      }
    };
    // all transfers but those of the last n stages have landed
    auto wait = [&](int n) {
      __builtin_amdgcn_sched_barrier(0);
      if (n >= NS - 2) __builtin_amdgcn_s_waitcnt(vmcnt_imm((NS - 2) * T));
#define IMM_LATER(k) else if (NS - 2 > k && n == k) __builtin_amdgcn_s_waitcnt(vmcnt_imm(k * T));
      IMM_LATER(6) IMM_LATER(5) IMM_LATER(4) IMM_LATER(3) IMM_LATER(2) IMM_LATER(1)
#undef IMM_LATER
      else __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
      __builtin_amdgcn_sched_barrier(0);
    };
    for (int t = 0; t < NS - 1 && t < nt; ++t) move(t);
    for (int t = 0; t < nt; ++t) {
      wait(nt - 1 - t);
      __builtin_amdgcn_s_barrier();
      if (t + NS - 1 < nt) move(t + NS - 1);
    }
    return;
  }

  // ---- the multiplying waves
  const int lr = lane % 16, hq = lane / 16;
  const int64_t row0 = m0 + 16 * w;
  const auto xbuf = buffer_at(static_cast<const char*>(g.A) + row0 * K, kMaxOffset * 2);
  const unsigned x_off = row0 + lr < g.M ? (unsigned)(lr * K + 32 * hq) : OOB;
  i32x8 x[2][8];
  auto load_x = [&](int t, i32x8 (&v)[8]) {
    const bool partial = (t + 1) * kStageK > K;
#pragma unroll
    for (int s = 0; s < 8; ++s)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int k = t * kStageK + s * 128 + e * 16;
        const unsigned off = partial && k + 32 * hq >= K ? OOB : x_off + k;
        const i32x4 q = __builtin_bit_cast(i32x4, load_b128(xbuf, off));
#pragma unroll
        for (int d = 0; d < 4; ++d) v[s][4 * e + d] = q[d];
      }
  };
  // chunk 8 s + 2 hq + e of column lr: four places, 256 bytes apart for every two steps
  int at[2][2];
#pragma unroll
  for (int o = 0; o < 2; ++o)
#pragma unroll
    for (int e = 0; e < 2; ++e) at[o][e] = lr * kStageK + (((8 * o + 2 * hq + e) ^ lr) & 15) * 16;
  f32x4 acc[CB];
#pragma unroll
  for (int j = 0; j < CB; ++j) acc[j] = f32x4{};
  auto stage = [&](auto BUF, int t) {
    constexpr int b = decltype(BUF)::value;
    if (t + 1 < nt) load_x(t + 1, x[1 - b]);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    const char* const slot = ring + t % NS * STAGE;
    auto steps = [&](int n) {
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        if (s >= n) break;
#pragma unroll
        for (int j = 0; j < CB; ++j) {
          i32x8 v;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const i32x4 q = *reinterpret_cast<const i32x4*>(slot + j * 16 * kStageK + at[s & 1][e] + s / 2 * 256);
#pragma unroll
            for (int d = 0; d < 4; ++d) v[4 * e + d] = q[d];
          }
          acc[j] = mfma16_f8<IN>(x[b][s], v, acc[j]);
        }
      }
    };
    const int left = K - t * kStageK;
    if (left >= kStageK)
      steps(8);
    else
      steps((left + 127) / 128);
  };
  if (nt > 0) load_x(0, x[0]);
  for (int t = 0; t < nt;) {
    stage(std::integral_constant<int, 0>{}, t++);
    if (t >= nt) break;
    stage(std::integral_constant<int, 1>{}, t++);
  }
#pragma unroll
  for (int j = 0; j < CB; ++j) {
    const int64_t col = n0 + 16 * j + lr;
    if (col >= g.N) continue;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma clang fp contract(off)
      const int64_t row = row0 + 4 * hq + r;
      if (row >= g.M) continue;
      const float v = acc[j][r];
      float s = g.scale == 1.0f ? v : v * g.scale;
      s = (s * g.row_scale[row]) * g.col_scale[col];
      store_final<OUT>(g.C, row * g.N + col, s, 1.0f, g.bias, col);
    }
  }
}

template <int IN, int OUT>
hipError_t launch_out(const ScaledArgs& a, hipStream_t s) {
  auto launch = [&](auto RB, auto CB, auto NS) {
    constexpr int rb = decltype(RB)::value, cb = decltype(CB)::value, ns = decltype(NS)::value;
    const dim3 grid((unsigned)((a.N + 16 * cb - 1) / (16 * cb)), (unsigned)((a.M + 16 * rb - 1) / (16 * rb)));
    hipLaunchKernelGGL((f8_rows_kernel<IN, OUT, rb, cb, ns>), grid, dim3((kMovers + rb) * 64), 0, s, a);
    return hipGetLastError();
  };
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I4 = std::integral_constant<int, 4>;
  if (a.M <= 16) return launch(I1{}, I1{}, I4{});
  if (a.M <= 32) return launch(I2{}, I1{}, I4{});
  return launch(I4{}, I1{}, I4{});
}

template <int IN>
hipError_t launch_in(int out, const ScaledArgs& a, hipStream_t s) {
  if (out == GEMM_F32) return launch_out<IN, GEMM_F32>(a, s);
  if (out == GEMM_F16) return launch_out<IN, GEMM_F16>(a, s);
  return launch_out<IN, GEMM_BF16>(a, s);
}

}  // namespace

bool f8_rows_take(int64_t M, int64_t N, int64_t K) {
  return M <= 64 && 64 * K < kMaxOffset;
}

hipError_t launch_f8_rows(int in, int out, const ScaledArgs& a, hipStream_t s) {
  return in == GEMM_F8_E4M3 ? launch_in<GEMM_F8_E4M3>(out, a, s) : launch_in<GEMM_F8_E5M2>(out, a, s);
}

}  // namespace imm
