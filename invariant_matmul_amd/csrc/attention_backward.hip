// The gradients of attention.  With p_ij = e^(scale q_i k_j - lse_i) and
// delta_i = sum_d do_id o_id:
//   dv_j = sum_i p_ij do_i
//   ds_ij = p_ij (do_i v_j - delta_i)
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i
//
// Three kernels: delta; dk and dv, a workgroup per 128 keys of a key head, which walks
// through the rows that see them; dq, a workgroup per 128 rows, which walks through
// their keys.  p and ds are made twice, so that every sum is one chain in one workgroup:
// no atomics, and the gradients of a sequence depend on that sequence alone.
// p and ds are rounded to the input's type for their products, all else is fp32.
#include "attention_common.h"
#include "rows16.h"

namespace imm {
namespace {
using namespace dev;

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kKeys = 32 * kWaves;   // keys of a workgroup (dk, dv)
constexpr int kRows = 32 * kWaves;   // rows of a workgroup (dq)
constexpr float kLog2e = 1.44269504088896340736f;

// delta: 16 lanes a row, 8 elements each.  With o alone, the rounding of o is as large a part of
// the gradients' error as the rounding of ds; with what it left (o_low) that is gone
// (1500 bf16 keys of 128: dq is off by 0.00245 of itself instead of 0.00305, where its own
// rounding makes 0.00166).
template <int IN>
__global__ __launch_bounds__(256) void attention_delta_kernel(AttnArgs a) {
  const int64_t at = (int64_t)blockIdx.x * 16 + threadIdx.x / 16;
  const int c = threadIdx.x % 16 * 8;
  const bool in = at < a.q_rows * a.q_heads && c < a.dim;
  float sum = 0.0f;
  if (in) {
    float o[8], g[8];
    widen8<IN>(*reinterpret_cast<const u32x4_t*>(static_cast<const char*>(a.o) + 2 * (at * a.dim + c)), o);
    widen8<IN>(*reinterpret_cast<const u32x4_t*>(static_cast<const char*>(a.d_o) + 2 * (at * a.dim + c)), g);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(o[e], g[e], sum);
    if (a.o_low) {
      widen8<IN>(*reinterpret_cast<const u32x4_t*>(static_cast<const char*>(a.o_low) + 2 * (at * a.dim + c)), o);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(o[e], g[e], sum);
    }
  }
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if (c == 0 && at < a.q_rows * a.q_heads) a.delta[at] = sum;
}

// A row set as the second operand: rows (lane % 16), dimensions 32 ks + 8 quad.
template <int DP>
__device__ __forceinline__ void row_operand(i32x4 (&f)[TileOf<DP>::KS], const char* row, bool ok, int dim) {
#pragma unroll
  for (int ks = 0; ks < TileOf<DP>::KS; ++ks) {
    const int d = 32 * ks + 8 * ((threadIdx.x & 63) / 16);
    f[ks] = i32x4{};
    if (ok && d < dim) f[ks] = *reinterpret_cast<const i32x4*>(row + 2 * d);
  }
}

// Segment i of the keys: as for the queries, with the rows before and behind the sequences.
__device__ __forceinline__ int64_t key_start(const AttnArgs& a, int i) {
  return i <= 0 ? 0 : i > a.batch + 1 ? a.k_rows : k_start(a, i - 1);
}

template <int IN, int DP>
__global__ __launch_bounds__(kThreads, 1) void attention_dkv_kernel(AttnArgs a) {
  using T = TileOf<DP>;
  __shared__ __attribute__((aligned(16))) char lds[2][2][kTile * T::PITCH];
  __shared__ __attribute__((aligned(16))) float stat[2][2][kTile];
  __shared__ __attribute__((aligned(16))) int sees[2][kTile];
  const int lane = threadIdx.x & 63, wave = threadIdx.x / 64, quad = lane / 16, col = lane % 16;
  const int kh = blockIdx.x % a.k_heads;
  const int64_t tile = blockIdx.x / a.k_heads;  // the first keys (the most rows) first
  int lo = 0, hi = a.batch + 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (key_start(a, mid) / kKeys + mid <= tile) lo = mid;
    else hi = mid - 1;
  }
  const int64_t k_first = key_start(a, lo);
  const int64_t k_end = lo == a.batch + 1 ? a.k_rows : key_start(a, lo + 1);
  const int64_t c0 = (tile - (k_first / kKeys + lo)) * kKeys;  // of the segment
  if (c0 >= k_end - k_first) return;
  const Sequence s = segment(a, lo);
  const int64_t rows = s.n * a.group;
  const int64_t w0 = c0 + 32 * wave;

  i32x4 kf[2][T::KS], vf[2][T::KS];
  f32x4 dk[2][T::DB], dv[2][T::DB];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t key = w0 + 16 * j + col;
    const bool ok = key < s.m;
    row_operand<DP>(kf[j], static_cast<const char*>(a.k) + 2 * ((k_first + key) * a.k_token + kh * a.k_head), ok, a.dim);
    row_operand<DP>(vf[j], static_cast<const char*>(a.v) + 2 * ((k_first + key) * a.v_token + kh * a.v_head), ok, a.dim);
#pragma unroll
    for (int d = 0; d < T::DB; ++d) dk[j][d] = dv[j][d] = f32x4{};
  }
  // the first query that sees a key
  auto first_row = [&](int64_t key) {
    if (key >= s.m) return rows;
    return a.causal ? clamp64(key - (s.m - s.n), 0, s.n) * a.group : (int64_t)0;
  };
  const int64_t from = first_row(c0) / kTile * kTile;
  const int64_t wave_from = first_row(w0);

  constexpr int N = kTile * T::SLOTS / kThreads;
  u32x4 nq[N], ng[N];
  float n_lse = 0.0f, n_delta = 0.0f;
  int n_seen = 0;
  auto fetch = [&](int64_t r0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = threadIdx.x + i * kThreads, r = at / T::SLOTS, c = at % T::SLOTS;
      const int64_t row = r0 + r, t = row / a.group;
      const int64_t h = kh * a.group + (row - t * a.group);
      nq[i] = ng[i] = u32x4{};
      if (row < rows && c * 8 < a.dim) {
        nq[i] = *reinterpret_cast<const u32x4*>(static_cast<const char*>(a.q) + 2 * ((s.q0 + t) * a.q_token + h * a.q_head) + 16 * c);
        ng[i] = *reinterpret_cast<const u32x4*>(static_cast<const char*>(a.d_o) + 2 * ((s.q0 + t) * a.q_heads + h) * a.dim + 16 * c);
      }
    }
    if (threadIdx.x < kTile) {
      const int64_t row = r0 + threadIdx.x, t = row / a.group;
      n_seen = 0;
      n_lse = n_delta = 0.0f;
      if (row < rows) {
        const int64_t at = (s.q0 + t) * a.q_heads + kh * a.group + (row - t * a.group);
        n_seen = (int)keys_seen(a, s, t);
        n_lse = a.lse[at] * kLog2e;
        n_delta = a.delta[at];
      }
    }
  };
  auto put = [&](int stage) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = threadIdx.x + i * kThreads, r = at / T::SLOTS, c = at % T::SLOTS;
      *reinterpret_cast<u32x4*>(lds[stage][0] + T::at(r, c)) = nq[i];
      *reinterpret_cast<u32x4*>(lds[stage][1] + T::at(r, c)) = ng[i];
    }
    if (threadIdx.x < kTile) {
      stat[stage][0][threadIdx.x] = n_lse;
      stat[stage][1][threadIdx.x] = n_delta;
      sees[stage][threadIdx.x] = n_seen;
    }
  };
  if (from < rows) {
    fetch(from);
    put(0);
  }
  __syncthreads();
  Lanes<DP> lanes;
  int stage = 0;
  for (int64_t r0 = from; r0 < rows; r0 += kTile) {
    const bool more = r0 + kTile < rows;
    if (more) fetch(r0 + kTile);
    const char* const qt = lds[stage][0];
    const char* const gt = lds[stage][1];
    if (r0 + kTile > wave_from && w0 < s.m) {
      // all rows of the step see all of the wave's keys
      const bool all = r0 + kTile <= rows && w0 + 32 <= sees[stage][0];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        f32x4 sc[2][2], dp[2][2];  // [block of rows][block of keys]
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          sc[b][0] = sc[b][1] = dp[b][0] = dp[b][1] = f32x4{};
#pragma unroll
          for (int ks = 0; ks < T::KS; ++ks) {
            const i32x4 qf = row_fragment<DP>(qt, lanes, 2 * half + b, ks);
            const i32x4 gf = row_fragment<DP>(gt, lanes, 2 * half + b, ks);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              sc[b][j] = mfma16_v<IN>(qf, kf[j][ks], sc[b][j]);
              dp[b][j] = mfma16_v<IN>(gf, vf[j][ks], dp[b][j]);
            }
          }
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int at = 32 * half + 16 * b + 4 * quad;
          const f32x4 lse = *reinterpret_cast<const f32x4*>(&stat[stage][0][at]);
          const f32x4 delta = *reinterpret_cast<const f32x4*>(&stat[stage][1][at]);
          const i32x4 seen = *reinterpret_cast<const i32x4*>(&sees[stage][at]);
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              float p = __builtin_amdgcn_exp2f(fmaf(sc[b][j][r], a.scale_log2, -lse[r]));
              if (!all && w0 + 16 * j + col >= seen[r]) p = 0.0f;
              const bool off = !all && w0 + 16 * j + col >= seen[r];
              sc[b][j][r] = p;
              dp[b][j][r] = off ? 0.0f : p * (dp[b][j][r] - delta[r]);
            }
        }
        i32x4 pf[2], sf[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          pf[j] = pack_blocks<IN>(sc[0][j], sc[1][j]);
          sf[j] = pack_blocks<IN>(dp[0][j], dp[1][j]);
        }
#pragma unroll
        for (int d = 0; d < T::DB; ++d) {
          const i32x4 gf = column_fragment<DP>(gt, lanes, half, d);
          const i32x4 qf = column_fragment<DP>(qt, lanes, half, d);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            dv[j][d] = mfma16_v<IN>(gf, pf[j], dv[j][d]);
            dk[j][d] = mfma16_v<IN>(qf, sf[j], dk[j][d]);
          }
        }
      }
    }
    if (more) {
      stage ^= 1;
      put(stage);
    }
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t key = w0 + 16 * j + col;
    if (key >= k_end - k_first) continue;
    const int64_t at = ((k_first + key) * a.k_heads + kh) * a.dim;
#pragma unroll
    for (int d = 0; d < T::DB; ++d) {
      const int c = 16 * d + 4 * quad;
      if (c < a.dim) {
        const f32x4 x = dk[j][d] * a.scale, y = dv[j][d];
        *reinterpret_cast<i32x2*>(static_cast<char*>(a.dk) + 2 * (at + c)) = i32x2{pack2<IN>(x[0], x[1]), pack2<IN>(x[2], x[3])};
        *reinterpret_cast<i32x2*>(static_cast<char*>(a.dv) + 2 * (at + c)) = i32x2{pack2<IN>(y[0], y[1]), pack2<IN>(y[2], y[3])};
      }
    }
  }
}

template <int IN, int DP>
__global__ __launch_bounds__(kThreads, 1) void attention_dq_kernel(AttnArgs a) {
  using T = TileOf<DP>;
  __shared__ __attribute__((aligned(16))) char lds[2][2][kTile * T::PITCH];
  const int lane = threadIdx.x & 63, wave = threadIdx.x / 64, quad = lane / 16, col = lane % 16;
  const int64_t tiles = gridDim.x / a.k_heads;
  const int kh = blockIdx.x % a.k_heads;
  const int64_t tile = tiles - 1 - blockIdx.x / a.k_heads;
  const int seg = segment_of_tile(a, tile, kRows);
  const Sequence s = segment(a, seg);
  const int64_t r0 = (tile - (s.q0 * a.group / kRows + seg)) * kRows;
  const int64_t rows = s.n * a.group;
  if (r0 >= rows) return;

  int64_t out[2];
  bool live[2];
  int seen[2];
  float lse[2], delta[2];
  i32x4 qf[2][T::KS], gf[2][T::KS];
  f32x4 dq[2][T::DB];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t row = r0 + 32 * wave + 16 * i + col, t = row / a.group;
    const int64_t h = kh * a.group + (row - t * a.group);
    live[i] = row < rows;
    out[i] = (s.q0 + t) * a.q_heads + h;
    seen[i] = (int)keys_seen(a, s, t);
    lse[i] = live[i] ? a.lse[out[i]] * kLog2e : 0.0f;
    delta[i] = live[i] ? a.delta[out[i]] : 0.0f;
    row_operand<DP>(qf[i], static_cast<const char*>(a.q) + 2 * ((s.q0 + t) * a.q_token + h * a.q_head), live[i], a.dim);
    row_operand<DP>(gf[i], static_cast<const char*>(a.d_o) + 2 * out[i] * a.dim, live[i], a.dim);
#pragma unroll
    for (int d = 0; d < T::DB; ++d) dq[i][d] = f32x4{};
  }
  auto seen_of = [&](int64_t r) { return (int)keys_seen(a, s, (r < rows ? r : rows - 1) / a.group); };
  const int need = __builtin_amdgcn_readfirstlane(seen_of(r0 + kRows - 1));
  const int64_t w0 = r0 + 32 * wave;
  const int wave_need = __builtin_amdgcn_readfirstlane(w0 < rows ? seen_of(w0 + 31) : 0);
  const int wave_all = __builtin_amdgcn_readfirstlane(w0 + 31 < rows ? seen_of(w0) : 0);

  const int64_t k_bytes = 2 * a.k_token, v_bytes = 2 * a.v_token;
  const char* const kp = static_cast<const char*>(a.k) + 2 * (s.k0 * a.k_token + kh * a.k_head);
  const char* const vp = static_cast<const char*>(a.v) + 2 * (s.k0 * a.v_token + kh * a.v_head);
  constexpr int N = kTile * T::SLOTS / kThreads;
  u32x4 nk[N], nv[N];
  auto fetch = [&](int64_t k0) {
    const auto kb = buffer_at(kp + k0 * k_bytes), vb = buffer_at(vp + k0 * v_bytes);
    const int left = (int)(s.m - k0 < kTile ? s.m - k0 : kTile);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = threadIdx.x + i * kThreads, r = at / T::SLOTS, c = at % T::SLOTS;
      const bool ok = r < left && c * 8 < a.dim;
      nk[i] = load_b128(kb, ok ? (unsigned)(r * (int)k_bytes + c * 16) : OOB);
      nv[i] = load_b128(vb, ok ? (unsigned)(r * (int)v_bytes + c * 16) : OOB);
    }
  };
  auto put = [&](int stage) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = threadIdx.x + i * kThreads, r = at / T::SLOTS, c = at % T::SLOTS;
      *reinterpret_cast<u32x4*>(lds[stage][0] + T::at(r, c)) = nk[i];
      *reinterpret_cast<u32x4*>(lds[stage][1] + T::at(r, c)) = nv[i];
    }
  };
  if (need > 0) {
    fetch(0);
    put(0);
  }
  __syncthreads();
  Lanes<DP> lanes;
  int stage = 0;
  for (int k0 = 0; k0 < need; k0 += kTile) {
    const bool more = k0 + kTile < need;
    if (more) fetch(k0 + kTile);
    const char* const kt = lds[stage][0];
    const char* const vt = lds[stage][1];
    if (k0 < wave_need) {
      const bool all = k0 + kTile <= wave_all;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        f32x4 sc[2][2], dp[2][2];  // [row set][block of keys]
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          sc[0][b] = sc[1][b] = dp[0][b] = dp[1][b] = f32x4{};
#pragma unroll
          for (int ks = 0; ks < T::KS; ++ks) {
            const i32x4 kf = row_fragment<DP>(kt, lanes, 2 * half + b, ks);
            const i32x4 vf = row_fragment<DP>(vt, lanes, 2 * half + b, ks);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              sc[i][b] = mfma16_v<IN>(kf, qf[i][ks], sc[i][b]);
              dp[i][b] = mfma16_v<IN>(vf, gf[i][ks], dp[i][b]);
            }
          }
        }
        i32x4 sf[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const bool off = !all && k0 + 32 * half + 16 * b + 4 * quad + r >= seen[i];
              const float p = __builtin_amdgcn_exp2f(fmaf(sc[i][b][r], a.scale_log2, -lse[i]));
              dp[i][b][r] = off ? 0.0f : p * (dp[i][b][r] - delta[i]);
            }
          sf[i] = pack_blocks<IN>(dp[i][0], dp[i][1]);
        }
#pragma unroll
        for (int d = 0; d < T::DB; ++d) {
          const i32x4 kf = column_fragment<DP>(kt, lanes, half, d);
          dq[0][d] = mfma16_v<IN>(kf, sf[0], dq[0][d]);
          dq[1][d] = mfma16_v<IN>(kf, sf[1], dq[1][d]);
        }
      }
    }
    if (more) {
      stage ^= 1;
      put(stage);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (!live[i]) continue;
#pragma unroll
    for (int d = 0; d < T::DB; ++d) {
      const int c = 16 * d + 4 * quad;
      if (c < a.dim) {
        const f32x4 x = dq[i][d] * a.scale;
        *reinterpret_cast<i32x2*>(static_cast<char*>(a.dq) + 2 * (out[i] * a.dim + c)) =
            i32x2{pack2<IN>(x[0], x[1]), pack2<IN>(x[2], x[3])};
      }
    }
  }
}

template <int IN, int DP>
hipError_t launch_in(const AttnArgs& a, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (a.q_rows > 0) {
    hipLaunchKernelGGL(attention_delta_kernel<IN>, dim3((unsigned)((a.q_rows * a.q_heads + 15) / 16)),
                       dim3(256), 0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t tiles = a.q_rows * a.group / kRows + a.batch + 2;
    hipLaunchKernelGGL((attention_dq_kernel<IN, DP>), dim3((unsigned)(tiles * a.k_heads)), dim3(kThreads),
                       0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.k_rows > 0) {
    const int64_t tiles = a.k_rows / kKeys + a.batch + 2;
    hipLaunchKernelGGL((attention_dkv_kernel<IN, DP>), dim3((unsigned)(tiles * a.k_heads)), dim3(kThreads),
                       0, s, a);
    e = hipGetLastError();
  }
  return e;
}

template <int IN>
hipError_t launch_dim(const AttnArgs& a, hipStream_t s) {
  if (a.dim <= 64) return launch_in<IN, 64>(a, s);
  if (a.dim <= 96) return launch_in<IN, 96>(a, s);
  return launch_in<IN, 128>(a, s);
}

}  // namespace

hipError_t launch_attention_backward(int in, const AttnArgs& a, hipStream_t s) {
  return in == GEMM_F16 ? launch_dim<GEMM_F16>(a, s) : launch_dim<GEMM_BF16>(a, s);
}

}  // namespace imm
