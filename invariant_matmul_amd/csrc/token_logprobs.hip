// Log probabilities of given tokens, the entropy and the most likely tokens of
// rows of logits, and the gradient of the logits.
//
//   M = max_v x_v, S = sum_v e^(x_v - M), T = sum_v e^(x_v - M) (x_v - M)
//   logp_v = (x_v - M) - ln S, entropy = -sum_v p_v logp_v = ln S - T / S
//   dx_v = sum_n g_n (1[v = token_n] - p_v) - h p_v (logp_v + entropy)
//
// The forward pass reads the logits once.  A wave holds a unit of 2048 logits
// in registers (32 a lane): its maximum, then S and T about each lane's own
// maximum, joined over the lanes; the units' (M, S, T) are joined at the end in
// an order that their number alone fixes.  So the bits of a row follow from its
// values and the vocabulary, whatever workgroup summed which unit: many rows run
// with a workgroup each, few rows are cut into parts whose results a second kernel
// joins.
//
// The most likely tokens are ordered by value (NaN above every number, as the
// largest), equal values by the lower token: the order of a 64-bit key of both,
// so the result needs no order of work.  A wave keeps its best as a sorted list, one
// entry a lane; a unit none of whose maxima passes the last entry costs one
// comparison.
//
// Many rows are bound by the bytes: 4093 rows of 100003 fp32 logits with 5 alternatives 305 us
// (5.4 TB/s), 4096 of 65536 in bf16 forward and backward 140 + 200 us (3.8 and 5.4 TB/s: the forward pass's
// vector units are busy 73 % of its cycles, with some 15 instructions a logit).  Few rows are bound by latency: 16 of 131072 with 20
// alternatives 10 us and the join 6, with the units' candidates kept one by one instead of by a threshold and a sort 53.
#include "decoder_internal.h"
#include "kernel_common.h"
#include "lanes.h"
#include "rows16.h"

// A product and a sum are fused where the code says fmaf and nowhere else: the kernels of whole rows and of parts
// round alike.
#pragma clang fp contract(off)

namespace imm {
namespace {
using namespace dev;

constexpr int kWaves = kLogprobsWaves, kThreads = 64 * kWaves;
constexpr int kUnit = kLogprobsUnit, kVecs = kUnit / 512;  // 8 logits of a lane at a time
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kNone = -__builtin_inff();

typedef u32x4_t u32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

template <int IN>
struct Size {
  static constexpr int value = IN == GEMM_F32 ? 4 : 2;
};

template <int IN>
__device__ __forceinline__ float load1(const void* x, int64_t i) {
  if constexpr (IN == GEMM_F32) return static_cast<const float*>(x)[i];
  else if constexpr (IN == GEMM_F16) return (float)static_cast<const _Float16*>(x)[i];
  else return __uint_as_float((unsigned)static_cast<const unsigned short*>(x)[i] << 16);
}

// Eight logits from element i on; elements from `end` on are -infinity and not
// read.  (Rows may begin at any element: the loads need no alignment.)
template <int IN>
__device__ __forceinline__ void load8(const void* x, int64_t i, int64_t end, float (&f)[8]) {
  if (i + 8 <= end) {
    if constexpr (IN == GEMM_F32) {
      const f32x4 a = *reinterpret_cast<const f32x4_any*>(static_cast<const float*>(x) + i);
      const f32x4 b = *reinterpret_cast<const f32x4_any*>(static_cast<const float*>(x) + i + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[e] = a[e];
        f[4 + e] = b[e];
      }
    } else {
      const u32x4_t v = *reinterpret_cast<const u32x4_any*>(static_cast<const char*>(x) + 2 * i);
      widen8<IN>(v, f);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = i + e < end ? load1<IN>(x, i + e) : kNone;
  }
}

// The order of the most likely tokens as unsigned keys: larger is better.
// Zeros of both signs are equal, NaN is above every number.
__device__ __forceinline__ unsigned order(float x) {
  const unsigned b = __float_as_uint(x == 0.0f ? 0.0f : x);
  return x != x ? 0xffffffffu : b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(unsigned key) {
  if (key == 0xffffffffu) return __builtin_nanf("");
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}
__device__ __forceinline__ uint64_t key_of(float x, int64_t token) {
  return (uint64_t)order(x) << 32 | (0xffffffffu - (unsigned)token);
}

__device__ __forceinline__ uint64_t lane_of(uint64_t v, int lane) {
  return (uint64_t)(unsigned)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
         (unsigned)__builtin_amdgcn_readlane((int)v, lane);
}

__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t smaller(uint64_t a, uint64_t b) { return a < b ? a : b; }
// A step of a bitonic network over the lanes: the larger of two keys that are D lanes
// apart goes to the lower lane, or to the higher one.
template <int D>
__device__ __forceinline__ uint64_t exchange(uint64_t key, bool falling) {
  const uint64_t other = lane_xor<D>(key);
  return ((threadIdx.x & D) == 0) == falling ? larger(key, other) : smaller(key, other);
}
// Keys of a wave in falling order (a bitonic sort).
__device__ __forceinline__ uint64_t sorted(uint64_t key) {
  each_up([&](auto k) {
    constexpr int K = decltype(k)::value;
    each_down<K>([&](auto d) { key = exchange<decltype(d)::value>(key, (threadIdx.x & 63 & (2 * K)) == 0); });
  });
  return key;
}

// A wave's 64 best keys, in falling order over its lanes (0: none); `last` is entry top - 1.
struct Best {
  uint64_t mine, last;
  int top;
  uint64_t* room;  // LDS for 128 keys
  __device__ __forceinline__ void insert(uint64_t key) {  // uniform, > last
    const uint64_t up = __shfl_up(mine, 1);
    const int lane = threadIdx.x & 63;
    const int at = __popcll(__ballot(mine > key));
    mine = lane < at ? mine : lane == at ? key : up;
    last = lane_of(mine, top - 1);
  }
  // 64 keys in falling order: the larger of each and of the opposite place are the best 64, in
  // bitonic order.
  __device__ __forceinline__ void join(uint64_t key) {
    mine = larger(mine, __shfl(key, 63 - (threadIdx.x & 63)));
    each_down<32>([&](auto d) { mine = exchange<decltype(d)::value>(mine, true); });
    last = lane_of(mine, top - 1);
  }
  // The first `n` keys of the room (n <= 64): by insertion where they are few.
  __device__ __forceinline__ void take(int n) {
    const int lane = threadIdx.x & 63;
    const uint64_t key = lane < n ? room[lane] : 0;
    if (n > 8) {
      join(sorted(key));
      return;
    }
    for (int i = 0; i < n; ++i) {
      const uint64_t k = lane_of(key, i);
      if (k > last) insert(k);
    }
  }
  // E keys of every lane, the largest of which is `largest`.  Keys that cannot be among
  // the best are passed by: those below `last`, and, of the first keys, those whose value is
  // below the top-th largest of the lanes' own largest (to 16 bits, which bf16 values have).  The
  // others are gathered in LDS.
  template <int E, class KEY>
  __device__ __forceinline__ void offer(uint64_t largest, KEY&& key) {
    if (!__any(largest > last)) return;
    uint64_t least = last;
    if (last == 0) {
      unsigned value = 0;
      for (unsigned bit = 1u << 31; bit >= 1u << 16; bit >>= 1)
        if (__popcll(__ballot((unsigned)(largest >> 32) >= (value | bit))) >= top) value |= bit;
      least = value ? ((uint64_t)value << 32) - 1 : 0;
    }
    const int lane = threadIdx.x & 63;
    int n = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint64_t k = key(e);
      const uint64_t found = __ballot(k > least);
      if (!found) continue;
      if (k > least) room[n + __popcll(found & ((1ull << lane) - 1))] = k;
      n += __popcll(found);
      if (n >= 64) {
        wait_lds();
        take(64);
        least = larger(least, last);
        n -= 64;
        const uint64_t rest = room[64 + lane];
        wait_lds();
        if (lane < n) room[lane] = rest;
      }
    }
    if (n) {
      wait_lds();
      take(n);
      wait_lds();  // before the room is used again
    }
  }
  // (the room is one wave's: its own LDS operations are in order)
  __device__ __forceinline__ static void wait_lds() { __builtin_amdgcn_wave_barrier(); }
};

struct Sums {
  float m, s, t;
};
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }
// Below this e^d is 0 in fp32; d stays finite, so that 0 d is 0.
constexpr float kLeast = -1000.0f;
// The sums of both, about the larger maximum.  The first's products are fused with the second's, so that two lanes
// that join each other's sums may differ in the last bit: lane 0's are the result.  (Without the
// fused sums they agree, and 4093 rows of 100003 fp32 logits take 311 us instead of 307.)
__device__ __forceinline__ Sums join(Sums a, Sums b) {
  // (NaN maxima do not occur: a NaN among the logits is in s and t)
  const float m = fmaxf(a.m, b.m);
  if (m == kNone) return Sums{m, a.s + b.s, a.t + b.t};
  const float da = fmaxf(a.m - m, kLeast), ea = exp_of(da), db = fmaxf(b.m - m, kLeast), eb = exp_of(db);
  return Sums{m, fmaf(a.s, ea, b.s * eb), fmaf(fmaf(a.s, da, a.t), ea, fmaf(b.s, db, b.t) * eb)};
}
__device__ __forceinline__ Sums join_lanes(Sums a) {
  each_up([&](auto d) {
    constexpr int D = decltype(d)::value;
    a = join(a, Sums{lane_xor<D>(a.m), lane_xor<D>(a.s), lane_xor<D>(a.t)});
  });
  return a;
}
__device__ __forceinline__ float of_lane_0(float v) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
}

// One unit: its sums (lane 0's), and its logits offered to `best`.
template <int IN, bool TOP>
__device__ __forceinline__ Sums take_unit(const void* row, int64_t v0, int64_t vocab, Best& best) {
  const int lane = threadIdx.x & 63;
  float x[kVecs][8];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) load8<IN>(row, v0 + 512 * i + 8 * lane, vocab, x[i]);
  float m = kNone;
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, x[i][e]);
  const float about = m == kNone ? 0.0f : m;
  float s = 0.0f, t = 0.0f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = x[i][e] - about, p = exp_of(d);
      s += p;
      t = fmaf(p, fmaxf(d, kLeast), t);
    }
  const Sums all = join_lanes(Sums{m, s, t});
  if constexpr (TOP) {
    unsigned highest = order(m);
    if (__any(s != s)) {  // a NaN, which takes no part in m, or an infinity
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) highest = max(highest, order(x[i][e]));
    }
    const uint64_t largest = (uint64_t)highest << 32 | 0xffffffffu;
    best.offer<8 * kVecs>(largest, [&](int e) {
      const int64_t v = v0 + 512 * (e / 8) + 8 * lane + e % 8;
      return v < vocab ? key_of(x[e / 8][e % 8], v) : 0ull;
    });
  }
  return all;
}

// The row's results from its units' sums and the waves' lists, by one wave.
template <int IN>
__device__ __forceinline__ void finish(const LogprobsArgs& g, int64_t row, const float* sums,
                                       const uint64_t* lists, int nlists, uint64_t* room) {
  const int lane = threadIdx.x & 63;
  Sums a{kNone, 0.0f, 0.0f};
  for (int u = lane; u < g.units; u += 64)
    a = join(a, Sums{sums[3 * u], sums[3 * u + 1], sums[3 * u + 2]});
  a = join_lanes(a);
  a = Sums{of_lane_0(a.m), of_lane_0(a.s), of_lane_0(a.t)};  // every column's and every alternative's
  const float ln_s = logf(a.s);
  if (lane == 0) {
    g.entropy[row] = ln_s - a.t / a.s;
    if (g.norm) {
      g.norm[2 * row] = a.m;
      g.norm[2 * row + 1] = ln_s;
    }
  }
  const char* const x = static_cast<const char*>(g.x) + row * g.row_stride * Size<IN>::value;
  for (int i = lane; i < g.n; i += 64) {
    const int64_t t = g.tokens[row * g.n + i];
    float lp = 0.0f;  // no token
    if (t >= g.vocab) lp = __builtin_nanf("");
    else if (t >= 0) lp = (load1<IN>(x, t) - a.m) - ln_s;
    g.logprob[row * g.n + i] = lp;
  }
  if (g.top) {
    Best best{0, 0, g.top, room};
    // a list a lane, 16 entries at a time (they fall: the first is the largest)
    for (int l0 = 0; l0 < nlists; l0 += 64) {
      const uint64_t* const list = lists + (int64_t)(l0 + lane) * g.top;
      const bool mine = l0 + lane < nlists;
      for (int e0 = 0; e0 < g.top; e0 += 16) {
        uint64_t k[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) k[e] = mine && e0 + e < g.top ? list[e0 + e] : 0;
        best.offer<16>(k[0], [&](int e) { return k[e]; });
      }
    }
    if (lane < g.top) {
      g.top_logprob[row * g.top + lane] = (value_of((unsigned)(best.mine >> 32)) - a.m) - ln_s;
      g.top_token[row * g.top + lane] = 0xffffffffu - (unsigned)best.mine;
    }
  }
}

// PARTS: the workgroup's part of a row, to the workspace; otherwise a whole row.
template <int IN, bool PARTS, bool TOP>
__global__ __launch_bounds__(kThreads, PARTS ? 5 : 6) void logprobs_kernel(LogprobsArgs g) {
  extern __shared__ float shared[];  // sums [units, 3] of a whole row
  __shared__ uint64_t lists[kWaves][kLogprobsMaxTop], room[kWaves][128];
  const int wave = threadIdx.x / 64, lane = threadIdx.x & 63;
  const int64_t row = PARTS ? blockIdx.x / g.parts : blockIdx.x;
  const int part = PARTS ? (int)(blockIdx.x % g.parts) : 0;
  const char* const x = static_cast<const char*>(g.x) + row * g.row_stride * Size<IN>::value;
  float* const sums = PARTS ? g.sums + row * g.units * 3 : shared;
  Best best{0, 0, g.top ? g.top : 1, room[wave]};
  const int step = PARTS ? kWaves * g.parts : kWaves;
  for (int u = part * kWaves + wave; u < g.units; u += step) {
    const Sums a = take_unit<IN, TOP>(x, (int64_t)u * kUnit, g.vocab, best);
    if (lane == 0) {
      sums[3 * u] = a.m;
      sums[3 * u + 1] = a.s;
      sums[3 * u + 2] = a.t;
    }
  }
  if constexpr (PARTS) {
    if (lane < g.top)
      g.best[((row * g.parts + part) * kWaves + wave) * g.top + lane] = best.mine;
  } else {
    if (lane < g.top) lists[0][wave * g.top + lane] = best.mine;
    __syncthreads();
    if (wave == 0) finish<IN>(g, row, sums, lists[0], kWaves, room[0]);
  }
}

template <int IN>
__global__ __launch_bounds__(64) void logprobs_join_kernel(LogprobsArgs g) {
  const int64_t row = blockIdx.x;
  __shared__ uint64_t room[128];
  const int lists = g.parts * kWaves;
  finish<IN>(g, row, g.sums + row * g.units * 3, g.best + row * lists * g.top, lists, room);
}

// The gradient of the logits: a workgroup takes 2048 logits of a row.
template <int IN>
__global__ __launch_bounds__(kThreads) void logprobs_backward_kernel(LogprobsArgs g) {
  const int64_t blocks = (g.vocab + 8 * kThreads - 1) / (8 * kThreads);
  const int64_t row = blockIdx.x / blocks;
  const int64_t v0 = (blockIdx.x - row * blocks) * 8 * kThreads + threadIdx.x * 8;
  const char* const x = static_cast<const char*>(g.x) + row * g.row_stride * Size<IN>::value;
  if (v0 >= g.vocab) return;
  float f[8];
  load8<IN>(x, v0, g.vocab, f);
  const float m = g.norm[2 * row], ln_s = g.norm[2 * row + 1];
  const float h = g.d_entropy ? g.d_entropy[row] : 0.0f, ent = g.entropy[row];
  float all = 0.0f, mine[8] = {};
  for (int i = 0; i < g.n; ++i) {
    const int64_t t = g.tokens[row * g.n + i];
    if (t < 0 || !g.d_logprob) continue;
    const float d = t < g.vocab ? g.d_logprob[row * g.n + i] : __builtin_nanf("");
    all += d;
#pragma unroll
    for (int e = 0; e < 8; ++e) mine[e] += v0 + e == t ? d : 0.0f;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float logp = (f[e] - m) - ln_s, p = exp_of(logp);
    f[e] = fmaf(-p, fmaf(h, fmaxf(logp, kLeast) + ent, all), mine[e]);
  }
  char* const out = static_cast<char*>(g.dx) + row * g.vocab * Size<IN>::value;
  if (v0 + 8 <= g.vocab) {
    if constexpr (IN == GEMM_F32) {
      *reinterpret_cast<f32x4_any*>(out + 4 * v0) = f32x4{f[0], f[1], f[2], f[3]};
      *reinterpret_cast<f32x4_any*>(out + 4 * v0 + 16) = f32x4{f[4], f[5], f[6], f[7]};
    } else {
      *reinterpret_cast<u32x4_any*>(out + 2 * v0) = narrow8<IN>(f);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (v0 + e < g.vocab) store_out<IN>(out, v0 + e, f[e]);
  }
}

template <class F>
void with_type(int in, F&& f) {
  if (in == GEMM_F16) f(std::integral_constant<int, GEMM_F16>{});
  else if (in == GEMM_BF16) f(std::integral_constant<int, GEMM_BF16>{});
  else f(std::integral_constant<int, GEMM_F32>{});
}

LogprobsArgs from_row(const LogprobsArgs& a, int in, int64_t r, int64_t rows) {
  LogprobsArgs b = a;
  const int64_t size = in == GEMM_F32 ? 4 : 2;
  b.rows = rows;
  b.x = static_cast<const char*>(a.x) + r * a.row_stride * size;
  b.tokens = a.tokens ? a.tokens + r * a.n : nullptr;
  b.logprob = a.logprob ? a.logprob + r * a.n : nullptr;
  b.entropy = a.entropy + r;
  b.norm = a.norm ? a.norm + 2 * r : nullptr;
  b.top_logprob = a.top_logprob ? a.top_logprob + r * a.top : nullptr;
  b.top_token = a.top_token ? a.top_token + r * a.top : nullptr;
  b.d_logprob = a.d_logprob ? a.d_logprob + r * a.n : nullptr;
  b.d_entropy = a.d_entropy ? a.d_entropy + r : nullptr;
  b.dx = a.dx ? static_cast<char*>(a.dx) + r * a.vocab * size : nullptr;
  return b;
}

}  // namespace

// Workgroups of a row: one from 1024 rows on; below, as many as leave every
// wave a unit, up to 1024 in all.
int logprobs_parts(int64_t rows, int64_t vocab) {
  const int64_t units = (vocab + kUnit - 1) / kUnit, most = (units + kWaves - 1) / kWaves;
  if (rows <= 0) return 1;
  const int64_t want = 1024 / rows;
  return (int)(want < 1 ? 1 : want < most ? want : most);
}

hipError_t launch_logprobs(int in, const LogprobsArgs& a, hipStream_t s) {
  hipError_t e = hipSuccess;
  with_type(in, [&](auto dt) {
    constexpr int IN = decltype(dt)::value;
    if (a.parts > 1) {
      const auto kernel = a.top ? logprobs_kernel<IN, true, true> : logprobs_kernel<IN, true, false>;
      hipLaunchKernelGGL(kernel, dim3((unsigned)(a.rows * a.parts)), dim3(kThreads), 0, s, a);
      e = hipGetLastError();
      if (e != hipSuccess) return;
      hipLaunchKernelGGL(logprobs_join_kernel<IN>, dim3((unsigned)a.rows), dim3(64), 0, s, a);
      e = hipGetLastError();
      return;
    }
    const auto kernel = a.top ? logprobs_kernel<IN, false, true> : logprobs_kernel<IN, false, false>;
    const int64_t most = (int64_t)1 << 23;  // (a launch holds fewer than 2^32 threads)
    for (int64_t r = 0; r < a.rows && e == hipSuccess; r += most) {
      const int64_t rows = a.rows - r < most ? a.rows - r : most;
      hipLaunchKernelGGL(kernel, dim3((unsigned)rows), dim3(kThreads), a.units * 3 * sizeof(float), s, from_row(a, in, r, rows));
      e = hipGetLastError();
    }
  });
  return e;
}

hipError_t launch_logprobs_backward(int in, const LogprobsArgs& a, hipStream_t s) {
  hipError_t e = hipSuccess;
  const int64_t blocks = (a.vocab + 8 * kThreads - 1) / (8 * kThreads);
  const int64_t most = ((int64_t)1 << 23) / blocks;
  with_type(in, [&](auto dt) {
    for (int64_t r = 0; r < a.rows && e == hipSuccess; r += most) {
      const int64_t rows = a.rows - r < most ? a.rows - r : most;
      hipLaunchKernelGGL(logprobs_backward_kernel<decltype(dt)::value>, dim3((unsigned)(rows * blocks)),
                         dim3(kThreads), 0, s, from_row(a, in, r, rows));
      e = hipGetLastError();
    }
  });
  return e;
}

}  // namespace imm
