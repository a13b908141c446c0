// The gradients of attention.  With p_ij = e^(scale q_i k_j - lse_i) and
// delta_i = sum_d do_id o_id:
//   dv_j = sum_i p_ij do_i
//   ds_ij = p_ij (do_i v_j - delta_i)
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i
//
// One kernel makes lse and delta of every row ready, one makes the gradients: its workgroups
// have a role each, dq of 128 rows, which walk through their keys, and dk or dv of 128
// keys, which walk through the rows that see them (64 of each in small calls).  p is made by
// all three and ds by two, so that every sum is one chain in one workgroup: no atomics, and
// the gradients of a sequence depend on that sequence alone.  dk and dv apart cost one product
// more (q k twice) than together, but fit a wave into half of a SIMD's registers: with both at
// once (254 + 256 registers, one wave a SIMD) that kernel took 3180 us for 8192 tokens of 8 key
// heads and 32 query heads of 128 where now all three take 2000 (matrix units busy 39 %,
// then exponentials, differences and packing, waits 28 %).
// p and ds are rounded to the input's type for their products (the rest of large ds follows),
// all else is fp32.
#include "attention_common.h"
#include "rows16.h"

namespace imm {
namespace {
using namespace dev;

template <int SETS>
constexpr int kBlock = 16 * SETS * kWaves;  // rows (dq) or keys (dk, dv) of a workgroup
constexpr float kLog2e = 1.44269504088896340736f;

// -lse log2(e) and delta of every row in the order of the packed rows, [key head][query][head
// of the group]; 16 lanes a row, 8 elements each.  With o alone, the rounding of o is as large a part of
// the gradients' error as the rounding of ds; with what it left (o_low) that is gone
// (1500 bf16 keys of 128: dq is off by 0.00245 of itself instead of 0.00305, where its own
// rounding makes 0.00166).
template <int IN>
__global__ __launch_bounds__(256) void attention_delta_kernel(AttnArgs a) {
  const int64_t at = (int64_t)(blockIdx.y * gridDim.x + blockIdx.x) * 16 + threadIdx.x / 16;
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
  if (c == 0 && at < a.q_rows * a.q_heads) {
    const int q = (unsigned)at / (unsigned)a.q_heads;
    const int head = (int)at - q * a.q_heads, kh = head / a.group;
    const int64_t to = ((int64_t)kh * a.q_rows + q) * a.group + (head - kh * a.group);
    a.stats[to] = -a.lse[at] * kLog2e;
    a.stats[a.q_rows * a.q_heads + to] = sum;
  }
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

// Two sets of 16 results, dimension by row or key, to 16-bit rows.
template <int IN, int DP>
__device__ __forceinline__ void store_rows(const f32x4 (&x)[TileOf<DP>::DB], float scale, void* to, int64_t at, int dim) {
  const int quad = (threadIdx.x & 63) / 16;
#pragma unroll
  for (int d = 0; d < TileOf<DP>::DB; ++d) {
    const int c = 16 * d + 4 * quad;
    const f32x4 y = x[d] * scale;
    if (c < dim)
      *reinterpret_cast<i32x2*>(static_cast<char*>(to) + 2 * (at + c)) = i32x2{pack2<IN>(y[0], y[1]), pack2<IN>(y[2], y[3])};
  }
}

// What the rounding of two blocks of ds left, where p is large.  The rounding of ds is the
// largest error of dq and dk, and the few large p of a row make much of it: their rest goes
// through the product too, in the steps that have one.  (Packed bf16 documents of 200 to 3500
// tokens: dq is off by 0.0023 of itself instead of 0.0025, with the rests of all p by 0.0018,
// and its own rounding makes 0.0017.  It costs 5 to 8 % of the kernel's time, as much by the
// branch as by the products.)  A rule of the element alone: zeros add nothing.
constexpr float kLarge = 0.25f;
template <int IN>
__device__ __forceinline__ i32x4 rest_of(const f32x4& a, const f32x4& b, const f32x4& pa, const f32x4& pb,
                                         const i32x4& rounded) {
  i32x4 rest;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const f32x4 &x = e < 2 ? a : b, &p = e < 2 ? pa : pb;
    const int i = 2 * (e % 2);
    const int kept = (p[i] >= kLarge ? 0xffff : 0) | (p[i + 1] >= kLarge ? (int)0xffff0000 : 0);
    rest[e] = pack2_rest<IN>(x[i], x[i + 1], rounded[e]) & kept;
  }
  return rest;
}

// Results that are not finite.  A step multiplies by 0 what a row or key does not see, and 0 times an infinity or a
// NaN is a NaN: how far one reaches beyond what the formula gives follows from the steps that a wave
// walks, and so from the number of its rows or keys.  A workgroup of two sets a wave that finds such
// results therefore makes them again with one set a wave, as all smaller calls do: the reach, at most 15 + 63
// places, and every bit are then the sequence's own.
template <int SETS, int DB>
__device__ __forceinline__ bool not_finite(const f32x4 (&x)[SETS][DB]) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < SETS; ++i)
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) bad |= !(fabsf(x[i][d][r]) < __builtin_inff());
  return bad;
}
// The kernel's argument from memory once more.  (The compiler would otherwise hold what the rare second
// pass needs through the loops ahead: 145 scalar registers spilled, the training case 577 us instead of 556, with no
// second pass at all 553.)
__device__ __forceinline__ const AttnArgs& again(const AttnArgs& a) {
#if defined(__HIP_DEVICE_COMPILE__)
  auto p = (const __attribute__((address_space(4))) AttnArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const AttnArgs*)p;
#else
  return a;
#endif
}
// f(first) of the two halves of a tile, once every wave is done with the stages.
template <class F>
__device__ __forceinline__ void by_halves(int first, F&& f) {
  for (int half = 0; half < 2; ++half) {
    __syncthreads();
    f(first + half * kBlock<1>);
  }
}

template <int DP>
struct Stages {  // (arrays of their own, as in the forward kernel)
  char *x0, *y0, *x1, *y1;
  float *n0, *d0, *n1, *d1;
};

// dq of a sequence's rows from r0 on.
template <int IN, int DP, int SETS>
__device__ __forceinline__ void rows_role(const AttnArgs& a, const Sequence& s, int r0, int kh, const Stages<DP>& st) {
  using T = TileOf<DP>;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int quad = lane / 16, col = lane % 16;
  const int rows = s.n * a.group;
  if (r0 >= rows) return;

  int seen[SETS];
  float nl[SETS], delta[SETS];
  i32x4 qf[SETS][T::KS], gf[SETS][T::KS];
  f32x4 dq[SETS][T::DB];
  const int w0 = r0 + 16 * SETS * wave;
#pragma unroll
  for (int i = 0; i < SETS; ++i) {
    const int row = w0 + 16 * i + col, t = row / a.group;
    const int h = kh * a.group + (row - t * a.group);
    const bool live = row < rows;
    seen[i] = keys_seen(a, s, t);
    const int64_t at = ((int64_t)kh * a.q_rows + s.q0) * a.group + row;
    nl[i] = live ? a.stats[at] : 0.0f;
    delta[i] = live ? a.stats[a.q_rows * a.q_heads + at] : 0.0f;
    row_operand<DP>(qf[i], static_cast<const char*>(a.q) + 2 * ((s.q0 + t) * a.q_token + h * a.q_head), live, a.dim);
    row_operand<DP>(gf[i], static_cast<const char*>(a.d_o) + 2 * ((int64_t)(s.q0 + t) * a.q_heads + h) * a.dim, live, a.dim);
#pragma unroll
    for (int d = 0; d < T::DB; ++d) dq[i][d] = f32x4{};
  }
  auto seen_of = [&](int r) { return keys_seen(a, s, (r < rows ? r : rows - 1) / a.group); };
  const int need = __builtin_amdgcn_readfirstlane(seen_of(r0 + kBlock<SETS> - 1));
  const int wave_need = __builtin_amdgcn_readfirstlane(w0 < rows ? seen_of(w0 + 16 * SETS - 1) : 0);
  const int wave_all = __builtin_amdgcn_readfirstlane(w0 < rows ? seen_of(w0) : 0);

  const int64_t k_bytes = 2 * a.k_token, v_bytes = 2 * a.v_token;
  const char* const kp = static_cast<const char*>(a.k) + 2 * (s.k0 * a.k_token + kh * a.k_head);
  const char* const vp = static_cast<const char*>(a.v) + 2 * (s.k0 * a.v_token + kh * a.v_head);
  const Mover<DP> km(k_bytes, a.dim), vm(v_bytes, a.dim);
  Lanes<DP> lanes;
  auto fetch = [&](int k0, char* kt, char* vt) {
    km.move(kp + k0 * k_bytes, kt, s.m - k0, k_bytes, a.dim);
    vm.move(vp + k0 * v_bytes, vt, s.m - k0, v_bytes, a.dim);
  };
  auto one = [&](int k0, const char* kt, const char* vt, char* next_k, char* next_v) {
    landed();
    if (k0 + kTile < need) fetch(k0 + kTile, next_k, next_v);
    if (k0 >= wave_need) return;
    const bool all = k0 + kTile <= wave_all;
    lanes.again();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      f32x4 sc[SETS][2], dp[SETS][2];  // [row set][block of keys]
#pragma unroll
      for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int i = 0; i < SETS; ++i) sc[i][b] = dp[i][b] = f32x4{};
#pragma unroll
        for (int ks = 0; ks < T::KS; ++ks) {
          const i32x4 kf = row_fragment<DP>(kt, lanes, 2 * half + b, ks);
          const i32x4 vf = row_fragment<DP>(vt, lanes, 2 * half + b, ks);
#pragma unroll
          for (int i = 0; i < SETS; ++i) {
            sc[i][b] = mfma16_v<IN>(kf, qf[i][ks], sc[i][b]);
            dp[i][b] = mfma16_v<IN>(vf, gf[i][ks], dp[i][b]);
          }
        }
      }
      i32x4 sf[SETS];
      float largest = 0.0f;
#pragma unroll
      for (int i = 0; i < SETS; ++i) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            sc[i][b][r] = __builtin_amdgcn_exp2f(fmaf(sc[i][b][r], a.scale_log2, nl[i]));
            dp[i][b][r] = sc[i][b][r] * (dp[i][b][r] - delta[i]);
            largest = fmaxf(largest, sc[i][b][r]);
          }
        if (!all) {
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (k0 + 32 * half + 16 * b + 4 * quad + r >= seen[i]) dp[i][b][r] = 0.0f;
        }
        sf[i] = pack_blocks<IN>(dp[i][0], dp[i][1]);
      }
#pragma unroll
      for (int d = 0; d < T::DB; ++d) {
        const i32x4 kf = column_fragment<DP>(kt, lanes, half, d);
#pragma unroll
        for (int i = 0; i < SETS; ++i) dq[i][d] = mfma16_v<IN>(kf, sf[i], dq[i][d]);
      }
      if (__any(largest >= kLarge)) {
#pragma unroll
        for (int i = 0; i < SETS; ++i) sf[i] = rest_of<IN>(dp[i][0], dp[i][1], sc[i][0], sc[i][1], sf[i]);
#pragma unroll
        for (int d = 0; d < T::DB; ++d) {
          const i32x4 kf = column_fragment<DP>(kt, lanes, half, d);
#pragma unroll
          for (int i = 0; i < SETS; ++i) dq[i][d] = mfma16_v<IN>(kf, sf[i], dq[i][d]);
        }
      }
    }
  };
  if (need > 0) fetch(0, st.x0, st.y0);
  for (int k0 = 0; k0 < need; k0 += 2 * kTile) {
    one(k0, st.x0, st.y0, st.x1, st.y1);
    if (k0 + kTile < need) one(k0 + kTile, st.x1, st.y1, st.x0, st.y0);
  }
  if constexpr (SETS == 2) {
    if (__syncthreads_or(not_finite(dq)))
      return by_halves(r0, [&](int first) { rows_role<IN, DP, 1>(again(a), s, first, kh, st); });
  }
#pragma unroll
  for (int i = 0; i < SETS; ++i) {
    const int row = w0 + 16 * i + col, t = row / a.group;
    if (seen[i] == 0) {  // (whatever the wave's other rows see)
#pragma unroll
      for (int d = 0; d < T::DB; ++d) dq[i][d] = f32x4{};
    }
    const int64_t h = kh * a.group + (row - t * a.group);
    if (row < rows) store_rows<IN, DP>(dq[i], a.scale, a.dq, ((int64_t)(s.q0 + t) * a.q_heads + h) * a.dim, a.dim);
  }
}

// Moves 64 packed rows of a sequence's q or do to LDS (rows past the last: zeros).  The rows of
// a thread keep their query and head as counts that advance by 64 rows.
template <int DP>
struct RowMover {
  static constexpr int N = kTile * TileOf<DP>::SLOTS / kThreads, ROWS = kThreads / TileOf<DP>::SLOTS;
  int query[N], head[N];  // of the group
  int first, first_head;  // of the step's first row
  int per, rest;          // queries of 64 rows, and the heads left over
  unsigned slot;          // its byte, or OOB
  __device__ __forceinline__ RowMover(int from, int group, int dim) {
    per = kTile / group;
    rest = kTile - per * group;
    first = __builtin_amdgcn_readfirstlane(from / group);
    first_head = from - first * group;
    const int row = threadIdx.x / TileOf<DP>::SLOTS;
    const int c = (threadIdx.x % TileOf<DP>::SLOTS) ^ (row & (TileOf<DP>::SLOTS - 1));
    slot = c * 8 < dim ? c * 16 : OOB;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = from + row + i * ROWS;
      query[i] = r / group;
      head[i] = r - query[i] * group;
    }
  }
  __device__ __forceinline__ void advance(int& q, int& h, int group) const {
    h += rest;
    const bool over = h >= group;
    h -= over ? group : 0;
    q += over ? per + 1 : per;
  }
  __device__ __forceinline__ void advance(int group) {
#pragma unroll
    for (int i = 0; i < N; ++i) advance(query[i], head[i], group);
    advance(first, first_head, group);
  }
  // base: the sequence's first query's first head of the group
  __device__ __forceinline__ void move(const char* base, int64_t token_bytes, int64_t head_bytes, int64_t queries,
                                       char* to) const {
    const auto buf = buffer_at(base + first * token_bytes);
    char* const mine = to + __builtin_amdgcn_readfirstlane(threadIdx.x & ~63) * 16;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const unsigned off = (unsigned)((query[i] - first) * (int)token_bytes) + (unsigned)(head[i] * (int)head_bytes) + slot;
      dma16(buf, mine + i * kThreads * 16, query[i] < queries && slot != OOB ? off : OOB, 0);
    }
  }
};

// Binary places by which p is raised for dv's products, and the sums lowered: in fp16 a p below 2^-14 would
// lose bits, one below 2^-25 all of them, as the p of ten thousand keys that a row sees do (64 queries over 65536 keys
// of 64, logits of standard deviation 1: dv would be off by 0.00072 of itself, it is by 0.00030).  p is at most 1 and fp16 reaches 2^15.  (bf16 needs none, and its
// values times 2^14 may leave fp32's range.)
template <int IN>
constexpr int kRaised = IN == GEMM_F16 ? 14 : 0;

// dk (DK) or dv of a segment's keys from c0 on.
template <int IN, int DP, bool DK, int SETS>
__device__ __forceinline__ void keys_role(const AttnArgs& a, const Found& found, int c0, int kh, const Stages<DP>& st) {
  using T = TileOf<DP>;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int quad = lane / 16, col = lane % 16;
  const Sequence s = found.s;
  const int k_first = s.k0, k_end = found.k_end;
  if (c0 >= k_end - k_first) return;
  const int rows = s.n * a.group;
  const int w0 = c0 + 16 * SETS * wave;
  // the first row that sees a key
  auto first_row = [&](int key) {
    if (key >= s.m) return rows;
    return a.causal ? clamped(key - (s.m - s.n), 0, s.n) * a.group : 0;
  };
  i32x4 kf[SETS][T::KS], vf[DK ? SETS : 1][T::KS];
  f32x4 sum[SETS][T::DB];
  int from_row[SETS];
#pragma unroll
  for (int j = 0; j < SETS; ++j) {
    const int key = w0 + 16 * j + col;
    row_operand<DP>(kf[j], static_cast<const char*>(a.k) + 2 * ((k_first + key) * a.k_token + kh * a.k_head), key < s.m, a.dim);
    if constexpr (DK)
      row_operand<DP>(vf[j], static_cast<const char*>(a.v) + 2 * ((k_first + key) * a.v_token + kh * a.v_head), key < s.m, a.dim);
    from_row[j] = first_row(key);
#pragma unroll
    for (int d = 0; d < T::DB; ++d) sum[j][d] = f32x4{};
  }
  const int from = first_row(c0) / kTile * kTile;
  const int wave_from = first_row(w0), wave_all = first_row(w0 + 16 * SETS - 1);

  const char* const qp = static_cast<const char*>(a.q) + 2 * (s.q0 * a.q_token + (int64_t)kh * a.group * a.q_head);
  const char* const gp = static_cast<const char*>(a.d_o) + 2 * ((int64_t)s.q0 * a.q_heads + kh * a.group) * a.dim;
  const float* const stats = a.stats + ((int64_t)kh * a.q_rows + s.q0) * a.group;
  const int64_t all_rows = a.q_rows * a.q_heads;
  RowMover<DP> rm(from, a.group, a.dim);
  Lanes<DP> lanes;
  auto fetch = [&](int r0, char* qt, char* gt, float* nl, float* delta) {
    rm.move(qp, 2 * a.q_token, 2 * a.q_head, s.n, qt);
    rm.move(gp, 2 * (int64_t)a.q_heads * a.dim, 2 * a.dim, s.n, gt);
    rm.advance(a.group);
    // a wave moves each of the two numbers of the rows
    if (wave < (DK ? 2 : 1)) {
      const auto buf = buffer_at(stats + (wave ? all_rows : 0) + r0);
      dma4(buf, reinterpret_cast<char*>(wave ? delta : nl), r0 + lane < rows ? (unsigned)(lane * 4) : OOB);
    }
  };
  auto one = [&](int r0, const char* qt, const char* gt, const float* nls, const float* deltas, char* next_q, char* next_g,
                 float* next_n, float* next_d) {
    landed();
    if (r0 + kTile < rows) fetch(r0 + kTile, next_q, next_g, next_n, next_d);
    if (r0 + kTile <= wave_from) return;
    const bool all = r0 >= wave_all;  // (rows past the last are zeros and add nothing)
    lanes.again();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float largest = 0.0f;
      f32x4 sc[2][SETS], dp[2][SETS];  // [block of rows][block of keys]
#pragma unroll
      for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int j = 0; j < SETS; ++j) sc[b][j] = dp[b][j] = f32x4{};
#pragma unroll
        for (int ks = 0; ks < T::KS; ++ks) {
          const i32x4 qf = row_fragment<DP>(qt, lanes, 2 * half + b, ks);
#pragma unroll
          for (int j = 0; j < SETS; ++j) sc[b][j] = mfma16_v<IN>(qf, kf[j][ks], sc[b][j]);
          if constexpr (DK) {
            const i32x4 gf = row_fragment<DP>(gt, lanes, 2 * half + b, ks);
#pragma unroll
            for (int j = 0; j < SETS; ++j) dp[b][j] = mfma16_v<IN>(gf, vf[j][ks], dp[b][j]);
          }
        }
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int at = 32 * half + 16 * b + 4 * quad;
        f32x4 nl = *reinterpret_cast<const f32x4*>(nls + at);
        if constexpr (!DK && kRaised<IN> != 0) nl += (float)kRaised<IN>;
        f32x4 delta{};
        if constexpr (DK) delta = *reinterpret_cast<const f32x4*>(deltas + at);
#pragma unroll
        for (int j = 0; j < SETS; ++j) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            sc[b][j][r] = __builtin_amdgcn_exp2f(fmaf(sc[b][j][r], a.scale_log2, nl[r]));
            if constexpr (DK) {
              dp[b][j][r] = sc[b][j][r] * (dp[b][j][r] - delta[r]);
              largest = fmaxf(largest, sc[b][j][r]);
            }
          }
          if (!all) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (r0 + at + r < from_row[j]) (DK ? dp : sc)[b][j][r] = 0.0f;
          }
        }
      }
      i32x4 f[SETS];
#pragma unroll
      for (int j = 0; j < SETS; ++j) f[j] = pack_blocks<IN>((DK ? dp : sc)[0][j], (DK ? dp : sc)[1][j]);
#pragma unroll
      for (int d = 0; d < T::DB; ++d) {
        const i32x4 x = column_fragment<DP>(DK ? qt : gt, lanes, half, d);
#pragma unroll
        for (int j = 0; j < SETS; ++j) sum[j][d] = mfma16_v<IN>(x, f[j], sum[j][d]);
      }
      if (DK && __any(largest >= kLarge)) {
#pragma unroll
        for (int j = 0; j < SETS; ++j) f[j] = rest_of<IN>(dp[0][j], dp[1][j], sc[0][j], sc[1][j], f[j]);
#pragma unroll
        for (int d = 0; d < T::DB; ++d) {
          const i32x4 x = column_fragment<DP>(qt, lanes, half, d);
#pragma unroll
          for (int j = 0; j < SETS; ++j) sum[j][d] = mfma16_v<IN>(x, f[j], sum[j][d]);
        }
      }
    }
  };
  if (from < rows) fetch(from, st.x0, st.y0, st.n0, st.d0);
  for (int r0 = from; r0 < rows; r0 += 2 * kTile) {
    one(r0, st.x0, st.y0, st.n0, st.d0, st.x1, st.y1, st.n1, st.d1);
    if (r0 + kTile < rows) one(r0 + kTile, st.x1, st.y1, st.n1, st.d1, st.x0, st.y0, st.n0, st.d0);
  }
  if constexpr (SETS == 2) {
    if (__syncthreads_or(not_finite(sum)))
      return by_halves(c0, [&](int first) { keys_role<IN, DP, DK, 1>(again(a), found, first, kh, st); });
  }
#pragma unroll
  for (int j = 0; j < SETS; ++j) {
    const int key = w0 + 16 * j + col;
    if (key >= s.m) {  // (the room of a cache)
#pragma unroll
      for (int d = 0; d < T::DB; ++d) sum[j][d] = f32x4{};
    }
    if (key < k_end - k_first)
      store_rows<IN, DP>(sum[j], DK ? a.scale : 1.0f / (1 << kRaised<IN>), DK ? a.dk : a.dv, ((int64_t)(k_first + key) * a.k_heads + kh) * a.dim, a.dim);
  }
}

// Workgroups: the tiles of keys, 8 for dk and the same 8 for dv in turn, which then read the same
// rows at the same time, and the tiles of rows for dq; a sequence's tiles in descending order of work.
// (All of dk, then dq, then all of dv: 2380 us instead of 1981 for 8192 tokens of 8 key heads and 32
// query heads of 128, 453 instead of 390 for 5 sequences of 183 to 3544 tokens, 16 query heads.)
constexpr int kTurn = 8;
template <int IN, int DP, int SETS>
__global__ __launch_bounds__(kThreads, 2) void attention_backward_kernel(AttnArgs a) {
  constexpr int BYTES = kTile * TileOf<DP>::PITCH;
  __shared__ __attribute__((aligned(1024))) char x0[BYTES], y0[BYTES], x1[BYTES], y1[BYTES];
  __shared__ __attribute__((aligned(256))) float n0[kTile], d0[kTile], n1[kTile], d1[kTile];
  const Stages<DP> st{x0, y0, x1, y1, n0, d0, n1, d1};
  const int kh = blockIdx.x % (unsigned)a.k_heads;
  int tile = blockIdx.x / (unsigned)a.k_heads;
  const int turns = a.k_turns * 2 * kTurn;
  if (tile >= turns) {
    const FoundTile f = tile_of_rows<kBlock<SETS>>(a, (int)a.q_tiles - 1 - (tile - turns));
    return rows_role<IN, DP, SETS>(a, f.found.s, f.first, kh, st);
  }
  const bool dk = tile / kTurn % 2 == 0;
  tile = tile / (2 * kTurn) * kTurn + tile % kTurn;
  if (tile >= a.k_tiles) return;
  const FoundTile f = tile_of_keys<kBlock<SETS>>(a, tile);
  if (dk) keys_role<IN, DP, true, SETS>(a, f.found, f.first, kh, st);
  else keys_role<IN, DP, false, SETS>(a, f.found, f.first, kh, st);
}

// Up to three workgroups of 128 rows or keys a compute unit, the longest chain of steps is what
// the call takes: waves then take 16 rows or keys instead of 32 (8 key heads of 128: 2000 tokens
// with 4 query heads each, 770 workgroups, 266 -> 205 us; 900 with 2 each, 250 workgroups, 67 ->
// 51; 3544 with 2 each, 900 workgroups, 252 -> 259).  The bits are the same.
constexpr int64_t kSmallGroups = 800;

template <int IN, int DP, int SETS>
void launch_roles(AttnArgs a, hipStream_t s) {
  a.q_tiles = a.q_rows > 0 ? a.q_rows * a.group / kBlock<SETS> + a.batch + 2 : 0;
  a.k_tiles = a.k_rows > 0 ? a.k_rows / kBlock<SETS> + a.batch + 2 : 0;
  a.k_turns = (int)((a.k_tiles + kTurn - 1) / kTurn);
  const int64_t grid = (a.q_tiles + 2 * kTurn * a.k_turns) * a.k_heads;
  hipLaunchKernelGGL((attention_backward_kernel<IN, DP, SETS>), dim3((unsigned)grid), dim3(kThreads), 0, s, a);
}

template <int IN, int DP>
hipError_t launch_in(AttnArgs a, hipStream_t s) {
  if (a.q_rows > 0) {
    hipLaunchKernelGGL(attention_delta_kernel<IN>, grid_of((a.q_rows * a.q_heads + 15) / 16), dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t groups = (a.q_rows * a.group / kBlock<2> + 2 * (a.k_rows / kBlock<2>) + 3 * a.batch) * a.k_heads;
  if (groups <= kSmallGroups) launch_roles<IN, DP, 1>(a, s);
  else launch_roles<IN, DP, 2>(a, s);
  return hipGetLastError();
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
