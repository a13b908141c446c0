// Attention over packed sequences and caches:
//   o_i = sum_j p_ij v_j, p_ij = e^(scale q_i k_j) / sum_j e^(scale q_i k_j),
// over the keys j that query i sees; lse_i = ln of that sum.
//
// A row's bits are a function of its query and the keys and values it sees, in
// their order, alone: they do not depend on how many queries the call holds, on the other
// sequences, on the room behind a cache or on which kernel runs.  A prompt
// taken at once, in pieces or token by token gives the same bits.  For that, every
// kernel sums in one order.  Keys are cut from the sequence's first one on into chunks of 256
// and steps of 64.  Within a chunk a reference of the logits, the sums and the output go from
// step to step (each step: S on the matrix cores, p about the reference, p rounded to the
// input's type, two steps of 32 keys into the output's chain); a chunk's results start anew,
// and chunks are joined in ascending order by fp32 products and one fma.  So chunks can be
// worked on by workgroups of their own (few rows) or one after the other (many rows).
//
// Rounding.  p is rounded to 16 bits for the product with v, and o is divided by the sum of
// the rounded p, in fp32: the weights then add up to 1, and where one key has most of the weight
// its rounding drops out of o (packed bf16 tokens: o is off by 0.0019 of itself, with the sum of
// the unrounded p by 0.0020, in the same time; about the exact maximum by 0.0017, but 6 %
// slower.  Its own rounding makes 0.0017).
// lse is of the unrounded sum, in fp32 too.
//
// Values that are not finite.  In the products they would reach rows that do not see them (0
// times infinity), and be NaN in the rows that see them with a probability that rounds to 0, as
// in any row whose factors later fall to 0.  So the sums are of the finite values, and the row's
// others are added to the quotient at the end: o is infinite or NaN where the row
// sees such a value, whatever its weight.  Only calls that hold some pay for it.
#include "attention_common.h"

namespace imm {
namespace {
using namespace dev;

// ---- Many rows -----------------------------------------------------------------
// A workgroup takes 128 rows of a key head, 32 a wave (or 64, 16 a wave: SETS sets of 16), and
// walks through their keys 64 at a time: the next step's keys and values go by DMA into the
// other half of a two-stage LDS buffer while this one's are used.  Two workgroups share a compute
// unit, so that one's exponentials run beside the other's products: 16384 causal tokens, 32
// query and 8 key heads of 128 in bf16, take 2040 to 2150 us (1020 to 1080 TFLOP/s; matrix units busy 46 %,
// vector units, with exponentials and packing, 50 %, waves waiting 21 %), of 64 1180 to 1240 (41 %, 72 % and 19 %).  With one workgroup of 8 waves a unit that took
// 2407, with every new maximum as the reference 2240, with a step's first values read
// after the softmax 2156.

template <int IN>
__device__ __forceinline__ bool not_finite(unsigned two) {
  constexpr unsigned E = IN == GEMM_F16 ? 0x7c00u : 0x7f80u;
  return (two & E) == E || (two & (E << 16)) == (E << 16);
}
// ... and zeros in the place of values that are not finite.
template <int IN>
__device__ __forceinline__ u32x4 only_finite(u32x4 v) {
  constexpr unsigned E = IN == GEMM_F16 ? 0x7c00u : 0x7f80u;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if ((v[e] & E) == E) v[e] &= 0xffff0000u;
    if ((v[e] & (E << 16)) == (E << 16)) v[e] &= 0xffffu;
  }
  return v;
}

// x + value R of a pair if that is not finite, otherwise x as it is.
template <int IN, int R>
__device__ __forceinline__ float plus_not_finite(float x, unsigned two) {
  constexpr unsigned E = IN == GEMM_F16 ? 0x7c00u : 0x7f80u;
  const unsigned bits = R ? two >> 16 : two & 0xffffu;
  // (infinity or NaN in fp32: an fp16 fraction moves up with its sign)
  const unsigned wide = IN == GEMM_F16 ? (bits & 0x8000u) << 16 | 0x7f800000u | (bits & 0x3ffu) << 13 : bits << 16;
  return (bits & E) == E ? x + __uint_as_float(wide) : x;
}

// The rows of a wave through one step.
template <int IN, int DP, bool SAVE, int SETS>
struct WaveRows {
  using T = TileOf<DP>;
  i32x4 q[SETS][T::KS];
  f32x4 O[SETS][T::DB], o[SETS][T::DB];  // of the chunks so far, of this chunk
  float M[SETS], L[SETS], E[SETS], m[SETS], l[SETS], e[SETS];  // references and sums (E, e: with SAVE)
  int seen[SETS];  // keys of this lane's rows
  Lanes<DP> at;
  float scale_log2;

  __device__ __forceinline__ void clear_all() {
#pragma unroll
    for (int i = 0; i < SETS; ++i) {
      M[i] = kNegInf;
      L[i] = E[i] = 0.0f;
#pragma unroll
      for (int d = 0; d < T::DB; ++d) O[i][d] = f32x4{};
    }
  }
  // FIRST: the first step of a chunk.  masked: some row of the wave does not see all of the
  // step's keys.
  template <bool FIRST>
  __device__ __forceinline__ void step(const char* kt, const char* vt, int k0, bool masked) {
    const int quad = (threadIdx.x & 63) / 16;
    at.again();
    f32x4 sc[SETS][4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
#pragma unroll
      for (int i = 0; i < SETS; ++i) sc[i][b] = f32x4{};
#pragma unroll
      for (int ks = 0; ks < T::KS; ++ks) {
        const i32x4 kf = row_fragment<DP>(kt, at, b, ks);
#pragma unroll
        for (int i = 0; i < SETS; ++i) sc[i][b] = mfma16_v<IN>(kf, q[i][ks], sc[i][b]);
      }
    }
    if (masked) {
#pragma unroll
      for (int i = 0; i < SETS; ++i)
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (k0 + 16 * b + 4 * quad + r >= seen[i]) sc[i][b][r] = kNegInf;
    }
    constexpr int PRE = 3;
    i32x4 pre[PRE];
#pragma unroll
    for (int d = 0; d < PRE; ++d) pre[d] = column_fragment<DP>(vt, at, 0, d);
    i32x4 pf[SETS][2];
#pragma unroll
    for (int i = 0; i < SETS; ++i) {
      const float top = lane_max(sc[i]) * scale_log2;
      if constexpr (FIRST) {
        m[i] = reference(kNegInf, row_max(top));
        l[i] = e[i] = 0.0f;
      } else {
        // (no lane has a logit that sets the reference of its row again: nothing changes)
        if (__any(reference(m[i], top) != m[i])) {
          const float to = reference(m[i], row_max(top));
          const float f = shrink(m[i], to);
          m[i] = to;
          l[i] *= f;
          if (SAVE) e[i] *= f;
#pragma unroll
          for (int d = 0; d < T::DB; ++d) o[i][d] *= f;
        }
      }
      probabilities(sc[i], scale_log2, m[i]);
      if (SAVE) e[i] += sum_of(sc[i]);
      pf[i][0] = pack_blocks<IN>(sc[i][0], sc[i][1]);
      pf[i][1] = pack_blocks<IN>(sc[i][2], sc[i][3]);
      l[i] = add_pairs<IN>(pf[i][1], add_pairs<IN>(pf[i][0], l[i]));
    }
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int d = 0; d < T::DB; ++d) {
        const i32x4 vf = p == 0 && d < PRE ? pre[d < PRE ? d : 0] : column_fragment<DP>(vt, at, p, d);
#pragma unroll
        for (int i = 0; i < SETS; ++i) o[i][d] = mfma16_v<IN>(vf, pf[i][p], FIRST && p == 0 ? f32x4{} : o[i][d]);
      }
  }
  // O + the values of a step that are not finite, for the rows that see them.
  __device__ __forceinline__ void add_not_finite(const char* v, int64_t v_bytes, int k0, int end, int dim) {
    const int quad = (threadIdx.x & 63) / 16;
    for (int j = k0; j < k0 + kTile && j < end; ++j) {
#pragma unroll
      for (int d = 0; d < T::DB; ++d) {
        const int c = 16 * d + 4 * quad;
        i32x2 x{};
        if (c < dim) x = *reinterpret_cast<const i32x2*>(v + j * v_bytes + 2 * c);
#pragma unroll
        for (int i = 0; i < SETS; ++i)
          if (j < seen[i]) {
            O[i][d][0] = plus_not_finite<IN, 0>(O[i][d][0], x[0]);
            O[i][d][1] = plus_not_finite<IN, 1>(O[i][d][1], x[0]);
            O[i][d][2] = plus_not_finite<IN, 0>(O[i][d][2], x[1]);
            O[i][d][3] = plus_not_finite<IN, 1>(O[i][d][3], x[1]);
          }
      }
    }
  }
  // The end of the chunk that begins at c0.
  __device__ __forceinline__ void join(int c0) {
#pragma unroll
    for (int i = 0; i < SETS; ++i) {
      // (a chunk that the row does not see leaves it as it is, to the sign of a zero)
      if (c0 < seen[i]) {
        const Join j = join_chunk(M[i], m[i]);
        M[i] = j.m;
        L[i] = joined(L[i], row_sum(l[i]), j);
        if (SAVE) E[i] = joined(E[i], row_sum(e[i]), j);
        // (a product with 1 changes nothing)
        if (__any(j.a != 1.0f)) {
#pragma unroll
          for (int d = 0; d < T::DB; ++d) O[i][d] *= j.a;
        }
#pragma unroll
        for (int d = 0; d < T::DB; ++d)
#pragma unroll
          for (int r = 0; r < 4; ++r) O[i][d][r] = fmaf(o[i][d][r], j.b, O[i][d][r]);
      }
    }
  }
};

// SAVE: lse and what o's rounding left too, for the backward pass.
template <int IN, int DP, bool SAVE, int SETS>
__global__ __launch_bounds__(kThreads, 2) void attention_kernel(AttnArgs a) {
  constexpr int kRows = 16 * SETS * kWaves;
  using T = TileOf<DP>;
  // (arrays of their own: the compiler then knows that a transfer into one stage does not
  // touch the other, and lets the reads of that go on)
  __shared__ __attribute__((aligned(1024))) char k_a[kTile * T::PITCH], v_a[kTile * T::PITCH];
  __shared__ __attribute__((aligned(1024))) char k_b[kTile * T::PITCH], v_b[kTile * T::PITCH];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int quad = lane / 16, col = lane % 16;
  // heads vary fastest: neighbouring workgroups go to different XCDs, so a key
  // head's workgroups meet in few of the L2s.  The last rows (the most keys) first.
  const int tiles = gridDim.x / (unsigned)a.k_heads;
  const int kh = blockIdx.x % (unsigned)a.k_heads;
  const int tile = blockIdx.x / (unsigned)a.k_heads;
  const FoundTile f = a.sorted ? longest_first<kRows>(a, tile) : tile_of_rows<kRows>(a, tiles - 1 - tile);
  const Found found = f.found;
  const Sequence s = found.s;
  const int r0 = f.first;
  const int rows = s.n * a.group;
  if (r0 >= rows) return;

  // this lane's rows: column `col` of the two blocks of 16 of its wave
  const int w0 = r0 + 16 * SETS * wave;
  WaveRows<IN, DP, SAVE, SETS> w;
  w.scale_log2 = a.scale_log2;
#pragma unroll
  for (int i = 0; i < SETS; ++i) {
    const int row = w0 + 16 * i + col, t = row / a.group;
    const int h = row - t * a.group;
    w.seen[i] = keys_seen(a, s, t);
    const char* const q = static_cast<const char*>(a.q) + 2 * ((s.q0 + t) * a.q_token + (kh * a.group + h) * a.q_head);
#pragma unroll
    for (int ks = 0; ks < T::KS; ++ks) {
      const int d = 32 * ks + 8 * quad;
      w.q[i][ks] = i32x4{};
      if (row < rows && d < a.dim) w.q[i][ks] = *reinterpret_cast<const i32x4*>(q + 2 * d);
    }
  }
  // keys that any row of the workgroup, and of the wave, sees, and those that all of the
  // wave's see (rows past the end see none, which needs no mask)
  auto seen_of = [&](int r) { return keys_seen(a, s, (r < rows ? r : rows - 1) / a.group); };
  const int need = __builtin_amdgcn_readfirstlane(seen_of(r0 + kRows - 1));
  const int wave_need = __builtin_amdgcn_readfirstlane(w0 < rows ? seen_of(w0 + 16 * SETS - 1) : 0);
  const int wave_all = __builtin_amdgcn_readfirstlane(w0 < rows ? seen_of(w0) : 0);

  const int64_t k_bytes = 2 * a.k_token, v_bytes = 2 * a.v_token;
  const char* const kp = static_cast<const char*>(a.k) + 2 * (s.k0 * a.k_token + kh * a.k_head);
  const char* const vp = static_cast<const char*>(a.v) + 2 * (s.k0 * a.v_token + kh * a.v_head);
  const Mover<DP> km(k_bytes, a.dim), vm(v_bytes, a.dim);
  auto fetch = [&](int k0, char* kt, char* vt) {
    km.move(kp + k0 * k_bytes, kt, s.m - k0, k_bytes, a.dim);
    vm.move(vp + k0 * v_bytes, vt, s.m - k0, v_bytes, a.dim);
  };
  // Zeros in the place of a tile's values that are not finite.
  auto clean = [&](char* vt) {
    u32x4* const mine = reinterpret_cast<u32x4*>(vt) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < Mover<DP>::N; ++i) mine[i * kThreads] = only_finite<IN>(mine[i * kThreads]);
    __syncthreads();
  };
  bool careful = false;
  auto one = [&](auto first, int k0, char* kt, char* vt, char* next_k, char* next_v) {
    landed();  // this step's tiles are there, and the other stage has been read
    if (k0 + kTile < need) fetch(k0 + kTile, next_k, next_v);
    if (careful) clean(vt);
    if (k0 < wave_need) w.template step<decltype(first)::value>(kt, vt, k0, k0 + kTile > wave_all);
  };
  const std::true_type first;
  const std::false_type further;
  for (;;) {
    w.clear_all();
    if (need > 0) fetch(0, k_a, v_a);
    for (int c0 = 0; c0 < need; c0 += kAttnChunk) {
      one(first, c0, k_a, v_a, k_b, v_b);
      for (int k0 = c0 + kTile; k0 < c0 + kAttnChunk && k0 < need; k0 += 2 * kTile) {
        one(further, k0, k_b, v_b, k_a, v_a);
        if (k0 + kTile < c0 + kAttnChunk && k0 + kTile < need) one(further, k0 + kTile, k_a, v_a, k_b, v_b);
      }
      if (c0 < wave_need) w.join(c0);
    }
    // A value that is not finite, seen or not, has left a result that is not finite in every row whose
    // steps held it; if there are such, all steps once more without those values.  (The
    // barrier is also the one before the stages are filled again.)
    bool bad = false;
#pragma unroll
    for (int i = 0; i < SETS; ++i)
#pragma unroll
      for (int d = 0; d < T::DB; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) bad |= !(fabsf(w.O[i][d][r]) < __builtin_inff());
    if (careful || !__syncthreads_or(bad)) break;
    careful = true;
  }

  // (rows that are past the call's are not stored)
#pragma unroll
  for (int i = 0; i < SETS; ++i) {
    const int t = (w0 + 16 * i + col) / a.group;
    // a row without keys is zero; one whose keys are all -infinity is 0 / 0; and NaN is what a
    // sequence longer than the call said has past that, here as in the kernel of few rows
    const bool unsaid = t >= a.max_q && found.segment >= 1 && found.segment <= a.batch;
    if (unsaid) w.L[i] = w.E[i] = __builtin_nanf("");
    const float inv = w.seen[i] == 0 && !unsaid ? 0.0f : 1.0f / w.L[i];
    if (unsaid) w.seen[i] = 1;
#pragma unroll
    for (int d = 0; d < T::DB; ++d) w.O[i][d] *= inv;
  }
  if (careful) {
    for (int k0 = 0; k0 < need; k0 += kTile) {
      bool bad = false;
#pragma unroll
      for (int i = 0; i < Mover<DP>::N; ++i) {
        const int at = threadIdx.x + i * kThreads, key = k0 + at / T::SLOTS, c = at % T::SLOTS * 8;
        if (key >= s.m || c >= a.dim) continue;
        const u32x4 v = *reinterpret_cast<const u32x4*>(vp + key * v_bytes + 2 * c);
#pragma unroll
        for (int e = 0; e < 4; ++e) bad |= not_finite<IN>(v[e]);
      }
      if (__syncthreads_or(bad) && k0 < wave_need) w.add_not_finite(vp, v_bytes, k0, s.m, a.dim);
    }
  }
#pragma unroll
  for (int i = 0; i < SETS; ++i) {
    const int row = w0 + 16 * i + col;
    if (row >= rows) continue;
    const int t = row / a.group;
    const int64_t at = (s.q0 + t) * a.q_heads + kh * a.group + (row - t * a.group);
#pragma unroll
    for (int d = 0; d < T::DB; ++d) {
      const int c = 16 * d + 4 * quad;
      if (c >= a.dim) continue;
      const f32x4 x = w.O[i][d];
      const i32x2 y{pack2<IN>(x[0], x[1]), pack2<IN>(x[2], x[3])};
      const int64_t to = 2 * (at * a.dim + c);
      *reinterpret_cast<i32x2*>(static_cast<char*>(a.o) + to) = y;
      if (SAVE && a.o_low)
        *reinterpret_cast<i32x2*>(static_cast<char*>(a.o_low) + to) =
            i32x2{pack2_rest<IN>(x[0], x[1], y[0]), pack2_rest<IN>(x[2], x[3], y[1])};
    }
    if (SAVE && a.lse && quad == 0)
      a.lse[at] = w.seen[i] == 0 ? kNegInf : (w.M[i] + __builtin_amdgcn_logf(w.E[i])) * kLn2;
  }
}

// ---- Few rows ------------------------------------------------------------------
// A workgroup takes one chunk of 256 keys of one key head, all of whose bytes it asks for
// at once: the keys as fragments in registers (each of the four waves its step of 64), the
// values through registers to LDS.  Each wave makes its step's logits and their
// maximum; with the maxima of the steps before, which LDS holds, every wave has the
// reference that one wave alone would have had, so the probabilities are
// those of the chain; then each wave takes a quarter of the output's dimensions through
// all four steps.
// Memory bounds it where there are many chunks (61 caches of up to 8192 keys, 32 query and 4
// key heads of 128: 125 us, 4.4 TB/s, and the join 8), latency where there are few (8192 keys
// of 8 heads: 12 us and the join 6, most of them launches and trips to memory).  The launch has a workgroup
// for every 256 rows of room: 61 caches of 900 to 1000 keys take 29 us in 1024 rows of room each, 40 in 8192, 122 in 65536.
constexpr int kFewWaves = 4, kFewThreads = 64 * kFewWaves;

template <int IN, int DP>
__global__ __launch_bounds__(kFewThreads, 2) void attention_few_kernel(AttnArgs a) {
  using T = TileOf<DP>;
  __shared__ __attribute__((aligned(16))) char vt[kFewWaves][kTile * T::PITCH];
  // (with a second set of these, and a barrier less, two workgroups would not fit into the LDS)
  __shared__ i32x4 pl[kFewWaves][2][64];
  __shared__ float ml[kFewWaves][16], se[kFewWaves][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int quad = lane / 16, col = lane % 16;
  const int kh = blockIdx.x % (unsigned)a.k_heads;
  const int slot = blockIdx.x / (unsigned)a.k_heads;
  const FoundTile chunk = chunk_of_slot(a, slot);
  const Sequence s = chunk.found.s;
  const int c0 = chunk.first;
  if (c0 >= s.m || s.n == 0) return;  // (a segment that is no sequence has no keys)
  const int queries = s.n < a.max_q ? s.n : (int)a.max_q;
  if (c0 >= keys_seen(a, s, queries - 1)) return;
  const int left = s.m - c0 < kAttnChunk ? s.m - c0 : kAttnChunk;

  const auto kb = buffer_at(static_cast<const char*>(a.k) + 2 * ((s.k0 + c0) * a.k_token + kh * a.k_head));
  const auto vb = buffer_at(static_cast<const char*>(a.v) + 2 * ((s.k0 + c0) * a.v_token + kh * a.v_head));
  const int rows = queries * a.group;
  i32x4 kf[4][T::KS], qf[T::KS];
  auto load_rows = [&](int r0) {
    const int row = r0 + col, t = row / a.group, h = row - t * a.group;
    const char* const q = static_cast<const char*>(a.q) + 2 * ((s.q0 + t) * a.q_token + (kh * a.group + h) * a.q_head);
#pragma unroll
    for (int ks = 0; ks < T::KS; ++ks) {
      const int d = 32 * ks + 8 * quad;
      qf[ks] = i32x4{};
      if (row < rows && d < a.dim) qf[ks] = *reinterpret_cast<const i32x4*>(q + 2 * d);
    }
  };
  load_rows(0);
#pragma unroll
  for (int b = 0; b < 4; ++b)
#pragma unroll
    for (int ks = 0; ks < T::KS; ++ks) {
      const int key = 64 * wave + 16 * b + col, d = 32 * ks + 8 * quad;
      kf[b][ks] = __builtin_bit_cast(
          i32x4, load_b128(kb, key < left && d < a.dim ? (unsigned)(key * (int)(2 * a.k_token) + 2 * d) : OOB));
    }
  constexpr int NV = kAttnChunk * T::SLOTS / kFewThreads;
  u32x4 vv[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = threadIdx.x + i * kFewThreads, key = at / T::SLOTS, c = at % T::SLOTS;
    vv[i] = load_b128(vb, key < left && c * 8 < a.dim ? (unsigned)(key * (int)(2 * a.v_token) + c * 16) : OOB);
  }
  bool bad = false;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = threadIdx.x + i * kFewThreads, key = at / T::SLOTS, c = at % T::SLOTS;
    *reinterpret_cast<u32x4*>(&vt[key / kTile][T::at(key % kTile, c)]) = vv[i];
#pragma unroll
    for (int e = 0; e < 4; ++e) bad |= not_finite<IN>(vv[i][e]);
  }
  // values that are not finite are taken out of the chunk, and told of: the join adds them
  const bool told = __syncthreads_or(bad);
  if (told) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = threadIdx.x + i * kFewThreads, key = at / T::SLOTS, c = at % T::SLOTS;
      *reinterpret_cast<u32x4*>(&vt[key / kTile][T::at(key % kTile, c)]) = only_finite<IN>(vv[i]);
    }
    __syncthreads();
  }

  const Lanes<DP> lanes;
  for (int r0 = 0; r0 < rows; r0 += 16) {
    const int row = r0 + col, t = row / a.group;
    const int seen = clamped((row < rows ? keys_seen(a, s, t) : 0) - c0, 0, kAttnChunk);
    f32x4 sc[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      sc[b] = f32x4{};
#pragma unroll
      for (int ks = 0; ks < T::KS; ++ks) sc[b] = mfma16_v<IN>(kf[b][ks], qf[ks], sc[b]);
    }
    if (r0 + 16 < rows) load_rows(r0 + 16);
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (64 * wave + 16 * b + 4 * quad + r >= seen) sc[b][r] = kNegInf;
    const float mine = row_max(lane_max(sc)) * a.scale_log2;
    if (quad == 0) ml[wave][col] = mine;
    __syncthreads();
    float m[kFewWaves];
    m[0] = reference(kNegInf, ml[0][col]);
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) m[w] = reference(m[w - 1], ml[w][col]);
    const float about = wave == 0 ? m[0] : wave == 1 ? m[1] : wave == 2 ? m[2] : m[3];
    probabilities(sc, a.scale_log2, about);
    se[wave][lane] = sum_of(sc);
    pl[wave][0][lane] = pack_blocks<IN>(sc[0], sc[1]);
    pl[wave][1][lane] = pack_blocks<IN>(sc[2], sc[3]);
    __syncthreads();
    f32x4 o[(T::DB + kFewWaves - 1) / kFewWaves];
#pragma unroll
    for (auto& x : o) x = f32x4{};
    float l = 0.0f, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) {
      const float f = w == 0 ? shrink(kNegInf, m[0]) : shrink(m[w - 1], m[w]);
      l *= f;
      sum = sum * f + se[w][lane];
#pragma unroll
      for (int p = 0; p < 2; ++p) l = add_pairs<IN>(pl[w][p][lane], l);
#pragma unroll
      for (int i = 0; i < (T::DB + kFewWaves - 1) / kFewWaves; ++i) {
        const int d = kFewWaves * i + wave;
        if (d < T::DB) {
          o[i] *= f;
#pragma unroll
          for (int p = 0; p < 2; ++p) o[i] = mfma16_v<IN>(column_fragment<DP>(vt[w], lanes, p, d), pl[w][p][lane], o[i]);
        }
      }
    }
    l = row_sum(l);
    sum = row_sum(sum);
    const int64_t at = ((int64_t)slot * a.k_heads + kh) * a.part_rows + row;
    if (row < rows) {
      if (wave == 0 && quad == 0) {
        reinterpret_cast<f32x4*>(a.part_ml)[at] = f32x4{m[kFewWaves - 1], l, sum, told ? 1.0f : 0.0f};
      }
#pragma unroll
      for (int i = 0; i < (T::DB + kFewWaves - 1) / kFewWaves; ++i) {
        const int d = 16 * (kFewWaves * i + wave) + 4 * quad;
        if (d < a.dim && d < DP) *reinterpret_cast<f32x4*>(a.part_o + at * a.dim + d) = o[i];
      }
    }
    __syncthreads();  // before the next rows use ml, se and pl
  }
}

// The chunks of a row, joined in ascending order: a wave per query and head, two
// dimensions a lane.  Latency bounds it, that of the code too (each of its lines is
// fetched for one pass): the references and factors of 64 chunks are made by a lane
// each, and two groups of 8 chunks' results are in flight in a short loop.
template <int IN>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a) {
  constexpr int U = 8;
  const int lane = threadIdx.x & 63;
  const unsigned at = (blockIdx.y * gridDim.x + blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  if (at >= (unsigned)a.q_rows * a.q_heads) return;
  const int q = at / (unsigned)a.q_heads, head = at - q * a.q_heads;
  const int kh = head / (unsigned)a.group;
  const Found found = segment_of_query(a, q);
  const Sequence s = found.s;
  const int t = q - s.q0;
  const bool said = t < a.max_q || found.segment == 0 || found.segment > a.batch;  // (rows in no sequence have no keys)
  const int seen = keys_seen(a, s, t);
  float M = kNegInf, L = 0.0f, E = 0.0f, O0 = 0.0f, O1 = 0.0f;
  const bool mine = 2 * lane < a.dim;
  const int64_t step = (int64_t)a.k_heads * a.part_rows;
  bool told = false;  // of values that are not finite
  if (said && seen > 0) {
    const int64_t first = (int64_t)first_slot(found) * step + kh * a.part_rows + t * a.group + (head - kh * a.group);
    const int chunks = (seen + kAttnChunk - 1) / kAttnChunk;
    const f32x4* ml_at = reinterpret_cast<const f32x4*>(a.part_ml) + first + lane * step;
    const char* o_at = reinterpret_cast<const char*>(a.part_o + first * a.dim + 2 * lane);
    const int64_t o_step = step * a.dim * 4;
    // (rows past the last chunk are loaded as the last once more)
    float2 o[U], next[U];
    int asked = 0;
    auto load = [&](float2(&to)[U]) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (mine) to[u] = *reinterpret_cast<const float2*>(o_at);
        o_at += ++asked < chunks ? o_step : 0;
      }
    };
    load(next);
    for (int c0 = 0; c0 < chunks; c0 += 64) {
      const int n = chunks - c0 < 64 ? chunks - c0 : 64;
      f32x4 ml{kNegInf, 0.0f, 0.0f, 0.0f};
      if (lane < n) ml = *ml_at;
      ml_at += 64 * step;
      told |= __any(ml[3] != 0.0f);
      // the reference after each chunk: it is set again at few of them
      float before = M, after = M;
      for (int from = 0;;) {
        const uint64_t set = __ballot(lane >= from && reference(M, ml[0]) != M);
        if (!set) break;
        const int l = __ffsll((unsigned long long)set) - 1;
        const float to = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ml[0]), l));
        if (lane > l) before = to;
        if (lane >= l) after = to;
        M = to;
        from = l + 1;
      }
      const float fa = shrink(before, after);
      const float fb = ml[0] == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(ml[0] - after);
      const bool ones = __all(fa == 1.0f);
      for (int u0 = 0; u0 < n; u0 += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) o[u] = next[u];
        if (c0 + u0 + U < chunks) load(next);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float b = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(fb), u0 + u));
          const float l = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ml[1]), u0 + u));
          const float e = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ml[2]), u0 + u));
          if (!ones) {  // (a product with 1 changes nothing)
            const float f = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(fa), u0 + u));
            L *= f;
            E *= f;
            O0 *= f;
            O1 *= f;
          }
          if (u0 + u < n) {
            L = fmaf(l, b, L);
            E = fmaf(e, b, E);
            O0 = fmaf(o[u].x, b, O0);
            O1 = fmaf(o[u].y, b, O1);
          }
        }
      }
    }
  }
  if (!said) L = E = O0 = O1 = __builtin_nanf("");  // a sequence longer than the call said
  const bool empty = seen == 0 && said;
  const float inv = empty ? 0.0f : 1.0f / L;
  O0 *= inv;
  O1 *= inv;
  if (told && mine) {
    const float* ml = a.part_ml + 4 * ((int64_t)first_slot(found) * step + kh * a.part_rows + t * a.group + (head - kh * a.group));
    const char* v = static_cast<const char*>(a.v) + 2 * (s.k0 * a.v_token + kh * a.v_head) + 4 * lane;
    for (int c0 = 0; c0 < seen; c0 += kAttnChunk, ml += 4 * step) {
      if (ml[3] == 0.0f) continue;
      for (int j = c0; j < c0 + kAttnChunk && j < seen; ++j) {
        const unsigned two = *reinterpret_cast<const unsigned*>(v + 2 * j * a.v_token);
        O0 = plus_not_finite<IN, 0>(O0, two);
        O1 = plus_not_finite<IN, 1>(O1, two);
      }
    }
  }
  if (mine) {
    const int y = pack2<IN>(O0, O1);
    const int64_t to = (int64_t)at * a.dim / 2 + lane;
    static_cast<int*>(a.o)[to] = y;
    if (a.o_low) static_cast<int*>(a.o_low)[to] = pack2_rest<IN>(O0, O1, y);
  }
  if (a.lse && lane == 0) a.lse[at] = empty ? kNegInf : (M + __builtin_amdgcn_logf(E)) * kLn2;
}

// Workgroups of 128 rows.
int64_t groups_of(const AttnArgs& a) { return (a.q_rows * a.group / (32 * kWaves) + a.batch) * a.k_heads; }
// Up to two of them a compute unit, what one takes for its keys alone is what the call takes:
// waves then take 16 rows instead of 32, which halves a step's products and exponentials, not its reads
// (8 key heads of 128, 4 query heads each: 1000 tokens 30 -> 23 us, 2000 56 -> 54, but 4000, with
// 1024 workgroups, 155 -> 184).
constexpr int64_t kSmallGroups = 512;
// While they are few rounds of what the compute units hold, those with the most keys go first: 13
// sequences of 169 to 1340 tokens, 2 key heads of 64, 16 query heads, 38 -> 34 us; 5 of 183 to
// 3544, 8 key heads of 128, 142 -> 133.  (Equal sequences lose up to 2 us by it, and with
// 4096 workgroups it gives nothing.)
constexpr int64_t kSortedGroups = 2048;

template <int IN, int DP, int SETS>
void launch_rows(AttnArgs a, hipStream_t s) {
  const int64_t tiles = a.q_rows * a.group / (16 * SETS * kWaves) + a.batch + 2;
  a.sorted = a.batch > 1 && a.batch + 2 <= kSortedSegments && groups_of(a) <= kSortedGroups;
  const auto kernel = a.lse || a.o_low ? attention_kernel<IN, DP, true, SETS> : attention_kernel<IN, DP, false, SETS>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles * a.k_heads)), dim3(kThreads), 0, s, a);
}

template <int IN, int DP>
hipError_t launch_in(const AttnArgs& a, hipStream_t s) {
  if (a.part_o) {
    if (a.chunks > 0)
      hipLaunchKernelGGL((attention_few_kernel<IN, DP>), dim3((unsigned)(a.chunks * a.k_heads)),
                         dim3(kFewThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(attention_join_kernel<IN>, grid_of((a.q_rows * a.q_heads + 3) / 4), dim3(256), 0, s, a);
    return hipGetLastError();
  }
  if (groups_of(a) <= kSmallGroups) launch_rows<IN, DP, 1>(a, s);
  else launch_rows<IN, DP, 2>(a, s);
  return hipGetLastError();
}

template <int IN>
hipError_t launch_dim(const AttnArgs& a, hipStream_t s) {
  if (a.dim <= 64) return launch_in<IN, 64>(a, s);
  if (a.dim <= 96) return launch_in<IN, 96>(a, s);
  return launch_in<IN, 128>(a, s);
}

}  // namespace

// Which kernel takes a call (the bits are the same): the one with the least estimated time, in us,
// from what the host knows.  Both wait for memory and launch (6, or 8 with the join).  The kernel of
// many rows takes 1.02 for a step of 64 keys (0.6 up to 64 dimensions), and as much for each
// 256 workgroups where these fill the compute units; the kernel of few rows 3 for a chunk's
// keys and 1.3 (1.7 shared) for each 16 rows, and its results go to the caches and back at
// 6 TB/s.  Measured, few against many rows' kernel, bf16, 8 key heads of 128 with 4 query heads each:
//   1 sequence of 8192 keys, 32 queries 31 and 133, 100 queries 71 and 135, 500 queries 290 and 136;
//   4 of 16384 keys, 100 queries 273 and 265; 1 of 16384 keys, 300 queries 276 and 265;
//   4 of 4096 keys, 64 queries 59 and 71; 16 of 2048 keys, 100 queries 106 and 58.
bool attention_few_rows(const AttnArgs& a) {
  constexpr double kMostBytes = 512e6;  // of workspace
  const double rows = (double)a.max_q * a.group, keys = (double)a.k_rows / a.batch;
  const double slots = (double)attention_chunk_slots(a.k_rows, a.batch) * a.k_heads;
  const double bytes = slots * rows * (a.dim + 4) * 4;
  if (bytes > kMostBytes || slots >= 1 << 24 || a.k_rows == 0) return false;
  const double rounds = slots <= 512 ? 1 : slots / 512, tiles = (rows + 15) / 16;
  const double few = 8 + rounds * (3 + tiles * (slots <= 256 ? 1.3 : 1.7)) + 2 * bytes / 6e6;
  const double groups = (double)groups_of(a);
  const double step = a.dim <= 64 ? 0.6 : 1.02;
  const double many = 6 + (keys / kTile + 1) * step * (groups <= kSmallGroups ? 1 : groups / 256);
  return few < many;
}
int64_t attention_chunk_slots(int64_t k_rows, int batch) { return k_rows / kAttnChunk + batch; }

hipError_t launch_attention(int in, const AttnArgs& a, hipStream_t s) {
  return in == GEMM_F16 ? launch_dim<GEMM_F16>(a, s) : launch_dim<GEMM_BF16>(a, s);
}

}  // namespace imm
