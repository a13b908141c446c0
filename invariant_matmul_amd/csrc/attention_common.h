// Parts that the attention kernels share: tiles in LDS, matrix steps and the softmax of a
// step.  (Sequences: attention_sequences.h.)
//
// Layout.  The rows of a sequence that share a key head are one matrix: row
// r = t group + h is query t of the sequence and query head h of the key
// head's group.  All products run on the 16x16x32 step with the operand whose
// index stays in a lane as the second one: S^T = K Q^T leaves a lane the logits of
// one row (lane % 16) against keys 4 (lane / 16) + 0..3 of each block of 16, and
// these are, as they lie, the second operand of O^T = V^T P^T: the step sums over
// its 32 places in an order of its own, and its place 8 q + j stands for key
// 4 q + j of the first block of 16 (j < 4) or key 4 q + j - 4 of the second.
// The first operand, V^T, comes in the same order from a transposing LDS read.  So
// no probability ever moves between lanes, and the sum of a row's
// probabilities is a sum within four lanes.
#pragma once

#include "attention_sequences.h"
#include "buffer_access.h"
#include "decoder_internal.h"
#include "kernel_common.h"

// From here on a product and a sum are fused where the code says fmaf and nowhere else: the kernels
// that a call may be given to have to round alike.
#pragma clang fp contract(off)

namespace imm {
namespace dev {

constexpr int kTile = kAttnTile;
constexpr float kNegInf = -__builtin_inff();
constexpr float kLn2 = 0.693147180559945309417f;

// Workgroups in two axes: a launch holds fewer than 2^32 threads along one.  (Those past the last do nothing.)
inline dim3 grid_of(int64_t groups) {
  const int64_t x = groups < 1 << 20 ? groups : 1 << 20;
  return dim3((unsigned)x, (unsigned)((groups + x - 1) / x));
}

// 16 bytes of a buffer; zeros past its end.
__device__ __forceinline__ u32x4 load_b128(__amdgpu_buffer_rsrc_t buf, unsigned off) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(buf, off, 0, 0));
#else
  return u32x4{};
#endif
}

// A tile of rows in LDS: 16-byte slot c of row r lies at slot c ^ (r % SLOTS).  The 16
// rows of a fragment read are then on different banks.
template <int DP>
struct TileOf {
  static constexpr int SLOTS = DP <= 64 ? 8 : 16;
  static constexpr int PITCH = SLOTS * 16;
  static constexpr int KS = DP / 32;   // steps over the dimension
  static constexpr int DB = DP / 16;   // blocks of it
  __device__ __forceinline__ static int at(int row, int slot) {
    return row * PITCH + ((slot ^ (row & (SLOTS - 1))) * 16);
  }
};

// Workgroups of the kernels that walk through a sequence: four waves with 32 rows or keys
// each, two workgroups on a compute unit.
constexpr int kWaves = 4, kThreads = 64 * kWaves;

// Moves a tile of keys or values to LDS; what lies past its `left` rows or past the
// dimension is zeros.  A wave fills 1 KB at a time, lane l the 16 bytes at 16 l: each
// lane fetches what belongs in its fixed slot.  The workgroup's next rows have a buffer of
// their own, so that one offset serves all.
template <int DP>
struct Mover {
  static constexpr int N = kTile * TileOf<DP>::SLOTS / kThreads, ROWS = kThreads / TileOf<DP>::SLOTS;
  static_assert(ROWS % TileOf<DP>::SLOTS == 0, "the rows of a thread have the same slot");
  unsigned off;  // of the thread's first row
  __device__ __forceinline__ Mover(int64_t row_bytes, int dim) {
    const int row = threadIdx.x / TileOf<DP>::SLOTS;
    const int slot = (threadIdx.x % TileOf<DP>::SLOTS) ^ (row & (TileOf<DP>::SLOTS - 1));
    off = slot * 8 < dim ? (unsigned)(row * (int)row_bytes + slot * 16) : OOB;
  }
  __device__ __forceinline__ void move(const char* from, char* to, int64_t left, int64_t row_bytes, int dim) const {
    // (rows behind the last: past the buffer's end, or, where rows overlap, values that no row sees)
    const int rows = (int)(left < kTile ? left : kTile);
    char* const mine = to + __builtin_amdgcn_readfirstlane(threadIdx.x & ~63) * 16;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int last = rows - 1 - i * ROWS;
      const auto buf = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(from) + i * ROWS * row_bytes, 0,
                                                         last < 0 ? 0 : last * (int)row_bytes + 2 * dim, 0x00020000);
      dma16(buf, mine + i * kThreads * 16, off, 0);
    }
  }
};

// This wave's transfers have landed, and everyone's; and everyone has read what it read before.
__device__ __forceinline__ void landed() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
}

// Where a lane's pieces of a tile lie.  Slots are XORed, so a piece's place is that of the
// first one XOR a constant: `again` keeps the compiler from holding all of them in
// registers over a loop.
template <int DP>
struct Lanes {
  unsigned row, column;
  __device__ __forceinline__ Lanes() {
    const int l = threadIdx.x & 63, r = 4 * (l / 16) + (l % 16) / 4;
    row = TileOf<DP>::at(l % 16, l / 16);
    column = TileOf<DP>::at(r, (l % 4) / 2) + (l % 2) * 8;
  }
  __device__ __forceinline__ void again() { asm volatile("" : "+v"(row), "+v"(column)); }
};

// Rows 16 b + lane % 16 of a tile, dimensions 32 ks + 8 (lane / 16) .. + 7.
template <int DP>
__device__ __forceinline__ i32x4 row_fragment(const char* tile, const Lanes<DP>& at, int b, int ks) {
  return *reinterpret_cast<const i32x4*>(tile + (at.row ^ (64 * ks)) + 16 * TileOf<DP>::PITCH * b);
}

// The transposed piece: dimension 16 db + lane % 16 of the rows 4 q + 0..3 of the
// blocks 2 s and 2 s + 1 of 16 rows, q = lane / 16.
template <int DP>
__device__ __forceinline__ i32x4 column_fragment(const char* tile, const Lanes<DP>& at, int s, int db) {
  i32x4 r{};
#if defined(__HIP_DEVICE_COMPILE__)
  typedef short v4i16 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) v4i16 lds_v4;
  const char* const p = tile + (at.column ^ (32 * db)) + 32 * TileOf<DP>::PITCH * s;
  const i32x2 lo = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4*)p));
  const i32x2 hi = __builtin_bit_cast(
      i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4*)(p + 16 * TileOf<DP>::PITCH)));
  r = i32x4{lo[0], lo[1], hi[0], hi[1]};
#endif
  return r;
}

template <int IN>
__device__ __forceinline__ int pack2(float a, float b) {
  if constexpr (IN == GEMM_F16) {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(int, f16x2{(_Float16)a, (_Float16)b});
  } else {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(int, bf16x2{(__bf16)a, (__bf16)b});
  }
}
// What rounding to IN left of a pair, rounded to IN.
template <int IN>
__device__ __forceinline__ int pack2_rest(float a, float b, int rounded) {
  if constexpr (IN == GEMM_F16) {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    const f16x2 r = __builtin_bit_cast(f16x2, rounded);
    return pack2<IN>(a - (float)r[0], b - (float)r[1]);
  } else {
    return pack2<IN>(a - __uint_as_float((unsigned)rounded << 16),
                     b - __uint_as_float((unsigned)rounded & 0xffff0000u));
  }
}
// Two blocks of 16 keys of one row set as the second operand of a step.
template <int IN>
__device__ __forceinline__ i32x4 pack_blocks(const f32x4& a, const f32x4& b) {
  return i32x4{pack2<IN>(a[0], a[1]), pack2<IN>(a[2], a[3]), pack2<IN>(b[0], b[1]),
               pack2<IN>(b[2], b[3])};
}

// sum + the four pairs of 16-bit values of a.
template <int IN>
__device__ __forceinline__ float add_pairs(const i32x4& a, float sum) {
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int two = a[e];
    if constexpr (IN == GEMM_F16) {
      typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
      sum = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, two), f16x2{1, 1}, sum, false);
    } else {
      typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
      sum = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, two), bf16x2{1, 1}, sum, false);
    }
  }
#endif
  return sum;
}

// Over the four lanes of a row.  (The swaps of 16 and 32 lanes hand every lane both values.)
struct Both {
  float a, b;
};
__device__ __forceinline__ Both swap16(float v) {
#if defined(__HIP_DEVICE_COMPILE__)
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return Both{__uint_as_float(r[0]), __uint_as_float(r[1])};
#else
  return Both{v, v};
#endif
}
__device__ __forceinline__ Both swap32(float v) {
#if defined(__HIP_DEVICE_COMPILE__)
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return Both{__uint_as_float(r[0]), __uint_as_float(r[1])};
#else
  return Both{v, v};
#endif
}
__device__ __forceinline__ float row_max(float v) {
  const Both x = swap16(v);
  const Both y = swap32(fmaxf(x.a, x.b));
  return fmaxf(y.a, y.b);
}
__device__ __forceinline__ float row_sum(float v) {
  const Both x = swap16(v);
  const Both y = swap32(x.a + x.b);
  return y.a + y.b;
}

// The largest of a step's logits of a row, in its own lane.  (A NaN is left out here and
// shows in the probabilities.)
__device__ __forceinline__ float lane_max(const f32x4 (&s)[4]) {
  float m = kNegInf;
#pragma unroll
  for (int b = 0; b < 4; ++b)
#pragma unroll
    for (int r = 0; r < 4; ++r) m = fmaxf(m, s[b][r]);
  return m;
}
// The reference of a row's probabilities, from step to step: the largest scaled logit of the
// step where it was last set.  It is set again only where a logit passes it by more than
// 8 (binary): probabilities are then at most 2^8, which fp32 sums and 16-bit values hold
// as well as 1, and the sums so far, which a new reference makes a pass over the
// output's registers for, mostly stay as they are.  A rule of the row's own logits.
__device__ __forceinline__ float reference(float m, float step_max) {
  return step_max > m + 8.0f ? step_max : m;
}
// What a reference that grew from a to b leaves of earlier sums (without any, there is nothing
// to change).
__device__ __forceinline__ float shrink(float a, float b) {
  return a == b || a == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(a - b);
}
// Probabilities about the reference m (of a row without any, 0), in place.
__device__ __forceinline__ void probabilities(f32x4 (&s)[4], float scale_log2, float m) {
  const float about = m == kNegInf ? 0.0f : m;
#pragma unroll
  for (int b = 0; b < 4; ++b)
#pragma unroll
    for (int r = 0; r < 4; ++r) s[b][r] = __builtin_amdgcn_exp2f(fmaf(s[b][r], scale_log2, -about));
}
__device__ __forceinline__ float sum_of(const f32x4 (&s)[4]) {
  float sum = 0.0f;
#pragma unroll
  for (int b = 0; b < 4; ++b) sum += (s[b][0] + s[b][1]) + (s[b][2] + s[b][3]);
  return sum;
}

// The result of the keys so far and that of one more chunk, about a reference that follows the
// chunks' as theirs follow the logits: o = o a + chunk_o b, and so the sums.
struct Join {
  float m, a, b;
};
__device__ __forceinline__ Join join_chunk(float m, float chunk_m) {
  const float to = reference(m, chunk_m);
  return Join{to, shrink(m, to), chunk_m == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(chunk_m - to)};
}
__device__ __forceinline__ float joined(float o, float chunk_o, const Join& j) {
  return fmaf(chunk_o, j.b, o * j.a);
}

}  // namespace dev
}  // namespace imm
