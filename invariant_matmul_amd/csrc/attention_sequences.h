// Which rows of q and which keys a workgroup or a wave of the attention kernels works on,
// from the call's arrays in device memory.  (Plain arithmetic and exchanges between lanes: a
// host program that supplies those walks through it too.)
#pragma once

#include "decoder_internal.h"

namespace imm {
namespace dev {

// A sequence of a call: its rows of q and its keys.  What the device's arrays say is
// clamped to the operands, so that no contents of theirs reach outside.  (Keys are counted in
// 30 bits, rows times heads in 31.)
struct Sequence {
  int q0, k0;   // first query, first key row
  int n, m;     // queries, keys
};

__device__ __forceinline__ int clamped(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// Segment i: sequence i - 1, or the rows before the first sequence (0) or behind the last
// (batch + 1), which have no keys.  Where its queries and keys begin:
__device__ __forceinline__ int q_start(const AttnArgs& a, int i) {
  const int rows = (int)a.q_rows;
  if (i <= 0) return 0;
  if (i > a.batch + 1) return rows;
  if (!a.cu_q) return i == 1 ? 0 : rows;
  return clamped(a.cu_q[i - 1], 0, rows);
}
__device__ __forceinline__ int key_start(const AttnArgs& a, int i) {
  const int rows = (int)a.k_rows;
  if (i <= 0) return 0;
  if (i > a.batch + 1) return rows;
  if (!a.cu_k) return i == 1 ? 0 : rows;
  return clamped(a.cu_k[i - 1], 0, rows);
}

// A segment for which begins(i, its first query, its first key) holds, and what it is: the last
// one where the arrays ascend.  begins(0) holds.  The segment is the last lane's that says yes, not their
// number: with arrays that do not ascend that one may begin behind what is looked for, whose
// place in it would be negative.  A lane looks at a segment: a call waits for memory once (and
// once more for each factor of 64 in the number of sequences), where a binary search waits at
// every step.
struct Found {
  int segment;
  int k_end;  // of its room
  Sequence s;
};
// (some lane's bit is set: begins(lo) holds throughout)
__device__ __forceinline__ int last_lane(uint64_t lanes) { return 63 - __builtin_clzll(lanes); }
template <class F>
__device__ __forceinline__ Found find_segment(const AttnArgs& a, F&& begins) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = a.batch + 2;
  while (n > 63) {
    const int step = (n + 63) / 64, i = lo + lane * step;
    const bool ok = i < lo + n && begins(i, q_start(a, i), key_start(a, i));
    const int skip = last_lane(__ballot(ok)) * step;
    lo += skip;
    n = n - skip < step ? n - skip : step;
  }
  const int i = lo + lane;
  int len = 0x7fffffff;
  if (a.k_lens && i >= 1 && i <= a.batch) len = a.k_lens[i - 1];
  const int q = q_start(a, i), k = key_start(a, i);
  const int l = last_lane(__ballot(lane < n && begins(i, q, k)));
  Found f{};
  f.segment = lo + l;
  f.s.q0 = __builtin_amdgcn_readlane(q, l);
  f.s.k0 = __builtin_amdgcn_readlane(k, l);
  const int q_end = __builtin_amdgcn_readlane(q, l + 1), k_end = __builtin_amdgcn_readlane(k, l + 1);
  f.k_end = k_end > f.s.k0 ? k_end : f.s.k0;
  f.s.n = q_end > f.s.q0 ? q_end - f.s.q0 : 0;
  if (f.segment >= 1 && f.segment <= a.batch) f.s.m = clamped(__builtin_amdgcn_readlane(len, l), 0, f.k_end - f.s.k0);
  return f;
}
// A tile of a segment's packed rows or keys, or a chunk of its keys.
struct FoundTile {
  Found found;
  int first;  // of the segment's; past its last if there is no such tile
};
// Tiles of ROWS packed rows: segment i begins at tile start(i) group / ROWS + i,
// so that every segment has the tiles it needs and no sum over segments is taken.
template <int ROWS>
__device__ __forceinline__ FoundTile tile_of_rows(const AttnArgs& a, int t) {
  FoundTile f;
  f.found = find_segment(a, [&](int i, int q, int) { return q * a.group / ROWS + i <= t; });
  f.first = (t - (f.found.s.q0 * a.group / ROWS + f.found.segment)) * ROWS;
  return f;
}
// Tiles of KEYS keys, those of a cache's room too: the same rule.
template <int KEYS>
__device__ __forceinline__ FoundTile tile_of_keys(const AttnArgs& a, int t) {
  FoundTile f;
  f.found = find_segment(a, [&](int i, int, int k) { return k / KEYS + i <= t; });
  f.first = (t - (f.found.s.k0 / KEYS + f.found.segment)) * KEYS;
  return f;
}
// Chunks of keys: sequence b's begin at slot (its first key) / 256 + b, so that every sequence has the
// slots that it needs.  (Slots before the first sequence's: segment 0, which has no keys.)
__device__ __forceinline__ int first_slot(const Found& f) { return f.s.k0 / kAttnChunk + f.segment - 1; }
__device__ __forceinline__ FoundTile chunk_of_slot(const AttnArgs& a, int slot) {
  FoundTile f;
  f.found = find_segment(a, [&](int i, int, int k) {
    return i == 0 || (i <= a.batch && k / kAttnChunk + (i - 1) <= slot);
  });
  f.first = (slot - first_slot(f.found)) * kAttnChunk;
  return f;
}
// The segment of a row of q.
__device__ __forceinline__ Found segment_of_query(const AttnArgs& a, int q) {
  return find_segment(a, [&](int, int first, int) { return first <= q; });
}

// The same tiles, none empty, with the longest sequence's first and each sequence's last rows first
// (up to kSortedSegments segments, a lane each).
constexpr int kSortedSegments = 32;
template <int ROWS>
__device__ __forceinline__ FoundTile longest_first(const AttnArgs& a, int t) {
  const int lane = threadIdx.x & 63, segments = a.batch + 2;
  int len = 0x7fffffff;
  if (a.k_lens && lane >= 1 && lane <= a.batch) len = a.k_lens[lane - 1];
  const int q = q_start(a, lane), k = key_start(a, lane);
  const int q_end = q_start(a, lane + 1), k_end = key_start(a, lane + 1);
  const int n = q_end > q ? q_end - q : 0, room = k_end > k ? k_end - k : 0;
  const int m = lane >= 1 && lane <= a.batch ? clamped(len, 0, room) : 0;
  const int tiles = lane < segments ? (n * a.group + ROWS - 1) / ROWS : 0;
  int before = 0;
  for (int j = 0; j < segments; ++j) {
    const int mj = __builtin_amdgcn_readlane(m, j), tj = __builtin_amdgcn_readlane(tiles, j);
    before += mj > m || (mj == m && j < lane) ? tj : 0;
  }
  const uint64_t in = __ballot(t >= before && t - before < tiles);
  FoundTile f{};
  if (in == 0) return f;
  const int l = __builtin_ctzll(in);
  f.found.segment = l;
  f.found.s.q0 = __builtin_amdgcn_readlane(q, l);
  f.found.s.k0 = __builtin_amdgcn_readlane(k, l);
  f.found.s.n = __builtin_amdgcn_readlane(n, l);
  f.found.s.m = __builtin_amdgcn_readlane(m, l);
  f.found.k_end = f.found.s.k0 + __builtin_amdgcn_readlane(room, l);
  f.first = (__builtin_amdgcn_readlane(tiles, l) - 1 - (t - __builtin_amdgcn_readlane(before, l))) * ROWS;
  return f;
}

// Keys that query t of a sequence sees: [0, seen).
__device__ __forceinline__ int keys_seen(const AttnArgs& a, const Sequence& s, int t) {
  if (t >= s.n) return 0;
  return a.causal ? clamped(s.m - s.n + t + 1, 0, s.m) : s.m;
}

}  // namespace dev
}  // namespace imm
