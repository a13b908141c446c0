// Host walk through csrc/attention_sequences.h: 64 lanes as contexts that meet at every exchange.
//   check MODE q_rows k_rows q_heads k_heads max_q causal cu_q.. -- cu_k.. -- k_lens..   (k_lens may be empty)
// For every tile, chunk and row of the modes below, the rows of q and keys that the kernels would
// touch are inside the operands, and where the arrays ascend every row and key has
// its place once.  Prints what is wrong; exit status 1.
#include <ucontext.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <map>
#include <set>
#include <string>
#include <utility>
#include <vector>

namespace wave {
struct Context {
  ucontext_t uc;
  std::vector<char> stack;
  bool done;
};
static Context lanes[64];
static ucontext_t home;
static int current;
static uint64_t offered[64], seen[64];
static std::function<void()> body;
static void meet(uint64_t v) {
  offered[current] = v;
  swapcontext(&lanes[current].uc, &home);
}
static void enter() {
  body();
  lanes[current].done = true;
  swapcontext(&lanes[current].uc, &home);
}
// f by 64 lanes in step
static void run(std::function<void()> f) {
  body = std::move(f);
  for (int l = 0; l < 64; ++l) {
    Context& c = lanes[l];
    c.stack.resize(1 << 16);
    c.done = false;
    getcontext(&c.uc);
    c.uc.uc_stack.ss_sp = c.stack.data();
    c.uc.uc_stack.ss_size = c.stack.size();
    c.uc.uc_link = &home;
    makecontext(&c.uc, enter, 0);
  }
  for (;;) {
    int done = 0;
    for (current = 0; current < 64; ++current) {
      swapcontext(&home, &lanes[current].uc);
      done += lanes[current].done;
    }
    if (done == 64) return;
    if (done) {
      std::printf("%d lanes left early\n", done);
      std::exit(1);
    }
    std::memcpy(seen, offered, sizeof seen);
  }
}
struct Index {
  struct X {
    operator unsigned() const { return (unsigned)current; }
  } x;
};
}  // namespace wave

static wave::Index threadIdx;
static inline uint64_t __ballot(bool v) {
  wave::meet(v);
  uint64_t r = 0;
  for (int l = 0; l < 64; ++l) r |= (wave::seen[l] & 1) << l;
  return r;
}
static inline int __popcll(uint64_t v) { return __builtin_popcountll(v); }
static inline int __builtin_amdgcn_readlane(int v, int lane) {
  wave::meet((uint64_t)(unsigned)v | (uint64_t)(unsigned)lane << 32);
  for (int l = 0; l < 64; ++l)
    if ((int)(wave::seen[l] >> 32) != lane) {
      std::printf("lanes ask for different lanes\n");
      std::exit(1);
    }
  if (lane < 0 || lane > 63) {
    std::printf("lane %d\n", lane);
    std::exit(1);
  }
  return (int)(unsigned)wave::seen[lane];
}

#include "attention_sequences.h"

using namespace imm;
using namespace imm::dev;

static AttnArgs a;
static std::vector<int> arrays[3];
static bool good_arrays;  // they ascend, from 0 to the rows, and no sequence has more queries than said

static void wrong(const char* what, long at, long x, long lo, long hi) {
  std::printf("%s at %ld: %ld outside [%ld, %ld]\n", what, at, x, lo, hi);
  std::exit(1);
}
static void inside(const char* what, long at, long x, long lo, long hi) {
  if (x < lo || x > hi) wrong(what, at, x, lo, hi);
}
static FoundTile found(const std::function<FoundTile()>& f) {
  FoundTile r{};
  wave::run([&] {
    const FoundTile x = f();
    if (wave::current == 0) r = x;
  });
  return r;
}
static void sequence_inside(const char* what, long at, const Found& f) {
  inside(what, at, f.segment, 0, a.batch + 1);
  inside(what, at, f.s.q0, 0, a.q_rows);
  inside(what, at, f.s.n, 0, a.q_rows - f.s.q0);
  inside(what, at, f.s.k0, 0, a.k_rows);
  inside(what, at, f.s.m, 0, a.k_rows - f.s.k0);
  inside(what, at, f.k_end, f.s.k0, a.k_rows);
}

static std::map<long, int> rows_done, keys_done;
template <int ROWS>
static void rows_of(const char* what, long t, const FoundTile& f) {
  sequence_inside(what, t, f.found);
  const Sequence& s = f.found.s;
  const long rows = (long)s.n * a.group;
  if (f.first >= rows) return;
  inside(what, t, f.first, 0, rows);
  for (long r = f.first; r < f.first + ROWS && r < rows; ++r) {
    const int q = (int)(r / a.group);
    inside(what, t, s.q0 + q, 0, a.q_rows - 1);
    inside(what, t, keys_seen(a, s, q), 0, s.m);
    ++rows_done[(long)s.q0 * a.group + r];
  }
}
static void all_rows_once(const char* what) {
  if (good_arrays) {
    for (long r = 0; r < a.q_rows * a.group; ++r) inside(what, r, rows_done[r], 1, 1);
    inside(what, -1, (long)rows_done.size(), a.q_rows * a.group, a.q_rows * a.group);
  }
  rows_done.clear();
}
template <int ROWS>
static void tiles_of_rows(bool sorted) {
  // (the grid of the forward kernel; the backward pass has the same)
  const long tiles = a.q_rows * a.group / ROWS + a.batch + 2;
  for (long t = 0; t < tiles; ++t)
    rows_of<ROWS>(sorted ? "longest_first" : "tile_of_rows", t,
                  found([&] { return sorted ? longest_first<ROWS>(a, (int)t) : tile_of_rows<ROWS>(a, (int)t); }));
  all_rows_once("rows");
}
template <int KEYS>
static void tiles_of_keys() {
  const long tiles = a.k_rows / KEYS + a.batch + 2;
  for (long t = 0; t < tiles; ++t) {
    const FoundTile f = found([&] { return tile_of_keys<KEYS>(a, (int)t); });
    sequence_inside("tile_of_keys", t, f.found);
    const Sequence& s = f.found.s;
    const long room = f.found.k_end - s.k0;
    if (f.first >= room) continue;
    inside("tile_of_keys", t, f.first, 0, room);
    for (long k = f.first; k < f.first + KEYS && k < room; ++k) {
      inside("key", t, s.k0 + k, 0, a.k_rows - 1);
      ++keys_done[s.k0 + k];
    }
  }
  if (good_arrays)
    for (long k = 0; k < a.k_rows; ++k) inside("keys", k, keys_done[k], 1, 1);
  keys_done.clear();
}
static void chunks_and_joins() {
  const long slots = a.k_rows / kAttnChunk + a.batch;
  std::set<std::pair<long, long>> written;  // (slot, row of the slot)
  for (long slot = 0; slot < slots; ++slot) {
    const FoundTile f = found([&] { return chunk_of_slot(a, (int)slot); });
    sequence_inside("chunk_of_slot", slot, f.found);
    const Sequence& s = f.found.s;
    if (f.first >= s.m || s.n == 0) continue;
    inside("chunk_of_slot", slot, f.first, 0, s.m);
    const int queries = s.n < a.max_q ? s.n : (int)a.max_q;
    if (f.first >= keys_seen(a, s, queries - 1)) continue;
    inside("rows of a slot", slot, (long)queries * a.group, 0, a.part_rows);
    for (int r = 0; r < queries * a.group; ++r) written.insert({slot, r});
  }
  for (long q = 0; q < a.q_rows; ++q) {
    const Found f = found([&] { return FoundTile{segment_of_query(a, (int)q), 0}; }).found;
    sequence_inside("segment_of_query", q, f);
    const int t = (int)q - f.s.q0;
    const int seen = keys_seen(a, f.s, t);
    inside("keys of a query", q, seen, 0, f.s.m);
    const bool said = t < a.max_q || f.segment == 0 || f.segment > a.batch;
    if (!said || seen == 0) continue;
    inside("row of a slot", q, t, 0, a.max_q - 1);
    for (long c = 0; c < (seen + kAttnChunk - 1) / kAttnChunk; ++c) {
      inside("slot of a row", q, first_slot(f) + c, 0, slots - 1);
      if (good_arrays && !written.count({first_slot(f) + c, (long)t * a.group})) wrong("slot that no one wrote", q, c, 0, -1);
    }
  }
}

int main(int argc, char** argv) {
  if (argc < 8) return 2;
  const std::string mode = argv[1];
  a.q_rows = std::atol(argv[2]), a.k_rows = std::atol(argv[3]);
  a.q_heads = std::atoi(argv[4]), a.k_heads = std::atoi(argv[5]);
  a.group = a.q_heads / a.k_heads;
  a.max_q = std::atol(argv[6]), a.causal = std::atoi(argv[7]);
  a.part_rows = (int)(a.max_q * a.group);
  int which = 0;
  for (int i = 8; i < argc; ++i) {
    if (std::string(argv[i]) == "--") ++which;
    else arrays[which].push_back((int)std::strtol(argv[i], nullptr, 10));
  }
  a.batch = (int)arrays[0].size() - 1;
  a.cu_q = arrays[0].data(), a.cu_k = arrays[1].data();
  a.k_lens = arrays[2].empty() ? nullptr : arrays[2].data();
  good_arrays = true;
  for (int w = 0; w < 2; ++w)
    for (size_t i = 0; i < arrays[w].size(); ++i)
      good_arrays &= arrays[w][i] >= (i ? arrays[w][i - 1] : 0) && arrays[w][i] <= (w ? a.k_rows : a.q_rows);
  for (int i = 0; i < a.batch; ++i) good_arrays &= arrays[0][i + 1] - arrays[0][i] <= a.max_q;
  if (mode == "rows") {
    tiles_of_rows<64>(false);
    tiles_of_rows<128>(false);
  } else if (mode == "sorted") {
    tiles_of_rows<64>(true);
    tiles_of_rows<128>(true);
  } else if (mode == "keys") {
    tiles_of_keys<64>();
    tiles_of_keys<128>();
  } else {
    chunks_and_joins();
  }
  return 0;
}
