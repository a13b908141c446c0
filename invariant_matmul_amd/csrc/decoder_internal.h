// Internal declarations of the calls between and behind the products of a
// decoder (decoder_api.cpp and its kernels): norms of heads with the rotation of
// their position, attention, log probabilities of tokens.
#pragma once

#include "imm_internal.h"

namespace imm {

// ---- Norm and rotation of heads (head_rope.hip) --------------------------------
constexpr int kRopeMaxDim = 512;     // 64 lanes of 8 elements
constexpr int kRopeMaxAxes = 4;
// Workgroups of the backward pass with weights (each leaves its parts of the
// weights' gradients): four per compute unit of a 256-CU MI355X.
constexpr int64_t kRopeBwdGroups = 1024;
struct HeadRopeArgs {
  // [0] queries, [1] keys: x[t * token_stride + h * head_stride + d]
  const void* x[2];
  int64_t token_stride[2], head_stride[2];
  const void* weight[2];   // [dim] or null: ones
  void* out[2];            // [tokens, heads, dim]; the backward pass: the gradients of x
  const void* dy[2];       // the backward pass: [tokens, heads, dim]
  float* parts;            // [groups, 2, dim] or null
  const int64_t* positions;  // [axes, tokens]
  const double* inv_freq;    // [rot / 2]
  int64_t tokens;
  int heads[2];
  int dim, rot;
  int axes, section_end[kRopeMaxAxes];
  int norm, interleaved;
  float eps;
  int share;                 // 2^share waves take a token
};
int64_t head_rope_groups(int64_t tokens, int heads, int dim);
hipError_t launch_head_rope(int in, HeadRopeArgs a, hipStream_t s);
// dweight[i]: [dim] in the input's type, or null
hipError_t launch_head_rope_backward(int in, HeadRopeArgs a, void* const* dweight, hipStream_t s);

// ---- Attention (attention.hip, attention_backward.hip) --------------------------
constexpr int kAttnMaxDim = 128;
constexpr int kAttnChunk = 256;  // keys whose products one softmax partial holds
constexpr int kAttnTile = 64;    // keys of a step
struct AttnArgs {
  const void *q, *k, *v;
  void* o;                 // [q_rows, q_heads, dim]
  void* o_low;             // what o's rounding left, for the backward pass, or null
  float* lse;              // [q_rows, q_heads] or null
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;  // strides, elements
  const int *cu_q, *cu_k;  // [batch + 1], or null: one sequence
  const int* k_lens;       // [batch] or null
  int64_t q_rows, k_rows;
  int batch, q_heads, k_heads, group, dim;
  int64_t max_q;
  float scale, scale_log2;  // scale log2(e)
  int causal;
  int sorted;              // many rows: the longest sequences first
  // few rows: partial results per (chunk, key head, row): o [.., dim] and
  // (reference, sum of rounded, sum of unrounded probabilities, whether the chunk holds values that
  // are not finite)
  float *part_o, *part_ml;
  int64_t chunks;          // chunk slots of all sequences
  int part_rows;           // rows a chunk slot holds: max_q group
  // backward
  const void* d_o;         // [q_rows, q_heads, dim]
  float* stats;            // -lse log2(e) and delta, [2, k_heads, q_rows, group]
  int64_t q_tiles, k_tiles;
  int k_turns;
  void *dq, *dk, *dv;      // contiguous
};
bool attention_few_rows(const AttnArgs& a);  // by its sizes
int64_t attention_chunk_slots(int64_t k_rows, int batch);
hipError_t launch_attention(int in, const AttnArgs& a, hipStream_t s);
hipError_t launch_attention_backward(int in, const AttnArgs& a, hipStream_t s);

// ---- Log probabilities of tokens (token_logprobs.hip) ---------------------------
constexpr int kLogprobsMaxTop = 64;         // a lane each
constexpr int64_t kLogprobsMaxVocab = (int64_t)1 << 22;
constexpr int kLogprobsUnit = 2048;         // logits one wave sums at a time
constexpr int kLogprobsWaves = 4;
struct LogprobsArgs {
  const void* x;
  int64_t row_stride;      // elements
  const int64_t* tokens;   // [rows, n]
  int64_t rows, vocab;
  int n, top;
  float *logprob, *entropy, *norm;  // [rows, n], [rows], [rows, 2] or null
  float* top_logprob;      // [rows, top]
  int64_t* top_token;
  // rows cut into parts: the units' sums [rows, units, 3] and the waves' best
  float* sums;
  uint64_t* best;          // [rows, parts * waves, top]
  int units, parts;
  // backward
  const float *d_logprob, *d_entropy;  // [rows, n] and [rows], or null
  void* dx;                // [rows, vocab]
};
int logprobs_parts(int64_t rows, int64_t vocab);
hipError_t launch_logprobs(int in, const LogprobsArgs& a, hipStream_t s);
hipError_t launch_logprobs_backward(int in, const LogprobsArgs& a, hipStream_t s);

}  // namespace imm
