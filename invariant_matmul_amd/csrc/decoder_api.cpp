// Host side of the calls between and behind the products of a decoder: norms of
// heads with their rotation, attention, log probabilities of tokens.
// Validation and launches only; the plans hold sizes, types and options.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <new>

#include "decoder_internal.h"
#include "host_internal.h"

using namespace imm;

struct head_rope_plan_s {
  int64_t tokens;
  int heads[2], dim, rot, dtype, axes, section_end[kRopeMaxAxes];
  bool norm, interleaved;
  float eps;
};

struct attention_plan_s {
  int64_t q_rows, k_rows, max_q;
  int batch, q_heads, k_heads, dim, dtype;
  bool causal, few;
  float scale;
};

struct logprobs_plan_s {
  int64_t rows, vocab;
  int n, top, dtype, parts, units;
};

namespace {

bool is_16bit(int dt) { return dt == GEMM_F16 || dt == GEMM_BF16; }
bool aligned(const void* p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}
bool good(const void* p, unsigned bytes) { return p && aligned(p, bytes); }
gemm_status status_of(hipError_t e) { return e == hipSuccess ? GEMM_OK : record_hip_error(e); }

// Strides in elements: 16-byte steps, and no further than 2^40 in all.
bool strides_ok(int64_t tokens, int heads, int64_t token, int64_t head) {
  const int64_t most = (int64_t)1 << 40;
  return token >= 0 && head >= 0 && token % 8 == 0 && head % 8 == 0 && token <= most &&
         head <= most && (tokens <= 1 || token <= most / tokens) && (heads <= 1 || head <= most / heads);
}
size_t strided_bytes(int64_t tokens, int heads, int64_t token, int64_t head, int dim) {
  if (tokens == 0 || heads == 0) return 0;
  return 2 * ((size_t)(tokens - 1) * (size_t)token + (size_t)(heads - 1) * (size_t)head + (size_t)dim);
}

}  // namespace

extern "C" {

gemm_status head_rope_plan(int64_t tokens, int q_heads, int k_heads, int dim, int rot,
                           gemm_dtype dtype, int norm, float eps, int interleaved, int axes,
                           const int* sections, head_rope_plan_t* plan) {
  if (!plan) return GEMM_ERR_INVALID_VALUE;
  *plan = nullptr;
  if (tokens < 0 || q_heads < 0 || k_heads < 0 || dim < 0 || rot < 0 || (axes > 1 && !sections))
    return GEMM_ERR_INVALID_VALUE;
  if (!is_16bit(dtype) || dim == 0 || dim % 8 != 0 || dim > kRopeMaxDim || rot % 16 != 0 ||
      rot > dim || axes < 1 || axes > kRopeMaxAxes || tokens > INT_MAX || q_heads > 65536 ||
      k_heads > 65536)
    return GEMM_ERR_UNSUPPORTED;
  if (norm && (!std::isfinite(eps) || eps < 0.0f)) return GEMM_ERR_UNSUPPORTED;
  head_rope_plan_s p{tokens, {q_heads, k_heads}, dim, rot, dtype, axes, {}, norm != 0, interleaved != 0, eps};
  int64_t end = 0;
  for (int i = 0; i < axes; ++i) {
    const int n = sections ? sections[i] : rot / 2;
    if (n < 0) return GEMM_ERR_INVALID_VALUE;
    end += n;
    if (end > rot / 2) return GEMM_ERR_INVALID_VALUE;
    p.section_end[i] = (int)end;
  }
  if (end != rot / 2) return GEMM_ERR_INVALID_VALUE;
  *plan = new (std::nothrow) head_rope_plan_s(p);
  return *plan ? GEMM_OK : GEMM_ERR_INVALID_VALUE;
}

size_t head_rope_workspace_size(head_rope_plan_t p) {
  if (!p || !p->norm) return 0;
  return (size_t)head_rope_groups(p->tokens, p->heads[0] + p->heads[1], p->dim) * 2 * (size_t)p->dim *
         sizeof(float);
}

static gemm_status rope_args(head_rope_plan_t p, const void* q, int64_t q_token, int64_t q_head,
                             const void* k, int64_t k_token, int64_t k_head,
                             const int64_t* positions, const double* inv_freq,
                             const void* q_weight, const void* k_weight, void* q_out, void* k_out,
                             HeadRopeArgs* a) {
  *a = HeadRopeArgs{{q, k}, {q_token, k_token}, {q_head, k_head}, {q_weight, k_weight}, {q_out, k_out},
                    {nullptr, nullptr}, nullptr, positions, inv_freq, p->tokens,
                    {p->heads[0], p->heads[1]}, p->dim, p->rot, p->axes, {}, p->norm, p->interleaved,
                    p->eps, 1};
  for (int i = 0; i < kRopeMaxAxes; ++i) a->section_end[i] = p->section_end[i];
  for (int i = 0; i < 2; ++i) {
    if (p->heads[i] == 0) continue;
    if (!good(a->out[i], 16) || !aligned(a->weight[i], 16) || (a->weight[i] && !p->norm) ||
        !strides_ok(p->tokens, p->heads[i], a->token_stride[i], a->head_stride[i]))
      return GEMM_ERR_INVALID_VALUE;
  }
  if (p->rot > 0 && (!good(positions, 8) || !good(inv_freq, 8))) return GEMM_ERR_INVALID_VALUE;
  return GEMM_OK;
}

gemm_status head_rope_run(head_rope_plan_t p, const void* q, int64_t q_token, int64_t q_head,
                          const void* k, int64_t k_token, int64_t k_head, const int64_t* positions,
                          const double* inv_freq, const void* q_weight, const void* k_weight,
                          void* q_out, void* k_out, void* stream) {
  if (!p) return GEMM_ERR_INVALID_VALUE;
  if (p->tokens == 0 || p->heads[0] + p->heads[1] == 0) return GEMM_OK;
  HeadRopeArgs a;
  gemm_status st = rope_args(p, q, q_token, q_head, k, k_token, k_head, positions, inv_freq, q_weight,
                             k_weight, q_out, k_out, &a);
  if (st != GEMM_OK) return st;
  if ((p->heads[0] && !good(q, 16)) || (p->heads[1] && !good(k, 16))) return GEMM_ERR_INVALID_VALUE;
  const size_t dim = (size_t)p->dim, n = (size_t)p->tokens * dim * 2;
  const bool hq = p->heads[0] > 0, hk = p->heads[1] > 0;
  st = check_device_operands(
      {{hq ? q : nullptr, strided_bytes(p->tokens, p->heads[0], q_token, q_head, p->dim)},
       {hk ? k : nullptr, strided_bytes(p->tokens, p->heads[1], k_token, k_head, p->dim)},
       {p->rot ? positions : nullptr, (size_t)p->tokens * (size_t)p->axes * 8},
       {p->rot ? inv_freq : nullptr, (size_t)p->rot * 4},
       {hq ? q_weight : nullptr, 2 * dim},
       {hk ? k_weight : nullptr, 2 * dim},
       {hq ? q_out : nullptr, n * (size_t)p->heads[0]},
       {hk ? k_out : nullptr, n * (size_t)p->heads[1]}});
  if (st != GEMM_OK) return st;
  return status_of(launch_head_rope(p->dtype, a, static_cast<hipStream_t>(stream)));
}

gemm_status head_rope_backward(head_rope_plan_t p, const void* dq_out, const void* dk_out,
                               const void* q, int64_t q_token, int64_t q_head, const void* k,
                               int64_t k_token, int64_t k_head, const int64_t* positions,
                               const double* inv_freq, const void* q_weight, const void* k_weight,
                               void* dq, void* dk, void* dq_weight, void* dk_weight,
                               void* workspace, size_t workspace_bytes, void* stream) {
  if (!p) return GEMM_ERR_INVALID_VALUE;
  const bool weights = dq_weight || dk_weight;
  if (weights && !p->norm) return GEMM_ERR_INVALID_VALUE;
  if (!aligned(dq_weight, 16) || !aligned(dk_weight, 16)) return GEMM_ERR_INVALID_VALUE;
  const bool any = p->tokens > 0 && p->heads[0] + p->heads[1] > 0;
  if (!any && !weights) return GEMM_OK;
  HeadRopeArgs a{};
  gemm_status st = GEMM_OK;
  const size_t need = weights && any ? head_rope_workspace_size(p) : 0;
  if (any) {
    st = rope_args(p, q, q_token, q_head, k, k_token, k_head, positions, inv_freq, q_weight, k_weight,
                   dq, dk, &a);
    if (st != GEMM_OK) return st;
    a.dy[0] = dq_out;
    a.dy[1] = dk_out;
    for (int i = 0; i < 2; ++i)
      if (p->heads[i] && (!good(a.dy[i], 16) || (p->norm && !good(a.x[i], 16)))) return GEMM_ERR_INVALID_VALUE;
    if (need) {
      if (!workspace || workspace_bytes < need) return GEMM_ERR_WORKSPACE;
      if (!aligned(workspace, 16)) return GEMM_ERR_INVALID_VALUE;
      a.parts = static_cast<float*>(workspace);
    }
  }
  a.dim = p->dim;
  const size_t dim = (size_t)p->dim, n = (size_t)p->tokens * dim * 2;
  const bool hq = any && p->heads[0] > 0, hk = any && p->heads[1] > 0;
  const size_t nq = n * (size_t)p->heads[0], nk = n * (size_t)p->heads[1];
  st = check_device_operands(
      {{hq ? dq_out : nullptr, nq},
       {hk ? dk_out : nullptr, nk},
       {hq && p->norm ? q : nullptr, strided_bytes(p->tokens, p->heads[0], q_token, q_head, p->dim)},
       {hk && p->norm ? k : nullptr, strided_bytes(p->tokens, p->heads[1], k_token, k_head, p->dim)},
       {any && p->rot ? positions : nullptr, (size_t)p->tokens * (size_t)p->axes * 8},
       {any && p->rot ? inv_freq : nullptr, (size_t)p->rot * 4},
       {hq ? q_weight : nullptr, 2 * dim},
       {hk ? k_weight : nullptr, 2 * dim},
       {hq ? dq : nullptr, nq},
       {hk ? dk : nullptr, nk},
       {dq_weight, 2 * dim},
       {dk_weight, 2 * dim},
       {need ? workspace : nullptr, need}});
  if (st != GEMM_OK) return st;
  void* const dw[2] = {dq_weight, dk_weight};
  return status_of(launch_head_rope_backward(p->dtype, a, dw, static_cast<hipStream_t>(stream)));
}

void head_rope_plan_destroy(head_rope_plan_t p) { delete p; }

gemm_status attention_plan(int64_t q_rows, int64_t k_rows, int64_t batch, int q_heads, int k_heads,
                           int dim, gemm_dtype dtype, int causal, float scale, int64_t max_q,
                           attention_plan_t* plan) {
  if (!plan) return GEMM_ERR_INVALID_VALUE;
  *plan = nullptr;
  if (q_rows < 0 || k_rows < 0 || batch < 1 || q_heads < 0 || k_heads < 0 || dim < 0 || max_q < 0)
    return GEMM_ERR_INVALID_VALUE;
  if (!is_16bit(dtype) || dim == 0 || dim % 8 != 0 || dim > kAttnMaxDim || k_heads == 0 ||
      q_heads == 0 || q_heads % k_heads != 0 || q_heads > 65536)
    return GEMM_ERR_UNSUPPORTED;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return GEMM_ERR_UNSUPPORTED;
  const int64_t group = q_heads / k_heads;
  // 31-bit counts of keys, of a sequence's rows and of rows and heads, and launches of
  // fewer than 2^32 threads
  if (q_rows > INT_MAX / q_heads || k_rows > (int64_t)1 << 30 || batch > 1 << 20 ||
      (q_rows * group / 128 + batch + 2) * k_heads >= (int64_t)1 << 23 ||
      (k_rows / 128 + batch + 10) * k_heads >= (int64_t)1 << 22)
    return GEMM_ERR_UNSUPPORTED;
  attention_plan_s p{q_rows, k_rows, max_q, (int)batch, q_heads, k_heads, dim, dtype, causal != 0, false, scale};
  if (p.max_q == 0 || p.max_q > q_rows) p.max_q = q_rows;
  AttnArgs sizes{};
  sizes.q_rows = q_rows, sizes.k_rows = k_rows, sizes.batch = (int)batch, sizes.k_heads = k_heads;
  sizes.group = (int)group, sizes.dim = dim, sizes.max_q = p.max_q;
  p.few = q_rows > 0 && attention_few_rows(sizes);
  *plan = new (std::nothrow) attention_plan_s(p);
  return *plan ? GEMM_OK : GEMM_ERR_INVALID_VALUE;
}

size_t attention_workspace_size(attention_plan_t p) {
  if (!p || !p->few) return 0;
  const size_t slots = (size_t)attention_chunk_slots(p->k_rows, p->batch);
  return slots * (size_t)(p->q_heads * p->max_q) * (size_t)(p->dim + 4) * sizeof(float);
}

size_t attention_backward_workspace_size(attention_plan_t p) {
  return p ? 2 * (size_t)p->q_rows * (size_t)p->q_heads * sizeof(float) : 0;
}

static gemm_status attention_args(attention_plan_t p, const void* q, int64_t q_token,
                                  int64_t q_head, const void* k, int64_t k_token, int64_t k_head,
                                  const void* v, int64_t v_token, int64_t v_head, const int* cu_q,
                                  const int* cu_k, const int* k_lens, AttnArgs* a) {
  *a = AttnArgs{};
  a->q = q, a->k = k, a->v = v;
  a->q_token = q_token, a->q_head = q_head, a->k_token = k_token, a->k_head = k_head;
  a->v_token = v_token, a->v_head = v_head;
  a->cu_q = cu_q, a->cu_k = cu_k, a->k_lens = k_lens;
  a->q_rows = p->q_rows, a->k_rows = p->k_rows, a->batch = p->batch;
  a->q_heads = p->q_heads, a->k_heads = p->k_heads, a->group = p->q_heads / p->k_heads, a->dim = p->dim;
  a->max_q = p->max_q;
  a->scale = p->scale, a->scale_log2 = (float)(p->scale * 1.4426950408889634);
  a->causal = p->causal;
  // one sequence needs no arrays, several need both
  if (!cu_q != !cu_k || (!cu_q && p->batch != 1) || !aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(k_lens, 4))
    return GEMM_ERR_INVALID_VALUE;
  if (p->q_rows > 0 && (!good(q, 16) || !strides_ok(p->q_rows, p->q_heads, q_token, q_head)))
    return GEMM_ERR_INVALID_VALUE;
  if (p->k_rows > 0 && (!good(k, 16) || !good(v, 16) || !strides_ok(p->k_rows, p->k_heads, k_token, k_head) ||
                        !strides_ok(p->k_rows, p->k_heads, v_token, v_head)))
    return GEMM_ERR_INVALID_VALUE;
  // 256 rows of keys or values within 31 bits
  const int64_t most = ((int64_t)1 << 31) / (2 * kAttnChunk) - kAttnMaxDim;
  if (p->k_rows > 0 && (k_token > most || v_token > most)) return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

gemm_status attention_run(attention_plan_t p, const void* q, int64_t q_token, int64_t q_head,
                          const void* k, int64_t k_token, int64_t k_head, const void* v,
                          int64_t v_token, int64_t v_head, const int* cu_q, const int* cu_k,
                          const int* k_lens, void* o, void* o_low, float* lse, void* workspace,
                          size_t workspace_bytes, void* stream) {
  if (!p) return GEMM_ERR_INVALID_VALUE;
  if (p->q_rows == 0) return GEMM_OK;
  AttnArgs a;
  gemm_status st = attention_args(p, q, q_token, q_head, k, k_token, k_head, v, v_token, v_head, cu_q,
                                  cu_k, k_lens, &a);
  if (st != GEMM_OK) return st;
  if (!good(o, 16) || !aligned(o_low, 16) || !aligned(lse, 4)) return GEMM_ERR_INVALID_VALUE;
  const size_t need = attention_workspace_size(p);
  if (need) {
    if (!workspace || workspace_bytes < need) return GEMM_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return GEMM_ERR_INVALID_VALUE;
  }
  const size_t all = (size_t)p->q_rows * (size_t)p->q_heads, b = (size_t)p->batch;
  const bool keys = p->k_rows > 0;
  st = check_device_operands({{q, strided_bytes(p->q_rows, p->q_heads, q_token, q_head, p->dim)},
                              {keys ? k : nullptr, strided_bytes(p->k_rows, p->k_heads, k_token, k_head, p->dim)},
                              {keys ? v : nullptr, strided_bytes(p->k_rows, p->k_heads, v_token, v_head, p->dim)},
                              {cu_q, 4 * (b + 1)},
                              {cu_k, 4 * (b + 1)},
                              {k_lens, 4 * b},
                              {o, 2 * all * (size_t)p->dim},
                              {o_low, 2 * all * (size_t)p->dim},
                              {lse, 4 * all},
                              {need ? workspace : nullptr, need}});
  if (st != GEMM_OK) return st;
  a.o = o;
  a.o_low = o_low;
  a.lse = lse;
  if (p->few) {
    a.chunks = attention_chunk_slots(p->k_rows, p->batch);
    a.part_rows = (int)(p->max_q * a.group);
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = a.part_o + (size_t)a.chunks * (size_t)a.k_heads * (size_t)a.part_rows * (size_t)p->dim;
  }
  return status_of(launch_attention(p->dtype, a, static_cast<hipStream_t>(stream)));
}

gemm_status attention_backward(attention_plan_t p, const void* d_o, const void* q, int64_t q_token,
                               int64_t q_head, const void* k, int64_t k_token, int64_t k_head,
                               const void* v, int64_t v_token, int64_t v_head, const void* o,
                               const void* o_low, const float* lse, const int* cu_q, const int* cu_k,
                               const int* k_lens, void* dq, void* dk, void* dv, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (!p) return GEMM_ERR_INVALID_VALUE;
  if (p->q_rows == 0 && p->k_rows == 0) return GEMM_OK;
  AttnArgs a;
  gemm_status st = attention_args(p, q, q_token, q_head, k, k_token, k_head, v, v_token, v_head, cu_q,
                                  cu_k, k_lens, &a);
  if (st != GEMM_OK) return st;
  const bool rows = p->q_rows > 0, keys = p->k_rows > 0;
  // 64 packed rows of q, and of the contiguous gradient, within 31 bits
  const int64_t reach = ((int64_t)1 << 30) - kAttnMaxDim;
  if (rows && (q_token > reach / 128 || (a.group > 1 && q_head > reach / 2 / (a.group - 1)) ||
               (int64_t)p->q_heads * p->dim > reach / 128))
    return GEMM_ERR_UNSUPPORTED;
  const size_t need = attention_backward_workspace_size(p);
  if (rows && (!good(d_o, 16) || !good(o, 16) || !aligned(o_low, 16) || !good(lse, 4) || !good(dq, 16))) return GEMM_ERR_INVALID_VALUE;
  if (keys && (!good(dk, 16) || !good(dv, 16))) return GEMM_ERR_INVALID_VALUE;
  if (need) {
    if (!workspace || workspace_bytes < need) return GEMM_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return GEMM_ERR_INVALID_VALUE;
  }
  const size_t all = (size_t)p->q_rows * (size_t)p->q_heads, b = (size_t)p->batch;
  const size_t nq = 2 * all * (size_t)p->dim, nk = 2 * (size_t)p->k_rows * (size_t)p->k_heads * (size_t)p->dim;
  st = check_device_operands({{rows ? q : nullptr, strided_bytes(p->q_rows, p->q_heads, q_token, q_head, p->dim)},
                              {keys ? k : nullptr, strided_bytes(p->k_rows, p->k_heads, k_token, k_head, p->dim)},
                              {keys ? v : nullptr, strided_bytes(p->k_rows, p->k_heads, v_token, v_head, p->dim)},
                              {rows ? d_o : nullptr, nq},
                              {rows ? o : nullptr, nq},
                              {rows ? o_low : nullptr, nq},
                              {rows ? lse : nullptr, 4 * all},
                              {rows ? dq : nullptr, nq},
                              {keys ? dk : nullptr, nk},
                              {keys ? dv : nullptr, nk},
                              {cu_q, 4 * (b + 1)},
                              {cu_k, 4 * (b + 1)},
                              {k_lens, 4 * b},
                              {need ? workspace : nullptr, need}});
  if (st != GEMM_OK) return st;
  a.d_o = d_o;
  a.o = const_cast<void*>(o);
  a.o_low = const_cast<void*>(o_low);
  a.lse = const_cast<float*>(lse);
  a.stats = static_cast<float*>(workspace);
  a.dq = dq, a.dk = dk, a.dv = dv;
  return status_of(launch_attention_backward(p->dtype, a, static_cast<hipStream_t>(stream)));
}

void attention_plan_destroy(attention_plan_t p) { delete p; }

gemm_status logprobs_plan(int64_t rows, int64_t vocab, int tokens_per_row, int top,
                          gemm_dtype dtype, logprobs_plan_t* plan) {
  if (!plan) return GEMM_ERR_INVALID_VALUE;
  *plan = nullptr;
  if (rows < 0 || vocab < 1 || tokens_per_row < 0 || top < 0 || top > vocab) return GEMM_ERR_INVALID_VALUE;
  if ((!is_16bit(dtype) && dtype != GEMM_F32) || rows > INT_MAX || vocab > kLogprobsMaxVocab ||
      tokens_per_row > 1024 || top > kLogprobsMaxTop)
    return GEMM_ERR_UNSUPPORTED;
  *plan = new (std::nothrow) logprobs_plan_s{
      rows, vocab, tokens_per_row, top, dtype, logprobs_parts(rows, vocab),
      (int)((vocab + kLogprobsUnit - 1) / kLogprobsUnit)};
  return *plan ? GEMM_OK : GEMM_ERR_INVALID_VALUE;
}

size_t logprobs_workspace_size(logprobs_plan_t p) {
  if (!p || p->parts <= 1) return 0;
  const size_t sums = ((size_t)p->units * 12 + 7) & ~(size_t)7;
  return (size_t)p->rows * (sums + (size_t)p->parts * kLogprobsWaves * (size_t)p->top * 8);
}

gemm_status logprobs_run(logprobs_plan_t p, const void* logits, int64_t row_stride,
                         const int64_t* tokens, float* logprob, float* entropy, float* norm,
                         float* top_logprob, int64_t* top_token, void* workspace,
                         size_t workspace_bytes, void* stream) {
  if (!p) return GEMM_ERR_INVALID_VALUE;
  if (p->rows == 0) return GEMM_OK;
  const unsigned size = p->dtype == GEMM_F32 ? 4 : 2;
  if (!good(logits, size) || row_stride < 0 || (row_stride && row_stride > ((int64_t)1 << 46) / p->rows) ||
      (p->n && (!good(tokens, 8) || !good(logprob, 4))) || !good(entropy, 4) || !aligned(norm, 4) ||
      (p->top && (!good(top_logprob, 4) || !good(top_token, 8))))
    return GEMM_ERR_INVALID_VALUE;
  const size_t need = logprobs_workspace_size(p);
  if (need) {
    if (!workspace || workspace_bytes < need) return GEMM_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return GEMM_ERR_INVALID_VALUE;
  }
  const size_t rows = (size_t)p->rows, n = rows * (size_t)p->n, top = rows * (size_t)p->top;
  const gemm_status st = check_device_operands(
      {{logits, ((rows - 1) * (size_t)row_stride + (size_t)p->vocab) * size},
       {p->n ? tokens : nullptr, 8 * n},
       {p->n ? logprob : nullptr, 4 * n},
       {entropy, 4 * rows},
       {norm, 8 * rows},
       {p->top ? top_logprob : nullptr, 4 * top},
       {p->top ? top_token : nullptr, 8 * top},
       {need ? workspace : nullptr, need}});
  if (st != GEMM_OK) return st;
  LogprobsArgs a{};
  a.x = logits, a.row_stride = row_stride, a.tokens = tokens, a.rows = p->rows, a.vocab = p->vocab;
  a.n = p->n, a.top = p->top, a.logprob = logprob, a.entropy = entropy, a.norm = norm;
  a.top_logprob = top_logprob, a.top_token = top_token;
  a.units = p->units, a.parts = p->parts;
  if (need) {
    // the lists of 64-bit keys first
    a.best = static_cast<uint64_t*>(workspace);
    a.sums = reinterpret_cast<float*>(a.best + rows * (size_t)p->parts * kLogprobsWaves * (size_t)p->top);
  }
  return status_of(launch_logprobs(p->dtype, a, static_cast<hipStream_t>(stream)));
}

gemm_status logprobs_backward(logprobs_plan_t p, const float* d_logprob, const float* d_entropy,
                              const void* logits, int64_t row_stride, const int64_t* tokens,
                              const float* norm, const float* entropy, void* d_logits,
                              void* stream) {
  if (!p) return GEMM_ERR_INVALID_VALUE;
  if (p->rows == 0) return GEMM_OK;
  const unsigned size = p->dtype == GEMM_F32 ? 4 : 2;
  if (!good(logits, size) || row_stride < 0 || (row_stride && row_stride > ((int64_t)1 << 46) / p->rows) ||
      (p->n && !good(tokens, 8)) || !aligned(d_logprob, 4) || !aligned(d_entropy, 4) || !good(norm, 4) ||
      !good(entropy, 4) || !good(d_logits, 16))
    return GEMM_ERR_INVALID_VALUE;
  const size_t rows = (size_t)p->rows, n = rows * (size_t)p->n;
  const gemm_status st = check_device_operands(
      {{logits, ((rows - 1) * (size_t)row_stride + (size_t)p->vocab) * size},
       {p->n ? tokens : nullptr, 8 * n},
       {p->n ? d_logprob : nullptr, 4 * n},
       {d_entropy, 4 * rows},
       {norm, 8 * rows},
       {entropy, 4 * rows},
       {d_logits, rows * (size_t)p->vocab * size}});
  if (st != GEMM_OK) return st;
  LogprobsArgs a{};
  a.x = logits, a.row_stride = row_stride, a.tokens = tokens, a.rows = p->rows, a.vocab = p->vocab;
  a.n = p->n, a.norm = const_cast<float*>(norm), a.entropy = const_cast<float*>(entropy);
  a.d_logprob = d_logprob, a.d_entropy = d_entropy, a.dx = d_logits;
  return status_of(launch_logprobs_backward(p->dtype, a, static_cast<hipStream_t>(stream)));
}

void logprobs_plan_destroy(logprobs_plan_t p) { delete p; }

}  // extern "C"
