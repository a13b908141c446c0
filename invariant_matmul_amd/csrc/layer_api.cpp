// Host side of the calls around a linear layer: the row norm, fp8 rows, 4-bit
// weights.
// Validation and launches only; the plans hold sizes and types.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <new>

#include "host_internal.h"
#include "layer_internal.h"

using namespace imm;

struct rms_norm_plan_s {
  int64_t rows, cols;
  int in, out;
  float eps;
};

struct w4_plan_s {
  int64_t M, N, K;
  int dtype, group;
  int64_t nblocks, kblocks, groups;  // of 16 outputs, of 128 K, of `group` K
};

namespace {

bool is_f8(int dt) { return dt == GEMM_F8_E4M3 || dt == GEMM_F8_E5M2; }
bool is_16bit(int dt) { return dt == GEMM_F16 || dt == GEMM_BF16; }
bool aligned(const void* p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}
// A required operand: present and aligned.
bool good(const void* p, unsigned bytes) { return p && aligned(p, bytes); }

gemm_status status_of(hipError_t e) { return e == hipSuccess ? GEMM_OK : record_hip_error(e); }

gemm_status check_rows(int64_t rows, int64_t cols, int in, int out) {
  if (rows < 0 || cols < 0) return GEMM_ERR_INVALID_VALUE;
  if (!is_16bit(in) || (out != in && !is_f8(out))) return GEMM_ERR_UNSUPPORTED;
  if (rows > INT_MAX || cols > kMaxRowCols || cols % (is_f8(out) ? 16 : 8) != 0)
    return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

}  // namespace

extern "C" {

gemm_status rms_norm_plan(int64_t rows, int64_t cols, gemm_dtype in, gemm_dtype out, float eps,
                          rms_norm_plan_t* plan) {
  if (!plan) return GEMM_ERR_INVALID_VALUE;
  *plan = nullptr;
  const gemm_status st = check_rows(rows, cols, in, out);
  if (st != GEMM_OK) return st;
  if (!std::isfinite(eps) || eps < 0.0f) return GEMM_ERR_UNSUPPORTED;
  rms_norm_plan_s* p = new (std::nothrow) rms_norm_plan_s{rows, cols, in, out, eps};
  if (!p) return GEMM_ERR_INVALID_VALUE;
  *plan = p;
  return GEMM_OK;
}

gemm_status rms_norm_run(rms_norm_plan_t p, const void* x, const void* residual,
                         const void* weight, void* out, float* row_scale, void* residual_out,
                         float* rstd, void* stream) {
  if (!p) return GEMM_ERR_INVALID_VALUE;
  // (rows without columns still have their values per row)
  const bool f8 = is_f8(p->out), any = p->cols > 0;
  if (p->rows == 0 || (!any && !row_scale && !rstd)) return GEMM_OK;
  if ((any && (!good(x, 16) || !good(out, 16))) || !aligned(weight, 16) || !aligned(rstd, 4))
    return GEMM_ERR_INVALID_VALUE;
  if (any && (!residual != !residual_out || !aligned(residual, 16) || !aligned(residual_out, 16)))
    return GEMM_ERR_INVALID_VALUE;
  if (f8 ? (any && !row_scale) || !aligned(row_scale, 4) : row_scale != nullptr)
    return GEMM_ERR_INVALID_VALUE;
  const size_t n = (size_t)p->rows * (size_t)p->cols;
  const size_t per_row = (size_t)p->rows * sizeof(float);
  const gemm_status st = check_device_operands({{any ? x : nullptr, 2 * n},
                                                {any ? residual : nullptr, 2 * n},
                                                {any ? weight : nullptr, 2 * (size_t)p->cols},
                                                {any ? out : nullptr, f8 ? n : 2 * n},
                                                {row_scale, per_row},
                                                {any ? residual_out : nullptr, 2 * n},
                                                {rstd, per_row}});
  if (st != GEMM_OK) return st;
  const RmsNormArgs a{x,    residual, weight,  out,     row_scale, residual_out,
                      rstd, p->rows,  p->cols, p->eps};
  return status_of(launch_rms_norm(p->in, p->out, true, a, static_cast<hipStream_t>(stream)));
}

size_t rms_norm_workspace_size(rms_norm_plan_t p) {
  if (!p || is_f8(p->out)) return 0;
  return (size_t)rms_norm_backward_groups(p->rows, p->cols) * (size_t)p->cols * sizeof(float);
}

gemm_status rms_norm_backward(rms_norm_plan_t p, const void* dy, const void* h,
                              const void* weight, const float* rstd, const void* dh, void* dx,
                              void* dweight, void* workspace, size_t workspace_bytes,
                              void* stream) {
  if (!p) return GEMM_ERR_INVALID_VALUE;
  if (is_f8(p->out)) return GEMM_ERR_UNSUPPORTED;
  if (p->cols == 0 || (p->rows == 0 && !dweight)) return GEMM_OK;
  if (!aligned(dweight, 16)) return GEMM_ERR_INVALID_VALUE;
  const size_t n = (size_t)p->rows * (size_t)p->cols, need = rms_norm_workspace_size(p);
  if (p->rows > 0) {
    if (!good(dy, 16) || !good(h, 16) || !aligned(weight, 16) || !good(rstd, 4) ||
        !aligned(dh, 16) || !good(dx, 16))
      return GEMM_ERR_INVALID_VALUE;
    if (dweight) {
      if (!workspace || workspace_bytes < need) return GEMM_ERR_WORKSPACE;
      if (!aligned(workspace, 16)) return GEMM_ERR_INVALID_VALUE;
    }
  }
  const bool any = p->rows > 0;
  const gemm_status st = check_device_operands({{any ? dy : nullptr, 2 * n},
                                                {any ? h : nullptr, 2 * n},
                                                {any ? weight : nullptr, 2 * (size_t)p->cols},
                                                {any ? rstd : nullptr, (size_t)p->rows * 4},
                                                {any ? dh : nullptr, 2 * n},
                                                {any ? dx : nullptr, 2 * n},
                                                {dweight, 2 * (size_t)p->cols},
                                                {any && dweight ? workspace : nullptr, need}});
  if (st != GEMM_OK) return st;
  const RmsNormBwdArgs a{dy, h,  weight, rstd,
                         dh, dx, any && dweight ? static_cast<float*>(workspace) : nullptr,
                         p->rows, p->cols};
  return status_of(launch_rms_norm_backward(p->in, a, dweight, static_cast<hipStream_t>(stream)));
}

void rms_norm_plan_destroy(rms_norm_plan_t p) { delete p; }

gemm_status quantize_rows(int64_t rows, int64_t cols, gemm_dtype in, gemm_dtype out, const void* x,
                          void* q, float* row_scale, void* stream) {
  if (!is_f8(out)) return GEMM_ERR_UNSUPPORTED;
  gemm_status st = check_rows(rows, cols, in, out);
  if (st != GEMM_OK) return st;
  const bool any = cols > 0;
  if (rows == 0 || (!any && !row_scale)) return GEMM_OK;
  if ((any && (!good(x, 16) || !good(q, 16))) || !good(row_scale, 4)) return GEMM_ERR_INVALID_VALUE;
  const size_t n = (size_t)rows * (size_t)cols;
  st = check_device_operands({{any ? x : nullptr, 2 * n},
                              {any ? q : nullptr, n},
                              {row_scale, (size_t)rows * sizeof(float)}});
  if (st != GEMM_OK) return st;
  const RmsNormArgs a{x,       nullptr, nullptr, q,   row_scale, nullptr,
                      nullptr, rows,    cols,    0.0f};
  return status_of(launch_rms_norm(in, out, false, a, static_cast<hipStream_t>(stream)));
}

gemm_status w4_plan(int64_t M, int64_t N, int64_t K, gemm_dtype dtype, int group, w4_plan_t* plan) {
  if (!plan) return GEMM_ERR_INVALID_VALUE;
  *plan = nullptr;
  if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_VALUE;
  if (!is_16bit(dtype) || (group != 32 && group != 64 && group != 128)) return GEMM_ERR_UNSUPPORTED;
  if (M > INT_MAX || N > INT_MAX || K > INT_MAX || N % 8 != 0 || K % group != 0)
    return GEMM_ERR_UNSUPPORTED;
  const int64_t nblocks = (N + 15) / 16, kblocks = (K + 127) / 128, groups = K / group;
  // fewer than 2^32 threads on tiles of 64 x 128, 31-bit counts of blocks and
  // groups, and the few-rows kernel's 31-bit offsets: 32 rows of x, a stage's
  // groups of scale words
  if ((M + 63) / 64 * ((N + 127) / 128) >= (int64_t)1 << 24 || nblocks * kblocks > INT_MAX ||
      nblocks * groups > INT_MAX || 64 * K > kMaxOffset || 512 * N > kMaxOffset)
    return GEMM_ERR_UNSUPPORTED;
  w4_plan_s* p = new (std::nothrow) w4_plan_s{M, N, K, dtype, group, nblocks, kblocks, groups};
  if (!p) return GEMM_ERR_INVALID_VALUE;
  *plan = p;
  return GEMM_OK;
}

size_t w4_packed_size(w4_plan_t p) {
  if (!p) return 0;
  return (size_t)p->nblocks * ((size_t)p->kblocks * 1024 + (size_t)p->groups * 64);
}

gemm_status w4_pack(w4_plan_t p, const void* q, const void* scales, const void* zeros,
                    void* packed, void* stream) {
  if (!p) return GEMM_ERR_INVALID_VALUE;
  if (p->N == 0 || p->K == 0) return GEMM_OK;
  if (!q || !good(scales, 2) || !good(packed, 16)) return GEMM_ERR_INVALID_VALUE;
  const size_t pairs = (size_t)p->N * (size_t)p->groups;
  const gemm_status st = check_device_operands({{q, (size_t)p->N * (size_t)p->K / 2},
                                                {scales, 2 * pairs},
                                                {zeros, pairs},
                                                {packed, w4_packed_size(p)}});
  if (st != GEMM_OK) return st;
  return status_of(launch_w4_pack(p->N, p->K, p->group, q, scales, zeros, packed,
                                  static_cast<hipStream_t>(stream)));
}

size_t w4_workspace_size(w4_plan_t p) {
  if (!p || p->N == 0 || !w4_uses_tiles(p->M, p->N, p->K, p->group)) return 0;
  return (size_t)p->groups * (size_t)((p->M + kW4RowPad - 1) / kW4RowPad * kW4RowPad) * 8;
}

gemm_status w4_run(w4_plan_t p, const void* x, const void* packed, const float* bias, void* y,
                   void* workspace, size_t workspace_bytes, void* stream) {
  if (!p) return GEMM_ERR_INVALID_VALUE;
  if (p->M == 0 || p->N == 0) return GEMM_OK;
  if (!good(y, 16) || !aligned(bias, 4)) return GEMM_ERR_INVALID_VALUE;
  const bool any = p->K > 0;
  if (any && (!good(x, 16) || !good(packed, 16))) return GEMM_ERR_INVALID_VALUE;
  const size_t need = w4_workspace_size(p);
  if (need) {
    if (!workspace || workspace_bytes < need) return GEMM_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return GEMM_ERR_INVALID_VALUE;
  }
  const size_t M = (size_t)p->M, N = (size_t)p->N, K = (size_t)p->K;
  const gemm_status st = check_device_operands({{any ? x : nullptr, 2 * M * K},
                                                {any ? packed : nullptr, w4_packed_size(p)},
                                                {bias, N * sizeof(float)},
                                                {y, 2 * M * N},
                                                {need ? workspace : nullptr, need}});
  if (st != GEMM_OK) return st;
  const char* const sz = static_cast<const char*>(packed) + p->nblocks * p->kblocks * 1024;
  const W4Args a{x,    packed, reinterpret_cast<const unsigned*>(any ? sz : nullptr),
                 bias, y,      p->M,
                 p->N, p->K,   p->nblocks,
                 p->kblocks,   p->groups,
                 p->group,     need ? workspace : nullptr,
                 (p->M + kW4RowPad - 1) / kW4RowPad * kW4RowPad,
                 0,            0,      0};
  return status_of(launch_w4(p->dtype, a, static_cast<hipStream_t>(stream)));
}

void w4_plan_destroy(w4_plan_t p) { delete p; }

}  // extern "C"
