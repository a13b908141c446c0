// Internal declarations of the calls around a linear layer (layer_api.cpp and
// its kernels).
#pragma once

#include "imm_internal.h"

namespace imm {

// Row kernels (rms_norm.hip).  cols is a multiple of 8, at most kMaxRowCols;
// every pointer is 16-byte aligned (row_scale, rstd: 4).
constexpr int64_t kMaxRowCols = 32768;  // 1024 threads of four 8-element vectors
// Workgroups of the backward pass (each leaves its parts of dw): two per
// compute unit of a 256-CU MI355X.
constexpr int64_t kRmsNormBwdGroups = 512;
struct RmsNormArgs {
  const void* x;
  const void* residual;  // or null
  const void* weight;    // or null: ones
  void* out;
  float* row_scale;      // fp8 outputs
  void* residual_out;    // with residual
  float* rstd;           // or null
  int64_t rows, cols;
  float eps;
};
struct RmsNormBwdArgs {
  const void* dy;
  const void* h;
  const void* weight;    // or null: ones
  const float* rstd;
  const void* dh;        // or null
  void* dx;
  float* parts;          // [rms_norm_backward_groups, cols], or null: no dw
  int64_t rows, cols;
};
// norm = false: the plain quantisation of rows (out is an fp8 type).
hipError_t launch_rms_norm(int in, int out, bool norm, const RmsNormArgs& a, hipStream_t s);
hipError_t launch_rms_norm_backward(int in, const RmsNormBwdArgs& a, void* dweight, hipStream_t s);
int64_t rms_norm_backward_groups(int64_t rows, int64_t cols);

// 4-bit weights (w4.hip).  packed: nblocks x kblocks blocks of 16 outputs x 128 K
// (1 KB each), followed by sz [groups, 16 nblocks].
struct W4Args {
  const void* x;         // [M, K]
  const void* packed;
  const unsigned* sz;
  const float* bias;     // fp32 [N] or null
  void* y;               // [M, N]
  int64_t M, N, K;
  int64_t nblocks, kblocks, groups;
  int group;
  // the tile kernel: sums of x per group as three bf16 pieces, 8 bytes each,
  // [groups, m_pad] (workspace; null selects the few-rows kernel), and its grid
  void* sums;
  int64_t m_pad;
  int64_t tiles_m, tiles_n, grid;
};
// Whether a product of M rows runs on the tile kernel (and needs the sums).
bool w4_uses_tiles(int64_t M, int64_t N, int64_t K, int group);
constexpr int64_t kMaxOffset = ((int64_t)1 << 31) - (1 << 16);
constexpr int64_t kW4RowPad = 128;  // rows of the largest tile; m_pad: M rounded up to it
hipError_t launch_w4_pack(int64_t N, int64_t K, int group, const void* q, const void* scales,
                          const void* zeros, void* packed, hipStream_t s);
hipError_t launch_w4(int in, const W4Args& a, hipStream_t s);

// Few fp8 rows with row and column scales (f8_rows.hip), bitwise equal to
// launch_gemm_scaled; whether a product runs there.
bool f8_rows_take(int64_t M, int64_t N, int64_t K);
hipError_t launch_f8_rows(int in, int out, const ScaledArgs& a, hipStream_t s);

}  // namespace imm
