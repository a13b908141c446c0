/*
 * invariant_matmul.h -- C ABI of a batch-invariant GEMM library for AMD
 * MI355X (gfx950).
 *
 * It computes C = scale_a * scale_b * (A x B) with A [M,K], B [K,N] and
 * C [M,N], all row-major and contiguous (leading dimensions K, N and N), from
 * fp16, bf16 or OCP fp8 (e4m3fn / e5m2) inputs with fp32 accumulation.  The
 * problem statement, the matrix shapes and the element formula follow the
 * Tencent engineer article on deterministic LLM inference ("AI インフラの深化：
 * 大規模モデルに確定的な出力を実現する方法"), section "Batch Invariance の由来"
 * (C = A x B with A [M,K], B [K,N]; C_ij is the dot product of row i of A and
 * column j of B over k).
 *
 * Batch invariance.  The same article (same section) shows that the
 * spatial tile sizes and the workgroup order do not change any bit, while the
 * reduction step and the split of K do.  This library therefore fixes the
 * matrix-core instruction per input dtype and fixes the K order, the K-step
 * and the split of K from (N, K, dtypes, explicit options) alone -- never
 * from M.  For one plan key the bits of row i of C are a function of row i of
 * A and of B only: they do not depend on M, on other rows, on concurrently
 * running work, on the stream or on how often the call has run.
 *
 * Calls, their passages (each call's own comment below repeats its passage):
 *   gemm_plan, gemm_plan_ex, gemm_plan_ex2
 *                     the problem statement C = A x B with A [M,K], B [K,N],
 *                     C [M,N] and a configuration fixed from (N, K, dtypes)
 *                     alone (article, section "Batch Invariance の由来"; section
 *                     "演算子チューニング" shows the M-driven tile and split
 *                     choices this planner does not make).
 *   gemm_plan_info    the configuration a plan fixed: BLOCK_M / BLOCK_N /
 *                     BLOCK_K, SPLIT_K, GROUP_M and the waves (the tuning
 *                     parameters of section "演算子チューニング").
 *   gemm_workspace_size
 *                     bytes of the [split_k, M, N] fp32 partial-sum workspace
 *                     (section "Split-K").
 *   gemm_plan_tile_of the workgroup -> output tile order (section "GROUP_M -
 *                     Swizzle L2 Cache").
 *   gemm_run          one workgroup per output tile running the K loop
 *                     (section "Tiling - 分塊行列乗算": accumulator init,
 *                     load/compute/accumulate per K step, one write-back);
 *                     tiles visited in GROUP_M order (section "GROUP_M -
 *                     Swizzle L2 Cache").
 *   gemm_run_bias, gemm_splitk_run_bias
 *                     the same plus the bias of a linear layer (the vLLM
 *                     batch-invariant linear operator listed in the article's
 *                     closing section).
 *   gemm_splitk_run   split-K through a [split_k, M, N] fp32 workspace and a
 *                     separate reduction kernel on the same stream, no atomics
 *                     (section "Split-K", the workspace variant).
 *   ozaki_*           the fp64 product by the Ozaki scheme (Insight Edge blog
 *                     on cuTile Python, section "倍精度行列積エミュレーション").
 *   gemm_plan_destroy, ozaki_plan_destroy, gemm_status_string,
 *   gemm_last_hip_error
 *                     library housekeeping (freeing a host plan, naming a
 *                     status, the last HIP error); no passage defines them.
 *
 * Conventions for every call:
 *   - All matrices and the workspace are DEVICE memory owned by the caller; the
 *     library never allocates device memory.  A plan is host memory owned by
 *     the caller (free it with gemm_plan_destroy).  Plans are immutable and
 *     may be used from several host threads / streams at once (each concurrent
 *     split-K call needs its own workspace).
 *   - `stream` is a hipStream_t passed as void* (NULL means the null stream),
 *     so that a caller needs no HIP header to include this one; a hipStream_t
 *     converts to void* implicitly in C and C++.  Run calls only enqueue work
 *     on it: they never synchronise the host.
 *   - Inputs are read-only.  C is fully overwritten (there is no beta).  The
 *     workspace holds no meaningful data after the call.
 *   - Every argument is validated before anything is enqueued (the checks
 *     that need no runtime come first, so they also run without a GPU); on
 *     error nothing is enqueued and C is untouched.  A status other than
 *     GEMM_OK is returned:
 *       GEMM_ERR_INVALID_VALUE  negative size, NULL pointer for a non-empty
 *                               operand, pointer not 16-byte aligned, NULL
 *                               plan or output handle; on a machine with a
 *                               GPU also an operand that does not lie
 *                               wholly inside one device allocation of the
 *                               current device (host memory, another
 *                               device's memory, or a buffer shorter than
 *                               the operand), checked with the runtime's
 *                               pointer queries before anything is enqueued;
 *       GEMM_ERR_UNSUPPORTED    unsupported dtype pair, N or K not a multiple of
 *                               16 bytes' worth of elements (8 for 16-bit
 *                               inputs, 16 for fp8), bad option value;
 *       GEMM_ERR_WORKSPACE      workspace NULL or smaller than
 *                               gemm_workspace_size();
 *       GEMM_ERR_HIP            no usable GPU, or a launch failed (the HIP
 *                               error is then available from hipGetLastError
 *                               semantics inside the library: call
 *                               gemm_last_hip_error() for its code).
 *   - Empty products: M == 0 or N == 0 enqueue nothing and return GEMM_OK;
 *     K == 0 writes C = 0.
 */
#ifndef INVARIANT_MATMUL_H
#define INVARIANT_MATMUL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  GEMM_OK = 0,
  GEMM_ERR_INVALID_VALUE = 1,
  GEMM_ERR_UNSUPPORTED = 2,
  GEMM_ERR_WORKSPACE = 3,
  GEMM_ERR_HIP = 4
} gemm_status;

/* Element types.  Inputs: F16, BF16, F8_E4M3 (OCP e4m3fn), F8_E5M2 (OCP e5m2).
 * Outputs: F32, BF16 or F16 (round to nearest, ties to even; fp16 keeps
 * subnormals and overflows to infinity). */
typedef enum {
  GEMM_F16 = 0,
  GEMM_BF16 = 1,
  GEMM_F8_E4M3 = 2,
  GEMM_F8_E5M2 = 3,
  GEMM_F32 = 4,
  GEMM_I8 = 5   /* int8, as Ozaki-scheme slices only (ozaki_plan) */
} gemm_dtype;

/* Output-tile shapes (rows x columns of C per workgroup).  All tiles of one
 * input dtype use the same matrix-core instruction and the same K order, so
 * for a fixed split of K they produce identical bits; the choice only moves
 * work in space. */
typedef enum {
  GEMM_TILE_DEFAULT = 0,    /* chosen from (N, K, dtype) */
  GEMM_TILE_256x256 = 1,    /* 8 waves, LDS ring filled by buffer->LDS DMA */
  GEMM_TILE_128x128 = 2,    /* 4 waves, register-staged LDS tiles */
  GEMM_TILE_32x128 = 3,     /* 4 waves, register-staged LDS tiles */
  GEMM_TILE_256x256_RS = 4, /* 8 waves, register-staged LDS tiles */
  GEMM_TILE_32x256 = 5,     /* 4 waves, DMA ring; narrow tile for skinny or
                               reduction-dominated shapes */
  GEMM_TILE_64x256 = 6,     /* 4 waves, DMA ring */
  GEMM_TILE_128x256 = 7,    /* 8 waves, DMA ring of 3 stages */
  GEMM_TILE_32x64 = 8,      /* 2 waves, DMA ring of 3 stages of 256 bytes of
                               K (two workgroups per compute unit); fp16 /
                               bf16 only: narrow tile for small M (4x the
                               workgroups of 32x256) */
  GEMM_TILE_64x64 = 9,      /* 2 waves, DMA ring of 2 stages of 256 bytes of
                               K (two workgroups per compute unit); fp16 /
                               bf16 only */
  GEMM_TILE_32x32 = 10      /* 2 waves, DMA ring of 3 stages of 256 bytes of
                               K (three workgroups per compute unit); fp16 /
                               bf16 only: twice the workgroups of 32x64 for
                               small M */
} gemm_tile;

/* Plan flags (gemm_plan_ex2). */
typedef enum {
  /* B is given transposed: a [N, K] row-major matrix W with B = W^T (the
   * weight layout of a linear layer, y = x W^T + b, as in the vLLM
   * batch-invariant operators the Tencent article lists in its closing
   * section).  Only the DMA tiles (256x256, 128x256, 64x256, 32x256, 64x64, 32x64,
   * 32x32) read this layout;
   * the bits of C are those of the [K, N] layout holding the same values. */
  GEMM_PLAN_B_TRANSPOSED = 1,
  /* gemm_run / gemm_run_bias with the 256x256 tile launch at most one
   * workgroup per compute unit, each walking the tiles of the one-tile-per-
   * workgroup grid in the same raster order, with its LDS pipeline running
   * on from one tile into the next (the persistent batch-invariant matmul of
   * the Tencent article's closing section).  The bits of C are those of the
   * plan without the flag; other tiles and the split-K path ignore it. */
  GEMM_PLAN_PERSISTENT = 2,
  /* gemm_run / gemm_run_bias take their tile from M instead of from (N, K,
   * dtype): the DMA tile (32x32, 32x64, 64x64, 32x256, 64x256, 128x256 or
   * 256x256; fp8 inputs skip the first three) with the least estimated time,
   * rounds of 256 workgroups times a per-tile time that grows with the
   * tile's size.  gemm_splitk_run of a wide reduction-dominated shape
   * (K >= 2N, N > 512) takes from M the tile with the fewest row tiles (32-row,
   * 64x256, 128x256 or 256x256); the split of K stays the one (N, K, dtype)
   * gives.  Every tile uses the same matrix-core instruction and K order, so
   * C is bitwise that of the plan without the flag for every M (tile sizes do
   * not change bits: the Tencent article, "Batch Invariance の由来"); only the
   * time changes.  An explicit tile, and the split-K path of other shapes,
   * ignore it. */
  GEMM_PLAN_TILE_BY_M = 4,
  /* fp8 inputs (GEMM_F8_E4M3, GEMM_F8_E5M2) only: every fp8 value is widened
   * to fp16 in registers (exactly: both formats are subsets of fp16) and the
   * products are accumulated by the 16x16x32 fp16 matrix-core step in fp32,
   * in ascending K, instead of by the 16x16x128 fp8 step.  The fp8 step adds
   * each group of 8 consecutive products in a window that drops what lies
   * more than 13 binades below the group's largest product, so its error is
   * bounded by K * 2^-24 * sum |a||b| (the fp32 accumulation the Tencent
   * article's "背景" assumes) only for long K or benign inputs; with this flag
   * that bound holds for every K and every input.  The bits are this mode's
   * own (equal to those of the fp8 step only where no product is dropped) and
   * are batch-invariant by the same rule as every plan: one instruction and
   * one K order for every tile and M.  It runs the fp8 data at the fp16
   * matrix rate.  DMA tiles only: an explicit register-staged tile, or a K so
   * large that the DMA tiles' 32-bit offsets overflow, gives
   * GEMM_ERR_UNSUPPORTED, as does another input dtype. */
  GEMM_PLAN_FP8_FP32_ACCUM = 8
} gemm_plan_flags;

typedef struct gemm_plan_s* gemm_plan_t;

/* A plan holds one tile for each entry point: tile / block_m / block_n /
 * waves / tiles_m / tiles_n describe gemm_splitk_run's partial kernel, the
 * run_* fields gemm_run's single pass.  Both are chosen from (N, K, dtype,
 * options) alone (with GEMM_PLAN_TILE_BY_M, also from M), and the bits of C
 * depend on neither: only split_k and k_per_split, which never depend on M,
 * decide them. */
typedef struct {
  int64_t M, N, K;
  int32_t in_dtype, out_dtype;  /* gemm_dtype values */
  int32_t tile;                 /* gemm_tile value of the split-K path */
  int32_t block_m, block_n;     /* its output tile */
  int32_t block_k;              /* K elements staged per main-loop step */
  int32_t mfma_m, mfma_n, mfma_k; /* matrix-core instruction shape */
  int32_t waves;                /* 64-lane wavefronts per workgroup (split-K path) */
  int32_t group_m;              /* GROUP_M of the tile raster */
  int32_t split_k;              /* K slices used by gemm_splitk_run */
  int64_t k_per_split;          /* K elements per slice (multiple of block_k) */
  int64_t tiles_m, tiles_n;     /* output tiles along M and N (split-K path) */
  int64_t grid_run;             /* workgroups launched by gemm_run */
  int64_t grid_splitk;          /* workgroups of the split-K partial kernel */
  uint64_t workspace_bytes;     /* split_k * M * N * 4 */
  float scale_a, scale_b;
  int32_t run_tile;             /* gemm_tile value of gemm_run */
  int32_t run_block_m, run_block_n;
  int32_t run_waves;
  int64_t run_tiles_m, run_tiles_n;
} gemm_plan_info_t;

/* Plan C[M,N] = A[M,K] x B[K,N] (Tencent article, "Batch Invariance の由来":
 * the problem statement, and the conclusion that the K step and the split of
 * K must not follow the batch size) with default options: fp32 output for
 * fp16 / bf16 inputs and bf16 output for fp8 inputs, split and tile chosen
 * from (N, K, dtype), GROUP_M = 8, scales 1.0.  M only sizes the grid and the
 * workspace.  On success *out receives a new plan (host memory; free it with
 * gemm_plan_destroy). */
gemm_status gemm_plan(int64_t M, int64_t N, int64_t K, gemm_dtype in, gemm_plan_t* out);

/* As gemm_plan with explicit options (same passage).  out_dtype: GEMM_F32,
 * GEMM_BF16 or GEMM_F16.
 * split_k: 0 = default, else 1..4096 (the slice length is rounded up to a
 * multiple of block_k; the split actually used is reported by
 * gemm_plan_info).  group_m: 0 = default (8), else >= 1.  scale_a, scale_b:
 * per-tensor scales multiplied into the result (their fp32 product is applied
 * to the fp32 sum before the output conversion); must be finite. */
gemm_status gemm_plan_ex(int64_t M, int64_t N, int64_t K, gemm_dtype in, gemm_dtype out,
                         int split_k, int group_m, float scale_a, float scale_b,
                         gemm_plan_t* plan);

/* As gemm_plan_ex with an explicit output tile and plan flags (same passage;
 * the tile is the article's BLOCK_M / BLOCK_N, which it shows changes no bit).
 * tile: a gemm_tile value (GEMM_TILE_DEFAULT: chosen from (N, K, dtype)).
 * flags: a bitwise OR of gemm_plan_flags; unknown bits give
 * GEMM_ERR_UNSUPPORTED.  With GEMM_PLAN_B_TRANSPOSED, B is read as [N, K]
 * row-major; an explicit register-staged tile, or a K so large that the DMA
 * tiles' 32-bit offsets overflow, gives GEMM_ERR_UNSUPPORTED. */
gemm_status gemm_plan_ex2(int64_t M, int64_t N, int64_t K, gemm_dtype in, gemm_dtype out,
                          int split_k, int group_m, int tile, float scale_a, float scale_b,
                          unsigned flags, gemm_plan_t* plan);

/* The configuration a plan fixed (Tencent article, "演算子チューニング": the
 * tile sizes, the K step, SPLIT_K and GROUP_M of its parameter table), into
 * *info.  Pure host call.  GEMM_ERR_INVALID_VALUE for a NULL argument. */
gemm_status gemm_plan_info(gemm_plan_t plan, gemm_plan_info_t* info);

/* Bytes of workspace gemm_splitk_run needs: split_k * M * N * sizeof(float),
 * the [split_k, M, N] fp32 partial sums (Tencent article, "Split-K").  0 for
 * a NULL plan. */
size_t gemm_workspace_size(gemm_plan_t plan);

/* Tile raster: the (k_slice, pid_m, pid_n) that workgroup `workgroup` of the
 * split-K partial kernel computes (k_slice is 0 for gemm_run's grid), after
 * the XCD remap and the GROUP_M order (Tencent article, "GROUP_M - Swizzle L2
 * Cache").  Pure host function, exposed so the raster can be checked to be a
 * bijection.  GEMM_ERR_INVALID_VALUE for a workgroup outside the grid. */
gemm_status gemm_plan_tile_of(gemm_plan_t plan, int64_t workgroup, int64_t* k_slice,
                              int64_t* pid_m, int64_t* pid_n);

/* C = A x B in one pass: one workgroup per output tile, full K in order
 * (Tencent article, "Tiling - 分塊行列乗算").  A, B, C: device memory,
 * row-major, 16-byte aligned; enqueued on `stream`. */
gemm_status gemm_run(gemm_plan_t plan, const void* A, const void* B, void* C, void* stream);

/* As gemm_run plus a bias: C[i, j] = convert(scale * sum_ij + bias[j]), one
 * fp32 add after the scale.  bias: device fp32 [N], 4-byte aligned, or NULL
 * (then exactly gemm_run).  The bias term of a linear layer (the vLLM
 * batch-invariant linear operator in the Tencent article's closing section). */
gemm_status gemm_run_bias(gemm_plan_t plan, const void* A, const void* B, const float* bias,
                          void* C, void* stream);

/* C = A x B through the split-K workspace (Tencent article, "Split-K", the
 * workspace variant): the partial kernel writes slice s of K to
 * workspace[s, :, :] (fp32, no atomics), then a reduction kernel sums the
 * slices in ascending s and writes C.  With split_k == 1 the result is
 * bitwise identical to gemm_run.  workspace: device memory of at least
 * gemm_workspace_size(plan) bytes, 16-byte aligned, owned by the caller. */
gemm_status gemm_splitk_run(gemm_plan_t plan, const void* A, const void* B, void* C,
                            void* workspace, size_t workspace_bytes, void* stream);

/* As gemm_splitk_run plus a bias, added by the reduction kernel after the
 * ascending-slice sum and the scale (same rule as gemm_run_bias). */
gemm_status gemm_splitk_run_bias(gemm_plan_t plan, const void* A, const void* B,
                                 const float* bias, void* C, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* As gemm_run_bias with one scale per row of A and one per column of B, the
 * product of fp8 rows that carry their scales (activations
 * from rms_norm_run or quantize_rows, weights [N, K] with a scale per output):
 *   C[i, j] = convert(((scale sum_ij) row_scale[i]) col_scale[j] + bias[j]),
 * each product and the sum rounded in fp32.  row_scale: device fp32 [M],
 * col_scale: device fp32 [N], 4-byte aligned, both required.  Plans with fp8
 * inputs and GEMM_PLAN_B_TRANSPOSED only (GEMM_ERR_UNSUPPORTED otherwise);
 * GEMM_PLAN_PERSISTENT is ignored.  sum_ij is the fp8 step's (8 neighbouring products
 * in a window of 13 binades, then fp32), or with GEMM_PLAN_FP8_FP32_ACCUM the fp16
 * step's, on the tiles at every M.  Few rows, and the few rows that tiles would
 * leave for another round, run on a kernel of their own with the same bits.  No
 * passage of the pages defines them. */
gemm_status gemm_run_scaled(gemm_plan_t plan, const void* A, const void* B, const float* row_scale,
                            const float* col_scale, const float* bias, void* C, void* stream);

/* Frees a host plan (NULL is ignored).  Housekeeping: no passage. */
void gemm_plan_destroy(gemm_plan_t plan);

/* The largest split-K workspace gemm_splitk_run_noalloc serves: 64 MiB (for
 * example the decode product 128 x 4096 x 14336 bf16 at its default 16 slices
 * needs 32 MiB; 256 x 4096 x 14336 needs 64 MiB exactly). */
#define GEMM_NOALLOC_WORKSPACE_BYTES ((size_t)64 << 20)

/* For callers that cannot allocate device memory -- code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc: as
 * gemm_splitk_run, with the [split_k, M, N] fp32 workspace taken from an array
 * inside the library instead of from the caller.  The library holds one such
 * array of GEMM_NOALLOC_WORKSPACE_BYTES on every GPU it runs on, from the
 * first call on that GPU until the process ends; the call itself allocates
 * nothing.  C is bitwise what gemm_splitk_run gives for the same plan.
 * Errors: as gemm_splitk_run; GEMM_ERR_WORKSPACE if gemm_workspace_size(plan)
 * exceeds GEMM_NOALLOC_WORKSPACE_BYTES (nothing is enqueued).  All calls on
 * one GPU share its array: calls that overlap on one GPU (other streams or
 * host threads) race and must be serialised by the caller. */
gemm_status gemm_splitk_run_noalloc(gemm_plan_t plan, const void* A, const void* B, void* C,
                                    void* stream);

/* ---------------------------------------------------------------------------
 * fp64 matrix product by the Ozaki scheme: C = A x B with A [M,K], B [K,N]
 * and C [M,N] in fp64 (row-major, contiguous), computed on the matrix cores
 * from low-precision slices: bf16 or fp8 e4m3 with fp32 accumulation, or
 * int8 with int32 accumulation.  Insight Edge blog on
 * cuTile Python, section "倍精度行列積エミュレーション":
 *   split ("分解(Split)", equations (1)-(5)): every row of A and every column
 *     of B is cut into `slices` Type2 slices (bf16, fp8 e4m3 or int8) with
 *     c0 = ceil(log2 max|x|) of that row / column, c_p = c0 - p*delta,
 *     sigma = 0.75*2^(rho+c_p), v = (x+sigma)-sigma, x -= v,
 *     slice_p = Type2(v*2^-c_p);
 *   product ("行列積の計算", equations (10), (11)): for each slice pair (p,q),
 *     p ascending then q ascending, without the pairs with p+q >= d ("Fast
 *     Mode（GEMMの削減）"), the fp32 product of the two slices, scaled by
 *     2^(c_p(row) + c_q(column)), is added to an fp64 sum starting at +0.
 * K is cut into chunks of `chunk` products; for each pair the exact fp32
 * product of every chunk is added to the fp64 sum in ascending chunk order
 * (the page's exactness argument in "最適化後の結果" is per K tile).
 * Precision parameter ("分解(Split)"): rho = max(gamma, xi),
 * gamma = ceil(53 - (m_Type3 - log2 k)/2), xi = 53 - m_Type2 (m_Type2 = 8 for
 * bf16, 4 for e4m3, 6 for int8 -- an int8 entry n * 2^-b needs |n| <= 2^b <=
 * 127; m_Type3 = 24 for fp32, 31 for int32 accumulation), with k = min(K,
 * chunk) the length of one accumulation chain.  A slice
 * carries b = 53 - rho bits, so every fp32 chunk product is exact and the
 * result does not depend on any summation order inside the matrix cores: it
 * is a bitwise function of row i of A, of B, of K and of (type2, slices, d,
 * chunk).  delta = b + 1.
 * Defaults: chunk = 2^(m_Type3 - 2 m_Type2), the longest exact chain with
 * all of Type2's bits (256 for bf16, 65536 for e4m3, 2^19 for int8);
 * slices = min(ceil(53 / b), 20) (7 for bf16, 14 for e4m3, 9 for int8; 20 is
 * the most the page's split routine makes),
 * d = slices + 2 (39 products for 7 bf16 slices, 130 for 14 e4m3 slices, the
 * page's "最適化後の結果" tables; 60 for 9 int8 slices).
 * Domain: finite inputs whose nonzero row / column maxima lie in
 * [2^-300, 2^300].  There every slice value, scaled term and partial sum is
 * a normal fp64 number, so the kernel may apply 2^(c0(row) + c0(column)) once
 * at the end instead of to every term without changing a bit.  A row of A or
 * a column of B outside it (holding a NaN or an infinity, a magnitude above
 * 2^300, or a nonzero maximum below 2^-300) gets the exponent -2^30 in the
 * workspace and zero slices, and its whole row / column of C is NaN; every
 * other entry of C is unaffected (no error is reported).
 *
 * Workspace (device memory, caller-owned, 16-byte aligned, at least
 * ozaki_workspace_size bytes), with the offsets that ozaki_plan_info reports:
 *   a_slices  [slices, M, k_pad] Type2, row-major (k_pad = K rounded up to 16)
 *   b_slices  [slices, k_pad, n_pad] Type2 (n_pad = N rounded up to 16)
 *   a_exp     [M] int32 c0 of each row of A
 *   b_exp     [n_pad] int32 c0 of each column of B
 *   scratch   column maxima of B
 * Padding entries of the slices are zero.  The contents stay valid after a
 * call until the workspace is used again.
 * ------------------------------------------------------------------------- */
typedef struct ozaki_plan_s* ozaki_plan_t;

typedef struct {
  int64_t M, N, K;
  int32_t type2;              /* GEMM_BF16, GEMM_F8_E4M3 or GEMM_I8 */
  int32_t rho, bits, delta;   /* precision parameter, bits per slice, exponent step */
  int32_t slices, d, pairs;   /* slices per operand, Fast Mode threshold, products */
  int64_t chunk;              /* products per exact fp32 chain */
  int32_t tile_m, tile_n;     /* output tile of the product kernel */
  int64_t k_pad, n_pad;
  int64_t grid;               /* workgroups of the product kernel */
  uint64_t workspace_bytes;
  uint64_t a_slices_offset, b_slices_offset, a_exp_offset, b_exp_offset, scratch_offset;
} ozaki_plan_info_t;

/* Plan an Ozaki-scheme product.  type2: GEMM_BF16, GEMM_F8_E4M3 or GEMM_I8.
 * slices: 0 = default, else 1..20; d: 0 = default, else >= 1; chunk: 0 =
 * default, else a multiple of 128 (at most 2^22).  M, N, K >= 0; K below 2^23
 * (bf16), 2^25 (e4m3) or 2^24 (int8), N below 2^23 (32-bit offsets inside one
 * tile).
 * Errors: GEMM_ERR_INVALID_VALUE (negative size, NULL
 * handle), GEMM_ERR_UNSUPPORTED (other type2, slices, d or chunk out of range,
 * sizes too large). */
gemm_status ozaki_plan(int64_t M, int64_t N, int64_t K, gemm_dtype type2, int slices, int d,
                       int64_t chunk, ozaki_plan_t* plan);

gemm_status ozaki_plan_info(ozaki_plan_t plan, ozaki_plan_info_t* info);

size_t ozaki_workspace_size(ozaki_plan_t plan);

/* The split of one operand into the workspace: operand 0 = A (x is [M, K]),
 * 1 = B (x is [K, N]); x is device fp64, 8-byte aligned.  Enqueues the
 * exponent and split kernels on `stream`. */
gemm_status ozaki_split(ozaki_plan_t plan, int operand, const double* x, void* workspace,
                        size_t workspace_bytes, void* stream);

/* The slice-pair product from a workspace holding both operands' slices and
 * exponents (after ozaki_split of A and of B): writes C (device fp64 [M, N],
 * 8-byte aligned). */
gemm_status ozaki_multiply(ozaki_plan_t plan, const void* workspace, size_t workspace_bytes,
                           double* C, void* stream);

/* ozaki_split(A), ozaki_split(B), ozaki_multiply on one stream. */
gemm_status ozaki_run(ozaki_plan_t plan, const double* A, const double* B, double* C,
                      void* workspace, size_t workspace_bytes, void* stream);

void ozaki_plan_destroy(ozaki_plan_t plan);

/* ---------------------------------------------------------------------------
 * Root-mean-square norm of rows, with the residual's addition, and fp8 rows
 * with a scale each: what stands in front of a linear layer.  x is
 * [rows, cols] row-major and contiguous, fp16 or bf16; cols a multiple of 8
 * (16 for fp8 outputs, the K rule of the fp8 product) and at most 32768.
 *   h = round(x + residual), the residual stream in its own type (h = x
 *       without a residual);
 *   rstd = 1 / sqrt(sum_k h_k^2 / cols + eps), t_k = (h_k rstd) weight_k, fp32;
 *   out = round(t) in the input's type, or, with an fp8 output,
 *   row_scale = max(max_k |t_k| / FMAX, 2^-120), FMAX = 448 (e4m3) or 57344
 *       (e5m2), and out = round8(t / row_scale), both quotients rounded in fp32: the
 *       row is out * row_scale.
 * Row i of every output is a bitwise function of row i of the inputs, the
 * weight, cols and eps.  Sums are fp32; where a row's sum of squares would leave
 * fp32's range, its values are multiplied by a power of two first, so finite rows of
 * every magnitude have the formula's result.  (rstd itself is an fp32 number: above
 * 2^126 it keeps 21 bits or more, and with eps = 0 it is infinite for a row whose root
 * mean square is below 2^-128: out is right there, gradients are not finite.)
 * A row that holds a NaN or an infinity is NaN where
 * the formula is (a 16-bit output), or NaN throughout (an fp8 output, whose
 * row_scale is then infinite or NaN); other rows are unaffected.  Rows without
 * columns (cols = 0) have row_scale = 2^-120, the scale of a row of zeros, and
 * rstd = NaN, 0 / 0; their matrices, weight and row_scale may then be NULL.
 * No passage of the pages defines these calls.
 * ------------------------------------------------------------------------- */
typedef struct rms_norm_plan_s* rms_norm_plan_t;

/* Plan a norm.  in: GEMM_F16 or GEMM_BF16; out: the same type, GEMM_F8_E4M3 or
 * GEMM_F8_E5M2; eps finite and >= 0.  GEMM_ERR_INVALID_VALUE for a negative
 * size or a NULL handle, GEMM_ERR_UNSUPPORTED for other types, cols or eps. */
gemm_status rms_norm_plan(int64_t rows, int64_t cols, gemm_dtype in, gemm_dtype out, float eps,
                          rms_norm_plan_t* plan);

/* The norm, on `stream`.  residual and residual_out: [rows, cols] in the input's
 * type, both NULL or both given (residual_out receives h and may be x or
 * residual itself; no other operands may overlap).  weight: [cols] in the
 * input's type, or NULL for ones.  row_scale: fp32 [rows], for fp8 outputs
 * (NULL otherwise).  rstd: fp32 [rows] for the backward pass, or NULL.
 * Matrices and weight are 16-byte aligned, row_scale and rstd 4-byte. */
gemm_status rms_norm_run(rms_norm_plan_t plan, const void* x, const void* residual,
                         const void* weight, void* out, float* row_scale, void* residual_out,
                         float* rstd, void* stream);

/* Bytes of workspace rms_norm_backward needs for the weight's gradient (the
 * fp32 sums of row groups).  0 for a NULL plan. */
size_t rms_norm_workspace_size(rms_norm_plan_t plan);

/* Gradients of the norm (plans with a 16-bit output).  dy: the gradient of out;
 * h: the residual stream the norm read (residual_out, or x without a
 * residual); rstd: as rms_norm_run left it; dh: the gradient that reaches h from
 * elsewhere, or NULL.  With n = h rstd and g = weight dy:
 *   dx = round(rstd (g - n sum_j(g_j n_j) / cols) + dh),
 * the gradient of x and of the residual alike, and
 *   dweight = round(sum over rows of dy n), [cols] in the input's type, or NULL
 * (then no workspace is needed).  dx may be dy or dh itself.  dweight sums the
 * rows in an order that (rows, cols) fix, without atomics; dx is a function of
 * its row alone. */
gemm_status rms_norm_backward(rms_norm_plan_t plan, const void* dy, const void* h,
                              const void* weight, const float* rstd, const void* dh, void* dx,
                              void* dweight, void* workspace, size_t workspace_bytes,
                              void* stream);

void rms_norm_plan_destroy(rms_norm_plan_t plan);

/* The fp8 rows of x [rows, cols] alone: t = x in the formula above (activations
 * that no norm precedes, or a weight [N, K] with a scale per output). */
gemm_status quantize_rows(int64_t rows, int64_t cols, gemm_dtype in, gemm_dtype out, const void* x,
                          void* q, float* row_scale, void* stream);

/* ---------------------------------------------------------------------------
 * Linear layer with 4-bit weights and group scales: y = x W^T + bias with
 *   W[n, k] = scale[n, g] (q[n, k] - zero[n, g]), g = k / group,
 * q in 0..15.  x [M, K] and y [M, N] are fp16 or bf16, row-major, contiguous;
 * N a multiple of 8, K a multiple of group, group 32, 64 or 128.  The sums of
 * a group run over x and the integers q on the matrix cores in fp32:
 *   X = sum_k x;  P = -zero X + sum_k x q;  acc = fma(scale, P, acc)
 * with the groups in ascending order, and y = round(acc + bias): no weight is
 * rounded.  P is a difference of two fp32 sums: its error goes with sum_k |x| (q + zero)
 * (x with q = zero throughout need not give 0), and bf16 x for which that passes 2^128
 * overflows.  Row i of y is a bitwise function of row i of x, of the weights and
 * bias, N, K and group.  A row of x that holds a NaN or an infinity has no
 * finite element in y.  No passage of the pages defines these calls.
 * ------------------------------------------------------------------------- */
typedef struct w4_plan_s* w4_plan_t;

/* Plan y[M, N] = x[M, K] W^T.  dtype: GEMM_F16 or GEMM_BF16 (of x, the scales
 * and y).  GEMM_ERR_INVALID_VALUE for a negative size or a NULL handle,
 * GEMM_ERR_UNSUPPORTED for other types, groups or sizes (N up to
 * 4194176 and K up to 33553408, fewer than 2^24 tiles of 64 x 128 outputs and
 * 2^31 blocks of 16 x 128 weights and pairs of an output block and a group). */
gemm_status w4_plan(int64_t M, int64_t N, int64_t K, gemm_dtype dtype, int group, w4_plan_t* plan);

/* Bytes of the packed weight, which (N, K, group) alone fix: any plan with
 * the same N, K, dtype and group reads it, whatever its M.  0 for a NULL plan. */
size_t w4_packed_size(w4_plan_t plan);

/* Lays a weight out for w4_run, once.  q: [N, K / 2] bytes, byte j of a row
 * holding element 2 j in its low and 2 j + 1 in its high half; scales:
 * [N, K / group] of the plan's dtype; zeros: [N, K / group] bytes, or NULL for 8
 * (symmetric weights).  packed: w4_packed_size(plan) bytes, 16-byte aligned
 * (scales 2-byte). */
gemm_status w4_pack(w4_plan_t plan, const void* q, const void* scales, const void* zeros,
                    void* packed, void* stream);

/* Bytes of workspace w4_run needs (the sums of x per group, for many rows; 0
 * for few rows or a NULL plan). */
size_t w4_workspace_size(w4_plan_t plan);

/* y = x W^T + bias on `stream`.  x, packed and y 16-byte aligned; bias: fp32
 * [N], 4-byte aligned, or NULL; workspace: w4_workspace_size(plan) bytes,
 * 16-byte aligned (NULL where that is 0). */
gemm_status w4_run(w4_plan_t plan, const void* x, const void* packed, const float* bias, void* y,
                   void* workspace, size_t workspace_bytes, void* stream);

void w4_plan_destroy(w4_plan_t plan);

/* ---------------------------------------------------------------------------
 * Norm and rotation of the query and key heads: what stands between the
 * projection of a layer's input and attention.  For every token t and head,
 *   n = x / sqrt(sum_d x_d^2 / dim + eps), y = n weight (y = x without the norm),
 *   angle_i = positions[axis(i), t] inv_freq[i] for i < rot / 2, in fp64,
 *   (z_a, z_b) = (y_a cos - y_b sin, y_b cos + y_a sin) with (a, b) =
 *       (i, i + rot / 2), or (2 i, 2 i + 1) if interleaved,
 *   z_d = y_d from rot on, out = round(z).
 * axis(i): the frequencies are cut into `axes` sections (time, height, width of a
 * video; one axis for text), and those of section s turn by positions[s].
 * q and k are fp16 or bf16, element d of head h of token t at
 * t token_stride + h head_stride + d (strides in elements, multiples of 8: both may lie in
 * the output of a fused projection).  The outputs are contiguous [tokens, heads, dim].
 * Sums are fp32 and out is rounded once.  A head of the result is a bitwise function of
 * that head, its position, the weight and the sizes.  No passage of the pages
 * defines these calls.
 * ------------------------------------------------------------------------- */
typedef struct head_rope_plan_s* head_rope_plan_t;

/* Plan the call.  dim a multiple of 8 up to 512, rot a multiple of 16 up to dim (0: no
 * rotation); norm: 0 or 1; eps finite and >= 0; axes 1 to 4, sections: the frequencies
 * of each axis, which add up to rot / 2 (NULL for one axis).
 * GEMM_ERR_INVALID_VALUE for a negative size, sections that do not add up or a NULL
 * handle, GEMM_ERR_UNSUPPORTED for other types or sizes. */
gemm_status head_rope_plan(int64_t tokens, int q_heads, int k_heads, int dim, int rot,
                           gemm_dtype dtype, int norm, float eps, int interleaved, int axes,
                           const int* sections, head_rope_plan_t* plan);

/* The outputs, on `stream`.  positions: int64 [axes, tokens]; inv_freq: fp64 [rot / 2];
 * weights: [dim] in the input's type, or NULL for ones (NULL without the norm).
 * Tensors of heads and weights are 16-byte aligned.  No operand may overlap an output. */
gemm_status head_rope_run(head_rope_plan_t plan, const void* q, int64_t q_token_stride,
                          int64_t q_head_stride, const void* k, int64_t k_token_stride,
                          int64_t k_head_stride, const int64_t* positions, const double* inv_freq,
                          const void* q_weight, const void* k_weight, void* q_out, void* k_out,
                          void* stream);

/* Bytes of workspace head_rope_backward needs for the weights' gradients; 0
 * without the norm or for a NULL plan. */
size_t head_rope_workspace_size(head_rope_plan_t plan);

/* The gradients: dq_out and dk_out, those of the outputs, contiguous; dq and dk, those of q
 * and k, contiguous; dq_weight and dk_weight: [dim] in the input's type, each may be
 * NULL (both: no workspace is needed).  q and k are read with the norm only.
 * The weights' gradients sum tokens and heads in an order that the sizes fix, without atomics. */
gemm_status head_rope_backward(head_rope_plan_t plan, const void* dq_out, const void* dk_out,
                               const void* q, int64_t q_token_stride, int64_t q_head_stride,
                               const void* k, int64_t k_token_stride, int64_t k_head_stride,
                               const int64_t* positions, const double* inv_freq,
                               const void* q_weight, const void* k_weight, void* dq, void* dk,
                               void* dq_weight, void* dk_weight, void* workspace,
                               size_t workspace_bytes, void* stream);

void head_rope_plan_destroy(head_rope_plan_t plan);

/* ---------------------------------------------------------------------------
 * Attention of packed sequences:
 *   o_i = sum_j p_ij v_j,  p_ij = e^(scale q_i k_j) / e^lse_i,
 *   lse_i = ln sum_j e^(scale q_i k_j)
 * over the keys j that query i sees.  Sequence b has the n queries cu_q[b] ..
 * cu_q[b + 1] - 1 and the m keys from cu_k[b] on: up to cu_k[b + 1], or k_lens[b]
 * of them (a cache with room).  With `causal`, query i of n sees the keys j <= m - n + i,
 * otherwise all; query head h uses key head h / (q_heads / k_heads).  A
 * query without keys has o = 0 and lse = -infinity, also a row of q in no sequence.
 *
 * q [q_rows, q_heads, dim], k and v [k_rows, k_heads, dim] are fp16 or bf16 with
 * strides as above; dim a multiple of 8 up to 128.  o is contiguous, lse fp32
 * [q_rows, q_heads].  Logits, statistics and sums are fp32; probabilities (about a
 * reference of the row's own logits, at most 2^8) are rounded to the input's type for
 * their product with v and for the sum that o is divided by, not for lse.
 * (Sums of probabilities times v that pass fp32's range are infinite, as bf16 values above
 * 2^120 divided by the number of keys can make them.)
 *
 * A row of o is a bitwise function of its query and of the keys and values it sees,
 * in their order (and of dim and scale): not of the number of queries of the call or
 * of its sequence, other sequences, room in a cache, or max_q.  A prompt taken at
 * once, in pieces or token by token over a cache has the same bits.  What lies in k and
 * v where a row does not see it does not reach the row, NaN included.  A value of v that is not
 * finite and that the row sees is added to the row's result as it is, whatever its weight: o is
 * that infinity there, or NaN (a NaN, or infinities of both signs).
 *
 * cu_q, cu_k (int32 [batch + 1]) and k_lens (int32 [batch]) are device memory, read by the
 * kernels: values that ascend, from 0 to the rows.  Others are clamped to the operands:
 * results are then unspecified, but nothing outside is touched.  No passage of the
 * pages defines these calls.
 * ------------------------------------------------------------------------- */
typedef struct attention_plan_s* attention_plan_t;

/* Plan the call.  max_q: no sequence has more queries (0: q_rows).  Where it is small and caches are
 * long, a kernel of few rows takes the call (the bits are the same); a sequence with more
 * queries than max_q says has NaN in the rows past it.  scale > 0.  GEMM_ERR_INVALID_VALUE for a
 * negative size, batch < 1 or a NULL handle, GEMM_ERR_UNSUPPORTED for other types, scales or sizes
 * (batch up to 2^20, k_rows up to 2^30, fewer than 2^23 tiles of 128 rows of the key
 * heads and 2^22 of 128 keys). */
gemm_status attention_plan(int64_t q_rows, int64_t k_rows, int64_t batch, int q_heads, int k_heads,
                           int dim, gemm_dtype dtype, int causal, float scale, int64_t max_q,
                           attention_plan_t* plan);

/* Bytes of workspace attention_run needs: the chunks' results of few rows, 0 otherwise. */
size_t attention_workspace_size(attention_plan_t plan);

/* o, and for the backward pass lse and o_low, on `stream`.  o_low has the form of o and
 * receives what the rounding of o left, rounded to the type; each may be NULL.  cu_q and cu_k
 * may both be NULL for one sequence of all rows.  q, k, v and o are 16-byte aligned,
 * strides multiples of 8 elements. */
gemm_status attention_run(attention_plan_t plan, const void* q, int64_t q_token_stride,
                          int64_t q_head_stride, const void* k, int64_t k_token_stride,
                          int64_t k_head_stride, const void* v, int64_t v_token_stride,
                          int64_t v_head_stride, const int* cu_q, const int* cu_k,
                          const int* k_lens, void* o, void* o_low, float* lse, void* workspace,
                          size_t workspace_bytes, void* stream);

/* Bytes of workspace attention_backward needs: two numbers a row and head. */
size_t attention_backward_workspace_size(attention_plan_t plan);

/* The gradients dq, dk and dv (contiguous) from that of o (contiguous), o, o_low (or NULL:
 * then the rounding of o is in the gradients) and lse:
 *   ds_ij = p_ij (do_i v_j - sum_d do_id (o + o_low)_id), dv_j = sum_i p_ij do_i,
 *   dq_i = scale sum_j ds_ij k_j, dk_j = scale sum_i ds_ij q_i,
 * p and ds rounded to the input's type for their products (fp16: p is raised by 2^14 for
 * dv's; a ds below 2^-25 is lost, so gradients need the scaling of the loss that fp16 training has).  Rows in no
 * sequence and keys past k_lens have zero gradients.  Sums in a fixed order, without
 * atomics: the gradients of a sequence are a bitwise function of it alone.  A NaN or infinity
 * in q, k, v or d_o stays in its sequence; there it may reach, beyond the formula's
 * gradients, those of queries and keys up to 78 places away that do not see each other (a wave
 * works on 16 rows or keys in steps of 64), and an infinite gradient may be NaN. */
gemm_status attention_backward(attention_plan_t plan, const void* d_o, const void* q,
                               int64_t q_token_stride, int64_t q_head_stride, const void* k,
                               int64_t k_token_stride, int64_t k_head_stride, const void* v,
                               int64_t v_token_stride, int64_t v_head_stride, const void* o,
                               const void* o_low, const float* lse, const int* cu_q, const int* cu_k,
                               const int* k_lens, void* dq, void* dk, void* dv, void* workspace,
                               size_t workspace_bytes, void* stream);

void attention_plan_destroy(attention_plan_t plan);

/* ---------------------------------------------------------------------------
 * Log probabilities of given tokens, the entropy and the most likely tokens of
 * rows of logits (the last product's output): with max = max_v x_v and
 * log_sum = ln sum_v e^(x_v - max),
 *   logprob[n] = (x[token_n] - max) - log_sum, entropy = -sum_v p_v ln p_v,
 * and the `top` tokens of the largest logits with their log probabilities, the
 * largest first, the lower token first among equals (NaN counts as the largest).
 * A token below 0 is no token (logprob 0, no gradient); one from vocab on gives NaN.
 * A logit of -infinity has probability 0; a row that holds NaN or +infinity, or
 * -infinity alone, has NaN results.  logits: fp32, fp16 or bf16, row i from element
 * i row_stride on (any stride: rows need no alignment).  Sums are fp32.  Row i of every
 * output is a bitwise function of row i.  No passage of the pages defines these
 * calls.
 * ------------------------------------------------------------------------- */
typedef struct logprobs_plan_s* logprobs_plan_t;

/* Plan the call.  tokens_per_row 0 to 1024, top 0 to 64, vocab up to 2^22.
 * GEMM_ERR_INVALID_VALUE for a negative size, vocab < 1, top > vocab or a NULL handle,
 * GEMM_ERR_UNSUPPORTED for other types or sizes. */
gemm_status logprobs_plan(int64_t rows, int64_t vocab, int tokens_per_row, int top,
                          gemm_dtype dtype, logprobs_plan_t* plan);

/* Bytes of workspace logprobs_run needs (few rows are cut into parts). */
size_t logprobs_workspace_size(logprobs_plan_t plan);

/* tokens: int64 [rows, tokens_per_row]; logprob: fp32 [rows, tokens_per_row]; entropy:
 * fp32 [rows]; norm: fp32 [rows, 2], (max, log_sum) for the backward pass, or NULL;
 * top_logprob: fp32 and top_token: int64 [rows, top] (NULL where top is 0). */
gemm_status logprobs_run(logprobs_plan_t plan, const void* logits, int64_t row_stride,
                         const int64_t* tokens, float* logprob, float* entropy, float* norm,
                         float* top_logprob, int64_t* top_token, void* workspace,
                         size_t workspace_bytes, void* stream);

/* The gradient of the logits, contiguous [rows, vocab] in their type, rounded once:
 *   d_logits_v = sum_n g_n (1[v = token_n] - p_v) - h p_v (ln p_v + entropy)
 * with g = d_logprob [rows, tokens_per_row] and h = d_entropy [rows], each fp32 or NULL.
 * norm and entropy as logprobs_run left them; d_logits 16-byte aligned, and no operand's
 * memory. */
gemm_status logprobs_backward(logprobs_plan_t plan, const float* d_logprob, const float* d_entropy,
                              const void* logits, int64_t row_stride, const int64_t* tokens,
                              const float* norm, const float* entropy, void* d_logits,
                              void* stream);

void logprobs_plan_destroy(logprobs_plan_t plan);

/* Name of a status ("GEMM_OK", ...); a static string.  Housekeeping. */
const char* gemm_status_string(gemm_status status);

/* HIP error code (hipError_t as int) of the most recent GEMM_ERR_HIP return on
 * this host thread, 0 if none. */
int gemm_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* INVARIANT_MATMUL_H */
