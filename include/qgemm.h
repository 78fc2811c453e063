/*
 * qgemm — weight-quantized mixed-precision matrix product for AMD MI355X (gfx950).
 *
 *     C[M,N] = A[M,K] . dequant(Wq[K,N])
 *
 * Problem statement: BitBLAS issue #252 ("Default Backend Should be changed
 * into tilelang ..."), reproduction script — a MatmulConfig is M, N, K,
 * A_dtype, W_dtype, out_dtype, accum_dtype, layout "nt", with_bias,
 * group_size, with_scaling, with_zeros, zeros_mode.  Parallel-k (k-parts)
 * follows hidet issue #364 ("[Graph][Quantization] Multi-stage software
 * pipelining and update parallel k rule"): K is split into parts whose
 * partial products are reduced with atomics.  Affine dequantisation
 * w = (q - z) * s follows torchao issue #2752 (AffineQuantizedTensor).
 * int8 products accumulate into and return int32 (Triton PR #3595).
 *
 * Supported formats (a_dtype, w_dtype, out_dtype, accum_dtype):
 *   W4A16 : (F16, I4 | U4, F16, F32)   per-group fp16 scales, optional zero points (U4)
 *   dense : (F16, F16,     F16, F32)
 *   W8A8  : (I8,  I8,      I32, I32)   exact
 *   W2A8  : (I8,  I2,      I32, I32)   exact
 *   W8A8 / W2A8 dequantised: (I8, I8 | I2, F16, I32), run with per-row and
 *           per-column fp32 scales through qgemm_run_scaled
 * Any other tuple returns QGEMM_ERR_UNSUPPORTED (fp16 accumulation and int8
 * output are not provided: the int8 narrowing rule is unspecified).
 *
 * Canonical input layout ("nt"; all row-major, little-endian):
 *   A        [M, K]      fp16 or int8
 *   W  I4/U4 uint32 [N, K/8]   value (k, n) in bits 4*(k%8) of word n*(K/8) + k/8
 *      I2    uint32 [N, K/16]  value (k, n) in bits 2*(k%16) of word n*(K/16) + k/16
 *      I8    int8   [N, K]     F16 fp16 [N, K]
 *      signed values are two's complement of the field width; U4 is plain binary.
 *   scales   fp16 [N, G], zeros fp16 [N, G]; G = K/g for g > 0, G = 1 for g = -1.
 *   C        [M, N]      fp16 or int32
 * Dequantised weight: w = q (g == 0), w = q*s (no zeros), w = (q - z)*s (zeros),
 * with s, z taken at column n and group k / g.
 *
 * Packed weights: qgemm_pack_weights writes an opaque blob of packed_bytes
 * (weights pre-shuffled into the MFMA operand order of gfx950, 1 KiB per
 * 16-column x KB-row block, plus relaid scales and zeros).  The blob depends
 * only on (N, K, w_dtype, group_size, has_zeros): plans that differ only in M,
 * k_parts or flags can share one packed weight.
 *
 * Ownership and streams: every device buffer is allocated and owned by the
 * caller; the library allocates no device memory.  A plan owns only host
 * memory and is immutable after creation, so it may be used from several
 * threads at once.  `stream` is a hipStream_t passed as void* (NULL = the
 * null stream); every device call is asynchronous on it.  Concurrent
 * qgemm_run calls on one plan need distinct workspaces and outputs.
 *
 * Errors: every call returns a status; nothing is thrown across the ABI.
 * Argument errors are found before any device call (qgemm_create makes no
 * HIP call at all).  A failed launch returns QGEMM_ERR_DEVICE.
 */
#ifndef QGEMM_H
#define QGEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct qgemm_plan qgemm_plan;

typedef enum {
  QGEMM_OK = 0,
  QGEMM_ERR_INVALID_ARG = 1, /* NULL pointer, non-positive size, bad flag, too-small buffer */
  QGEMM_ERR_UNSUPPORTED = 2, /* legal request outside the supported formats or shapes */
  QGEMM_ERR_NO_MEMORY = 3,   /* host allocation of the plan failed */
  QGEMM_ERR_DEVICE = 4       /* a kernel launch failed */
} qgemm_status;

typedef enum {
  QGEMM_F16 = 1,
  QGEMM_F32 = 2,
  QGEMM_I32 = 3,
  QGEMM_I8 = 4,
  QGEMM_I4 = 5, /* signed int4, [-8, 7] */
  QGEMM_U4 = 6, /* unsigned int4, [0, 15] */
  QGEMM_I2 = 7  /* signed int2, [-2, 1] */
} qgemm_dtype;

/* flags for qgemm_create (k_parts > 1 only; without flags the parts are reduced
   with global atomics, the parallel-k reduction of hidet issue #364) */
#define QGEMM_DETERMINISTIC 1u /* fixed-order two-pass reduction: bitwise reproducible */
#define QGEMM_SPLIT_AUTO 2u    /* the reduction that measured faster for the plan's shape:
                                  two-pass for fp16 outputs and for int32 outputs from 128
                                  rows while the partials stay within 256 MiB, else atomics;
                                  QGEMM_DETERMINISTIC takes precedence */

/* execution path chosen by a plan (qgemm_plan_path) */
#define QGEMM_PATH_GEMV 1 /* M <= 8: skinny kernels streaming the weights once (dot products at
                             one row; matrix cores from 2 rows, 3 for int4) */
#define QGEMM_PATH_MFMA 2 /* M > 8: matrix cores (skinny kernels up to 32 rows, then
                             LDS-staged tiles) */

/*
 * Create a plan: the problem statement of BitBLAS issue #252's Matmul
 * configuration (M, N, K, A_dtype, W_dtype, out_dtype, accum_dtype, group_size,
 * with_scaling as group_size != 0, with_zeros) plus hidet issue #364's k-parts.
 * No device call.
 *   M, N, K       problem sizes, each >= 1.  K must be a multiple of the values
 *                 per canonical word: 8 (I4/U4), 16 (I2), 1 (I8/F16), and of
 *                 group_size when that is > 0, else QGEMM_ERR_UNSUPPORTED.  The
 *                 kernels work on whole granules of 128 (I4/U4, I8), 256 (I2) or
 *                 64 (F16) positions: when K is not a multiple of the granule,
 *                 the blob is zero-padded and every run first copies A into the
 *                 workspace with its rows zero-padded (the workspace then also
 *                 holds M * roundup(K, granule) activation elements).  The
 *                 activations, M * roundup(K, granule) elements, must stay below
 *                 4 GiB, else QGEMM_ERR_UNSUPPORTED.
 *   group_size    0 = no scaling (with_scaling False), -1 = one group per output
 *                 column over all of K, g > 0 = groups of g along K.  Scaled
 *                 formats are I4/U4 only; g > 0 must divide K and be a multiple
 *                 of 32.  Other weight formats require 0.
 *   has_zeros     0 or 1; 1 only with w_dtype U4 and group_size != 0.
 *                 Scales of U4 weights: |s| < 64, and with zero points
 *                 |s| * (1024 + z) < 65504 with 0 <= z < 1024; of I4 weights
 *                 with g > 0: |s| < 63; for rows that take the 256 x 256 tiles
 *                 (large M): those tiles upcast and scale a weight with one
 *                 fp16 fma whose addend, -1024 s, -fp16(1024 + z) s or -1032 s,
 *                 must be finite (BitBLAS issue #252, the int4 / uint4 op
 *                 configs with scaling and zero points).
 *   k_parts       >= 1: number of contiguous, group-aligned K ranges computed by
 *                 separate workgroups and reduced with fp32/int32 global atomics
 *                 (default) or by ordered partials and one summing pass
 *                 (QGEMM_DETERMINISTIC; see qgemm_run).  At most K / unit, where
 *                 unit = group_size when it is a multiple of 128 (and larger),
 *                 else the granule (K rounded up to it).
 *   flags         0, or QGEMM_DETERMINISTIC and / or QGEMM_SPLIT_AUTO.
 *   packed_bytes  out: size of the packed blob for qgemm_pack_weights/qgemm_run.
 *   workspace_bytes out: size of the device workspace qgemm_run needs (0 if none).
 *                 A plan of k_parts 1 may need one too: for I4 / U4 weights and
 *                 K >= 8192 the library splits K itself and sums the partial
 *                 products in a fixed order, so results stay bitwise reproducible;
 *                 the workspace holds those parts' fp32 partials.  With 33 to 256
 *                 rows and N >= 4096: 2, 4 or 8 parts (as many as one wave of 256
 *                 workgroups of 128 x 128 output tiles takes), for runs of more than
 *                 32 rows.  With 9 to 32 rows, N <= 4096 and groups of whole
 *                 superblocks (or none): 4 parts for runs of 17 rows or more when the
 *                 plan has more than 16 rows, else 2 parts for runs of 9 or more.
 *                 U4 with zero points and groups that are whole multiples of 128
 *                 (or one group over K), and I4 with such groups (its offset 8
 *                 as the zero point): runs that take the 256 x 256 tiles apply
 *                 the zero points after their K loop as sum_g R[m, g] P[g, n],
 *                 with R the row sums of A over each group and P from the scales
 *                 and zeros (each held as two bf16 planes of roundup(G, 32)
 *                 values per row of A and per padded column); the workspace then
 *                 ends with those planes, sized for the largest run of the plan
 *                 that takes those tiles.
 */
qgemm_status qgemm_create(qgemm_plan** out, int64_t M, int64_t N, int64_t K,
                          qgemm_dtype a_dtype, qgemm_dtype w_dtype, qgemm_dtype out_dtype,
                          qgemm_dtype accum_dtype, int32_t group_size, int32_t has_zeros,
                          int32_t k_parts, uint32_t flags, size_t* packed_bytes,
                          size_t* workspace_bytes);

/*
 * Pack canonical weights (device memory, layout above) into the plan's blob: the
 * backend-specific pre-shuffled weight of torchao issue #2752's "dtype +
 * packing_format" tensors, built from BitBLAS issue #252's "nt" weight layout.
 *   w       device, canonical weights.
 *   scales  device, fp16 [N, G]; required iff group_size != 0, else ignored.
 *   zeros   device, fp16 [N, G]; required iff has_zeros, else ignored.
 *   packed  device, >= packed_bytes, 16-byte aligned; fully overwritten.
 * Asynchronous on `stream`; run once per weight, outside the hot loop.
 */
qgemm_status qgemm_pack_weights(const qgemm_plan* plan, const void* w, const void* scales,
                                const void* zeros, void* packed, void* stream);

/*
 * C = A . dequant(W) on `stream` (the quantized matmul of hidet issue #364 and
 * BitBLAS issue #252; int8 x int8 / int2 products accumulate and return int32,
 * Triton PR #3595).
 *   A          device, [M, K] fp16 or int8, 16-byte aligned (rows are K elements
 *              apart, whatever their alignment).
 *   packed     device, the blob written by qgemm_pack_weights.
 *   C          device, [M, N] fp16 or int32; fully overwritten.
 *   workspace  device, >= workspace_bytes (may be NULL when that is 0),
 *              16-byte aligned; scratch for split-K and padded activations, its
 *              contents on entry are ignored.
 * Split-K (k_parts > 1) reduces the parts with global atomics unless a flag says
 * otherwise: fp16 outputs add fp32 partials into the zero-filled workspace
 * (M * N * 4 bytes), which one more pass rounds into C; int32 outputs add
 * straight into C (no workspace).  fp32 atomics add in the order the parts
 * finish, so fp16 results may differ in the last bits between runs (each within
 * the accuracy of the fp32 sum); int32 results are exact and identical.  With
 * QGEMM_DETERMINISTIC (and with QGEMM_SPLIT_AUTO where it picks them) the parts
 * write ordered partials (k_parts * M * N * 4 bytes) that one pass sums in part
 * order: bitwise reproducible.
 */
qgemm_status qgemm_run(const qgemm_plan* plan, const void* A, const void* packed, void* C,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * C = A . dequant(W) (+ bias) for a run-time number of rows, on `stream`: the
 * serving form of qgemm_run (decode batches vary from call to call), and the
 * bias epilogue that BitBLAS's Matmul configuration names with_bias (its
 * benchmark configurations leave it off; BitBLAS issue #252, reproduction script).
 *   M          rows this call computes, 1 <= M <= the plan's M, else
 *              QGEMM_ERR_INVALID_ARG.  The kernels are chosen for this M (as
 *              qgemm_create would for a plan of M rows); the plan's workspace
 *              size covers every M.
 *   A          device, [M, K], as in qgemm_run.
 *   packed     device, the plan's blob.
 *   bias       device, [N] of the output type (fp16 or int32), or NULL for none:
 *              C[m, n] = sum + bias[n].  fp16 outputs add it in fp32 before the
 *              one rounding to fp16; int32 outputs add it exactly.  Naturally
 *              aligned (2 / 4 bytes), else QGEMM_ERR_INVALID_ARG.
 *   C          device, [M, N]; fully overwritten.
 *   workspace, workspace_bytes, stream: as in qgemm_run.
 * qgemm_run(plan, A, packed, C, ...) is qgemm_run_ex with the plan's M and no bias.
 */
qgemm_status qgemm_run_ex(const qgemm_plan* plan, int64_t M, const void* A, const void* packed,
                          const void* bias, void* C, void* workspace, size_t workspace_bytes,
                          void* stream);

/*
 * qgemm_run_ex without a workspace argument, for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc).  Split-K runs in a fixed scratch array inside the
 * library, one per GPU, of QGEMM_NOALLOC_MAX_SCRATCH bytes, which each GPU the
 * library runs on holds until the process ends; this call itself allocates
 * nothing.  It needs the workspace that qgemm_run_ex would for run-time M (the
 * atomic accumulator or the two-pass partials, plus the zero-padded activation
 * rows when K is not a whole number of blocks, plus the zero-point planes of U4 /
 * I4 plans on the 256 x 256 tiles; none for an unsplit plan of
 * whole blocks otherwise); more than the maximum returns QGEMM_ERR_UNSUPPORTED
 * before any device call.
 * Every call on one GPU shares that GPU's scratch: calls that may overlap in
 * time on one GPU (other streams, other threads) race and must be serialised by
 * the caller.  The stream must belong to the current device.  Plans with
 * dequantised int8 output (qgemm_run_scaled) are rejected (QGEMM_ERR_INVALID_ARG).
 *   M, A, packed, bias, C, stream: as in qgemm_run_ex.
 * The first call that needs scratch on a device looks up its address
 * (QGEMM_ERR_DEVICE if that fails).
 */
#define QGEMM_NOALLOC_MAX_SCRATCH ((size_t)32 << 20)
qgemm_status qgemm_run_noalloc(const qgemm_plan* plan, int64_t M, const void* A, const void* packed,
                               const void* bias, void* C, void* stream);

/*
 * int8 activations with fp16 output (plans created with the tuple
 * (I8, I8 | I2, F16, I32)): C[m, n] = fp16(acc[m, n] * row_scales[m] *
 * col_scales[n] (+ bias[n])), the dequantising epilogue of the int8
 * dynamic-activation configurations (torchao issue #2752), computed in fp32
 * from the exact int32 accumulator with one rounding.  Such plans run only
 * through this call (qgemm_run / qgemm_run_ex return QGEMM_ERR_INVALID_ARG).
 *   M          rows, 1 <= M <= the plan's M.
 *   A          device, int8 [M, K] (e.g. from qgemm_quantize_rows).
 *   row_scales device, fp32 [M] (per-token activation scales).
 *   col_scales device, fp32 [N] (per-channel weight scales).
 *   bias       device, fp16 [N], or NULL.
 *   C          device, fp16 [M, N]; fully overwritten.
 *   workspace, workspace_bytes, stream: as in qgemm_run.
 */
qgemm_status qgemm_run_scaled(const qgemm_plan* plan, int64_t M, const void* A, const void* packed,
                              const float* row_scales, const float* col_scales, const void* bias,
                              void* C, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Dynamic per-token int8 quantisation of fp16 activations (the activation step
 * of torchao issue #2752's Int8DynamicActivation* configurations), symmetric
 * with one scale per row:
 *   scales[m] = max_k |A[m, k]| / 127                  (fp32, round to nearest)
 *   Q[m, k]   = clamp(rint(A[m, k] / scales[m]), -127, 127)
 * with the division in fp32, correctly rounded, rint to nearest even; an
 * all-zero row gets scale 0 and codes 0.
 *   A       device, fp16 [M, K], 16-byte aligned.
 *   M, K    M >= 1; K >= 8 and a multiple of 8.
 *   Q       device, int8 [M, K], 8-byte aligned; fully overwritten.
 *   scales  device, fp32 [M], 4-byte aligned; fully overwritten.
 * Asynchronous on `stream`.  QGEMM_ERR_INVALID_ARG on a bad argument (checked
 * before any launch), QGEMM_ERR_DEVICE if the launch fails.
 */
qgemm_status qgemm_quantize_rows(const void* A, int64_t M, int64_t K, void* Q, float* scales,
                                 void* stream);

/* ---- gated feed-forward block ------------------------------------------------
 *
 *     C[M,N] = act(A . dequant(Wg) + bg) * (A . dequant(Wu) + bu)
 *
 * Both projections, the activation and the product in one kernel (one more summing
 * pass where the library splits K, as for the plain product).  A gated plan packs the
 * two weights into one blob whose 16-column blocks alternate, so that a lane of every
 * kernel holds the two sums of an output; they stay in fp32 (int32 for int8
 * activations) up to the one rounding of C.
 */
typedef enum {
  QGEMM_ACT_SILU = 1,     /* x sigmoid(x) */
  QGEMM_ACT_GELU_TANH = 2 /* 0.5 x (1 + tanh(sqrt(2 / pi) (x + 0.044715 x^3))) */
} qgemm_act;

/*
 * Create a gated plan.  The arguments are those of qgemm_create, with N the columns of
 * C and of each projection; the output type is QGEMM_F16 (else QGEMM_ERR_UNSUPPORTED),
 * so the tuples are (F16, I4 | U4 | F16, F16, F32) and (I8, I8 | I2, F16, I32).  K is not
 * split by the caller (the library splits it where qgemm_create's plans do).  The size
 * limits hold for the 2 * roundup(N, 16) columns of both projections.
 *   act            the activation, else QGEMM_ERR_INVALID_ARG.
 *   packed_bytes   out: size of the blob that qgemm_pack_gated writes.
 *   workspace_bytes out: size of the workspace of qgemm_run_gated (0 if none).  Runs of more
 *                  than 128 rows whose groups are not multiples of 128 keep the weights there
 *                  as fp16 (4 K N bytes and their padding).
 * Gated plans run through qgemm_pack_gated, qgemm_run_gated and qgemm_gated_backward
 * (the plain calls return QGEMM_ERR_INVALID_ARG for them) and are destroyed by
 * qgemm_destroy.
 */
qgemm_status qgemm_create_gated(qgemm_plan** out, int64_t M, int64_t N, int64_t K,
                                qgemm_dtype a_dtype, qgemm_dtype w_dtype, qgemm_dtype out_dtype,
                                qgemm_dtype accum_dtype, int32_t group_size, int32_t has_zeros,
                                qgemm_act act, size_t* packed_bytes, size_t* workspace_bytes);

/*
 * Pack the canonical weights of both projections (each as in qgemm_pack_weights: w
 * [N, K], 16-byte aligned; s and z fp16 [N, G], required iff the plan has them) into
 * the plan's blob.  Asynchronous on `stream`.
 */
qgemm_status qgemm_pack_gated(const qgemm_plan* plan, const void* w_gate, const void* s_gate,
                              const void* z_gate, const void* w_up, const void* s_up,
                              const void* z_up, void* packed, void* stream);

/*
 * Run a gated plan on `stream` for M rows, 1 <= M <= the plan's M (the kernels are
 * chosen for this M).
 *   A              device, [M, K] fp16 or int8, 16-byte aligned.
 *   packed         device, the blob of qgemm_pack_gated, 16-byte aligned.
 *   row_scales     device, fp32 [M]; col_scales_gate / _up fp32 [N]: the scales of
 *                  int8 activations and weights as in qgemm_run_scaled.  Required iff
 *                  the activations are int8, else all three must be NULL.
 *   bias_gate, bias_up  device, fp16 [N], each may be NULL (none).
 *   preact         device, fp16 [M, 2 N] or NULL: receives the two pre-activations of each
 *                  row (gate, then up), rounded to fp16, for qgemm_gated_backward.
 *   C              device, fp16 [M, N]; fully overwritten.
 *   workspace, workspace_bytes: as in qgemm_run.
 */
qgemm_status qgemm_run_gated(const qgemm_plan* plan, int64_t M, const void* A, const void* packed,
                             const float* row_scales, const float* col_scales_gate,
                             const float* col_scales_up, const void* bias_gate, const void* bias_up,
                             void* preact, void* C, void* workspace, size_t workspace_bytes,
                             void* stream);

/*
 * Workspace of qgemm_gated_backward for M rows; weight_grads: whether any weight or bias
 * gradient will be asked for.  QGEMM_ERR_UNSUPPORTED for int8 activations, for weight
 * gradients of quantised weights (which are frozen), and where an operand of the
 * products passes the size limits of qgemm_create.
 */
qgemm_status qgemm_gated_backward_workspace(const qgemm_plan* plan, int64_t M, int32_t weight_grads,
                                            size_t* workspace_bytes);

/*
 * Gradients of a gated run of M rows from the gradient of its output:
 *   dU = dC act(g), dG = dC u act'(g);  dA = dG . Wg^T + dU . Wu^T,
 *   dWg = dG^T . A, dWu = dU^T . A, dbg and dbu the column sums of dG and dU
 * with g and u the pre-activations as kept (rounded to fp16; a kept infinity stands for
 * 65504 of its sign) and dG, dU rounded to fp16 as operands of the products, which sum in
 * fp32.  A row of them (for dA) or a column (for dW) whose largest value lies past fp16 or
 * below 2^-6 is scaled by a power of two for that, so that it neither overflows nor
 * vanishes; the sums are scaled back before they are rounded.  Bias gradients sum the
 * unrounded values.  Quantised weights enter dA as (q - z) s rounded to fp16.
 *   A          device, fp16 [M, K] (needed for weight gradients), 16-byte aligned.
 *   packed     device, the forward's blob (needed for dA), 16-byte aligned.
 *   preact     device, fp16 [M, 2 N], from the forward.
 *   dC         device, fp16 [M, N].
 *   dA         device, fp16 [M, K], or NULL.
 *   dw_gate, dw_up       device, fp16 [N, K], both or neither (fp16 weights only); where
 *              dw_up follows dw_gate in memory one product computes both.
 *   dbias_gate, dbias_up device, fp16 [N], each may be NULL (fp16 weights only).
 *   workspace  device, >= the bytes of qgemm_gated_backward_workspace, 16-byte aligned.
 * Every output asked for is fully overwritten; the sums' order is fixed, so results are
 * bitwise reproducible.  Asynchronous on `stream`.
 */
qgemm_status qgemm_gated_backward(const qgemm_plan* plan, int64_t M, const void* A,
                                  const void* packed, const void* preact, const void* dC, void* dA,
                                  void* dw_gate, void* dw_up, void* dbias_gate, void* dbias_up,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* ---- paged key / value cache ---------------------------------------------------
 *
 * Keys and values of past tokens in fp16 pages: k and v are device arrays
 * [n_pages, kv_heads, page_size, head_dim], contiguous, 16-byte aligned, owned by the
 * caller.  page_size is a power of two up to 65536; head_dim a multiple of 8 up to 256
 * (else QGEMM_ERR_UNSUPPORTED).  A token's slot is page * page_size + its place in the
 * page.  Offsets are 64 bits wide: a cache may pass 2^32 values.
 */
typedef struct {
  void* k;
  void* v;
  int64_t n_pages;
  int32_t page_size;
  int32_t kv_heads;
  int32_t head_dim;
} qgemm_kv_cache;

/*
 * Rotate the queries and keys of T new tokens and write the keys and values into the
 * cache.  Head h of a token is its values h * head_dim .. of the row; of each the first
 * rot_dim values turn by the token's angles (fp32, one rounding), the others are copied:
 *   (a, b) -> (a c - b s, b c + a s),  c = cos[p, j], s = sin[p, j], p = positions[t],
 * over the pairs (j, j + rot_dim / 2), or (2 j, 2 j + 1) when interleaved.
 *   T           tokens, >= 0 (0: nothing is launched).
 *   q_heads     query heads, a multiple of the cache's kv_heads.
 *   q, k, v     device, fp16; row t starts t * stride values in (strides >= the row's
 *               length, so that they may be slices of one projection's output).
 *   cos, sin    device, fp32 [n_positions, rot_dim / 2].
 *   rot_dim     even, 0 .. head_dim (0: cos and sin may be NULL).
 *   positions   device, int32 [T].  A token whose position is outside [0, n_positions) is
 *               not stored, and its queries become NaN.
 *   slots       device, int64 [T], distinct.  A token whose slot is outside the cache
 *               (negative in unused places of a batch) is not stored.
 *   q_out       device, fp16 [T, q_heads, head_dim]; may be q itself when q_stride is
 *               q_heads * head_dim.
 * 16-byte aligned arrays with strides of whole 8 values take the widest accesses.  More
 * than 65535 * 512 values a token (all heads) return QGEMM_ERR_UNSUPPORTED.
 */
qgemm_status qgemm_kv_append(const qgemm_kv_cache* cache, int64_t T, int32_t q_heads, const void* q,
                             int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                             int64_t v_stride, const float* cos, const float* sin,
                             int64_t n_positions, int32_t rot_dim, int32_t interleaved,
                             const int32_t* positions, const int64_t* slots, void* q_out,
                             void* stream);

/*
 * Workspace of qgemm_attention for these sizes (0 where no work is split).
 */
qgemm_status qgemm_attention_workspace(const qgemm_kv_cache* cache, int64_t T, int32_t q_heads,
                                       int64_t B, int64_t max_q, int64_t max_len,
                                       int64_t prefix_len, size_t* workspace_bytes);

/*
 * Causal attention of B sequences over the cache, all of which may begin with one shared
 * prefix: out = softmax(scale q K^T) V per query and head (scale positive and scale log2 e
 * finite in fp32), with scores, softmax and sums in fp32 and the probabilities rounded to fp16
 * as operands of the product with V.
 * Query head h reads key / value head h / (q_heads / kv_heads).
 *   T            rows of q: the queries of all sequences, one after the other.  With 0 of them
 *                nothing is launched, and B and max_q may be 0 (else they are at least 1).
 *   q            device, fp16, row t at t * q_stride values (q_stride >= q_heads *
 *                head_dim, a multiple of 8; q 16-byte aligned).
 *   q_starts     device, int32 [B + 1]: sequence b has the rows q_starts[b] ..
 *                q_starts[b + 1] - 1 (n of them; none is allowed), at most max_q.
 *   kv_lens      device, int32 [B]: own tokens of each sequence in the cache, the n new
 *                ones included, at most max_len.
 *   tables       device, int32 [B, table_width]: pages of each sequence's own tokens,
 *                in order; entries past its last page are not read.
 *   prefix_table device, int32: pages of the prefix (NULL when prefix_len is 0).
 *   prefix_len   tokens of the prefix, >= 0; every query sees all of them.
 * Query i of a sequence sees own token j iff j <= kv_lens[b] - n + i.  A query that sees
 * nothing gets zeros (and lse -inf).  Keys and values that a query does not see never
 * enter its result, whatever they hold (NaN and infinities included).
 *   max_q, max_len  bounds of n and kv_lens (host values, so that a captured call can be
 *                replayed with other lengths); rows past max_q are not written, tokens past
 *                max_len or the table not read.  A page number outside the cache reads
 *                page 0.
 *   out          device, fp16 [T, q_heads, head_dim], 16-byte aligned; rows of no
 *                sequence are not written.
 *   lse          device, fp32 [T, q_heads] or NULL: ln(sum exp(scale q k)) of each row.
 *   workspace, workspace_bytes: as stated by qgemm_attention_workspace, 16-byte aligned.
 * More than 65535 sequences, 2^31 - 65537 tokens of one sequence and the prefix, or work of
 * 2^24 workgroups return QGEMM_ERR_UNSUPPORTED.
 * The prefix is read once for rows of all sequences where sequences have few rows each;
 * keys are split over workgroups where rows are few, and the parts' results joined in a
 * fixed order: results are bitwise reproducible for the same sizes.
 */
qgemm_status qgemm_attention(const qgemm_kv_cache* cache, int64_t T, int32_t q_heads, const void* q,
                             int64_t q_stride, int64_t B, const int32_t* q_starts,
                             const int32_t* kv_lens, const int32_t* tables, int64_t table_width,
                             const int32_t* prefix_table, int64_t prefix_len, int64_t max_q,
                             int64_t max_len, float scale, void* out, float* lse, void* workspace,
                             size_t workspace_bytes, void* stream);

/* Release a plan; NULL is a no-op.  Device buffers are the caller's. */
void qgemm_destroy(qgemm_plan* plan);

/* Path the plan chose (QGEMM_PATH_GEMV or QGEMM_PATH_MFMA), or -1 for NULL. */
int32_t qgemm_plan_path(const qgemm_plan* plan);

/* Short static description of a status code. */
const char* qgemm_status_string(qgemm_status status);

#ifdef __cplusplus
}
#endif

#endif /* QGEMM_H */
