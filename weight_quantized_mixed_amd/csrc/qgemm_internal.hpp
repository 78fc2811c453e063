// Internal definitions shared by the host ABI and the kernels of libqgemm.
//
// Packed blob layout (written by the pack kernel, read by every compute kernel)
// ---------------------------------------------------------------------------
// Columns are padded to Npad = roundup(N, 256).  The weight region is a grid of
// 1 KiB "superblocks", each 16 columns x KB reduction positions:
//     superblock (nb, kb) at byte ((kb * (Npad/16)) + nb) * 1024
// KB = 128 (int4), 256 (int2), 64 (int8), 32 (fp16): 16 bytes per column per
// quarter of the block.  Inside a superblock, the 16-byte "piece" of column
// nn = n % 16 and quarter kq sits at byte (kq*16 + nn) * 16, so one wave-wide
// 16-byte load (lane l -> piece l) fetches the whole block in the lane order of
// a gfx950 16x16 MFMA B operand (lane l: column l%16, K slice l/16).  A piece
// covers the KB/4 consecutive positions kb*KB + kq*KB/4 + [0, KB/4):
//   int4  4 words x 8 values; word t holds positions 8t..8t+7 with nibble
//         slots (0..7) <- positions (0,2,4,6,1,3,5,7), stored offset-binary
//         (q + 8 for signed, q for unsigned), so (w >> 4j) & 0x000F000F,
//         or-ed with 0x6400 per half, is the fp16 pair (1024 + s[2j], 1024 + s[2j+1]).
//   int2  4 words x 16 values; word t holds positions 16t..16t+15, value e in
//         byte e%4 at bit 2*(e/4), so (w >> 2j) & 0x03030303 gives the four
//         consecutive positions 4j..4j+3.  Classes j = 0..2 are stored
//         offset-binary (q + 2); class 3 (bits 6..7 of each byte) is stored two's
//         complement, so w & 0xC0C0C0C0 reads as the signed bytes 64q.
//   int8  16 bytes = 16 consecutive positions.
//   fp16  8 halves = 8 consecutive positions.
// After the weights (256-byte aligned) come the scales as [G][Npad] fp16, or
// (scale, zero) half pairs as [G][Npad] when zero points are present.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qgemm.h"

namespace qg {

enum Fmt : int { FMT_I4 = 0, FMT_U4 = 1, FMT_F16 = 2, FMT_I8 = 3, FMT_I2 = 4 };

// output modes of a compute kernel
enum OutMode : int {
  OUT_STORE = 0,    // write C directly (k_parts == 1)
  OUT_ATOMIC = 1,   // atomic add into fp32 workspace (fp16 out) or into C (int32 out)
  OUT_PARTIAL = 2,  // write the part's partial to workspace[part][M][N] (two-pass)
  OUT_GATE = 3      // gated plans, one part: C = act(gate) * up from neighbouring column blocks
};

// scale modes
enum ScaleMode : int {
  SC_NONE = 0,   // group_size == 0
  SC_BLOCK = 1,  // one group per superblock (g >= KB or g == -1)
  SC_PIECE = 2   // one group per 32-position piece (g in {32, 64} for int4)
};

constexpr int kb_of(int fmt) {
  return fmt == FMT_I2 ? 256 : fmt == FMT_I8 ? 64 : fmt == FMT_F16 ? 32 : 128;
}

// fp16 / int8 direct-load MFMA stages of two superblocks (128-byte activation rows;
// 1) or one (64-byte rows; 0).  A direct load of 16 rows x 64 bytes moves half as
// many bytes per clock as one of 8 rows x 128 bytes (a probe of global_load_lds_dwordx4
// from L2 at a 32 KiB row stride: 70 against 143 bytes per ns per CU).
#ifndef QG_DL_WIDE
#define QG_DL_WIDE 1
#endif
// K granule of a format: K is padded to it and k-parts split at it (two superblocks
// for fp16 / int8 with two-superblock stages, else one)
constexpr int kgrain_of(int fmt) {
  return (QG_DL_WIDE && (fmt == FMT_F16 || fmt == FMT_I8)) ? 2 * kb_of(fmt) : kb_of(fmt);
}

// K is padded to whole K granules (Kpad = roundup(K, kgrain_of)): the blob holds zero
// codes at positions K .. Kpad - 1 and, where scale groups are smaller than a
// superblock, zero scales for the groups past K (G_store rows in all), and runs
// read activations zero-padded to Kpad, so those positions add exactly nothing.
struct Layout {
  int fmt;
  int64_t N, K, Kpad, Npad, NB, nkb;
  int32_t group_size;  // as given: 0, -1 or g > 0
  int64_t G;           // number of scale groups of the input table (0 without scaling)
  int64_t G_store;     // scale rows in the blob (G, or more to cover Kpad)
  bool zeros;
  size_t w_bytes, s_offset, s_bytes, total;
};

// Gated plans (C = act(A Wg + bg) * (A Wu + bu)) run both projections as one product
// whose 16-column blocks alternate: inner column 32 b + i (i < 16) is column 16 b + i of
// the gate projection and 32 b + 16 + i the same column of the up projection.  Every
// compute kernel then holds the two sums of an output in one lane, in neighbouring
// column blocks, and the block padding of N is the same for both.
__host__ __device__ constexpr int64_t gate_inner(int64_t N) { return (N + 15) / 16 * 32; }

// canonical weight values per 32-bit word (int8 / fp16 rows are plain arrays)
constexpr int pack_factor(int fmt) { return fmt == FMT_I2 ? 16 : (fmt == FMT_I4 || fmt == FMT_U4) ? 8 : 1; }

// Arguments of every compute kernel (GEMV and MFMA), passed by value.
struct RunArgs {
  const void* A;        // [M, K]
  const uint4* W;       // packed superblocks
  const void* S;        // scales (half) or (scale, zero) half2 pairs, [G][Npad]
  void* C;              // [M, N] fp16 or int32
  void* ws;             // fp32/int32 workspace
  int32_t M, N, K;
  int32_t Npad, NB, nkb;
  int32_t group_size;   // 0, -1 or g
  int32_t smode;        // ScaleMode
  int32_t zeros;        // 0/1
  int32_t out_mode;     // OutMode
  int32_t k_parts;
  int32_t unit_kb;      // superblocks per split unit
  int32_t n_units;      // nkb / unit_kb
  int32_t waves;        // GEMV: waves per workgroup (K split inside the workgroup)
  int32_t sb_per_group; // superblocks per scale group (nkb when one group spans K)
  int32_t g_shift;      // group of position p = p >> g_shift, or -1: p / group_size
  int32_t gemv_cb;      // matrix-core GEMV: 16-column blocks per workgroup (1, 2 or 4)
  const void* bias;     // [N] of the output type, or null
  // int8 activations with fp16 output: C = fp16(acc * row_scale[m] * col_scale[n]
  // (+ bias)); null for int32 output.  fp16 weights: C = fp16(acc * row_scale[m] (+ bias))
  // where row_scale is given (the gradient products)
  const float* row_scale;
  const float* col_scale;
  // int4 / uint4 with one scale group over K and no zero points on the matrix-core
  // tiles: the per-column scale applied to the fp32 sum in the epilogue (the tiles
  // then upcast without it); null otherwise
  const _Float16* epi_scale;
  // uint4 with zero points (and signed int4, its offset 8 as the zero point) on the
  // 256 x 256 tiles of four waves: the zero points are folded out of the K loop
  // (C = sum_k A q s - sum_g R[m, g] s[g, n] z[g, n], R the row sums of A over scale
  // group g).  zr holds R of each row, zp the per-column term P of each column (Npad of
  // them), each as two bf16 planes of zr_gp values, [hi | lo] with hi = bf16(x),
  // lo = bf16(x - hi), groups zr_G .. zr_gp - 1 zero; both null without the folding
  const uint16_t* zr;
  const uint16_t* zp;
  int32_t zr_gp;  // groups per plane: zr_G rounded up to 32
  int32_t zr_G;   // scale groups over K
  // gated plans (gate_n != 0): N counts the inner columns, gate_n the output's; bias and
  // col_scale are the gate projection's, these the up projection's; act(x) =
  // x sigmoid(x (act_c0 + act_c1 x^2)); preact, if given, receives the rounded
  // pre-activations [M][2 gate_n] (gate | up)
  int32_t gate_n;
  float act_c0, act_c1;
  const void* bias_up;
  const float* col_scale_up;
  _Float16* preact;
};

// bias of output column col (0 without bias): fp16 outputs add it in fp32 before
// their one rounding, int32 outputs exactly
__device__ __forceinline__ float bias_f(const RunArgs& a, int col) {
  return a.bias ? (float)static_cast<const _Float16*>(a.bias)[col] : 0.f;
}
__device__ __forceinline__ int bias_i(const RunArgs& a, int col) {
  return a.bias ? static_cast<const int*>(a.bias)[col] : 0;
}
// fp16 output of an int32 accumulator: the per-row (activation) and per-column
// (weight) scales and the bias applied in fp32, one rounding to fp16
__device__ __forceinline__ _Float16 dq_out(const RunArgs& a, int row, int col, int acc) {
  return (_Float16)((float)acc * a.row_scale[row] * a.col_scale[col] + bias_f(a, col));
}
// One output column of a gated plan, from the inner column of its gate sum: the
// scales that turn the two sums into pre-activations, and the biases.
struct GateCol {
  float sg, su, bg, bu;
  int col;  // output column
  bool in;
};
__device__ __forceinline__ GateCol gate_col(const RunArgs& a, int icol) {
  GateCol c;
  c.col = (icol >> 5) * 16 + (icol & 15);
  c.in = c.col < a.gate_n;
  c.sg = c.su = 1.f;
  c.bg = c.bu = 0.f;
  if (!c.in) return c;
  if (a.epi_scale) {
    c.sg = (float)a.epi_scale[icol];
    c.su = (float)a.epi_scale[icol + 16];
  } else if (a.col_scale) {
    c.sg = a.col_scale[c.col];
    c.su = a.col_scale_up[c.col];
  }
  if (a.bias) c.bg = (float)static_cast<const _Float16*>(a.bias)[c.col];
  if (a.bias_up) c.bu = (float)static_cast<const _Float16*>(a.bias_up)[c.col];
  return c;
}
// x sigmoid(t), t = x (c0 + c1 x^2): silu with (1, 0); the tanh form of gelu with
// (2 c, 2 c 0.044715), c = sqrt(2 / pi), since (1 + tanh y) / 2 = sigmoid(2 y).  The
// hardware exponential and reciprocal are within a few ulp in fp32.
// sigmoid(x (c0 + c1 x^2)), with the constants times -log2 e taken out of the exponent; the
// square stays finite, since silu's c1 of 0 times an infinite one (|x| from 1.8e19) would be NaN
__device__ __forceinline__ float gate_sigmoid(float c0, float c1, float x) {
  constexpr float L = -1.4426950408889634f;
  const float xx = fminf(x * x, 3.4e38f);
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x * (c0 * L + c1 * L * xx)));
}
__device__ __forceinline__ float gate_act(const RunArgs& a, float x) { return x * gate_sigmoid(a.act_c0, a.act_c1, x); }
// stores output (row, c.col) from the two sums, in fp32 up to the one rounding of the
// output (and one of each pre-activation, where they are kept for the backward pass: half the
// bytes to write and to read again; the output does not see it, the gradients start from it)
__device__ __forceinline__ void gate_store(const RunArgs& a, int row, const GateCol& c, float g, float u) {
  if (a.row_scale) {
    const float rs = a.row_scale[row];
    g *= rs;
    u *= rs;
  }
  g = g * c.sg + c.bg;
  u = u * c.su + c.bu;
  if (a.preact) {
    _Float16* p = a.preact + (size_t)row * 2 * a.gate_n + c.col;
    p[0] = (_Float16)g;
    p[a.gate_n] = (_Float16)u;
  }
  static_cast<_Float16*>(a.C)[(size_t)row * a.gate_n + c.col] = (_Float16)(gate_act(a, g) * u);
}
// where integer split-K atomics add up: C itself, or the workspace when the
// output is dequantised afterwards
__device__ __forceinline__ int* int_atomic_target(const RunArgs& a) {
  return static_cast<int*>(a.row_scale ? a.ws : a.C);
}

// Split units [u0, u1) of K part `part` (contiguous, as even as integers allow).
// Without a split the 64-bit division, which costs a measurable part of a
// microsecond-scale kernel's start, is skipped.
__device__ __forceinline__ void part_units(const RunArgs& a, int part, int& u0, int& u1) {
  u0 = 0;
  u1 = a.n_units;
  if (a.k_parts != 1) {
    u0 = (int)((int64_t)part * a.n_units / a.k_parts);
    u1 = (int)((int64_t)(part + 1) * a.n_units / a.k_parts);
  }
}

// the 256 x 256 tiles of four 128 x 128 waves (mfma_big.hip) for the formats that
// take them (0: the eight-wave tile of mfma_dl.hip for every format)
#ifndef QG_BIG4
#define QG_BIG4 1
#endif

// kernel launchers (return hipSuccess or the launch error)
// canonical arrays of a projection: words or values [N, K], scales and zero points [N, G]
struct Canonical {
  const void *w, *s, *z;
};
// up, if given, is the up projection of a gated plan of N output columns per projection
// (L.N is then gate_inner(N))
hipError_t launch_pack(const Layout& L, int64_t N, const Canonical& gate, const Canonical* up, void* packed,
                       hipStream_t st);
hipError_t launch_gemv(int fmt, const RunArgs& a, hipStream_t st);
// M = 1 with 16-column workgroups (gemv16.hip), for matrices with few 64-column blocks
hipError_t launch_gemv16(int fmt, const RunArgs& a, hipStream_t st);
// int8 / int2 skinny-M on the matrix cores, B operands straight from the blob (gemv_mfma.hip)
hipError_t launch_gemv_mfma(int fmt, const RunArgs& a, hipStream_t st);
// int4 / uint4 skinny-M (M <= 32) on the matrix cores, bias-folded B operands (gemv_mfma4.hip)
hipError_t launch_gemv_mfma4(int fmt, const RunArgs& a, hipStream_t st);
hipError_t launch_mfma(int fmt, int tile, const RunArgs& a, hipStream_t st);
// direct-load ring kernel (mfma_dl.hip): the tile for a problem, or -1 when the
// problem needs the LDS-staged kernel (int4 with per-piece scale groups)
enum DlTile : int {
  DL_32x64 = 0, DL_32x128, DL_32x256, DL_64x128, DL_64x256, DL_128x256, DL_256x256, DL_128x128, DL_NUM
};
void dl_tile_dims(int tile, int* bm, int* bn);
int choose_dl_tile(int fmt, int64_t M, int64_t N, int k_parts, int smode, bool gated);
hipError_t launch_mfma_dl(int fmt, int tile, const RunArgs& a, hipStream_t st);
hipError_t launch_mfma_dl_gated(int fmt, int tile, const RunArgs& a, hipStream_t st);
hipError_t launch_mfma_dl_rows(int tile, const RunArgs& a, hipStream_t st);  // fp16 weights with a.row_scale
// 256 x 256 tiles of four 128 x 128 waves (mfma_big.hip) for the formats that
// big_tile_takes; same arguments and stage layout as launch_mfma_dl's 256 x 256 tile
bool big_tile_takes(int fmt, const RunArgs& a);
hipError_t launch_mfma_big(int fmt, const RunArgs& a, hipStream_t st);
// fp16 product against the transpose of the blob a.W (a.NB, a.nkb: that blob's), on the same
// tiles: a.N output columns are the blob's positions, a.K its columns in whole granules
hipError_t launch_mfma_big_transposed(const RunArgs& a, hipStream_t st);
hipError_t launch_fill_zero(void* p, size_t bytes, hipStream_t st);
// zr = the bf16 planes [R_hi | R_lo] of the group row sums of a.A (rows of a.K fp16
// values, scale groups of a.group_size positions, or one group when it is negative)
// for the zero-point folding of the 256 x 256 tiles; a.K / 32 <= ROWSUM_MAX_UNITS
constexpr int ROWSUM_MAX_UNITS = 8192;
hipError_t launch_group_rowsum(const RunArgs& a, uint16_t* zr, hipStream_t st);
// zp = the bf16 planes [P_hi | P_lo] of the per-column term of the folding for each of
// the Npad columns, from the (scale, zero) pairs a.S ([zr_G][Npad]), or for signed int4
// (a.zeros 0) from its fp16 scales with the offset 8 as the zero point
hipError_t launch_zero_planes(const RunArgs& a, uint16_t* zp, hipStream_t st);
// dst[m, k] = k < K ? A[m, k] : 0 for rows of Kpad elements of esz bytes (Kpad * esz a
// multiple of 16, dst 16-byte aligned; A any alignment of its element size)
hipError_t launch_pad_rows(const void* A, void* dst, int64_t M, int64_t K, int64_t Kpad, int esz,
                           hipStream_t st);
// C[m, n] = bias[n] (int32) for the integer atomics to add into
hipError_t launch_fill_bias(const RunArgs& a, hipStream_t st);
// per-row symmetric int8 quantisation of fp16 activations (quant.hip)
hipError_t launch_quantize_rows(const void* A, int64_t M, int64_t K, void* Q, float* scales, hipStream_t st);
// sums the per-part partials (or converts the atomic accumulator) into C;
// acc_fp: fp32 accumulator (fp16 activations), else int32
hipError_t launch_finalize(const RunArgs& a, int acc_fp, hipStream_t st);
// the same for a gated plan: sums the parts of both projections and writes C
hipError_t launch_finalize_gate(const RunArgs& a, int acc_fp, hipStream_t st);

// Passes of the gated backward (gated.hip): gradients of the pre-activations of M rows and
// N columns, row by row (inner column order, rows of kd values, times 1 / row_scale) if
// rowwise is given, and column by column (gate, then up: 2 N rows of mp values, times 1 /
// col_scale) if colwise is, with the bias gradients (each may be null) if bias_part is.
// row_top, col_top and bias_part are scratch: [gate_grad_col_tiles(N)][M],
// [gate_grad_row_tiles(M)][N] and [gate_grad_row_tiles(M)][2 N].
struct GateGradArgs {
  const _Float16 *preact, *dC;
  _Float16 *rowwise, *colwise, *dbias_gate, *dbias_up;
  float *row_scale, *col_scale, *row_top, *bias_part;
  uint32_t* col_top;
  int64_t mp;
  int32_t M, N, kd;
  float c0, c1;  // the activation's
};
hipError_t launch_gate_grad(const GateGradArgs& a, hipStream_t st);
int64_t gate_grad_row_tiles(int64_t M);
int64_t gate_grad_col_tiles(int64_t N);
// the transposed weights of a gated plan, and transposed fp16 rows, as fp16 blobs of layout `to`
hipError_t launch_transpose_blob(const Layout& L, int64_t gate_n, const void* packed, const Layout& to, void* out,
                                 hipStream_t st);
// the weights of an int4 / uint4 blob with scales as an fp16 blob of layout `to` (same columns)
hipError_t launch_expand_blob(const Layout& L, const void* packed, const Layout& to, void* out, hipStream_t st);
hipError_t launch_transpose_rows(const void* X, int64_t M, int64_t K, const Layout& to, void* out, hipStream_t st);

// rotation of new queries and keys, keys and values into the paged cache (kv_append.hip)
struct AppendArgs {
  const _Float16 *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // values between rows
  const float *cos, *sin;                // [n_positions][rot / 2]
  const int32_t* positions;
  const int64_t* slots;
  _Float16 *q_out, *k_cache, *v_cache;
  int64_t n_positions, n_pages;
  int32_t page, q_heads, kv_heads, D, rot, interleaved;
};
hipError_t launch_kv_append(const AppendArgs& a, int64_t T, hipStream_t st);

// attention over the paged cache (attention.hip)
struct AttnArgs {
  const _Float16 *q, *k, *v;
  _Float16* out;
  float* lse;
  const int32_t *q_starts, *kv_lens, *tables, *prefix_table;
  int64_t q_stride, table_width, prefix_len;
  int32_t T, q_heads, kv_heads, D, n_pages, page_shift, max_q, max_len;
  float scale;
};
// sizes that the host knows, which choose the split of the work
struct AttnShape {
  int64_t T, B, max_q, max_len, prefix_len;
  int32_t q_heads, kv_heads, D;
};
bool attention_grid_fits(const AttnShape& s);  // row numbers in 32 bits, work items in a launch
size_t attention_ws_bytes(const AttnShape& s);
hipError_t launch_attention(const AttnArgs& a, const AttnShape& s, void* ws, hipStream_t st);

// GEMV tuning: most waves per workgroup (they split the workgroup's K range)
// and superblocks per register stage
#ifndef QG_GEMV_MAX_WAVES
#define QG_GEMV_MAX_WAVES 8
#endif
#ifndef QG_GEMV_UNR
#define QG_GEMV_UNR 1
#endif
#ifndef QG_GEMV_UNR_I2
#define QG_GEMV_UNR_I2 1
#endif
constexpr int GEMV_MAX_WAVES = QG_GEMV_MAX_WAVES;

// tiles of the LDS-staged MFMA kernel (mfma.hip), used where the direct-load kernel
// is not: TILE_BIG is 256 x 256 for fp16 / int8 and 256 x 128 for int4 / int2
enum Tile : int { TILE_32x64 = 0, TILE_64x64 = 1, TILE_128x128 = 2, TILE_BIG = 3 };
void tile_dims(int fmt, int tile, int* bm, int* bn);

}  // namespace qg
