// Backward pass of the gated feed-forward block C = act(g) * u, g = A Wg + bg,
// u = A Wu + bu, from the pre-activations that the forward kept:
//   dU = dC act(g)     dG = dC u act'(g)
//   dA = dG Wg^T + dU Wu^T     dWg = dG^T A     dWu = dU^T A     db = column sums
// The three products are the library's fp16 products ("nt": both operands run along the
// reduction), so this file holds the passes that bring their operands into that form:
// the gradients of the pre-activations, once per row (operand of dA) and once per
// column (operand of dW), and the transposed weights and activations in the packed
// superblocks of the fp16 format.  The gradients of the pre-activations are rounded to fp16
// for that, the operand type of the matrix cores at their full rate (split into two halves they
// would double the products), each sum's terms at a common scale where fp16's range asks for
// one.  All of the passes read and write each value once and are
// bound by HBM; the transposes go through LDS so that both sides are contiguous (N = 11008,
// K = 4096: gradients of the pre-activations both ways at M = 2048 58 us for 319 MB and 5 us to
// check their range, row by row at M = 1024 23 us for 114 MB and 5 us; the transposed int4
// weights 47 us for 225 MB; X of 2048 rows 8 us).
//
// dA runs as one product over the inner columns of the gated plan (gate and up blocks of
// 16 alternate), so its weight operand is the transpose of the forward's blob, whatever
// format that has.  Where the product takes the 256 x 256 tiles and the weights are fp16, it
// reads that blob itself (mfma_big.hip), and no transposed copy is made.
#include "qgemm_internal.hpp"

namespace qg {
namespace {

typedef _Float16 half8v __attribute__((ext_vector_type(8)));

__device__ __forceinline__ _Float16 as_half(uint32_t x) { return __builtin_bit_cast(_Float16, (uint16_t)x); }

// A pre-activation past fp16 was kept as infinity: the largest value instead, since infinity
// times 0 (a saturated gate's act', or a dC of 0) would be NaN.  A gate there has act' 0 or 1
// already; an up projection's share in dG is the one of 65504.  NaN stays.
__device__ __forceinline__ float kept(_Float16 h) {
  const float x = (float)h;
  return fabsf(x) == INFINITY ? copysignf(65504.f, x) : x;
}

// ---- gradients of the pre-activations: tiles of 64 rows x 64 output columns
constexpr int GT = 64;
constexpr int GPITCH = GT + 8;  // halves per LDS row (16-byte aligned rows, banks shifted by 4)

// A sum's terms (a row of dG and dU for dA, a column of one of them for dW) are fp16 operands,
// 11 bits of any term from 2^-14 on.  Where the largest term is past fp16 or below 2^-6
// (from there up, 22016 terms lose below 2^-25 what the rounding of the largest alone loses),
// all of them are taken times 2^-e, which brings the largest to 2^13 .. 2^14, and the
// product's fp32 sum times 2^e.  Ordinary rows and columns have e = 0.
// top: the largest term, cut to the upper half of its bits (65280 then stands for all up to
// 65536).
constexpr float TOP_MOST = 65280.f, TOP_LEAST = 0x1p-6f;
__device__ __forceinline__ int range_shift(float top) {
  if (!(top > 0.f) || top == INFINITY || (top >= TOP_LEAST && top < TOP_MOST)) return 0;
  return max(ilogbf(top) - 13, -64);
}
// two magnitudes' upper halves in a word, and their maxima (the bits order like the values)
__device__ __forceinline__ uint32_t upper_halves(float lo, float hi) {
  return (__float_as_uint(hi) & 0xFFFF0000u) | (__float_as_uint(lo) >> 16);
}
__device__ __forceinline__ uint32_t larger_halves(uint32_t x, uint32_t y) {
  typedef uint16_t ushort2v __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(ushort2v, x), __builtin_bit_cast(ushort2v, y)));
}

// dG and dU of V outputs in fp32
template <int V>
struct GateGrads {
  float g[V], u[V];
};
template <int V, typename VEC>
__device__ __forceinline__ GateGrads<V> gate_grads(const GateGradArgs& a, const VEC& g, const VEC& u, const VEC& d) {
  GateGrads<V> r;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float x = kept(g[e]), dc = (float)d[e];
    const float sg = gate_sigmoid(a.c0, a.c1, x);
    // act'(x) = sg + x sg (1 - sg) t'(x)
    r.g[e] = dc * kept(u[e]) * (sg + x * sg * (1.f - sg) * (a.c0 + 3.f * a.c1 * x * x));
    r.u[e] = dc * x * sg;
  }
  return r;
}

// [gate, up][column][row] of a tile; the threads' shares of the columns' maxima (both
// projections' in a word) or of their sums
template <int V>
union GradTile {
  _Float16 t[2][GT][GPITCH];
  uint32_t top[256 / (GT / V)][GT];
  float sum[256 / (GT / V)][2][GT];
};

// an LDS tile to its places in colwise
template <int V>
__device__ __forceinline__ void store_columns(const GateGradArgs& a, const GradTile<V>& lds, int m0, int n0) {
  for (int i = threadIdx.x; i < 2 * GT * (GT / 8); i += 256) {
    const int p = i / (GT * GT / 8), c = (i / (GT / 8)) % GT, m = (i % (GT / 8)) * 8, n = n0 + c;
    if (n < a.N)
      *reinterpret_cast<half8v*>(a.colwise + ((size_t)p * a.N + n) * a.mp + m0 + m) =
          *reinterpret_cast<const half8v*>(&lds.t[p][c][m]);
  }
}

// rows [m][2 N] of preact and [m][N] of dC -> rowwise [m][kd] (inner order, zero past the
// last inner column) and, if colwise is given, [2 N][mp] (gate rows, then up rows; zero
// for m in [M, mp)), all unscaled, with the largest magnitudes of the tile's rows and
// columns, and bias_part [row tile][2 N], the sums over the tile's rows in fp32, of
// the values before their rounding (rounded, those below 2^-25 would be lost one by one).
// V: values per access (8 or 2 where N and the pointers allow it).
template <int V>
__global__ __launch_bounds__(256) void gate_grad_kernel(GateGradArgs a) {
  constexpr int PER_ROW = GT / V, STEPS = GT * PER_ROW / 256, AT_ONCE = STEPS < 4 ? STEPS : 4;
  typedef _Float16 vec __attribute__((ext_vector_type(V)));
  __shared__ __attribute__((aligned(16))) GradTile<V> lds;
  const int m0 = blockIdx.y * GT, n0 = blockIdx.x * GT, N = a.N;
  // a thread's rows lie in the same V columns
  float sum[2][V] = {}, top[2][V] = {};
#pragma unroll 1
  for (int s0 = 0; s0 < STEPS; s0 += AT_ONCE) {
    // the loads of a few steps before their first use
    vec g[AT_ONCE], u[AT_ONCE], d[AT_ONCE];
#pragma unroll
    for (int s = 0; s < AT_ONCE; ++s) {
      const int i = (s0 + s) * 256 + threadIdx.x, m = m0 + i / PER_ROW, n = n0 + (i % PER_ROW) * V;
      g[s] = u[s] = d[s] = vec{};
      if (m < a.M && n < N) {  // N is a multiple of V
        const _Float16* p = a.preact + (size_t)m * 2 * N + n;
        g[s] = *reinterpret_cast<const vec*>(p);
        u[s] = *reinterpret_cast<const vec*>(p + N);
        d[s] = *reinterpret_cast<const vec*>(a.dC + (size_t)m * N + n);
      }
    }
#pragma unroll
    for (int s = 0; s < AT_ONCE; ++s) {
      const int i = (s0 + s) * 256 + threadIdx.x, r = i / PER_ROW, m = m0 + r, n = n0 + (i % PER_ROW) * V;
      const GateGrads<V> x = gate_grads<V>(a, g[s], u[s], d[s]);
      vec dg, du;
      float most = 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        sum[0][e] += x.g[e];
        sum[1][e] += x.u[e];
        top[0][e] = fmaxf(top[0][e], fabsf(x.g[e]));
        top[1][e] = fmaxf(top[1][e], fabsf(x.u[e]));
        most = fmaxf(most, fmaxf(fabsf(x.g[e]), fabsf(x.u[e])));
        dg[e] = (_Float16)x.g[e];
        du[e] = (_Float16)x.u[e];
      }
      if (a.rowwise) {
        if (m < a.M) {
          const int c = (n >> 4) * 32 + (n & 15);
          _Float16* o = a.rowwise + (size_t)m * a.kd + c;
          if (c < a.kd) *reinterpret_cast<vec*>(o) = dg;
          if (c + 16 < a.kd) *reinterpret_cast<vec*>(o + 16) = du;
        }
#pragma unroll
        for (int o = PER_ROW / 2; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor(most, o, 64));
        if (i % PER_ROW == 0 && m < a.M) a.row_top[(size_t)blockIdx.x * a.M + m] = most;
      }
      if (a.colwise) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          lds.t[0][n - n0 + e][r] = dg[e];
          lds.t[1][n - n0 + e][r] = du[e];
        }
      }
    }
  }
  if (!a.colwise) return;
  __syncthreads();
  store_columns<V>(a, lds, m0, n0);
  // over the threads of a column, in order
  const int own_row = threadIdx.x / PER_ROW, own_col = threadIdx.x % PER_ROW * V;
  __syncthreads();
#pragma unroll
  for (int e = 0; e < V; ++e) lds.top[own_row][own_col + e] = upper_halves(top[0][e], top[1][e]);
  __syncthreads();
  if (threadIdx.x < GT && n0 + (int)threadIdx.x < N) {
    uint32_t x = 0;
#pragma unroll 8
    for (int r = 0; r < 256 / PER_ROW; ++r) x = larger_halves(x, lds.top[r][threadIdx.x]);
    a.col_top[(size_t)blockIdx.y * N + n0 + threadIdx.x] = x;
  }
  if (!a.bias_part) return;
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int e = 0; e < V; ++e) lds.sum[own_row][p][own_col + e] = sum[p][e];
  __syncthreads();
  const int p = threadIdx.x / GT, c = threadIdx.x % GT;
  if (p < 2 && n0 + c < N) {
    float x = 0.f;
    for (int r = 0; r < 256 / PER_ROW; ++r) x += lds.sum[r][p][c];
    a.bias_part[(size_t)blockIdx.y * 2 * N + (size_t)p * N + n0 + c] = x;
  }
}

// What is left when every tile is done: the scales of rows and columns from their tiles'
// largest magnitudes, the rows and columns whose scale is not 1 over again, scaled, and the
// bias gradients, the tiles' sums in tile order.  The first row_blocks workgroups take a row a
// wave, the next col_blocks a strip of 64 columns, the others 256 bias gradients.  Ordinary
// gradients leave it at reading the magnitudes, one or two in 64 of the values.
template <int V>
__global__ __launch_bounds__(256) void gate_grad_range_kernel(GateGradArgs a, int row_blocks, int col_blocks, int col_tiles,
                                                              int row_tiles) {
  constexpr int PER_ROW = GT / V;
  typedef _Float16 vec __attribute__((ext_vector_type(V)));
  __shared__ __attribute__((aligned(16))) GradTile<V> lds;
  __shared__ float factor[2][GT];
  const int N = a.N;
  if ((int)blockIdx.x < row_blocks) {
    const int lane = threadIdx.x & 63, m = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (m >= a.M) return;
    float top = 0.f;
    for (int i = lane; i < col_tiles; i += 64) top = fmaxf(top, a.row_top[(size_t)i * a.M + m]);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    const int e = range_shift(__uint_as_float(__float_as_uint(top) & 0xFFFF0000u));
    if (lane == 0) a.row_scale[m] = ldexpf(1.f, e);
    if (e == 0) return;
    const float f = ldexpf(1.f, -e);
    for (int n = lane * V; n < N; n += 64 * V) {
      const _Float16* p = a.preact + (size_t)m * 2 * N + n;
      const GateGrads<V> x = gate_grads<V>(a, *reinterpret_cast<const vec*>(p), *reinterpret_cast<const vec*>(p + N),
                                           *reinterpret_cast<const vec*>(a.dC + (size_t)m * N + n));
      vec dg, du;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        dg[i] = (_Float16)(x.g[i] * f);
        du[i] = (_Float16)(x.u[i] * f);
      }
      _Float16* o = a.rowwise + (size_t)m * a.kd + (n >> 4) * 32 + (n & 15);
      *reinterpret_cast<vec*>(o) = dg;
      *reinterpret_cast<vec*>(o + 16) = du;
    }
    return;
  }
  if ((int)blockIdx.x >= row_blocks + col_blocks) {
    const int n = ((int)blockIdx.x - row_blocks - col_blocks) * 256 + threadIdx.x;
    _Float16* out = n < N ? a.dbias_gate : a.dbias_up;
    if (n >= 2 * N || !out) return;
    float s = 0.f;
#pragma unroll 8
    for (int t = 0; t < row_tiles; ++t) s += a.bias_part[(size_t)t * 2 * N + n];
    out[n < N ? n : n - N] = (_Float16)s;
    return;
  }
  const int n0 = ((int)blockIdx.x - row_blocks) * GT, n = n0 + threadIdx.x % GT;
  uint32_t top = 0;  // a quarter of the tiles a wave
  if (n < N) {
#pragma unroll 8
    for (int t = threadIdx.x / GT; t < row_tiles; t += 4) top = larger_halves(top, a.col_top[(size_t)t * N + n]);
  }
  lds.top[threadIdx.x / GT][threadIdx.x % GT] = top;
  __syncthreads();
  int e = 0;
  if (threadIdx.x < 2 * GT) {
    const int p = threadIdx.x / GT, c = threadIdx.x % GT;
    for (int w = 0; w < 4; ++w) top = larger_halves(top, lds.top[w][c]);
    e = range_shift(__uint_as_float(p ? top & 0xFFFF0000u : top << 16));
    factor[p][c] = ldexpf(1.f, -e);
    if (n < N) a.col_scale[(size_t)p * N + n] = ldexpf(1.f, e);
  }
  if (!__syncthreads_or(e != 0)) return;
  for (int m0 = 0; m0 < a.M; m0 += GT) {
    for (int i = threadIdx.x; i < GT * PER_ROW; i += 256) {
      const int r = i / PER_ROW, m = m0 + r, n = n0 + (i % PER_ROW) * V;
      vec g = {}, u = {}, d = {};
      if (m < a.M && n < N) {
        const _Float16* p = a.preact + (size_t)m * 2 * N + n;
        g = *reinterpret_cast<const vec*>(p);
        u = *reinterpret_cast<const vec*>(p + N);
        d = *reinterpret_cast<const vec*>(a.dC + (size_t)m * N + n);
      }
      const GateGrads<V> x = gate_grads<V>(a, g, u, d);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        lds.t[0][n - n0 + j][r] = (_Float16)(x.g[j] * factor[0][n - n0 + j]);
        lds.t[1][n - n0 + j][r] = (_Float16)(x.u[j] * factor[1][n - n0 + j]);
      }
    }
    __syncthreads();
    store_columns<V>(a, lds, m0, n0);
    __syncthreads();
  }
}

// ---- transposed operands: tiles of 32 reduction positions x 128 columns through LDS
constexpr int TP = 32, TC = 128, TPITCH = TC + 8;

// writes the LDS tile t[position][column] as the 8 superblocks (16 columns x 32 positions)
// of an fp16 blob of nb column blocks: tile row kb, tile columns col0 ..
__device__ __forceinline__ void store_superblocks(const _Float16 (&t)[TP][TPITCH], uint4* __restrict__ out, int kb,
                                                  int col0, int nb) {
  for (int i = threadIdx.x; i < TC / 16 * 64; i += 256) {
    const int b = i >> 6, q = (i >> 4) & 3, c = b * 16 + (i & 15);
    if (col0 / 16 + b >= nb) continue;
    half8v v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = t[q * 8 + e][c];
    out[((size_t)kb * nb + col0 / 16 + b) * 64 + (i & 63)] = __builtin_bit_cast(uint4, v);
  }
}

// Transpose of a gated plan's blob into the fp16 blob of the dA product: its columns are
// the K positions of the forward's weights, its reduction the inner columns.  A value is
// (q - z) s in fp32, rounded once to fp16, the operand type of the product (a scale cannot leave
// the sum here: it changes along the reduction).
template <int FMT>
__global__ __launch_bounds__(256) void transpose_blob_kernel(const uint4* __restrict__ W, const void* __restrict__ S,
                                                             int NB, int Npad, int nkb, int gate_n, int group_size,
                                                             int zeros, uint4* __restrict__ out, int out_nb) {
  __shared__ _Float16 t[TP][TPITCH];
  const int col0 = blockIdx.x * TC, kb = blockIdx.y, c0 = kb * TP;  // forward positions, inner columns
  constexpr int KB = kb_of(FMT), Q = KB / 4;
  constexpr int PIECES = TP * (TC / Q);  // pieces of 16 bytes: Q positions of an inner column
  for (int i = threadIdx.x; i < PIECES; i += 256) {
    const int l = i & 63, sb = i >> 6;                       // lane order of a superblock
    const int cb = sb % (TP / 16), kk = sb / (TP / 16);      // its column block and K block within the tile
    const int c = c0 + cb * 16 + (l & 15), k0 = col0 + kk * KB + (l >> 4) * Q;
    const int src = (c >> 5) * 16 + (c & 15);
    const bool in = c < NB * 16 && src < gate_n && k0 / KB < nkb;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (in) w = W[((size_t)(k0 / KB) * NB + c / 16) * 64 + l];
    _Float16* dst = &t[cb * 16 + (l & 15)][k0 - col0];
    const uint32_t wd[4] = {w.x, w.y, w.z, w.w};
    if constexpr (FMT == FMT_F16) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        dst[2 * e] = as_half(wd[e] & 0xFFFFu);
        dst[2 * e + 1] = as_half(wd[e] >> 16);
      }
    } else {
      float s = 1.f, z = 0.f;
      if (in && S) {
        const size_t o = (size_t)(group_size > 0 ? k0 / group_size : 0) * Npad + c;
        if (zeros) {
          const uint32_t sz = static_cast<const uint32_t*>(S)[o];
          s = (float)as_half(sz & 0xFFFFu);
          z = (float)as_half(sz >> 16);
        } else {
          s = (float)as_half(static_cast<const uint16_t*>(S)[o]);
        }
      }
      if (FMT == FMT_I4) z += 8.f;  // codes are stored as q + 8
      if (!in) s = 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int slot = (e & 1) ? 4 + (e >> 1) : (e >> 1);
          dst[8 * x + e] = (_Float16)(((float)((wd[x] >> (4 * slot)) & 15u) - z) * s);
        }
    }
  }
  __syncthreads();
  store_superblocks(t, out, kb, col0, out_nb);
}

// (q - z) s of a packed int4 / uint4 blob, rounded once, as the fp16 blob of the same columns.
// A thread takes a piece of 32 positions of a column (they share a group) to the four
// pieces of 8 of one fp16 superblock; a wave's 16-byte stores fill whole superblocks.
// Bound by HBM: 22016 columns, K = 4096, groups of 64 (228 MB) 36 us, 6.3 TB/s.
template <int FMT>
__global__ __launch_bounds__(256) void expand_blob_kernel(const uint4* __restrict__ W, const void* __restrict__ S, int NB,
                                                          int Npad, int64_t pieces, int group_size, int zeros,
                                                          uint4* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= pieces) return;
  const int l = (int)(i & 63), q = l >> 4, c16 = l & 15;
  const int64_t sb = i >> 6, kb = sb / NB;
  const int cb = (int)(sb % NB);
  const size_t o = (size_t)((kb * kb_of(FMT) + q * 32) / group_size) * Npad + cb * 16 + c16;
  float s, z = 0.f;
  if (zeros) {
    const uint32_t sz = static_cast<const uint32_t*>(S)[o];
    s = (float)as_half(sz & 0xFFFFu);
    z = (float)as_half(sz >> 16);
  } else {
    s = (float)as_half(static_cast<const uint16_t*>(S)[o]);
  }
  if (FMT == FMT_I4) z += 8.f;  // codes are stored as q + 8
  const uint4 w = W[i];
  const uint32_t wd[4] = {w.x, w.y, w.z, w.w};
  uint4* dst = out + ((kb * (kb_of(FMT) / 32) + q) * NB + cb) * 64 + c16;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    typedef _Float16 half8v __attribute__((ext_vector_type(8)));
    half8v v;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int slot = (e & 1) ? 4 + (e >> 1) : (e >> 1);
      v[e] = (_Float16)(((float)((wd[x] >> (4 * slot)) & 15u) - z) * s);
    }
    dst[16 * x] = __builtin_bit_cast(uint4, v);
  }
}

// Transpose of fp16 rows X [M][K] into the fp16 blob of the dW products: columns K,
// reduction over the rows (zero past M).  VEC: rows are whole aligned 16-byte groups.
template <bool VEC>
__global__ __launch_bounds__(256) void transpose_rows_kernel(const _Float16* __restrict__ X, int M, int K,
                                                             uint4* __restrict__ out, int out_nb) {
  __shared__ __attribute__((aligned(16))) _Float16 t[TP][TPITCH];
  const int col0 = blockIdx.x * TC, kb = blockIdx.y;
  constexpr int V = VEC ? 8 : 1;
  typedef _Float16 vec __attribute__((ext_vector_type(V)));
  for (int i = threadIdx.x; i < TP * TC / V; i += 256) {
    const int r = i / (TC / V), c = (i % (TC / V)) * V, m = kb * TP + r;
    vec v = {};
    if (m < M && col0 + c < K) v = *reinterpret_cast<const vec*>(X + (size_t)m * K + col0 + c);
    *reinterpret_cast<vec*>(&t[r][c]) = v;
  }
  __syncthreads();
  store_superblocks(t, out, kb, col0, out_nb);
}

}  // namespace

hipError_t launch_gate_grad(const GateGradArgs& a, hipStream_t st) {
  const int64_t cols = gate_grad_col_tiles(a.N), rows = gate_grad_row_tiles(a.M);
  const int row_blocks = a.rowwise ? (a.M + 3) / 4 : 0, col_blocks = a.colwise ? (a.N + GT - 1) / GT : 0;
  const int bias_blocks = a.bias_part ? (2 * a.N + 255) / 256 : 0;
  auto go = [&](auto first, auto second) {
    hipLaunchKernelGGL(first, dim3((unsigned)cols, (unsigned)rows), dim3(256), 0, st, a);
    hipLaunchKernelGGL(second, dim3((unsigned)(row_blocks + col_blocks + bias_blocks)), dim3(256), 0, st, a, row_blocks,
                       col_blocks, (int)cols, (int)rows);
  };
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.preact) | reinterpret_cast<uintptr_t>(a.dC);
  if (a.N % 8 == 0 && (at & 15) == 0) go(gate_grad_kernel<8>, gate_grad_range_kernel<8>);
  else if (a.N % 2 == 0 && (at & 3) == 0) go(gate_grad_kernel<2>, gate_grad_range_kernel<2>);
  else go(gate_grad_kernel<1>, gate_grad_range_kernel<1>);
  return hipGetLastError();
}

int64_t gate_grad_row_tiles(int64_t M) { return (M + GT - 1) / GT; }
// the inner columns' padding of rowwise too (whole granules of 64 inner columns, 32 of the output)
int64_t gate_grad_col_tiles(int64_t N) { return ((gate_inner(N) + 63) / 64 * 32 + GT - 1) / GT; }

hipError_t launch_transpose_blob(const Layout& L, int64_t gate_n, const void* packed, const Layout& to, void* out,
                                 hipStream_t st) {
  const dim3 grid((unsigned)((to.Npad + TC - 1) / TC), (unsigned)to.nkb);
  const void* S = L.G ? static_cast<const char*>(packed) + L.s_offset : nullptr;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, static_cast<const uint4*>(packed), S, (int)L.NB, (int)L.Npad,
                       (int)L.nkb, (int)gate_n, (int)L.group_size, L.zeros ? 1 : 0, static_cast<uint4*>(out),
                       (int)to.NB);
  };
  switch (L.fmt) {
    case FMT_I4: go(transpose_blob_kernel<FMT_I4>); break;
    case FMT_U4: go(transpose_blob_kernel<FMT_U4>); break;
    case FMT_F16: go(transpose_blob_kernel<FMT_F16>); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t launch_expand_blob(const Layout& L, const void* packed, const Layout& to, void* out, hipStream_t st) {
  static_assert(kb_of(FMT_I4) == 128 && kb_of(FMT_U4) == 128 && kb_of(FMT_F16) == 32, "pieces of 32 and 8 positions");
  if (L.NB != to.NB || L.nkb * 4 != to.nkb || L.group_size < 32) return hipErrorInvalidValue;
  const int64_t pieces = L.nkb * L.NB * 64;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)((pieces + 255) / 256)), dim3(256), 0, st, static_cast<const uint4*>(packed),
                       static_cast<const char*>(packed) + L.s_offset, (int)L.NB, (int)L.Npad, pieces, (int)L.group_size,
                       L.zeros ? 1 : 0, static_cast<uint4*>(out));
    return hipGetLastError();
  };
  return L.fmt == FMT_I4 ? go(expand_blob_kernel<FMT_I4>)
         : L.fmt == FMT_U4 ? go(expand_blob_kernel<FMT_U4>)
                           : hipErrorInvalidValue;
}

hipError_t launch_transpose_rows(const void* X, int64_t M, int64_t K, const Layout& to, void* out, hipStream_t st) {
  const dim3 grid((unsigned)((to.Npad + TC - 1) / TC), (unsigned)to.nkb);
  const bool vec = K % 8 == 0 && (reinterpret_cast<uintptr_t>(X) & 15) == 0;
  if (vec)
    hipLaunchKernelGGL(transpose_rows_kernel<true>, grid, dim3(256), 0, st, static_cast<const _Float16*>(X), (int)M,
                       (int)K, static_cast<uint4*>(out), (int)to.NB);
  else
    hipLaunchKernelGGL(transpose_rows_kernel<false>, grid, dim3(256), 0, st, static_cast<const _Float16*>(X), (int)M,
                       (int)K, static_cast<uint4*>(out), (int)to.NB);
  return hipGetLastError();
}

}  // namespace qg
