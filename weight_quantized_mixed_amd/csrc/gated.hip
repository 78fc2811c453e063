// Backward pass of the gated feed-forward block C = act(g) * u, g = A Wg + bg,
// u = A Wu + bu, from the pre-activations that the forward kept:
//   dU = dC act(g)     dG = dC u act'(g)
//   dA = dG Wg^T + dU Wu^T     dWg = dG^T A     dWu = dU^T A     db = column sums
// The three products are the library's fp16 products ("nt": both operands run along the
// reduction), so this file holds the passes that bring their operands into that form:
// the gradients of the pre-activations, once per row (operand of dA) and once per
// column (operand of dW), and the transposed weights and activations in the packed
// superblocks of the fp16 format.  All of them read and write each value once and are
// bound by HBM; the transposes go through LDS so that both sides are contiguous (N = 11008,
// K = 4096: gradients of the pre-activations both ways at M = 2048 57 us for 315 MB, row by
// row at M = 1024 24 us for 113 MB; the transposed int4 weights 47 us for 225 MB; X of 2048
// rows 7 us).
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

// rows [m][2 N] of preact and [m][N] of dC -> rowwise [m][kd] (inner order, zero past the
// last inner column) and, if colwise is given, [2 N][mp] (gate rows, then up rows; zero
// for m in [M, mp)) and bias_part [row tile][2 N], the sums over the tile's rows in fp32, of
// the values before their rounding (rounded, those below 2^-25 would be lost one by one).
// V: values per access (8 or 2 where N and the pointers allow it).
template <int V>
__global__ __launch_bounds__(256) void gate_grad_kernel(const _Float16* __restrict__ preact,
                                                        const _Float16* __restrict__ dC, int M, int N, int kd,
                                                        int64_t mp, float c0, float c1,
                                                        _Float16* __restrict__ rowwise,
                                                        _Float16* __restrict__ colwise,
                                                        float* __restrict__ bias_part) {
  constexpr int PER_ROW = GT / V, STEPS = GT * PER_ROW / 256, AT_ONCE = STEPS < 4 ? STEPS : 4;
  __shared__ __attribute__((aligned(16))) union {
    _Float16 t[2][GT][GPITCH];          // [gate, up][column][row]
    float sums[256 / PER_ROW][2][GT];   // then the column sums of the threads' rows
  } lds;
  auto& t = lds.t;
  const int m0 = blockIdx.y * GT, n0 = blockIdx.x * GT;
  float sum[2][V] = {};  // a thread's rows lie in the same V columns
  typedef _Float16 vec __attribute__((ext_vector_type(V)));
#pragma unroll 1
  for (int s0 = 0; s0 < STEPS; s0 += AT_ONCE) {
    // the loads of a few steps before their first use
    vec g[AT_ONCE], u[AT_ONCE], d[AT_ONCE];
#pragma unroll
    for (int s = 0; s < AT_ONCE; ++s) {
      const int i = (s0 + s) * 256 + threadIdx.x, m = m0 + i / PER_ROW, n = n0 + (i % PER_ROW) * V;
      g[s] = u[s] = d[s] = vec{};
      if (m < M && n < N) {  // N is a multiple of V
        const _Float16* p = preact + (size_t)m * 2 * N + n;
        g[s] = *reinterpret_cast<const vec*>(p);
        u[s] = *reinterpret_cast<const vec*>(p + N);
        d[s] = *reinterpret_cast<const vec*>(dC + (size_t)m * N + n);
      }
    }
#pragma unroll
    for (int s = 0; s < AT_ONCE; ++s) {
      const int i = (s0 + s) * 256 + threadIdx.x, r = i / PER_ROW, m = m0 + r, n = n0 + (i % PER_ROW) * V;
      vec dg, du;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float x = kept(g[s][e]), dc = (float)d[s][e];
        const float sg = gate_sigmoid(c0, c1, x);
        // act'(x) = sg + x sg (1 - sg) t'(x)
        const float gx = dc * kept(u[s][e]) * (sg + x * sg * (1.f - sg) * (c0 + 3.f * c1 * x * x)), ux = dc * x * sg;
        sum[0][e] += gx;
        sum[1][e] += ux;
        dg[e] = (_Float16)gx;
        du[e] = (_Float16)ux;
      }
      if (rowwise && m < M) {
        const int c = (n >> 4) * 32 + (n & 15);
        _Float16* o = rowwise + (size_t)m * kd + c;
        if (c < kd) *reinterpret_cast<vec*>(o) = dg;
        if (c + 16 < kd) *reinterpret_cast<vec*>(o + 16) = du;
      }
      if (colwise) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          t[0][n - n0 + e][r] = dg[e];
          t[1][n - n0 + e][r] = du[e];
        }
      }
    }
  }
  if (!colwise) return;
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * GT * (GT / 8); i += 256) {
    const int p = i / (GT * GT / 8), c = (i / (GT / 8)) % GT, m = (i % (GT / 8)) * 8, n = n0 + c;
    if (n < N) *reinterpret_cast<half8v*>(colwise + ((size_t)p * N + n) * mp + m0 + m) = *reinterpret_cast<half8v*>(&t[p][c][m]);
  }
  if (!bias_part) return;
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int e = 0; e < V; ++e) lds.sums[threadIdx.x / PER_ROW][p][threadIdx.x % PER_ROW * V + e] = sum[p][e];
  __syncthreads();
  if (threadIdx.x < 2 * GT) {
    const int p = threadIdx.x / GT, c = threadIdx.x % GT;
    float s = 0.f;
    for (int r = 0; r < 256 / PER_ROW; ++r) s += lds.sums[r][p][c];
    if (n0 + c < N) bias_part[(size_t)blockIdx.y * 2 * N + (size_t)p * N + n0 + c] = s;
  }
}

// column sums of the tiles' sums, in tile order
__global__ void bias_grad_kernel(const float* __restrict__ part, int tiles, int N, _Float16* __restrict__ dbg,
                                 _Float16* __restrict__ dbu) {
  const int n = blockIdx.x * blockDim.x + threadIdx.x;
  if (n >= 2 * N) return;
  float s = 0.f;
  for (int t = 0; t < tiles; ++t) s += part[(size_t)t * 2 * N + n];
  _Float16* out = n < N ? dbg : dbu;
  if (out) out[n < N ? n : n - N] = (_Float16)s;
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
// (q - z) s in fp32, rounded once to fp16 (the operand type of the product).
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
// Bound by HBM: 22016 columns, K = 4096 (208 MB) 37 us, 5.6 TB/s.
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

hipError_t launch_gate_grad(const void* preact, const void* dC, int64_t M, int64_t N, int64_t kd, int64_t mp, float c0,
                            float c1, void* rowwise, void* colwise, float* bias_part, hipStream_t st) {
  // column tiles cover the inner columns' padding of rowwise too (kd / 2 output columns)
  const int64_t cols = rowwise && kd / 2 > N ? kd / 2 : N;
  const dim3 grid((unsigned)((cols + GT - 1) / GT), (unsigned)((M + GT - 1) / GT));
  const uintptr_t at = reinterpret_cast<uintptr_t>(preact) | reinterpret_cast<uintptr_t>(dC);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, static_cast<const _Float16*>(preact),
                       static_cast<const _Float16*>(dC), (int)M, (int)N, (int)kd, mp, c0, c1,
                       static_cast<_Float16*>(rowwise), static_cast<_Float16*>(colwise), bias_part);
  };
  if (N % 8 == 0 && (at & 15) == 0) go(gate_grad_kernel<8>);
  else if (N % 2 == 0 && (at & 3) == 0) go(gate_grad_kernel<2>);
  else go(gate_grad_kernel<1>);
  return hipGetLastError();
}

hipError_t launch_bias_grad(const float* part, int64_t M, int64_t N, void* dbg, void* dbu, hipStream_t st) {
  hipLaunchKernelGGL(bias_grad_kernel, dim3((unsigned)((2 * N + 255) / 256)), dim3(256), 0, st, part,
                     (int)((M + GT - 1) / GT), (int)N, static_cast<_Float16*>(dbg), static_cast<_Float16*>(dbu));
  return hipGetLastError();
}

int64_t gate_grad_row_tiles(int64_t M) { return (M + GT - 1) / GT; }

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
