// Norms of queries and keys for each head with the rotation of their positions in one pass,
// and the gradients of both.
//
//   r = (mean x^2 + eps)^(-1/2),  n = x r w,  y = R(p) n
//   g = R(-p) dy,  dw = sum x r g,  h = g w,  dx = r h - x r^3 mean(x h)
// with R(p) the rotation of the pairs by the angles of position p, whose transpose is its
// inverse for angles on the unit circle (for any others g takes the transpose, as a gradient
// does).
//
// Every value is read once and written once, so the passes are bound by HBM (long prompts) or
// by the launch (a decode batch).  A head belongs to LPH lanes (4, 8 or 16 for up to 64, 128 or
// 256 values) of 16 values each, which are whole pairs: its sums are taken over those lanes by
// DPP, its pairs turn in registers, and nothing passes through LDS.  A lane's values are 8 / V
// pieces of V pairs, where V is what alignment, strides and sizes allow in one access each.
//
// Measured: 48 tokens 3.7 us; 8190 tokens of 32 + 8 + 8 heads of 128 (201 MB) 35 to 39 us, as the
// caches have it; gradients of 4096 tokens of 32 + 8 heads (126 MB) 24.5 us, 5.1 TB/s (a
// 2 GiB copy reaches 4.85), the weights' second pass 4.0 us.
//
// The gradient of a norm's weight sums over tokens and heads: each lane adds up its own places
// over the rows that its workgroup walks (at most CHAIN), the workgroup joins its lanes and
// leaves one row of partial sums, and a second pass adds those in order (bitwise reproducible).
#include <type_traits>

#include "qgemm_internal.hpp"

namespace qg {
namespace {

template <int V>
struct Vec {
  typedef _Float16 h __attribute__((ext_vector_type(V)));
  typedef float f __attribute__((ext_vector_type(V)));
};

// sum over the LPH lanes of a head, in all of them
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
  v = add_dpp<0xB1>(v);                             // lanes 1 0 3 2 of each four
  v = add_dpp<0x4E>(v);                             // lanes 2 3 0 1
  if constexpr (LPH >= 8) v = add_dpp<0x141>(v);    // the other four of each eight (mirrored)
  if constexpr (LPH >= 16) v = add_dpp<0x140>(v);   // the other eight of each sixteen
  return v;
}

// where a lane's piece c of a head lies: places of its two V-vectors, and whether they turn
template <int V, bool INTERLEAVED>
struct Piece {
  int o0, o1, j;
  bool live, turn;
  __device__ __forceinline__ Piece(int c, int D, int half, bool turns) {
    j = c * V;
    live = j < D / 2;
    turn = turns && j < half;
    o0 = turn && !INTERLEAVED ? j : 2 * j;
    o1 = turn && !INTERLEAVED ? j + half : 2 * j + V;
  }
};

// places of pair e among the 2 V values of a turned piece
template <int V, bool INTERLEAVED>
__device__ __forceinline__ int first_of(int e) { return INTERLEAVED ? 2 * e : e; }
template <int V, bool INTERLEAVED>
__device__ __forceinline__ int second_of(int e) { return INTERLEAVED ? 2 * e + 1 : V + e; }

template <int V>
__device__ __forceinline__ void read(const _Float16* from, int o0, int o1, float* x) {
  typedef typename Vec<V>::h hv;
  const hv a = *reinterpret_cast<const hv*>(from + o0), b = *reinterpret_cast<const hv*>(from + o1);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    x[e] = (float)a[e];
    x[V + e] = (float)b[e];
  }
}
template <int V>
__device__ __forceinline__ void write(_Float16* to, int o0, int o1, const float* x) {
  typedef typename Vec<V>::h hv;
  hv a, b;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    a[e] = (_Float16)x[e];
    b[e] = (_Float16)x[V + e];
  }
  *reinterpret_cast<hv*>(to + o0) = a;
  *reinterpret_cast<hv*>(to + o1) = b;
}

// turns the pairs of a piece by the angles of position pos, or back (BACK: the transpose)
template <int V, bool INTERLEAVED, bool BACK>
__device__ __forceinline__ void rotate(float* x, const float* cos, const float* sin, int64_t at) {
  typedef typename Vec<V>::f fv;
  const fv c = *reinterpret_cast<const fv*>(cos + at), s = *reinterpret_cast<const fv*>(sin + at);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int ia = first_of<V, INTERLEAVED>(e), ib = second_of<V, INTERLEAVED>(e);
    const float p = x[ia], q = x[ib], t = BACK ? -s[e] : s[e];
    x[ia] = p * c[e] - q * t;
    x[ib] = q * c[e] + p * t;
  }
}

// Forward.  Heads of a token in order: queries, keys, and with a cache the values (copied); the
// heads of all tokens one after the other, LPH lanes each (a token to a row of workgroups left lanes
// idle where its heads do not fill them: 8000 tokens of 96 heads of 128, 393 MB, 84 us; so 75 us, 5.2 TB/s).
template <int V, int LPH, bool INTERLEAVED>
__global__ __launch_bounds__(256) void norm_rotate_kernel(NormArgs a, int tokens) {
  constexpr int PIECES = 8 / V;
  const uint32_t heads = a.q_heads + (a.k_out ? 1 : 2) * a.kv_heads;
  const uint32_t row = blockIdx.x * (256 / LPH) + threadIdx.x / LPH, token = row / heads;
  const int sub = threadIdx.x % LPH, h = (int)(row - token * heads);
  const int64_t t = token;
  if (t >= tokens) return;
  const int half = a.rot / 2;
  const bool is_q = h < a.q_heads, is_v = h >= a.q_heads + a.kv_heads;

  // the head is read before its position and slot are known: one wait for memory
  // less (8190 tokens of 32 + 8 + 8 heads, three inputs in turn, 42.8 -> 39.0 us)
  typedef typename Vec<V>::h hv;
  const int kh = is_v ? h - a.q_heads - a.kv_heads : h - a.q_heads;
  const _Float16* src = is_q ? a.q + t * a.q_stride + (int64_t)h * a.D
                             : (is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride) + (int64_t)kh * a.D;
  hv first[PIECES], second[PIECES];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const Piece<V, INTERLEAVED> p(i * LPH + sub, a.D, half, !is_v);
    if (!p.live) continue;
    first[i] = *reinterpret_cast<const hv*>(src + p.o0);
    second[i] = *reinterpret_cast<const hv*>(src + p.o1);
  }
  const int64_t pos = a.rot ? a.positions[t] : 0;
  const bool pos_ok = !a.rot || (pos >= 0 && pos < a.n_positions);
  const int64_t slot = a.k_out ? 0 : a.slots[t];
  if (!is_q && !a.k_out && !(pos_ok && slot >= 0 && slot < a.n_pages * a.page)) return;
  _Float16* dst;
  if (is_q) dst = a.q_out + (t * a.q_heads + h) * a.D;
  else if (a.k_out) dst = a.k_out + (t * a.kv_heads + kh) * a.D;
  else {
    const int64_t page = slot / a.page, in_page = slot - page * a.page;
    dst = (is_v ? a.v_cache : a.k_cache) + ((page * a.kv_heads + kh) * a.page + in_page) * a.D;
  }

  if (is_v) {  // as it is, bit by bit
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const Piece<V, INTERLEAVED> p(i * LPH + sub, a.D, half, false);
      if (!p.live) continue;
      *reinterpret_cast<hv*>(dst + p.o0) = first[i];
      *reinterpret_cast<hv*>(dst + p.o1) = second[i];
    }
    return;
  }
  float x[PIECES][2 * V], sum = 0.f;
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const Piece<V, INTERLEAVED> p(i * LPH + sub, a.D, half, true);
    if (!p.live) continue;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      x[i][e] = (float)first[i][e];
      x[i][V + e] = (float)second[i][e];
    }
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) sum = __builtin_fmaf(x[i][e], x[i][e], sum);
  }
  const float r = rsqrtf(head_sum<LPH>(sum) / (float)a.D + a.eps);
  const _Float16* w = is_q ? a.q_weight : a.k_weight;
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const Piece<V, INTERLEAVED> p(i * LPH + sub, a.D, half, true);
    if (!p.live) continue;
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) x[i][e] *= r;
    if (w) {
      float f[2 * V];
      read<V>(w, p.o0, p.o1, f);
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) x[i][e] *= f[e];
    }
    if (!pos_ok) {
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) x[i][e] = __builtin_nanf("");
    } else if (p.turn) {
      rotate<V, INTERLEAVED, false>(x[i], a.cos, a.sin, pos * half + p.j);
    }
    write<V>(dst, p.o0, p.o1, x[i]);
  }
}

// Workgroups of the gradients of queries, and of keys: each leaves a row of partial sums.  512 up to CHAIN rows
// a lane (a step of 2870 tokens of 16 + 8 heads of 80 took 25.9 us with 1024, of which some walked one row and some
// two, 22.7 with 512; of 4096 tokens of 32 + 8 heads of 128 44.9 and 43.7), beyond as many as keep it at that: no
// value passes more than CHAIN additions in fp32 here and 33 behind them, however many the rows (67 million rows of
// heads of 8 by 512 workgroups are 2048 a lane, whose sum in fp32 was off by 2^-15).
constexpr int GRAD_BLOCKS = 512, CHAIN = 64;

// Gradients: blockIdx.y 0 walks the rows (token, head) of the queries, 1 those of the keys.
template <int V, int LPH, bool INTERLEAVED>
__global__ __launch_bounds__(256) void norm_rotate_grad_kernel(NormGradArgs a) {
  constexpr int PIECES = 8 / V, GROUPS = 256 / LPH;
  __shared__ float sums[4][256];
  const bool is_k = blockIdx.y != 0;
  const int sub = threadIdx.x % LPH, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int heads = is_k ? a.kv_heads : a.q_heads, half = a.rot / 2;
  const _Float16* X = is_k ? a.k : a.q;
  const _Float16* DY = is_k ? a.dk_out : a.dq_out;
  _Float16* DX = is_k ? a.dk : a.dq;
  const int64_t stride = is_k ? a.k_stride : a.q_stride, out_stride = is_k ? a.dk_stride : a.dq_stride;
  const _Float16* w = is_k ? a.k_weight : a.q_weight;
  float* dw = is_k ? a.dk_weight : a.dq_weight;
  const uint32_t rows = (uint32_t)a.T * (uint32_t)heads;  // below 2^31 (checked)

  float acc[PIECES][2 * V], wf[PIECES][2 * V];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const Piece<V, INTERLEAVED> p(i * LPH + sub, a.D, half, true);
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) acc[i][e] = 0.f, wf[i][e] = 1.f;
    if (w && p.live) read<V>(w, p.o0, p.o1, wf[i]);
  }
  for (uint32_t row = blockIdx.x * GROUPS + threadIdx.x / LPH; row < rows; row += gridDim.x * GROUPS) {
    const uint32_t t = row / (uint32_t)heads, h = row - t * (uint32_t)heads;
    const int64_t pos = a.rot ? a.positions[t] : 0;
    const bool pos_ok = !a.rot || (pos >= 0 && pos < a.n_positions);
    const _Float16* src = X + t * stride + (int64_t)h * a.D;
    const _Float16* dsrc = DY + (int64_t)row * a.D;
    _Float16* dst = DX + t * out_stride + (int64_t)h * a.D;
    float x[PIECES][2 * V], g[PIECES][2 * V], xx = 0.f;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const Piece<V, INTERLEAVED> p(i * LPH + sub, a.D, half, true);
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) x[i][e] = g[i][e] = 0.f;
      if (!p.live || !pos_ok) continue;
      read<V>(src, p.o0, p.o1, x[i]);
      read<V>(dsrc, p.o0, p.o1, g[i]);
      if (p.turn) rotate<V, INTERLEAVED, true>(g[i], a.cos, a.sin, pos * half + p.j);
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) xx = __builtin_fmaf(x[i][e], x[i][e], xx);
    }
    const float r = rsqrtf(head_sum<LPH>(xx) / (float)a.D + a.eps);
    float xh = 0.f;
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) {
        x[i][e] *= r;
        acc[i][e] = __builtin_fmaf(x[i][e], g[i][e], acc[i][e]);
        g[i][e] *= wf[i][e];
        xh = __builtin_fmaf(x[i][e], g[i][e], xh);
      }
    const float mean = head_sum<LPH>(xh) / (float)a.D;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const Piece<V, INTERLEAVED> p(i * LPH + sub, a.D, half, true);
      if (!p.live) continue;
      float d[2 * V];
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) d[e] = pos_ok ? r * (g[i][e] - x[i][e] * mean) : 0.f;
      write<V>(dst, p.o0, p.o1, d);
    }
  }
  if (!dw) return;
  // this workgroup's sums, of the lanes with the same places
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const Piece<V, INTERLEAVED> p(i * LPH + sub, a.D, half, true);
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) {
      float s = acc[i][e];
#pragma unroll
      for (int o = LPH; o < 64; o <<= 1) s += __shfl_xor(s, o, 64);
      if (lane < LPH && p.live) sums[wave][e < V ? p.o0 + e : p.o1 + e - V] = s;
    }
  }
  __syncthreads();
  if ((int)threadIdx.x < a.D) {
    const int d = threadIdx.x;
    a.part[((int64_t)(is_k ? gridDim.x : 0) + blockIdx.x) * a.D + d] = sums[0][d] + sums[1][d] + sums[2][d] + sums[3][d];
  }
}

// The workgroups' partial sums added up in order: 16 places of a weight a workgroup (64 bytes of a
// row), 64 rows at a time, the loads of GRAD_BLOCKS rows in flight together, and the sums of these in 64 bits.
__global__ __launch_bounds__(1024) void norm_weight_grad_kernel(NormGradArgs a, int blocks, int q_blocks, int k_blocks) {
  __shared__ float sums[16][16];
  const bool is_k = blockIdx.y != 0;
  float* out = is_k ? a.dk_weight : a.dq_weight;
  if (!out) return;
  const int n = is_k ? k_blocks : q_blocks, col = threadIdx.x % 16, r0 = threadIdx.x / 16, d = blockIdx.x * 16 + col;
  const float* part = a.part + (int64_t)(is_k ? blocks : 0) * a.D + min(d, a.D - 1);
  double total = 0.;
  for (int n0 = 0; n0 < n; n0 += GRAD_BLOCKS) {
    float v[GRAD_BLOCKS / 64];
#pragma unroll
    for (int i = 0; i < GRAD_BLOCKS / 64; ++i) {
      const int r = n0 + r0 + 64 * i;
      v[i] = r < n ? part[(int64_t)r * a.D] : 0.f;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < GRAD_BLOCKS / 64; ++i) s += v[i];
    total += s;
  }
  float s = (float)total;
  s += __shfl_xor(s, 16, 64);
  s += __shfl_xor(s, 32, 64);
  if ((threadIdx.x & 63) < 16) sums[threadIdx.x >> 6][col] = s;
  __syncthreads();
  if (threadIdx.x < 16 && d < a.D) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += sums[i][col];
    out[d] = s;
  }
}

// Calls f with the widest V that divides the pairs of the turned and of the copied part and every
// row stride (`counts` has all of them ored), to which fp16 arrays (`halves`) and angles (`floats`)
// are aligned, and with the lanes of a head.
template <typename F>
void dispatch(int D, bool interleaved, uintptr_t halves, uintptr_t floats, int64_t counts, F f) {
  auto fits = [&](int v) {
    return counts % v == 0 && (halves & (2 * v - 1)) == 0 && (floats & ((v > 4 ? 16 : 4 * v) - 1)) == 0;
  };
  auto lanes = [&](auto v, auto il) {
    if (D <= 64) f(v, std::integral_constant<int, 4>{}, il);
    else if (D <= 128) f(v, std::integral_constant<int, 8>{}, il);
    else f(v, std::integral_constant<int, 16>{}, il);
  };
  auto order = [&](auto v) {
    if (interleaved) lanes(v, std::true_type{});
    else lanes(v, std::false_type{});
  };
  if (fits(8)) order(std::integral_constant<int, 8>{});
  else if (fits(4)) order(std::integral_constant<int, 4>{});
  else if (fits(2)) order(std::integral_constant<int, 2>{});
  else order(std::integral_constant<int, 1>{});
}

template <typename... P>
uintptr_t bits(P... p) {
  return (reinterpret_cast<uintptr_t>(p) | ...);
}

int64_t grad_blocks(int64_t rows, int groups) {
  const int64_t n = (rows + groups - 1) / groups, least = (n + CHAIN - 1) / CHAIN;
  return least > GRAD_BLOCKS ? least : n < GRAD_BLOCKS ? n : GRAD_BLOCKS;
}

}  // namespace

hipError_t launch_norm_rotate(const NormArgs& a, int64_t T, hipStream_t st) {
  const uintptr_t halves = bits(a.q, a.k, a.v, a.q_out, a.k_out, a.k_cache, a.v_cache, a.q_weight, a.k_weight);
  const int64_t counts = (int64_t)(a.rot / 2) | (a.D / 2) | a.D | a.q_stride | a.k_stride | a.v_stride;
  dispatch(a.D, a.interleaved != 0, halves, bits(a.cos, a.sin), counts, [&](auto v, auto lph, auto il) {
    constexpr int GROUPS = 256 / decltype(lph)::value;
    const int heads = a.q_heads + (a.k_out ? 1 : 2) * a.kv_heads;
    const int64_t most = ((int64_t)1 << 31) / ((int64_t)heads * decltype(lph)::value);  // tokens: a launch ends below 2^32 threads
    for (int64_t t0 = 0; t0 < T; t0 += most) {
      NormArgs b = a;
      b.q += t0 * a.q_stride;
      b.k += t0 * a.k_stride;
      if (b.v) b.v += t0 * a.v_stride;
      b.q_out += t0 * a.q_heads * a.D;
      if (b.k_out) b.k_out += t0 * a.kv_heads * a.D;
      if (b.positions) b.positions += t0;
      if (b.slots) b.slots += t0;
      const int64_t n = T - t0 < most ? T - t0 : most;
      const dim3 grid((unsigned)((n * heads + GROUPS - 1) / GROUPS));
      hipLaunchKernelGGL((norm_rotate_kernel<decltype(v)::value, decltype(lph)::value, decltype(il)::value>), grid, dim3(256),
                         0, st, b, (int)n);
    }
  });
  return hipGetLastError();
}

size_t norm_grad_ws_bytes(int64_t T, int32_t q_heads, int32_t kv_heads, int32_t D) {
  const int groups = D <= 64 ? 64 : D <= 128 ? 32 : 16;  // heads of a workgroup, as in dispatch
  const int64_t n = grad_blocks(T * (q_heads > kv_heads ? q_heads : kv_heads), groups);
  return (size_t)2 * (n > GRAD_BLOCKS ? n : GRAD_BLOCKS) * D * sizeof(float);
}

hipError_t launch_norm_rotate_grad(const NormGradArgs& a, hipStream_t st) {
  const uintptr_t halves = bits(a.q, a.k, a.dq_out, a.dk_out, a.dq, a.dk, a.q_weight, a.k_weight);
  const int64_t counts = (int64_t)(a.rot / 2) | (a.D / 2) | a.D | a.q_stride | a.k_stride | a.dq_stride | a.dk_stride;
  int64_t blocks = 0, nq = 0, nk = 0;  // of the launch, and those that have rows of queries and of keys
  dispatch(a.D, a.interleaved != 0, halves, bits(a.cos, a.sin), counts, [&](auto v, auto lph, auto il) {
    constexpr int GROUPS = 256 / decltype(lph)::value;
    const int64_t rows_q = (int64_t)a.T * a.q_heads, rows_k = (int64_t)a.T * a.kv_heads;
    blocks = grad_blocks(rows_q > rows_k ? rows_q : rows_k, GROUPS);
    auto with_rows = [&](int64_t rows) {
      const int64_t n = (rows + GROUPS - 1) / GROUPS;
      return n < blocks ? n : blocks;
    };
    nq = with_rows(rows_q);
    nk = with_rows(rows_k);
    if (a.T > 0) hipLaunchKernelGGL((norm_rotate_grad_kernel<decltype(v)::value, decltype(lph)::value, decltype(il)::value>),
                       dim3((unsigned)blocks, 2), dim3(256), 0, st, a);
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!a.dq_weight && !a.dk_weight)) return e;
  hipLaunchKernelGGL(norm_weight_grad_kernel, dim3((unsigned)((a.D + 15) / 16), 2), dim3(1024), 0, st, a, (int)blocks, (int)nq, (int)nk);
  return hipGetLastError();
}

}  // namespace qg
