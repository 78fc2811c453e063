// Rotary positions on new queries and keys, and their keys and values written into the
// paged cache.
//
// Every value is read once and written once: 2 T (q_heads + 2 kv_heads) head_dim halves,
// bound by HBM for long prompts and by the launch for a decode batch.  One thread takes V
// pairs of one head of one token (two V-value vectors: the halves j and j + rot / 2 of V
// pairs, or 2 V consecutive values of the interleaved order or of the part that is only
// copied), so no thread needs another's values and loads and stores are as wide as V.
// blockIdx.x is the token, which makes its position, slot and row addresses scalar; the
// threads of a workgroup walk the token's heads in order, so consecutive threads touch
// consecutive memory on both sides.  The angles of a token are read by all its heads from
// cache.  Rotation in fp32, one rounding to fp16.  8190 tokens of 32 + 32 + 32 heads of 128
// (405 MB): 78 us, 5.2 TB/s (a 2 GiB copy reaches 4.9); 48 tokens: 3.0 us, the launch.
#include "qgemm_internal.hpp"

namespace qg {
namespace {

template <int V>
struct Vec {
  typedef _Float16 h __attribute__((ext_vector_type(V)));
  typedef float f __attribute__((ext_vector_type(V)));
};

template <int V, bool INTERLEAVED>
__global__ __launch_bounds__(256) void kv_append_kernel(AppendArgs a) {
  typedef typename Vec<V>::h hv;
  typedef typename Vec<V>::f fv;
  const int64_t t = blockIdx.x;
  const int per_head = a.D / 2 / V;  // work items of a head: V pairs each
  const int item = blockIdx.y * 256 + threadIdx.x;
  if (item >= (a.q_heads + 2 * a.kv_heads) * per_head) return;
  const int h = item / per_head, j = (item - h * per_head) * V;  // head of the token, first pair
  const int half = a.rot / 2;
  const bool is_q = h < a.q_heads, is_v = h >= a.q_heads + a.kv_heads;

  const int64_t pos = a.rot ? a.positions[t] : 0;
  const bool pos_ok = !a.rot || (pos >= 0 && pos < a.n_positions);
  const int64_t slot = a.slots[t];
  const bool store = is_q || (pos_ok && slot >= 0 && slot < a.n_pages * a.page);
  if (!store) return;

  const bool turn = !is_v && j < half;
  // places of the two vectors within the head
  int o0, o1;
  if (is_v) {
    o0 = 2 * j;
    o1 = o0 + V;
  } else if (turn) {
    o0 = INTERLEAVED ? 2 * j : j;
    o1 = INTERLEAVED ? o0 + V : j + half;
  } else {
    o0 = 2 * j;  // rot + 2 (j - half)
    o1 = o0 + V;
  }
  const _Float16* src;
  _Float16* dst;
  if (is_q) {
    src = a.q + t * a.q_stride + (int64_t)h * a.D;
    dst = a.q_out + (t * a.q_heads + h) * a.D;
  } else {
    const int kh = is_v ? h - a.q_heads - a.kv_heads : h - a.q_heads;
    src = (is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride) + (int64_t)kh * a.D;
    const int64_t page = slot / a.page, in_page = slot - page * a.page;
    dst = (is_v ? a.v_cache : a.k_cache) + ((page * a.kv_heads + kh) * a.page + in_page) * a.D;
  }
  hv x = *reinterpret_cast<const hv*>(src + o0), y = *reinterpret_cast<const hv*>(src + o1);
  if (turn && pos_ok) {
    const fv c = *reinterpret_cast<const fv*>(a.cos + pos * half + j);
    const fv s = *reinterpret_cast<const fv*>(a.sin + pos * half + j);
    float val[2 * V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      val[e] = (float)x[e];
      val[V + e] = (float)y[e];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      // places of pair e among the 2 V values
      const int ia = INTERLEAVED ? 2 * e : e, ib = INTERLEAVED ? 2 * e + 1 : V + e;
      const float p = val[ia], r = val[ib];
      val[ia] = p * c[e] - r * s[e];
      val[ib] = r * c[e] + p * s[e];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      x[e] = (_Float16)val[e];
      y[e] = (_Float16)val[V + e];
    }
  } else if (!pos_ok) {
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = y[e] = __builtin_bit_cast(_Float16, (uint16_t)0x7E00);
  }
  *reinterpret_cast<hv*>(dst + o0) = x;
  *reinterpret_cast<hv*>(dst + o1) = y;
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs& a, int64_t T, hipStream_t st) {
  // The widest vector that divides the pairs of the turned and of the copied part and
  // every row stride, and to which every array is aligned (fp32 angles: twice as wide).
  const uintptr_t halves = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) |
                           reinterpret_cast<uintptr_t>(a.v) | reinterpret_cast<uintptr_t>(a.q_out) |
                           reinterpret_cast<uintptr_t>(a.k_cache) | reinterpret_cast<uintptr_t>(a.v_cache);
  const uintptr_t floats = reinterpret_cast<uintptr_t>(a.cos) | reinterpret_cast<uintptr_t>(a.sin);
  const int64_t counts = (int64_t)(a.rot / 2) | (a.D / 2) | a.D | a.q_stride | a.k_stride | a.v_stride;
  auto fits = [&](int v) {
    return counts % v == 0 && (halves & (2 * v - 1)) == 0 && (floats & ((v > 4 ? 16 : 4 * v) - 1)) == 0;
  };
  // a launch holds fewer than 2^32 threads along its first dimension, the tokens'
  constexpr int64_t MOST = (int64_t)1 << 23;
  auto go = [&](auto kernel, int v) {
    const int items = (a.q_heads + 2 * a.kv_heads) * (a.D / 2 / v);
    for (int64_t t0 = 0; t0 < T; t0 += MOST) {
      AppendArgs b = a;
      b.q += t0 * a.q_stride;
      b.k += t0 * a.k_stride;
      b.v += t0 * a.v_stride;
      b.q_out += t0 * a.q_heads * a.D;
      if (b.positions) b.positions += t0;
      b.slots += t0;
      const unsigned n = (unsigned)(T - t0 < MOST ? T - t0 : MOST);
      hipLaunchKernelGGL(kernel, dim3(n, (unsigned)((items + 255) / 256)), dim3(256), 0, st, b);
    }
  };
  const bool il = a.interleaved != 0;
  if (fits(8)) il ? go(kv_append_kernel<8, true>, 8) : go(kv_append_kernel<8, false>, 8);
  else if (fits(4)) il ? go(kv_append_kernel<4, true>, 4) : go(kv_append_kernel<4, false>, 4);
  else if (fits(2)) il ? go(kv_append_kernel<2, true>, 2) : go(kv_append_kernel<2, false>, 2);
  else il ? go(kv_append_kernel<1, true>, 1) : go(kv_append_kernel<1, false>, 1);
  return hipGetLastError();
}

}  // namespace qg
