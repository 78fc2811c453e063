// Causal attention of a ragged batch over the paged cache, behind one shared prefix.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(s_j - m),  s_j = scale q . k_j,  m = max s_j
// in one pass over the keys: when a block of keys raises the running maximum from m to m',
// the sums so far shrink by exp(m - m').
//
// One wave per query and head.  A lane scores one key of a block of 64, the block's
// probabilities meet in the wave, and then a lane owns head_dim / 64 places of the output.
#include "qgemm_internal.hpp"

namespace qg {
namespace {

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// offset of token t of sequence b's keys (prefix tokens first) in the cache arrays
__device__ __forceinline__ int64_t token_offset(const AttnArgs& a, int b, int64_t t, int head) {
  int64_t own = t - a.prefix_len;
  const int32_t* table = own < 0 ? a.prefix_table : a.tables + (int64_t)b * a.table_width;
  if (own < 0) own = t;
  int page = table[own >> a.page_shift];
  if ((uint32_t)page >= (uint32_t)a.n_pages) page = 0;
  const int in_page = (int)(own & ((1 << a.page_shift) - 1));
  return (((int64_t)page * a.kv_heads + head) << a.page_shift) * a.D + (int64_t)in_page * a.D;
}

__global__ __launch_bounds__(64) void attend_simple_kernel(AttnArgs a) {
  const int lane = threadIdx.x, b = blockIdx.z, i = blockIdx.y, h = blockIdx.x;
  const int start = a.q_starts[b], n = min(a.q_starts[b + 1] - start, a.max_q);
  if (i >= n) return;
  const int64_t row = start + i;
  if (row < 0 || row >= a.T) return;
  const int64_t held = min((int64_t)min(a.kv_lens[b], a.max_len), a.table_width << a.page_shift);
  const int64_t seen = max((int64_t)0, held - n + i + 1);
  const int64_t keys = a.prefix_len + seen;
  const int kvh = h / (a.q_heads / a.kv_heads);
  const _Float16* q = a.q + row * a.q_stride + (int64_t)h * a.D;
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t t0 = 0; t0 < keys; t0 += 64) {
    const int64_t t = t0 + lane;
    float s = -INFINITY;
    int64_t at = 0;
    if (t < keys) {
      at = token_offset(a, b, t, kvh);
      s = 0.f;
      for (int d = 0; d < a.D; ++d) s += (float)q[d] * (float)a.k[at + d];
      s *= a.scale;
    }
    const float m2 = fmaxf(m, wave_max(s));
    const float base = m2 == -INFINITY ? 0.f : m2;
    const float keep = __expf(m - base), p = t < keys ? __expf(s - base) : 0.f;
    l = l * keep + wave_sum(p);
    m = m2;
    for (int e = 0; e < 4; ++e) o[e] *= keep;
    const int cnt = (int)min((int64_t)64, keys - t0);
    for (int j = 0; j < cnt; ++j) {
      const float pj = __shfl(p, j, 64);
      const int64_t vj = __shfl(at, j, 64);
      for (int e = 0; e < 4; ++e)
        if (e * 64 + lane < a.D) o[e] += pj * (float)a.v[vj + e * 64 + lane];
    }
  }
  _Float16* out = a.out + (row * a.q_heads + h) * a.D;
  for (int e = 0; e < 4; ++e)
    if (e * 64 + lane < a.D) out[e * 64 + lane] = (_Float16)(keys > 0 ? o[e] / l : 0.f);
  if (a.lse && lane == 0) a.lse[row * a.q_heads + h] = keys > 0 ? m + __logf(l) : -INFINITY;
}

}  // namespace

size_t attention_ws_bytes(const AttnShape&) { return 0; }

hipError_t launch_attention(const AttnArgs& a, const AttnShape& s, void*, hipStream_t st) {
  hipLaunchKernelGGL(attend_simple_kernel, dim3(a.q_heads, (unsigned)a.max_q, (unsigned)s.B), dim3(64), 0, st, a);
  return hipGetLastError();
}

}  // namespace qg
