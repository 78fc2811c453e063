// Attention over the paged cache: how a call's work is split, and the pass that joins the
// parts (the tiles: attention_kernel.hpp).
#include "attention_kernel.hpp"

namespace qg {
namespace {

// Joins the partial results of every row, one wave a row: lane s weighs slot s, then the
// lanes own places of the output and sum the slots' in order, eight loads in flight (one
// after the other, each behind its slot's maximum, 17 slots took 12.9 us for 2048 rows).
constexpr int JOIN_SLOTS = 64;
__global__ __launch_bounds__(256) void attend_join_kernel(AttnArgs a, AttnSplit sp) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int start, n;
  queries_of(a, blockIdx.y, start, n);
  const int64_t x = (int64_t)blockIdx.x * 4 + wave;  // row of the sequence: query * q_heads + head
  if (x >= (int64_t)n * a.q_heads) return;
  const int64_t th = (int64_t)start * a.q_heads + x, step = (int64_t)a.T * a.q_heads;
  float2 ml = make_float2(-INFINITY, 0.f);
  if (lane < sp.slots) ml = sp.part_ml[lane * step + th];
  // a slot without keys weighs nothing; NaN sums stay (they have a maximum of -inf at least)
  float top = ml.x;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
  const bool live = !(ml.x == -INFINITY && ml.y == 0.f);
  const float w = !live ? 0.f : ml.x == top ? 1.f : exp2_f(ml.x - top);
  float sum = live ? w * ml.y : 0.f;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
  const bool none = top == -INFINITY && sum == 0.f;
  // lanes past D read its last values again: each lane holds a slot's weight, so all stay in
  const int d0 = min(lane * 4, a.D - 4);
  const float* po = sp.part_o + th * a.D + d0;
  float4v v = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < sp.slots; s0 += 8) {
    float4v p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int s = min(s0 + i, sp.slots - 1);
      p[i] = *reinterpret_cast<const float4v*>(po + s * step * a.D);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float ws = __shfl(w, s0 + i, 64);  // 0 past the last slot
      if (ws != 0.f) v += ws * p[i];
    }
  }
  if (lane * 4 < a.D) {
    half4v h;
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = (_Float16)(none ? 0.f : v[i] / sum);
    *reinterpret_cast<half4v*>(a.out + th * a.D + d0) = h;
  }
  if (a.lse && lane == 0) a.lse[th] = none ? -INFINITY : (top + __log2f(sum)) * 0.6931471805599453f;
}

int64_t div_up(int64_t x, int64_t y) { return (x + y - 1) / y; }

// keys per part and parts, so that about `want` items run (parts of at least min_chunk keys)
void split_keys(int64_t keys, int64_t items, int64_t want, int64_t min_chunk, int* chunk, int* splits) {
  int64_t s = div_up(want, items < 1 ? 1 : items);
  const int64_t most = div_up(keys < 1 ? 1 : keys, min_chunk);
  if (s > most) s = most;
  if (s > JOIN_SLOTS / 2) s = JOIN_SLOTS / 2;  // prefix and own parts together fit a wave
  if (s < 1) s = 1;
  *chunk = (int)(div_up(div_up(keys < 1 ? 1 : keys, s), 64) * 64);
  *splits = (int)div_up(keys < 1 ? 1 : keys, *chunk);
}

// The same for a window, whose few keys make a join dear (300 queries with a window of 100, 32 / 8
// heads of 128, three sequences: 11 us whole and 28 us in two parts): the number of parts whose sum of
// three terms is least, each as measured, in us.  A block of 64 keys (KEYS: 128, by four waves) takes a CU
// 0.65, 1.0 and 1.7 (128 rows: 2.4; KEYS: a quarter more) with heads of 64, 128 and 256; an item's beginning and end as
// long as about two and a half of them; items run a CU each, then the next.  A join is 4 and the partial
// results at 4.85 TB/s both ways.  Over 120 batches of 20 to 1000 queries and windows of 100 to 6000 this
// takes 0.78 of the time that as many parts as make 512 items take (geometric mean; 0.37 to 1.06), over 114
// of one or two queries 0.96 (0.70 to 1.04).
// With heads past 128 the tiles of 64 rows, which one workgroup is soonest done with, are weighed against
// those of 128 (8 / 2 heads of 256, window 100: 300 queries 11 and 17 us, 3000 queries 24 and 20).
void split_window(const AttnShape& s, AttnSplit* p) {
  const int64_t G = s.q_heads / s.kv_heads, max_rows = s.max_q * G;
  const double part = 2.0 * s.T * s.q_heads * (s.D + 2) * sizeof(float) / 4.85e6;
  double best = INFINITY;
  auto weigh = [&](int kind, double block) {
    const int64_t rows = tile_rows(kind), step = kind == TILE_KEYS ? 128 : 64;
    // the window of a tile's last query, what its earlier ones see before that, and the first keys
    const int64_t queries = (rows - 1) / G + 2, all = s.max_len + s.prefix_len;
    const int64_t list = s.window + (queries < s.max_q ? queries : s.max_q) + s.sinks;
    const int64_t keys = all < 1 ? 1 : list < all ? list : all;
    // (the tiles that have rows, as many as there may be)
    const int64_t of_rows = s.B + s.T * G / rows, most = s.B * div_up(max_rows, rows);
    const int64_t items = (of_rows < most ? of_rows : most) * s.kv_heads;
    for (int n = 1; n <= JOIN_SLOTS / 2; ++n) {
      const int64_t chunk = div_up(div_up(keys, n), step) * step, parts = div_up(keys, chunk);
      if (parts < n) {  // (these parts have been looked at)
        if (chunk == step) break;
        continue;
      }
      const double us = div_up(items * parts, 256) * (chunk / step + 2.5) * block + (parts > 1 ? 4 + parts * part : 0);
      if (us >= best) continue;
      best = us;
      p->kind_s = kind;
      p->s_tiles = (int)div_up(max_rows, rows);
      p->s_chunk = (int)chunk;
      p->s_splits = (int)parts;
    }
  };
  const double width = s.D <= 64 ? 0.65 : s.D <= 128 ? 1.0 : 1.7;
  if (max_rows <= 16) weigh(TILE_KEYS, 1.25 * width);
  else if (max_rows <= 64) weigh(TILE_ROWS64, width);
  else if (s.D <= 128) weigh(TILE_ROWS128, width);
  else weigh(TILE_ROWS64, width), weigh(TILE_ROWS128, 2.4);
}

// (head dimensions past 128 keep 64 rows: with 128 the accumulators of a wave spilled)
int kind_for(int64_t rows, int D) {
  return rows <= 16 ? TILE_KEYS : rows <= 64 || D > 128 ? TILE_ROWS64 : TILE_ROWS128;
}

AttnSplit choose_split(const AttnShape& s) {
  AttnSplit p = {};
  p.kind_p = TILE_NONE;
  if (s.window) {  // (each sequence reads what it sees of the prefix by itself)
    split_window(s, &p);
    p.s_items = (int)(s.B * s.kv_heads * p.s_tiles * p.s_splits);
    p.slots = p.s_splits > 1 ? p.s_splits : 0;
    return p;
  }
  const int64_t G = s.q_heads / s.kv_heads, rows = s.max_q * G;
  int64_t keys = s.max_len + s.prefix_len;  // of one item
  p.kind_s = kind_for(rows, s.D);
  p.shared = s.prefix_len > 0 && s.B > 1 && rows <= 64;
  p.s_tiles = (int)div_up(rows, tile_rows(p.kind_s));
  const int64_t s_base = s.B * s.kv_heads * p.s_tiles;
  if (p.shared) {
    p.kind_p = kind_for(s.T * G, s.D);
    p.p_tiles = (int)div_up(s.T * G, tile_rows(p.kind_p));
    split_keys(s.prefix_len, (int64_t)p.p_tiles * s.kv_heads, 256, 128, &p.p_chunk, &p.p_splits);
    p.p_items = p.p_tiles * p.p_splits * s.kv_heads;
    keys = s.max_len;
  }
  split_keys(keys, s_base, 512, 128, &p.s_chunk, &p.s_splits);
  p.s_items = (int)(s_base * p.s_splits);
  p.slots = (p.shared ? p.p_splits : 0) + p.s_splits;
  if (p.slots == 1) p.slots = 0;
  return p;
}

size_t part_o_bytes(const AttnShape& s, const AttnSplit& p) {
  return (size_t)p.slots * s.T * s.q_heads * s.D * sizeof(float);
}

template <int DP>
hipError_t launch_dim(const AttnArgs& a, const AttnSplit& p, hipStream_t st) {
  if (p.kind_p == TILE_NONE) {
    if (p.kind_s == TILE_KEYS) return launch_kinds<DP, TILE_NONE, TILE_KEYS>(a, p, st);
    if (p.kind_s == TILE_ROWS64) return launch_kinds<DP, TILE_NONE, TILE_ROWS64>(a, p, st);
    if constexpr (DP <= 128) return launch_kinds<DP, TILE_NONE, TILE_ROWS128>(a, p, st);
  } else if (p.kind_s == TILE_KEYS) {
    if (p.kind_p == TILE_KEYS) return launch_kinds<DP, TILE_KEYS, TILE_KEYS>(a, p, st);
    if (p.kind_p == TILE_ROWS64) return launch_kinds<DP, TILE_ROWS64, TILE_KEYS>(a, p, st);
    if constexpr (DP <= 128) return launch_kinds<DP, TILE_ROWS128, TILE_KEYS>(a, p, st);
  } else {  // more than 16 rows a sequence, so more than 16 in all
    if (p.kind_p == TILE_ROWS64) return launch_kinds<DP, TILE_ROWS64, TILE_ROWS64>(a, p, st);
    if constexpr (DP <= 128) return launch_kinds<DP, TILE_ROWS128, TILE_ROWS64>(a, p, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace

bool attention_grid_fits(const AttnShape& s) {
  const int64_t G = s.q_heads / s.kv_heads, tiles = div_up(s.max_q * G, 16), all = div_up(s.T * G, 16);
  const int64_t most = (s.B * tiles + all) * s.kv_heads * 64;  // items, with every part that there can be
  if (most >= INT32_MAX || s.T * G >= INT32_MAX / 2 || s.max_q * s.q_heads >= INT32_MAX) return false;
  // a launch holds fewer than 2^32 threads along a dimension, 256 a workgroup here
  constexpr int64_t MOST = (int64_t)1 << 24;
  if (most < MOST) return true;
  const AttnSplit p = choose_split(s);
  return (int64_t)p.p_items + p.s_items < MOST && (!p.slots || div_up(s.max_q * s.q_heads, 4) < MOST);
}

size_t attention_ws_bytes(const AttnShape& s) {
  const AttnSplit p = choose_split(s);
  if (!p.slots) return 0;
  return part_o_bytes(s, p) + (size_t)p.slots * s.T * s.q_heads * sizeof(float2);
}

hipError_t launch_attention(const WindowArgs& a, const AttnShape& s, void* ws, hipStream_t st) {
  AttnSplit p = choose_split(s);
  if (p.slots) {
    p.part_o = static_cast<float*>(ws);
    p.part_ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + part_o_bytes(s, p));
  }
  const AttnArgs& b = a;
  hipError_t e = s.window ? launch_window_tiles(a, p, st)
                 : s.D <= 64 ? launch_dim<64>(b, p, st) : s.D <= 128 ? launch_dim<128>(b, p, st) : launch_dim<256>(b, p, st);
  if (e != hipSuccess || !p.slots) return e;
  hipLaunchKernelGGL(attend_join_kernel, dim3((unsigned)div_up(s.max_q * s.q_heads, 4), (unsigned)s.B), dim3(256), 0, st,
                     b, p);
  return hipGetLastError();
}

}  // namespace qg
