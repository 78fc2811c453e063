// Causal attention of a ragged batch over the paged cache, behind one shared prefix.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(s_j - m),  s_j = scale q . k_j,  m = max s_j
// in one pass over the keys: when a block of keys raises the running maximum, the sums so
// far shrink by exp(old - new).  The results of parts of the keys join the same way.
//
// Packed rows.  All q_heads / kv_heads = G query heads of a key / value head share its
// keys, so a row of a tile is a (query token, head of the group) pair: row r is token
// r / G, head r % G.  A tile's rows read every key once.
//
// Work items (one workgroup of four waves each):
//   prefix item    a tile of the rows of ALL sequences against a chunk of the prefix, which
//                  every query sees whole: no mask, and the prefix is read once per tile of
//                  up to 128 rows instead of once per sequence;
//   sequence item  a tile of one sequence's rows against a chunk of its own tokens, or of
//                  prefix and own tokens one after the other where the sequence's rows fill
//                  tiles by themselves (sharing then saves nothing).
// Both kinds run in one launch; items whose keys are split leave (m, l, o) in fp32 in the
// workspace, which a second pass joins in slot order.
//
// Two tile shapes.  KEYS: few rows (up to 16): the four waves take blocks of 32 keys in
// turn, each with LDS of its own and no barrier, and meet in LDS at the end; bound by HBM.
// ROWS: 64 or 128 rows, each wave its own 16 or 32, all from one block of 64 keys in LDS;
// bound by the matrix cores and the exponentials.
//
// The products.  S^T = K Q^T (keys x rows) and O^T = V^T P^T on 16x16x32 MFMAs: the lane
// that holds a score column (row l % 16, keys 4 (l / 16) + i) holds exactly its operand of
// the second product, since the order of the keys within a product is free as long as P
// and V agree, so probabilities never leave their lane.  V^T comes from LDS by transposed
// reads (ds_read_b64_tr_b16: lane i of 16 gets column i of a 4 x 16 block).  Keys and
// values go from memory to LDS directly (global_load_lds_dwordx4), and so do the page
// numbers of the block after next, so that no wait for a page number ever waits for the
// data loads behind it.
//
// Measured (heads of 128): KEYS, 64 sequences of 512 own tokens, 8 key / value heads 23 us
// (5.7 TB/s of keys and values), 16 sequences of 8000 tokens 111 us (4.7 TB/s); one sequence of
// 777 tokens, 32 heads 6.1 us and 4 us to join its 7 parts.  ROWS, 4096 tokens of 32 / 8 heads
// 178-189 us (727-772 TFLOP/s), 2048 queries behind 16384 keys 677 us (863 TFLOP/s): a block of
// 64 keys takes 128 rows 64 MFMAs (1024 cycles) and about 210 vector instructions (1220
// cycles, 512 of them exponentials) a wave, two waves share a SIMD, and the two pipes
// overlap only in part.
//
// Precision: scores, maxima and sums in fp32, exponentials as 2^(s c - m) with c = scale
// log2 e; probabilities round to fp16 as operands (the matrix cores' full rate; error against 64
// bits 2.6e-4 to 2.9e-4, 2.1e-4 of it the result's own rounding).  The maximum used may lag the true one
// by up to 8 (probabilities up to 2^8, far inside fp16), which spares most of the
// rescaling.
//
// Keys a row does not see: their scores become -inf by selection, so what K holds there
// never matters; where a block holds such keys, V's infinities and NaN are added to the
// rows that do see them and taken out of the product (0 times infinity would be NaN).
//
// Windows (WindowArgs; instances of their own): of the c keys up to its own a query sees the
// last `window` and the first `sinks`.  A tile then walks a list of keys in an order of its
// own, since a softmax does not ask for one: first those from the latest window's beginning
// on, which all rows see up to their own ends, then those that only the earlier rows still
// see, then the first ones.  So the whole blocks come first, as without a window, and the
// masked ones are few and at the end: 2 of 17 blocks of a prompt behind a window of 1024.
#pragma once

#include "dl_common.hpp"

namespace qg {

enum TileKind : int { TILE_NONE = -1, TILE_KEYS = 0, TILE_ROWS64 = 1, TILE_ROWS128 = 2 };
constexpr int tile_rows(int kind) { return kind == TILE_KEYS ? 16 : kind == TILE_ROWS64 ? 64 : 128; }

// how the host split the work of a call
struct AttnSplit {
  int shared;                      // the prefix has items of its own
  int kind_p, kind_s;
  int p_tiles, p_splits, p_chunk;  // row tiles, parts of the keys, keys per part
  int s_tiles, s_splits, s_chunk;
  int p_items, s_items;
  int slots;                       // partial results per row (0: results go out directly)
  float* part_o;                   // [slot][T][q_heads][D]
  float2* part_ml;                 // [slot][T][q_heads]: running maximum (log2) and sum
};

namespace {
using namespace dl;

typedef short short4v __attribute__((ext_vector_type(4)));
typedef _Float16 half4v __attribute__((ext_vector_type(4)));

constexpr float RAISE = 8.f;  // log2 of how far the maximum used may lag

__device__ __forceinline__ float exp2_f(float x) { return __builtin_amdgcn_exp2f(x); }

// over the four 16-lane rows of a wave (the lanes of one score column)
template <typename F>
__device__ __forceinline__ float across_rows(float v, F f) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = f(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return f(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// 4-byte direct global -> LDS load (lane l's value lands at lds_base + 4 l)
__device__ __forceinline__ void dma4(const void* g, uint32_t lds_base) {
  asm volatile("global_load_lds_dword %0, off" : : "v"(g), "{m0}"(lds_base) : "memory");
}
// 16-byte form (lane l's bytes land at lds_base + 16 l)
__device__ __forceinline__ void dma16v(const void* g, uint32_t lds_base) {
  asm volatile("global_load_lds_dwordx4 %0, off" : : "v"(g), "{m0}"(lds_base) : "memory");
}
// every LDS read of this wave has returned (its buffer may be loaded over)
__device__ __forceinline__ void reads_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
// all but the newest N loads have landed, and no LDS read moves above
template <int N>
__device__ __forceinline__ void landed() {
  wait_vmcnt<N>();
  asm volatile("" ::: "memory");
}

// query heads of a key / value head, and the query of an item's row; with a window without a division
// (a tile of a small one takes about 10 us, of which those at its start were 1)
__device__ __forceinline__ int heads_per_kv(const AttnArgs& a) { return a.q_heads / a.kv_heads; }
__device__ __forceinline__ int heads_per_kv(const WindowArgs& a) { return a.per_head; }
__device__ __forceinline__ int query_of(const AttnArgs&, int row, int per_head) { return row / per_head; }
__device__ __forceinline__ int query_of(const WindowArgs& a, int row, int) { return a.by_per_head(row); }

// Geometry of a tile kind for head dimensions up to DP.
template <int DP, int KIND>
struct TileGeo {
  static constexpr bool KEYS = KIND == TILE_KEYS;
  static constexpr int NT = KIND == TILE_ROWS128 ? 2 : 1;  // 16-row blocks per wave
  static constexpr int BM = tile_rows(KIND);
  static constexpr int KT = KEYS ? 32 : 64;                // keys per block
  static constexpr int ROWB = DP * 2, SL = ROWB / 16;      // bytes and 16-byte slots of a key
  static constexpr int RPI = 64 / SL;                      // keys per 1 KiB load
  static constexpr int BLOCK = KT * ROWB;                  // bytes of a block of keys (or values)
  static constexpr int LOADS = BLOCK / 1024 / (KEYS ? 1 : 4);  // per wave
  // KEYS: each wave one block of keys and one of values; ROWS: two of each, shared
  static constexpr int PAGES = 2 * 256;                    // page numbers of two blocks, per wave
  static constexpr int BUF = KEYS ? 4 * 2 * BLOCK : 2 * 2 * BLOCK;
  static constexpr int RED = KEYS ? 4 * 16 * (DP + 4) * 4 + 4 * 16 * 8 : 0;  // the waves' results at the end
  static constexpr int LDS = (BUF > RED ? BUF : RED) + 4 * PAGES;
};

// Position of 16-byte slot c of key r in its LDS row: c XOR f(r), f linear in the bits of
// r.  The LDS serves the 64 lanes of a read in groups of 16, 32 or all, each of which
// should touch every 16-byte slot of 256, 512 or 1024 bytes once.  A fragment read of K
// takes 16 keys (lane % 16) at 4 neighbouring slots (lane / 16), a transposed read of V 16
// keys at 2 neighbouring slots, 8 keys by half a wave; f is chosen so that both are free of
// conflicts (checked for all keys and slots on the host; with f = 4 (r / 4), which spreads
// the keys over 1024 bytes only, conflicts were 74 % of the LDS cycles of a prefill).
template <int SL>
__device__ __forceinline__ int slot_of(int r, int c) {
  if constexpr (SL == 8) return c ^ (r & 6) ^ (((r >> 3) & 1) * 7);
  const int f = (r ^ ((r & 1) << 3)) & 15;
  if constexpr (SL == 16) return c ^ f;
  return c ^ f ^ ((((r >> 3) ^ (r >> 1)) & 1) << 4);
}

// what a work item covers
struct Item {
  int kvh, row0, rows;   // key / value head; first row of the tile, rows in all
  int tok0, last_tok;    // query token of row 0; last query token of the item's rows
  int key0, key1;        // keys of the part
  int pre;               // keys [0, pre) are the prefix's
  int lim0;              // row r sees keys below pre_lim + max(0, lim0 + r / G) and key1, ...
  int pre_lim;           // ... with lim0 = INT_MIN / 2 for rows that see pre_lim keys
  int slot;
  const int32_t* own;    // pages of the keys from pre on
  // Of a window: key0 and key1 count in the tile's list of keys, which holds n_late keys from
  // late on, n_early from early on (those before late that earlier rows see), and then the
  // first ones, up to list keys; held is where the sequence's keys end.
  int late, n_late, early, n_early, list, held;
};

// keys up to the place of query i of an item's tile, the prefix's among them
__device__ __forceinline__ int end_at(const Item& it, int i) {
  return it.pre_lim + min(INT32_MAX - it.pre_lim, max(0, it.lim0 + i));
}

// the key at place x of an item's list
__device__ __forceinline__ int key_at(const Item& it, int x) {
  const int before = it.n_late + it.n_early;
  return x + (x < it.n_late ? it.late : x < before ? it.early - it.n_late : -before);
}

// places of an item's list that a row sees: those below late, n_early of them from early on,
// and n_first from the first keys' place on
struct Seen {
  int late, early, first;
  uint32_t n_early, n_first;
  // (written without branches: the row differs from lane to lane)
  __device__ __forceinline__ bool operator()(int x) const {
    return (x < late) | ((uint32_t)(x - early) < n_early) | ((uint32_t)(x - first) < n_first);
  }
  // the same of the 64 places from x on, a bit each
  __device__ __forceinline__ uint64_t from(int x) const {
    auto below = [&](int to) {
      const int n = min(max(to - x, 0), 64);
      return n < 64 ? ((uint64_t)1 << n) - 1 : ~(uint64_t)0;
    };
    return below(late) | (below(early + (int)n_early) & ~below(early)) | (below(first + (int)n_first) & ~below(first));
  }
};
// score s where bit `at` of the places seen is set, else -inf: two instructions, where the three
// intervals took ten for each score
__device__ __forceinline__ float where_seen(uint64_t bits, int at, float s) {
  const uint32_t keep = (uint32_t)__builtin_amdgcn_sbfe((int)(uint32_t)(bits >> (at & 32)), at & 31, 1);
  return __uint_as_float((__float_as_uint(s) & keep) | (0xFF800000u & ~keep));
}
// ... of a row that ends at key `end`, below place `stop`
__device__ __forceinline__ Seen seen_by(const Item& it, int end, int window, int stop) {
  auto length = [](int from, int to) { return (uint32_t)max(to - from, 0); };
  Seen s;
  s.late = min(stop, min(max(min(end, it.held) - it.late, 0), it.n_late));
  s.early = it.n_late + max(end - window - it.early, 0);
  s.n_early = length(s.early, min(stop, it.n_late + min(max(end - it.early, 0), it.n_early)));
  s.first = it.n_late + it.n_early;
  s.n_first = length(s.first, min(stop, s.first + min(end, it.list - s.first)));
  return s;
}

// what keys hold past D: zeros, which add nothing to a score whatever the key's own values are
// (another place of the key would: zero times its infinity is NaN)
__device__ const uint4 PAST_D = {0, 0, 0, 0};

// FULL: D is DP; else D is less, and the places past it are PAST_D in keys, the value's first ones
// in values (whose products there go nowhere); an instance of its own, since branches on D cost the
// full tiles 2 to 8 %
template <int DP, int KIND, bool FULL, typename Args>
__device__ __forceinline__ void attend_tile(const Args& a, const AttnSplit& sp, const Item& it, uint8_t* lds) {
  using T = TileGeo<DP, KIND>;
  constexpr bool KEYS = T::KEYS, WIN = std::is_same_v<Args, WindowArgs>;
  constexpr int NT = T::NT, KT = T::KT, SL = T::SL, RPI = T::RPI, LOADS = T::LOADS;
  constexpr int NSUB = KT / 16, NK = KT / 32, ND = DP / 16, NQ = DP / 32;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, l16 = lane & 15;
  const int G = heads_per_kv(a), D = a.D;

  // ---- rows of this wave, and the keys that they see (the smaller of the two bounds before
  // pre_lim is added: the lengths that a call holds may pass the ones it states)
  const int wrow0 = it.row0 + (KEYS ? 0 : wave * NT * 16);
  const int cap = it.key1 - it.pre_lim;
  // keys up to row r's own, the prefix's among them
  auto end_of = [&](int r) { return end_at(it, query_of(a, min(r, it.rows - 1), G)); };
  // ... and in the order of the item: the keys below this are seen, and (without a window) no others
  auto limit_of = [&](int r) {
    if constexpr (WIN) return min(it.key1, max(0, min(end_of(r), it.held) - it.late));
    else return it.pre_lim + min(cap, max(0, it.lim0 + min(r, it.rows - 1) / G));
  };
  int lim[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) lim[nt] = limit_of(wrow0 + nt * 16 + l16);
  // over the tile's last row (the limits grow with the row), this wave's first and last
  const int kend = __builtin_amdgcn_readfirstlane(WIN ? it.key1 : limit_of(it.row0 + T::BM - 1));
  const int wave_lo = __builtin_amdgcn_readfirstlane(limit_of(wrow0));
  const int wave_hi = __builtin_amdgcn_readfirstlane(wrow0 < it.rows ? limit_of(wrow0 + NT * 16 - 1) : 0);

  // blocks of this wave: all of them (ROWS), or every fourth (KEYS)
  const int nblk = kend > it.key0 ? (kend - it.key0 + KT - 1) / KT : 0;
  const int j0 = KEYS ? wave : 0, jstep = KEYS ? 4 : 1;
  const int cnt = nblk > j0 ? (nblk - j0 + jstep - 1) / jstep : 0;
  auto base_of = [&](int j) { return it.key0 + (j0 + j * jstep) * KT; };
  // whether row block nt sees what is at place x of the item's order
  Seen seen[WIN ? NT : 1];
  if constexpr (WIN) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) seen[nt] = seen_by(it, end_of(wrow0 + nt * 16 + l16), a.window, kend);
  }
  auto sees = [&](int nt, int x) {
    if constexpr (WIN) return seen[nt](x);
    else return x < lim[nt];
  };
  // whether any row of this wave may see keys of the block from base on
  auto busy = [&](int base) {
    if constexpr (!WIN) return base < wave_hi;
    else return base < kend && (base < wave_hi || (base + KT > it.n_late && wrow0 < it.rows));
  };

  float4v o[NT][ND];
  float m[NT], l[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt] = -INFINITY;
    l[nt] = 0.f;
#pragma unroll
    for (int d = 0; d < ND; ++d) o[nt][d] = float4v{0.f, 0.f, 0.f, 0.f};
  }

  if (cnt > 0) {
    // ---- operands of the rows: lane holds row l % 16, values 32 t + 8 g .. + 7 (zero past D)
    half8v qf[NT][NQ];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = min(wrow0 + nt * 16 + l16, it.rows - 1);
      int tok, head;
      if constexpr (WIN) {
        const int i = query_of(a, r, G);
        tok = min(it.tok0 + i, it.last_tok);
        head = it.kvh * G + (r - i * G);
      } else {
        tok = min(it.tok0 + r / G, it.last_tok);
        head = it.kvh * G + r % G;
      }
      const _Float16* q = a.q + (int64_t)tok * a.q_stride + (int64_t)head * D;
#pragma unroll
      for (int t = 0; t < NQ; ++t) {
        const int d = 32 * t + 8 * g;
        qf[nt][t] = d < D ? *reinterpret_cast<const half8v*>(q + d) : half8v{0, 0, 0, 0, 0, 0, 0, 0};
      }
    }
    const float c = a.scale * 1.4426950408889634f;

    // ---- staging
    uint8_t* const kbuf = lds + (KEYS ? wave * 2 * T::BLOCK : 0);
    uint8_t* const pages = lds + (T::LDS - 4 * T::PAGES) + wave * T::PAGES;
    const uint32_t kbuf_at = __builtin_amdgcn_readfirstlane(lds_off(kbuf));
    const uint32_t pages_at = __builtin_amdgcn_readfirstlane(lds_off(pages));
    const int page_mask = (1 << a.page_shift) - 1;
    const uint32_t row_bytes = (uint32_t)D * 2;
    const uint32_t page_bytes = (uint32_t)a.kv_heads * row_bytes << a.page_shift;  // below 2^32 (checked)
    const uint32_t head_bytes = (uint32_t)it.kvh * row_bytes << a.page_shift;
    // token of place x of block j, as its place in the prefix's or the sequence's own pages
    auto place = [&](int j, int x, bool& own) {
      int t = min(base_of(j) + x, kend - 1);
      if constexpr (WIN) t = key_at(it, t);
      own = t >= it.pre;
      return own ? t - it.pre : t;
    };
    // page numbers of block j (one lane each) into ring slot j & 1
    auto load_pages = [&](int j) {
      bool own;
      const int t = place(j, lane & (KT - 1), own);
      const int32_t* e = (own ? it.own : a.prefix_table) + (t >> a.page_shift);
      dma4(e, pages_at + (j & 1) * 256);
    };
    // byte offsets in the cache of the rows that this lane loads of block j
    const int c_lane = lane % SL, r_lane = lane / SL;
    auto row_of_load = [&](int i) { return (KEYS ? i : i * 4 + wave) * RPI + r_lane; };
    int64_t off[LOADS];
    uint32_t past = 0;  // loads whose place lies past D, a bit each
    auto find_rows = [&](int j) {
      past = 0;
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int x = row_of_load(i);
        uint32_t page = reinterpret_cast<const uint32_t*>(pages + (j & 1) * 256)[x];
        if (page >= (uint32_t)a.n_pages) page = 0;
        bool own;
        const int t = place(j, x, own);
        const int slot = slot_of<SL>(x, c_lane);
        const uint32_t in_page = head_bytes + (uint32_t)(t & page_mask) * row_bytes + (FULL || slot * 8 < D ? slot * 16 : 0);
        if (!FULL && slot * 8 >= D) past |= 1u << i;
        off[i] = (int64_t)((uint64_t)page * page_bytes + in_page);
      }
    };
    auto load_block = [&](const _Float16* cache, uint32_t at, auto KEY) {
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const uint8_t* from = reinterpret_cast<const uint8_t*>(cache) + off[i];
        if (!FULL && KEY && (past >> i & 1)) from = reinterpret_cast<const uint8_t*>(&PAST_D);
        dma16v(from, at + (KEYS ? i : i * 4 + wave) * 1024);
      }
    };

    half8v p[NT][NK];
    typedef float4v Scores[NT][NSUB];
    // operand of K: lane holds values 32 t + 8 g .. + 7 of key 16 u + l % 16
    auto k_operand = [&](const uint8_t* kb, int u, int t) {
      const int r = u * 16 + l16;
      return *reinterpret_cast<const half8v*>(kb + r * T::ROWB + slot_of<SL>(r, 4 * t + g) * 16);
    };
    auto score_step = [&](const half8v& kf, Scores& s, int u, int t) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        s[nt][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[nt][t], t ? s[nt][u] : float4v{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
    };
    // S^T of a block: lane holds keys 16 u + 4 g + i of row l % 16
    auto scores = [&](const uint8_t* kb, Scores& s) {
#pragma unroll
      for (int u = 0; u < NSUB; ++u)
#pragma unroll
        for (int t = 0; t < NQ; ++t) score_step(k_operand(kb, u, t), s, u, t);
    };
    // the scores of keys that a row does not see
    auto hide = [&](Scores& s, int base) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int n = lim[nt] - base - 4 * g;
        uint64_t bits = 0;
        if constexpr (WIN) bits = seen[nt].from(base + 4 * g);
#pragma unroll
        for (int u = 0; u < NSUB; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (WIN) s[nt][u][i] = where_seen(bits, u * 16 + i, s[nt][u][i]);
            else s[nt][u][i] = u * 16 + i < n ? s[nt][u][i] : -INFINITY;
          }
      }
    };
    // the largest score of each row of a block (log2 units)
    auto largest = [&](const Scores& s, float (&top)[NT]) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x = -INFINITY;
#pragma unroll
        for (int u = 0; u < NSUB; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) x = fmaxf(x, s[nt][u][i]);
        top[nt] = across_rows(x, [](float p, float q) { return fmaxf(p, q); }) * c;
      }
    };
    // raises the maxima that lag too far, row by row (a row's result does not depend on the
    // rows beside it), with what the rows have summed so far
    auto raise = [&](const float (&top)[NT]) {
      bool any = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) any |= top[nt] > m[nt] + RAISE;
      if (__any(any)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float to = top[nt] > m[nt] + RAISE ? top[nt] : m[nt];
          const float keep = m[nt] == to ? 1.f : exp2_f(m[nt] - to);
          m[nt] = to;
          l[nt] *= keep;
#pragma unroll
          for (int d = 0; d < ND; ++d) o[nt][d] *= keep;
        }
      }
    };
    // probabilities from scores, two at a time: pair x of a block (key half x / (4 NT),
    // then row block, then pairs of its 8 keys), against ref = m or 0 where m is -inf
    float ref[NT];
    auto set_ref = [&] {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) ref[nt] = m[nt] == -INFINITY ? 0.f : m[nt];
    };
    auto exp_pair = [&](const Scores& s, int x) {
      const int k = x / (4 * NT), nt = x / 4 % NT, y = x % 4 * 2;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int u = 2 * k + (y + e) / 4, i = (y + e) % 4;
        const float v = exp2_f(__builtin_fmaf(s[nt][u][i], c, -ref[nt]));
        l[nt] += v;
        p[nt][k][y + e] = (_Float16)v;
      }
    };
    auto exponentials = [&](const Scores& s) {
      set_ref();
#pragma unroll
      for (int x = 0; x < NK * NT * 4; ++x) exp_pair(s, x);
    };
    // operand of V^T: lane holds value 16 d + l % 16 of keys 32 k + 4 g + (0..3) and + 16
    auto v_operand = [&](const uint8_t* vb, int d, int k) {
      half8v v;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int r = k * 32 + hf * 16 + 4 * g + (l16 >> 2);
        const int slot = slot_of<SL>(r, 2 * d + ((l16 >> 1) & 1));
        const uint8_t* at = vb + r * T::ROWB + slot * 16 + (l16 & 1) * 8;
        const short4v x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) short4v*)(__attribute__((address_space(3))) void*)at);
        const half4v y = __builtin_bit_cast(half4v, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[hf * 4 + i] = y[i];
      }
      return v;
    };
    auto product = [&](const uint8_t* vb) {
#pragma unroll
      for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          const half8v v = v_operand(vb, d, k);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) o[nt][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, p[nt][k], o[nt][d], 0, 0, 0);
        }
    };
    // whether a block of values holds no infinity and no NaN
    auto finite = [&](const uint8_t* vb) {
      uint32_t carry = 0;  // an exponent of all ones, plus one, carries into the sign's place
#pragma unroll
      for (int i = 0; i < T::BLOCK / 1024; ++i) {
        const uint4 w = *reinterpret_cast<const uint4*>(vb + i * 1024 + lane * 16);
        carry |= ((w.x & 0x7C007C00u) + 0x04000400u) | ((w.y & 0x7C007C00u) + 0x04000400u) |
                 ((w.z & 0x7C007C00u) + 0x04000400u) | ((w.w & 0x7C007C00u) + 0x04000400u);
      }
      return !__any((carry & 0x80008000u) != 0);
    };
    // Takes the infinities and NaN out of a block of values that some rows do not see whole
    // (0 times one would be NaN): first each is added to the rows that see its key, then it
    // becomes 0 in LDS.  Rare, and small rather than fast: one element at a time.
    auto set_apart = [&](uint8_t* vb, int base) {
      constexpr int PER = DP / 64;  // values of a key that a lane looks at
#pragma unroll 1
      for (int x = 0; x < KT; ++x) {
#pragma unroll 1
        for (int h = 0; h < PER; ++h) {
          const int e = lane * PER + h;
          const uint32_t bits =
              *reinterpret_cast<const uint16_t*>(vb + x * T::ROWB + slot_of<SL>(x, e / 8) * 16 + e % 8 * 2);
          uint64_t bad = __ballot((bits & 0x7C00u) == 0x7C00u);
          while (bad) {
            const int from = __builtin_ctzll(bad);
            bad &= bad - 1;
            const uint32_t b16 = (uint32_t)__builtin_amdgcn_readlane((int)bits, from);
            const float val = (float)__builtin_bit_cast(_Float16, (uint16_t)b16);
            const int at = from * PER + h;  // place of the value: register (at / 16, at % 4) of lanes with g = at / 4 % 4
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float add = g == (at >> 2 & 3) && sees(nt, base + x) ? val : 0.f;
#pragma unroll
              for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (d == at >> 4 && i == (at & 3)) o[nt][d][i] += add;
            }
          }
        }
      }
      reads_done();
      if constexpr (!KEYS) asm volatile("s_barrier" ::: "memory");  // (no wave cleans what another still looks at)
#pragma unroll 1
      for (int i = KEYS ? 0 : wave; i < T::BLOCK / 1024; i += KEYS ? 1 : 4) {
        uint4* at = reinterpret_cast<uint4*>(vb + i * 1024 + lane * 16);
        uint4 w = *at;
        auto clean = [](uint32_t& x) {
          if ((x & 0x7C00u) == 0x7C00u) x &= 0xFFFF0000u;
          if ((x & 0x7C000000u) == 0x7C000000u) x &= 0xFFFFu;
        };
        clean(w.x);
        clean(w.y);
        clean(w.z);
        clean(w.w);
        *at = w;
      }
      reads_done();
      if constexpr (!KEYS) asm volatile("s_barrier" ::: "memory");
    };

    if constexpr (KEYS) {
      // One block of keys and one of values per wave: the next keys load from the moment
      // the scores are done, the next values from the moment the product is.  Loads land
      // in order, so a count of newer ones says when a block is there.
      load_pages(0);
      landed<0>();
      find_rows(0);
      reads_done();
      load_pages(1);
      load_block(a.k, kbuf_at, std::true_type{});
      load_block(a.v, kbuf_at + T::BLOCK, std::false_type{});
      for (int j = 0; j < cnt; ++j) {
        const bool more = j + 1 < cnt;
        const int base = base_of(j);
        const bool masked = base + KT > wave_lo;
        landed<LOADS>();  // the values may still be on their way
        Scores s;
        scores(kbuf, s);
        if (more) find_rows(j + 1);
        reads_done();
        if (more) {
          load_pages(j + 2);
          load_block(a.k, kbuf_at, std::true_type{});
        }
        if (masked) hide(s, base);
        float top[NT];
        largest(s, top);
        raise(top);
        exponentials(s);
        if (more) landed<LOADS + 1>();
        else landed<0>();
        if (masked && !finite(kbuf + T::BLOCK)) set_apart(kbuf + T::BLOCK, base);
        product(kbuf + T::BLOCK);
        reads_done();
        if (more) load_block(a.v, kbuf_at + T::BLOCK, std::false_type{});
      }
    } else {
      // Two blocks each of keys and values for the workgroup, of which a wave loads a
      // quarter.  Keys run one block ahead of the values: while the vector units take the
      // exponentials of block j, the matrix cores score block j + 1, and while they
      // multiply block j with its values, its successor's maxima are found.
      uint8_t* const vbuf = kbuf + 2 * T::BLOCK;
      const uint32_t vbuf_at = kbuf_at + 2 * T::BLOCK;
      load_pages(0);
      load_pages(1);
      landed<0>();
      find_rows(0);
      load_block(a.k, kbuf_at, std::true_type{});
      load_block(a.v, vbuf_at, std::false_type{});
      find_rows(1);
      reads_done();
      load_pages(2);
      if (cnt > 1) load_block(a.k, kbuf_at + T::BLOCK, std::true_type{});
      // blocks that every row of the tile sees whole
      const int whole = (max(limit_of(it.row0), it.key0) - it.key0) / KT;
      Scores sa, sb;
      float top[NT];
      landed<0>();
      asm volatile("s_barrier" ::: "memory");
      scores(kbuf, sa);
      if (whole < 1) hide(sa, it.key0);
      largest(sa, top);
      raise(top);
      // block j and the loads behind it; LDS halves of the two parities
      auto stage = [&](int j, int odd) {
        landed<0>();
        reads_done();
        asm volatile("s_barrier" ::: "memory");  // keys j + 1 and values j are whole; keys j, values j - 1 no longer read
        if (j + 1 < cnt) load_block(a.v, vbuf_at + (odd ^ 1) * T::BLOCK, std::false_type{});
        if (j + 2 < cnt) {
          find_rows(j + 2);
          reads_done();
          load_pages(j + 3);
          load_block(a.k, kbuf_at + odd * T::BLOCK, std::true_type{});
        }
      };
      // A block that every row sees whole, in a fixed order of small steps (the fences keep
      // the scheduler from hoisting all reads to the front, which spilled): each step has
      // its MFMAs, the LDS read of the operand AHEAD steps on, and a share of the vector
      // work that fits in their shadow: in the scores of the next block the exponentials
      // of this one's first 32 keys, in the first half of the product those of the other
      // 32, in its second half the next block's maxima.
      auto whole_block = [&](int j, int odd, Scores& now, Scores& next) {
        constexpr int AHEAD = 4, NS = NSUB * NQ, NP = NK * ND, PAIRS = NT * 4;
        stage(j, odd);
        const uint8_t* kb = kbuf + (odd ^ 1) * T::BLOCK;
        const uint8_t* vb = vbuf + odd * T::BLOCK;
        auto fence = [] { __builtin_amdgcn_sched_barrier(0); };
        half8v f[AHEAD];
        set_ref();
#pragma unroll
        for (int x = 0; x < AHEAD; ++x) f[x] = k_operand(kb, x / NQ, x % NQ);
        fence();
        static_for(std::make_integer_sequence<int, NS>{}, [&](auto X) {
          constexpr int x = decltype(X)::value;
          score_step(f[x % AHEAD], next, x / NQ, x % NQ);
          if constexpr (x + AHEAD < NS) f[x % AHEAD] = k_operand(kb, (x + AHEAD) / NQ, (x + AHEAD) % NQ);
          else f[x % AHEAD] = v_operand(vb, x + AHEAD - NS, 0);
#pragma unroll
          for (int y = x * PAIRS / NS; y < (x + 1) * PAIRS / NS; ++y) exp_pair(now, y);
          fence();
        });
        static_assert(NS % AHEAD == 0 && ND >= AHEAD && NK == 2, "operand ring");
        float part[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) part[nt] = -INFINITY;
        static_for(std::make_integer_sequence<int, NP>{}, [&](auto X) {
          constexpr int x = decltype(X)::value, k = x / ND, d = x % ND;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            o[nt][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f[x % AHEAD], p[nt][k], o[nt][d], 0, 0, 0);
          if constexpr (x + AHEAD < NP) f[x % AHEAD] = v_operand(vb, (x + AHEAD) % ND, (x + AHEAD) / ND);
          if constexpr (k == 0) {
#pragma unroll
            for (int y = d * PAIRS / ND; y < (d + 1) * PAIRS / ND; ++y) exp_pair(now, PAIRS + y);
          } else {
#pragma unroll
            for (int y = d * NSUB * NT / ND; y < (d + 1) * NSUB * NT / ND; ++y)
#pragma unroll
              for (int i = 0; i < 4; ++i) part[y % NT] = fmaxf(part[y % NT], next[y % NT][y / NT][i]);
          }
          fence();
        });
        if (j + 1 < whole) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) top[nt] = across_rows(part[nt], [](float x, float y) { return fmaxf(x, y); }) * c;
        } else {  // (past the last block: nothing is seen of what its buffer holds)
          hide(next, base_of(j + 1));
          largest(next, top);
        }
        raise(top);
      };
      int j = 0;
      for (; j + 1 < whole; j += 2) {
        whole_block(j, 0, sa, sb);
        whole_block(j + 1, 1, sb, sa);
      }
      if (j < whole) {
        whole_block(j, 0, sa, sb);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int u = 0; u < NSUB; ++u) sa[nt][u] = sb[nt][u];
        ++j;
      }
#pragma unroll 1
      for (; j < cnt; ++j) {
        stage(j, j & 1);
        const int base = base_of(j);
        uint8_t* const vb = vbuf + (j & 1) * T::BLOCK;
        if (!finite(vb)) set_apart(vb, base);  // all four waves or none
        if (busy(base)) {
          exponentials(sa);
          product(vb);
        }
        if (busy(base + KT)) {
          scores(kbuf + ((j & 1) ^ 1) * T::BLOCK, sa);
          if (base + 2 * KT > wave_lo) hide(sa, base + KT);
          largest(sa, top);
          raise(top);
        }
      }
    }
    landed<0>();  // no load outlives the workgroup's LDS
  }

  // ---- results: lane holds values 16 d + 4 g + i of row l % 16
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) l[nt] = across_rows(l[nt], [](float x, float y) { return x + y; });
  // number of row r among all (query, head) pairs
  auto pair_of = [&](int r) {
    const int i = query_of(a, r, G);
    return (int64_t)(it.tok0 + i) * a.q_heads + it.kvh * G + (r - i * G);
  };
  // (m, l, o) of a pair: into its partial slot, or divided into the output
  const int64_t slot0 = (int64_t)it.slot * a.T * a.q_heads;
  auto emit4 = [&](int64_t th, int d0, float4v v, float mm, float ll, float inv) {
    if (sp.slots) {
      *reinterpret_cast<float4v*>(sp.part_o + (slot0 + th) * D + d0) = v;
      if (d0 == 0) sp.part_ml[slot0 + th] = make_float2(mm, ll);
    } else {
      const bool none = mm == -INFINITY && ll == 0.f;  // a row that saw nothing
      half4v h;
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = (_Float16)(none ? 0.f : v[i] * inv);
      *reinterpret_cast<half4v*>(a.out + th * D + d0) = h;
      if (a.lse && d0 == 0) a.lse[th] = none ? -INFINITY : (mm + __log2f(ll)) * 0.6931471805599453f;
    }
  };
  if constexpr (KEYS) {
    __syncthreads();
    float* ro = reinterpret_cast<float*>(lds);                        // [wave][row][DP + 4]
    float2* rml = reinterpret_cast<float2*>(ro + 4 * 16 * (DP + 4));  // [wave][row]
#pragma unroll
    for (int d = 0; d < ND; ++d) *reinterpret_cast<float4v*>(ro + (wave * 16 + l16) * (DP + 4) + d * 16 + 4 * g) = o[0][d];
    if (g == 0) rml[wave * 16 + l16] = make_float2(m[0], l[0]);
    __syncthreads();
    for (int x = threadIdx.x; x < 16 * (DP / 4); x += 256) {
      const int r = x / (DP / 4), d0 = x % (DP / 4) * 4;
      if (it.row0 + r >= it.rows || d0 >= D) continue;
      float mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) mm = fmaxf(mm, rml[w * 16 + r].x);
      float4v v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float2 ml = rml[w * 16 + r];
        if (ml.x == -INFINITY && ml.y == 0.f) continue;
        const float f = ml.x == mm ? 1.f : exp2_f(ml.x - mm);
        ll += f * ml.y;
        v += f * *reinterpret_cast<const float4v*>(ro + (w * 16 + r) * (DP + 4) + d0);
      }
      emit4(pair_of(it.row0 + r), d0, v, mm, ll, 1.f / ll);
    }
  } else {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = wrow0 + nt * 16 + l16;
      if (r >= it.rows) continue;
      const int64_t th = pair_of(r);
      const float inv = 1.f / l[nt];
#pragma unroll
      for (int d = 0; d < ND; ++d)
        if (d * 16 + 4 * g < D) emit4(th, d * 16 + 4 * g, o[nt][d], m[nt], l[nt], inv);
    }
  }
}

// queries of sequence b: first row of q, how many within q, and n of them within max_q
__device__ __forceinline__ int queries_of(const AttnArgs& a, int b, int& start, int& n) {
  start = min(max(a.q_starts[b], 0), a.T);
  const int all = min(max(a.q_starts[b + 1], start), a.T) - start;
  n = min(all, a.max_q);
  return all;
}

// The w-th item of a call with a window; false where it has no rows.  (Placed as in attend_kernel
// below, whose items are written out there: through a function of their own its tiles of 128 rows
// took other registers and 4 % longer.)
template <int KIND>
__device__ __forceinline__ bool window_item(const WindowArgs& a, const AttnSplit& sp, int w, Item& it) {
  const int above = a.by_groups(w), tile = sp.s_tiles - 1 - above, group = w - above * a.groups;
  const int pair = a.by_kv_heads(group), b = a.by_splits(pair), part = pair - b * sp.s_splits;
  it.kvh = group - pair * a.kv_heads;
  int n;
  const int all = queries_of(a, b, it.tok0, n);
  it.row0 = tile * tile_rows(KIND);
  it.rows = n * a.per_head;
  if (it.row0 >= it.rows) return false;
  it.last_tok = it.tok0 + n - 1;
  const int64_t room = a.table_width << a.page_shift;
  const int len = max(a.kv_lens[b], 0), held = (int)min((int64_t)min(len, a.max_len), room);
  it.pre = it.pre_lim = (int)a.prefix_len;
  it.lim0 = len - all + 1;
  it.key0 = part * sp.s_chunk;
  it.slot = part;
  it.own = a.tables + (int64_t)b * a.table_width;
  // the ends of the tile's first and last row, and where their windows begin
  const int end0 = end_at(it, a.by_per_head(it.row0));
  const int end1 = end_at(it, a.by_per_head(min(it.row0 + tile_rows(KIND), it.rows) - 1));
  const int begin1 = end1 - a.window;
  it.held = it.pre + held;
  it.late = it.early = it.n_early = 0;
  int n_first = 0;
  if (begin1 > a.sinks) {  // (else no row has a key between its first ones and its window)
    it.late = begin1;
    it.early = max(a.sinks, end0 - a.window);
    it.n_early = max(0, min(it.late, it.held) - it.early);
    n_first = min(a.sinks, it.held);
  }
  it.n_late = max(0, min(end1, it.held) - it.late);
  it.list = it.n_late + it.n_early + n_first;
  it.key1 = min(it.list, it.key0 + sp.s_chunk);
  return true;
}

template <int DP, int KIND_P, int KIND_S, bool FULL, typename Args>
__global__ __launch_bounds__(256, DP == 256 ? 1 : 2) void attend_kernel(Args a, AttnSplit sp) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  int w = blockIdx.x;
  Item it;
  if constexpr (std::is_same_v<Args, WindowArgs>) {
    if (window_item<KIND_S>(a, sp, w, it)) attend_tile<DP, KIND_S, FULL>(a, sp, it, lds);
    return;
  }
  const int G = a.q_heads / a.kv_heads;
  if (KIND_P != TILE_NONE && w < sp.p_items) {
    // workgroups go to the 8 XCDs in turn: the tiles of one part and head (the same keys)
    // follow each other in one of them
    const int groups = a.kv_heads * sp.p_splits;
    int group, tile;
    if ((groups & 7) == 0) {
      group = (w >> 3) / sp.p_tiles * 8 + (w & 7);
      tile = (w >> 3) % sp.p_tiles;
    } else {
      group = w / sp.p_tiles;
      tile = w % sp.p_tiles;
    }
    const int part = group % sp.p_splits;
    it.kvh = group / sp.p_splits;
    it.row0 = tile * tile_rows(KIND_P);
    it.rows = a.T * G;
    it.tok0 = 0;
    it.last_tok = a.T - 1;
    it.key0 = part * sp.p_chunk;
    it.key1 = min((int)a.prefix_len, it.key0 + sp.p_chunk);
    it.pre = it.pre_lim = (int)a.prefix_len;
    it.lim0 = INT32_MIN / 2;
    it.slot = part;
    it.own = nullptr;
    if constexpr (KIND_P != TILE_NONE) attend_tile<DP, KIND_P, FULL>(a, sp, it, lds);
    return;
  }
  if (KIND_P != TILE_NONE) w -= sp.p_items;
  // The last tiles of the sequences see the most keys: they start first, of all sequences.
  // A group (sequence, part, head: the same keys) stays in one XCD where the groups divide
  // evenly, and the heads of a sequence, which cost the same, go to different ones (with a
  // sequence in one XCD, four prompts of 700 to 1024 tokens took 165 us).
  const int groups = sp.s_items / sp.s_tiles;
  int tile, group;
  if ((groups & 7) == 0) {
    tile = sp.s_tiles - 1 - (w >> 3) / (groups >> 3);
    group = (w >> 3) % (groups >> 3) * 8 + (w & 7);
  } else {
    tile = sp.s_tiles - 1 - w / groups;
    group = w % groups;
  }
  it.kvh = group % a.kv_heads;
  const int part = group / a.kv_heads % sp.s_splits;
  const int b = group / a.kv_heads / sp.s_splits;
  int n;
  const int all = queries_of(a, b, it.tok0, n);
  it.row0 = tile * tile_rows(KIND_S);
  it.rows = n * G;
  if (it.row0 >= it.rows) return;
  it.last_tok = it.tok0 + n - 1;
  const int64_t room = a.table_width << a.page_shift;
  const int len = max(a.kv_lens[b], 0), held = (int)min((int64_t)min(len, a.max_len), room);
  it.pre = it.pre_lim = sp.shared ? 0 : (int)a.prefix_len;
  it.lim0 = len - all + 1;  // from the true lengths, also where rows or tokens past the call's bounds are left out
  it.key0 = part * sp.s_chunk;
  it.key1 = min(it.pre + held, it.key0 + sp.s_chunk);
  it.slot = (sp.shared ? sp.p_splits : 0) + part;
  it.own = a.tables + (int64_t)b * a.table_width;
  attend_tile<DP, KIND_S, FULL>(a, sp, it, lds);
}

template <int DP, int KIND_P, int KIND_S, typename Args>
hipError_t launch_kinds(const Args& a, const AttnSplit& p, hipStream_t st) {
  constexpr int ls = TileGeo<DP, KIND_S>::LDS;
  constexpr int lp = KIND_P == TILE_NONE ? 0 : TileGeo<DP, KIND_P == TILE_NONE ? KIND_S : KIND_P>::LDS;
  constexpr int lds = ls > lp ? ls : lp;
  static_assert(lds <= 160 * 1024, "LDS budget");
  const dim3 grid((unsigned)(p.p_items + p.s_items));
  if (a.D == DP) hipLaunchKernelGGL((attend_kernel<DP, KIND_P, KIND_S, true, Args>), grid, dim3(256), lds, st, a, p);
  else hipLaunchKernelGGL((attend_kernel<DP, KIND_P, KIND_S, false, Args>), grid, dim3(256), lds, st, a, p);
  return hipGetLastError();
}

}  // namespace
}  // namespace qg
