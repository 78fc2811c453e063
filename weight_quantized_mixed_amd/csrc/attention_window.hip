// Attention with a window: tiles of 128 rows on 32 x 32 x 16 MFMAs (up to 64 rows a sequence take the
// tiles of attention_kernel.hpp).
//
// A wave has 32 rows.  S^T = K Q^T takes 32 keys at a time and 16 places of the head, O^T = V^T P^T
// 32 places of the head and 16 keys.  Lane l holds row l % 32; of a product's 32 results per row
// (keys, or places) it has 8 q + 4 (l / 32) + i for q, i < 4, and its scores are the operand of the
// second product as they are, as in the 16 x 16 tiles, with half as many maxima and sums to bring
// together.  Why 32 x 32: next to a matrix instruction the vector unit stands still for about 8
// cycles whatever the shape, so with two waves on a SIMD 32 cycles of matrix work beside four
// fused multiply-adds and one exponential took 38 cycles a wave as one 32 x 32 x 16 and 47 as two
// 16 x 16 x 32 (measured alone).
//
// A block of 64 keys, the same for whole and for masked ones: while the matrix cores score block
// j + 1 the vector units take the exponentials of block j, and while they multiply those with the
// values the maxima of block j + 1 are found; steps of one MFMA, the LDS reads four steps ahead
// (the compiler may move things between the steps: fences kept them apart for nothing, but sums and
// maxima that it gathered behind the loop cost 2 %).
//
// Measured (8192 tokens of one prompt, 32 / 8 heads of 128): window 64 46 us, 256 72 us, 1024
// 162 us (807 TFLOP/s), 4096 426 us (970); 32 / 4 heads of 64: 26, 40, 96 and 261 us.  The 16 x 16 x
// 32 tiles took 78, 111, 200 and 466 us with heads of 128, these 54, 79, 169 and 435 as they were
// first; then scores hidden by bits instead of intervals (window 64 54 -> 49 us) and items placed
// without divisions (49 -> 46).  16 / 4 heads of 256 (one workgroup a CU, sums in the accumulation
// registers): 67, 95, 199 and 482 us, on 16 x 16 x 32 tiles of 64 rows 94, 146, 325 and 816.  Heads of
// 136 to 248, whose loads past the head are set apart, spill 11 registers (24 / 8 heads of 192, window
// 1024 272 us).  Precision: as in attention_kernel.hpp, with the probabilities in fp16 as operands.
//
// With heads of 128 a block of two workgroups takes a CU about 3850 cycles (4650 on the 16 x 16 tiles)
// at 1.84 GHz (2.04): the clock gives way to the matrix cores, so fewer stalls buy less time than
// cycles, and neither deeper operand rings, other orders of the steps nor wave priorities moved it by
// 1 %.  The LDS gives each wave the whole block, 32 KiB of keys and values: 1024 cycles for the four
// waves, as many as their products; 64 rows a wave would halve that, but left one wave to a SIMD and
// took no less time.
//
// Where a key's row lies in the cache one lane of each wave finds out, two blocks ahead of its
// loads, and leaves it in LDS for the lanes that load (found by every lane for itself it took about
// 50 more vector instructions a block).
#include "attention_kernel.hpp"

namespace qg {
namespace {

constexpr int KT = 64;  // keys of a block

template <int DP>
struct RowsGeo {
  static constexpr int ROWB = DP * 2, SL = ROWB / 16;  // bytes and 16-byte slots of a key
  static constexpr int RPI = 64 / SL;                  // keys per 1 KiB load
  static constexpr int BLOCK = KT * ROWB;              // bytes of a block of keys, or of values
  static constexpr int LOADS = BLOCK / 4096;           // per wave
  static constexpr int NQ = DP / 16, ND = DP / 32;     // steps of a score, 32-place blocks of a result
  static constexpr int RING = 2 * KT * 8;              // where the rows of two blocks lie, per wave
  static constexpr int LDS = 4 * BLOCK + 4 * RING + 16;
};

// Slot c of key r lies at c XOR f(r), f linear in the bits of r.  A read of keys takes 32 keys at
// one slot and its neighbour, one of values 8 keys at 4 neighbouring slots; with these every 16, 32
// and 64 lanes (values: 32 and 64) touch every bank of 256, 512 or 1024 bytes once (checked for all
// reads on the host).  Values depend on the three lowest bits only, which a lane's reads share.
template <int SL>
__device__ __forceinline__ constexpr int key_swizzle(int r) {
  if constexpr (SL == 8) return ((r >> 2) & 3) | ((((r >> 4) ^ (r >> 1)) & 1) << 2);
  return ((r >> 1) & 15) ^ ((r & 1) << 3);
}
template <int SL>
__device__ __forceinline__ constexpr int value_swizzle(int r) {
  if constexpr (SL == 8) return (((r >> 1) ^ (r >> 2)) & 1) << 2;
  return (((r ^ (r >> 2)) & 1) << 3) | (((r >> 1) & 1) << 2);
}

typedef float float16v __attribute__((ext_vector_type(16)));

// keeps the computation of v where it is written
__device__ __forceinline__ void stay(float& v) { asm volatile("" : "+v"(v)); }

template <int DP, bool FULL>
__global__ __launch_bounds__(256, DP == 64 ? 3 : DP == 128 ? 2 : 1) void window_rows_kernel(WindowArgs a, AttnSplit sp) {
  using T = RowsGeo<DP>;
  constexpr int SL = T::SL, LOADS = T::LOADS, NQ = T::NQ, ND = T::ND;
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  Item it;
  if (!window_item<TILE_ROWS128>(a, sp, blockIdx.x, it)) return;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, l32 = lane & 31, l16 = lane & 15;
  const int G = a.per_head, D = a.D;
  const int kend = __builtin_amdgcn_readfirstlane(it.key1);
  const int cnt = kend > it.key0 ? (kend - it.key0 + KT - 1) / KT : 0;
  auto base_of = [&](int j) { return it.key0 + j * KT; };

  // this lane's row, its place among the tokens and what it sees
  const int row = min(it.row0 + wave * 32 + l32, it.rows - 1), query = a.by_per_head(row);
  const Seen seen = seen_by(it, end_at(it, query), a.window, kend);
  // blocks that every row of the tile sees whole
  const int first_end = end_at(it, a.by_per_head(it.row0));
  const int whole = (max(min(kend, min(max(min(first_end, it.held) - it.late, 0), it.n_late)), it.key0) - it.key0) / KT;

  // ... the leading ones, and among the first keys (of which later rows see what the tile's first does:
  // 8192 tokens of 32 / 8 heads of 128, window 1024 and 512 first ones 228 -> 218 us)
  const int first_at = it.n_late + it.n_early, first_to = min(kend, first_at + min(first_end, it.list - first_at));
  auto masked = [&](int j) { return j >= whole && !(base_of(j) >= first_at && base_of(j) + KT <= first_to); };

  float16v o[ND];
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;

  if (cnt > 0) {
    const float c = a.scale * 1.4426950408889634f;

    // ---- staging
    uint64_t* const ring = reinterpret_cast<uint64_t*>(lds + 4 * T::BLOCK + wave * T::RING);
    const uint32_t lds_at = __builtin_amdgcn_readfirstlane(lds_off(lds)) + wave * 1024;
    const uint32_t row_bytes = (uint32_t)D * 2;
    const uint32_t page_bytes = (uint32_t)a.kv_heads * row_bytes << a.page_shift;  // below 2^32 (checked)
    const uint32_t head_bytes = (uint32_t)it.kvh * row_bytes << a.page_shift;
    const uint32_t page_mask = (1u << a.page_shift) - 1;
    // of key `lane` of a block: its page's number, on its way, and its place in the page
    struct Where {
      uint32_t page, in_page;
    };
    auto find = [&](int j) {
      const int key = key_at(it, min(base_of(j) + lane, kend - 1));
      const bool own = key >= it.pre;
      const int t = own ? key - it.pre : key;
      Where w;
      w.page = (uint32_t)(own ? it.own : a.prefix_table)[t >> a.page_shift];
      w.in_page = head_bytes + ((uint32_t)t & page_mask) * row_bytes;
      return w;
    };
    auto publish = [&](int j, Where w) {
      if (w.page >= (uint32_t)a.n_pages) w.page = 0;
      ring[(j & 1) * KT + lane] = (uint64_t)w.page * page_bytes + w.in_page;
      __builtin_amdgcn_wave_barrier();  // (read by other lanes)
    };
    // key that load i of this lane takes, and the 16 bytes of it (load i differs by an XOR)
    const int c_lane = lane % SL, r_lane = wave * T::RPI + lane / SL;
    auto row_of_load = [&](int i) { return i * 4 * T::RPI + r_lane; };
    const int key_slot = c_lane ^ key_swizzle<SL>(r_lane), value_slot = c_lane ^ value_swizzle<SL>(r_lane);
    auto rows_of = [&](int j, uint64_t (&off)[LOADS]) {
#pragma unroll
      for (int i = 0; i < LOADS; ++i) off[i] = ring[(j & 1) * KT + row_of_load(i)];
    };
    auto load_block = [&](const _Float16* cache, const uint64_t (&off)[LOADS], uint32_t at, auto KEY) {
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        int slot = KEY ? key_slot ^ key_swizzle<SL>(i * 4 * T::RPI) : value_slot ^ value_swizzle<SL>(i * 4 * T::RPI);
        const bool past = !FULL && slot * 8 >= D;  // zeros in keys, what is at hand in values
        if (past) slot = 0;
        const uint8_t* from = reinterpret_cast<const uint8_t*>(cache) + off[i] + (uint32_t)slot * 16;
        if (KEY && past) from = reinterpret_cast<const uint8_t*>(&PAST_D);
        dma16v(from, lds_at + at + i * 4096);
      }
    };
    constexpr uint32_t VALUES = 2 * T::BLOCK;
    auto load_keys = [&](int j, const uint64_t (&off)[LOADS]) { load_block(a.k, off, (j & 1) * T::BLOCK, std::true_type{}); };
    auto load_values = [&](int j, const uint64_t (&off)[LOADS]) {
      load_block(a.v, off, VALUES + (j & 1) * T::BLOCK, std::false_type{});
    };

    Where w0 = find(0), w1 = find(1);
    publish(0, w0);
    publish(1, w1);
    Where next_rows = find(2);
    uint64_t off[LOADS];
    rows_of(0, off);
    load_keys(0, off);
    load_values(0, off);
    rows_of(1, off);
    if (cnt > 1) load_keys(1, off);

    // ---- operands: lane holds values 16 t + 8 half .. + 7 of its row (zero past D)
    half8v qf[NQ];
    {
      const int tok = min(it.tok0 + query, it.last_tok), head = it.kvh * G + (row - query * G);
      const _Float16* q = a.q + (int64_t)tok * a.q_stride + (int64_t)head * D;
#pragma unroll
      for (int t = 0; t < NQ; ++t) {
        const int d = 16 * t + 8 * half;
        qf[t] = FULL || d < D ? *reinterpret_cast<const half8v*>(q + d) : half8v{0, 0, 0, 0, 0, 0, 0, 0};
      }
    }
    // ... values 16 t + 8 half .. + 7 of key 32 u + l % 32
    const uint32_t key_read = l32 * T::ROWB + ((half ^ key_swizzle<SL>(l32)) * 16);
    auto k_operand = [&](int odd, int u, int t) {
      return *reinterpret_cast<const half8v*>(lds + odd * T::BLOCK + u * 32 * T::ROWB + (key_read ^ (t * 32)));
    };
    // ... value 32 d + l % 32 of keys 16 k + 4 half + (0..3) and + 8
    uint32_t value_read;
    {
      const int r = 4 * half + (l16 >> 2), lo = 2 * ((lane >> 4) & 1) + ((l16 >> 1) & 1);
      value_read = r * T::ROWB + (value_swizzle<SL>(r) + lo) * 16 + (l16 & 1) * 8;
    }
    auto v_operand = [&](int odd, int d, int k) {
      half8v v;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const uint8_t* at = lds + VALUES + odd * T::BLOCK + (16 * k + 8 * hf) * T::ROWB + (value_read ^ (d * 64));
        const short4v x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) short4v*)(__attribute__((address_space(3))) void*)at);
        const half4v y = __builtin_bit_cast(half4v, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[hf * 4 + i] = y[i];
      }
      return v;
    };

    typedef float16v Scores[2];
    half8v p[4];
    auto score_step = [&](const half8v& kf, Scores& s, int u, int t) {
      if (t == 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[u][i] = 0.f;
      }
      s[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, qf[t], s[u], 0, 0, 0);
    };
    auto hide = [&](Scores& s, int base) {
      const uint64_t bits = seen.from(base + 4 * half);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[u][i] = where_seen(bits, 32 * u + 8 * (i / 4) + i % 4, s[u][i]);
    };
    // over the two lanes of a row
    auto both = [&](float v, auto f) {
      const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
      return f(__uint_as_float(x[0]), __uint_as_float(x[1]));
    };
    auto larger = [](float x, float y) { return fmaxf(x, y); };
    auto largest = [&](const Scores& s) {
      float x = -INFINITY;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) x = fmaxf(x, s[u][i]);
      return both(x, larger) * c;
    };
    float ref = 0.f;
    // raises the maxima that lag too far, with what the rows have summed so far
    auto raise = [&](float top) {
      if (__any(top > m + RAISE)) {
        const float to = top > m + RAISE ? top : m;
        const float keep = m == to ? 1.f : exp2_f(m - to);
        m = to;
        l *= keep;
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          // (in accumulation registers with heads of 256: read here, and not on the way to the branch, 213 -> 199 us)
          if constexpr (DP == 256) asm volatile("" : "+a"(o[d]));
          o[d] *= keep;
        }
      }
      ref = m == -INFINITY ? 0.f : m;
    };
    // probabilities, two at a time: pair x of a block (keys 16 (x / 4) .., the lane's places 2 (x % 4) and + 1)
    auto exp_pair = [&](const Scores& s, int x) {
      const int k = x / 4, y = x % 4 * 2;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float v = exp2_f(__builtin_fmaf(s[k / 2][8 * (k % 2) + y + e], c, -ref));
        l += v;
        p[k][y + e] = (_Float16)v;
      }
      stay(l);
    };
    auto product_step = [&](const half8v& v, int d, int k) { o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, p[k], o[d], 0, 0, 0); };

    // Takes the infinities and NaN out of a block of values that some rows do not see whole (0 times
    // one would be NaN): they become 0 in LDS, and are added behind the last block.  A quarter of the
    // block is looked at by each wave; the rest is rare.
    uint32_t* const flag = reinterpret_cast<uint32_t*>(lds + 4 * T::BLOCK + 4 * T::RING);
    int cleaned_from = cnt, cleaned_to = 0;  // all blocks that were changed are among these
    auto clean = [&](int j, int odd) {
      int lane = threadIdx.x & 63;
      asm volatile("" : "+v"(lane));  // (addresses made here, rather than kept through the loop and spilled)
      uint8_t* const vb = lds + VALUES + odd * T::BLOCK;
      uint32_t carry = 0;  // an exponent of all ones, plus one, carries into the sign's place
#pragma unroll
      for (int i = 0; i < T::BLOCK / 4096; ++i) {
        const uint4 w = *reinterpret_cast<const uint4*>(vb + (i * 4 + wave) * 1024 + lane * 16);
        carry |= ((w.x & 0x7C007C00u) + 0x04000400u) | ((w.y & 0x7C007C00u) + 0x04000400u) |
                 ((w.z & 0x7C007C00u) + 0x04000400u) | ((w.w & 0x7C007C00u) + 0x04000400u);
      }
      const bool bad_here = __any((carry & 0x80008000u) != 0);
      if (lane == 0) flag[wave] = bad_here;
      reads_done();
      asm volatile("s_barrier" ::: "memory");
      const uint4 f = *reinterpret_cast<const uint4*>(flag);
      if (__builtin_amdgcn_readfirstlane(f.x | f.y | f.z | f.w) != 0) {
        cleaned_from = min(cleaned_from, j);
        cleaned_to = j + 1;
#pragma unroll 1
        for (int i = wave; i < T::BLOCK / 1024; i += 4) {
          uint4* at = reinterpret_cast<uint4*>(vb + i * 1024 + lane * 16);
          uint4 w = *at;
          auto zero = [](uint32_t& x) {
            if ((x & 0x7C00u) == 0x7C00u) x &= 0xFFFF0000u;
            if ((x & 0x7C000000u) == 0x7C000000u) x &= 0xFFFFu;
          };
          zero(w.x);
          zero(w.y);
          zero(w.z);
          zero(w.w);
          *at = w;
        }
        reads_done();
        asm volatile("s_barrier" ::: "memory");
      }
    };
    // ... and adds each to the rows that see its key: the values of those blocks read again from the cache, one
    // value of a key at a time (in the loop, with heads of 256, it drove the sums into memory).  Blocks of first
    // keys that all rows see were not cleaned and may lie between them.
    auto add_cleaned = [&] {
      constexpr int PER = DP / 64;  // values of a key that a lane looks at
#pragma unroll 1
      for (int x = base_of(cleaned_from); x < min(base_of(cleaned_to), kend); ++x) {
        if (!masked((x - it.key0) / KT)) continue;
        const int key = key_at(it, x);
        const bool own = key >= it.pre;
        const int t = own ? key - it.pre : key;
        uint32_t page = (uint32_t)(own ? it.own : a.prefix_table)[t >> a.page_shift];
        if (page >= (uint32_t)a.n_pages) page = 0;
        const _Float16* const row = a.v + ((uint64_t)page * page_bytes + head_bytes + ((uint32_t)t & page_mask) * row_bytes) / 2;
#pragma unroll 1
        for (int h = 0; h < PER; ++h) {
          const int e = lane * PER + h;
          const uint32_t bits = FULL || e < D ? __builtin_bit_cast(uint16_t, row[e]) : 0;
          uint64_t bad = __ballot((bits & 0x7C00u) == 0x7C00u);
          while (bad) {
            const int from = __builtin_ctzll(bad);
            bad &= bad - 1;
            const float val = (float)__builtin_bit_cast(_Float16, (uint16_t)__builtin_amdgcn_readlane((int)bits, from));
            const int at = from * PER + h;  // place of the value: o[at / 32][4 (at / 8 % 4) + at % 4] of lanes with half at / 4 % 2
            const float add = half == (at >> 2 & 1) && seen(x) ? val : 0.f;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
              for (int i = 0; i < 16; ++i)
                o[d][i] += d == at >> 5 && i == (at >> 3 & 3) * 4 + (at & 3) ? add : 0.f;
          }
        }
      }
    };

    // Keys j + 1 and values j are whole, keys j and values j - 1 no longer read: their successors load.
    auto stage = [&](int j) {
      uint64_t more[LOADS];
      rows_of(j + 2, more);
      landed<0>();
      reads_done();
      asm volatile("s_barrier" ::: "memory");
      if (j + 1 < cnt) load_values(j + 1, off);
      if (j + 2 < cnt) load_keys(j + 2, more);
#pragma unroll
      for (int i = 0; i < LOADS; ++i) off[i] = more[i];
      publish(j + 3, next_rows);
      next_rows = find(j + 4);
    };
    // (three workgroups a CU with heads of 64, which leaves registers for two operands ahead and spills three: window 64
    // 32 -> 28 us, 1024 101 -> 98 us; eight ahead with heads of 256 were level; PS pairs of the 16 beside
    // the scores)
    constexpr int AHEAD = DP == 64 ? 2 : 4, NS = 2 * NQ, NP = 4 * ND, PS = 12;
    static_assert(NS % AHEAD == 0 && NP >= AHEAD, "operand ring");
    // a block that is not the last one: its probabilities and product, and the scores of the next
    auto block = [&](int j, auto ODD, Scores& now, Scores& next) {
      constexpr int odd = decltype(ODD)::value;
      stage(j);
      if (masked(j)) clean(j, odd);
      half8v f[AHEAD];
#pragma unroll
      for (int x = 0; x < AHEAD; ++x) f[x] = k_operand(odd ^ 1, x % 2, x / 2);
      static_for(std::make_integer_sequence<int, NS>{}, [&](auto X) {
        constexpr int x = decltype(X)::value;
        score_step(f[x % AHEAD], next, x % 2, x / 2);
        if constexpr (x + AHEAD < NS) f[x % AHEAD] = k_operand(odd ^ 1, (x + AHEAD) % 2, (x + AHEAD) / 2);
        else f[x % AHEAD] = v_operand(odd, (x + AHEAD - NS) % ND, (x + AHEAD - NS) / ND);
#pragma unroll
        for (int y = x * PS / NS; y < (x + 1) * PS / NS; ++y) exp_pair(now, y);
      });
      float part = -INFINITY;
      static_for(std::make_integer_sequence<int, NP>{}, [&](auto X) {
        constexpr int x = decltype(X)::value, PX = 3 * ND;  // the last pairs before the keys that need them
        product_step(f[x % AHEAD], x % ND, x / ND);
        if constexpr (x + AHEAD < NP) f[x % AHEAD] = v_operand(odd, (x + AHEAD) % ND, (x + AHEAD) / ND);
        if constexpr (x < PX) {
#pragma unroll
          for (int y = PS + x * (16 - PS) / PX; y < PS + (x + 1) * (16 - PS) / PX; ++y) exp_pair(now, y);
        }
#pragma unroll
        for (int y = x * 32 / NP; y < (x + 1) * 32 / NP; ++y) part = fmaxf(part, next[y / 16][y % 16]);
        stay(part);
      });
      float top;
      if (!masked(j + 1)) top = both(part, larger) * c;
      else {
        hide(next, base_of(j + 1));
        top = largest(next);
      }
      raise(top);
    };

    landed<0>();
    reads_done();
    asm volatile("s_barrier" ::: "memory");
    publish(2, next_rows);
    next_rows = find(3);
    Scores sa, sb;
#pragma unroll
    for (int t = 0; t < NQ; ++t)
#pragma unroll
      for (int u = 0; u < 2; ++u) score_step(k_operand(0, u, t), sa, u, t);
    if (masked(0)) hide(sa, it.key0);
    raise(largest(sa));
    int j = 0;
    for (; j + 2 < cnt; j += 2) {
      block(j, std::integral_constant<int, 0>{}, sa, sb);
      block(j + 1, std::integral_constant<int, 1>{}, sb, sa);
    }
    if (j + 1 < cnt) {
      block(j, std::integral_constant<int, 0>{}, sa, sb);
      sa[0] = sb[0];
      sa[1] = sb[1];
      ++j;
    }
    // the last block
    landed<0>();
    reads_done();
    asm volatile("s_barrier" ::: "memory");
    const int odd = j & 1;
    if (masked(j)) clean(j, odd);
#pragma unroll
    for (int x = 0; x < 16; ++x) exp_pair(sa, x);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int d = 0; d < ND; ++d) product_step(v_operand(odd, d, k), d, k);
    if (cleaned_to) add_cleaned();
    l = both(l, [](float x, float y) { return x + y; });
  }

  // ---- results: lane holds places 32 d + 8 q + 4 half + i of its row
  const bool mine = it.row0 + wave * 32 + l32 < it.rows, none = m == -INFINITY && l == 0.f;  // (none: a row that saw nothing)
  const int64_t pair = (int64_t)(it.tok0 + query) * a.q_heads + it.kvh * G + (row - query * G);
  if (sp.slots) {
    const int64_t at = (int64_t)it.slot * a.T * a.q_heads + pair;
    if (!mine) return;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int d0 = 32 * d + 8 * q + 4 * half;
        if (FULL || d0 < D) *reinterpret_cast<float4v*>(sp.part_o + at * D + d0) = float4v{o[d][4 * q], o[d][4 * q + 1], o[d][4 * q + 2], o[d][4 * q + 3]};
      }
    if (half == 0) sp.part_ml[at] = make_float2(m, l);
    return;
  }
  // rounded, and through LDS so that rows leave whole, 16 bytes a lane
  __syncthreads();
  uint8_t* const tile = lds + wave * 32 * T::ROWB;
  const float inv = 1.f / l;
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      half4v h;
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = (_Float16)(none ? 0.f : o[d][4 * q + i] * inv);
      *reinterpret_cast<half4v*>(tile + l32 * T::ROWB + ((4 * d + q) ^ (l32 & (SL - 1))) * 16 + half * 8) = h;
    }
  if (a.lse && half == 0 && mine) a.lse[pair] = none ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
  reads_done();
  constexpr int ROWS = 64 / SL;  // rows of a store
#pragma unroll
  for (int i = 0; i < 32 / ROWS; ++i) {
    const int r = i * ROWS + lane / SL, cl = lane % SL;
    const uint4 w = *reinterpret_cast<const uint4*>(tile + r * T::ROWB + (cl ^ (r & (SL - 1))) * 16);
    const int64_t to = __shfl(pair, r, 64);
    if (it.row0 + wave * 32 + r < it.rows && (FULL || cl * 8 < D)) *reinterpret_cast<uint4*>(a.out + to * D + cl * 8) = w;
  }
}

template <int DP>
hipError_t launch_rows(const WindowArgs& a, const AttnSplit& p, hipStream_t st) {
  constexpr int lds = RowsGeo<DP>::LDS;
  static_assert(lds <= 160 * 1024, "LDS budget");
  const dim3 grid((unsigned)p.s_items);
  if (a.D == DP) hipLaunchKernelGGL((window_rows_kernel<DP, true>), grid, dim3(256), lds, st, a, p);
  else hipLaunchKernelGGL((window_rows_kernel<DP, false>), grid, dim3(256), lds, st, a, p);
  return hipGetLastError();
}

template <int DP>
hipError_t launch_dim(const WindowArgs& a, const AttnSplit& p, hipStream_t st) {
  if (p.kind_s == TILE_KEYS) return launch_kinds<DP, TILE_NONE, TILE_KEYS>(a, p, st);
  if (p.kind_s == TILE_ROWS64) return launch_kinds<DP, TILE_NONE, TILE_ROWS64>(a, p, st);
  return launch_rows<DP>(a, p, st);
}

}  // namespace

hipError_t launch_window_tiles(const WindowArgs& args, const AttnSplit& p, hipStream_t st) {
  WindowArgs a = args;
  a.per_head = a.q_heads / a.kv_heads;
  a.groups = p.s_items / p.s_tiles;
  a.by_per_head = Divide::by(a.per_head);
  a.by_groups = Divide::by(a.groups);
  a.by_kv_heads = Divide::by(a.kv_heads);
  a.by_splits = Divide::by(p.s_splits);
  return a.D <= 64 ? launch_dim<64>(a, p, st) : a.D <= 128 ? launch_dim<128>(a, p, st) : launch_dim<256>(a, p, st);
}

}  // namespace qg
