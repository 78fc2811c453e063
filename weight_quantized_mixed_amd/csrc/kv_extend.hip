// Block tables and slot maps of a batch's new tokens, from its request lengths.
//
// With L own tokens in the cache and n new ones, a sequence grows from old = ceil(L / page)
// to ceil((L + n) / page) pages.  Three sums over the sequences place everything: of the new
// tokens (the rows of the batch), of the pages wanted (which page of the pool a new one is)
// and of the pages given back (where in the pool they go).  The pool is a ring, so that no
// list is moved: pages are taken from its head and put behind its last one, and a page given
// back by a call is taken by a later call.
//
// One workgroup takes the sums, 1024 sequences at a time (DPP scans of a wave, the waves'
// totals through LDS), and writes what there is one of per sequence.  Then a token finds its
// sequence by bisection of the rows' starts, its page in the table (the last page held, which
// it may fill up) or in the ring, and the first token of a new page writes the table's entry;
// a page given back finds its sequence and its place in the table the same way, a thread each.
// For few tokens the same workgroup does that, from LDS (one_launch); more go to a second launch of
// many workgroups, which reads the sequences from the workspace.
//
// Measured: 1 sequence 3.7 us, 48 sequences of up to 8000 tokens 4.8 us (a launch with nothing in it
// about 2.5); 24 sequences of 8400 tokens 3.7 + 3.4 us, 1500 of 30000 tokens 5.8 + 5.1 us.  Nothing but
// latency bounds it: the sums wait for two barriers a thousand sequences, a token for the reads of
// its bisection, which lie one behind the other.
//
// Sums saturate at 2^32 - 1 instead of wrapping, which is past every limit they are held
// against (tokens of the batch, pages of the pool), and saturated sums can be joined in any order.
#include "qgemm_internal.hpp"

namespace qg {
namespace {

constexpr int THREADS = 1024, WAVES = THREADS / 64;
constexpr int ONE_LAUNCH_SEQUENCES = 2048;

__device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) { return __builtin_elementwise_add_sat(a, b); }

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t add_from(uint32_t v) {
  return add(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, true));
}

// sum of v over lanes 0 .. this one
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v = add_from<0x111, 0xF>(v);  // from 1, 2, 4 and 8 lanes before, within rows of 16
  v = add_from<0x112, 0xF>(v);
  v = add_from<0x114, 0xF>(v);
  v = add_from<0x118, 0xF>(v);
  v = add_from<0x142, 0xA>(v);  // row 0's last lane into row 1, row 2's into row 3
  return add_from<0x143, 0xC>(v);  // row 1's last lane into rows 2 and 3
}

// Sums of N values over the threads before this one, each behind its `carry`, which grows by
// all threads' sum.
template <int N>
__device__ __forceinline__ void block_scan(uint32_t (&v)[N], uint32_t (&carry)[N], uint32_t (*totals)[WAVES]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t before[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t upto = wave_scan(v[i]);
    before[i] = __shfl_up(upto, 1, 64);
    if (lane == 0) before[i] = 0;
    if (lane == 63) totals[i][wave] = upto;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t all = carry[i], mine = carry[i];
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      if (w < wave) mine = add(mine, totals[i][w]);
      all = add(all, totals[i][w]);
    }
    carry[i] = all;
    v[i] = add(mine, before[i]);
  }
  __syncthreads();  // (the totals may be written again)
}

// What the second part asks of a sequence: where its rows and the pages that it gives back
// begin among all, and the rest.
struct Rest {
  int32_t len;    // tokens held before
  int32_t taken;  // pages that the sequences before take from the pool, or -1: refused
  // pages given back, as their places in its table: [0, to0), then from1 on
  int32_t to0, from1;
};
struct Steps {
  Rest* rest;
  uint32_t *starts, *puts;
};
// totals of a call, and the ring as it was found
struct Totals {
  int32_t rows, back, head, free;
};

__device__ __forceinline__ int pages_of(int64_t tokens, int shift) { return (int)((tokens + (1 << shift) - 1) >> shift); }

// the last of n ascending starts that is at most x (n >= 1, start(0) is 0)
__device__ __forceinline__ int sequence_of(uint32_t x, int n, const uint32_t* starts) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// token t of the batch, of sequence b (s) that begins in row start
__device__ __forceinline__ void place_token(const ExtendArgs& a, int t, int b, int start, const Rest& s, int head) {
  int pos = -1;
  int64_t slot = -1;
  if (s.taken >= 0) {
    const int j = s.len + (t - start), p = j >> a.page_shift, in_page = j & ((1 << a.page_shift) - 1);
    const int old = pages_of(s.len, a.page_shift);
    int32_t* entry = a.tables + (int64_t)b * a.table_width + p;
    int32_t page;
    if (p < old) page = *entry;
    else {
      const int64_t at = (int64_t)head + s.taken + (p - old);
      page = a.ring[at < a.ring_size ? at : at - a.ring_size];
      if (in_page == 0) *entry = page;
    }
    pos = (int)a.prefix_len + j;
    slot = ((int64_t)page << a.page_shift) | in_page;
  }
  a.positions[t] = pos;
  a.slots[t] = slot;
}

// the i-th page given back, the nth of sequence b; the pool never holds more than it has places
__device__ __forceinline__ void give_back(const ExtendArgs& a, uint32_t i, int b, uint32_t nth, const Rest& s, const Totals& t) {
  const int64_t place = (int64_t)t.free + i, x = (int64_t)t.head + place;
  if (place < a.ring_size)
    a.ring[x < a.ring_size ? x : x - a.ring_size] =
        a.tables[(int64_t)b * a.table_width + ((int)nth < s.to0 ? nth : s.from1 + (int)nth - s.to0)];
}

// The sums, and what there is one of per sequence.  ALL: tokens and pages given back too.
template <bool ALL>
__global__ __launch_bounds__(THREADS) void extend_kernel(ExtendArgs a, Steps steps, Totals* end) {
  constexpr int HELD = ALL ? ONE_LAUNCH_SEQUENCES : 1;
  __shared__ uint32_t totals[2][WAVES];
  __shared__ Rest held_rest[HELD];
  __shared__ uint32_t held_starts[HELD], held_puts[HELD];
  if constexpr (ALL) steps = {held_rest, held_starts, held_puts};
  const int lane = threadIdx.x & 63, R = a.ring_size;
  int head = a.ring_state[0], free = a.ring_state[1];
  // (a state that no call left is brought into range, so that nothing is touched outside the pool)
  head = head < 0 || head >= R ? 0 : head;
  free = min(max(free, 0), R);
  uint32_t sums[2] = {0, 0}, wanted[1] = {0}, taken = 0;  // rows and pages given back; pages asked for
  for (int b0 = 0; b0 < a.B; b0 += THREADS) {
    const int b = b0 + threadIdx.x;
    const bool in = b < a.B;
    const int asked = in ? a.new_tokens[b] : 0, n = max(asked, 0);
    const int len = in ? max(a.lens[b], 0) : 0, gone = in && a.window ? max(a.gone[b], 0) : 0;
    const int old = pages_of(len, a.page_shift), now = pages_of((int64_t)len + n, a.page_shift);
    // what goes back, of the pages that the table has
    const int held = (int)min((int64_t)old, a.table_width);
    int to0 = 0, from1 = 0, to1 = 0, gone_now = 0;
    if (asked < 0) {
      to0 = gone > a.first_page ? min(a.first_page, held) : 0;
      from1 = gone > a.first_page ? gone : 0;
      to1 = held;
    } else if (a.window) {
      const int past = (int)(max((int64_t)len - a.window + 1, (int64_t)0) >> a.page_shift);
      from1 = max(a.first_page, gone);
      to1 = min(past, held);
      gone_now = past > a.first_page ? max(gone, past) : gone;
    }
    uint32_t first[2] = {(uint32_t)n, (uint32_t)(to0 + max(to1 - from1, 0))};
    block_scan(first, sums, totals);
    // what no other sequence can help
    const uint32_t start = first[0];
    const bool fits = now <= a.table_width && a.prefix_len + len + n <= INT32_MAX && add(start, (uint32_t)n) <= (uint32_t)a.T;
    const uint32_t need = fits ? now - old : 0;
    uint32_t before[1] = {need};
    block_scan(before, wanted, totals);
    const bool refused = n > 0 && (!fits || (need > 0 && add(before[0], need) > (uint32_t)free));
    if (in) {
      const uint32_t row = min(start, (uint32_t)a.T);
      a.q_starts[b] = (int)row;
      a.refused[b] = refused;
      a.lens_out[b] = asked < 0 ? 0 : refused ? len : len + n;
      a.gone_out[b] = gone_now;
      steps.starts[b] = row;
      steps.puts[b] = first[1];
      steps.rest[b] = {len, refused ? -1 : (int)before[0], to0, from1};
    }
    // those that were not refused come first
    if (need > 0 && !refused) taken = max(taken, add(before[0], need));
  }
  // over the workgroup: the largest of `taken`
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) taken = max(taken, (uint32_t)__shfl_xor(taken, o, 64));
  if (lane == 0) totals[0][threadIdx.x >> 6] = taken;
  __syncthreads();
  const Totals t = {(int)min(sums[0], (uint32_t)a.T), (int)min(sums[1], (uint32_t)R), head, free};
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < WAVES; ++w) taken = max(taken, totals[0][w]);
    const int64_t next = (int64_t)head + taken;
    a.q_starts[a.B] = t.rows;
    a.ring_state_out[0] = (int)(next < R ? next : next - R);
    a.ring_state_out[1] = (int)(min((int64_t)free + t.back, (int64_t)R) - taken);
    if constexpr (!ALL) *end = t;
  }
  if constexpr (ALL) {
    for (int i = threadIdx.x; i < a.T; i += THREADS) {
      if (i < t.rows) {
        const int b = sequence_of(i, a.B, held_starts);
        place_token(a, i, b, held_starts[b], held_rest[b], head);
      } else {
        a.positions[i] = 0;
        a.slots[i] = -1;
      }
    }
    for (int i = threadIdx.x; i < t.back; i += THREADS) {
      const int b = sequence_of(i, a.B, held_puts);
      give_back(a, i, b, i - held_puts[b], held_rest[b], t);
    }
  }
}

// Tokens, and pages given back, of many: the first GIVING workgroups take the pages, the others
// a token a thread.  Up to STAGED sequences their starts are bisected in LDS (1500 sequences:
// with 11 reads from the L2 one behind the other the tokens alone took 5.2 us).
constexpr int GIVING = 32, STAGED = 4096;
__global__ __launch_bounds__(256) void place_kernel(ExtendArgs a, Steps steps, const Totals* end) {
  __shared__ uint32_t held[STAGED];
  const Totals t = *end;
  const bool giving = blockIdx.x < GIVING;
  const uint32_t* starts = giving ? steps.puts : steps.starts;
  const int64_t i0 = (int64_t)(giving ? blockIdx.x : blockIdx.x - GIVING) * 256, i = i0 + threadIdx.x;
  if (a.B <= STAGED && i0 < (giving ? t.back : t.rows)) {
    for (int b = threadIdx.x; b < a.B; b += 256) held[b] = starts[b];
    __syncthreads();
    starts = held;
  }
  if (giving) {
    for (int64_t k = i; k < t.back; k += GIVING * 256) {
      const int b = sequence_of((uint32_t)k, a.B, starts);
      give_back(a, (uint32_t)k, b, (uint32_t)k - starts[b], steps.rest[b], t);
    }
  } else if (i < t.rows) {
    const int b = sequence_of((uint32_t)i, a.B, starts);
    place_token(a, (int)i, b, starts[b], steps.rest[b], t.head);
  } else if (i < a.T) {
    a.positions[i] = 0;
    a.slots[i] = -1;
  }
}

// One workgroup takes 0.24 us for a thousand tokens and 0.08 more for each step of the bisection, a second
// launch 4.5 in all: 24 sequences of 4800 tokens 7.9 us as one and 10.4 as two, of 19200 16.8 and 10.7;
// 300 sequences of 9300 tokens 14.9 and 10.7.
// The rule leaves out what comes back, which the host does not know: that takes one workgroup as long as as many tokens,
// and the second launch 0.14 us a thousand pages.  In the long run as many come back as are taken, one a sequence in
// page_size steps, for which the launch does not pay (2048 sequences of 8000 tokens, one more each: 8.8 us as one, 2049 of
// them 13.0 as two); in a step in which very many end it would (pages of 16, one of fifty ending: 29.5 and 15.1 us, one of
// two, 512000 pages: 570 and 84).
bool one_launch(int64_t B, int64_t T) {
  int steps = 0;
  while (((int64_t)1 << steps) < B) ++steps;
  return B <= ONE_LAUNCH_SEQUENCES && T * (3 + steps) <= 57600;
}

}  // namespace

size_t extend_ws_bytes(int64_t B, int64_t T) {
  return one_launch(B, T) ? 0 : sizeof(Totals) + (size_t)B * (sizeof(Rest) + 2 * sizeof(uint32_t));
}

hipError_t launch_kv_extend(const ExtendArgs& a, hipStream_t st) {
  if (one_launch(a.B, a.T)) {
    hipLaunchKernelGGL(extend_kernel<true>, dim3(1), dim3(THREADS), 0, st, a, Steps{}, nullptr);
    return hipGetLastError();
  }
  Totals* end = static_cast<Totals*>(a.scratch);
  Steps steps;
  steps.rest = reinterpret_cast<Rest*>(end + 1);
  steps.starts = reinterpret_cast<uint32_t*>(steps.rest + a.B);
  steps.puts = steps.starts + a.B;
  hipLaunchKernelGGL(extend_kernel<false>, dim3(1), dim3(THREADS), 0, st, a, steps, end);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(place_kernel, dim3((unsigned)(GIVING + ((int64_t)a.T + 255) / 256)), dim3(256), 0, st, a, steps, end);
  return hipGetLastError();
}

}  // namespace qg
