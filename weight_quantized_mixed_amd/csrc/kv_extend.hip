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
// totals through LDS), writes what there is one of per sequence, and gives pages back.  Then
// a token finds its sequence by bisection of the rows' starts, its page in the table (the
// last page held, which it may fill up) or in the ring, and the first token of a new page
// writes the table's entry.  Up to ONE_LAUNCH tokens the same workgroup does that, from LDS;
// more go to a second launch of many workgroups, which reads the sequences from the workspace.
//
// Sums saturate at 2^32 - 1 instead of wrapping, which is past every limit they are held
// against (tokens of the batch, pages of the pool), and saturated sums can be joined in any order.
#include "qgemm_internal.hpp"

namespace qg {
namespace {

constexpr int THREADS = 1024, WAVES = THREADS / 64;
constexpr int ONE_LAUNCH = 4096, ONE_LAUNCH_SEQUENCES = 2048;

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

// sum of v over the threads before this one, behind `carry`, which grows by all threads' sum
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t& carry, uint32_t* totals) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t upto = wave_scan(v);
  uint32_t before = __shfl_up(upto, 1, 64);
  if (lane == 0) before = 0;
  if (lane == 63) totals[wave] = upto;
  __syncthreads();
  uint32_t all = carry, mine = carry;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    if (w < wave) mine = add(mine, totals[w]);
    all = add(all, totals[w]);
  }
  __syncthreads();  // (the totals may be written again)
  carry = all;
  return add(mine, before);
}

// what a token asks of its sequence
struct Grown {
  int32_t start;  // first row
  int32_t len;    // tokens held before
  int32_t taken;  // pages that the sequences before take from the pool, or -1: refused
};

__device__ __forceinline__ int pages_of(int64_t tokens, int shift) { return (int)((tokens + (1 << shift) - 1) >> shift); }

// token t of the batch, in sequence b (or in none)
__device__ __forceinline__ void place_token(const ExtendArgs& a, int t, int b, Grown s, int head) {
  int pos = 0;
  int64_t slot = -1;
  if (b < a.B && s.taken < 0) pos = -1;
  if (b < a.B && s.taken >= 0) {
    const int j = s.len + (t - s.start), p = j >> a.page_shift, in_page = j & ((1 << a.page_shift) - 1);
    const int old = pages_of(s.len, a.page_shift);
    int32_t* entry = a.tables + (int64_t)b * a.table_width + p;
    int32_t page;
    if (p < old) page = *entry;
    else {
      int64_t at = (int64_t)head + s.taken + (p - old);
      page = a.ring[at < a.ring_size ? at : at - a.ring_size];
      if (in_page == 0) *entry = page;
    }
    pos = (int)a.prefix_len + j;
    slot = ((int64_t)page << a.page_shift) | in_page;
  }
  a.positions[t] = pos;
  a.slots[t] = slot;
}

// the last of n ascending starts that is at most t (n if there is none: n >= 1, start(0) is 0)
template <typename F>
__device__ __forceinline__ int sequence_of(int t, int n, F start) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start(mid) <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ALL: the tokens too
template <bool ALL>
__global__ __launch_bounds__(THREADS) void extend_kernel(ExtendArgs a) {
  __shared__ uint32_t totals[WAVES];
  __shared__ Grown grown[ALL ? ONE_LAUNCH_SEQUENCES : 1];
  const int lane = threadIdx.x & 63;
  const int R = a.ring_size;
  int head = a.ring_state[0], free = a.ring_state[1];
  // (a state that no call left is brought into range, so that nothing is touched outside the pool)
  head = head < 0 || head >= R ? 0 : head;
  free = min(max(free, 0), R);
  uint32_t rows = 0, wanted = 0, taken = 0, back = 0;
  for (int b0 = 0; b0 < a.B; b0 += THREADS) {
    const int b = b0 + threadIdx.x;
    const bool in = b < a.B;
    const int asked = in ? a.new_tokens[b] : 0, n = max(asked, 0);
    const int len = in ? max(a.lens[b], 0) : 0, gone = in && a.window ? max(a.gone[b], 0) : 0;
    const int old = pages_of(len, a.page_shift), now = pages_of((int64_t)len + n, a.page_shift);
    const uint32_t start = block_scan((uint32_t)n, rows, totals);
    // what no other sequence can help
    const bool fits = now <= a.table_width && a.prefix_len + len + n <= INT32_MAX && add(start, (uint32_t)n) <= (uint32_t)a.T;
    const uint32_t need = fits ? now - old : 0;
    const uint32_t before = block_scan(need, wanted, totals);
    const bool refused = n > 0 && (!fits || (need > 0 && add(before, need) > (uint32_t)free));
    // pages given back: [from0, to0) and [from1, to1), of those that the table has
    const int held = min((int64_t)old, a.table_width);
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
    const int n1 = max(to1 - from1, 0), given = to0 + n1;
    const uint32_t put = block_scan((uint32_t)given, back, totals);
    // the i-th page given back by a sequence; the pool never holds more than it has places
    auto give = [&](int of, uint32_t at, int i, int to0, int from1) {
      const int64_t place = (int64_t)free + at + i;
      if (place >= R) return;
      const int64_t x = head + place;
      a.ring[x < R ? x : x - R] = a.tables[(int64_t)of * a.table_width + (i < to0 ? i : from1 + i - to0)];
    };
    // a sequence's few pages by its own thread, many by the wave
    if (given > 0 && given <= 2)
      for (int i = 0; i < given; ++i) give(b, put, i, to0, from1);
    for (uint64_t many = __ballot(given > 2); many; many &= many - 1) {
      const int from = __builtin_ctzll(many);
      const int g = __shfl(given, from, 64), t0 = __shfl(to0, from, 64), f1 = __shfl(from1, from, 64);
      const uint32_t at = __shfl(put, from, 64);
      for (int i = lane; i < g; i += 64) give(b - lane + from, at, i, t0, f1);
    }
    if (in) {
      const int first = (int)min(start, (uint32_t)a.T);
      a.q_starts[b] = first;
      a.refused[b] = refused;
      a.lens_out[b] = asked < 0 ? 0 : refused ? len : len + n;
      a.gone_out[b] = gone_now;
      const Grown s = {first, len, refused ? -1 : (int)before};
      if constexpr (ALL) grown[b] = s;
      else reinterpret_cast<Grown*>(a.scratch)[b] = s;
    }
    // the pages of those that were not refused, who come first
    if (need > 0 && !refused) taken = max(taken, add(before, need));
  }
  // over the workgroup: the largest of `taken`
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) taken = max(taken, (uint32_t)__shfl_xor(taken, o, 64));
  if (lane == 0) totals[threadIdx.x >> 6] = taken;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < WAVES; ++w) taken = max(taken, totals[w]);
    const int64_t next = (int64_t)head + taken;
    a.q_starts[a.B] = (int)min(rows, (uint32_t)a.T);
    a.ring_state_out[0] = (int)(next < R ? next : next - R);
    a.ring_state_out[1] = (int)(min((int64_t)free + back, (int64_t)R) - taken);
    if constexpr (!ALL) reinterpret_cast<Grown*>(a.scratch)[a.B] = {(int)min(rows, (uint32_t)a.T), head, 0};
  }
  if constexpr (ALL) {
    const int end = (int)min(rows, (uint32_t)a.T);
    for (int t = threadIdx.x; t < a.T; t += THREADS) {
      int b = a.B;
      if (t < end) b = sequence_of(t, a.B, [&](int i) { return grown[i].start; });
      place_token(a, t, b, b < a.B ? grown[b] : Grown{0, 0, 0}, head);
    }
  }
}

__global__ __launch_bounds__(256) void place_tokens_kernel(ExtendArgs a) {
  const Grown* grown = reinterpret_cast<const Grown*>(a.scratch);
  const int end = grown[a.B].start, head = grown[a.B].len;
  const int t = (int)(blockIdx.x * 256 + threadIdx.x);
  if (t >= a.T) return;
  int b = a.B;
  if (t < end) b = sequence_of(t, a.B, [&](int i) { return grown[i].start; });
  place_token(a, t, b, b < a.B ? grown[b] : Grown{0, 0, 0}, head);
}

bool one_launch(int64_t B, int64_t T) { return T <= ONE_LAUNCH && B <= ONE_LAUNCH_SEQUENCES; }

}  // namespace

size_t extend_ws_bytes(int64_t B, int64_t T) {
  return one_launch(B, T) ? 0 : (size_t)(B + 1) * sizeof(Grown);
}

hipError_t launch_kv_extend(const ExtendArgs& a, hipStream_t st) {
  if (one_launch(a.B, a.T)) {
    hipLaunchKernelGGL(extend_kernel<true>, dim3(1), dim3(THREADS), 0, st, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(extend_kernel<false>, dim3(1), dim3(THREADS), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.T == 0) return e;
  hipLaunchKernelGGL(place_tokens_kernel, dim3((unsigned)(((int64_t)a.T + 255) / 256)), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace qg
