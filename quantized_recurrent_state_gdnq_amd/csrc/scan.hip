// Gated linear recurrence over channels, h_t = a_t h_{t-1} + b_t (see
// gdnq_scan_* in gdnq.h): forward with the states for the backward pass, the
// backward pass, and the single-token step.
//
// Forward and backward are one pass over the tokens each.  The tokens of the
// whole call (all sequences, back to back) are cut into chunks, and a
// workgroup takes one chunk of 64 or 128 channels: lanes hold channels, waves
// hold runs of 8 to 32 tokens, whose inputs stay in registers.
//   1. Each wave folds its run to the pair (A, H) with h_out = A h_in + H.  A
//      sequence's first token has A = 0 (its state comes from h0), so runs,
//      waves and chunks may hold any number of sequence borders.
//   2. The waves' pairs go through LDS to the chunk's pair, which is published
//      in the workspace.  Every 16th chunk publishes the pair of its group of 16
//      chunks as well, every 256th its outgoing state, so the state that enters
//      a chunk is folded from at most one state, 15 groups and 15 chunks, back
//      to the chunk that holds its first token's sequence start.  Handing a
//      state on costs about 3 us; with a state per group instead of two levels
//      of pairs those hops bounded long sequences.  The fold's order is fixed
//      by the sizes alone.
//   3. Every wave walks its run again from the state it now knows and writes.
// Waiting: chunks are taken by ticket (a counter per channel tile), so the
// chunk before the one a workgroup waits for is always held by a workgroup
// that runs already and, by induction over the tickets, ends: no order of
// dispatch is assumed.  A published pair carries its own mark (the workspace
// starts as all ones, which no published pair has), so a single relaxed
// 8-byte atomic is the whole hand-over.
//
// Bound by memory in fp32: 262144 x 640 forward 365 us, 5.6 TB/s; 65536 x 1024
// backward 222, 6.0 TB/s.  In bf16 the vector instructions weigh as much: 32768
// x 2048 forward 98 us a call with given gates (4.1 TB/s), 109 with logits (the
// kernel 104 of it, 115 to 117 under the profiler); 65536 x 2048 backward with
// given gates 258 (5.2 TB/s); 32768 x 5120 with logits, 48 sequences: forward
// 236, backward 370 (4.4 and 4.7 TB/s).  An odd number of channels takes one a
// lane: 65536 x 1023 forward 142, backward 196 (2.8 and 3.4 TB/s).  All but the
// calls' by the profiler's medians.
#include <hip/hip_runtime.h>

#include "../../include/gdnq.h"
#include "device_common.h"
#include "launch.h"
#include "vec_io.h"

namespace gdnq {
namespace {

// Waves of a workgroup, tokens per wave and waves per SIMD (by the registers)
// for V channels per lane.  Two channels of bf16 and their gates take two
// registers and a half per token, so half as many waves hold twice the tokens:
// 98 us for 32768 tokens of 2048 channels with given gates, 114 with 8 waves of
// 16 tokens; the shape of one channel spills.  One channel of fp32: 377 us for
// 262144 tokens of 640 channels, 413 with 8 waves of 32 tokens.
template <int V>
struct ForwardShape {
  static constexpr int WAVES = V == 1 ? 16 : 8, RUN = V == 1 ? 16 : 32, PER_SIMD = V == 1 ? 8 : 4;
};
constexpr int FWD_CHUNK = 256;
// The backward pass holds three values and a state per token.
constexpr int BWD_WAVES = 16, BWD_RUN = 8, BWD_PER_SIMD = 8, BWD_CHUNK = BWD_WAVES * BWD_RUN;
constexpr int GROUP = 16;  // chunks per published group, groups per published state
static_assert(BWD_CHUNK == GDNQ_SCAN_CHUNK && FWD_CHUNK % GDNQ_SCAN_CHUNK == 0, "carry rows are chunk borders");

// Words between the tiles' ticket counters: a cache line of their own each.
constexpr int TICKET_STRIDE = 64;

constexpr unsigned long long EMPTY = ~0ull;

// The chain of chunks in the workspace: a ticket counter per channel tile, then
// per channel a pair per chunk, a pair per group and a state per GROUP groups.
struct Chain {
  uint32_t* ticket;  // null: the call is one chunk
  unsigned long long* pair;
  unsigned long long* group;
  unsigned long long* state;
};

// V channels of one token: in memory, and as the registers that hold them.
template <typename E, int V>
struct Cell;
template <>
struct Cell<bf16, 2> {
  uint32_t w;
  __device__ __forceinline__ void load(const bf16* p) { w = *reinterpret_cast<const uint32_t*>(p); }
  __device__ __forceinline__ float get(int i) const { return i ? bf16_hi(w) : bf16_lo(w); }
  // Between walks: the compiler would keep both values apart, in two registers.
  __device__ __forceinline__ void forget() { asm volatile("" : "+v"(w)); }
  __device__ static __forceinline__ void store(bf16* p, const float (&v)[2]) {
    *reinterpret_cast<bf16x2*>(p) = __builtin_convertvector(f32x2{v[0], v[1]}, bf16x2);
  }
};
template <typename E>
struct Cell<E, 1> {
  E w;
  __device__ __forceinline__ void load(const E* p) { w = *p; }
  __device__ __forceinline__ float get(int) const { return to_f32(w); }
  __device__ __forceinline__ void forget() {}
  __device__ static __forceinline__ void store(E* p, const float (&v)[1]) { store_f32(p, v[0]); }
};

// V gates of one token: a = gate or sigmoid(gate) and keep = 1 - a, from what
// they were loaded as (load, then settle once).  From logits one value is
// kept in fp32, the smaller of a and keep with the logit's sign, and the other
// is one minus it: the exponential and the reciprocal are taken once however
// many times a token is walked over (they, not the memory, bounded the
// kernels that took them in every walk).
template <typename E, int V, bool LOGITS>
struct Gates;
template <typename E, int V>
struct Gates<E, V, false> {
  Cell<E, V> g;
  __device__ __forceinline__ void load(const E* p) { g.load(p); }
  __device__ __forceinline__ void settle() {}
  __device__ __forceinline__ void forget() {}
  __device__ __forceinline__ void get(int i, float& a, float& keep) const {
    a = g.get(i);
    keep = 1.0f - a;
  }
};
template <typename E, int V>
struct Gates<E, V, true> {
  Cell<E, V> g;
  float t[V];
  __device__ __forceinline__ void load(const E* p) { g.load(p); }
  __device__ __forceinline__ void settle() {
#pragma unroll
    for (int i = 0; i < V; ++i) t[i] = sigmoid_tail<E>(g.get(i));
  }
  __device__ __forceinline__ void get(int i, float& a, float& keep) const { sigmoid_of_tail(t[i], a, keep); }
  // Between walks: the compiler would keep a and b of every token from the
  // first one in registers, four values instead of two, and spill them.
  __device__ __forceinline__ void forget() {
#pragma unroll
    for (int i = 0; i < V; ++i) asm volatile("" : "+v"(t[i]));
  }
};

// What a wave needs to know of the run of tokens from row0 on: bit r of the
// masks is token row0 + r; lane r holds its sequence.
struct Rows {
  uint32_t valid, start, end;
  int seq;
  __device__ __forceinline__ int seq_of(int r) const { return __builtin_amdgcn_readlane(seq, r); }
  // All of them in the middle of one sequence.
  template <int RUN>
  __device__ __forceinline__ bool plain() const {
    return valid == uint32_t((uint64_t(1) << RUN) - 1) && (start | end) == 0;
  }
};

// f(Plain or Mixed): most runs are plain, and their walks need no question per
// token, whose branches cost as much as the arithmetic (32768 x 2048 bf16: 98
// us, 114 with them).  With gates from logits the two kinds of walk together
// keep more values in registers than there are, and spill (156 us against
// 112), so there all are Mixed.
struct Plain {
  static constexpr bool value = true;
};
struct Mixed {
  static constexpr bool value = false;
};
template <bool LOGITS, typename F>
__device__ __forceinline__ void by_kind(bool plain, F&& f) {
  if constexpr (!LOGITS) {
    if (plain) return f(Plain{});
  }
  f(Mixed{});
}

// The last offset that is <= row among cu[0..B] (-1: none).
__device__ __forceinline__ int sequence_at(const int32_t* cu, int B, int row) {
  int lo = 0, hi = B + 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= row) lo = mid + 1;
    else hi = mid;
  }
  return lo - 1;
}

// first: the first token of the sequence that holds row0 (row0 + 1 if none does).
template <int RUN>
__device__ __forceinline__ Rows rows_of(const int32_t* __restrict__ cu, int B, int T, int64_t N, int row0, int lane,
                                        int& first) {
  const int row = row0 + lane;
  bool valid = lane < RUN && row < N, start, end;
  Rows w;
  if (cu) {
    const int s0 = sequence_at(cu, B, row0);
    int s = s0;
    start = s >= 0 && cu[max(s, 0)] == row;
    end = false;
    for (int j = s0 + 1; j <= B; ++j) {
      const int c = cu[j];
      if (c > row0 + RUN) break;
      if (c <= row) {
        s = j;
        start = c == row;
      }
      end |= c == row + 1;
    }
    valid &= s >= 0 && s < B;
    w.seq = s;
    first = s0 >= 0 && s0 < B ? max(cu[max(s0, 0)], 0) : row0 + 1;
  } else {
    const uint32_t s = uint32_t(row) / uint32_t(T), t = uint32_t(row) - s * uint32_t(T);
    w.seq = int(s);
    start = t == 0;
    end = t + 1 == uint32_t(T);
    first = row0 < N ? int(uint32_t(row0) / uint32_t(T) * uint32_t(T)) : row0 + 1;
  }
  w.valid = uint32_t(__builtin_amdgcn_ballot_w64(valid));
  w.start = uint32_t(__builtin_amdgcn_ballot_w64(valid && start));
  w.end = uint32_t(__builtin_amdgcn_ballot_w64(valid && end));
  return w;
}

__device__ __forceinline__ unsigned long long pack_pair(float a, float h) {
  uint32_t lo = __float_as_uint(a);
  if (lo == 0xffffffffu) lo = 0x7fc00000u;  // another NaN: the mark stays free
  return (static_cast<unsigned long long>(__float_as_uint(h)) << 32) | lo;
}

template <int V>
__device__ __forceinline__ void publish(unsigned long long* p, const float (&a)[V], const float (&h)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i)
    __hip_atomic_store(p + i, pack_pair(a[i], h[i]), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <int V>
__device__ __forceinline__ void await(const unsigned long long* p, float (&a)[V], float (&h)[V]) {
  unsigned long long w[V];
  for (;;) {
    bool there = true;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      w[i] = __hip_atomic_load(p + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      there &= w[i] != EMPTY;
    }
    if (there) break;
    __builtin_amdgcn_s_sleep(1);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    a[i] = __uint_as_float(uint32_t(w[i]));
    h[i] = __uint_as_float(uint32_t(w[i] >> 32));
  }
}

// A tile of LDS: a pair per wave (or chunk of the group) and channel.
template <int V>
__device__ __forceinline__ void put(f32x2* p, const float (&a)[V], const float (&h)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) p[i] = f32x2{a[i], h[i]};
}

// (a, h) := the pair (pa, ph) after (a, h).  Behind a border (cut) neither
// enters: the pair is the border's own, (0, ph).  As products with its zero a
// NaN or an infinity of one sequence would reach the next one.
__device__ __forceinline__ void join(float pa, float ph, bool cut, float& a, float& h) {
  h = cut ? ph : fmaf(pa, h, ph);
  a = cut ? 0.0f : a * pa;
}

// The same with the pair of every channel at p.
template <int V>
__device__ __forceinline__ void then(const f32x2* p, bool cut, float (&a)[V], float (&h)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) join(p[i].x, p[i].y, cut, a[i], h[i]);
}

// Which waves of the workgroup have a border in their run (bit per wave).
template <int WAVES>
__device__ __forceinline__ uint32_t waves_with(const uint32_t* borders, int lane) {
  return uint32_t(__builtin_amdgcn_ballot_w64(lane < WAVES && borders[lane & (WAVES - 1)] != 0));
}

// What a chunk's fold needs, in LDS.
template <int V>
struct Fold {
  f32x2 pair[GROUP][64 * V], group[GROUP][64 * V];
  float carry[64 * V];   // the states that enter the chunk
  f32x2 so_far[64 * V];  // the pair of the group's chunks before this one
};

// The states that enter a chunk, by all waves of its workgroup: place is the
// chunk's place in the order of the chain, from the first place whose pair it
// needs (place itself: none).  Ends with a barrier.
template <int V, int WAVES>
__device__ __forceinline__ void enter_chunk(const Chain& chain, int place, int from, int C, int c, bool active, int wave,
                                            int lane, Fold<V>& f) {
  const int border = place / GROUP * GROUP, group = place / GROUP, outer = group / GROUP * GROUP;
  const bool base = from < outer * GROUP;
  const int lo = max(from, border), glo = from >= border ? group : base ? outer : from / GROUP;
  // a wave takes one of each: all of its loads are under way together
#pragma unroll
  for (int k = 0; k < GROUP; k += WAVES) {
    const bool p = active && lo + k + wave < place, g = active && glo + k + wave < group;
    float a[V], h[V];
    if (g) {
      await<V>(chain.group + int64_t(glo + k + wave) * C + c, a, h);
      put<V>(&f.group[k + wave][lane * V], a, h);
    }
    if (p) {
      await<V>(chain.pair + int64_t(lo + k + wave) * C + c, a, h);
      put<V>(&f.pair[k + wave][lane * V], a, h);
    }
  }
  if (wave == WAVES - 1 && active) {  // (never a pair to wait for where WAVES = GROUP)
    float a[V], h[V] = {};
    if (base) await<V>(chain.state + int64_t(outer / GROUP - 1) * C + c, a, h);
#pragma unroll
    for (int i = 0; i < V; ++i) f.carry[lane * V + i] = h[i];
  }
  __syncthreads();
  if (wave == 0 && active) {
    float a[V], h[V], ga[V] = {}, gh[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      a[i] = 1.0f;
      h[i] = 0.0f;
      gh[i] = f.carry[lane * V + i];
    }
    for (int j = glo; j < group; ++j) then<V>(&f.group[j - glo][lane * V], false, ga, gh);
    for (int j = lo; j < place; ++j) then<V>(&f.pair[j - lo][lane * V], false, a, h);
    put<V>(&f.so_far[lane * V], a, h);
#pragma unroll
    for (int i = 0; i < V; ++i) f.carry[lane * V + i] = fmaf(a[i], gh[i], h[i]);
  }
  __syncthreads();
}

// After enter_chunk, by one wave: the chunk's own pair (a, h), with or without
// a border (cut) in it, to its group's pair and outgoing state, where due.
template <int V>
__device__ __forceinline__ void leave_chunk(const Chain& chain, int place, int C, int c, int lane, bool cut, const float (&a)[V],
                                            const float (&h)[V], const Fold<V>& f) {
  if (place % GROUP != GROUP - 1) return;
  float ga[V], gh[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    ga[i] = f.so_far[lane * V + i].x;
    gh[i] = f.so_far[lane * V + i].y;
    join(a[i], h[i], cut, ga[i], gh[i]);
  }
  publish<V>(chain.group + int64_t(place / GROUP) * C + c, ga, gh);
  if (place % (GROUP * GROUP) != GROUP * GROUP - 1) return;
#pragma unroll
  for (int i = 0; i < V; ++i) gh[i] = cut ? h[i] : fmaf(a[i], f.carry[lane * V + i], h[i]);
  publish<V>(chain.state + int64_t(place / (GROUP * GROUP)) * C + c, ga, gh);
}

template <int V>
__device__ __forceinline__ void add_h0(const float* h0, int seq, int C, int c, const float (&a)[V], float (&b)[V]) {
  if (!h0) return;
#pragma unroll
  for (int i = 0; i < V; ++i) b[i] = fmaf(a[i], h0[int64_t(seq) * C + c + i], b[i]);
}

__device__ __forceinline__ int take_ticket(uint32_t* ticket) {
  __shared__ int mine;
  if (threadIdx.x == 0)
    mine = int(__hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(mine);
}

template <typename E, int V, bool LOGITS, bool LERP>
__global__ __launch_bounds__(ForwardShape<V>::WAVES * 64, ForwardShape<V>::PER_SIMD) void scan_forward_kernel(ScanLaunch L, Chain chain, const int32_t* __restrict__ cu,
                                                                      const E* __restrict__ xs, const E* __restrict__ gates, int tiles) {
  constexpr int WAVES = ForwardShape<V>::WAVES, RUN = ForwardShape<V>::RUN, CT = 64 * V;
  static_assert(WAVES * RUN == FWD_CHUNK, "a chunk is the workgroup's runs");
  __shared__ f32x2 wave_pair[WAVES][CT];
  __shared__ Fold<V> fold;
  __shared__ uint32_t borders[WAVES];
  __shared__ int first_row;
  const int tile = blockIdx.x % tiles;
  const int chunk = chain.ticket ? take_ticket(chain.ticket + tile * TICKET_STRIDE) : 0;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int c = tile * CT + lane * V, C = L.C;
  const bool active = c < C;
  const int row0 = chunk * FWD_CHUNK + wave * RUN;

  Cell<E, V> x[RUN];
  Gates<E, V, LOGITS> g[RUN];
  const int cl = active ? c : 0, last = int(L.N) - 1;
#pragma unroll
  for (int r = 0; r < RUN; ++r) {
    // Lanes differ in the channel alone.  Plain walks wait for one token's loads
    // at a time, if no branch parts them: beyond the end these read the last
    // token.  Under a branch they are issued a token at a time, which Mixed
    // walks take better (prefill with logits 113 us, 119 without the branch).
    if (LOGITS && row0 + r > last) continue;
    const int64_t at = int64_t(min(row0 + r, last)) * C;
    x[r].load(xs + at + cl);
    g[r].load(gates + at + cl);
  }
  int first;
  const Rows rows = rows_of<RUN>(cu, L.B, L.T, L.N, row0, lane, first);
  if (threadIdx.x == 0) first_row = first;

  float A[V], H[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    A[i] = 1.0f;
    H[i] = 0.0f;
  }
  // a and b of token r of the run
  auto input = [&](int r, float (&a)[V], float (&b)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float keep;
      g[r].get(i, a[i], keep);
      b[i] = LERP ? keep * x[r].get(i) : x[r].get(i);
    }
  };
  auto fold_run = [&](auto PLAIN) {
#pragma unroll
    for (int r = 0; r < RUN; ++r) {
      if (!PLAIN.value && !(rows.valid >> r & 1)) continue;
      float a[V], b[V];
      g[r].settle();
      input(r, a, b);
      if (!PLAIN.value && (rows.start >> r & 1)) {
        if (active) add_h0<V>(L.h0, rows.seq_of(r), C, c, a, b);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          A[i] = 0.0f;
          H[i] = b[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          H[i] = fmaf(a[i], H[i], b[i]);
          A[i] *= a[i];
        }
      }
    }
  };
  by_kind<LOGITS>(rows.template plain<RUN>(), fold_run);
  put<V>(&wave_pair[wave][lane * V], A, H);
  if (lane == 0) borders[wave] = rows.start;
  __syncthreads();

  // the pair of the waves before this one
  const uint32_t cuts = waves_with<WAVES>(borders, lane);
  float pa[V], ph[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    pa[i] = 1.0f;
    ph[i] = 0.0f;
  }
  for (int w = 0; w < wave; ++w) then<V>(&wave_pair[w][lane * V], cuts >> w & 1, pa, ph);
  float in[V] = {};
  if (chain.ticket) {
    if (wave == WAVES - 1) {  // the chunk's pair
#pragma unroll
      for (int i = 0; i < V; ++i) {
        H[i] = rows.start ? H[i] : fmaf(A[i], ph[i], H[i]);
        A[i] = cuts ? 0.0f : A[i] * pa[i];
      }
      if (active) publish<V>(chain.pair + int64_t(chunk) * C + c, A, H);
    }
    const int start = first_row;
    const int from = start >= chunk * FWD_CHUNK ? chunk : start / FWD_CHUNK;
    enter_chunk<V, WAVES>(chain, chunk, from, C, c, active, wave, lane, fold);
#pragma unroll
    for (int i = 0; i < V; ++i) in[i] = fold.carry[lane * V + i];
    if (wave == WAVES - 1 && active) leave_chunk<V>(chain, chunk, C, c, lane, cuts != 0, A, H, fold);
  }

  float h[V];
#pragma unroll
  for (int i = 0; i < V; ++i) h[i] = cuts & ((1u << wave) - 1) ? ph[i] : fmaf(pa[i], in[i], ph[i]);
  if (L.carry && wave % (GDNQ_SCAN_CHUNK / RUN) == 0 && active && row0 < L.N) {
#pragma unroll
    for (int i = 0; i < V; ++i) L.carry[int64_t(row0 / GDNQ_SCAN_CHUNK) * C + c + i] = h[i];
  }
  E* ys = static_cast<E*>(L.y);
#pragma unroll
  for (int r = 0; r < RUN; ++r) {
    g[r].forget();
    if (!LOGITS) x[r].forget();
  }
  auto write_run = [&](auto PLAIN) {
#pragma unroll
    for (int r = 0; r < RUN; ++r) {
      if (!PLAIN.value && !(rows.valid >> r & 1)) continue;
      float a[V], b[V];
      input(r, a, b);
      if (!PLAIN.value && (rows.start >> r & 1)) {
        add_h0<V>(L.h0, rows.seq_of(r), C, c, a, b);
#pragma unroll
        for (int i = 0; i < V; ++i) h[i] = b[i];
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) h[i] = fmaf(a[i], h[i], b[i]);
      }
      Cell<E, V>::store(ys + int64_t(row0 + r) * C + c, h);
      if (!PLAIN.value && L.h_last && (rows.end >> r & 1)) {
#pragma unroll
        for (int i = 0; i < V; ++i) L.h_last[int64_t(rows.seq_of(r)) * C + c + i] = h[i];
      }
    }
  };
  if (active) by_kind<LOGITS>(rows.template plain<RUN>(), write_run);
}

// The backward pass runs the chain from the last chunk to the first with
// m_t = a_t l_t, what token t passes on to the token before it:
//   l_t = dy_t (+ dh_last at a sequence's last token) + m_{t+1},
// again pairs with m_out = A m_in + H, A = 0 over a sequence border.  The
// states h_{t-1} are formed again from the chunk's row of carry.
template <typename E, int V, bool LOGITS, bool LERP>
__global__ __launch_bounds__(BWD_WAVES * 64, BWD_PER_SIMD) void scan_backward_kernel(ScanLaunch L, Chain chain, const int32_t* __restrict__ cu,
                                                                       const E* __restrict__ xs, const E* __restrict__ gates,
                                                                       const E* __restrict__ dys, int tiles, int chunks) {
  constexpr int WAVES = BWD_WAVES, RUN = BWD_RUN, CT = 64 * V;
  __shared__ f32x2 wave_pair[WAVES][CT];  // of h, forwards
  __shared__ f32x2 wave_back[WAVES][CT];  // of m, backwards
  __shared__ Fold<V> fold;
  __shared__ uint32_t starts[WAVES], borders[WAVES];
  __shared__ int last_row;
  const int tile = blockIdx.x % tiles;
  const int place = chain.ticket ? take_ticket(chain.ticket + tile * TICKET_STRIDE) : 0, chunk = chunks - 1 - place;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int c = tile * CT + lane * V, C = L.C;
  const bool active = c < C;
  const int row0 = chunk * BWD_CHUNK + wave * RUN;

  Cell<E, V> x[RUN], dy[RUN];
  Gates<E, V, LOGITS> g[RUN];
  const int cl = active ? c : 0, last = int(L.N) - 1;
#pragma unroll
  for (int r = 0; r < RUN; ++r) {  // as in the forward pass
    if (LOGITS && row0 + r > last) continue;
    const int64_t at = int64_t(min(row0 + r, last)) * C;
    x[r].load(xs + at + cl);
    g[r].load(gates + at + cl);
    dy[r].load(dys + at + cl);
  }
  float h_in[V];
#pragma unroll
  for (int i = 0; i < V; ++i) h_in[i] = L.carry[int64_t(chunk) * C + cl + i];
  int first;
  const Rows rows = rows_of<RUN>(cu, L.B, L.T, L.N, row0, lane, first);
  if (threadIdx.x == WAVES * 64 - 64) {
    // the last token of the sequence that holds the chunk's last token (the
    // chunk's own last where none does, or where it ends there)
    const int at = chunk * BWD_CHUNK + BWD_CHUNK - 1;
    int e = at;
    if (at < L.N) {
      if (cu) {
        const int s = sequence_at(cu, L.B, at);
        if (s >= 0 && s < L.B) e = max(int(min(int64_t(cu[s + 1]), L.N)) - 1, at);
      } else {
        e = int((uint32_t(at) / uint32_t(L.T) + 1) * uint32_t(L.T)) - 1;
      }
    }
    last_row = e;
  }

  float A[V], H[V], M[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    A[i] = 1.0f;
    H[i] = M[i] = 0.0f;
  }
  // m behind a sequence's last token
  auto last_gradient = [&](int r, float (&m)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) m[i] = L.dh_last ? L.dh_last[int64_t(rows.seq_of(r)) * C + cl + i] : 0.0f;
  };
  // a and b of token r of the run
  auto input = [&](int r, float (&a)[V], float (&b)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float keep;
      g[r].get(i, a[i], keep);
      b[i] = LERP ? keep * x[r].get(i) : x[r].get(i);
    }
  };
  auto fold_run = [&](auto PLAIN) {
#pragma unroll
    for (int r = 0; r < RUN; ++r) {
      if (!PLAIN.value && !(rows.valid >> r & 1)) continue;
      float a[V], b[V];
      g[r].settle();
      input(r, a, b);
      if (!PLAIN.value && (rows.start >> r & 1)) {
        if (active) add_h0<V>(L.h0, rows.seq_of(r), C, c, a, b);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          A[i] = 0.0f;
          H[i] = b[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          H[i] = fmaf(a[i], H[i], b[i]);
          A[i] *= a[i];
        }
      }
    }
  };
  by_kind<LOGITS>(rows.template plain<RUN>(), fold_run);
  auto fold_back = [&](auto PLAIN) {
#pragma unroll
    for (int r = RUN - 1; r >= 0; --r) {
      if constexpr (!PLAIN.value) {
        if (!(rows.valid >> r & 1)) continue;
        if (rows.start >> r & 1) {
#pragma unroll
          for (int i = 0; i < V; ++i) M[i] = 0.0f;
          continue;
        }
        if (rows.end >> r & 1) last_gradient(r, M);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float a, keep;
        g[r].get(i, a, keep);
        M[i] = a * (dy[r].get(i) + M[i]);
      }
    }
  };
  by_kind<LOGITS>(rows.template plain<RUN>(), fold_back);
  put<V>(&wave_pair[wave][lane * V], A, H);
  // a border behind the run's last token is a border of m too, but not of h
  const bool border = rows.start != 0 || rows.end != 0;
#pragma unroll
  for (int i = 0; i < V; ++i) H[i] = border ? 0.0f : A[i];
  put<V>(&wave_back[wave][lane * V], H, M);
  if (lane == 0) {
    starts[wave] = rows.start;
    borders[wave] = border;
  }
  __syncthreads();

  {
    const uint32_t cuts = waves_with<WAVES>(starts, lane);
    float a[V] = {};
    for (int w = 0; w < wave; ++w) then<V>(&wave_pair[w][lane * V], cuts >> w & 1, a, h_in);
  }
  const uint32_t cuts = waves_with<WAVES>(borders, lane);
  // the pair of the waves behind this one
  float pa[V], pm[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    pa[i] = 1.0f;
    pm[i] = 0.0f;
  }
  for (int w = WAVES - 1; w > wave; --w) then<V>(&wave_back[w][lane * V], cuts >> w & 1, pa, pm);
  float in[V] = {};
  if (chain.ticket) {
    if (wave == 0) {  // the chunk's pair
#pragma unroll
      for (int i = 0; i < V; ++i) {
        M[i] = border ? M[i] : fmaf(H[i], pm[i], M[i]);
        H[i] = cuts ? 0.0f : H[i] * pa[i];
      }
      if (active) publish<V>(chain.pair + int64_t(place) * C + c, H, M);
    }
    const int from = min(place, max(0, chunks - 1 - last_row / BWD_CHUNK));
    enter_chunk<V, WAVES>(chain, place, from, C, c, active, wave, lane, fold);
#pragma unroll
    for (int i = 0; i < V; ++i) in[i] = fold.carry[lane * V + i];
    if (wave == 0 && active) leave_chunk<V>(chain, place, C, c, lane, cuts != 0, H, M, fold);
  }
  float m[V];
#pragma unroll
  for (int i = 0; i < V; ++i) m[i] = cuts >> (wave + 1) ? pm[i] : fmaf(pa[i], in[i], pm[i]);

  float before[RUN][V];
#pragma unroll
  for (int r = 0; r < RUN; ++r) {
    g[r].forget();
    if (!LOGITS) x[r].forget();
    if (!LOGITS) dy[r].forget();
  }
  E* dxs = static_cast<E*>(L.dx);
  E* dgs = static_cast<E*>(L.dgate);
  auto write_run = [&](auto PLAIN) {
#pragma unroll
    for (int r = 0; r < RUN; ++r) {
      if constexpr (!PLAIN.value) {
        if (!(rows.valid >> r & 1)) continue;
        if (rows.start >> r & 1) {
#pragma unroll
          for (int i = 0; i < V; ++i) h_in[i] = L.h0 ? L.h0[int64_t(rows.seq_of(r)) * C + c + i] : 0.0f;
        }
      }
      float a[V], b[V];
      input(r, a, b);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        before[r][i] = h_in[i];
        h_in[i] = fmaf(a[i], h_in[i], b[i]);
      }
    }
#pragma unroll
    for (int r = RUN - 1; r >= 0; --r) {
      if constexpr (!PLAIN.value) {
        if (!(rows.valid >> r & 1)) continue;
        if (rows.end >> r & 1) last_gradient(r, m);
      }
      float dx[V], dg[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float a, keep;
        g[r].get(i, a, keep);
        const float lam = dy[r].get(i) + m[i];
        const float da = lam * (LERP ? before[r][i] - x[r].get(i) : before[r][i]);
        dx[i] = LERP ? keep * lam : lam;
        dg[i] = LOGITS ? da * (a * keep) : da;
        m[i] = a * lam;
      }
      const int64_t at = int64_t(row0 + r) * C + c;
      Cell<E, V>::store(dxs + at, dx);
      Cell<E, V>::store(dgs + at, dg);
      if (!PLAIN.value && L.dh0 && (rows.start >> r & 1)) {
#pragma unroll
        for (int i = 0; i < V; ++i) L.dh0[int64_t(rows.seq_of(r)) * C + c + i] = m[i];
      }
    }
  };
  if (active) by_kind<LOGITS>(rows.template plain<RUN>(), write_run);
}

// What has to be done before the pass: the chain is emptied (tickets 0, pairs
// and states all ones), and out[s] = in[s] (zero where in is null) for the
// sequences without tokens, whose states pass through.  A wave looks at 64
// sequences at a time.
__global__ __launch_bounds__(256) void scan_begin_kernel(uint32_t* ticket, int tiles, ulonglong2* rest, int64_t n,
                                                         const int32_t* __restrict__ cu, const float* __restrict__ in,
                                                         float* __restrict__ out, int B, int C, int N) {
  const int64_t i = blockIdx.x * int64_t(256) + threadIdx.x;
  if (i < tiles) ticket[i * TICKET_STRIDE] = 0;
  if (i < n) rest[i] = ulonglong2{EMPTY, EMPTY};
  bool empty = out && i < B;
  if (empty && cu) empty = min(max(cu[i], 0), N) >= min(max(cu[i + 1], 0), N);
  const int lane = threadIdx.x & 63;
  for (uint64_t left = __builtin_amdgcn_ballot_w64(empty); left; left &= left - 1) {
    const int64_t at = (i - lane + __builtin_ctzll(left)) * C;
    for (int c = lane; c < C; c += 64) out[at + c] = in ? in[at + c] : 0.0f;
  }
}

// One value a lane: 64 x 4096 takes 2.8 us, little more than a launch; 1024 x
// 8192 in bf16 17.9 us (117 MB, in part from the last-level cache), fp32 21.7 (168 MB).
template <typename E, bool LOGITS, bool LERP>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanLaunch L) {
  const int64_t n = int64_t(L.B) * L.C, i = blockIdx.x * int64_t(256) + threadIdx.x;
  if (i >= n) return;
  Gates<E, 1, LOGITS> g;
  g.load(static_cast<const E*>(L.gate) + i);
  g.settle();
  float a, keep;
  g.get(0, a, keep);
  const float v = to_f32(static_cast<const E*>(L.x)[i]);
  const float h = fmaf(a, L.h0[i], LERP ? keep * v : v);
  L.h_last[i] = h;
  store_f32(static_cast<E*>(L.y) + i, h);
}

struct Layout {
  int tiles;
  int64_t chunks, words;  // 8-byte words of pairs and states
  size_t bytes;
};

Layout layout_of(int64_t N, int C, int chunk, int V) {
  Layout l;
  l.tiles = (C + 64 * V - 1) / (64 * V);
  l.chunks = (N + chunk - 1) / chunk;
  l.words = (l.chunks + l.chunks / GROUP + l.chunks / (GROUP * GROUP)) * C + 1;
  l.bytes = l.chunks > 1 ? size_t(l.tiles) * TICKET_STRIDE * 4 + size_t(l.words + 1) / 2 * 16 : 0;
  return l;
}

// The chain in the workspace (none for a call of one chunk), emptied, and the
// sequences without tokens.
hipError_t begin(const ScanLaunch& L, const Layout& l, const float* in, float* out, Chain& chain, hipStream_t stream) {
  chain = Chain{};
  const bool linked = l.chunks > 1;
  if (!L.cu_seqlens && L.N > 0) out = nullptr;  // every sequence has tokens
  if (!linked && !out) return hipSuccess;
  if (linked) {
    chain.ticket = static_cast<uint32_t*>(L.workspace);
    chain.pair = reinterpret_cast<unsigned long long*>(chain.ticket + size_t(l.tiles) * TICKET_STRIDE);
    chain.group = chain.pair + l.chunks * L.C;
    chain.state = chain.group + l.chunks / GROUP * L.C;
  }
  const int64_t words = linked ? (l.words + 1) / 2 : 0, tiles = linked ? l.tiles : 0;
  int64_t most = words > tiles ? words : tiles;
  if (out && L.B > most) most = L.B;
  scan_begin_kernel<<<uint32_t((most + 255) / 256), 256, 0, stream>>>(chain.ticket, int(tiles),
                                                                    reinterpret_cast<ulonglong2*>(chain.pair), words,
                                                                    L.cu_seqlens, in, out, L.B, L.C, int(L.N));
  return hipGetLastError();
}

template <typename E, int V, bool LOGITS, bool LERP>
struct Forward {
  static hipError_t go(const ScanLaunch& L, hipStream_t stream) {
    const Layout l = layout_of(L.N, L.C, FWD_CHUNK, V);
    Chain chain;
    if (hipError_t e = begin(L, l, L.h0, L.h_last, chain, stream)) return e;
    if (L.N == 0) return hipSuccess;
    scan_forward_kernel<E, V, LOGITS, LERP><<<uint32_t(l.chunks * l.tiles), ForwardShape<V>::WAVES * 64, 0, stream>>>(
        L, chain, L.cu_seqlens, static_cast<const E*>(L.x), static_cast<const E*>(L.gate), l.tiles);
    return hipGetLastError();
  }
};

template <typename E, int V, bool LOGITS, bool LERP>
struct Backward {
  static hipError_t go(const ScanLaunch& L, hipStream_t stream) {
    const Layout l = layout_of(L.N, L.C, BWD_CHUNK, V);
    Chain chain;
    if (hipError_t e = begin(L, l, L.dh_last, L.dh0, chain, stream)) return e;
    if (L.N == 0) return hipSuccess;
    scan_backward_kernel<E, V, LOGITS, LERP><<<uint32_t(l.chunks * l.tiles), BWD_WAVES * 64, 0, stream>>>(
        L, chain, L.cu_seqlens, static_cast<const E*>(L.x), static_cast<const E*>(L.gate), static_cast<const E*>(L.dy), l.tiles,
        int(l.chunks));
    return hipGetLastError();
  }
};

template <typename E, int V, bool LOGITS, bool LERP>
struct Step {
  static hipError_t go(const ScanLaunch& L, hipStream_t stream) {
    scan_step_kernel<E, LOGITS, LERP><<<uint32_t((int64_t(L.B) * L.C + 255) / 256), 256, 0, stream>>>(L);
    return hipGetLastError();
  }
};

template <template <typename, int, bool, bool> class F, typename E, int V>
hipError_t by_flags(const ScanLaunch& L, hipStream_t stream) {
  if (L.logits) return L.lerp ? F<E, V, true, true>::go(L, stream) : F<E, V, true, false>::go(L, stream);
  return L.lerp ? F<E, V, false, true>::go(L, stream) : F<E, V, false, false>::go(L, stream);
}

// Channels per lane: a wave's row is 256 bytes in fp32 and, in pairs, in
// bf16; an odd number of bf16 channels leaves rows unaligned to pairs and
// takes one channel per lane.
template <template <typename, int, bool, bool> class F>
hipError_t dispatch(const ScanLaunch& L, hipStream_t stream) {
  if (!L.bf16) return by_flags<F, float, 1>(L, stream);
  return L.C % 2 ? by_flags<F, bf16, 1>(L, stream) : by_flags<F, bf16, 2>(L, stream);
}

}  // namespace

size_t scan_workspace_bytes(int64_t N, int C, bool is_bf16) {
  const int V = is_bf16 && C % 2 == 0 ? 2 : 1;
  const size_t f = layout_of(N, C, FWD_CHUNK, V).bytes, b = layout_of(N, C, BWD_CHUNK, V).bytes;
  return f > b ? f : b;
}
hipError_t launch_scan_forward(const ScanLaunch& L, hipStream_t s) { return dispatch<Forward>(L, s); }
hipError_t launch_scan_backward(const ScanLaunch& L, hipStream_t s) { return dispatch<Backward>(L, s); }
hipError_t launch_scan_step(const ScanLaunch& L, hipStream_t s) { return dispatch<Step>(L, s); }

}  // namespace gdnq
