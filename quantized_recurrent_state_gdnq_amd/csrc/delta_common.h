// Shared parts of the trained delta rule (delta_rule.hip, delta_rule_backward.hip):
// where chunks lie, what the workspace and the carry hold, and the layouts of
// the matrix operands.
//
// A chunk is 64 tokens of one sequence, counted from the sequence's start.  With
//   c_i   the running product of alpha inside the chunk, rho_ij = c_i / c_j,
//   At_ij = rho_ij k_i.k_j (j < i),   M_ij = rho_ij q_i.k_j (j <= i),
//   B     = diag(beta),   S the state that enters the chunk,
// the chunk is
//   w = (I + At B)^-1 (V - c K S^T),   u = B w      (w: what each token writes, u: times beta)
//   O = c Q S^T + M u,                 S' = c_64 S + u^T (c_64 / c) K
// and its gradient, from dS' and dO,
//   du = M^T dO + (c_64 / c) K dS'^T,  z = (I + B At)^-T du,  dx = B z
//   dS = c_64 dS' + dO^T c Q - dx^T c K,   dV = dx,   dbeta = w . z
// (the rest at the gradient kernel).  Only S and dS pass from chunk to chunk,
// and each of their rows by itself: a wave carries 16 rows.
//
// Operands of the products are bf16: q, k, v and dO as they are, fp32 values in
// parts, bf16(x), bf16(x less that) and so on.  What passes to a state, a gate's
// gradient or the next chunk has three, 24 bits and more; the inverse two, 16 to 17
// bits, and so does what goes to a bf16 result alone (M, O's S and w, dM and dAt).
// Products of parts beyond the longer operand's last (2^-25 of a term of three, 2^-18
// of two) are left out.  Sums are fp32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.h"
#include "launch.h"
#include "mfma.h"
#include "vec_io.h"

namespace gdnq {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int DELTA_CHUNK = 64;
// A triangle of 64 x 64 as the first operand of a product: of its 16 x 32
// blocks six are not zero.  A block is 64 lanes of 16 bytes; a part lies behind another.
constexpr int TRI_BLOCKS = 6, TRI_PART = TRI_BLOCKS * 1024, TRI_BYTES = 2 * TRI_PART;
// Of one chunk of one value head in the workspace: two such triangles (the backward
// pass's second in three parts), then rows of 64: c, beta c_64 / c, c_64 / c, beta c
// (the chains' kilobyte), beta, and log2 c as a whole number and a rest.
__host__ __device__ constexpr int delta_scalars(bool back) { return (back ? 5 : 4) * TRI_PART; }
enum { ROW_C, ROW_TAIL_BETA, ROW_TAIL, ROW_C_BETA, ROW_BETA, ROW_WHOLE, ROW_REST, ROWS };
__host__ __device__ constexpr int delta_chunk_bytes(bool back) { return delta_scalars(back) + 8 * 256; }

inline int64_t delta_slots(const DeltaLaunch& L) {
  return L.cu_seqlens ? L.N / DELTA_CHUNK + L.B : int64_t(L.B) * ((int64_t(L.T) + DELTA_CHUNK - 1) / DELTA_CHUNK);
}
__host__ __device__ inline int64_t delta_align(int64_t n) { return (n + 255) / 256 * 256; }
// What a chain leaves of a chunk and head, in fp32: a state, and behind it the
// chunk's w or z, [d_v][64].  Both are in tiles of 16 rows and 16 columns, a kilobyte,
// the columns those of a chain's tile (chain_row): a store of a wave is then whole
// lines (rows as they are leave half a line each: 4 x 8192 tokens, 16 heads, chain 640
// us, with tiles 583).
__host__ __device__ inline int64_t delta_state_floats(const DeltaLaunch& L) {
  return int64_t((L.dv + 15) / 16) * ((L.dk + 31) / 32) * 512;
}
__host__ __device__ inline int64_t delta_left_bytes(const DeltaLaunch& L) {
  return delta_state_floats(L) * 4 + int64_t((L.dv + 15) / 16) * 4096;
}
// Where, in floats, a lane's four values of a tile are, of rows of so many tiles.
__host__ __device__ inline int left_place(int row, int tile, int tiles, int g) {
  return ((row >> 4) * tiles + tile) * 256 + (row & 15) * 16 + g * 4;
}

// Few chains of many chunks are cut into segments that run at once.  A segment
// maps the state that enters it linearly, S' = S P + R: a first pass carries R
// from zero and P from the identity (d_k more rows, without V and O), a second
// one joins them, and the chains then start from the states that enter.  That is
// 1.9 times the work (without the outputs, and with two parts of each value, 82 of
// 176 products a chunk and row), so it pays where chains leave three in four of the
// 256 CUs idle: 65536 tokens, 8 heads, 16 workgroups: the call takes 3.3 ms in one
// piece, 0.65 cut.  What enters a segment is good to the two parts' bits, 5e-6 of its
// norm; three would be half as many products again in both passes.
//   Packed sequences differ: those of more than `split_above` chunks, three times what
// a CU's share of all chunks would be, are cut into segments of that share (their
// lengths are known on the device alone).  16384 tokens, 16 heads, forward: one of all
// 873 -> 316 us; 10000, 4000, 1500 and 884 570 -> 371; where none is long enough the two
// empty launches cost 8 to 10 of 230.  Twice and half the share: 356 and 455.
//   In the workspace for each segment of a cut sequence and each head: R (then the
// state behind the segment) [d_v][d_k] fp32, P [2][d_k][d_k] in two bf16 parts.
constexpr int DELTA_ORDERED = 64;  // packed sequences that a wave puts in order
inline void delta_split(DeltaLaunch& L, int64_t at) {
  const int64_t rows = int64_t(L.H) * ((L.dv + 63) / 64), chains = rows * L.B;
  const int64_t chunks = ((L.cu_seqlens ? L.N : int64_t(L.T)) + DELTA_CHUNK - 1) / DELTA_CHUNK;
  L.segments = 1;
  L.seg_chunks = L.split_above = 0x7fffffff;
  L.seg_slots = 0;
  L.seg_at = delta_align(at);
  if (chains == 0) return;
  if (L.cu_seqlens) {
    const int64_t share = chunks * rows / 256;
    const int64_t above = share > 5 ? 3 * share : 16;
    if (L.B > DELTA_ORDERED || chunks <= above) return;
    L.split_above = int(above);
    L.seg_chunks = int(share > 8 ? share : 8);
    L.segments = int((chunks + L.seg_chunks - 1) / L.seg_chunks);
    // every cut sequence has one more than its whole segments, and is longer than split_above
    L.seg_slots = chunks / L.seg_chunks + chunks / above + 1;
  } else {
    if (chains > 64) return;
    const int64_t want = 256 / chains;
    if (chunks < 8 * want) return;
    L.split_above = 0;
    L.seg_chunks = int((chunks + want - 1) / want);
    L.segments = int((chunks + L.seg_chunks - 1) / L.seg_chunks);
    L.seg_slots = int64_t(L.B) * L.segments;
  }
}
// Segments and whole sequences of a call, at most; of a first pass, the segments that another follows.
inline int64_t delta_items(const DeltaLaunch& L, bool pass) {
  if (L.segments == 1) return L.B;
  if (!L.cu_seqlens) return int64_t(L.B) * (L.segments - pass);
  return L.N / DELTA_CHUNK / L.seg_chunks + (pass ? 1 : L.B);
}
__host__ __device__ inline int64_t delta_segment_bytes(const DeltaLaunch& L) { return int64_t(L.dk) * (L.dv + L.dk) * 4; }
// The bytes up to the end of what the segments take.
inline int64_t delta_split_bytes(const DeltaLaunch& L) { return L.seg_at + L.seg_slots * L.H * delta_segment_bytes(L); }

#ifdef __HIPCC__

__device__ __forceinline__ uint8_t* delta_segment(const DeltaLaunch& L, int at, int h) {
  return static_cast<uint8_t*>(L.workspace) + L.seg_at + (int64_t(at) * L.H + h) * delta_segment_bytes(L);
}

template <int V>
using Int = std::integral_constant<int, V>;
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (I < N) {
    f(Int<I>{});
    each<N, I + 1>(static_cast<F&&>(f));
  }
}

struct DeltaSpan {
  int64_t first, slot;  // first token in the call, first chunk slot
  int tokens;
};

// The offsets of sequence b: malformed ones are clamped into [0, N].
__device__ __forceinline__ int64_t delta_offset(const DeltaLaunch& L, int b) {
  return min(max(int64_t(L.cu_seqlens[b]), int64_t(0)), L.N);
}

// Slots of packed sequences need no map: sequence b's start at cu[b] / 64 + b,
// and those of the next lie far enough behind, since floor(y / 64) -
// floor(x / 64) + 1 >= ceil((y - x) / 64).
__device__ __forceinline__ DeltaSpan delta_sequence(const DeltaLaunch& L, int b) {
  if (!L.cu_seqlens) {
    const int chunks = (L.T + DELTA_CHUNK - 1) / DELTA_CHUNK;
    return {int64_t(b) * L.T, int64_t(b) * chunks, L.T};
  }
  const int64_t first = delta_offset(L, b), end = delta_offset(L, b + 1);
  return {first, first / DELTA_CHUNK + b, int(max(end - first, int64_t(0)))};
}

// Workgroups that read the same (a key head's) on the same XCD, whose L2 they
// share: of a grid of units of `size` workgroups, eight units at a time, one for each
// XCD, as workgroups are dealt out; the last units, fewer than eight, in order.
// 65536 tokens, 8 heads, first pass 216 -> 206 us; 16384 packed tokens, 16 heads, chains 328 -> 317
// and 334 -> 323.
__device__ __forceinline__ int xcd_unit(int size, int& within) {
  const int block = int(blockIdx.x), full = int(gridDim.x) / size & ~7;
  if (block < full * size) {
    const int r = block % (8 * size);
    within = r >> 3;
    return block / (8 * size) * 8 + (r & 7);
  }
  within = (block - full * size) % size;
  return full + (block - full * size) / size;
}

// What the workgroups of a chain take: a sequence, or a segment of one.
struct DeltaItem {
  int b, seg, segments;  // b < 0: none
  int64_t at;            // its sequence's first segment in the workspace
};
// Of packed sequences (up to 64, a lane each) the longest come first, so that no
// long chain starts beside the last short ones (12 sequences of 16384 tokens, 16
// heads: 326 -> 317 us, and 336 -> 323 back).  Malformed offsets can ask for more
// items or segments than there are: those beyond are left out.  More than 64 sequences
// are taken as they lie, uncut: 16000 tokens and 64 short ones take 867 us forward and
// 1486 back, with 63 short ones 463 and 1036.
__device__ __forceinline__ DeltaItem delta_packed(const DeltaLaunch& L, int index, int b, bool pass) {
  const int lane = threadIdx.x & 63;
  const int tokens = lane < L.B ? delta_sequence(L, lane).tokens : -1;
  const int chunks = (tokens + DELTA_CHUNK - 1) / DELTA_CHUNK;
  const int segments = chunks > L.split_above ? (chunks + L.seg_chunks - 1) / L.seg_chunks : 1;
  const int items = lane < L.B ? segments - pass : 0, slots = segments > 1 ? segments : 0;
  int before = 0;
  int64_t at = 0;
  for (int i = 0; i < L.B; ++i) {
    const int other = __builtin_amdgcn_readlane(tokens, i);
    const bool first = other > tokens || (other == tokens && i < lane);
    before += first ? __builtin_amdgcn_readlane(items, i) : 0;
    at += first ? __builtin_amdgcn_readlane(slots, i) : 0;
  }
  const bool fits = at + slots <= L.seg_slots;
  const bool here = b < 0 ? index >= before && index - before < items : lane == b;
  const uint64_t found = __builtin_amdgcn_ballot_w64(here && fits);
  if (!found) return {-1, 0, 1, 0};
  const int from = __builtin_ctzll(found);
  return {from, index - __builtin_amdgcn_readlane(before, from), __builtin_amdgcn_readlane(segments, from),
          __builtin_amdgcn_readlane(int(at), from)};
}
// The index-th item.
__device__ __forceinline__ DeltaItem delta_item(const DeltaLaunch& L, int index, bool pass) {
  if (L.cu_seqlens && L.B <= DELTA_ORDERED) return delta_packed(L, index, -1, pass);
  const int n = L.segments - pass;
  return {index / n, index % n, L.segments, int64_t(index / n) * L.segments};
}
// All of sequence b.
__device__ __forceinline__ DeltaItem delta_whole(const DeltaLaunch& L, int b) {
  if (L.cu_seqlens && L.B <= DELTA_ORDERED) return delta_packed(L, 0, b, false);
  return {b, 0, L.segments, int64_t(b) * L.segments};
}

// The tokens of a slot: how many (0: none) and the first.
__device__ __forceinline__ int delta_slot_tokens(const DeltaLaunch& L, int slot, int64_t& first) {
  int b;
  if (!L.cu_seqlens) {
    const int chunks = (L.T + DELTA_CHUNK - 1) / DELTA_CHUNK;
    b = slot / chunks;
  } else {
    int low = 0, high = L.B - 1;  // the last sequence that starts at or before the slot
    while (low < high) {
      const int mid = (low + high + 1) / 2;
      if (delta_offset(L, mid) / DELTA_CHUNK + mid <= slot)
        low = mid;
      else
        high = mid - 1;
    }
    b = low;
  }
  const DeltaSpan s = delta_sequence(L, b);
  const int64_t at = (slot - s.slot) * DELTA_CHUNK;
  first = s.first + at;
  return at < 0 ? 0 : int(min(int64_t(DELTA_CHUNK), s.tokens - at > 0 ? s.tokens - at : int64_t(0)));
}

// Rows of D bf16 in LDS in 16-byte blocks, permuted by the row's number so
// that neither sixteen rows at one block nor the 4 rows x 32 (or 4 x 8) bytes of
// a transposing read meet in a bank.
template <int D>
__device__ __forceinline__ int lds_block(int row, int block) {
  if constexpr (D == 128)
    return row * 256 + ((block ^ ((row & 3) << 2 | (row >> 2 & 3))) << 4);
  else
    return row * 128 + ((block ^ ((row >> 1 & 1) << 2 | (row >> 2 & 3))) << 4);
}

// Loads are made whatever the token or column, from a clamped address, and cut
// to zero where they are used: a branch around a load waits for it on the spot.
__device__ __forceinline__ u32x4 only_if(bool keep, const u32x4& x) {
  const uint32_t m = keep ? ~0u : 0u;
  return x & m;
}

__device__ __forceinline__ bf16x8 lds_frag(const uint8_t* p) { return *reinterpret_cast<const bf16x8*>(p); }

// 4 x 16 values of 16 bits per 16 lanes, transposed: lane 4 t + p gives the
// address of four adjacent values of row t, lane i gets column i of four rows.
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ bf16x8 lds_transposed(const uint8_t* a, const uint8_t* b) {
  typedef __attribute__((address_space(3))) s16x4* lds4;
  const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(a));
  const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(b));
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  return __builtin_bit_cast(bf16x8, s16x8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]});
}

// Products of fp32 values in two parts.
__device__ __forceinline__ f32x4 mfma_exact_split(const bf16x8& a, const bf16x8& bh, const bf16x8& bl, f32x4 c) {
  return mfma16(a, bh, mfma16(a, bl, c));
}
__device__ __forceinline__ f32x4 mfma_split_split(const bf16x8& ah, const bf16x8& al, const bf16x8& bh, const bf16x8& bl,
                                                  f32x4 c) {
  return mfma16(ah, bh, mfma16(ah, bl, mfma16(al, bh, c)));
}

// Two values in P parts, five instructions for each part but the last.
template <int P>
__device__ __forceinline__ void split_pair(f32x2 x, uint32_t (&parts)[P]) {
#pragma unroll
  for (int p = 0; p < P; ++p) {
    parts[p] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
    if (p + 1 == P) break;
    uint32_t word = parts[p];
    asm("" : "+v"(word));  // or the compiler rounds each value again to have it by itself
    x = f32x2{x[0] - __uint_as_float(word << 16), x[1] - __uint_as_float(word & 0xffff0000u)};
  }
}
// Eight values in P parts.
template <int P>
__device__ __forceinline__ void split8(const f32x4& a, const f32x4& b, bf16x8 (&x)[P]) {
  u32x4 words[P];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t parts[P];
    split_pair(i < 2 ? f32x2{a[2 * i], a[2 * i + 1]} : f32x2{b[2 * i - 4], b[2 * i - 3]}, parts);
#pragma unroll
    for (int p = 0; p < P; ++p) words[p][i] = parts[p];
  }
#pragma unroll
  for (int p = 0; p < P; ++p) x[p] = __builtin_bit_cast(bf16x8, words[p]);
}
// f(i, j) for the parts of a product of PA and PB that are not left out, the
// smallest terms first.
template <int PA, int PB, typename F>
__device__ __forceinline__ void part_terms(F&& f) {
  constexpr int N = PA > PB ? PA : PB;
  each<N * PA>([&](auto n) {
    constexpr int i = PA - 1 - n.value % PA, j = N - 1 - n.value / PA - i;
    if constexpr (j >= 0 && j < PB) f(Int<i>{}, Int<j>{});
  });
}

// 2^(a - b) of numbers given as whole part and rest.
__device__ __forceinline__ float exp2_difference(float ar, int aw, float br, int bw) {
  return ldexpf(__builtin_amdgcn_exp2f(ar - br), aw - bw);
}

// In the chains a wave's tile it of 16 tokens holds, in row 4 g + e, token
// 32 (it / 2) + 8 g + 4 (it % 2) + e, and tile t of 16 state columns likewise:
// so the results of two tiles are, in their lanes, the second operand of a
// product over those 32, in order.
__device__ __forceinline__ int chain_row(int tile, int row) {
  return (tile >> 1) * 32 + (row >> 2) * 8 + (tile & 1) * 4 + (row & 3);
}

// What the workgroup of a chain (256 threads, 64 rows of a state) has in LDS of
// a chunk: K, Q, the two triangles, 64 columns of V (or dO), and the kilobyte of
// decays.  All of it comes straight from memory, 16 bytes a lane and 1 KB a wave
// at a time, in the order of LDS: the permutation of the blocks is in the address
// that each lane loads from.
// The first pass over segments of the forward call needs neither Q nor the second
// triangle, and two of its workgroups fit a CU.
template <int DK, bool BACK, bool BARE>
struct ChainBuffer {
  static constexpr int TRI_PIECES = delta_scalars(BACK) / 1024;
  uint8_t k[64 * DK * 2], q[64 * DK * 2], tri[delta_scalars(BACK)], v[64 * 128], rows[1024];
};
template <int DK, bool BACK>
struct ChainBuffer<DK, BACK, true> {
  static constexpr int TRI_PIECES = TRI_BYTES / 1024;
  uint8_t k[64 * DK * 2], tri[TRI_BYTES], v[64 * 128], rows[1024];
};

__device__ const uint8_t delta_zeros[16] __attribute__((aligned(16))) = {};

// As a statement that writes no register: the compiler, which would wait for
// all such loads before any read of LDS, does not know of it, and the kernel
// waits itself (vmcnt) before the barrier that lets the buffer be read.  The
// s_nop is the wait that a load into LDS needs behind a scalar write of M0, where
// the chip takes its place from.
__device__ __forceinline__ void to_lds(const void* base, uint32_t offset, void* to) {
  const uint32_t lds = uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)to));
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(offset), "s"(base) : "m0", "memory");
}
__device__ __forceinline__ void to_lds(const void* p, void* to) {
  const uint32_t lds = uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)to));
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p) : "m0", "memory");
}

// The row and block that lane place p of a matrix of rows of D bf16 is: the
// inverse of lds_block.
template <int D>
__device__ __forceinline__ void lds_place(int p, int& row, int& block) {
  row = p / (D / 8);
  block = (lds_block<D>(row, p % (D / 8)) >> 4) % (D / 8);
}

template <int DK, bool BACK>
struct ChainLoader {
  static constexpr int LOADS = 64 * (DK / 8) / 256;
  template <bool BARE>
  using Buffer = ChainBuffer<DK, BACK, BARE>;
  uint32_t at_k[LOADS], at_v[2];  // byte offsets in a whole chunk
  const uint8_t *k, *q, *v;       // of the call's first token, this head, this group of columns
  const uint8_t* space;           // the workspace at this head
  int64_t krow, vrow, chunk_stride;
  int dk, cols, wave, lane;
  bool exact;                     // no columns of K to be zero
  uint32_t beyond;                // else bit i: the lane's block of load i is such a column

  __device__ __forceinline__ void init(const DeltaLaunch& L, const void* values, int h, int group, int wave_, int lane_) {
    wave = wave_;
    lane = lane_;
    dk = L.dk;
    exact = L.dk == DK;
    const int kh = h / (L.H / L.G);
    krow = int64_t(L.G) * L.dk * 2;
    vrow = int64_t(L.H) * L.dv * 2;
    k = static_cast<const uint8_t*>(L.k) + int64_t(kh) * L.dk * 2;
    q = static_cast<const uint8_t*>(L.q) + int64_t(kh) * L.dk * 2;
    v = static_cast<const uint8_t*>(values) + (int64_t(h) * L.dv + group * 64) * 2;
    cols = min(64, L.dv - group * 64);
    space = static_cast<const uint8_t*>(L.workspace) + int64_t(h) * delta_chunk_bytes(BACK);
    chunk_stride = int64_t(L.H) * delta_chunk_bytes(BACK);
    int row, block;
    beyond = 0;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      lds_place<DK>((i * 4 + wave) * 64 + lane, row, block);
      at_k[i] = uint32_t(row) * uint32_t(krow) + block * 16;
      beyond |= uint32_t(block * 8 >= dk) << i;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      lds_place<64>((i * 4 + wave) * 64 + lane, row, block);
      at_v[i] = uint32_t(row) * uint32_t(vrow) + min(block * 8, cols - 8) * 2;  // columns beyond the last: no matter
    }
  }

  // The next chunk to load: n tokens from `first` on, chunk slot `slot`.
  struct Next {
    const uint8_t *ws, *k, *q, *v;
    int n;
    bool whole;
  };
  __device__ __forceinline__ Next next(int64_t first, int n, int64_t slot) const {
    return {space + slot * chunk_stride, k + first * krow, q + first * krow, v + first * vrow, n, n == 64};
  }

  // A whole chunk's loads are made in STEPS parts of one or two, between the
  // products of the chunk before: all at once they hold the wave up until the
  // queue has room (2600 of a chunk's 8100 cycles).
  static constexpr int TRI_STEPS = (delta_scalars(BACK) / 1024 + 7) / 8, STEPS = LOADS + 1 + TRI_STEPS + 1;
  template <int STEP, bool BARE>
  __device__ __forceinline__ void step(Buffer<BARE>& to, const Next& x) const {
    constexpr int PIECES = Buffer<BARE>::TRI_PIECES;
    if constexpr (STEP < LOADS) {
      if (exact || !(beyond >> STEP & 1)) {  // lanes of columns beyond the last write nothing
        to_lds(x.k, at_k[STEP], to.k + (STEP * 4 + wave) * 1024);
        if constexpr (!BARE) to_lds(x.q, at_k[STEP], to.q + (STEP * 4 + wave) * 1024);
      }
    } else if constexpr (STEP == LOADS) {
#pragma unroll
      for (int i = 0; i < 2; ++i) to_lds(x.v, at_v[i], to.v + (i * 4 + wave) * 1024);
    } else if constexpr (STEP < LOADS + 1 + TRI_STEPS) {
#pragma unroll
      for (int i = (STEP - LOADS - 1) * 2; i < (STEP - LOADS) * 2 && i * 4 < PIECES; ++i)
        if (i * 4 + 4 <= PIECES || i * 4 + wave < PIECES)
          to_lds(x.ws, (i * 4 + wave) * 1024 + lane * 16, to.tri + (i * 4 + wave) * 1024);
    } else {
      if (wave == 0) to_lds(x.ws + delta_scalars(BACK), lane * 16, to.rows);
    }
  }

  // The columns beyond the last, zero in both buffers before the first load, so that
  // their chunks too are loaded in steps (1003 tokens, heads of 72: chain 52 -> 49 us).
  template <bool BARE>
  __device__ __forceinline__ void clear(Buffer<BARE>& to) const {
    if (exact) return;
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      if (beyond >> i & 1) {
        const int at = (i * 4 + wave) * 1024 + lane * 16;
        *reinterpret_cast<u32x4*>(to.k + at) = u32x4{0, 0, 0, 0};
        if constexpr (!BARE) *reinterpret_cast<u32x4*>(to.q + at) = u32x4{0, 0, 0, 0};
      }
  }

  // Any chunk at once.  Rows behind the last token are the last one's again (beta
  // is 0 there), or zeros where ZERO_V; columns behind the last are zero.
  template <bool ZERO_V, bool BARE>
  __device__ __forceinline__ void load(Buffer<BARE>& to, const Next& x) const {
    each<STEPS - LOADS - 1>([&](auto i) { step<LOADS + 1 + i.value, BARE>(to, x); });
    int row, block;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      lds_place<DK>((i * 4 + wave) * 64 + lane, row, block);
      const int64_t at = min(row, x.n - 1) * krow + block * 16;
      to_lds(block * 8 < dk ? x.k + at : delta_zeros, to.k + (i * 4 + wave) * 1024);
      if constexpr (!BARE) to_lds(block * 8 < dk ? x.q + at : delta_zeros, to.q + (i * 4 + wave) * 1024);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      lds_place<64>((i * 4 + wave) * 64 + lane, row, block);
      const uint8_t* p = x.v + min(row, x.n - 1) * vrow + min(block * 8, cols - 8) * 2;
      to_lds(ZERO_V && row >= x.n ? delta_zeros : p, to.v + (i * 4 + wave) * 1024);
    }
  }
};

// What the chains read of K or Q: the 64 tokens in chain order with 32 columns
// each (an operand of a product over d_k), and 64 columns in chain order with
// their tokens (of one over the tokens).  Operands are read some products ahead
// of their own, and kept there (the sched_barriers): left to the compiler each
// was read just before its product, and waited for.
template <int DK>
__device__ __forceinline__ void chain_rows(const uint8_t* m, int lane, int j, bf16x8 (&f)[4]) {
#pragma unroll
  for (int it = 0; it < 4; ++it) f[it] = lds_frag(m + lds_block<DK>(chain_row(it, lane & 15), j * 4 + (lane >> 4)));
}
template <int DK>
__device__ __forceinline__ void chain_columns(const uint8_t* m, int lane, int tiles, bf16x8 (&f)[4][2]) {
  const int c = lane & 15, g = lane >> 4;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int row = j * 32 + g * 8 + (c >> 2), block = ((tiles * 4 + t) >> 1) * 4 + (c & 3), half = (t & 1) * 8;
      f[t][j] = lds_transposed(m + lds_block<DK>(row, block) + half, m + lds_block<DK>(row + 4, block) + half);
    }
}
// Four tiles of S^T += columns^T x, x in P parts, 32 tokens each.
template <int P>
__device__ __forceinline__ void chain_update(f32x4* S, const bf16x8 (&f)[4][2], const bf16x8 (&x)[2][P]) {
#pragma unroll
  for (int p = P - 1; p >= 0; --p)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int t = 0; t < 4; ++t) S[t] = mfma16(f[t][j], x[j][p], S[t]);
}
// The six blocks of a triangle, in its first P parts.
template <int P>
__device__ __forceinline__ void chain_triangle(const uint8_t* tri, int lane, bf16x8 (&m)[P][TRI_BLOCKS]) {
#pragma unroll
  for (int i = 0; i < TRI_BLOCKS; ++i)
#pragma unroll
    for (int p = 0; p < P; ++p) m[p][i] = lds_frag(tri + p * TRI_PART + i * 1024 + lane * 16);
}
__device__ __forceinline__ void phase() { __builtin_amdgcn_sched_barrier(0); }

// Four tokens of tile it of a lane's column, out of the 64 columns in LDS.
__device__ __forceinline__ s16x4 chain_column(const uint8_t* v, int it, int wave, int lane) {
  const int c = lane & 15, g = lane >> 4;
  typedef __attribute__((address_space(3))) s16x4* lds4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (lds4)(v + lds_block<64>(chain_row(it, g * 4) + (c >> 2), wave * 2 + ((c & 3) >> 1)) + (c & 1) * 8));
}
__device__ __forceinline__ float bf16_value(short x) { return __uint_as_float(uint32_t(uint16_t(x)) << 16); }

// Where the workgroup of a chain is: rows [64 group, ..) of head h, an item's chunks.
// Of a first pass the groups behind those of V carry the identity.
struct ChainPlace {
  int h, group, first, end;  // chunks
  bool identity;
};
__device__ __forceinline__ ChainPlace chain_place(const DeltaLaunch& L, int groups, int chunks, const DeltaItem& item, int key_head,
                                                 int within) {
  ChainPlace p;
  p.group = within % groups;
  p.h = key_head * (L.H / L.G) + within / groups;
  const int dv_groups = (L.dv + 63) / 64;
  p.identity = p.group >= dv_groups;
  if (p.identity) p.group -= dv_groups;
  p.first = item.seg > 0 ? int(min(int64_t(item.seg) * L.seg_chunks, int64_t(chunks))) : 0;
  p.end = item.seg + 1 < item.segments ? int(min(int64_t(p.first) + L.seg_chunks, int64_t(chunks))) : chunks;
  return p;
}
// A chain's state tiles from a matrix of fp32 rows (or none: zero), or the identity.
template <int TILES>
__device__ __forceinline__ void chain_load_state(f32x4 (&S)[TILES], const float* rows, int dk, int row, bool here, int g) {
#pragma unroll
  for (int t = 0; t < TILES; ++t) {
    const int at = chain_row(t, g * 4);
    S[t] = f32x4{0, 0, 0, 0};
    if (rows && here && at < dk) S[t] = *reinterpret_cast<const f32x4*>(rows + int64_t(row) * dk + at);
  }
}
template <int TILES>
__device__ __forceinline__ void chain_identity(f32x4 (&S)[TILES], int row, int g) {
#pragma unroll
  for (int t = 0; t < TILES; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) S[t][e] = chain_row(t, g * 4) + e == row ? 1.0f : 0.0f;
}
// What a first pass leaves: R in fp32, or P in two parts.
template <int TILES>
__device__ __forceinline__ void chain_leave(const DeltaLaunch& L, const DeltaItem& item, const ChainPlace& p, const f32x4 (&S)[TILES], int row, int g) {
  uint8_t* to = delta_segment(L, int(item.at) + item.seg, p.h);
  if (!p.identity) {
    if (row >= L.dv) return;
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const int at = chain_row(t, g * 4);
      if (at < L.dk) *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(to) + int64_t(row) * L.dk + at) = S[t];
    }
    return;
  }
  if (row >= L.dk) return;
  bf16* pm = reinterpret_cast<bf16*>(to + int64_t(L.dv) * L.dk * 4);
#pragma unroll
  for (int j = 0; j < TILES / 2; ++j) {
    const int at = j * 32 + g * 8;
    bf16x8 x[2];
    split8(S[2 * j], S[2 * j + 1], x);
    if (at < L.dk) {
      *reinterpret_cast<bf16x8*>(pm + row * L.dk + at) = x[0];
      *reinterpret_cast<bf16x8*>(pm + (L.dk + row) * L.dk + at) = x[1];
    }
  }
}

// The segments of a sequence and head joined: S = S P + R from the first on (or,
// for the gradient, from the last), each R replaced by the state behind it.  A
// workgroup takes 64 rows of S, in the chains' layout; P goes through LDS.  4.8 us a
// step at 128 x 128, bound by what one CU can fetch of matrices that other XCDs
// wrote (96 KB): R a step ahead and more sums at once measured the same.
template <int DK, bool BACK>
__global__ __launch_bounds__(256) void delta_join_kernel(DeltaLaunch L, int groups) {
  constexpr int TILES = DK / 16, KB = DK / 32, PIECES = 2 * DK * DK * 2 / 1024;
  __shared__ __attribute__((aligned(1024))) uint8_t ps[2][2][DK * DK * 2];
  const int group = int(blockIdx.x) % groups, h = int(blockIdx.x) / groups % L.H, b = int(blockIdx.x) / groups / L.H;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int row = group * 64 + wave * 16 + c;
  const bool mine = row < L.dv;
  const DeltaItem item = delta_whole(L, b);
  const int steps = item.segments - 1;
  if (item.b < 0 || steps <= 0) return;
  auto load = [&](int step) {
    const uint8_t* from = delta_segment(L, int(item.at) + (BACK ? steps - step : step), h) + int64_t(L.dv) * L.dk * 4;
#pragma unroll 4
    for (int i = 0; i < PIECES / 4; ++i) {
      const int piece = i * 4 + wave, part = piece / (PIECES / 2);
      int r, block;
      lds_place<DK>(piece % (PIECES / 2) * 64 + lane, r, block);
      const uint8_t* p = from + (int64_t(part * L.dk + r) * L.dk + block * 8) * 2;
      to_lds(r < L.dk && block * 8 < L.dk ? p : delta_zeros, &ps[step & 1][0][0] + piece * 1024);
    }
  };
  f32x4 S[TILES];
  const float* start = BACK ? L.dh_last : L.h0;
  if (start) start += (int64_t(b) * L.H + h) * L.dv * L.dk;
  chain_load_state<TILES>(S, start, L.dk, row, mine, g);
  load(0);
  for (int step = 0; step < steps; ++step) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (step + 1 < steps) load(step + 1);
    float* state = reinterpret_cast<float*>(delta_segment(L, int(item.at) + (BACK ? steps - step : step), h));
    f32x4 R[TILES];
    chain_load_state<TILES>(R, state, L.dk, row, mine, g);
    bf16x8 s2[KB][2];
#pragma unroll
    for (int j = 0; j < KB; ++j) split8(S[2 * j], S[2 * j + 1], s2[j]);
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      f32x4 s = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        const int r = j * 32 + g * 8 + (c >> 2), block = (t >> 1) * 4 + (c & 3), half = (t & 1) * 8;
        const int x = lds_block<DK>(r, block) + half, y = lds_block<DK>(r + 4, block) + half;
        const uint8_t *ph = ps[step & 1][0], *pl = ps[step & 1][1];
        s = mfma_split_split(lds_transposed(ph + x, ph + y), lds_transposed(pl + x, pl + y), s2[j][0], s2[j][1], s);
      }
      S[t] = R[t] + s;
    }
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const int at = chain_row(t, g * 4);
      if (mine && at < L.dk) *reinterpret_cast<f32x4*>(state + int64_t(row) * L.dk + at) = S[t];
    }
  }
}

#endif  // __HIPCC__

}  // namespace gdnq
