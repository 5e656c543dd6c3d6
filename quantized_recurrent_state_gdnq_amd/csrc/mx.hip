// Microscaled 4-bit floating point (see gdnq_mx_* in gdnq.h): the codec and
// the product of rows in it on the scaled matrix instructions.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "../../include/gdnq.h"
#include "device_common.h"
#include "launch.h"
#include "vec_io.h"

namespace gdnq {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}
__device__ __forceinline__ void load8(const bf16* p, float (&v)[8]) {
  const i32x4 a = *reinterpret_cast<const i32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(uint32_t(a[i]));
    v[2 * i + 1] = bf16_hi(uint32_t(a[i]));
  }
}

// The scale byte of a block from the bits of its largest magnitude (the bits
// of non-negative floats order as the values do, NaN above infinity): its
// exponent field - 2, and 2^(127 - s), by which x / scale is an exact product.
__device__ __forceinline__ int scale_of(uint32_t top, float& inv) {
  const int field = int(top >> 23), s = field == 255 ? 255 : max(field - 2, 0);
  inv = __uint_as_float(uint32_t(254 - min(s, 253)) << 23);  // s = 254 cannot occur, 255 is NaN
  return s;
}

// The codes of eight values: the hardware's conversion rounds to the nearest,
// ties to the even code, and saturates.
__device__ __forceinline__ uint32_t eight_codes(const float (&v)[8], float inv) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0] * inv, v[1] * inv, 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2] * inv, v[3] * inv, 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4] * inv, v[5] * inv, 1.0f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6] * inv, v[7] * inv, 1.0f, 3);
}

// Four lanes per block of 32 values, eight values (one 4-byte word of codes)
// each.  Bound by memory: 16384 x 4096 bf16 in 29 us, 5.8 TB/s.
template <typename E>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const E* __restrict__ x, int64_t groups, uint32_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
  const int64_t i = blockIdx.x * int64_t(256) + threadIdx.x;  // a group of eight values
  if (i >= groups) return;  // whole blocks of four lanes leave together
  float v[8];
  load8(x + i * 8, v);
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
  top = max(top, uint32_t(__builtin_amdgcn_update_dpp(0, int(top), DPP_XOR1, 0xF, 0xF, true)));
  top = max(top, uint32_t(__builtin_amdgcn_update_dpp(0, int(top), DPP_XOR2, 0xF, 0xF, true)));
  float inv;
  const int s = scale_of(top, inv);
  codes[i] = eight_codes(v, inv);
  if ((i & 3) == 0) scales[i >> 2] = uint8_t(s);
}

// The matrix instruction takes 128 values of depth: lane l holds the 32 values
// (16 bytes) of one block of row l % 16 of its operand, and that block's
// scale, one block for each lane group q = l / 16.  Which four blocks those
// are is free as long as both operands agree.  Its first operand is W and its
// second the rows of A, so a lane's four results are four adjacent columns of
// row l % 16.  BW, BA: the byte of the scale register that is used.
template <int BW, int BA>
__device__ __forceinline__ f32x4 product(const i32x4& w, const i32x4& a, const f32x4& c, int sw, int sa) {
  const i32x8 w8 = {w[0], w[1], w[2], w[3], 0, 0, 0, 0}, a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w8, a8, c, 4, 4, BW, sw, BA, sa);
}

// f(integral constant) for 0 .. N - 1: the scale byte must be a constant.
template <int I>
struct Int {
  static constexpr int value = I;
};
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (I < N) {
    f(Int<I>{});
    each<N, I + 1>(f);
  }
}

// Four results of a lane: columns n .. n + 3 of row m.
template <typename E>
__device__ __forceinline__ void store4(E* y, int M, int N, int m, int n, const f32x4& v) {
  if (m >= M) return;
  E* p = y + int64_t(m) * N + n;
  if (N % 4 == 0) {  // rows start on 4 elements: aligned, and in or out together
    if (n >= N) return;
    if constexpr (sizeof(E) == 2) {
      typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
      *reinterpret_cast<bf16x4*>(p) = __builtin_convertvector(v, bf16x4);
    } else {
      *reinterpret_cast<f32x4*>(p) = v;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < N) store_f32(p + i, v[i]);
}

// ---------------------------------------------------------------- few rows
//
// Bound by the bytes of W.  A workgroup computes 16 columns x 16 MT rows, its
// waves a run of the depth each, operands straight from memory to registers
// (nothing is used twice but A, which the caches hold), and the waves' sums
// are added in LDS in wave order.  A lane takes N adjacent blocks of its row at
// a time: four, 64 bytes and one word of scales (single blocks with their own
// scale loads took 7.8 us for 32 x 4096 x 4096, against 5.8); where rows are
// quantized here two, so that more waves share that (1 x 4096 x 4096: 6.0 us,
// with four 7.6; 16 x 4096 x 4096: 8.0, 8.9).  As many rows in codes take two as
// well (5.4 us for 16, with four 5.0), so that mx_linear and mx_matmul of the
// same rows add in the same order.

// Scales of blocks b .. b + N - 1 of a row (beyond its end 0).
template <int N>
__device__ __forceinline__ int scales_at(const uint8_t* row, int b, int blocks) {
  uint32_t w = 0;
  if (b + N <= blocks) {
    __builtin_memcpy(&w, row + b, N);
  } else {
#pragma unroll
    for (int i = 0; i < N - 1; ++i)
      if (b + i < blocks) w |= uint32_t(row[b + i]) << (8 * i);
  }
  return int(w);
}

// A block of 32 values quantized by one lane: its scale, and its codes in w.
template <typename X>
__device__ __forceinline__ int quantize_block(const X* x, i32x4& w) {
  float v[32];
#pragma unroll
  for (int i = 0; i < 4; ++i) load8(x + 8 * i, *reinterpret_cast<float(*)[8]>(v + 8 * i));
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
  float inv;
  const int s = scale_of(top, inv);
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = int(eight_codes(*reinterpret_cast<float(*)[8]>(v + 8 * i), inv));
  return s;
}

// X: the type of A's rows where they are quantized here, in every workgroup,
// instead of by a launch of their own (void: they are codes).
template <int MT, int WAVES, int N, typename E, typename X>
__global__ __launch_bounds__(WAVES * 64) void mx_rows_kernel(MxLaunch L, int col_tiles) {
  __shared__ f32x4 sums[WAVES][MT][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x % col_tiles * 16, m0 = blockIdx.x / col_tiles * 16 * MT;
  const int blocks = L.K / 32;
  const int64_t wrow = min(n0 + r, L.N - 1);
  const uint8_t* wc = L.w_codes + wrow * (L.K / 2);
  const uint8_t* ws = L.w_scales + wrow * blocks;
  const uint8_t* ac[MT];
  const uint8_t* as[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t arow = min(m0 + t * 16 + r, L.M - 1);
    ac[t] = L.a_codes + arow * (L.K / 2);
    as[t] = L.a_scales + arow * blocks;
  }
  f32x4 acc[MT] = {};
  // runs of whole steps
  constexpr int STEP = 4 * N;
  const int steps = (blocks + STEP - 1) / STEP;
  const int first = steps * wave / WAVES, last = steps * (wave + 1) / WAVES;
  for (int step = first; step < last; ++step) {
    const int b = step * STEP + q * N;
    i32x4 w[N], a[MT][N];
#pragma unroll
    for (int s = 0; s < N; ++s) {
      w[s] = i32x4{0, 0, 0, 0};
      if (b + s < blocks) w[s] = *reinterpret_cast<const i32x4*>(wc + int64_t(b + s) * 16);
    }
    const int sw = scales_at<N>(ws, b, blocks);
    int sa[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
      for (int s = 0; s < N; ++s) a[t][s] = i32x4{0, 0, 0, 0};
      if constexpr (std::is_void_v<X>) {
#pragma unroll
        for (int s = 0; s < N; ++s)
          if (b + s < blocks) a[t][s] = *reinterpret_cast<const i32x4*>(ac[t] + int64_t(b + s) * 16);
        sa[t] = scales_at<N>(as[t], b, blocks);
      } else {
        const X* x = static_cast<const X*>(L.x) + int64_t(min(m0 + t * 16 + r, L.M - 1)) * L.K;
        sa[t] = 0;
#pragma unroll
        for (int s = 0; s < N; ++s)
          if (b + s < blocks) sa[t] |= quantize_block(x + (b + s) * 32, a[t][s]) << (8 * s);
      }
    }
    each<N>([&](auto s) {
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[t] = product<s.value, s.value>(w[s.value], a[t][s.value], acc[t], sw, sa[t]);
    });
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) sums[wave][t][lane] = acc[t];
  __syncthreads();
  for (int t = wave; t < MT; t += WAVES) {
    f32x4 s = sums[0][t][lane];
    for (int w = 1; w < WAVES; ++w) s += sums[w][t][lane];
    store4<E>(static_cast<E*>(L.y), L.M, L.N, m0 + t * 16 + r, n0 + q * 4, s);
  }
}

// ---------------------------------------------------------------- many rows
//
// Bound by the matrix units: 16384 x 8192 x 4096 takes 314 us of a call, 3.5
// PFLOP/s (under the profiler 325 to 348).  A step of 256 x 256 x 256 takes 1.76
// us, at the instruction's own rate 0.85; without its loads into LDS 1.39; the
// clock falls to 2.0 GHz meanwhile.  A tile costs 11 us beside its 16 steps, more
// than half of it to write its results; a CU works on one tile at a time, and
// nothing of that is hidden.
//   A workgroup computes BM x BN of y, its WGM x WGN
// waves an equal part each, in steps of DEPTH values (256, or 512 for small
// tiles): the step's rows of both operands are loaded straight into LDS, in two
// buffers.
//   The 32 x 32 x 64 instruction: lane l holds one block of row l % 32, of two
// blocks h = l / 32, and the results 8 g + 4 h + 0 .. 3 of column l % 32.  It
// reaches 9.5 PFLOP/s in a loop of its own, 16 x 16 x 128 only 4.8.  Half h
// takes the step's blocks of that half in turn, so four scale bytes are one
// word and the instruction step selects the byte.
//   In LDS the 16-byte blocks of a row are permuted by its number, so
// that the rows that a wave reads together at one block lie in different
// banks; the loads write LDS in lane order, so the permutation is in the
// address each lane loads from.
//   The operands of instruction step s + 1 are read from LDS while those of s
// are multiplied.  Before the last of a step's, the next step's buffer
// has to be filled and this one's reads done (one barrier a step); then the
// loads for the step after go into this one.
//   Rows beyond the end read the last row (their results are not stored);
// blocks beyond the depth read zeros.
__device__ const uint8_t zeros[16] __attribute__((aligned(16))) = {};

// What a row's block number is permuted by: the same for rows 16 apart.
template <int BLOCKS>
__device__ __forceinline__ int swizzle(int row) {
  return BLOCKS == 8 ? (row ^ (row >> 3 & 1)) & 7 : row & 15;
}

// One operand's ROWS rows of a step of BLOCKS blocks, 1 KB per wave and load.
template <int ROWS, int BLOCKS, int THREADS>
struct Stage {
  static constexpr int LOADS = ROWS * BLOCKS / THREADS, PER_KB = 64 / BLOCKS;
  const uint8_t* base;  // of the tile's first row
  uint32_t at[LOADS];   // the lane's block of its rows in a step
  __device__ __forceinline__ void init(const uint8_t* codes, int row0, int rows, int row_bytes, int wave, int lane) {
    base = codes + int64_t(row0) * row_bytes;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int row = (i * (THREADS / 64) + wave) * PER_KB + lane / BLOCKS;
      at[i] = uint32_t(min(row, rows - 1 - row0)) * uint32_t(row_bytes) + ((lane % BLOCKS ^ swizzle<BLOCKS>(row)) << 4);
    }
  }
  // 16 bytes a lane from p (base and the lane's offset) to LDS at `to`, in lane
  // order.  As an empty-handed statement (it writes no register), because the
  // compiler waits for all such loads before any read of LDS when it knows of
  // them, whichever buffer is read; the kernel waits itself (vmcnt) before the
  // barrier that lets the buffer be read.  The s_nop is the wait that a load
  // into LDS needs behind a scalar write of M0, where the chip takes its place
  // in LDS from; inside a statement the compiler adds none.  The compiler warns
  // that M0 is a reserved register: nothing else in this file uses it.
  __device__ __forceinline__ static void to_lds(const uint8_t* base, uint32_t offset, uint8_t* to) {
    const uint32_t lds = uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)to));
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(offset), "s"(base) : "m0", "memory");
  }
  __device__ __forceinline__ static void to_lds(const uint8_t* p, uint8_t* to) {
    const uint32_t lds = uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)to));
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p) : "m0", "memory");
  }
  // Loads the step from block k0 on to LDS at `to`.
  __device__ __forceinline__ void load(uint8_t* to, int k0, int wave) const {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) load_one(to, k0, wave, i);
  }
  __device__ __forceinline__ void load_one(uint8_t* to, int k0, int wave, int i) const {
    to_lds(base + int64_t(k0) * 16, at[i], to + (i * (THREADS / 64) + wave) * 1024);
  }
  // The same where the depth ends inside the step.
  __device__ __forceinline__ void load_end(uint8_t* to, int k0, int blocks, int wave, int lane) const {
    const uint8_t* from = base + int64_t(k0) * 16;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int piece = i * (THREADS / 64) + wave, row = piece * PER_KB + lane / BLOCKS;
      to_lds(k0 + (lane % BLOCKS ^ swizzle<BLOCKS>(row)) < blocks ? from + at[i] : zeros, to + piece * 1024);
    }
  }
};

template <int BW, int BA>
__device__ __forceinline__ f32x16 wide_product(const i32x4& w, const i32x4& a, const f32x16& c, int sw, int sa) {
  const i32x8 w8 = {w[0], w[1], w[2], w[3], 0, 0, 0, 0}, a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w8, a8, c, 4, 4, BW, sw, BA, sa);
}

template <int BM, int BN, int WGM, int WGN, int DEPTH, typename E>
__global__ __launch_bounds__(WGM* WGN * 64) void mx_tile_kernel(MxLaunch L, int row_tiles, int col_tiles) {
  constexpr int WAVES = WGM * WGN, THREADS = WAVES * 64;
  constexpr int TM = BM / WGM / 32, TN = BN / WGN / 32;  // 32 x 32 tiles of a wave
  constexpr int STEP_BYTES = DEPTH / 2, STEP_BLOCKS = DEPTH / 32;  // of a row
  constexpr int INSTRUCTIONS = STEP_BLOCKS / 2, WORDS = STEP_BLOCKS / 8;  // of a step; a half's words of scales
  static_assert(BM * BN <= (BM + BN) * STEP_BYTES, "the results of a pass fit the two buffers");
  constexpr int SCALE_ROWS = BM + BN > THREADS ? (BM + BN) / THREADS : 1;  // that a thread stages
  static_assert((SCALE_ROWS * THREADS) % (BM + BN) == 0, "every row's scales are staged");
  __shared__ __attribute__((aligned(1024))) uint8_t codes[2][(BM + BN) * STEP_BYTES];
  __shared__ uint64_t scales[2][BM + BN][WORDS];

  // Tiles in bands: the workgroups of one XCD (every eighth) take adjacent
  // ones, down GROUP rows of tiles and then to the right, so that its L2 holds
  // the operands they share.
  constexpr int GROUP = 8;
  const int tiles = row_tiles * col_tiles, b = blockIdx.x;
  const int per = tiles / 8, extra = tiles % 8, x = b % 8;
  const int id = x * per + min(x, extra) + b / 8;
  const int band = id / (GROUP * col_tiles), in_band = id % (GROUP * col_tiles);
  const int rows_here = min(GROUP, row_tiles - band * GROUP);
  const int m0 = (band * GROUP + in_band % rows_here) * BM, n0 = in_band / rows_here * BN;

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
  const int wm = wave % WGM * (BM / WGM), wn = wave / WGM * (BN / WGN);
  const int blocks = L.K / 32, row_bytes = L.K / 2;
  Stage<BM, STEP_BLOCKS, THREADS> sa;
  Stage<BN, STEP_BLOCKS, THREADS> sw;
  sa.init(L.a_codes, m0, L.M, row_bytes, wave, lane);
  sw.init(L.w_codes, n0, L.N, row_bytes, wave, lane);
  // thread t stages the scales of rows t, t + THREADS .. of A's tile, then W's
  const int t = threadIdx.x % (BM + BN);
  const uint8_t* scale_row[SCALE_ROWS];
#pragma unroll
  for (int q = 0; q < SCALE_ROWS; ++q) {
    const int row = t + q * THREADS;
    scale_row[q] = row < BM ? L.a_scales + int64_t(min(m0 + row, L.M - 1)) * blocks
                            : L.w_scales + int64_t(min(n0 + row - BM, L.N - 1)) * blocks;
  }
  const int full = blocks / STEP_BLOCKS, steps = (blocks + STEP_BLOCKS - 1) / STEP_BLOCKS;
  uint64_t staged[SCALE_ROWS][WORDS] = {};
  auto load_scales = [&](int step) {
#pragma unroll
    for (int q = 0; q < SCALE_ROWS; ++q) __builtin_memcpy(staged[q], scale_row[q] + step * STEP_BLOCKS, sizeof(staged[q]));
  };
  auto load_any = [&](int step) {  // a step beyond the last: none
    if (step >= steps) return;
    uint8_t* to = codes[step & 1];
    if (step < full) {
      sa.load(to, step * STEP_BLOCKS, wave);
      sw.load(to + BM * STEP_BYTES, step * STEP_BLOCKS, wave);
      load_scales(step);
      return;
    }
    sa.load_end(to, step * STEP_BLOCKS, blocks, wave, lane);
    sw.load_end(to + BM * STEP_BYTES, step * STEP_BLOCKS, blocks, wave, lane);
#pragma unroll
    for (int q = 0; q < SCALE_ROWS; ++q)
#pragma unroll
      for (int k = 0; k < WORDS; ++k) {
        staged[q][k] = 0;
#pragma unroll 1
        for (int i = step * STEP_BLOCKS + 8 * k, n = 0; n < 8 && i + n < blocks; ++n)
          staged[q][k] |= uint64_t(scale_row[q][i + n]) << (8 * n);
      }
  };
  auto put_scales = [&](int buf) {
#pragma unroll
    for (int q = 0; q < SCALE_ROWS; ++q)
#pragma unroll
      for (int k = 0; k < WORDS; ++k) scales[buf][t + q * THREADS][k] = staged[q][k];
  };

  f32x16 acc[TN][TM] = {};
  i32x4 a[2][TM], w[2][TN];
  int sca[TM][WORDS], scw[TN][WORDS], next_sca[TM][WORDS], next_scw[TN][WORDS];
  constexpr int PRODUCTS = TM * TN, READS = TM + TN;  // of a wave, in an instruction step
  constexpr int LOADS = decltype(sa)::LOADS + decltype(sw)::LOADS;
  // operand n of instruction step s of `buf`
  auto fetch = [&](int buf, auto s, int n) {
    constexpr int k = s.value;
    const int slot = ((INSTRUCTIONS * h + k) ^ swizzle<STEP_BLOCKS>(r)) << 4;
    const uint8_t* at = codes[buf] + r * STEP_BYTES + slot;
    if (n < TM)
      a[k & 1][n] = *reinterpret_cast<const i32x4*>(at + (wm + n * 32) * STEP_BYTES);
    else
      w[k & 1][n - TM] = *reinterpret_cast<const i32x4*>(at + (BM + wn + (n - TM) * 32) * STEP_BYTES);
  };
  auto fetch_scales = [&](int buf) {
    const int* p = reinterpret_cast<const int*>(scales[buf]);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int k = 0; k < WORDS; ++k) next_sca[i][k] = p[((wm + i * 32 + r) * 2 + h) * WORDS + k];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int k = 0; k < WORDS; ++k) next_scw[i][k] = p[((BM + wn + i * 32 + r) * 2 + h) * WORDS + k];
  };
  // The products of instruction step s.  Between them, and kept there: the reads
  // of step f's operands (READ) and the loads of a full `load` (LOAD), a share
  // before each product.  All at once ahead of the products they held these up
  // until the queues of LDS and of the loads had room (16384 x 8192 x 4096: 346
  // us, with waves of 128 x 128 333, with the reads and loads between 321).
  auto products = [&](auto s, int buf, auto f, auto READ, int load, auto LOAD) {
    constexpr int k = s.value;
    each<PRODUCTS>([&](auto q) {
      constexpr int j = q.value / TM, i = q.value % TM;
      if constexpr (READ.value != 0) {
        constexpr int SHARE = (READS + PRODUCTS - 1) / PRODUCTS;
#pragma unroll
        for (int n = q.value * SHARE; n < min((q.value + 1) * SHARE, READS); ++n) fetch(buf, f, n);
      }
      if constexpr (LOAD.value != 0) {
        constexpr int SHARE = (LOADS + PRODUCTS - 1) / PRODUCTS;
        uint8_t* to = codes[load & 1];
#pragma unroll
        for (int n = q.value * SHARE; n < min((q.value + 1) * SHARE, LOADS); ++n) {
          if (n < sa.LOADS)
            sa.load_one(to, load * STEP_BLOCKS, wave, n);
          else
            sw.load_one(to + BM * STEP_BYTES, load * STEP_BLOCKS, wave, n - sa.LOADS);
        }
      }
      acc[j][i] = wide_product<k & 3, k & 3>(w[k & 1][j], a[k & 1][i], acc[j][i], scw[j][k / 4], sca[i][k / 4]);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  // One step; LOAD: the step after the next is loaded, 1 full, 2 any; NEXT:
  // there is a next one.  The body of the main loop has no branch: the
  // compiler moves matrix instructions past one, behind the barrier.
  auto body = [&](int step, auto LOAD, auto NEXT) {
    const int buf = step & 1;
#pragma unroll
    for (int k = 0; k < WORDS; ++k) {
#pragma unroll
      for (int i = 0; i < TM; ++i) sca[i][k] = next_sca[i][k];
#pragma unroll
      for (int i = 0; i < TN; ++i) scw[i][k] = next_scw[i][k];
    }
    each<INSTRUCTIONS - 1>([&](auto s) { products(s, buf, Int<s.value + 1>{}, Int<1>{}, 0, Int<0>{}); });
    if constexpr (NEXT.value != 0) {
      put_scales(buf ^ 1);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's loads into LDS
      __syncthreads();
      if constexpr (LOAD.value == 1) load_scales(step + 2);
      if constexpr (LOAD.value == 2) load_any(step + 2);
      fetch_scales(buf ^ 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    products(Int<INSTRUCTIONS - 1>{}, buf ^ 1, Int<0>{}, NEXT, step + 2, Int<LOAD.value == 1>{});
  };
  load_any(0);
  put_scales(0);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  load_any(1);
#pragma unroll
  for (int n = 0; n < READS; ++n) fetch(0, Int<0>{}, n);
  fetch_scales(0);
  int step = 0;
  for (; step + 2 < full; ++step) body(step, Int<1>{}, Int<1>{});
  for (; step + 1 < steps; ++step) body(step, Int<2>{}, Int<1>{});
  body(step, Int<0>{}, Int<0>{});

  // The results go through LDS (BN 2-byte or half as many 4-byte values a row
  // at a time) so that they leave in whole rows: stored from the lanes, 16
  // bytes a row, they took 13 us of a tile's 52.  A row's 16-byte pieces are
  // permuted by its number.
  constexpr int PASSES = sizeof(E) / 2, COLS = BN / PASSES, PITCH = COLS * sizeof(E), PIECES = PITCH / 16;
  static_assert(BM * PIECES % THREADS == 0, "the loop below ends with whole rows of threads");
  typedef E e4 __attribute__((ext_vector_type(4)));
  uint8_t* out = codes[0];
  E* y = static_cast<E*>(L.y);
  for (int pass = 0; pass < PASSES; ++pass) {
    __syncthreads();
    if (wn / COLS == pass) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int row = wm + i * 32 + r, at = (wn % COLS + j * 32 + g * 8 + h * 4) * int(sizeof(E));
            const f32x4 v = {acc[j][i][4 * g], acc[j][i][4 * g + 1], acc[j][i][4 * g + 2], acc[j][i][4 * g + 3]};
            *reinterpret_cast<e4*>(out + row * PITCH + (((at >> 4) ^ row) & (PIECES - 1)) * 16 + (at & 15)) =
                __builtin_convertvector(v, e4);
          }
    }
    __syncthreads();
    const int n = n0 + pass * COLS;
    if (int64_t(L.N) * sizeof(E) % 16 == 0) {  // whole pieces, aligned, in or out together
#pragma unroll 8
      for (int i = 0; i < BM * PIECES; i += THREADS) {
        const int p = i + threadIdx.x, row = p / PIECES, piece = p % PIECES, col = n + piece * (16 / int(sizeof(E)));
        if (m0 + row < L.M && col < L.N)  // past L2, which the operands need (16384 x 8192 x 8192: 621 us, 612)
          __builtin_nontemporal_store(
              *reinterpret_cast<const i32x4*>(out + row * PITCH + ((piece ^ row) & (PIECES - 1)) * 16),
              reinterpret_cast<i32x4*>(y + int64_t(m0 + row) * L.N + col));
      }
    } else {
      for (int p = threadIdx.x; p < BM * COLS; p += THREADS) {
        const int row = p / COLS, at = p % COLS * int(sizeof(E)), col = n + p % COLS;
        if (m0 + row < L.M && col < L.N)
          y[int64_t(m0 + row) * L.N + col] =
              *reinterpret_cast<const E*>(out + row * PITCH + (((at >> 4) ^ row) & (PIECES - 1)) * 16 + (at & 15));
      }
    }
  }
}

template <int MT, int WAVES, int N, typename E, typename X>
hipError_t rows_product(const MxLaunch& L, hipStream_t stream) {
  const int cols = (L.N + 15) / 16;
  const int64_t grid = int64_t(cols) * ((L.M + 16 * MT - 1) / (16 * MT));
  mx_rows_kernel<MT, WAVES, N, E, X><<<uint32_t(grid), WAVES * 64, 0, stream>>>(L, cols);
  return hipGetLastError();
}

template <int BM, int BN, int WGM, int WGN, int DEPTH, typename E>
hipError_t tile_product(const MxLaunch& L, hipStream_t stream) {
  const int rows = (L.M + BM - 1) / BM, cols = (L.N + BN - 1) / BN;
  mx_tile_kernel<BM, BN, WGM, WGN, DEPTH, E><<<uint32_t(rows) * uint32_t(cols), WGM * WGN * 64, 0, stream>>>(L, rows, cols);
  return hipGetLastError();
}

// Up to FUSED_ROWS rows are quantized inside the product where it has at most
// one workgroup per CU: one launch less, and 16 rows are little to quantize
// again in every workgroup; at 64 rows that took longer than the launch.  (us
// on the GPU, one launch and two, 1 and 16 rows: 4096 columns x 512: 3.7 and 3.9,
// 4.4 and 4.6; x 4096: 6.0 and 7.9, 6.1 and 7.5; x 8192: 10.4 and 15.1, 9.3 and
// 11.3, where the second launch's 2 us of host time still make up for it.  With
// more columns a CU quantizes the rows again and again: 16384 x 4096: 19.4 and
// 28.2, 13.2 and 13.0; 32768 x 4096: 34.9 and 55.0, 17.7 and 17.7.)
constexpr int FUSED_ROWS = 16;
bool fused(const MxLaunch& L) { return L.M <= FUSED_ROWS && L.N <= 256 * 16; }

// Which kernel, by the number of workgroups each would have (us for a product
// of M x N x K with the choice, and with the one it was taken over):
//   few rows, 16 of them and 16 waves: at most one workgroup per CU
//     (16 x 4096 x 4096: 4.6, 64 x 64 tiles 6.3; 64 x 1024 x 8192: 6.9, 10.0);
//     for up to 16 rows two per CU from a depth of 1024 on (1 and 16 rows x 8192 x
//     4096: 6.8 and 8.4, by the rules below 9.9 and 10.0; x 8192 x 1024: 3.5 and
//     4.0, 4.0 and 4.1; but x 4112 x 512: 2.9 and 3.0, 2.8 and 2.9);
//   few rows, 32 of them: also up to 448 where the depth is small enough that
//     reading A in each of them costs little (32 x 4096 x 4096: 5.7, 6.3; 192 x
//     1111 x 2080: 4.3, 7.1; but 192 x 1024 x 8192: 15.6, 10.3; the border
//     between them rests on these three);
//   64 x 64 tiles, of which a CU holds two: up to 512, in steps of 512, since a
//     step takes its loads' latency (64 x 4096 x 4096: 6.5, in steps of 256
//     8.1, 128 x 128 tiles 11.9; 512 x 4096 x 4096: 11.6, 128 x 128 13.0);
//   128 x 128 tiles: up to 256 in steps of 512, one on a CU (1001 x 4096 x
//     4096: 15.1, 17.8), else in steps of 256, two on a CU (2048 x 4096 x
//     4096: 28.3, 31.3);
//   256 x 256 tiles from 192 on (4096 x 4096 x 4096: 42.7, 52.4; 2048 x 4096 x
//     4096, 128 of them: 33.1, 28.3).
template <typename E>
hipError_t matmul(const MxLaunch& L, hipStream_t stream) {
  auto count = [&](int64_t m, int64_t n) { return (L.M + m - 1) / m * ((L.N + n - 1) / n); };
  if (L.M <= FUSED_ROWS && count(16, 16) <= (L.K >= 1024 ? 512 : 256)) return rows_product<1, 16, 2, E, void>(L, stream);
  if (count(16, 16) <= 256) return rows_product<1, 16, 4, E, void>(L, stream);
  const int64_t rows = count(32, 16);
  if (rows <= 256 || (rows <= 448 && rows * L.K <= 1 << 20)) return rows_product<2, 8, 4, E, void>(L, stream);
  if (count(64, 64) <= 512) return tile_product<64, 64, 2, 2, 512, E>(L, stream);
  if (count(256, 256) >= 192) return tile_product<256, 256, 2, 2, 256, E>(L, stream);
  if (count(128, 128) <= 256) return tile_product<128, 128, 2, 2, 512, E>(L, stream);
  return tile_product<128, 128, 2, 2, 256, E>(L, stream);
}

}  // namespace

hipError_t launch_mx_quantize(const void* x, int64_t rows, int K, bool is_bf16, uint8_t* codes, uint8_t* scales,
                              hipStream_t stream) {
  // a thread per eight values; a launch has fewer than 2^32 threads
  constexpr int64_t PART = int64_t(1) << 31;
  const int64_t groups = rows * (K / 8);
  for (int64_t at = 0; at < groups; at += PART) {
    const int64_t n = groups - at < PART ? groups - at : PART;
    const uint32_t grid = uint32_t((n + 255) / 256);
    uint32_t* words = reinterpret_cast<uint32_t*>(codes) + at;
    if (is_bf16)
      mx_quantize_kernel<bf16><<<grid, 256, 0, stream>>>(static_cast<const bf16*>(x) + at * 8, n, words, scales + at / 4);
    else
      mx_quantize_kernel<float><<<grid, 256, 0, stream>>>(static_cast<const float*>(x) + at * 8, n, words, scales + at / 4);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

hipError_t launch_mx_matmul(const MxLaunch& L, hipStream_t stream) {
  return L.out_bf16 ? matmul<bf16>(L, stream) : matmul<float>(L, stream);
}

hipError_t launch_mx_linear(const MxLaunch& L, hipStream_t stream) {
  if (fused(L)) {
    if (L.in_bf16) return L.out_bf16 ? rows_product<1, 16, 2, bf16, bf16>(L, stream) : rows_product<1, 16, 2, float, bf16>(L, stream);
    return L.out_bf16 ? rows_product<1, 16, 2, bf16, float>(L, stream) : rows_product<1, 16, 2, float, float>(L, stream);
  }
  if (hipError_t e = launch_mx_quantize(L.x, L.M, L.K, L.in_bf16, const_cast<uint8_t*>(L.a_codes),
                                        const_cast<uint8_t*>(L.a_scales), stream))
    return e;
  return launch_mx_matmul(L, stream);
}

}  // namespace gdnq
