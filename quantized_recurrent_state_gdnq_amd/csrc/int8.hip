// Matrix product in 8-bit integers with a scale for every token and channel
// (see gdnq_int_* in gdnq.h): y = (A W^T) sa sw + bias, A and W codes of the
// library's row codec, their product in whole numbers.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "../../include/gdnq.h"
#include "device_common.h"
#include "launch.h"
#include "vec_io.h"

namespace gdnq {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

template <int V>
using Int = std::integral_constant<int, V>;
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (I < N) {
    f(Int<I>{});
    each<N, I + 1>(static_cast<F&&>(f));
  }
}

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

// ---------------------------------------------------------------- the codec
//
// A row per workgroup of THREADS lanes, EIGHTS times eight values a lane held in
// registers between the largest value and the codes (EIGHTS = 0: a row longer
// than that is read twice, the second time in part out of cache).  Bound by memory:
// 16384 rows of 4096 bf16 take 40 us (36 at best), 5.0 TB/s, of 8192 fp32 126 us, 5.3;
// of 12288 fp32, read twice, 264 us, 3.8 TB/s of the bytes as read once; 64 rows 4.0.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float scale, bool finite) {
  float c[8];
  codec_codes<8>(v, scale, c);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e / 4] |= (uint32_t(int(c[e])) & 255u) << (8 * (e & 3));
  return finite ? uint2{w[0], w[1]} : uint2{0, 0};
}

template <typename E, int THREADS, int EIGHTS>
__global__ __launch_bounds__(THREADS) void int8_quantize_kernel(const E* __restrict__ x, int64_t rows, int K, int8_t* codes,
                                                                float* scales) {
  __shared__ uint32_t tops[THREADS / 64];
  const int64_t row = blockIdx.x;
  x += row * K;
  codes += row * K;
  float v[EIGHTS ? EIGHTS : 1][8];
  uint32_t top = 0;  // bits of the largest magnitude: they order as the values do, NaN above infinity
  if constexpr (EIGHTS > 0) {
#pragma unroll
    for (int i = 0; i < EIGHTS; ++i) {
      const int at = (i * THREADS + threadIdx.x) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
      if (at < K) load8(x + at, v[i]);
    }
#pragma unroll
    for (int i = 0; i < EIGHTS; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[i][e]) & 0x7fffffffu);
  } else {
    for (int at = threadIdx.x * 8; at < K; at += THREADS * 8) {
      load8(x + at, v[0]);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[0][e]) & 0x7fffffffu);
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) top = max(top, uint32_t(__shfl_xor(int(top), d)));
  if constexpr (THREADS > 64) {
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) top = max(top, tops[w]);
  }
  const bool finite = top < 0x7f800000u;
  const float scale = finite ? codec_scale<127>(__uint_as_float(top)) : __uint_as_float(0x7fc00000u);
  if (threadIdx.x == 0) scales[row] = scale;
  if constexpr (EIGHTS > 0) {
#pragma unroll
    for (int i = 0; i < EIGHTS; ++i) {
      const int at = (i * THREADS + threadIdx.x) * 8;
      if (at < K) *reinterpret_cast<uint2*>(codes + at) = codes8(v[i], scale, finite);
    }
  } else {
    for (int at = threadIdx.x * 8; at < K; at += THREADS * 8) {
      load8(x + at, v[0]);
      *reinterpret_cast<uint2*>(codes + at) = codes8(v[0], scale, finite);
    }
  }
}

// ---------------------------------------------------------------- the results
__device__ __forceinline__ float result(int acc, float sa, float sw, float bias) { return fmaf(float(acc) * sa, sw, bias); }

template <typename E>
__device__ __forceinline__ void store4(E* y, int M, int N, int m, int n, const f32x4& v) {
  if (m >= M) return;
  E* p = y + int64_t(m) * N + n;
  if (N % 4 == 0) {  // rows start on 4 elements: aligned, and in or out together
    if (n >= N) return;
    typedef E e4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<e4*>(p) = __builtin_convertvector(v, e4);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < N) store_f32(p + i, v[i]);
}

// ---------------------------------------------------------------- few rows
//
// A workgroup computes 16 columns of 16 MT rows, the depth split over its
// waves; every lane loads whole 16-byte blocks of the weights straight into the
// instruction's operand (lane l: row l % 16, block l / 16 of 16 x 64).  Bound by the
// latency of these loads: 16 x 4096 x 4096 takes 8.2 us, its weights 3.3 at a copy's rate.
template <int MT, int WAVES, int N, typename E>
__global__ __launch_bounds__(WAVES * 64) void int8_rows_kernel(Int8Launch L, int col_tiles) {
  __shared__ i32x4 sums[WAVES][MT][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x % col_tiles * 16, m0 = blockIdx.x / col_tiles * 16 * MT;
  const int blocks = L.K / 16;
  const int8_t* wc = L.w_codes + int64_t(min(n0 + r, L.N - 1)) * L.K;
  const int8_t* ac[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) ac[t] = L.a_codes + int64_t(min(m0 + t * 16 + r, L.M - 1)) * L.K;
  i32x4 acc[MT] = {};
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
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int s = 0; s < N; ++s) {
        a[t][s] = i32x4{0, 0, 0, 0};
        if (b + s < blocks) a[t][s] = *reinterpret_cast<const i32x4*>(ac[t] + int64_t(b + s) * 16);
      }
#pragma unroll
    for (int s = 0; s < N; ++s)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[s], a[t][s], acc[t], 0, 0, 0);
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) sums[wave][t][lane] = acc[t];
  __syncthreads();
  for (int t = wave; t < MT; t += WAVES) {
    i32x4 s = sums[0][t][lane];
    for (int w = 1; w < WAVES; ++w) s += sums[w][t][lane];
    const int m = m0 + t * 16 + r;
    const float sa = L.a_scales[min(m, L.M - 1)];
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int n = min(n0 + q * 4 + e, L.N - 1);
      v[e] = result(s[e], sa, L.w_scales[n], L.bias ? L.bias[n] : 0.0f);
    }
    store4<E>(static_cast<E*>(L.y), L.M, L.N, m, n0 + q * 4, v);
  }
}

// ---------------------------------------------------------------- many rows
//
// Bound by the matrix units: 16384 x 8192 x 4096 takes 492 us at best, 2.24 POPS (a
// large library product of 8-bit integers reaches 2.18 on this card, 8192 x 8192 x
// 8192), and 540, 2.04 POPS, as the median of 20 in a row; eight waves of 128 x 64
// instead of four of 128 x 128 take 1% more.
//   A workgroup computes BM x BN of y, its WGM x WGN waves an equal part each, in
// steps of DEPTH values: the step's rows of both operands are loaded straight
// into LDS, in two buffers.  The 32 x 32 x 32 instruction: lane l holds 16 bytes
// of row l % 32, of two blocks h = l / 32, and the results 8 g + 4 h + 0 .. 3 of
// column l % 32; half h takes the step's blocks of that half in turn.
//   In LDS the 16-byte blocks of a row are permuted by its number, so that the
// rows that a wave reads together at one block lie in different banks; the loads
// write LDS in lane order, so the permutation is in the address each lane loads
// from.  The operands of instruction step s + 1 are read while those of s are
// multiplied; before the last of a step's, the next step's buffer has to be
// filled and this one's reads done (one barrier a step).
//   Rows beyond the end read the last row (their results are not stored);
// blocks beyond the depth read zeros.
__device__ const uint8_t zeros[16] __attribute__((aligned(16))) = {};

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
  __device__ __forceinline__ void init(const int8_t* codes, int row0, int rows, int row_bytes, int wave, int lane) {
    base = reinterpret_cast<const uint8_t*>(codes) + int64_t(row0) * row_bytes;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int row = (i * (THREADS / 64) + wave) * PER_KB + lane / BLOCKS;
      at[i] = uint32_t(min(row, rows - 1 - row0)) * uint32_t(row_bytes) + ((lane % BLOCKS ^ swizzle<BLOCKS>(row)) << 4);
    }
  }
  // 16 bytes a lane to LDS at `to`, in lane order, as a statement that writes no
  // register: the compiler, which would wait for all such loads before any read
  // of LDS, does not know of it, and the kernel waits itself (vmcnt) before the
  // barrier that lets the buffer be read.  The s_nop is the wait that a load into
  // LDS needs behind a scalar write of M0, where the chip takes its place from.
  __device__ __forceinline__ static void to_lds(const uint8_t* base, uint32_t offset, uint8_t* to) {
    const uint32_t lds = uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)to));
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(offset), "s"(base) : "m0", "memory");
  }
  __device__ __forceinline__ static void to_lds(const uint8_t* p, uint8_t* to) {
    const uint32_t lds = uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)to));
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p) : "m0", "memory");
  }
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

template <int BM, int BN, int WGM, int WGN, int DEPTH, typename E>
__global__ __launch_bounds__(WGM* WGN * 64) void int8_tile_kernel(Int8Launch L, int row_tiles, int col_tiles) {
  constexpr int WAVES = WGM * WGN, THREADS = WAVES * 64;
  constexpr int TM = BM / WGM / 32, TN = BN / WGN / 32;  // 32 x 32 tiles of a wave
  constexpr int STEP_BLOCKS = DEPTH / 16, INSTRUCTIONS = STEP_BLOCKS / 2;
  __shared__ __attribute__((aligned(1024))) uint8_t codes[2][(BM + BN) * DEPTH];

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
  const int blocks = L.K / 16;
  Stage<BM, STEP_BLOCKS, THREADS> sa;
  Stage<BN, STEP_BLOCKS, THREADS> sw;
  sa.init(L.a_codes, m0, L.M, L.K, wave, lane);
  sw.init(L.w_codes, n0, L.N, L.K, wave, lane);
  const int full = blocks / STEP_BLOCKS, steps = (blocks + STEP_BLOCKS - 1) / STEP_BLOCKS;
  auto load_any = [&](int step) {  // a step beyond the last: none
    if (step >= steps) return;
    uint8_t* to = codes[step & 1];
    if (step < full) {
      sa.load(to, step * STEP_BLOCKS, wave);
      sw.load(to + BM * DEPTH, step * STEP_BLOCKS, wave);
      return;
    }
    sa.load_end(to, step * STEP_BLOCKS, blocks, wave, lane);
    sw.load_end(to + BM * DEPTH, step * STEP_BLOCKS, blocks, wave, lane);
  };

  i32x16 acc[TN][TM] = {};
  i32x4 a[2][TM], w[2][TN];
  constexpr int PRODUCTS = TM * TN, READS = TM + TN;  // of a wave, in an instruction step
  constexpr int LOADS = decltype(sa)::LOADS + decltype(sw)::LOADS;
  // operand n of instruction step s of `buf`
  auto fetch = [&](int buf, auto s, int n) {
    constexpr int k = s.value;
    const int slot = ((INSTRUCTIONS * h + k) ^ swizzle<STEP_BLOCKS>(r)) << 4;
    const uint8_t* at = codes[buf] + r * DEPTH + slot;
    if (n < TM)
      a[k & 1][n] = *reinterpret_cast<const i32x4*>(at + (wm + n * 32) * DEPTH);
    else
      w[k & 1][n - TM] = *reinterpret_cast<const i32x4*>(at + (BM + wn + (n - TM) * 32) * DEPTH);
  };
  // The products of instruction step s.  Between them, and kept there: the reads
  // of step f's operands (READ) and the loads of a full `load` (LOAD), a share
  // before each product.
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
            sw.load_one(to + BM * DEPTH, load * STEP_BLOCKS, wave, n - sa.LOADS);
        }
      }
      acc[j][i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(w[k & 1][j], a[k & 1][i], acc[j][i], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  // One step; LOAD: the step after the next is loaded, 1 full, 2 any; NEXT:
  // there is a next one.  The body of the main loop has no branch: the
  // compiler moves matrix instructions past one, behind the barrier.
  auto body = [&](int step, auto LOAD, auto NEXT) {
    const int buf = step & 1;
    each<INSTRUCTIONS - 1>([&](auto s) { products(s, buf, Int<s.value + 1>{}, Int<1>{}, 0, Int<0>{}); });
    if constexpr (NEXT.value != 0) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's loads into LDS
      __syncthreads();
      if constexpr (LOAD.value == 2) load_any(step + 2);
      __builtin_amdgcn_sched_barrier(0);
    }
    products(Int<INSTRUCTIONS - 1>{}, buf ^ 1, Int<0>{}, NEXT, step + 2, Int<LOAD.value == 1>{});
  };
  load_any(0);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  load_any(1);
#pragma unroll
  for (int n = 0; n < READS; ++n) fetch(0, Int<0>{}, n);
  int step = 0;
  for (; step + 2 < full; ++step) body(step, Int<1>{}, Int<1>{});
  for (; step + 1 < steps; ++step) body(step, Int<2>{}, Int<1>{});
  body(step, Int<0>{}, Int<0>{});

  // The results go through LDS, so that they leave in whole rows.  A row's
  // 16-byte pieces are permuted by its number.
  constexpr int PASSES = BM * BN * sizeof(E) <= sizeof(codes) ? 1 : 2, COLS = BN / PASSES, PITCH = COLS * sizeof(E), PIECES = PITCH / 16;
  static_assert(BM * COLS * sizeof(E) <= sizeof(codes) && BN / WGN <= COLS, "a pass fits the two buffers, a wave's columns one pass");
  static_assert(BM * PIECES % THREADS == 0, "the loop below ends with whole rows of threads");
  typedef E e4 __attribute__((ext_vector_type(4)));
  float scale_a[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i) scale_a[i] = L.a_scales[min(m0 + wm + i * 32 + r, L.M - 1)];
  uint8_t* out = codes[0];
  E* y = static_cast<E*>(L.y);
  for (int pass = 0; pass < PASSES; ++pass) {
    __syncthreads();
    int column = n0 + wn + h * 4;
    asm volatile("" : "+v"(column));  // scales are read here, not kept from before the loop: that spilled
    if (wn / COLS == pass) {
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          f32x4 scale_w, bias = {0, 0, 0, 0};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int n = min(column + j * 32 + g * 8 + e, L.N - 1);
            scale_w[e] = L.w_scales[n];
            if (L.bias) bias[e] = L.bias[n];
          }
#pragma unroll
          for (int i = 0; i < TM; ++i) {
            const int row = wm + i * 32 + r, at = (wn % COLS + j * 32 + g * 8 + h * 4) * int(sizeof(E));
            f32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = result(acc[j][i][4 * g + e], scale_a[i], scale_w[e], bias[e]);
            *reinterpret_cast<e4*>(out + row * PITCH + (((at >> 4) ^ row) & (PIECES - 1)) * 16 + (at & 15)) =
                __builtin_convertvector(v, e4);
          }
        }
    }
    __syncthreads();
    const int n = n0 + pass * COLS;
    if (int64_t(L.N) * sizeof(E) % 16 == 0) {  // whole pieces, aligned, in or out together
#pragma unroll 8
      for (int i = 0; i < BM * PIECES; i += THREADS) {
        const int p = i + threadIdx.x, row = p / PIECES, piece = p % PIECES, col = n + piece * (16 / int(sizeof(E)));
        if (m0 + row < L.M && col < L.N)  // past L2, which the operands need
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

template <int MT, int WAVES, int N, typename E>
hipError_t rows_product(const Int8Launch& L, hipStream_t stream) {
  const int cols = (L.N + 15) / 16;
  const int64_t grid = int64_t(cols) * ((L.M + 16 * MT - 1) / (16 * MT));
  int8_rows_kernel<MT, WAVES, N, E><<<uint32_t(grid), WAVES * 64, 0, stream>>>(L, cols);
  return hipGetLastError();
}

template <int BM, int BN, int WGM, int WGN, int DEPTH, typename E>
hipError_t tile_product(const Int8Launch& L, hipStream_t stream) {
  const int rows = (L.M + BM - 1) / BM, cols = (L.N + BN - 1) / BN;
  int8_tile_kernel<BM, BN, WGM, WGN, DEPTH, E><<<uint32_t(rows) * uint32_t(cols), WGM * WGN * 64, 0, stream>>>(L, rows, cols);
  return hipGetLastError();
}

// Which kernel, by the number of workgroups each would have (us for a product of
// M x N x K with the choice, and with the one it was taken over):
//   few rows, 16 of them and 16 waves: at most one workgroup per CU (16 x 4096 x
//     4096: 8.2, 32 x 32 tiles 10.2; 64 x 1024 x 8192: 9.5, 13.0 with 32 rows);
//   few rows, 32 of them: also up to 448 where the depth is small enough that
//     reading A in each of them costs little (64 x 2048 x 4096: 8.4, 32 x 32 tiles
//     10.0; 192 x 1111 x 2064: 7.3, 8.2; but 48 x 4096 x 4096, 512 of them: 13.3,
//     10.3);
//   32 x 32 tiles of one wave: at most one per CU, since a CU takes about 25 to 45
//     bytes a nanosecond and 64 x 64 tiles leave most of them idle (64 x 4096 x
//     4096: 10.4, 12.1);
//   64 x 64 tiles in steps of 256, of which a CU holds two: up to 512 (512 x 4096
//     x 4096: 15.3, 128 x 128 tiles 22.7);
//   128 x 128 tiles: up to 256 in steps of 256, one on a CU (1001 x 4096 x 4096:
//     22.6, in steps of 128 24.7, 64 x 64 28.0), else in steps of 128, two on a CU
//     (2048 x 4096 x 4096: 35.7, 256 x 256 tiles 46.8);
//   256 x 256 tiles from 192 on (4096 x 4096 x 4096: 63.5, 71.0).
template <typename E>
hipError_t matmul(const Int8Launch& L, hipStream_t stream) {
  auto count = [&](int64_t m, int64_t n) { return (L.M + m - 1) / m * ((L.N + n - 1) / n); };
  if (count(16, 16) <= 256) return rows_product<1, 16, 4, E>(L, stream);
  const int64_t rows = count(32, 16);
  if (rows <= 256 || (rows <= 448 && rows * L.K <= 1 << 20)) return rows_product<2, 8, 4, E>(L, stream);
  if (count(32, 32) <= 256) return tile_product<32, 32, 1, 1, 256, E>(L, stream);
  if (count(64, 64) <= 512) return tile_product<64, 64, 2, 2, 256, E>(L, stream);
  if (count(256, 256) >= 192) return tile_product<256, 256, 2, 2, 128, E>(L, stream);
  if (count(128, 128) <= 256) return tile_product<128, 128, 2, 2, 256, E>(L, stream);
  return tile_product<128, 128, 2, 2, 128, E>(L, stream);
}

template <typename E>
hipError_t quantize(const E* x, int64_t rows, int K, int8_t* codes, float* scales, hipStream_t stream) {
  // a workgroup of up to 256 threads per row; a launch has fewer than 2^32 threads
  constexpr int64_t PART = int64_t(1) << 23;
  for (int64_t at = 0; at < rows; at += PART) {
    const uint32_t n = uint32_t(rows - at < PART ? rows - at : PART);
    const E* from = x + at * K;
    int8_t* to = codes + at * K;
    if (K <= 512)
      int8_quantize_kernel<E, 64, 1><<<n, 64, 0, stream>>>(from, n, K, to, scales + at);
    else if (K <= 2048)
      int8_quantize_kernel<E, 256, 1><<<n, 256, 0, stream>>>(from, n, K, to, scales + at);
    else if (K <= 4096)
      int8_quantize_kernel<E, 256, 2><<<n, 256, 0, stream>>>(from, n, K, to, scales + at);
    else if (K <= 8192)
      int8_quantize_kernel<E, 256, 4><<<n, 256, 0, stream>>>(from, n, K, to, scales + at);
    else
      int8_quantize_kernel<E, 256, 0><<<n, 256, 0, stream>>>(from, n, K, to, scales + at);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_int8_quantize(const void* x, int64_t rows, int K, bool is_bf16, int8_t* codes, float* scales,
                                hipStream_t stream) {
  return is_bf16 ? quantize(static_cast<const bf16*>(x), rows, K, codes, scales, stream)
                 : quantize(static_cast<const float*>(x), rows, K, codes, scales, stream);
}

hipError_t launch_int8_matmul(const Int8Launch& L, hipStream_t stream) {
  return L.out_bf16 ? matmul<bf16>(L, stream) : matmul<float>(L, stream);
}

}  // namespace gdnq
