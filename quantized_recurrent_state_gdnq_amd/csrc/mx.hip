// Microscaled 4-bit floating point (see gdnq_mx_* in gdnq.h): the codec and
// the product of rows in it on the scaled matrix instructions.
#include <hip/hip_runtime.h>

#include "../../include/gdnq.h"
#include "device_common.h"
#include "launch.h"
#include "vec_io.h"

namespace gdnq {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

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

// Four lanes per block of 32 values, eight values (one 4-byte word of codes)
// each.  The largest magnitude's exponent field is read from its bits (the
// bits of non-negative floats order as the values do, NaN above infinity), so
// s = field - 2, and x / scale is the product with the power of two
// 2^(127 - s), exact.  The hardware's conversion rounds to the nearest, ties
// to the even code, and saturates.
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
  const int field = int(top >> 23);
  const int s = field == 255 ? 255 : max(field - 2, 0);
  // 2^(127 - s), exponent field 254 - s; s = 254 cannot occur, 255 is NaN
  const float inv = __uint_as_float(uint32_t(254 - min(s, 253)) << 23);
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= inv;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], 1.0f, 3);
  codes[i] = w;
  if ((i & 3) == 0) scales[i >> 2] = uint8_t(s);
}

// A wave computes 16 columns x 16 MT rows of y, operands from memory to
// registers.  The matrix instruction takes 128 values of depth: lane l holds
// the 32 values (16 bytes) of one block of row l % 16 and that block's scale,
// for each of the four lane groups l / 16.  Its first operand is W and its
// second the rows of A, so a lane's four results are four adjacent columns.
template <int MT, typename E>
__global__ __launch_bounds__(64) void mx_direct_kernel(MxLaunch L) {
  const int lane = threadIdx.x, r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * MT;
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
  for (int b0 = 0; b0 < blocks; b0 += 4) {
    const bool in = b0 + q < blocks;
    const int b = in ? b0 + q : 0;
    i32x4 w = *reinterpret_cast<const i32x4*>(wc + int64_t(b) * 16);
    int sw = ws[b];
    if (!in) {
      w = i32x4{0, 0, 0, 0};
      sw = 127;
    }
    const i32x8 w8 = {w[0], w[1], w[2], w[3], 0, 0, 0, 0};
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      i32x4 a = *reinterpret_cast<const i32x4*>(ac[t] + int64_t(b) * 16);
      int sa = as[t][b];
      if (!in) {
        a = i32x4{0, 0, 0, 0};
        sa = 127;
      }
      const i32x8 a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
      acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w8, a8, acc[t], 4, 4, 0, sw, 0, sa);
    }
  }
  E* y = static_cast<E*>(L.y);
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int m = m0 + t * 16 + r;
    if (m >= L.M) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + q * 4 + i;
      if (n < L.N) store_f32(y + int64_t(m) * L.N + n, acc[t][i]);
    }
  }
}

}  // namespace

hipError_t launch_mx_quantize(const void* x, int64_t rows, int K, bool is_bf16, uint8_t* codes, uint8_t* scales,
                              hipStream_t stream) {
  const int64_t groups = rows * (K / 8);
  const uint32_t grid = uint32_t((groups + 255) / 256);
  uint32_t* words = reinterpret_cast<uint32_t*>(codes);
  if (is_bf16)
    mx_quantize_kernel<bf16><<<grid, 256, 0, stream>>>(static_cast<const bf16*>(x), groups, words, scales);
  else
    mx_quantize_kernel<float><<<grid, 256, 0, stream>>>(static_cast<const float*>(x), groups, words, scales);
  return hipGetLastError();
}

size_t mx_matmul_workspace_bytes(int, int, int) { return 0; }

hipError_t launch_mx_matmul(const MxLaunch& L, hipStream_t stream) {
  const dim3 grid((L.N + 15) / 16, (L.M + 63) / 64);
  if (L.out_bf16)
    mx_direct_kernel<4, bf16><<<grid, 64, 0, stream>>>(L);
  else
    mx_direct_kernel<4, float><<<grid, 64, 0, stream>>>(L);
  return hipGetLastError();
}

}  // namespace gdnq
