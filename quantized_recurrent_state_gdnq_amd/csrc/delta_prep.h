// What the chains of the trained delta rule need of every chunk and does not
// depend on the state: the inverse of I + At B (forward) or the transposed one
// of I + B At (backward), the triangle M B (so that the chain needs w alone) or
// the transpose of M, and the decays.
// One workgroup of four waves per chunk and value head, six on a CU.  Bound by
// latency: loads, the scan of the decays, sixteen dependent rows of a
// substitution and six tile products one after another (vector units 31% busy, LDS
// 24%); 8192 chunks and heads of 128 take 140 to 148 us, 26 KB written (32 backward) and
// 16 to 32 KB read each at 2.5 to 3.8 TB/s.
#pragma once

#include "delta_common.h"

namespace gdnq {

// A lower triangle of 64 x 64 fp32 in LDS: its ten 16 x 16 tiles, rows of 20.
constexpr int PREP_PITCH = 20, PREP_TILE = 16 * PREP_PITCH, PREP_FLOATS = 10 * PREP_TILE;
__device__ __forceinline__ constexpr int prep_tile(int it, int jt) { return (it * (it + 1) / 2 + jt) * PREP_TILE; }

// D += A B of such tiles: A in LDS, B in result layout; the contraction index of
// step s is 4 g + s, which a result tile holds in register s.
__device__ __forceinline__ f32x4 tile_product(const float* a, const f32x4& b, f32x4 d, int lane) {
  const f32x4 x = *reinterpret_cast<const f32x4*>(a + (lane & 15) * PREP_PITCH + (lane >> 4) * 4);
#pragma unroll
  for (int s = 0; s < 4; ++s) d = __builtin_amdgcn_mfma_f32_16x16x4f32(x[s], b[s], d, 0, 0, 0);
  return d;
}
__device__ __forceinline__ f32x4 load_tile(const float* a, int lane) {
  f32x4 x;
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = a[(4 * (lane >> 4) + e) * PREP_PITCH + (lane & 15)];
  return x;
}
__device__ __forceinline__ void store_tile(float* a, const f32x4& x, int lane, float sign) {
#pragma unroll
  for (int e = 0; e < 4; ++e) a[(4 * (lane >> 4) + e) * PREP_PITCH + (lane & 15)] = sign * x[e];
}

// (I + a)^-1 of a strictly lower triangle into n, fp32: the diagonal tiles by
// substitution, a lane per column, then [n1 0; -n2 a21 n1, n2] twice.
__device__ __forceinline__ void invert_triangle(const float* a, float* n, int wave, int lane) {
  if (lane < 16) {
    const float* block = a + prep_tile(wave, wave);
    float* to = n + prep_tile(wave, wave) + lane;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float row[16];
#pragma unroll
      for (int j = 0; j < i; j += 4) *reinterpret_cast<f32x4*>(row + j) = *reinterpret_cast<const f32x4*>(block + i * PREP_PITCH + j);
      float sum = i == lane ? 1.0f : 0.0f;
#pragma unroll
      for (int j = 0; j < i; ++j) sum = fmaf(-row[j], x[j], sum);
      x[i] = sum;
      to[i * PREP_PITCH] = sum;
    }
  }
  __syncthreads();
  if (wave < 2) {
    const int t = wave * 2;
    f32x4 p = tile_product(a + prep_tile(t + 1, t), load_tile(n + prep_tile(t, t), lane), f32x4{0, 0, 0, 0}, lane);
    p = tile_product(n + prep_tile(t + 1, t + 1), p, f32x4{0, 0, 0, 0}, lane);
    store_tile(n + prep_tile(t + 1, t), p, lane, -1.0f);
  }
  __syncthreads();
  const int rt = 2 + (wave >> 1), ct = wave & 1;
  f32x4 sum = {0, 0, 0, 0};
#pragma unroll
  for (int m = 2; m < 4; ++m) {
    if (m > rt) break;
    f32x4 p = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k < ct) continue;
      p = tile_product(a + prep_tile(m, k), load_tile(n + prep_tile(k, ct), lane), p, lane);
    }
    sum = tile_product(n + prep_tile(rt, m), p, sum, lane);
  }
  store_tile(n + prep_tile(rt, ct), sum, lane, -1.0f);
  __syncthreads();
}

// Inclusive prefix sum of the lanes in 64 bits, as wave_scan_incl.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_rows64(double x) {
  const int2 v = __builtin_bit_cast(int2, x);
  return __builtin_bit_cast(double, int2{__builtin_amdgcn_update_dpp(0, v.x, CTRL, ROWS, 0xF, false),
                                         __builtin_amdgcn_update_dpp(0, v.y, CTRL, ROWS, 0xF, false)});
}
__device__ __forceinline__ double wave_scan64(double x) {
  x += dpp_rows64<0x111, 0xF>(x);
  x += dpp_rows64<0x112, 0xF>(x);
  x += dpp_rows64<0x114, 0xF>(x);
  x += dpp_rows64<0x118, 0xF>(x);
  x += dpp_rows64<0x142, 0xA>(x);
  x += dpp_rows64<0x143, 0xC>(x);
  return x;
}

template <int DK, bool BACK>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaLaunch L) {
  constexpr int KB = DK / 32;
  __shared__ __attribute__((aligned(16))) float a[PREP_FLOATS], n[PREP_FLOATS];
  __shared__ float rest[64], beta[64];
  __shared__ int whole[64];
  int within;
  const int unit = xcd_unit(L.H / L.G, within), slot = unit / L.G, kh = unit % L.G, h = kh * (L.H / L.G) + within;
  int64_t first;
  const int tokens = delta_slot_tokens(L, slot, first);
  if (tokens == 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  uint8_t* out = static_cast<uint8_t*>(L.workspace) + (int64_t(slot) * L.H + h) * delta_chunk_bytes(BACK);

  // The decays, as log2 in 64 bits and then as a whole number and a rest, so
  // that the ratio of two tokens is good to fp32 whatever lies before them.  A
  // token's decay is at least 2^-64: what is left of a state then is below any
  // sum's rounding, and the gradient of a zero alpha can be told from it.
  if (wave == 0) {
    double x = 0.0;
    float bt = 0.0f;
    if (lane < tokens) {
      const int64_t at = (first + lane) * L.H + h;
      x = L.log_decay ? double(L.alpha[at]) * 1.4426950408889634074 : log2(double(L.alpha[at]));
      x = x < -64.0 ? -64.0 : x;
      bt = L.beta[at];
    }
    x = wave_scan64(x);
    const double w = rint(x);
    const float r = float(x - w);
    const int wi = int(w);
    rest[lane] = r;
    whole[lane] = wi;
    beta[lane] = bt;
    float* sc = reinterpret_cast<float*>(out + delta_scalars(BACK)) + lane;
    const float c1 = exp2_difference(r, wi, 0.0f, 0), tail = exp2_difference(__shfl(r, 63), __shfl(wi, 63), r, wi);
    sc[ROW_C * 64] = c1;
    sc[ROW_TAIL_BETA * 64] = tail * bt;
    sc[ROW_TAIL * 64] = tail;
    sc[ROW_C_BETA * 64] = c1 * bt;
    sc[ROW_BETA * 64] = bt;
    reinterpret_cast<int*>(sc)[ROW_WHOLE * 64] = wi;
    sc[ROW_REST * 64] = r;
  }
  // Wave it: the rows of tile it, against the tiles up to it.
  const bf16* kp = static_cast<const bf16*>(L.k) + int64_t(kh) * L.dk;
  const bf16* qp = static_cast<const bf16*>(L.q) + int64_t(kh) * L.dk;
  auto frag = [&](const bf16* p, int row, int j) {
    const int at = j * 32 + g * 8;
    const u32x4 x = *reinterpret_cast<const u32x4*>(p + (first + min(row, tokens - 1)) * (int64_t(L.G) * L.dk) + min(at, L.dk - 8));
    return __builtin_bit_cast(bf16x8, only_if(row < tokens && at < L.dk, x));
  };
  f32x4 kk[4] = {}, qk[4] = {};
#pragma unroll
  for (int j = 0; j < KB; ++j) {
    const bf16x8 kr = frag(kp, wave * 16 + c, j), qr = frag(qp, wave * 16 + c, j);
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      if (jt > wave) break;
      const bf16x8 kc = frag(kp, jt * 16 + c, j);
      kk[jt] = mfma16(kr, kc, kk[jt]);
      qk[jt] = mfma16(qr, kc, qk[jt]);
    }
  }
  __syncthreads();
  f32x4 m[4];
#pragma unroll
  for (int jt = 0; jt < 4; ++jt) {
    if (jt > wave) break;
    const int j = jt * 16 + c;
    f32x4 at;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = wave * 16 + g * 4 + e;
      const float rho = j <= i ? exp2_difference(rest[i], whole[i], rest[j], whole[j]) : 0.0f;
      m[jt][e] = BACK ? rho * qk[jt][e] : rho * qk[jt][e] * beta[j];
      at[e] = j < i ? rho * kk[jt][e] * beta[BACK ? i : j] : 0.0f;
    }
    store_tile(a + prep_tile(wave, jt), at, lane, 1.0f);
  }
  __syncthreads();
  invert_triangle(a, n, wave, lane);
#pragma unroll
  for (int jt = 0; jt < 4; ++jt)
    if (jt <= wave) store_tile(a + prep_tile(wave, jt), m[jt], lane, 1.0f);  // M in a's place
  __syncthreads();

  // Out as first operands: six blocks of each, rows in the chains' order.
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int f = wave * 3 + i, block = f % TRI_BLOCKS;
    const float* from = f < TRI_BLOCKS ? n : a;
    int it, j;
    if (!BACK) {
      it = block < 2 ? block : (block + 2) / 2;
      j = block < 2 ? 0 : block & 1;
    } else {  // transposed: tiles 0 and 1 have both blocks, 2 and 3 the second
      it = block < 4 ? block / 2 : block - 2;
      j = block < 4 ? block & 1 : 1;
    }
    const int row = chain_row(it, c), at = j * 32 + g * 8;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int r = BACK ? at + e : row, k = BACK ? row : at + e;  // at + e all lie in one tile
      x[e] = (at >> 4) > (row >> 4) == BACK || (at >> 4) == (row >> 4) ? from[prep_tile(r >> 4, k >> 4) + (r & 15) * PREP_PITCH + (k & 15)] : 0.0f;
    }
    bf16x8 parts[3];
    split3(x, parts[0], parts[1], parts[2]);
    uint8_t* to = out + (f < TRI_BLOCKS ? 0 : TRI_BYTES) + block * 1024 + lane * 16;
    *reinterpret_cast<bf16x8*>(to) = parts[0];
    *reinterpret_cast<bf16x8*>(to + TRI_PART) = parts[1];
    if (BACK && f >= TRI_BLOCKS) *reinterpret_cast<bf16x8*>(to + 2 * TRI_PART) = parts[2];
  }
}

}  // namespace gdnq
