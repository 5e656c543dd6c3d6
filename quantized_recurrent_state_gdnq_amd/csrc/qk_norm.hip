// Norms of queries and keys for each head with the position rotation in the
// same pass, forward and backward (see gdnq_qk_norm in gdnq.h).
//
//   n = x rstd weight,  rstd = 1 / sqrt(mean(x^2) + eps)   (L2: sum(x^2))
//   y: pairs (a, b) of the first `rotary` columns turned by the token's angle,
//      (a cos - b sin, a sin + b cos)
//   backward: dy turned back, dhat = dy weight,  hat = x rstd,
//      dx = rstd (dhat - hat mean(dhat hat)),  dweight = sum dy hat
//
// Every array is read or written once: a head's row is held in the registers of
// a team of 8 .. 64 lanes.  A workgroup takes a few tokens at a time, puts the
// sines and cosines of their angles into LDS (one of each per token and pair, for
// all its heads), and its teams take the tokens' rows in turn.
//   Bound by memory where there is work: 32768 tokens of 40 heads of 128, all columns
// turned, bf16, take 149 us forward (4.5 TB/s) and 242 back (4.2), the medians of 20,
// at best 138 (4.9) and 223 (4.5); a large copy 5.14 TB/s; 64 tokens of 32 heads take
// 6.2, a launch and two dependent loads.
//   WIDE: rows of a multiple of 8 columns, 16-byte aligned: a lane holds eight
// adjacent columns, and partners half the rotated columns apart are in another
// lane's same register where that half is a multiple of 8.  Else a lane holds
// every TEAM-th column, and partners are exchanged through LDS.
#include <hip/hip_runtime.h>

#include "../../include/gdnq.h"
#include "device_common.h"
#include "launch.h"
#include "vec_io.h"

namespace gdnq {
namespace {

constexpr int THREADS = 256;
// How partners lie: none, 2i and 2i+1, through LDS, in another lane, and in the
// lane half a team away where the whole row turns and fills the team.
enum { NONE = 0, PAIRS = 1, HALVES = 2, LANES = 3, WHOLE = 4 };

// The value of lane l ^ (TEAM / 2).
template <int TEAM>
__device__ __forceinline__ float across(float x) {
  if constexpr (TEAM == 8) return dpp<0x1B>(dpp<DPP_ROW_HALF_MIRROR>(x));  // 7 - l, then reversed in its four
  if constexpr (TEAM == 16) return dpp<0x128>(x);                          // the row of 16 turned by 8
  return __shfl_xor(x, TEAM / 2);
}

// The turn of position p: angle = p f is exact or nearly so in 64 bits, and is
// brought into [-pi, pi] there; the rest is rounded to fp32 once.
__device__ __forceinline__ void turn(double angle, float& c, float& s) {
  const double n = rint(angle * 0.15915494309189535);
  const double r = fma(-n, 2.4492935982947064e-16, fma(-n, 6.283185307179586, angle));
  sincosf(float(r), &s, &c);
}

template <typename E, int TEAM, bool WIDE>
struct Row {
  static __device__ __forceinline__ int column(int l, int j) { return WIDE ? l * 8 + j : j * TEAM + l; }
  // as they are in memory; outside the row 0
  static __device__ __forceinline__ void fetch(const E* p, int l, int D, E (&x)[8]) {
    if constexpr (WIDE) {
      if (l * 8 < D) {
        __builtin_memcpy(x, __builtin_assume_aligned(p + l * 8, 16), sizeof(x));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = E(0.0f);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = column(l, j) < D ? p[column(l, j)] : E(0.0f);
    }
  }
  static __device__ __forceinline__ void store(E* p, int l, int D, const float (&v)[8]) {
    if constexpr (WIDE) {
      E x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = E(v[j]);
      if (l * 8 < D) __builtin_memcpy(__builtin_assume_aligned(p + l * 8, 16), x, sizeof(x));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (column(l, j) < D) store_f32(p + column(l, j), v[j]);
    }
  }
  static __device__ __forceinline__ void weights(const float* w, int l, int D, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = w && column(l, j) < D ? w[column(l, j)] : 1.0f;
  }
};

// Turns the row's first r columns; sign -1: back.  cs, sn: the token's table of
// r / 2 pairs; box: the team's 8 TEAM floats of LDS (HALVES).
template <int TEAM, bool WIDE, int MODE, typename R>
__device__ __forceinline__ void rotate(float (&v)[8], int l, int r, const float* cs, const float* sn, float sign, float* box) {
  if constexpr (MODE == NONE) return;
  if constexpr (MODE == WHOLE) {
    const int pair = (l & (TEAM / 2 - 1)) * 8;
    const float s = l < TEAM / 2 ? -sign : sign;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = fmaf(v[j], cs[pair + j], sn[pair + j] * s * across<TEAM>(v[j]));
    return;
  }
  const int half = r / 2;
  float other[8];
  if constexpr (MODE == PAIRS) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (WIDE)
        other[j] = v[j ^ 1];
      else
        other[j] = dpp<DPP_XOR1>(v[j]);
    }
  } else if constexpr (MODE == LANES) {
    const int from = l * 8 < half ? l + half / 8 : l - half / 8;  // a lane behind the turned columns: no matter which
#pragma unroll
    for (int j = 0; j < 8; ++j) other[j] = __shfl(v[j], from, TEAM);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) box[R::column(l, j)] = v[j];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = R::column(l, j);
      other[j] = i < r ? box[i < half ? i + half : i - half] : 0.0f;
    }
    __builtin_amdgcn_wave_barrier();
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i = R::column(l, j);
    if (i < r) {
      const int pair = MODE == PAIRS ? i >> 1 : i < half ? i : i - half;
      const bool first = MODE == PAIRS ? (i & 1) == 0 : i < half;
      const float s = sn[pair] * sign;
      v[j] = fmaf(v[j], cs[pair], (first ? -s : s) * other[j]);
    }
  }
}

// The rows of a workgroup's tokens, `heads` each, in turns of `teams`.
struct Units {
  int token, h;
  __device__ __forceinline__ Units(int team, int heads) : token(team / heads), h(team % heads) {}
  __device__ __forceinline__ void next(int teams, int heads) {
    h += teams;
    while (h >= heads) h -= heads, ++token;
  }
};

// The tokens' tables, [token][pair].
__device__ __forceinline__ void tables(const QkLaunch& L, int64_t first, int tokens, float* cs, float* sn) {
  const int half = L.rotary / 2;
  for (int i = threadIdx.x; i < tokens * half; i += THREADS) {
    const int64_t row = first + i / half;
    const double p = L.pos64 ? double(static_cast<const int64_t*>(L.positions)[row]) : double(static_cast<const int32_t*>(L.positions)[row]);
    turn(p * double(L.inv_freq[i % half]), cs[i], sn[i]);
  }
}

template <typename E, int TEAM, bool WIDE, int MODE>
__global__ __launch_bounds__(THREADS) void qk_forward_kernel(QkLaunch L) {
  typedef Row<E, TEAM, WIDE> R;
  constexpr int TEAMS = THREADS / TEAM;
  extern __shared__ float lds[];
  float* cs = lds;
  float* sn = cs + L.group * (L.rotary / 2);
  float* box = sn + L.group * (L.rotary / 2) + threadIdx.x / TEAM * (8 * TEAM);
  const int l = threadIdx.x % TEAM, team = threadIdx.x / TEAM, D = L.D;
  const int64_t first = int64_t(blockIdx.x) * L.group;
  const int tokens = int(min(int64_t(L.group), L.R - first));
  if constexpr (MODE != NONE) {
    tables(L, first, tokens, cs, sn);
    __syncthreads();
  }
  const int heads = L.Hq + L.Hk;
  const float scale = L.l2 ? 1.0f : 1.0f / D;
  float wq[8], wk[8];
  R::weights(L.q_weight, l, D, wq);
  R::weights(L.k_weight, l, D, wk);
  auto from = [&](const Units& u) {
    return u.h < L.Hq ? static_cast<const E*>(L.q) + (first + u.token) * L.q_stride + u.h * D
                      : static_cast<const E*>(L.k) + (first + u.token) * L.k_stride + (u.h - L.Hq) * D;
  };
  // a row is loaded while the one before is worked on
  Units u(team, heads);
  E x[8], ahead[8];
  if (u.token < tokens) R::fetch(from(u), l, D, x);
  while (u.token < tokens) {
    Units n = u;
    n.next(TEAMS, heads);
    if (n.token < tokens) R::fetch(from(n), l, D, ahead);
    const bool is_q = u.h < L.Hq;
    float v[8], s = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = to_f32(x[j]);
      s = fmaf(v[j], v[j], s);
    }
    const float rstd = 1.0f / sqrtf(fmaf(group_sum<TEAM>(s), scale, L.eps));
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] * rstd * (is_q ? wq[j] : wk[j]);
    rotate<TEAM, WIDE, MODE, R>(v, l, L.rotary, cs + u.token * (L.rotary / 2), sn + u.token * (L.rotary / 2), 1.0f, box);
    const int64_t row = first + u.token;
    R::store(is_q ? static_cast<E*>(L.q_out) + (row * L.Hq + u.h) * D : static_cast<E*>(L.k_out) + (row * L.Hk + u.h - L.Hq) * D,
             l, D, v);
    u = n;
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = ahead[j];
  }
}

template <typename E, int TEAM, bool WIDE, int MODE>
__global__ __launch_bounds__(THREADS) void qk_backward_kernel(QkLaunch L, float* partial) {
  typedef Row<E, TEAM, WIDE> R;
  constexpr int TEAMS = THREADS / TEAM;
  extern __shared__ float lds[];
  float* cs = lds;
  float* sn = cs + L.group * (L.rotary / 2);
  float* boxes = sn + L.group * (L.rotary / 2);
  float* box = boxes + threadIdx.x / TEAM * (8 * TEAM);
  const int l = threadIdx.x % TEAM, team = threadIdx.x / TEAM, D = L.D;
  const float scale = L.l2 ? 1.0f : 1.0f / D;
  float sums[2][8] = {};
  for (int64_t g = blockIdx.x; g * L.group < L.R; g += gridDim.x) {
    const int64_t first = g * L.group;
    const int tokens = int(min(int64_t(L.group), L.R - first));
    if constexpr (MODE != NONE) {
      __syncthreads();
      tables(L, first, tokens, cs, sn);
      __syncthreads();
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const int heads = which ? L.Hk : L.Hq;
      const int64_t stride = which ? L.k_stride : L.q_stride;
      const E* x = static_cast<const E*>(which ? L.k : L.q) + first * stride;
      const E* dy = static_cast<const E*>(which ? L.dk_out : L.dq_out) + first * heads * D;
      E* dx = static_cast<E*>(which ? L.dk : L.dq) + first * heads * D;
      float w[8];
      R::weights(which ? L.k_weight : L.q_weight, l, D, w);
      Units u(team, heads);
      for (; u.token < tokens; u.next(TEAMS, heads)) {
        E x8[8], d8[8];
        R::fetch(x + u.token * stride + u.h * D, l, D, x8);
        R::fetch(dy + (u.token * heads + u.h) * D, l, D, d8);
        float v[8], d[8], s = 0.0f, inner = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] = to_f32(x8[j]);
          d[j] = to_f32(d8[j]);
          s = fmaf(v[j], v[j], s);
        }
        const float rstd = 1.0f / sqrtf(fmaf(group_sum<TEAM>(s), scale, L.eps));
        rotate<TEAM, WIDE, MODE, R>(d, l, L.rotary, cs + u.token * (L.rotary / 2), sn + u.token * (L.rotary / 2), -1.0f, box);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] *= rstd;
          sums[which][j] = fmaf(d[j], v[j], sums[which][j]);
          d[j] *= w[j];
          inner = fmaf(d[j], v[j], inner);
        }
        inner = group_sum<TEAM>(inner) * scale;
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = rstd * fmaf(-v[j], inner, d[j]);
        R::store(dx + (u.token * heads + u.h) * D, l, D, d);
      }
    }
  }
  if (!partial) return;
  // the workgroup's sums, [2][grid][D]
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) box[R::column(l, j)] = sums[which][j];
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += THREADS) {
      float s = 0.0f;
      for (int t = 0; t < TEAMS; ++t) s += boxes[t * (8 * TEAM) + c];
      partial[(int64_t(which) * gridDim.x + blockIdx.x) * D + c] = s;
    }
  }
}

// out[c] = sum over rows of partial[row][c]: a workgroup takes 16 adjacent
// columns, 64 rows at a time.
__global__ __launch_bounds__(1024) void qk_weights_kernel(const float* __restrict__ partial, int rows, int cols, float* dq_weight,
                                                          float* dk_weight) {
  __shared__ float part[64][17];
  float* out = blockIdx.y ? dk_weight : dq_weight;
  if (!out) return;
  partial += int64_t(blockIdx.y) * rows * cols;
  const int i = threadIdx.x & 15, r = threadIdx.x >> 4, c = blockIdx.x * 16 + i;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int row = r; row < rows; row += 64) s += partial[int64_t(row) * cols + c];
  }
  part[r][i] = s;
  __syncthreads();
  for (int n = 32; n > 0; n >>= 1) {
    if (r < n) part[r][i] += part[r + n][i];
    __syncthreads();
  }
  if (r == 0 && c < cols) out[c] = part[0][i];
}

constexpr int MAX_GRID = 1024;  // of the backward pass, as many as the CUs hold: rows of partial sums

// Tokens of a workgroup: more share a launch's fixed costs and the table's
// barrier, fewer spread a small call over the chip; the table is 16 KB at most (8
// tokens, 512 columns).  As many as leave 1024 workgroups, up to 8 (us forward / back of
// 32 heads of 128, all turned, with 1, 2, 4 and 8): 64 tokens 5.1 / 4.7, 6.4 / 6.2,
// 8.8 / 9.1, 13.9 / 15.1; 2048 20.6 / 12.8, 15.1 / 11.7, 13.4 / 13.8, 16.0 / 21.1; 8192
// 67.7 / 38.4, 42.2 / 34.7, 32.5 / 34.3, 30.1 / 35.2.
int group_of(const QkLaunch& L) {
  int group = 8;
  while (group > 1 && (L.R + group - 1) / group < 1024) group /= 2;
  return group;
}

template <typename E, int TEAM, bool WIDE, int MODE>
hipError_t go(QkLaunch L, bool back, hipStream_t stream) {
  L.group = group_of(L);
  const int64_t groups = (L.R + L.group - 1) / L.group;
  const size_t lds = (size_t(L.group) * L.rotary + (back || MODE == HALVES ? THREADS * 8 : 0)) * 4;
  if (!back) {
    qk_forward_kernel<E, TEAM, WIDE, MODE><<<uint32_t(groups), THREADS, lds, stream>>>(L);
    return hipGetLastError();
  }
  const bool weights = L.dq_weight || L.dk_weight;
  float* partial = weights ? static_cast<float*>(L.workspace) : nullptr;
  const int grid = int(groups < MAX_GRID ? groups : MAX_GRID);
  if (grid > 0) {
    qk_backward_kernel<E, TEAM, WIDE, MODE><<<grid, THREADS, lds, stream>>>(L, partial);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (!weights) return hipSuccess;
  qk_weights_kernel<<<dim3((L.D + 15) / 16, 2), 1024, 0, stream>>>(partial, grid, L.D, L.dq_weight, L.dk_weight);
  return hipGetLastError();
}

template <typename E, int TEAM, bool WIDE>
hipError_t by_mode(const QkLaunch& L, bool back, hipStream_t s) {
  if (L.rotary == 0) return go<E, TEAM, WIDE, NONE>(L, back, s);
  if (L.interleaved) return go<E, TEAM, WIDE, PAIRS>(L, back, s);
  if constexpr (WIDE) {
    if (L.rotary == 8 * TEAM) return go<E, TEAM, WIDE, WHOLE>(L, back, s);
    if (L.rotary % 16 == 0) return go<E, TEAM, WIDE, LANES>(L, back, s);
  }
  return go<E, TEAM, WIDE, HALVES>(L, back, s);
}

template <typename E, bool WIDE>
hipError_t by_width(const QkLaunch& L, bool back, hipStream_t s) {
  if (L.D <= 64) return by_mode<E, 8, WIDE>(L, back, s);
  if (L.D <= 128) return by_mode<E, 16, WIDE>(L, back, s);
  if (L.D <= 256) return by_mode<E, 32, WIDE>(L, back, s);
  return by_mode<E, 64, WIDE>(L, back, s);
}

hipError_t dispatch(const QkLaunch& L, bool back, hipStream_t s) {
  const int64_t per = L.bf16 ? 8 : 4;
  const bool wide = L.D % 8 == 0 && L.q_stride % per == 0 && L.k_stride % per == 0 &&
                    reinterpret_cast<uintptr_t>(L.q) % 16 == 0 && reinterpret_cast<uintptr_t>(L.k) % 16 == 0;
  if (L.bf16) return wide ? by_width<bf16, true>(L, back, s) : by_width<bf16, false>(L, back, s);
  return wide ? by_width<float, true>(L, back, s) : by_width<float, false>(L, back, s);
}

}  // namespace

size_t qk_workspace_bytes(const QkLaunch& L) {
  const int64_t group = group_of(L), groups = (L.R + group - 1) / group;
  return size_t(groups < MAX_GRID ? groups : MAX_GRID) * 2 * L.D * 4;
}

hipError_t launch_qk_forward(const QkLaunch& L, hipStream_t stream) { return dispatch(L, false, stream); }
hipError_t launch_qk_backward(const QkLaunch& L, hipStream_t stream) { return dispatch(L, true, stream); }

}  // namespace gdnq
