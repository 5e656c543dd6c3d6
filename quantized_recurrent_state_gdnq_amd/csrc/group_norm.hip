// Group norm with its activation, channels last, forward and backward (see
// gdnq_group_norm in gdnq.h).
//
//   hat = (x - mu) rstd,  n = hat w + b,  y = n f(gate) or f(n)
//   dn = dy f(gate) or dy f'(n),  dgate = dy n f'(gate)
//   dhat = dn w,  dx = rstd (dhat - [center] mean(dhat) - hat mean(dhat hat))
//   dw = sum dn hat,  db = sum dn   (over tokens; over groups too when shared)
//
// Every array is read or written once.  A group (one head of one token) is
// held in the registers of a team of TEAM lanes, EIGHTS times eight values
// each, so the statistics, the second sum of the backward pass and the outputs
// need no second read.  The variance is the mean of the centred squares, in
// fp32.
// Measured, gated bf16: 32768 x 16 groups of 128 forward 82 us (4.9 TB/s),
// backward 127 (5.3 TB/s); 16384 groups of 5120 forward 96 (5.2 TB/s).  Bound
// by memory from groups of about 48 aligned values on; not
//   below: a team has eight lanes of eight values, so of groups of 8 seven lanes
//     in eight idle (100 M values in bf16, forward and backward: groups of 8 603
//     and 999 us, of 16 284 and 486, of 24 189 and 338, of 48 101 and 182);
//   in the backward pass above 8192 values, where two eights of everything do
//     not fit the registers and 119 to 278 of a lane's are kept in scratch (100
//     M values in bf16: groups of 12288 715 us, of 16384 675, of 16383 965; 50 M
//     in fp32: 427, 420 and 465);
//   in the backward pass of unaligned bf16 (100 M values: groups of 171 283 us,
//     of 333 294, of 4999 370).
//   TEAM: the fewest lanes (8 .. 64) that hold the group with eight values
//   each; above 512 values a workgroup (TEAM = BLOCK) of as many waves as that
//   takes, with eight or sixteen values a lane (see forward_eights).
//   A lane holds eight adjacent values (16 bytes of bf16).  Where the width is
// a multiple of 8 (WIDE) they are aligned and all in the group or all out; else
// they are loaded unaligned, and the lane in which the group ends takes its last
// eight values, of which those of the lane before count once (forward and
// backward of 20000 x 4999 bf16: 583 us; 666 where that lane takes its own few
// one by one; 1499 where every lane takes every TEAM-th value, aligned).
#include <hip/hip_runtime.h>

#include "../../include/gdnq.h"
#include "device_common.h"
#include "launch.h"
#include "vec_io.h"

namespace gdnq {
namespace {

constexpr int THREADS = 256;  // of a workgroup with several teams
constexpr int BLOCK = 0;       // the team is the workgroup

template <int TEAM>
constexpr int bounds() { return TEAM == BLOCK ? 1024 : THREADS; }
template <int TEAM>
constexpr int teams_of() { return TEAM == BLOCK ? 1 : THREADS / (TEAM == BLOCK ? 1 : TEAM); }
// Whether the backward pass gives a workgroup one group of every token.
template <int TEAM>
constexpr bool by_group() { return TEAM != BLOCK && TEAM >= 16; }
template <int TEAM>
__device__ __forceinline__ int team_size() { return TEAM == BLOCK ? int(blockDim.x) : TEAM; }

// f(z) and f'(z); E: the type of the call.
template <typename E>
__device__ __forceinline__ void activation(int act, float z, float& f, float& df) {
  if (act == GDNQ_ACT_NONE) {
    f = z;
    df = 1.0f;
    return;
  }
  float p, q;
  sigmoid_pair<E>(z, p, q);
  f = act == GDNQ_ACT_SILU ? z * p : p;
  df = act == GDNQ_ACT_SILU ? p * fmaf(z, q, 1.0f) : p * q;
}

// Sum over a team: inside a wave, or over the workgroup's waves through LDS
// (box: a place of its own for every sum of a group, so that the barrier of
// the next one orders its use).
template <int TEAM>
__device__ __forceinline__ float team_sum(float x, float* box) {
  if constexpr (TEAM != BLOCK) {
    return group_sum<TEAM>(x);
  } else {
    x = group_sum<64>(x);
    if ((threadIdx.x & 63) == 0) box[threadIdx.x >> 6] = x;
    __syncthreads();
    const int waves = blockDim.x >> 6, lane = threadIdx.x & 15;
    return group_sum<16>(lane < waves ? box[lane] : 0.0f);
  }
}

// Where eighth e of lane l starts in its group: a lane in which the group ends
// starts early, so that its eight values are the group's last ones.
template <int TEAM, bool WIDE>
__device__ __forceinline__ int place(int l, int e, int D) {
  const int at = (e * team_size<TEAM>() + l) * 8;
  return !WIDE && at < D && D >= 8 ? min(at, D - 8) : at;
}
// Whether value j there is the lane's own: not also one of the lane before.
template <int TEAM, bool WIDE>
__device__ __forceinline__ bool own(int l, int e, int j, int D) {
  return WIDE || place<TEAM, WIDE>(l, e, D) + j >= (e * team_size<TEAM>() + l) * 8;
}

template <typename E, int TEAM, bool WIDE>
struct Eight {
  // as they are in memory; outside the group 0
  E v[8];
  __device__ __forceinline__ void load(const E* p, int l, int e, int D) {
    const int at = place<TEAM, WIDE>(l, e, D);
    if (at + (WIDE ? 0 : 7) < D) {
      if constexpr (WIDE) p = static_cast<const E*>(__builtin_assume_aligned(p, 16));
      __builtin_memcpy(v, p + at, sizeof(v));
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = !WIDE && at + j < D ? p[at + j] : E(0.0f);
  }
  __device__ __forceinline__ void store(E* p, int l, int e, int D) const {
    const int at = place<TEAM, WIDE>(l, e, D);
    if (at + (WIDE ? 0 : 7) < D) {
      if constexpr (WIDE) p = static_cast<E*>(__builtin_assume_aligned(p, 16));
      __builtin_memcpy(p + at, v, sizeof(v));
      return;
    }
    if constexpr (!WIDE) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at + j < D) p[at + j] = v[j];
    }
  }
};

template <int TEAM, bool WIDE, int EIGHTS>
__device__ __forceinline__ void load_params(const float* p, float other, int l, int D, float (&v)[EIGHTS][8]) {
  if (!p) {
#pragma unroll
    for (int e = 0; e < EIGHTS; ++e)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[e][j] = other;
    return;
  }
#pragma unroll
  for (int e = 0; e < EIGHTS; ++e) {
    Eight<float, TEAM, WIDE> r;
    r.load(p, l, e, D);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[e][j] = r.v[j];
  }
}

// mu and rstd of the group in v; afterwards v holds x - mu (0 outside).
template <int TEAM, bool WIDE, int EIGHTS>
__device__ __forceinline__ float normalise(const NormLaunch& L, float (&v)[EIGHTS][8], int l, float (*box)[16]) {
  const float inv = 1.0f / L.D;
  if (L.center) {
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < EIGHTS; ++e)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += own<TEAM, WIDE>(l, e, j, L.D) ? v[e][j] : 0.0f;
    const float mu = team_sum<TEAM>(s, box[0]) * inv;
#pragma unroll
    for (int e = 0; e < EIGHTS; ++e)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[e][j] = place<TEAM, WIDE>(l, e, L.D) + j < L.D ? v[e][j] - mu : 0.0f;
  }
  float s = 0.0f;
#pragma unroll
  for (int e = 0; e < EIGHTS; ++e)
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fmaf(v[e][j], own<TEAM, WIDE>(l, e, j, L.D) ? v[e][j] : 0.0f, s);
  return 1.0f / sqrtf(fmaf(team_sum<TEAM>(s, box[1]), inv, L.eps));
}

// A team takes every slots-th group from its own number on; unless all groups
// share the weights, slots is a multiple of the number of groups, so a team's
// groups have the same weights, read once.  The next group's values are
// loaded while the current one is worked on.
template <typename E, int TEAM, bool WIDE, int EIGHTS>
__global__ __launch_bounds__(bounds<TEAM>()) void norm_forward_kernel(NormLaunch L, int64_t units, int64_t slots) {
  __shared__ float box[4][16];
  int turn = 0;  // without the mean a group has one barrier: its sum's place alternates
  const int l = TEAM == BLOCK ? threadIdx.x : threadIdx.x % team_size<TEAM>(), D = L.D;
  const int64_t slot = blockIdx.x * int64_t(teams_of<TEAM>()) + threadIdx.x / team_size<TEAM>();
  if (slot >= slots) return;  // whole teams
  const E* xs = static_cast<const E*>(L.x);
  const E* gates = static_cast<const E*>(L.gate);
  Eight<E, TEAM, WIDE> x[EIGHTS], g[EIGHTS], xn[EIGHTS], gn[EIGHTS];
#pragma unroll
  for (int e = 0; e < EIGHTS; ++e) xn[e].load(xs + slot * D, l, e, D);
  if (gates) {
#pragma unroll
    for (int e = 0; e < EIGHTS; ++e) gn[e].load(gates + slot * D, l, e, D);
  }
  const int64_t wat = L.shared ? 0 : slot % L.G * D;
  float w[EIGHTS][8], b[EIGHTS][8];
  load_params<TEAM, WIDE>(L.weight ? L.weight + wat : nullptr, 1.0f, l, D, w);
  load_params<TEAM, WIDE>(L.bias ? L.bias + wat : nullptr, 0.0f, l, D, b);
  for (int64_t u = slot; u < units; u += slots, turn ^= 2) {
    const int64_t next = min(u + slots, units - 1) * D;
    float v[EIGHTS][8];
#pragma unroll
    for (int e = 0; e < EIGHTS; ++e) {
      x[e] = xn[e];
      g[e] = gn[e];
      xn[e].load(xs + next, l, e, D);
    }
    if (gates) {
#pragma unroll
      for (int e = 0; e < EIGHTS; ++e) gn[e].load(gates + next, l, e, D);
    }
#pragma unroll
    for (int e = 0; e < EIGHTS; ++e)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[e][j] = to_f32(x[e].v[j]);
    const float rstd = normalise<TEAM, WIDE>(L, v, l, box + turn);
#pragma unroll
    for (int e = 0; e < EIGHTS; ++e) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = fmaf(v[e][j] * rstd, w[e][j], b[e][j]);
        float f, df;
        activation<E>(L.act, gates ? to_f32(g[e].v[j]) : n, f, df);
        x[e].v[j] = E(gates ? n * f : f);
      }
      x[e].store(static_cast<E*>(L.y) + u * D, l, e, D);
    }
  }
}

// The teams take their groups as in the forward pass, or, with weights of
// every channel and groups wide enough (above 64 values) to be read apart from
// their neighbours, the teams of a workgroup take one group of the token each
// of the next tokens.  Either way a team adds the gradients of its weights up
// in registers, and where the workgroup's teams have the same weights they are
// added in LDS to one row of the partial sums, else a team has a row.
template <typename E, int TEAM, bool WIDE, int EIGHTS>
__global__ __launch_bounds__(bounds<TEAM>()) void norm_backward_kernel(NormLaunch L, int64_t units, int64_t slots, float* partial) {
  constexpr int TEAMS = teams_of<TEAM>();
  __shared__ float box[4][16];
  const int l = TEAM == BLOCK ? threadIdx.x : threadIdx.x % team_size<TEAM>(), D = L.D;
  const int64_t slot = blockIdx.x * int64_t(TEAMS) + threadIdx.x / team_size<TEAM>();
  const bool alike = L.shared || by_group<TEAM>();  // the workgroup's teams have the same weights
  const int64_t per_group = gridDim.x / L.G;         // workgroups (by_group)
  const int64_t group = by_group<TEAM>() && !L.shared ? blockIdx.x % L.G : slot % L.G;
  const int64_t wat = L.shared ? 0 : group * D;
  int64_t first = slot < slots ? slot : units, stride = slots;
  if (by_group<TEAM>() && !L.shared) {
    first = (blockIdx.x / L.G * TEAMS + threadIdx.x / team_size<TEAM>()) * L.G + group;
    stride = per_group * TEAMS * L.G;
  }
  float w[EIGHTS][8], b[EIGHTS][8], dw[EIGHTS][8] = {}, db[EIGHTS][8] = {};
  load_params<TEAM, WIDE>(L.weight ? L.weight + wat : nullptr, 1.0f, l, D, w);
  load_params<TEAM, WIDE>(L.bias ? L.bias + wat : nullptr, 0.0f, l, D, b);
  const E* xs = static_cast<const E*>(L.x);
  const E* gates = static_cast<const E*>(L.gate);
  const E* dys = static_cast<const E*>(L.dy);
  Eight<E, TEAM, WIDE> x[EIGHTS], g[EIGHTS], dy[EIGHTS], xn[EIGHTS], gn[EIGHTS], dyn[EIGHTS];
  // The next group's values are loaded while the current one is worked on,
  // where the registers still let four waves share a SIMD (20000 x 5120 bf16,
  // forward and backward: 394 us, 485 without; 20000 x 4999, unaligned, where
  // they do not: 727, 622 without).
  constexpr bool AHEAD = WIDE && sizeof(E) == 2;
  auto load = [&](int64_t u) {
    const int64_t at = min(u, units - 1) * D;
#pragma unroll
    for (int e = 0; e < EIGHTS; ++e) xn[e].load(xs + at, l, e, D);
    if (gates) {
#pragma unroll
      for (int e = 0; e < EIGHTS; ++e) gn[e].load(gates + at, l, e, D);
    }
#pragma unroll
    for (int e = 0; e < EIGHTS; ++e) dyn[e].load(dys + at, l, e, D);
  };
  if (AHEAD) load(first);
  for (int64_t u = first; u < units; u += stride) {
    const int64_t at = u * D;
    if (!AHEAD) load(u);
#pragma unroll
    for (int e = 0; e < EIGHTS; ++e) {
      x[e] = xn[e];
      g[e] = gn[e];
      dy[e] = dyn[e];
    }
    if (AHEAD) load(u + stride);
    float v[EIGHTS][8], d[EIGHTS][8];
#pragma unroll
    for (int e = 0; e < EIGHTS; ++e)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[e][j] = to_f32(x[e].v[j]);
    const float rstd = normalise<TEAM, WIDE>(L, v, l, box);
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int e = 0; e < EIGHTS; ++e) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float hat = v[e][j] * rstd, n = fmaf(hat, w[e][j], b[e][j]), y = to_f32(dy[e].v[j]);  // outside the group dy = 0
        float f, df;
        activation<E>(L.act, L.gate ? to_f32(g[e].v[j]) : n, f, df);
        const float dn = y * (L.gate ? f : df);
        if (L.gate) g[e].v[j] = E(y * n * df);
        dw[e][j] = fmaf(dn, hat, dw[e][j]);
        db[e][j] += dn;
        d[e][j] = dn * w[e][j];
        v[e][j] = hat;
        const float mine = own<TEAM, WIDE>(l, e, j, D) ? d[e][j] : 0.0f;
        s0 += mine;
        s1 = fmaf(mine, hat, s1);
      }
      if (L.gate) g[e].store(static_cast<E*>(L.dgate) + at, l, e, D);
    }
    const float inv = 1.0f / D;
    s0 = L.center ? team_sum<TEAM>(s0, box[2]) * inv : 0.0f;
    s1 = team_sum<TEAM>(s1, box[3]) * inv;
#pragma unroll
    for (int e = 0; e < EIGHTS; ++e) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[e].v[j] = E(rstd * fmaf(-v[e][j], s1, d[e][j] - s0));
      x[e].store(static_cast<E*>(L.dx) + at, l, e, D);
    }
  }
  if (!partial) return;
  // [2][rows][D]: dw, then db
  if constexpr (TEAMS > 1) {
    if (alike) {
      __shared__ float sums[2][TEAMS][TEAM * 8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sums[0][threadIdx.x / TEAM][l * 8 + j] = dw[0][j];
        sums[1][threadIdx.x / TEAM][l * 8 + j] = db[0][j];
      }
      __syncthreads();
      for (int i = threadIdx.x; i < 2 * TEAM * 8; i += THREADS) {
        const int which = i / (TEAM * 8), k = i % (TEAM * 8), c = place<TEAM, WIDE>(k / 8, 0, D) + k % 8;
        float s = 0.0f;
        for (int t = 0; t < TEAMS; ++t) s += sums[which][t][k];
        if (c < D && own<TEAM, WIDE>(k / 8, 0, k % 8, D)) partial[(int64_t(which) * gridDim.x + blockIdx.x) * D + c] = s;
      }
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < EIGHTS; ++e)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = place<TEAM, WIDE>(l, e, D) + j;
      if (c < D && slot < slots && own<TEAM, WIDE>(l, e, j, D)) {
        partial[slot * D + c] = dw[e][j];
        partial[(slots + slot) * D + c] = db[e][j];
      }
    }
}

// out[c] = sum over rows of partial[row][c]: a workgroup takes 16 adjacent
// columns, 64 rows at a time.
__global__ __launch_bounds__(1024) void norm_params_kernel(const float* __restrict__ partial, int64_t rows, int64_t cols,
                                                           float* dweight, float* dbias) {
  __shared__ float part[64][17];
  float* out = blockIdx.y ? dbias : dweight;
  if (!out) return;
  partial += int64_t(blockIdx.y) * rows * cols;
  const int i = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int64_t c = blockIdx.x * int64_t(16) + i;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int64_t row = r; row < rows; row += 64) s += partial[row * cols + c];
  }
  part[r][i] = s;
  __syncthreads();
  for (int n = 32; n > 0; n >>= 1) {
    if (r < n) part[r][i] += part[r + n][i];
    __syncthreads();
  }
  if (r == 0 && c < cols) out[c] = part[0][i];
}

// The team's lanes (BLOCK: threads of the workgroup).
int team_of(int D) { return D <= 64 ? 8 : D <= 128 ? 16 : D <= 256 ? 32 : D <= 512 ? 64 : BLOCK; }
int threads_of(int D, int eights) { return D <= 512 ? THREADS : (D + 512 * eights - 1) / (512 * eights) * 64; }
int teams_in(int D) { return team_of(D) == BLOCK ? 1 : THREADS / team_of(D); }

// Teams of a call: those of as many workgroups as the chip's 256 CUs hold at
// once, which then take the same number of groups each, rounded up to a
// multiple of G (the groups of a token, 1 for shared weights) so that a team's
// groups share their weights.  FORWARD_WAVES, waves of a CU in the forward
// grid, are as measured.  A grid of more than the registers hold runs a part of
// its workgroups after the others: 20000 x 4999 bf16 199 us with 32, 156 with
// 28; 20000 x 8 groups of 256 fp32 97 with 32, 94 with 28.  As many as they
// hold is not always better: above 512 values in aligned bf16 they hold 20
// (16384 x 5120: 115 us, with 16 96), up to 512 in unaligned bf16 32 (40000 x 16
// groups of 100: 94, with 28 95).
template <typename E, int TEAM, bool WIDE, int EIGHTS>
constexpr int FORWARD_WAVES = EIGHTS == 2 ? 16 : WIDE && sizeof(E) == 2 ? 32 : 28;
constexpr int BACKWARD_WAVES = 16;

// Eights of a lane where a group takes a workgroup: two above 8192 values, and
// in the forward pass
//   of aligned bf16 always, for fewer waves at a barrier (16384 x 5120: 96 us,
//   117 with one; 8192 x 5120 fp32 103 and 96);
//   of unaligned groups above 7168, of whose 15 waves a CU holds only one group
//   (16384 x 7169: 188 us, 234 with one; 16384 x 5121 158 and 130).
// The backward pass spills with two, so it takes them only above 8192 values,
// where one would need more than 1024 threads.
template <typename E, bool WIDE>
int forward_eights(int D) { return (WIDE && sizeof(E) == 2) || D > (WIDE ? 8192 : 7168) ? 2 : 1; }
int backward_eights(int D) { return D <= 8192 ? 1 : 2; }

int64_t slots_of(int64_t units, int G, int D, int eights, int waves) {
  const int own = threads_of(D, eights) / 64;
  const int64_t groups = 256 * (waves > own ? waves / own : 1);
  const int64_t most = groups * teams_in(D), want = units < most ? units : most;
  return (want + G - 1) / G * G;
}

template <typename E, int TEAM, bool WIDE, int EIGHTS>
struct Forward {
  static constexpr bool ONE = !WIDE || sizeof(E) == 4;  // whether groups of a workgroup may have one eight a lane
  static int eights(int D) { return forward_eights<E, WIDE>(D); }
  static hipError_t go(const NormLaunch& L, hipStream_t stream) {
    constexpr int TEAMS = teams_of<TEAM>();
    const int64_t units = int64_t(L.R) * L.G, slots = slots_of(units, L.shared ? 1 : L.G, L.D, EIGHTS, FORWARD_WAVES<E, TEAM, WIDE, EIGHTS>);
    norm_forward_kernel<E, TEAM, WIDE, EIGHTS><<<uint32_t((slots + TEAMS - 1) / TEAMS), threads_of(L.D, EIGHTS), 0, stream>>>(L, units, slots);
    return hipGetLastError();
  }
};

template <typename E, int TEAM, bool WIDE, int EIGHTS>
struct Backward {
  static constexpr bool ONE = true;
  static int eights(int D) { return backward_eights(D); }
  static hipError_t go(const NormLaunch& L, hipStream_t stream) {
    constexpr int TEAMS = teams_of<TEAM>();
    const int64_t units = int64_t(L.R) * L.G, slots = slots_of(units, L.shared ? 1 : L.G, L.D, EIGHTS, BACKWARD_WAVES);
    int64_t grid = (slots + TEAMS - 1) / TEAMS;
    if (by_group<TEAM>() && !L.shared) grid = (grid + L.G - 1) / L.G * L.G;
    const bool params = L.dweight || L.dbias;
    float* partial = params ? static_cast<float*>(L.workspace) : nullptr;
    if (units > 0) {
      norm_backward_kernel<E, TEAM, WIDE, EIGHTS><<<uint32_t(grid), threads_of(L.D, EIGHTS), 0, stream>>>(L, units, slots, partial);
      if (hipError_t e = hipGetLastError()) return e;
    }
    if (!params) return hipSuccess;
    // rows of D: one per workgroup whose teams have the same weights, else one
    // per team; without shared weights the groups repeat every G rows: [rows / G][G D]
    const int64_t all = L.shared || by_group<TEAM>() ? grid : slots;
    const int64_t rows = units == 0 ? 0 : L.shared ? all : all / L.G, cols = int64_t(L.shared ? 1 : L.G) * L.D;
    norm_params_kernel<<<dim3(uint32_t((cols + 15) / 16), 2), 1024, 0, stream>>>(partial, rows, cols, L.dweight, L.dbias);
    return hipGetLastError();
  }
};

template <template <typename, int, bool, int> class F, typename E, bool WIDE>
hipError_t by_width(const NormLaunch& L, hipStream_t s) {
  switch (team_of(L.D)) {
    case 8: return F<E, 8, WIDE, 1>::go(L, s);
    case 16: return F<E, 16, WIDE, 1>::go(L, s);
    case 32: return F<E, 32, WIDE, 1>::go(L, s);
    case 64: return F<E, 64, WIDE, 1>::go(L, s);
    default:
      if constexpr (F<E, BLOCK, WIDE, 1>::ONE) {
        if (F<E, BLOCK, WIDE, 1>::eights(L.D) == 1) return F<E, BLOCK, WIDE, 1>::go(L, s);
      }
      return F<E, BLOCK, WIDE, 2>::go(L, s);
  }
}

template <template <typename, int, bool, int> class F>
hipError_t dispatch(const NormLaunch& L, hipStream_t s) {
  const bool wide = L.D % 8 == 0;
  if (L.bf16) return wide ? by_width<F, bf16, true>(L, s) : by_width<F, bf16, false>(L, s);
  return wide ? by_width<F, float, true>(L, s) : by_width<F, float, false>(L, s);
}

}  // namespace

size_t norm_workspace_bytes(int R, int G, int D, bool shared) {
  return size_t(slots_of(int64_t(R) * G, shared ? 1 : G, D, backward_eights(D), BACKWARD_WAVES)) * D * 2 * 4;
}

hipError_t launch_norm_forward(const NormLaunch& L, hipStream_t stream) { return dispatch<Forward>(L, stream); }
hipError_t launch_norm_backward(const NormLaunch& L, hipStream_t stream) { return dispatch<Backward>(L, stream); }

}  // namespace gdnq
