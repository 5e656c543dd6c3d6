// Group norm with its activation, channels last, forward and backward (see
// gdnq_group_norm in gdnq.h).
//
//   hat = (x - mu) rstd,  n = hat w + b,  y = n f(gate) or f(n)
//   dn = dy f(gate) or dy f'(n),  dgate = dy n f'(gate)
//   dhat = dn w,  dx = rstd (dhat - [center] mean(dhat) - hat mean(dhat hat))
//   dw = sum dn hat,  db = sum dn   (over tokens; over groups too when shared)
//
// One wave per (token, group), its values read again from memory in every
// pass: the plain form.
#include <hip/hip_runtime.h>

#include "../../include/gdnq.h"
#include "device_common.h"
#include "launch.h"
#include "vec_io.h"

namespace gdnq {
namespace {

// f(z) and f'(z)
__device__ __forceinline__ void activation(int act, float z, float& f, float& df) {
  if (act == GDNQ_ACT_NONE) {
    f = z;
    df = 1.0f;
    return;
  }
  float p, q;
  sigmoid_pair(z, p, q);
  f = act == GDNQ_ACT_SILU ? z * p : p;
  df = act == GDNQ_ACT_SILU ? p * fmaf(z, q, 1.0f) : p * q;
}

template <typename E>
__device__ __forceinline__ void statistics(const NormLaunch& L, const E* x, float& mu, float& rstd) {
  mu = 0.0f;
  if (L.center) {
    float s = 0.0f;
    for (int i = threadIdx.x; i < L.D; i += 64) s += to_f32(x[i]);
    mu = group_sum<64>(s) / L.D;
  }
  float s = 0.0f;
  for (int i = threadIdx.x; i < L.D; i += 64) {
    const float d = to_f32(x[i]) - mu;
    s = fmaf(d, d, s);
  }
  rstd = 1.0f / sqrtf(group_sum<64>(s) / L.D + L.eps);
}

template <typename E>
__global__ __launch_bounds__(64) void norm_forward_kernel(NormLaunch L) {
  const int64_t u = blockIdx.x;
  const int g = L.shared ? 0 : int(u % L.G);
  const E* x = static_cast<const E*>(L.x) + u * L.D;
  const E* gate = L.gate ? static_cast<const E*>(L.gate) + u * L.D : nullptr;
  E* y = static_cast<E*>(L.y) + u * L.D;
  float mu, rstd;
  statistics(L, x, mu, rstd);
  for (int i = threadIdx.x; i < L.D; i += 64) {
    const float w = L.weight ? L.weight[int64_t(g) * L.D + i] : 1.0f, b = L.bias ? L.bias[int64_t(g) * L.D + i] : 0.0f;
    const float n = fmaf((to_f32(x[i]) - mu) * rstd, w, b);
    float f, df;
    activation(L.act, gate ? to_f32(gate[i]) : n, f, df);
    store_f32(y + i, gate ? n * f : f);
  }
}

template <typename E>
__global__ __launch_bounds__(64) void norm_backward_kernel(NormLaunch L) {
  const int64_t u = blockIdx.x;
  const int g = L.shared ? 0 : int(u % L.G);
  const E* x = static_cast<const E*>(L.x) + u * L.D;
  const E* dy = static_cast<const E*>(L.dy) + u * L.D;
  const E* gate = L.gate ? static_cast<const E*>(L.gate) + u * L.D : nullptr;
  float mu, rstd;
  statistics(L, x, mu, rstd);
  if (threadIdx.x == 0) {
    static_cast<float*>(L.workspace)[2 * u] = mu;
    static_cast<float*>(L.workspace)[2 * u + 1] = rstd;
  }
  float s0 = 0.0f, s1 = 0.0f;
  for (int pass = 0; pass < 2; ++pass) {
    for (int i = threadIdx.x; i < L.D; i += 64) {
      const float w = L.weight ? L.weight[int64_t(g) * L.D + i] : 1.0f, b = L.bias ? L.bias[int64_t(g) * L.D + i] : 0.0f;
      const float hat = (to_f32(x[i]) - mu) * rstd, n = fmaf(hat, w, b), d = to_f32(dy[i]);
      float f, df;
      activation(L.act, gate ? to_f32(gate[i]) : n, f, df);
      const float dhat = d * (gate ? f : df) * w;
      if (pass == 0) {
        s0 += dhat;
        s1 = fmaf(dhat, hat, s1);
      } else {
        if (gate) store_f32(static_cast<E*>(L.dgate) + u * L.D + i, d * n * df);
        store_f32(static_cast<E*>(L.dx) + u * L.D + i, rstd * (dhat - s0 - hat * s1));
      }
    }
    if (pass == 0) {
      s0 = L.center ? group_sum<64>(s0) / L.D : 0.0f;
      s1 = group_sum<64>(s1) / L.D;
    }
  }
}

// One thread per channel of the weights, over all its tokens (and groups).
template <typename E>
__global__ __launch_bounds__(64) void norm_params_kernel(NormLaunch L) {
  const int64_t c = blockIdx.x * int64_t(64) + threadIdx.x, channels = int64_t(L.shared ? 1 : L.G) * L.D;
  if (c >= channels) return;
  const int i = int(c % L.D);
  const float w = L.weight ? L.weight[c] : 1.0f, b = L.bias ? L.bias[c] : 0.0f;
  const float* stat = static_cast<const float*>(L.workspace);
  float sw = 0.0f, sb = 0.0f;
  const int64_t units = int64_t(L.R) * L.G;
  for (int64_t u = L.shared ? 0 : c / L.D; u < units; u += L.shared ? 1 : L.G) {
    const float hat = (to_f32(static_cast<const E*>(L.x)[u * L.D + i]) - stat[2 * u]) * stat[2 * u + 1];
    float f, df;
    activation(L.act, L.gate ? to_f32(static_cast<const E*>(L.gate)[u * L.D + i]) : fmaf(hat, w, b), f, df);
    const float dn = to_f32(static_cast<const E*>(L.dy)[u * L.D + i]) * (L.gate ? f : df);
    sw = fmaf(dn, hat, sw);
    sb += dn;
  }
  if (L.dweight) L.dweight[c] = sw;
  if (L.dbias) L.dbias[c] = sb;
}

template <typename E>
hipError_t forward(const NormLaunch& L, hipStream_t stream) {
  norm_forward_kernel<E><<<uint32_t(int64_t(L.R) * L.G), 64, 0, stream>>>(L);
  return hipGetLastError();
}

template <typename E>
hipError_t backward(const NormLaunch& L, hipStream_t stream) {
  if (L.R > 0) norm_backward_kernel<E><<<uint32_t(int64_t(L.R) * L.G), 64, 0, stream>>>(L);
  if (L.dweight || L.dbias)
    norm_params_kernel<E><<<uint32_t((int64_t(L.shared ? 1 : L.G) * L.D + 63) / 64), 64, 0, stream>>>(L);
  return hipGetLastError();
}

}  // namespace

size_t norm_workspace_bytes(int R, int G, int) { return size_t(R) * G * 8; }

hipError_t launch_norm_forward(const NormLaunch& L, hipStream_t stream) {
  return L.bf16 ? forward<bf16>(L, stream) : forward<float>(L, stream);
}

hipError_t launch_norm_backward(const NormLaunch& L, hipStream_t stream) {
  return L.bf16 ? backward<bf16>(L, stream) : backward<float>(L, stream);
}

}  // namespace gdnq
