// Gated linear recurrence over channels, h_t = a_t h_{t-1} + b_t (see
// gdnq_scan_* in gdnq.h): forward with the states for the backward pass, the
// backward pass, and the single-token step.
//
// One lane per channel and sequence walks the tokens in order: the plain form
// of the definition.
#include <hip/hip_runtime.h>

#include "../../include/gdnq.h"
#include "device_common.h"
#include "launch.h"
#include "vec_io.h"

namespace gdnq {
namespace {

constexpr int CHUNK = GDNQ_SCAN_CHUNK;

// a = gate or sigmoid(gate), and keep = 1 - a without cancellation.
template <bool LOGITS>
__device__ __forceinline__ void gate_of(float g, float& a, float& keep) {
  if constexpr (LOGITS) {
    sigmoid_pair(g, a, keep);
  } else {
    a = g;
    keep = 1.0f - g;
  }
}

__device__ __forceinline__ void sequence_of(const int32_t* cu, int b, int T, int64_t N, int64_t& t0, int64_t& t1) {
  if (cu) {
    t0 = min(max(int64_t(cu[b]), int64_t(0)), N);
    t1 = min(max(int64_t(cu[b + 1]), t0), N);
  } else {
    t0 = int64_t(b) * T;
    t1 = t0 + T;
  }
}

template <typename E, bool LOGITS, bool LERP>
__global__ __launch_bounds__(64) void scan_forward_kernel(ScanLaunch L) {
  const int c = blockIdx.x * 64 + threadIdx.x;
  if (c >= L.C) return;
  const E* x = static_cast<const E*>(L.x) + c;
  const E* gate = static_cast<const E*>(L.gate) + c;
  E* y = static_cast<E*>(L.y) + c;
  for (int b = blockIdx.y; b < L.B; b += gridDim.y) {
    int64_t t0, t1;
    sequence_of(L.cu_seqlens, b, L.T, L.N, t0, t1);
    float h = L.h0 ? L.h0[int64_t(b) * L.C + c] : 0.0f;
    for (int64_t t = t0; t < t1; ++t) {
      if (L.carry && t % CHUNK == 0) L.carry[t / CHUNK * L.C + c] = h;
      float a, keep;
      gate_of<LOGITS>(to_f32(gate[t * L.C]), a, keep);
      const float v = to_f32(x[t * L.C]);
      h = fmaf(a, h, LERP ? keep * v : v);
      store_f32(y + t * L.C, h);
    }
    if (L.h_last) L.h_last[int64_t(b) * L.C + c] = h;
  }
}

// Chunk by chunk from the back: the chunk's states from its carry, then the
// reverse recurrence over it.
template <typename E, bool LOGITS, bool LERP>
__global__ __launch_bounds__(64) void scan_backward_kernel(ScanLaunch L) {
  __shared__ float before[CHUNK][64];
  const int c = blockIdx.x * 64 + threadIdx.x;
  if (c >= L.C) return;
  const E* x = static_cast<const E*>(L.x) + c;
  const E* gate = static_cast<const E*>(L.gate) + c;
  const E* dy = static_cast<const E*>(L.dy) + c;
  E* dx = static_cast<E*>(L.dx) + c;
  E* dgate = static_cast<E*>(L.dgate) + c;
  for (int b = blockIdx.y; b < L.B; b += gridDim.y) {
    int64_t t0, t1;
    sequence_of(L.cu_seqlens, b, L.T, L.N, t0, t1);
    float m = L.dh_last ? L.dh_last[int64_t(b) * L.C + c] : 0.0f;
    for (int64_t end = t1; end > t0;) {
      const int64_t begin = max(t0, (end - 1) / CHUNK * CHUNK);
      float h = begin == t0 ? (L.h0 ? L.h0[int64_t(b) * L.C + c] : 0.0f) : L.carry[begin / CHUNK * L.C + c];
      for (int64_t t = begin; t < end; ++t) {
        before[t - begin][threadIdx.x] = h;
        float a, keep;
        gate_of<LOGITS>(to_f32(gate[t * L.C]), a, keep);
        const float v = to_f32(x[t * L.C]);
        h = fmaf(a, h, LERP ? keep * v : v);
      }
      for (int64_t t = end - 1; t >= begin; --t) {
        float a, keep;
        gate_of<LOGITS>(to_f32(gate[t * L.C]), a, keep);
        const float lam = to_f32(dy[t * L.C]) + m;
        float da = before[t - begin][threadIdx.x];
        if (LERP) da -= to_f32(x[t * L.C]);
        da *= lam;
        store_f32(dgate + t * L.C, LOGITS ? da * (a * keep) : da);
        store_f32(dx + t * L.C, LERP ? keep * lam : lam);
        m = a * lam;
      }
      end = begin;
    }
    if (L.dh0) L.dh0[int64_t(b) * L.C + c] = m;
  }
}

template <typename E, bool LOGITS, bool LERP>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanLaunch L) {
  const int64_t n = int64_t(L.B) * L.C, i = blockIdx.x * int64_t(256) + threadIdx.x;
  if (i >= n) return;
  float a, keep;
  gate_of<LOGITS>(to_f32(static_cast<const E*>(L.gate)[i]), a, keep);
  const float v = to_f32(static_cast<const E*>(L.x)[i]);
  const float h = fmaf(a, L.h0[i], LERP ? keep * v : v);
  L.h_last[i] = h;
  store_f32(static_cast<E*>(L.y) + i, h);
}

// F<E, LOGITS, LERP> for the call's type and flags.
template <template <typename, bool, bool> class F>
hipError_t dispatch(const ScanLaunch& L, hipStream_t stream) {
  if (L.bf16) {
    if (L.logits) return L.lerp ? F<bf16, true, true>::go(L, stream) : F<bf16, true, false>::go(L, stream);
    return L.lerp ? F<bf16, false, true>::go(L, stream) : F<bf16, false, false>::go(L, stream);
  }
  if (L.logits) return L.lerp ? F<float, true, true>::go(L, stream) : F<float, true, false>::go(L, stream);
  return L.lerp ? F<float, false, true>::go(L, stream) : F<float, false, false>::go(L, stream);
}

template <typename E, bool LOGITS, bool LERP>
struct Forward {
  static hipError_t go(const ScanLaunch& L, hipStream_t stream) {
    scan_forward_kernel<E, LOGITS, LERP><<<dim3((L.C + 63) / 64, min(L.B, 65535)), 64, 0, stream>>>(L);
    return hipGetLastError();
  }
};

template <typename E, bool LOGITS, bool LERP>
struct Backward {
  static hipError_t go(const ScanLaunch& L, hipStream_t stream) {
    scan_backward_kernel<E, LOGITS, LERP><<<dim3((L.C + 63) / 64, min(L.B, 65535)), 64, 0, stream>>>(L);
    return hipGetLastError();
  }
};

template <typename E, bool LOGITS, bool LERP>
struct Step {
  static hipError_t go(const ScanLaunch& L, hipStream_t stream) {
    scan_step_kernel<E, LOGITS, LERP><<<uint32_t((int64_t(L.B) * L.C + 255) / 256), 256, 0, stream>>>(L);
    return hipGetLastError();
  }
};

}  // namespace

size_t scan_workspace_bytes(int64_t, int, bool) { return 0; }
hipError_t launch_scan_forward(const ScanLaunch& L, hipStream_t s) { return dispatch<Forward>(L, s); }
hipError_t launch_scan_backward(const ScanLaunch& L, hipStream_t s) { return dispatch<Backward>(L, s); }
hipError_t launch_scan_step(const ScanLaunch& L, hipStream_t s) { return dispatch<Step>(L, s); }

}  // namespace gdnq
