// Element types and small vectors of the channel-wise kernels (scan,
// group norm): fp32 and bf16 in memory, fp32 in registers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdnq {

typedef __bf16 bf16;
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(bf16 x) { return float(x); }
// One rounding to the nearest even (NaN stays NaN).
__device__ __forceinline__ void store_f32(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_f32(bf16* p, float x) { *p = bf16(x); }

// The smaller of p = sigmoid(z) and q = 1 - p, with the sign of z: with
// u = e^-|z| it is u / (1 + u), and the larger is formed as one minus it, so
// neither cancels.  E is the type z was stored in.
//   fp32: good to a few units in the last place: the hardware's 2^x takes
// -|z| log2(e) in two parts (product and its rounding error), its reciprocal
// one Newton step.
//   bf16: neither, 12 instruction slots instead of 21 (2^x and the reciprocal
// are four each): the smaller side is off by up to 1.25 |z| 2^-24 of itself and a
// few units.  Results in bf16 are rounded to 2^-8; the fp32 ones of such calls
// (states, their gradients, weights' gradients) carry it, beside inputs that
// were rounded to 2^-8 (20 units for a gate of e^-16).
//   Either way a smaller side under 2^-126 (|z| above 87.3) is 0.
template <typename E>
__device__ __forceinline__ float sigmoid_tail(float z) {
  if constexpr (sizeof(E) == 2) {
    const float u = __builtin_amdgcn_exp2f(-fabsf(z) * 1.44269504f);
    return copysignf(u * __builtin_amdgcn_rcpf(1.0f + u), z);
  } else {
    float m = -fabsf(z);
    m = m < -128.0f ? -128.0f : m;  // u is 0 there (infinities, the type's lowest value); NaN passes
    const float t = m * 1.44269504f;
    const float low = fmaf(m, 1.44269504f, -t) + m * 1.92596299e-8f;  // log2(e) = 1.44269504 + 1.926e-8
    const float e = __builtin_amdgcn_exp2f(t);
    const float u = fmaf(e, low * 0.693147181f, e);
    const float d = 1.0f + u;
    float r = __builtin_amdgcn_rcpf(d);
    r = fmaf(fmaf(-d, r, 1.0f), r, r);
    return copysignf(u * r, z);
  }
}

__device__ __forceinline__ void sigmoid_of_tail(float t, float& p, float& q) {
  const float small = fabsf(t), large = 1.0f - small;
  const bool up = __float_as_int(t) >= 0;  // z >= 0; a zero tail keeps its sign
  p = up ? large : small;
  q = up ? small : large;
}

// p = sigmoid(z) and q = 1 - p.
template <typename E>
__device__ __forceinline__ void sigmoid_pair(float z, float& p, float& q) {
  sigmoid_of_tail(sigmoid_tail<E>(z), p, q);
}

}  // namespace gdnq
