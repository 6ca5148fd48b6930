// expert.cuh -- what the expert kernels share: the segments of a receive layout
// and the activations.
#pragma once

#include "ep_common.cuh"

namespace ep {

// The rows of every expert in a receive layout (normal: psum != nullptr;
// packed: each expert owns cap rows).
struct Segments {
  const int32_t* counts;   // [E]
  const int64_t* psum;     // [R, E_l + 1] or nullptr
  int E, E_l;
  int64_t cap;             // rows per rank (normal) or per expert (packed)
  int32_t* status;
};

struct Segment {
  int64_t start;   // first row
  int32_t count;
};

// Expert e's rows, cut to the buffer (a cut is reported as a capacity error).
__device__ __forceinline__ Segment segment_of(const Segments& s, int e) {
  int64_t base = 0, off = 0;
  if (s.psum != nullptr) {
    const int r = e / s.E_l, l = e - r * s.E_l;
    base = (int64_t)r * s.cap;
    off = s.psum[(int64_t)r * (s.E_l + 1) + l];
  } else {
    base = (int64_t)e * s.cap;
  }
  int64_t n = s.counts[e];
  if (off < 0 || off > s.cap) {
    if (n > 0) set_status(s.status, EP_ERR_CAPACITY);
    return {base, 0};
  }
  if (n < 0) n = 0;
  if (n > s.cap - off) {
    set_status(s.status, EP_ERR_CAPACITY);
    n = s.cap - off;
  }
  return {base + off, (int32_t)n};
}

// The ue8m0 byte of a 128-channel block whose largest magnitude is amax, as
// dispatch quantises: amax / 448 rounded up to a power of two, amax floored at
// 1e-4 and capped at the largest finite float.
__device__ __forceinline__ uint32_t ue8m0_of(float amax) {
  amax = fminf(fmaxf(amax, 1e-4f), 3.40282346638528859812e+38f);
  const uint32_t bits = __float_as_uint(__fdiv_rn(amax, 448.0f));
  return ((bits >> 23) & 0xffu) + ((bits & 0x7fffffu) ? 1u : 0u);
}

// ---------------------------------------------------------------- activations

// g = exp(-z^2 / 2) and Phi(z), the normal distribution up to z.  Its tail is
// Phi(-|z|) = g t Q(t), t = 1 / (1 + 0.36 |z|): the form of Hastings (Approximations
// for Digital Computers, 1955), Q fitted to erfc by its relative error, 2^-19.8 in
// 32 bits; with the exponential's argument 2^-17 at |z| = 12; 0 below 2^-126.
// 1 + erf(z / sqrt 2) is a multiple of 2^-24, 4 % off at z = -5 and 57 % at -5.5;
// erfcf is right but slow (8192 x 512 x 7168 with GELU: 130 us, 86 by erff, 71 so).
__device__ __forceinline__ float normal_cdf(float z, float& g) {
  const float u = fabsf(z);
  float t;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.36f, u, 1.0f)));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(g) : "f"(z * z * -0.72134752f));
  float q = 0.0473445728f;
  q = fmaf(q, t, -0.180751652f);
  q = fmaf(q, t, 0.182297572f);
  q = fmaf(q, t, 0.0256238226f);
  q = fmaf(q, t, 0.14005743f);
  q = fmaf(q, t, 0.141710669f);
  q = fmaf(q, t, 0.143717438f);
  const float tail = q * t * g;
  return z > 0.0f ? 1.0f - tail : tail;
}

template <int kAct>
__device__ __forceinline__ float act_value(float z) {
  if (kAct == EP_ACT_RELU) return z < 0.0f ? 0.0f : z;   // a NaN stays one
  if (kAct == EP_ACT_SILU) return __fdividef(z, 1.0f + __expf(-z));   // 2 ulp; 0 where the divisor passes 2^126
  if (kAct == EP_ACT_GELU) {
    float g;
    return z * normal_cdf(z, g);
  }
  return z;
}

// act(z) and act'(z)
template <int kAct>
__device__ __forceinline__ void act_both(float z, float& value, float& slope) {
  if (kAct == EP_ACT_RELU) {
    value = z < 0.0f ? 0.0f : z;
    slope = z > 0.0f ? 1.0f : 0.0f;
  } else if (kAct == EP_ACT_SILU) {
    const float q = __fdividef(1.0f, 1.0f + __expf(-z));
    value = z * q;
    slope = q * (1.0f + z * (1.0f - q));
  } else if (kAct == EP_ACT_GELU) {
    float g;
    const float c = normal_cdf(z, g);
    value = z * c;
    slope = c + z * 0.39894228f * g;
  } else {
    value = z;
    slope = 1.0f;
  }
}

}  // namespace ep
