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

template <int kAct>
__device__ __forceinline__ float act_value(float z) {
  if (kAct == EP_ACT_RELU) return z < 0.0f ? 0.0f : z;   // a NaN stays one
  if (kAct == EP_ACT_SILU) return __fdividef(z, 1.0f + __expf(-z));   // 2 ulp; 0 where the divisor passes 2^126
  if (kAct == EP_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678f));
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
    const float c = 0.5f * (1.0f + erff(z * 0.70710678f));
    value = z * c;
    slope = c + z * 0.39894228f * __expf(-0.5f * z * z);
  } else {
    value = z;
    slope = 1.0f;
  }
}

}  // namespace ep
