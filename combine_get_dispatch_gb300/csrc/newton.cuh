// newton.cuh -- what the kernels of the orthogonalised update share: their source,
// and how X is held.
#pragma once

#include "umma.cuh"

namespace ep {

constexpr float kHeld = 256.0f;           // X, A and P are held this many times as large

struct Source {
  const void* g;
  bool f32;
  float* m;               // or nullptr: u is the gradient
  float momentum;
  bool nesterov;
  int64_t each;           // elements of a matrix, a multiple of 8
  int64_t part;           // elements of a part, a multiple of 8 kSourceThreads
  int parts, count;
  bool early;             // the next kernel may come up while one runs: without an SM budget
  float eps;
  float* sums;            // [count, parts]
  float* factor;          // [count]
  int32_t* failed;        // set by products whose waits ran out, so that weights are not updated from what they left
  int rows, cols, stride; // of X: rows of `cols` elements, `stride` apart
  __half *hi, *lo;        // lo may be nullptr
};

// 8 elements as they lie in memory, read past the first-level cache.
struct SourceWords {
  uint4 a, b;   // b: of fp32
};
__device__ __forceinline__ SourceWords load_words(const void* from, bool f32, int64_t i) {
  SourceWords w{};
  if (f32) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(from) + i);
    w.a = __ldcg(p);
    w.b = __ldcg(p + 1);
  } else {
    w.a = __ldcg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(from) + i));
  }
  return w;
}
__device__ __forceinline__ void words_to_floats(const SourceWords& s, bool f32, float (&v)[8]) {
  const uint32_t w[8] = {s.a.x, s.a.y, s.a.z, s.a.w, s.b.x, s.b.y, s.b.z, s.b.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = f32 ? __uint_as_float(w[2 * k]) : bf16_lo(w[k]);
    v[2 * k + 1] = f32 ? __uint_as_float(w[2 * k + 1]) : bf16_hi(w[k]);
  }
}
// norm + eps -> the power of two that brings u near 2^8, and the factor that is
// left; NaN for both where the norm is not finite or passes 2^60.
__device__ __forceinline__ void source_scale(float square, float eps, float& up, float& factor) {
  const float norm = sqrtf(square) + eps;   // at least 1e-12
  const bool fits = norm <= 1.152921505e18f;
  // the least power of two that is not below 2^8 / norm
  up = fits ? __uint_as_float((uint32_t)(127 + 8 - ilogbf(norm)) << 23) : __uint_as_float(0x7fc00000u);
  factor = fits ? kHeld / (norm * up) : __uint_as_float(0x7fc00000u);
}

// Two numbers as hi and lo words.
__device__ __forceinline__ void split_f16(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 b = __half22float2(h);
  const __half2 l = __floats2half2_rn(x - b.x, y - b.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}
__device__ __forceinline__ float2 floats_of(uint32_t half2) { return __half22float2(*reinterpret_cast<const __half2*>(&half2)); }

// Instruction descriptor, fp16 operands and fp32 sums.
__device__ __forceinline__ uint32_t umma_idesc_f16(int m, int n, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Matrices whose X fits one SM's registers, and with the polynomial its shared memory.
constexpr int kSmallSide = 128, kSmallLength = 256;
struct SmallNewton {
  Source src;
  int M, N, steps;
  float abc[3 * 32];
  __nv_bfloat16* out;       // or nullptr and
  float* w;
  __nv_bfloat16* w16;
  float keep, step;
  int32_t* status;
};
int launch_newton_small(const SmallNewton& p, cudaStream_t stream);

}  // namespace ep
