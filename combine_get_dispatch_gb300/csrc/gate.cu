// gate.cu -- the router's top-k (ep_gate_topk) and its gradient
// (ep_gate_topk_backward): the topk_idx / topk_weights that dispatch and
// combine read.
//
//   m = max l, p_e = exp(l_e - m) / sum exp(l - m)
//   SOFTMAX       w_j = p of the chosen expert over all E experts
//   SOFTMAX_TOPK  the sum runs over the chosen experts only
//   gradient      SOFTMAX: dl_e = [e chosen] w_e g_e - p_e sum_j w_j g_j
//                 TOPK:    dl_e = [e chosen] w_e (g_e - sum_j w_j g_j)
//
// One warp per token.  Logits become order-preserving 32-bit keys, so the
// choice is exact in integers; -inf and NaN have key 0 and are never chosen.

#include "ep_common.cuh"

namespace ep {

constexpr int kGateThreads = 256;

struct GateParams {
  const void* logits;
  int64_t T;
  int E, k;
  const float* grad;
  int64_t* idx;
  float* w;
  void* grad_logits;
  int32_t* status;
};

// Order-preserving key of a logit: larger logit, larger key; 0 for -inf and
// NaN (never chosen).  +-0 compare equal, as the floats do.
__device__ __forceinline__ uint32_t gate_key(float l) {
  if (!(l > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(l + 0.0f);   // -0 + 0 = +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float gate_unkey(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

// exp(l - m) with m the row's largest logit; equal values give 1 (so that a
// +inf is 1 and everything below it 0), a key of 0 gives 0.
__device__ __forceinline__ float gate_exp(uint32_t key, float m) {
  if (key == 0u) return 0.0f;
  const float l = gate_unkey(key);
  return l == m ? 1.0f : expf(l - m);
}

template <bool kBf16>
__device__ __forceinline__ float gate_load(const void* logits, int64_t at) {
  if (kBf16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(logits)[at] << 16);
  return static_cast<const float*>(logits)[at];
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// kV: logits a lane holds (expert lane + 32 i).
template <int kV, bool kBf16, bool kTopk>
__global__ void __launch_bounds__(kGateThreads) k_gate(GateParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t warp0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  for (int64_t t = warp0; t < p.T; t += nwarps) {
    uint32_t key[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int e = lane + 32 * i;
      key[i] = e < p.E ? gate_key(gate_load<kBf16>(p.logits, t * p.E + e)) : 0u;
    }
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < kV; ++i) best = max(best, key[i]);
    const uint32_t mkey = __reduce_max_sync(0xffffffffu, best);
    const float m = gate_unkey(mkey);
    float total = 0.0f;
    if (!kTopk) {
#pragma unroll
      for (int i = 0; i < kV; ++i) total += gate_exp(key[i], m);
      total = warp_sum(total);
    }
    uint32_t my_key = 0;
    int my_idx = -1;
    for (int j = 0; j < p.k; ++j) {
      uint32_t b = 0;
      int at = 0;
#pragma unroll
      for (int i = 0; i < kV; ++i)
        if (key[i] > b) {
          b = key[i];
          at = i;
        }
      const uint32_t top = __reduce_max_sync(0xffffffffu, b);
      if (top == 0u) break;   // nothing left to choose
      const uint32_t e = b == top ? (uint32_t)(lane + 32 * at) : 0xffffffffu;
      const uint32_t win = __reduce_min_sync(0xffffffffu, e);
      if (lane == j) {
        my_key = top;
        my_idx = (int)win;
      }
#pragma unroll
      for (int i = 0; i < kV; ++i)
        if (win == (uint32_t)(lane + 32 * i)) key[i] = 0u;
    }
    const float ex = gate_exp(my_key, m);
    if (kTopk) total = warp_sum(ex);
    if (lane < p.k) {
      p.idx[t * p.k + lane] = my_idx;
      p.w[t * p.k + lane] = my_idx >= 0 ? ex / total : 0.0f;
    }
  }
}

template <int kV, bool kBf16, bool kTopk>
__global__ void __launch_bounds__(kGateThreads) k_gate_backward(GateParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t warp0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  for (int64_t t = warp0; t < p.T; t += nwarps) {
    int my_idx = -1;
    float g = 0.0f;
    if (lane < p.k) {
      const int64_t id = p.idx[t * p.k + lane];
      if (id < -1 || id >= p.E)
        set_status(p.status, EP_ERR_INVALID_ARG);
      else
        my_idx = (int)id;
      if (my_idx >= 0) g = p.grad[t * p.k + lane];
    }
    const uint32_t my_key = my_idx >= 0 ? gate_key(gate_load<kBf16>(p.logits, t * p.E + my_idx)) : 0u;
    if (my_key == 0u) g = 0.0f;
    uint32_t key[kV];
    uint32_t best = my_key;
    if (!kTopk) {
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const int e = lane + 32 * i;
        key[i] = e < p.E ? gate_key(gate_load<kBf16>(p.logits, t * p.E + e)) : 0u;
        best = max(best, key[i]);
      }
    }
    const float m = gate_unkey(__reduce_max_sync(0xffffffffu, best));
    const float mine = gate_exp(my_key, m);
    float total = mine;
    if (!kTopk) {
      total = 0.0f;
#pragma unroll
      for (int i = 0; i < kV; ++i) total += gate_exp(key[i], m);
    }
    total = warp_sum(total);
    const float inv = total > 0.0f ? 1.0f / total : 0.0f;
    const float w = mine * inv;
    const float inner = warp_sum(w * g);
    const float add = kTopk ? w * (g - inner) : w * g;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int e = lane + 32 * i;
      float d = kTopk ? 0.0f : -gate_exp(key[i], m) * inv * inner;
      for (int j = 0; j < p.k; ++j) {
        const int ej = __shfl_sync(0xffffffffu, my_idx, j);
        const float aj = __shfl_sync(0xffffffffu, add, j);
        if (ej == e) d += aj;
      }
      if (e < p.E) {
        if (kBf16)
          static_cast<__nv_bfloat16*>(p.grad_logits)[t * p.E + e] = __float2bfloat16_rn(d);
        else
          static_cast<float*>(p.grad_logits)[t * p.E + e] = d;
      }
    }
  }
}

template <int kV, bool kBf16, bool kTopk>
static int launch_gate_t(const GateParams& p, bool backward, cudaStream_t stream) {
  const int64_t warps = kGateThreads / kWarp;
  const int64_t want = (p.T + warps - 1) / warps;
  const int grid = (int)std::min<int64_t>(want, (int64_t)ep_host::num_sms() * 8);
  if (backward)
    k_gate_backward<kV, kBf16, kTopk><<<grid, kGateThreads, 0, stream>>>(p);
  else
    k_gate<kV, kBf16, kTopk><<<grid, kGateThreads, 0, stream>>>(p);
  ep_host::count_launch();
  return ep_host::check_launch();
}

template <int kV>
static int launch_gate_v(const GateParams& p, bool bf16, bool topk, bool backward, cudaStream_t s) {
  if (bf16)
    return topk ? launch_gate_t<kV, true, true>(p, backward, s) : launch_gate_t<kV, true, false>(p, backward, s);
  return topk ? launch_gate_t<kV, false, true>(p, backward, s) : launch_gate_t<kV, false, false>(p, backward, s);
}

static int launch_gate(const GateParams& p, int dtype, int score, bool backward, cudaStream_t s) {
  if (p.T == 0) return EP_OK;
  const bool bf16 = dtype == EP_DTYPE_BF16, topk = score == EP_GATE_SOFTMAX_TOPK;
  if (p.E <= 64) return launch_gate_v<2>(p, bf16, topk, backward, s);
  if (p.E <= 128) return launch_gate_v<4>(p, bf16, topk, backward, s);
  if (p.E <= 256) return launch_gate_v<8>(p, bf16, topk, backward, s);
  if (p.E <= 512) return launch_gate_v<16>(p, bf16, topk, backward, s);
  return launch_gate_v<32>(p, bf16, topk, backward, s);
}

static int check_gate(const void* logits, int dtype, int R, int T_r, int E, int k, int score) {
  if (R <= 0 || R > kMaxR || T_r < 0 || E <= 0 || E > kMaxE || E % R != 0 || k <= 0 || k > kMaxK ||
      k > E)
    return EP_ERR_INVALID_ARG;
  if (dtype != EP_DTYPE_F32 && dtype != EP_DTYPE_BF16) return EP_ERR_INVALID_ARG;
  if (score != EP_GATE_SOFTMAX && score != EP_GATE_SOFTMAX_TOPK) return EP_ERR_INVALID_ARG;
  if (T_r > 0 && logits == nullptr) return EP_ERR_INVALID_ARG;
  return EP_OK;
}

}  // namespace ep

extern "C" int ep_gate_topk(const void* logits, int dtype, int R, int T_r, int E, int k, int score,
                            int64_t* topk_idx, float* topk_weights, void* stream) {
  const int rc = ep::check_gate(logits, dtype, R, T_r, E, k, score);
  if (rc != EP_OK) return rc;
  if (T_r > 0 && (topk_idx == nullptr || topk_weights == nullptr)) return EP_ERR_INVALID_ARG;
  ep::GateParams p{};
  p.logits = logits;
  p.T = (int64_t)R * T_r;
  p.E = E;
  p.k = k;
  p.idx = topk_idx;
  p.w = topk_weights;
  return ep::launch_gate(p, dtype, score, false, static_cast<cudaStream_t>(stream));
}

extern "C" int ep_gate_topk_backward(const void* logits, int dtype, const int64_t* topk_idx,
                                     const float* grad_topk_weights, int R, int T_r, int E, int k,
                                     int score, void* grad_logits, int32_t* status, void* stream) {
  const int rc = ep::check_gate(logits, dtype, R, T_r, E, k, score);
  if (rc != EP_OK) return rc;
  if (T_r > 0 && (topk_idx == nullptr || grad_topk_weights == nullptr || grad_logits == nullptr))
    return EP_ERR_INVALID_ARG;
  ep::GateParams p{};
  p.logits = logits;
  p.T = (int64_t)R * T_r;
  p.E = E;
  p.k = k;
  p.idx = const_cast<int64_t*>(topk_idx);
  p.grad = grad_topk_weights;
  p.grad_logits = grad_logits;
  p.status = status;
  return ep::launch_gate(p, dtype, score, true, static_cast<cudaStream_t>(stream));
}
