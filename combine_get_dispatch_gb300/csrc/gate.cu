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
// One warp per token.  NaN becomes -inf on the way in; -inf is never chosen.

#include "ep_common.cuh"

namespace ep {

constexpr int kGateThreads = 256;
constexpr int kGateCtas = 6;   // CTAs an SM holds

struct GateParams {
  const void* logits;
  int64_t T;
  int E, k;
  const float* grad;
  int64_t* idx;
  float* w;
  void* grad_logits;
  int32_t* status;
  bool vec;   // rows start on 16 bytes, a lane's experts are all there or all not
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float warp_min(float v) {
  float r;
  asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

constexpr float kNone = -INFINITY;   // an expert that is never chosen

// exp(l - m): the difference rounds once and its product with log2(e) once, so
// it is off by |l - m| 2^-23 of itself.  m is finite.
__device__ __forceinline__ float gate_exp(float l, float m) { return __expf(l - m); }

// A logit as the kernels see it: NaN is an expert that is never chosen.
__device__ __forceinline__ float gate_clean(float l) { return fmaxf(l, kNone); }

template <bool kBf16>
__device__ __forceinline__ float gate_load(const void* logits, int64_t at) {
  if (kBf16) return gate_clean(__uint_as_float((uint32_t)static_cast<const uint16_t*>(logits)[at] << 16));
  return gate_clean(static_cast<const float*>(logits)[at]);
}

// The logits of a lane's kV experts, lane * kV on, of the row that starts at
// `row` (-inf past its end); vec: rows start on 16 bytes and E is a multiple of
// kV.
template <int kV, bool kBf16>
__device__ __forceinline__ void gate_row(const GateParams& p, int64_t row, int lane, float (&l)[kV]) {
  constexpr int kWords = kV * (kBf16 ? 2 : 4) / 4;   // 32-bit words a lane reads
  const int e0 = lane * kV;
  if (p.vec) {
    uint32_t w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = kBf16 ? 0xff80ff80u : 0xff800000u;   // -inf
    if (e0 < p.E) {
      const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.logits) + (row + e0) * (kBf16 ? 2 : 4));
      if (kWords >= 4) {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + i);
          w[4 * i] = v.x;
          w[4 * i + 1] = v.y;
          w[4 * i + 2] = v.z;
          w[4 * i + 3] = v.w;
        }
      } else if (kWords == 2) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
        w[0] = v.x;
        w[kWords - 1] = v.y;
      } else {
        w[0] = __ldg(src);
      }
    }
#pragma unroll
    for (int i = 0; i < kV; ++i)
      l[i] = gate_clean(kBf16 ? ((i & 1) ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2])) : __uint_as_float(w[kBf16 ? 0 : i]));
  } else {
#pragma unroll
    for (int i = 0; i < kV; ++i) l[i] = e0 + i < p.E ? gate_load<kBf16>(p.logits, row + e0 + i) : kNone;
  }
}

// The value to subtract, from the row's largest logit: itself, or 0 where nothing
// can be chosen.
__device__ __forceinline__ float gate_base(float most) { return most == kNone ? 0.0f : most; }

// As gate_exp in a row whose largest logit is +inf.
__device__ __forceinline__ float gate_share(float l) { return l == INFINITY ? 1.0f : 0.0f; }

// The k largest of the warp's logits, one round a choice: the largest, the
// lowest lane that holds it, that lane's lowest expert.  Lane j of the result
// holds choice j (-inf: none).
template <int kV>
__device__ __forceinline__ void gate_choose(float (&l)[kV], int k, int lane, float& my_l, int& my_idx) {
  my_l = kNone;
  my_idx = -1;
  for (int j = 0; j < k; ++j) {
    float b = kNone;
    int at = 0;
#pragma unroll
    for (int i = 0; i < kV; ++i)
      if (l[i] > b) {
        b = l[i];
        at = i;
      }
    const float top = warp_max(b);
    if (top == kNone) break;   // nothing left to choose
    const int win = __ffs(__ballot_sync(0xffffffffu, b == top)) - 1;
    const int e = __shfl_sync(0xffffffffu, lane * kV + at, win);
    if (lane == j) {
      my_l = top;
      my_idx = e;
    }
#pragma unroll
    for (int i = 0; i < kV; ++i)
      if (e == lane * kV + i) l[i] = kNone;
  }
}

// A round of choosing costs a warp about as many instructions as it holds
// logits, so most logits are thrown out first: 8 groups (16 for k > 8) of lanes
// have a largest logit each, the least of those is at most the k-th largest
// logit, and only logits at or above it can be chosen (some 15 of 256).  They
// are packed, in expert order, one to a lane, and a choice is then one reduction
// and one ballot.  Rows where more than 32 remain take the plain rounds.
template <int kV, bool kBf16, bool kTopk>
__global__ void __launch_bounds__(kGateThreads, kV <= 8 ? kGateCtas : 1) k_gate(GateParams p) {
  __shared__ uint2 packed[kGateThreads / kWarp][2 * kWarp];   // the upper half takes what is not packed
  const int lane = threadIdx.x & 31;
  uint2* mine = packed[threadIdx.x >> 5];
  const int64_t warp0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  for (int64_t t = warp0; t < p.T; t += nwarps) {
    float l[kV];
    gate_row<kV, kBf16>(p, t * p.E, lane, l);
    float best = l[0];
#pragma unroll
    for (int i = 1; i < kV; ++i) best = fmaxf(best, l[i]);
    const float m = gate_base(warp_max(best));
    float near = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 1)), far = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 16));
    if (p.k <= 8) {
      near = fmaxf(near, __shfl_xor_sync(0xffffffffu, near, 2));
      far = fmaxf(far, __shfl_xor_sync(0xffffffffu, far, 8));
    }
    // at least the type's lowest value, so that -inf is no candidate
    const float least = fmaxf(-3.40282346638528859812e+38f, fmaxf(warp_min(near), warp_min(far)));
    int n = 0;
#pragma unroll
    for (int i = 0; i < kV; ++i) n += l[i] >= least ? 1 : 0;
    int before = 0, all = 0;   // candidates of lower lanes, of all: a bit of n at a time
#pragma unroll
    for (int b = 0; (1 << b) <= kV; ++b) {
      const uint32_t has = __ballot_sync(0xffffffffu, (n >> b) & 1);
      before += __popc(has & lanemask_lt()) << b;
      all += __popc(has) << b;
    }
    float total = 0.0f;
    if (!kTopk) {
      if (m < INFINITY) {
#pragma unroll
        for (int i = 0; i < kV; ++i) total += gate_exp(l[i], m);
      } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) total += gate_share(l[i]);
      }
      total = warp_sum(total);
    }
    float my_l = kNone;
    int my_idx = -1, slot = p.k, found = 0;
    if (all <= kWarp) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const bool take = l[i] >= least;
        mine[take ? before : kWarp + lane] = make_uint2(__float_as_uint(l[i]), (uint32_t)(lane * kV + i));
        before += take ? 1 : 0;
      }
      __syncwarp();
      if (lane < all) {
        const uint2 c = mine[lane];
        my_l = __uint_as_float(c.x);
        my_idx = (int)c.y;
      }
      float left = my_l;
      const int rounds = min(p.k, all);
      for (; found < rounds; ++found) {
        const uint32_t who = __ballot_sync(0xffffffffu, left == warp_max(left));
        if (((who & (0u - who)) >> lane) == 1u) {   // the lowest lane of them
          slot = found;
          left = kNone;
        }
      }
      if (slot == p.k) my_l = kNone;
    } else {
      gate_choose<kV>(l, p.k, lane, my_l, my_idx);
      found = __popc(__ballot_sync(0xffffffffu, my_idx >= 0));
      slot = my_idx >= 0 ? lane : p.k;
    }
    const float ex = m < INFINITY ? gate_exp(my_l, m) : gate_share(my_l);
    if (kTopk) total = warp_sum(ex);
    if (slot < p.k) {
      p.idx[t * p.k + slot] = my_idx;
      p.w[t * p.k + slot] = ex / total;
    }
    if (lane >= found && lane < p.k) {
      p.idx[t * p.k + lane] = -1;
      p.w[t * p.k + lane] = 0.0f;
    }
  }
}

// The row of the gradient is laid out in shared memory (-p inner of the lane's
// own experts, or zeros), the k chosen experts add their own term to it in slot
// order, and the row is stored as it was read.
template <int kV, bool kBf16, bool kTopk>
__global__ void __launch_bounds__(kGateThreads) k_gate_backward(GateParams p) {
  extern __shared__ float rows[];
  const int lane = threadIdx.x & 31;
  float* mine = rows + (threadIdx.x >> 5) * (kV * kWarp);
  const int64_t warp0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  for (int64_t t = warp0; t < p.T; t += nwarps) {
    int my_idx = -1;
    float g = 0.0f, chosen = kNone;
    if (lane < p.k) {
      const int64_t id = p.idx[t * p.k + lane];
      if (id < -1 || id >= p.E)
        set_status(p.status, EP_ERR_INVALID_ARG);
      else
        my_idx = (int)id;
      if (my_idx >= 0) {
        g = p.grad[t * p.k + lane];
        chosen = gate_load<kBf16>(p.logits, t * p.E + my_idx);
      }
    }
    if (chosen == kNone) g = 0.0f;
    float l[kV];
    float best = chosen;
#pragma unroll
    for (int i = 0; i < kV; ++i) l[i] = kNone;
    if (!kTopk) {
      gate_row<kV, kBf16>(p, t * p.E, lane, l);
#pragma unroll
      for (int i = 0; i < kV; ++i) best = fmaxf(best, l[i]);
    }
    const float m = gate_base(warp_max(best));
    const float ex = m < INFINITY ? gate_exp(chosen, m) : gate_share(chosen);
    float total = ex;
    if (!kTopk) {
      total = 0.0f;
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        l[i] = m < INFINITY ? gate_exp(l[i], m) : gate_share(l[i]);
        total += l[i];
      }
    }
    total = warp_sum(total);
    const float inv = total > 0.0f ? 1.0f / total : 0.0f;
    const float w = ex * inv;
    const float inner = warp_sum(w * g);
    const float add = kTopk ? w * (g - inner) : w * g;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kV; ++i) mine[lane * kV + i] = kTopk ? 0.0f : -l[i] * inv * inner;
    __syncwarp();
    for (int j = 0; j < p.k; ++j) {   // in slot order, should a token name an expert twice
      if (lane == j && my_idx >= 0) mine[my_idx] += add;
      __syncwarp();
    }
    if (p.vec) {
      const int unit = kBf16 ? 8 : 4;   // 16 bytes
      for (int e = lane * unit; e < p.E; e += kWarp * unit) {
        uint4 v;
        if (kBf16)
          v = make_uint4(pack_bf16x2(mine[e], mine[e + 1]), pack_bf16x2(mine[e + 2], mine[e + 3]),
                         pack_bf16x2(mine[e + 4], mine[e + 5]), pack_bf16x2(mine[e + 6], mine[e + 7]));
        else
          v = ld_shared_v4(mine + e);
        st_v4(static_cast<uint8_t*>(p.grad_logits) + (t * p.E + e) * (kBf16 ? 2 : 4), v);
      }
    } else {
      for (int e = lane; e < p.E; e += kWarp) {
        if (kBf16)
          static_cast<__nv_bfloat16*>(p.grad_logits)[t * p.E + e] = __float2bfloat16_rn(mine[e]);
        else
          static_cast<float*>(p.grad_logits)[t * p.E + e] = mine[e];
      }
    }
  }
}

template <int kV, bool kBf16, bool kTopk>
static int launch_gate_t(const GateParams& p, bool backward, cudaStream_t stream) {
  const int64_t warps = kGateThreads / kWarp;
  const int64_t want = (p.T + warps - 1) / warps;
  const int grid = (int)std::min<int64_t>(want, (int64_t)ep_host::num_sms() * kGateCtas);
  if (backward)
    k_gate_backward<kV, kBf16, kTopk><<<grid, kGateThreads, kV * kGateThreads * sizeof(float), stream>>>(p);
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
  GateParams q = p;
  const int kv = p.E <= 64 ? 2 : p.E <= 128 ? 4 : p.E <= 256 ? 8 : p.E <= 512 ? 16 : 32;
  q.vec = p.E % std::max(kv, 8) == 0 && ep_host::aligned16(p.logits) && ep_host::aligned16(p.grad_logits);
  if (p.E <= 64) return launch_gate_v<2>(q, bf16, topk, backward, s);
  if (p.E <= 128) return launch_gate_v<4>(q, bf16, topk, backward, s);
  if (p.E <= 256) return launch_gate_v<8>(q, bf16, topk, backward, s);
  if (p.E <= 512) return launch_gate_v<16>(q, bf16, topk, backward, s);
  return launch_gate_v<32>(q, bf16, topk, backward, s);
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
