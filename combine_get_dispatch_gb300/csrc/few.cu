// few.cu -- a whole mixture-of-experts layer for a few tokens, in two kernels.

#include "expert.cuh"

namespace ep {

constexpr int kFewThreads = 256;

struct FewParams {
  const __nv_bfloat16* x;      // [T, H]
  const int64_t* idx;          // [T, k]
  const float* weights;
  const uint8_t* w_gu;         // bf16 or E4M3
  const uint8_t* gu_scales;
  const uint8_t* w_down;
  const uint8_t* down_scales;
  __nv_bfloat16* h;            // [T k, I], workspace
  __nv_bfloat16* out;
  int32_t* status;
  int T, k, E, H, I;
};

__device__ __forceinline__ float scale_of(uint32_t b) {
  return b == 255 ? __uint_as_float(0x7fc00000u) : b == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23);
}

// Sum over the row of 8 elements a lane and step.
template <bool kFp8>
__device__ __forceinline__ float dot(const uint8_t* w, int64_t row, const uint8_t* scales, int64_t scale_row, const __nv_bfloat16* v, int K, int lane) {
  float sum = 0.0f;
  for (int c = lane; c < K; c += 32) {
    float a;
    if (kFp8) {
      __half_raw r = __nv_cvt_fp8_to_halfraw(w[row * K + c], __NV_E4M3);
      a = __half2float(__half(r)) * scale_of(scales[scale_row * (K / kFp8Block) + c / kFp8Block]);
    } else {
      a = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(w)[row * K + c]);
    }
    sum = fmaf(a, __bfloat162float(v[c]), sum);
  }
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// h of every slot: a warp an element.
template <bool kFp8, int kAct>
__global__ void __launch_bounds__(kFewThreads) k_few_in(FewParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kFewThreads / kWarp), n = (int64_t)p.T * p.k * p.I;
  for (int64_t at = (int64_t)blockIdx.x * (kFewThreads / kWarp) + threadIdx.x / kWarp; at < n; at += warps) {
    const int slot = (int)(at / p.I), i = (int)(at - (int64_t)slot * p.I);
    const int64_t e = p.idx[slot];
    if (e < 0 || e >= p.E) {
      if (lane == 0 && e != -1) set_status(p.status, EP_ERR_INVALID_ARG);
      continue;
    }
    const __nv_bfloat16* v = p.x + (int64_t)(slot / p.k) * p.H;
    const int64_t row = e * 2 * p.I + i, block = e * 2 * (p.I / kFp8Block) + i / kFp8Block;
    const float gate = dot<kFp8>(p.w_gu, row, p.gu_scales, block, v, p.H, lane);
    const float up = dot<kFp8>(p.w_gu, row + p.I, p.gu_scales, block + p.I / kFp8Block, v, p.H, lane);
    if (lane == 0) p.h[at] = __float2bfloat16_rn(act_value<kAct>(gate) * up);
  }
}

// out: a warp an element, its token's slots in order of their experts.
template <bool kFp8>
__global__ void __launch_bounds__(kFewThreads) k_few_out(FewParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kFewThreads / kWarp), n = (int64_t)p.T * p.H;
  for (int64_t at = (int64_t)blockIdx.x * (kFewThreads / kWarp) + threadIdx.x / kWarp; at < n; at += warps) {
    const int t = (int)(at / p.H), c = (int)(at - (int64_t)t * p.H);
    const int64_t* idx = p.idx + (int64_t)t * p.k;
    float sum = 0.0f;
    for (int64_t last = -1;;) {   // the next expert above the last one
      int64_t e = p.E;
      for (int j = 0; j < p.k; ++j)
        if (idx[j] > last && idx[j] < e) e = idx[j];
      if (e >= p.E) break;
      last = e;
      for (int j = 0; j < p.k; ++j) {
        if (idx[j] != e) continue;
        const int slot = t * p.k + j;
        const float y = dot<kFp8>(p.w_down, e * p.H + c, p.down_scales, e * (p.H / kFp8Block) + c / kFp8Block, p.h + (int64_t)slot * p.I, p.I, lane);
        sum = fmaf(p.weights[slot], y, sum);
      }
    }
    if (lane == 0) p.out[at] = __float2bfloat16_rn(sum);
  }
}

template <bool kFp8, int kAct>
static int launch_few(const FewParams& p, cudaStream_t s) {
  const int grid = ep_host::grid_cap(4);
  k_few_in<kFp8, kAct><<<grid, kFewThreads, 0, s>>>(p);
  ep_host::count_launch();
  int rc = ep_host::check_launch();
  if (rc != EP_OK) return rc;
  k_few_out<kFp8><<<grid, kFewThreads, 0, s>>>(p);
  ep_host::count_launch();
  return ep_host::check_launch();
}

static bool few_sizes(int R, int T_r, int k, int E, int I) {
  return R > 0 && R <= kMaxR && T_r >= 0 && T_r <= EP_MOE_FEW_TOKENS && R * T_r <= EP_MOE_FEW_TOKENS && k > 0 && k <= kMaxK && E > 0 &&
         E <= kMaxE && E % R == 0 && I > 0 && I % 8 == 0 && I <= (1 << 24);
}

}  // namespace ep

extern "C" size_t ep_moe_few_workspace_size(int R, int T_r, int k, int E, int I) {
  if (!ep::few_sizes(R, T_r, k, E, I)) return 0;
  return std::max<size_t>(16, ((size_t)R * T_r * k * I * 2 + 15) / 16 * 16);
}

extern "C" int ep_moe_few(const void* x, const int64_t* topk_idx, const float* topk_weights, const void* w_gu,
                          const uint8_t* w_gu_scales, const void* w_down, const uint8_t* w_down_scales, int fp8_mode,
                          int R, int T_r, int k, int E, int H, int I, int act, void* out, void* workspace,
                          size_t workspace_bytes, int32_t* status, void* stream) {
  using namespace ep;
  if (fp8_mode != EP_FP8_NONE && fp8_mode != EP_FP8_E4M3_UE8M0) return EP_ERR_INVALID_ARG;
  const bool fp8 = fp8_mode != EP_FP8_NONE;
  if (!few_sizes(R, T_r, k, E, I) || H <= 0 || H > (1 << 24)) return EP_ERR_INVALID_ARG;
  const int unit = fp8 ? kFp8Block : 8;
  const int64_t lim = (int64_t)1 << 31;
  if (H % unit != 0 || I % unit != 0 || (int64_t)E * H >= lim || (int64_t)E * I >= lim) return EP_ERR_INVALID_ARG;
  if (act <= EP_ACT_NONE || act > EP_ACT_GELU) return EP_ERR_INVALID_ARG;
  if (fp8 != (w_gu_scales != nullptr) || fp8 != (w_down_scales != nullptr)) return EP_ERR_INVALID_ARG;
  if (T_r == 0) return EP_OK;
  for (const void* p : {x, w_gu, w_down, (const void*)out, (const void*)workspace})
    if (p == nullptr || !ep_host::aligned16(p)) return EP_ERR_INVALID_ARG;
  if (topk_idx == nullptr || topk_weights == nullptr || workspace_bytes < ep_moe_few_workspace_size(R, T_r, k, E, I))
    return EP_ERR_INVALID_ARG;
  FewParams p{};
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.idx = topk_idx;
  p.weights = topk_weights;
  p.w_gu = static_cast<const uint8_t*>(w_gu);
  p.gu_scales = w_gu_scales;
  p.w_down = static_cast<const uint8_t*>(w_down);
  p.down_scales = w_down_scales;
  p.h = static_cast<__nv_bfloat16*>(workspace);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.status = status;
  p.T = R * T_r;
  p.k = k;
  p.E = E;
  p.H = H;
  p.I = I;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (act) {
    case EP_ACT_RELU: return fp8 ? launch_few<true, EP_ACT_RELU>(p, s) : launch_few<false, EP_ACT_RELU>(p, s);
    case EP_ACT_SILU: return fp8 ? launch_few<true, EP_ACT_SILU>(p, s) : launch_few<false, EP_ACT_SILU>(p, s);
    default: return fp8 ? launch_few<true, EP_ACT_GELU>(p, s) : launch_few<false, EP_ACT_GELU>(p, s);
  }
}
