// newton.cu -- orthogonalised update of the experts' weights: momentum, norm,
// Newton-Schulz products, weight update.

#include <cmath>

#include "ep_common.cuh"

namespace ep {

constexpr int kTile = 32;

struct NewtonShape {
  int count, M, N, S;
};

// u of element i: the gradient, or with momentum what the step goes along.
struct Source {
  const void* g;
  bool f32;
  float* m;
  float momentum;
  bool nesterov;
};

// X = u, m updated; norms[matrix] = |u|: one CTA a matrix.
__global__ void __launch_bounds__(1024) k_newton_begin(Source src, int64_t each, float eps, float* x) {
  __shared__ float part[32];
  const int64_t base = blockIdx.x * each;
  float sum = 0.0f;
  for (int64_t i = threadIdx.x; i < each; i += blockDim.x) {
    float u = src.f32 ? static_cast<const float*>(src.g)[base + i] : __bfloat162float(static_cast<const __nv_bfloat16*>(src.g)[base + i]);
    if (src.m != nullptr) {
      const float g = u, m = fmaf(src.momentum, src.m[base + i], g);
      src.m[base + i] = m;
      u = src.nesterov ? fmaf(src.momentum, m, g) : m;
    }
    x[base + i] = u;
    sum = fmaf(u, u, sum);
  }
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
  __syncthreads();
  float all = 0.0f;
  for (int w = 0; w < 32; ++w) all += part[w];
  const float f = all <= 1.329228e36f ? 1.0f / (sqrtf(all) + eps) : __uint_as_float(0x7fc00000u);   // 2^120
  __syncthreads();
  for (int64_t i = threadIdx.x; i < each; i += blockDim.x) x[base + i] *= f;
}

// C = alpha P Q + beta D per matrix; element (i, j) of P at i p0 + j p1, of Q at i q0 + j q1.
struct Product {
  const float *P, *Q, *D;
  float* C;
  int64_t p0, p1, q0, q1, p_each, q_each, c_each;
  int rows, cols, inner;
  float alpha, beta;
};

__global__ void __launch_bounds__(1024) k_newton_product(Product a) {
  __shared__ float P[kTile][kTile + 1], Q[kTile][kTile + 1];
  const int tx = threadIdx.x % kTile, ty = threadIdx.x / kTile;
  const int i = blockIdx.y * kTile + ty, j = blockIdx.x * kTile + tx;
  for (int z = blockIdx.z;; z += gridDim.z) {
    const float *p = a.P + z * a.p_each, *q = a.Q + z * a.q_each;
    float sum = 0.0f;
    for (int k0 = 0; k0 < a.inner; k0 += kTile) {
      P[ty][tx] = i < a.rows && k0 + tx < a.inner ? p[i * a.p0 + (k0 + tx) * a.p1] : 0.0f;
      Q[ty][tx] = j < a.cols && k0 + ty < a.inner ? q[(k0 + ty) * a.q0 + j * a.q1] : 0.0f;
      __syncthreads();
      for (int k = 0; k < kTile; ++k) sum = fmaf(P[ty][k], Q[k][tx], sum);
      __syncthreads();
    }
    if (i < a.rows && j < a.cols) {
      const int64_t at = z * a.c_each + (int64_t)i * a.cols + j;
      a.C[at] = a.alpha * sum + (a.beta != 0.0f ? a.beta * a.D[at] : 0.0f);
    }
    break;
  }
}

__global__ void __launch_bounds__(256) k_newton_end(const float* x, int64_t n, __nv_bfloat16* out, float* w, __nv_bfloat16* w16, float keep, float step) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    if (out != nullptr) out[i] = __float2bfloat16_rn(x[i]);
    if (w != nullptr) {
      const float v = fmaf(-step, x[i], keep * w[i]);
      w[i] = v;
      if (w16 != nullptr) w16[i] = __float2bfloat16_rn(v);
    }
  }
}

static bool newton_sizes(int count, int M, int N) {
  return count >= 0 && count <= 65535 && M > 0 && N > 0 && N % 8 == 0 && M <= (1 << 20) && N <= (1 << 20) && (int64_t)count * M < ((int64_t)1 << 31);
}

static int newton(const Source& src, int count, int M, int N, int steps, const float* abc, float eps, __nv_bfloat16* out, float* w,
                  __nv_bfloat16* w16, float keep, float step, void* workspace, cudaStream_t s) {
  const int S = std::min(M, N);
  const int64_t each = (int64_t)M * N, square = (int64_t)S * S;
  float* x = static_cast<float*>(workspace);
  float *y = x + count * each, *A = y + count * each, *B = A + count * square;
  k_newton_begin<<<count, 1024, 0, s>>>(src, each, eps, x);
  ep_host::count_launch();
  const bool tall = M > N;
  auto product = [&](Product p) {
    k_newton_product<<<dim3((p.cols + kTile - 1) / kTile, (p.rows + kTile - 1) / kTile, count), 1024, 0, s>>>(p);
    ep_host::count_launch();
  };
  for (int t = 0; t < steps; ++t) {
    const float a = abc[3 * t], b = abc[3 * t + 1], c = abc[3 * t + 2];
    if (tall)
      product({x, x, nullptr, A, 1, N, N, 1, each, each, square, S, S, M, 1.0f, 0.0f});
    else
      product({x, x, nullptr, A, N, 1, 1, N, each, each, square, S, S, N, 1.0f, 0.0f});
    product({A, A, A, B, S, 1, S, 1, square, square, square, S, S, c != 0.0f ? S : 0, c, b});
    if (tall)
      product({x, B, x, y, N, 1, S, 1, each, square, each, M, N, S, 1.0f, a});
    else
      product({B, x, x, y, S, 1, N, 1, square, each, each, M, N, S, 1.0f, a});
    std::swap(x, y);
  }
  k_newton_end<<<ep_host::grid_cap(4), 256, 0, s>>>(x, count * each, out, w, w16, keep, step);
  ep_host::count_launch();
  return ep_host::check_launch();
}

static int check_newton(const void* g, int dtype, int count, int M, int N, int steps, const float* abc, float eps, const void* workspace,
                        size_t bytes) {
  if ((dtype != EP_DTYPE_F32 && dtype != EP_DTYPE_BF16) || !newton_sizes(count, M, N)) return EP_ERR_INVALID_ARG;
  if (steps < 1 || steps > 32 || abc == nullptr || !(eps >= 1e-12f) || !std::isfinite(eps)) return EP_ERR_INVALID_ARG;
  for (int i = 0; i < 3 * steps; ++i)
    if (!std::isfinite(abc[i])) return EP_ERR_INVALID_ARG;
  if (count > 0 && (g == nullptr || !ep_host::aligned16(g) || workspace == nullptr || !ep_host::aligned16(workspace) ||
                    bytes < ep_orthogonalize_workspace_size(count, M, N)))
    return EP_ERR_INVALID_ARG;
  return EP_OK;
}

}  // namespace ep

extern "C" size_t ep_orthogonalize_workspace_size(int count, int M, int N) {
  if (!ep::newton_sizes(count, M, N)) return 0;
  const size_t S = std::min(M, N);
  return std::max<size_t>(16, (size_t)count * ((size_t)M * N * 8 + S * S * 8));
}

extern "C" int ep_orthogonalize(const void* g, int dtype, int count, int M, int N, int steps, const float* coefficients, float eps, void* out,
                                void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
  using namespace ep;
  const int rc = check_newton(g, dtype, count, M, N, steps, coefficients, eps, workspace, workspace_bytes);
  if (rc != EP_OK) return rc;
  if (count == 0) return EP_OK;
  if (out == nullptr || !ep_host::aligned16(out)) return EP_ERR_INVALID_ARG;
  const Source src = {g, dtype == EP_DTYPE_F32, nullptr, 0.0f, false};
  return newton(src, count, M, N, steps, coefficients, eps, static_cast<__nv_bfloat16*>(out), nullptr, nullptr, 0.0f, 0.0f, workspace,
                static_cast<cudaStream_t>(stream));
}

extern "C" int ep_muon_update(const void* g, int dtype, float* m, float* w, void* w16, int count, int M, int N, float lr, float scale,
                              float momentum, int nesterov, float weight_decay, int steps, const float* coefficients, float eps,
                              void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
  using namespace ep;
  const int rc = check_newton(g, dtype, count, M, N, steps, coefficients, eps, workspace, workspace_bytes);
  if (rc != EP_OK) return rc;
  if (!std::isfinite(lr) || !std::isfinite(scale) || !std::isfinite(weight_decay) || !(momentum >= 0.0f && momentum < 1.0f))
    return EP_ERR_INVALID_ARG;
  if (count == 0) return EP_OK;
  if (m == nullptr || w == nullptr || !ep_host::aligned16(m) || !ep_host::aligned16(w) || !ep_host::aligned16(w16)) return EP_ERR_INVALID_ARG;
  const Source src = {g, dtype == EP_DTYPE_F32, m, momentum, nesterov != 0};
  return newton(src, count, M, N, steps, coefficients, eps, nullptr, w, static_cast<__nv_bfloat16*>(w16),
                (float)(1.0 - (double)lr * weight_decay), (float)((double)lr * scale), workspace, static_cast<cudaStream_t>(stream));
}
