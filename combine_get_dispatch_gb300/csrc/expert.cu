// expert.cu -- the experts' products over a receive layout: entry points and the
// elementwise half of the gradients.

#include "expert_gemm.cuh"
#include "umma.cuh"

namespace ep {

constexpr int kThreads = 256;
constexpr int kSlopeRows = 32, kSlopeCols = 512, kSlopeCtas = 4;   // a piece of k_glu_slope; CTAs of an SM

struct SlopeParams {
  Segments seg;
  const __nv_bfloat16* dy;    // dh [rows, N], or dy [rows, N]
  const __nv_bfloat16* pre;   // gu [rows, 2, N], or pre [rows, N]
  __nv_bfloat16* out;         // dgu, dpre; may be nullptr (sum only)
  __nv_bfloat16* dbias;       // [E, N] or nullptr
  int N;
};

// dgu = (dh * up * act'(gate), dh * act(gate)) over the rows of every segment,
// 8 columns a thread, two rows' loads at a time.  A CTA takes 32 rows x 512
// columns of an expert from the list of all of them, whatever the experts' shares
// are (one grid row an expert took 97 us where one of 32 experts had a quarter of
// 12288 rows x 1416; whole rows, one load at a time, 33, and 72 us for 96 rows x
// 3984 of 16 experts; now 28 and 14).  Memory bounds it: 65536 x 2048 198 us, 6.8 TB/s.
// dgu is rounded to bf16, the operand type of the products that follow: dx and dw
// are then 0.0023 off (relative norm, bf16 results), 0.0017 from 32-bit ones, which
// the tensor cores would take as two operands and twice the products.
template <int kAct>
__global__ void __launch_bounds__(kThreads, kSlopeCtas) k_glu_slope(SlopeParams p) {
  constexpr int kWide = kSlopeCols / 8, kStep = kThreads / kWide, kLoads = 2;
  __shared__ Tile next[2];
  __shared__ TileWalk walks[kWarp];   // not in registers, which the rows need
  const int lane = threadIdx.x & 31;
  TileWalk& walk = walks[lane];
  pdl_launch_dependents();
  pdl_wait();
  if (threadIdx.x < 32) walk.begin(p.seg, -1, kSlopeRows, (p.N + kSlopeCols - 1) / kSlopeCols, kSlopeCols, blockIdx.x == 0, lane);
  for (int64_t at = blockIdx.x, n = 0;; at += gridDim.x, ++n) {
    if (threadIdx.x < 32) {
      const Tile t = walk.at(at, lane);
      if (lane == 0) next[n & 1] = t;
    }
    __syncthreads();
    const Tile t = next[n & 1];
    if (t.e < 0) break;
    const int c = t.n0 + (int)(threadIdx.x % kWide) * 8;
    if (c >= p.N) continue;
    for (int r0 = threadIdx.x / kWide; r0 < t.rows; r0 += kLoads * kStep) {
      uint4 d[kLoads], g[kLoads], u[kLoads];
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        d[k] = g[k] = u[k] = make_uint4(0, 0, 0, 0);
        if (r0 + k * kStep < t.rows) {
          const int64_t row = (int64_t)t.start + t.m0 + r0 + k * kStep;
          d[k] = *reinterpret_cast<const uint4*>(p.dy + row * p.N + c);
          g[k] = *reinterpret_cast<const uint4*>(p.pre + row * 2 * p.N + c);
          u[k] = *reinterpret_cast<const uint4*>(p.pre + (row * 2 + 1) * p.N + c);
        }
      }
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int64_t row = (int64_t)t.start + t.m0 + r0 + k * kStep;
        const uint32_t dw[4] = {d[k].x, d[k].y, d[k].z, d[k].w}, gw[4] = {g[k].x, g[k].y, g[k].z, g[k].w};
        const uint32_t uw[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
        uint32_t og[4], ou[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v0, s0, v1, s1;
          act_both<kAct>(bf16_lo(gw[i]), v0, s0);
          act_both<kAct>(bf16_hi(gw[i]), v1, s1);
          const float d0 = bf16_lo(dw[i]), d1 = bf16_hi(dw[i]);
          og[i] = pack_bf16x2(d0 * bf16_lo(uw[i]) * s0, d1 * bf16_hi(uw[i]) * s1);
          ou[i] = pack_bf16x2(d0 * v0, d1 * v1);
        }
        if (r0 + k * kStep < t.rows) {
          st_v4(p.out + row * 2 * p.N + c, make_uint4(og[0], og[1], og[2], og[3]));
          st_v4(p.out + (row * 2 + 1) * p.N + c, make_uint4(ou[0], ou[1], ou[2], ou[3]));
        }
      }
    }
  }
}

// dpre = dy * act'(pre) and dbias = its sum over the expert's rows.  A cluster of
// kSplit CTAs owns 64 columns of one expert: 8 threads a row, 32 rows a CTA and
// step, four steps' loads at a time, the sums in 32 bits (before dpre is
// rounded, as dgu is above), added over the CTA's rows and then over the cluster in a fixed order.
// kAlone (under an SM budget): a CTA takes the shares of a cluster one after
// another, and as many column groups as its part of the grid is; the same sums in
// the same order.  Memory bounds it (50288 x 4072, sum only: read once, 410 MB).
template <int kAct, int kSplit, bool kAlone>
__global__ void __launch_bounds__(kThreads) k_linear_slope(SlopeParams p) {
  constexpr int kRows = kThreads / 8, kSteps = 4, kCluster = kAlone ? 1 : kSplit;
  __shared__ float part[kThreads / kWarp][64];
  const int c8 = threadIdx.x & 7, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = blockIdx.x % kCluster, groups = (p.N + 63) / 64;
  pdl_launch_dependents();   // the products come up while this runs
  pdl_wait();
  for (int item = blockIdx.x / kCluster; !kAlone || item < groups * p.seg.E; item += gridDim.x) {
    const int e = kAlone ? item / groups : blockIdx.y;
    const int c0 = (kAlone ? item % groups : item) * 64, c = c0 + c8 * 8;
    Segments seg = p.seg;
    if (c0 != 0 || rank != 0) seg.status = nullptr;
    const Segment s = segment_of(seg, e);
    float all = 0.0f;
    for (int share = rank;; ++share) {
      float sum[8] = {};
      if (c < p.N) {
        for (int64_t i0 = share * kRows + (threadIdx.x >> 3); i0 < s.count; i0 += kSplit * kRows * kSteps) {
          uint4 d[kSteps], z[kSteps];
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            const int64_t i = i0 + k * kSplit * kRows;
            d[k] = z[k] = make_uint4(0, 0, 0, 0);
            if (i < s.count) {
              const int64_t at = (s.start + i) * p.N + c;
              d[k] = *reinterpret_cast<const uint4*>(p.dy + at);
              if (kAct != EP_ACT_NONE) z[k] = *reinterpret_cast<const uint4*>(p.pre + at);
            }
          }
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            const int64_t i = i0 + k * kSplit * kRows;
            const uint32_t dw[4] = {d[k].x, d[k].y, d[k].z, d[k].w}, zw[4] = {z[k].x, z[k].y, z[k].z, z[k].w};
            uint32_t o[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float v, s0, s1;
              act_both<kAct>(bf16_lo(zw[q]), v, s0);
              act_both<kAct>(bf16_hi(zw[q]), v, s1);
              const float d0 = bf16_lo(dw[q]) * s0, d1 = bf16_hi(dw[q]) * s1;
              sum[2 * q] += d0;
              sum[2 * q + 1] += d1;
              o[q] = pack_bf16x2(d0, d1);
            }
            if (kAct != EP_ACT_NONE && i < s.count) st_v4(p.out + (s.start + i) * p.N + c, make_uint4(o[0], o[1], o[2], o[3]));
          }
        }
      }
      if (p.dbias != nullptr) {   // the same for every CTA of the cluster
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          sum[q] += __shfl_xor_sync(0xffffffffu, sum[q], 8);
          sum[q] += __shfl_xor_sync(0xffffffffu, sum[q], 16);
          if (lane < 8) part[warp][c8 * 8 + q] = sum[q];
        }
        __syncthreads();
        float rows = 0.0f;
        if (threadIdx.x < 64) {
#pragma unroll
          for (int w = 0; w < kThreads / kWarp; ++w) rows += part[w][threadIdx.x];
        }
        all = kAlone && share > 0 ? all + rows : rows;
        if (kSplit > 1 || kAlone) __syncthreads();   // part is written again
      }
      if (!kAlone || share + 1 == kSplit) break;
    }
    const int col = c0 + threadIdx.x;
    const bool writes = p.dbias != nullptr && rank == 0 && threadIdx.x < 64 && col < p.N;
    if (kCluster > 1 && p.dbias != nullptr) {
      if (threadIdx.x < 64) part[0][threadIdx.x] = all;
      cluster_sync();
      if (writes) {
        for (int r = 1; r < kCluster; ++r) all += ld_cluster_f32(map_to_rank(smem_addr(&part[0][threadIdx.x]), r));
      }
      cluster_sync();   // no CTA leaves while its sums are read
    }
    if (writes) p.dbias[(int64_t)e * p.N + col] = __float2bfloat16_rn(all);
    if (!kAlone) break;
  }
}

template <int kAct>
static int launch_glu_slope(const SlopeParams& p, int64_t rows, cudaStream_t s) {
  const int64_t tiles = (rows / kSlopeRows + p.seg.E) * ((p.N + kSlopeCols - 1) / kSlopeCols);
  const int grid = (int)std::min<int64_t>(tiles, ep_host::grid_cap(kSlopeCtas));
  if (ep_host::launch_dependent(k_glu_slope<kAct>, grid, kThreads, 0, s, p) != EP_OK) return EP_ERR_CUDA;
  ep_host::count_launch();
  return ep_host::check_launch();
}

template <int kAct, int kSplit>
static int launch_linear_slope_t(const SlopeParams& p, cudaStream_t s) {
  const int groups = (p.N + 63) / 64;
  const int rc =
      ep_host::sm_budget_set()
          ? ep_host::launch_dependent(k_linear_slope<kAct, kSplit, true>, std::min(groups * p.seg.E, ep_host::grid_cap(1)),
                                      kThreads, 0, s, p)
          : ep_host::launch_dependent(k_linear_slope<kAct, kSplit, false>, dim3(groups * kSplit, p.seg.E), kThreads, 0, s, p, kSplit);
  if (rc != EP_OK) return rc;
  ep_host::count_launch();
  return ep_host::check_launch();
}

// One CTA for 64 columns of an expert where those fill the SMs' 8 places several
// times; with fewer the rows are split over 2, so that one expert's many rows are
// not the kernel's time (11088 rows x 272, 224 experts of uneven sizes: 31 us
// whole, 17 by 2, 24 by 8; 37140 x 1400, 32 even experts: 52, 58-60, 78); with
// at most one an SM over 8 (777 x 2048, one expert: 13.2 us by 32 CTAs, 7.4).
// The split does not look at the SM budget, so that the sums are the same under one.
template <int kAct>
static int launch_linear_slope(const SlopeParams& p, cudaStream_t s) {
  const int64_t groups = (int64_t)((p.N + 63) / 64) * p.seg.E;
  const int sms = ep_host::num_sms();
  if (groups <= sms) return launch_linear_slope_t<kAct, 8>(p, s);
  return groups < 16 * sms ? launch_linear_slope_t<kAct, 2>(p, s) : launch_linear_slope_t<kAct, 1>(p, s);
}

static int64_t rows_of(const Segments& s) { return s.cap * (s.psum != nullptr ? s.E / s.E_l : s.E); }

// Which products let the kernel after them come up early: those that another expert
// kernel follows, in their call or in a layer (gated projection of 128 rows, call
// after call: 5.4 us without, 4.6 with).  Not those whose rows the combine reads
// (the product, the gated projection's dx and dw): its split of the tokens is static
// and takes its CTAs for evenly placed (projection of 12288 rows over 64 experts,
// 1408 -> 4096, and combine: 159.1 us, 156.7 without; over 32 experts by Zipf 1.2,
// 1416 -> 4096: 164.6, 161.3; 128 rows of 128 -> 256: 6.7, 7.1).

// dx = d W and dw = d^T x, over d [rows, N].  early: of the last of them.
static int launch_gradients(bool early, const Segments& seg, const void* d, const void* x, const void* w, int K, int N,
                            void* dx, void* dw, cudaStream_t s) {
  if (dw != nullptr && rows_of(seg) == 0) {   // no rows: zero weights' gradients
    if (cudaMemsetAsync(dw, 0, (size_t)seg.E * N * K * 2, s) != cudaSuccess) {
      cudaGetLastError();
      return EP_ERR_CUDA;
    }
    dw = nullptr;
  }
  if (dx != nullptr) {
    ProductParams p{};
    p.seg = seg;
    p.rows = rows_of(seg);
    p.a = d;
    p.b = w;
    p.K = N;
    p.N = K;
    p.out = dx;
    p.early = early || dw != nullptr;
    const int rc = launch_gemm_bf16(kDx, p, EP_ACT_NONE, s);
    if (rc != EP_OK) return rc;
  }
  if (dw != nullptr) {
    ProductParams p{};
    p.seg = seg;
    p.rows = rows_of(seg);
    p.a = d;
    p.b = x;
    p.K = N;
    p.N = K;
    p.out = dw;
    p.early = early;
    const int rc = launch_gemm_bf16(kDw, p, EP_ACT_NONE, s);
    if (rc != EP_OK) return rc;
  }
  return EP_OK;
}

static int check_expert(const int32_t* counts, const int64_t* psum, int R, int E, int K, int N, int64_t cap_rows,
                        int unit) {
  if (R <= 0 || R > kMaxR || E <= 0 || E > kMaxE || E % R != 0 || cap_rows < 0) return EP_ERR_INVALID_ARG;
  if (K <= 0 || N <= 0 || K % unit != 0 || N % unit != 0 || K > (1 << 24) || N > (1 << 24)) return EP_ERR_INVALID_ARG;
  const int64_t lim = (int64_t)1 << 31;
  const int64_t owners = psum != nullptr ? R : E;
  // coordinates run past a segment's end, by less than a tile, without leaving 31 bits
  if (cap_rows > (lim - (1 << 16)) / owners || (int64_t)E * K >= lim || (int64_t)E * N >= lim / 2) return EP_ERR_INVALID_ARG;
  if (counts == nullptr) return EP_ERR_INVALID_ARG;
  return EP_OK;
}

static bool good(const void* p) { return p != nullptr && ep_host::aligned16(p); }

static Segments segments(const int32_t* counts, const int64_t* psum, int R, int E, int64_t cap_rows, int32_t* status) {
  Segments s;
  s.counts = counts;
  s.psum = psum;
  s.E = E;
  s.E_l = E / R;
  s.cap = cap_rows;
  s.status = status;
  return s;
}

}  // namespace ep

extern "C" int ep_expert_glu(const void* x, const uint8_t* x_scales, const void* w, const uint8_t* w_scales,
                             int fp8_mode, const int32_t* counts, const int64_t* psum, int R, int E, int H,
                             int I, int64_t cap_rows, int act, void* h, uint8_t* h_scales, void* gu,
                             int32_t* status, void* stream) {
  using namespace ep;
  if (fp8_mode != EP_FP8_NONE && fp8_mode != EP_FP8_E4M3_UE8M0) return EP_ERR_INVALID_ARG;
  const bool fp8 = fp8_mode != EP_FP8_NONE;
  const int rc = check_expert(counts, psum, R, E, H, I, cap_rows, fp8 ? kFp8Block : 8);
  if (rc != EP_OK) return rc;
  if (act <= EP_ACT_NONE || act > EP_ACT_GELU) return EP_ERR_INVALID_ARG;
  if (fp8 ? (x_scales == nullptr || w_scales == nullptr || gu != nullptr) : h_scales != nullptr)
    return EP_ERR_INVALID_ARG;
  if (cap_rows == 0) return EP_OK;
  if (!good(x) || !good(w) || !good(h) || !ep_host::aligned16(gu)) return EP_ERR_INVALID_ARG;
  ProductParams p{};
  p.seg = segments(counts, psum, R, E, cap_rows, status);
  p.rows = rows_of(p.seg);
  p.a = x;
  p.a_scales = x_scales;
  p.b = w;
  p.b_scales = w_scales;
  p.K = H;
  p.N = I;
  p.out = h;
  p.out_scales = h_scales;
  p.keep = static_cast<__nv_bfloat16*>(gu);
  p.early = true;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return fp8 ? launch_gemm_e4m3(kGlu, p, act, s) : launch_gemm_bf16(kGlu, p, act, s);
}

extern "C" int ep_expert_glu_backward(const void* dh, const void* gu, const void* x, const void* w,
                                      const int32_t* counts, const int64_t* psum, int R, int E, int H, int I,
                                      int64_t cap_rows, int act, void* dgu, void* dx, void* dw,
                                      int32_t* status, void* stream) {
  using namespace ep;
  int rc = check_expert(counts, psum, R, E, H, I, cap_rows, 8);
  if (rc != EP_OK) return rc;
  if (act <= EP_ACT_NONE || act > EP_ACT_GELU) return EP_ERR_INVALID_ARG;
  if (cap_rows > 0 && (!good(dh) || !good(gu) || !good(dgu) || (dw != nullptr && !good(x)))) return EP_ERR_INVALID_ARG;
  if ((dx != nullptr && cap_rows > 0 && !good(w)) || !ep_host::aligned16(dx) || !ep_host::aligned16(dw))
    return EP_ERR_INVALID_ARG;
  SlopeParams p{};
  p.seg = segments(counts, psum, R, E, cap_rows, status);
  p.dy = static_cast<const __nv_bfloat16*>(dh);
  p.pre = static_cast<const __nv_bfloat16*>(gu);
  p.out = static_cast<__nv_bfloat16*>(dgu);
  p.N = I;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cap_rows > 0) {
    rc = act == EP_ACT_RELU ? launch_glu_slope<EP_ACT_RELU>(p, rows_of(p.seg), s)
       : act == EP_ACT_SILU ? launch_glu_slope<EP_ACT_SILU>(p, rows_of(p.seg), s) : launch_glu_slope<EP_ACT_GELU>(p, rows_of(p.seg), s);
    if (rc != EP_OK) return rc;
  } else {
    dx = nullptr;
  }
  return launch_gradients(false, p.seg, dgu, x, w, H, 2 * I, dx, dw, s);
}

extern "C" int ep_expert_linear(const void* x, const uint8_t* x_scales, const void* w, const uint8_t* w_scales,
                                int fp8_mode, const void* bias, const void* residual, const int32_t* counts,
                                const int64_t* psum, int R, int E, int K, int N, int64_t cap_rows, int act,
                                void* y, void* pre, int32_t* status, void* stream) {
  using namespace ep;
  if (fp8_mode != EP_FP8_NONE && fp8_mode != EP_FP8_E4M3_UE8M0) return EP_ERR_INVALID_ARG;
  const bool fp8 = fp8_mode != EP_FP8_NONE;
  const int rc = check_expert(counts, psum, R, E, K, N, cap_rows, fp8 ? kFp8Block : 8);
  if (rc != EP_OK) return rc;
  if (act < EP_ACT_NONE || act > EP_ACT_GELU) return EP_ERR_INVALID_ARG;
  if (fp8 && (x_scales == nullptr || w_scales == nullptr)) return EP_ERR_INVALID_ARG;
  if (cap_rows == 0) return EP_OK;
  if (!good(x) || !good(w) || !good(y) || !ep_host::aligned16(pre) || !ep_host::aligned16(residual) ||
      !ep_host::aligned16(bias))
    return EP_ERR_INVALID_ARG;
  ProductParams p{};
  p.seg = segments(counts, psum, R, E, cap_rows, status);
  p.rows = rows_of(p.seg);
  p.a = x;
  p.a_scales = x_scales;
  p.b = w;
  p.b_scales = w_scales;
  p.K = K;
  p.N = N;
  p.bias = static_cast<const __nv_bfloat16*>(bias);
  p.residual = static_cast<const __nv_bfloat16*>(residual);
  p.out = y;
  p.keep = static_cast<__nv_bfloat16*>(pre);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return fp8 ? launch_gemm_e4m3(kLinear, p, act, s) : launch_gemm_bf16(kLinear, p, act, s);
}

extern "C" int ep_expert_linear_backward(const void* dy, const void* pre, const void* x, const void* w,
                                         const int32_t* counts, const int64_t* psum, int R, int E, int K,
                                         int N, int64_t cap_rows, int act, void* dpre, void* dx, void* dw,
                                         void* dbias, int32_t* status, void* stream) {
  using namespace ep;
  int rc = check_expert(counts, psum, R, E, K, N, cap_rows, 8);
  if (rc != EP_OK) return rc;
  if (act < EP_ACT_NONE || act > EP_ACT_GELU) return EP_ERR_INVALID_ARG;
  const bool curved = act != EP_ACT_NONE;
  if (cap_rows > 0 && (!good(dy) || (curved && (!good(pre) || !good(dpre))) || (dw != nullptr && !good(x)) ||
                       (dx != nullptr && !good(w))))
    return EP_ERR_INVALID_ARG;
  if (!ep_host::aligned16(dx) || !ep_host::aligned16(dw) || !ep_host::aligned16(dbias)) return EP_ERR_INVALID_ARG;
  SlopeParams p{};
  p.seg = segments(counts, psum, R, E, cap_rows, status);
  p.dy = static_cast<const __nv_bfloat16*>(dy);
  p.pre = static_cast<const __nv_bfloat16*>(pre);
  p.out = static_cast<__nv_bfloat16*>(dpre);
  p.dbias = static_cast<__nv_bfloat16*>(dbias);
  p.N = N;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dbias != nullptr || (curved && cap_rows > 0)) {
    rc = act == EP_ACT_RELU   ? launch_linear_slope<EP_ACT_RELU>(p, s)
         : act == EP_ACT_SILU ? launch_linear_slope<EP_ACT_SILU>(p, s)
         : act == EP_ACT_GELU ? launch_linear_slope<EP_ACT_GELU>(p, s)
                              : launch_linear_slope<EP_ACT_NONE>(p, s);
    if (rc != EP_OK) return rc;
  }
  if (cap_rows == 0) dx = nullptr;
  return launch_gradients(true, p.seg, curved ? dpre : dy, x, w, K, N, dx, dw, s);
}
