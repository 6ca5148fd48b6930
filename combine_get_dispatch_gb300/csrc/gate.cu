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
// Issue slots bound the choice, memory nearly bounds the gradient.  NaN becomes
// -inf on the way in; -inf is never chosen.

#include "ep_common.cuh"

namespace ep {

constexpr int kForwardThreads = 256, kBackwardThreads = 128;
constexpr int kBackwardCtas = 8;   // of an SM
// Up to 8 logits a lane are loaded one row ahead; more take too many registers
// (131072 x 256, two tokens a warp: 70 us with the row ahead, 47 without; 45 now).
__host__ __device__ constexpr bool row_ahead(int logits) { return logits <= 8; }
__host__ __device__ constexpr int forward_ctas(int logits) { return row_ahead(logits) ? 5 : 4; }

struct GateParams {
  const void* logits;
  int64_t T;
  int E, k;
  const float* grad;
  int64_t* idx;
  float* w;
  void* grad_logits;
  int32_t* status;
  bool vec;   // rows are whole 16-byte pieces
};

// Over the kG lanes of a token; every lane has the result.
template <int kG, typename Op>
__device__ __forceinline__ float group_reduce(float v, Op op) {
#pragma unroll
  for (int o = kG / 2; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
struct Max {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct Min {
  __device__ __forceinline__ float operator()(float a, float b) const { return fminf(a, b); }
};
struct Sum {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};

// The same, by one instruction where the lanes are the whole warp.
template <int kG>
__device__ __forceinline__ float group_max(float v) {
  if (kG < kWarp) return group_reduce<kG>(v, Max());
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
template <int kG>
__device__ __forceinline__ float group_min(float v) {
  if (kG < kWarp) return group_reduce<kG>(v, Min());
  float r;
  asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
template <int kG>
__device__ __forceinline__ int group_total(int v) {
  if constexpr (kG == kWarp) {
    return __reduce_add_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = kG / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
}
// Sum over the lanes of a token up to this one.
template <int kG>
__device__ __forceinline__ int group_scan(int v) {
#pragma unroll
  for (int o = 1; o < kG; o <<= 1)
    asm volatile("{\n .reg .u32 r;\n .reg .pred p;\n shfl.sync.up.b32 r|p, %0, %1, %2, 0xffffffff;\n @p add.u32 %0, %0, r;\n}\n"
                 : "+r"(v)
                 : "r"(o), "n"((kWarp - kG) << 8));
  return v;
}

constexpr float kNone = -INFINITY;   // an expert that is never chosen
constexpr float kLowest = -3.40282346638528859812e+38f;

// exp(l - m): the difference rounds once and its product with log2(e) once, so
// it is off by |l - m| 2^-23 of itself; below 2^-126 it is 0.  m is finite.  Logits of
// a spread of 1.5: weights 6.4e-8 off (rms), 5.6e-8 by expf and a rounded quotient.
__device__ __forceinline__ float gate_exp(float l, float m) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"((l - m) * 1.44269504f));
  return r;
}

// A logit as the kernels see it: NaN is an expert that is never chosen.
__device__ __forceinline__ float gate_clean(float l) { return fmaxf(l, kNone); }

template <bool kBf16>
__device__ __forceinline__ float gate_load(const void* logits, int64_t at) {
  if (kBf16) return gate_clean(__uint_as_float((uint32_t)static_cast<const uint16_t*>(logits)[at] << 16));
  return gate_clean(static_cast<const float*>(logits)[at]);
}

// A lane's kV logits of a row, as they are stored (-inf past its end, or without
// one): pieces of kP in turn over the kG lanes, so that those read whole lines.
// vec: rows are whole 16-byte pieces.
template <int kG, int kV, bool kBf16>
struct Row {
  static constexpr int kP = kV < (kBf16 ? 8 : 4) ? kV : (kBf16 ? 8 : 4);
  static constexpr int kWords = kV * (kBf16 ? 2 : 4) / 4, kPieceWords = kP * (kBf16 ? 2 : 4) / 4;
  uint32_t w[kWords];

  // The expert of lane g's value i.
  static __device__ __forceinline__ int expert(int g, int i) { return (i / kP * kG + g) * kP + i % kP; }

  __device__ __forceinline__ void load(const GateParams& p, bool in, int64_t row, int g) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = kBf16 ? 0xff80ff80u : 0xff800000u;   // -inf
    if (!in) return;
    if (p.vec) {
      const uint8_t* src = static_cast<const uint8_t*>(p.logits) + (row + g * kP) * (kBf16 ? 2 : 4);
#pragma unroll
      for (int i = 0; i < kV / kP; ++i) {
        if (expert(g, i * kP) < p.E) {
          if (kPieceWords == 4) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + i * kG);
            w[kPieceWords * i] = v.x;
            w[kPieceWords * i + kPieceWords / 4] = v.y;
            w[kPieceWords * i + kPieceWords / 2] = v.z;
            w[kPieceWords * i + kPieceWords - 1] = v.w;
          } else if (kPieceWords == 2) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(src) + i * kG);
            w[kPieceWords * i] = v.x;
            w[kPieceWords * i + kPieceWords - 1] = v.y;
          } else {
            w[i] = __ldg(reinterpret_cast<const uint32_t*>(src) + i * kG);
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        if (expert(g, i) < p.E) {
          if (kBf16) {
            const uint32_t u = static_cast<const uint16_t*>(p.logits)[row + expert(g, i)];
            w[i / 2] = (i & 1) ? (w[i / 2] & 0xffffu) | u << 16 : (w[i / 2] & 0xffff0000u) | u;
          } else {
            w[kBf16 ? 0 : i] = static_cast<const uint32_t*>(p.logits)[row + expert(g, i)];
          }
        }
      }
    }
  }
  __device__ __forceinline__ void get(float (&l)[kV]) const {
#pragma unroll
    for (int i = 0; i < kV; ++i)
      l[i] = gate_clean(kBf16 ? ((i & 1) ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2])) : __uint_as_float(w[kBf16 ? 0 : i]));
  }
};

// The value to subtract, from the row's largest logit: itself, or 0 where nothing
// can be chosen.
__device__ __forceinline__ float gate_base(float most) { return most == kNone ? 0.0f : most; }

// As gate_exp in a row whose largest logit is +inf.
__device__ __forceinline__ float gate_share(float l) { return l == INFINITY ? 1.0f : 0.0f; }

__device__ __forceinline__ float gate_weight(float l, float m) { return m < INFINITY ? gate_exp(l, m) : gate_share(l); }

// The places of a lane's candidates in the falling order of the list: the number
// of larger logits, and (exact) of equal ones of a lower expert.  The list is
// padded with -inf to a multiple of 8.
template <int kOwn>
__device__ __forceinline__ void gate_places(const float* logits, int all, const float (&mine)[kOwn], int (&place)[kOwn]) {
#pragma unroll
  for (int o = 0; o < kOwn; ++o) place[o] = 0;
  for (int j = 0; j < all; j += 8) {
    const float4 x = *reinterpret_cast<const float4*>(logits + j), y = *reinterpret_cast<const float4*>(logits + j + 4);
#pragma unroll
    for (int o = 0; o < kOwn; ++o) {
      place[o] += (x.x > mine[o] ? 1 : 0) + (x.y > mine[o] ? 1 : 0) + (x.z > mine[o] ? 1 : 0) + (x.w > mine[o] ? 1 : 0);
      place[o] += (y.x > mine[o] ? 1 : 0) + (y.y > mine[o] ? 1 : 0) + (y.z > mine[o] ? 1 : 0) + (y.w > mine[o] ? 1 : 0);
    }
  }
}
__device__ __forceinline__ int gate_place_exact(const float* logits, const int* experts, int all, float mine, int expert) {
  int place = 0;
  for (int j = 0; j < all; ++j) {
    const float x = logits[j];
    place += x > mine || (x == mine && experts[j] < expert) ? 1 : 0;
  }
  return place;
}

// Writes a logit and its expert (32 words on) where the logit is a candidate, and
// moves on.
__device__ __forceinline__ void gate_put(uint32_t& at, float l, float least, int expert) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ge.f32 p, %1, %2;\n @p st.shared.f32 [%0], %1;\n @p st.shared.u32 [%0 + 128], %3;\n"
      " @p add.u32 %0, %0, 4;\n}\n"
      : "+r"(at)
      : "f"(l), "f"(least), "r"(expert)
      : "memory");
}

// A finite bf16 logit with its expert in the 16 bits below it: equal logits (and
// zeros of both signs) then fall in the order of their experts.
__device__ __forceinline__ float gate_unique(float l, int expert) {
  const uint32_t u = __float_as_uint(l + 0.0f);
  return __uint_as_float(u | (uint32_t)((u & 0x80000000u) ? expert : 0xffff - expert));
}

// The k largest of a token's logits, one round a choice: the largest, and the
// lowest expert that has it.  Lane j of the result holds choice j (-inf: none).
template <int kG, int kV, bool kBf16>
__device__ __forceinline__ void gate_choose(float (&l)[kV], int k, int g, float& my_l, int& my_idx) {
  my_l = kNone;
  my_idx = -1;
  for (int j = 0; j < k; ++j) {
    float b = kNone;
    int e = 0;
#pragma unroll
    for (int i = 0; i < kV; ++i)
      if (l[i] > b) {
        b = l[i];
        e = Row<kG, kV, kBf16>::expert(g, i);
      }
    const float top = group_max<kG>(b);   // -inf: nothing left to choose
    // below 2^24: whole numbers, larger is lower
    e = -(int)group_max<kG>(b == top ? (float)-e : kNone);
    if (g == j && top != kNone) {
      my_l = top;
      my_idx = e;
    }
#pragma unroll
    for (int i = 0; i < kV; ++i)
      if (e == Row<kG, kV, kBf16>::expert(g, i)) l[i] = kNone;
  }
}

// A lower bound of a row's k-th largest logit: the k-th of the lanes' largest, by
// their places.
template <int kG>
__device__ __forceinline__ float gate_bound(float* list, float best, int k, int g) {
  __syncwarp();
  list[g] = best;
  __syncwarp();
  int place[1];
  gate_places<1>(list, kG, {best}, place);
  return group_min<kG>(place[0] < k ? best : INFINITY);
}

// The same for 32 lanes and k <= 8, cheaper and not as close: eight disjoint groups
// of four lanes have a largest logit each, and the least of those is no larger;
// the better of two such groupings.  (For k = 16 groups of two lanes mostly kept
// more than 32 candidates of 512: 178 us for 65536 tokens.)
__device__ __forceinline__ float gate_bound8(float best) {
  float near = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 1)), far = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 16));
  near = fmaxf(near, __shfl_xor_sync(0xffffffffu, near, 2));
  far = fmaxf(far, __shfl_xor_sync(0xffffffffu, far, 8));
  return fmaxf(group_min<kWarp>(near), group_min<kWarp>(far));
}

// kG lanes (16: two tokens a warp; 32) per token, kV logits each.  Most logits are
// thrown out first: only those at or above a bound of the k-th largest can be
// chosen (11 to 17 of 256 on average for k = 8).  The others go to a list of 32, one or
// two to a lane, and the larger ones of each are counted.  Equal logits, in the
// order of their experts, are looked at only where they have left a gap in the
// places; bf16 logits, often equal, are made unique.  Rows where more than 32
// remain take their choices one round at a time.  Issue slots bound it (0.77 taken):
// about 300 instructions a token, 45 us for 131072 x 256, top-8 (21.7 us to read
// and write them).  A warp a token took 53 us there against 47, 24.6 against 20.5 for 65536 x
// 128, top-6, and 21.5 against 17.5 for 65536 x 64, top-2; 64 bytes in a row a
// lane instead of 16-byte pieces in turn 51, and 55 against 43 for 32768 x 1024.
// Slower: k rounds of a reduction and a ballot over the list; 8 lanes a token (99
// us: registers for half the warps).
template <int kG, int kV, bool kBf16, bool kTopk>
__global__ void __launch_bounds__(kForwardThreads, kV <= 16 ? forward_ctas(kV) : 1) k_gate(GateParams p) {
  constexpr int kOwn = kWarp / kG;   // tokens of a warp; places of the list a lane has
  __shared__ float4 lists[kForwardThreads / kG][2 * kWarp / 4];   // 32 logits, their 32 experts
  const int g = threadIdx.x % kG;
  float* list = reinterpret_cast<float*>(lists[threadIdx.x / kG]);
  const int* experts = reinterpret_cast<const int*>(list + kWarp);
  const uint32_t list_at = smem_addr(list);
  const int64_t step = (int64_t)gridDim.x * (kForwardThreads / kG);
  // all lanes of a warp go round as long as its first token is one
  int64_t t = (int64_t)blockIdx.x * (kForwardThreads / kG) + threadIdx.x / kG;
  Row<kG, kV, kBf16> row;
  if (row_ahead(kV)) row.load(p, t < p.T, t * p.E, g);
  for (; t - (threadIdx.x & 31) / kG < p.T; t += step) {
    float l[kV];
    if (!row_ahead(kV)) row.load(p, t < p.T, t * p.E, g);
    row.get(l);
    if (row_ahead(kV)) row.load(p, t + step < p.T, (t + step) * p.E, g);   // arrives while this one is worked on
    float best = l[0];
#pragma unroll
    for (int i = 1; i < kV; ++i) best = fmaxf(best, l[i]);
    const float m = gate_base(group_max<kG>(best));
    // at least the type's lowest value, so that -inf is no candidate
    const float least = fmaxf(kLowest, kG == kWarp && p.k <= 8 ? gate_bound8(best) : gate_bound<kG>(list, best, p.k, g));
    int own = 0;
#pragma unroll
    for (int i = 0; i < kV; ++i) own += l[i] >= least ? 1 : 0;
    const int upto = group_scan<kG>(own), all = __shfl_sync(0xffffffffu, upto, kG - 1, kG);
    float total = 0.0f;
    if (!kTopk) {
      if (m < INFINITY) {
#pragma unroll
        for (int i = 0; i < kV; ++i) total += gate_exp(l[i], m);
      } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) total += gate_share(l[i]);
      }
      total = group_reduce<kG>(total, Sum());
    }
    float my_l[kOwn];
    int my_idx[kOwn], place[kOwn], found = min(p.k, all);
#pragma unroll
    for (int j = 1; j < kOwn; ++j) {
      my_l[j] = kNone;
      my_idx[j] = -1;
      place[j] = p.k;
    }
    if (__all_sync(0xffffffffu, all <= kWarp)) {
      const bool more = kOwn > 1 && __any_sync(0xffffffffu, all > kG);   // a lane has a second candidate
      __syncwarp();
#pragma unroll
      for (int j = 0; j < kOwn; ++j) list[g + j * kG] = kNone;
      __syncwarp();
      uint32_t at = list_at + 4 * (upto - own);
#pragma unroll
      for (int i = 0; i < kV; ++i) gate_put(at, l[i], least, row.expert(g, i));
      __syncwarp();
      auto fetch = [&](int j) {
        my_l[j] = list[g + j * kG];
        my_idx[j] = experts[g + j * kG];
        return kBf16 && m < INFINITY ? gate_unique(my_l[j], my_idx[j]) : my_l[j];
      };
      float key[kOwn];
      key[0] = fetch(0);
      if (more) key[kOwn - 1] = fetch(kOwn - 1);
      if (kBf16) {
        __syncwarp();
        if (g < all) list[g] = key[0];
        if (more && g + kG < all) list[g + kG] = key[kOwn - 1];
        __syncwarp();
      }
      if (more)
        gate_places<kOwn>(list, all, key, place);
      else
        gate_places<1>(list, all, {key[0]}, reinterpret_cast<int(&)[1]>(place[0]));
      // the places below k are as many as there are choices, each once, unless equal logits share one
      int taken = 0;
#pragma unroll
      for (int j = 0; j < kOwn; ++j) taken += g + j * kG < all && place[j] < p.k ? (1 << 16) + place[j] : 0;
      taken = group_total<kG>(taken);
      if (taken != (found << 16) + found * (found - 1) / 2) {
        place[0] = gate_place_exact(list, experts, all, key[0], my_idx[0]);
        if (more) place[kOwn - 1] = gate_place_exact(list, experts, all, key[kOwn - 1], my_idx[kOwn - 1]);
      }
#pragma unroll
      for (int j = 0; j < kOwn; ++j)
        if (g + j * kG >= all) place[j] = p.k;
    } else {
      gate_choose<kG, kV, kBf16>(l, p.k, g, my_l[0], my_idx[0]);
      place[0] = my_idx[0] >= 0 ? g : p.k;
    }
    float ex[kOwn], chosen = 0.0f;
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      ex[j] = place[j] < p.k ? gate_weight(my_l[j], m) : 0.0f;
      chosen += ex[j];
    }
    if (kTopk) total = group_reduce<kG>(chosen, Sum());
    if (t < p.T) {
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        if (place[j] < p.k) {
          p.idx[t * p.k + place[j]] = my_idx[j];
          p.w[t * p.k + place[j]] = __fdividef(ex[j], total);   // 1 <= total <= E: within 2 ulp
        }
      }
      if (g >= found && g < p.k) {
        p.idx[t * p.k + g] = -1;
        p.w[t * p.k + g] = 0.0f;
      }
    }
  }
}

// In the gradient value v of lane g is expert (v / kP * kG + g) * kP + v % kP:
// 16-byte pieces in turn, so that the lanes of a token read whole lines.
template <bool kBf16>
struct Piece {
  static constexpr int kP = kBf16 ? 8 : 4;
};
// A lane's logits of the row at `row`, -inf past its end (or for no row at all).
// p.vec: rows are whole 16-byte pieces.
template <int kG, int kV, bool kBf16>
__device__ __forceinline__ void gate_pieces(const GateParams& p, bool in, const uint8_t* row, int g, float (&l)[kV]) {
  constexpr int kP = Piece<kBf16>::kP, kN = kV / kP;
  if (p.vec) {
    const uint32_t none = kBf16 ? 0xff80ff80u : 0xff800000u;
    uint4 x[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      x[i] = make_uint4(none, none, none, none);
      if (in && (i * kG + g) * kP < p.E) x[i] = __ldg(reinterpret_cast<const uint4*>(row + g * 16 + i * kG * 16));
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int c = 0; c < kP; ++c)
        l[i * kP + c] = gate_clean(kBf16 ? ((c & 1) ? bf16_hi(w[c / 2]) : bf16_lo(w[c / 2])) : __uint_as_float(w[c % 4]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int e = (i / kP * kG + g) * kP + i % kP;
      l[i] = in && e < p.E ? gate_load<kBf16>(row, e) : kNone;
    }
  }
}

// kG lanes (8, 16 or 32) hold a token's logits, up to 32 each, so that a warp works
// on several tokens at once (32768 x 256 fp32: 14.4 us, 4.9 TB/s; 16 lanes a
// token 15.5, a warp 18; memory bounds it).  All loads are issued before the
// first is used (one after another they took 22 us).  Every
// lane stores the gradient of its own logits (-p inner, or zero); then the lanes
// of the chosen experts store those whole.
template <int kG, int kV, bool kBf16, bool kTopk>
__global__ void __launch_bounds__(kBackwardThreads, kBackwardCtas) k_gate_backward(GateParams p) {
  constexpr int kTokens = kWarp / kG, kP = Piece<kBf16>::kP;
  const int lane = threadIdx.x & 31, g = lane % kG, token = lane / kG;
  const int64_t warp0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  for (int64_t t0 = warp0 * kTokens; t0 < p.T; t0 += nwarps * kTokens) {
    const int64_t t = t0 + token;
    const bool in = t < p.T;
    // every load that waits for nothing first: the slot's id and gradient, the row
    int64_t id = -1;   // of slot g (k <= kG)
    float grad = 0.0f;
    if (in && g < p.k) {
      id = p.idx[t * p.k + g];
      grad = p.grad[t * p.k + g];
    }
    float l[kV];
    if (!kTopk)
      gate_pieces<kG, kV, kBf16>(p, in, static_cast<const uint8_t*>(p.logits) + t * p.E * (kBf16 ? 2 : 4), g, l);
    int my_idx = -1;
    float chosen = kNone;
    if (id < -1 || id >= p.E)
      set_status(p.status, EP_ERR_INVALID_ARG);
    else if (id >= 0) {
      my_idx = (int)id;
      chosen = gate_load<kBf16>(p.logits, t * p.E + my_idx);
    }
    if (chosen == kNone) grad = 0.0f;
    float best = chosen;
    if (!kTopk) {
#pragma unroll
      for (int i = 0; i < kV; ++i) best = fmaxf(best, l[i]);
    }
    const float most = group_reduce<kG>(best, Max());
    const float m = most == kNone ? 0.0f : most;
    const float ex = gate_weight(chosen, m);
    float total = ex;
    if (!kTopk) {
      total = 0.0f;
      if (__all_sync(0xffffffffu, m < INFINITY)) {
#pragma unroll
        for (int i = 0; i < kV; ++i) l[i] = gate_exp(l[i], m);
      } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) l[i] = gate_weight(l[i], m);
      }
#pragma unroll
      for (int i = 0; i < kV; ++i) total += l[i];
    }
    total = group_reduce<kG>(total, Sum());
    const float inv = total > 0.0f ? 1.0f / total : 0.0f;
    const float w = ex * inv;
    const float inner = group_reduce<kG>(w * grad, Sum());
    const float add = kTopk ? w * (grad - inner) : w * grad;
    const float scale = -inv * inner;
#pragma unroll
    for (int i = 0; i < kV / kP; ++i) {
      const int e0 = (i * kG + g) * kP;
      float d[kP];
#pragma unroll
      for (int c = 0; c < kP; ++c) d[c] = kTopk ? 0.0f : l[i * kP + c] * scale;
      if (p.vec) {
        if (in && e0 < p.E) {
          uint4 x;
          if (kBf16)
            x = make_uint4(pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3]), pack_bf16x2(d[kP - 4], d[kP - 3]),
                           pack_bf16x2(d[kP - 2], d[kP - 1]));
          else
            x = make_uint4(__float_as_uint(d[0]), __float_as_uint(d[1]), __float_as_uint(d[2]), __float_as_uint(d[3]));
          st_v4(static_cast<uint8_t*>(p.grad_logits) + (t * p.E + e0) * (kBf16 ? 2 : 4), x);
        }
      } else {
#pragma unroll
        for (int c = 0; c < kP; ++c) {
          if (in && e0 + c < p.E) {
            if (kBf16)
              static_cast<__nv_bfloat16*>(p.grad_logits)[t * p.E + e0 + c] = __float2bfloat16_rn(d[c]);
            else
              static_cast<float*>(p.grad_logits)[t * p.E + e0 + c] = d[c];
          }
        }
      }
    }
    // a token that names an expert twice: the terms in slot order, the same sum from every slot
    float own = kTopk ? 0.0f : ex * scale;
    for (int j = 0; j < p.k; ++j) {
      const int ej = __shfl_sync(0xffffffffu, my_idx, j, kG);
      const float aj = __shfl_sync(0xffffffffu, add, j, kG);
      if (ej == my_idx) own += aj;
    }
    __syncwarp();   // the row's stores come first
    if (my_idx >= 0) {
      if (kBf16)
        static_cast<__nv_bfloat16*>(p.grad_logits)[t * p.E + my_idx] = __float2bfloat16_rn(own);
      else
        static_cast<float*>(p.grad_logits)[t * p.E + my_idx] = own;
    }
  }
}

template <int kG, int kV, bool kBf16, bool kTopk>
static int launch_backward_t(const GateParams& p, cudaStream_t stream) {
  constexpr int kTokens = kBackwardThreads / kG;   // of a CTA
  const int64_t want = (p.T + kTokens - 1) / kTokens;
  const int grid = (int)std::min<int64_t>(want, ep_host::grid_cap(kBackwardCtas));
  k_gate_backward<kG, kV, kBf16, kTopk><<<grid, kBackwardThreads, 0, stream>>>(p);
  ep_host::count_launch();
  return ep_host::check_launch();
}
template <int kG, int kV, bool kBf16, bool kTopk>
static int launch_forward_t(const GateParams& p, cudaStream_t stream) {
  constexpr int kTokens = kForwardThreads / kG;
  const int64_t want = (p.T + kTokens - 1) / kTokens;
  const int grid = (int)std::min<int64_t>(want, ep_host::grid_cap(forward_ctas(kV)));
  k_gate<kG, kV, kBf16, kTopk><<<grid, kForwardThreads, 0, stream>>>(p);
  ep_host::count_launch();
  return ep_host::check_launch();
}

template <int kG, int kV>
static int launch_backward(const GateParams& p, bool bf16, bool topk, cudaStream_t s) {
  if (bf16) return topk ? launch_backward_t<kG, kV, true, true>(p, s) : launch_backward_t<kG, kV, true, false>(p, s);
  return topk ? launch_backward_t<kG, kV, false, true>(p, s) : launch_backward_t<kG, kV, false, false>(p, s);
}
template <int kG, int kV>
static int launch_forward(const GateParams& p, bool bf16, bool topk, cudaStream_t s) {
  if (bf16) return topk ? launch_forward_t<kG, kV, true, true>(p, s) : launch_forward_t<kG, kV, true, false>(p, s);
  return topk ? launch_forward_t<kG, kV, false, true>(p, s) : launch_forward_t<kG, kV, false, false>(p, s);
}

static int launch_gate(const GateParams& params, int dtype, int score, bool backward, cudaStream_t s) {
  if (params.T == 0) return EP_OK;
  const bool bf16 = dtype == EP_DTYPE_BF16, topk = score == EP_GATE_SOFTMAX_TOPK;
  GateParams p = params;
  p.vec = p.E % (bf16 ? 8 : 4) == 0 && ep_host::aligned16(p.logits) && (!backward || ep_host::aligned16(p.grad_logits));
  if (!backward) {
    // Two tokens a warp while their lists mostly hold what is left of a row (131072 x 256: top-9 44 us against
    // 61 by a warp a token, top-12 57 against 61, top-13 77 against 63; x 64, top-16 86 against 51) and their
    // rows fit the registers (65536 x 512, top-8: 40 us either way).
    if (p.k <= 12) {
      if (p.E <= 64) return launch_forward<16, 4>(p, bf16, topk, s);
      if (p.E <= 128) return launch_forward<16, 8>(p, bf16, topk, s);
      if (p.E <= 256) return launch_forward<16, 16>(p, bf16, topk, s);
    }
    if (p.E <= 64) return launch_forward<32, 2>(p, bf16, topk, s);
    if (p.E <= 128) return launch_forward<32, 4>(p, bf16, topk, s);
    if (p.E <= 256) return launch_forward<32, 8>(p, bf16, topk, s);
    if (p.E <= 512) return launch_forward<32, 16>(p, bf16, topk, s);
    return launch_forward<32, 32>(p, bf16, topk, s);
  }
  // as few lanes a token as hold its logits in 32 registers each and its k slots in one each
  if (p.k <= 8) {
    if (p.E <= 64) return launch_backward<8, 8>(p, bf16, topk, s);
    if (p.E <= 128) return launch_backward<8, 16>(p, bf16, topk, s);
    if (p.E <= 256) return launch_backward<8, 32>(p, bf16, topk, s);
  }
  if (p.E <= 128) return launch_backward<16, 8>(p, bf16, topk, s);
  if (p.E <= 512) return launch_backward<16, 32>(p, bf16, topk, s);
  return launch_backward<32, 32>(p, bf16, topk, s);
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
