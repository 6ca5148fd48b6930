// few.cuh -- what the kernels of the layer for few tokens share: the call, its
// lists of used experts and their slots, a CTA's walk over its columns, waits.
#pragma once

#include "expert.cuh"
#include "umma.cuh"

namespace ep {

constexpr int kFewSmem = 226 * 1024;
constexpr int kCrossing = 16;   // columns: what a narrow unit at an expert's end costs by its products (one token: bf16 43 us without, 41 so; E4M3 76, 69)

// h between the kernels has more than bf16's 8 bits (with bf16 weights two words, with E4M3 fp32), so that the output
// is as near as its own rounding lets it be: with h rounded to bf16 it is 1.4 times as far off.  In every call, so that a
// token comes out the same whatever the batch, though 64 bf16 tokens through eight experts of 4096 x 2048 take 86 us
// and 74 with h in bf16, as tokens' bytes count there (one token 39 either way; 32 on E4M3 weights 763, 767).
constexpr int kHiddenBytes = 4;

struct FewCall {
  const uint8_t* scales;       // of E4M3 weights
  const __nv_bfloat16* v;      // kIn: x [T, H]; kOut: h [T k, 2, I], or fp32 [T k, I]
  const int64_t* idx;          // [T, k]
  const float* weights;
  __nv_bfloat16* out;          // kIn: h; kOut: out [T, H]
  int32_t* status;
  int T, k, E, K, N;           // K: inner extent; N: columns of h or out
  uint32_t wave;               // CTAs that run at once
};

// What every CTA works out first: the used experts in rising order, and their
// slots in rising order.
struct FewCounts {
  int group_slots[kMaxE / kWarp], group_used[kMaxE / kWarp], group_most[kMaxE / kWarp];   // of 32 experts
  int n_used, most;                    // used experts; slots of the largest
};
struct FewUsed {
  int16_t expert, first, count, pad;   // slots first .. first + count of the lists
};
template <int kUnitRows>
struct FewLists {
  FewUsed* used;             // [E]
  float* weight;             // [n], as the next three
  int16_t *slot, *token, *id;   // id: expert of a slot, -1: unused
  int16_t* start;            // [E]
  float* sums;               // kOut: [T][kUnitRows], the columns in hand
  static __host__ __device__ int bytes(int E, int T, int k) { return (E * 10 + T * k * 10 + T * kUnitRows * 4 + 127) / 128 * 128; }
  __device__ __forceinline__ FewLists(uint8_t* at, int E, int T, int k) {
    used = reinterpret_cast<FewUsed*>(at);
    sums = reinterpret_cast<float*>(used + E);
    weight = sums + T * kUnitRows;
    slot = reinterpret_cast<int16_t*>(weight + T * k);
    token = slot + T * k;
    id = token + T * k;
    start = id + T * k;
  }
};

// masks: a bit a slot for every expert; memory that nothing else uses yet.
template <int kThreads, int kUnitRows>
__device__ __forceinline__ void few_lists(const FewCall& p, FewCounts& sh, const FewLists<kUnitRows>& l, uint32_t* masks, bool report) {
  const int n = p.T * p.k, words = (n + 31) / 32, groups = (p.E + 31) / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (n <= kWarp) {   // one warp by itself, a slot a lane: places by counting the slots before (2.3 us more the other way, four tokens of two)
    if (warp == 0) {
      const int64_t id = lane < n ? p.idx[lane] : -1;
      const bool fits = id >= 0 && id < p.E;
      if (report && !fits && id != -1) set_status(p.status, EP_ERR_INVALID_ARG);
      const int e = fits ? (int)id : kMaxE;
      const float weight = fits ? p.weights[lane] : 0.0f;
      const uint32_t same = __match_any_sync(0xffffffffu, e);
      const bool leads = fits && (same & lanemask_lt()) == 0;
      int at = __popc(same & lanemask_lt()), d = 0;
      for (int i = 0; i < n; ++i) {
        const int other = __shfl_sync(0xffffffffu, e, i);
        const bool other_leads = __shfl_sync(0xffffffffu, leads, i);
        at += other < e;
        d += other < e && other_leads;
      }
      const int c = __popc(same);
      if (fits) {
        l.slot[at] = (int16_t)lane;
        l.token[at] = (int16_t)(lane / p.k);
        l.weight[at] = weight;
        if (leads) l.used[d] = {(int16_t)e, (int16_t)at, (int16_t)c, 0};
      }
      const int used = __popc(__ballot_sync(0xffffffffu, leads)), most = __reduce_max_sync(0xffffffffu, fits ? c : 0);
      if (lane == 0) {
        sh.n_used = used;
        sh.most = most;
      }
    }
    __syncthreads();
    return;
  }
  for (int i = threadIdx.x; i < p.E * words; i += kThreads) masks[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int64_t e = p.idx[i];
    const bool fits = e >= 0 && e < p.E;
    if (report && !fits && e != -1) set_status(p.status, EP_ERR_INVALID_ARG);
    if (fits) atomicOr(masks + (int)e * words + (i >> 5), 1u << (i & 31));
    l.id[i] = fits ? (int16_t)e : (int16_t)-1;
  }
  __syncthreads();
  auto count_of = [&](int e) {
    int c = 0;
    if (e < p.E)
      for (int w = 0; w < words; ++w) c += __popc(masks[e * words + w]);
    return c;
  };
  for (int q = warp; q < groups; q += kThreads / kWarp) {
    const int c = count_of(q * 32 + lane);
    const int all = __reduce_add_sync(0xffffffffu, c), most = __reduce_max_sync(0xffffffffu, c);
    const uint32_t some = __ballot_sync(0xffffffffu, c > 0);
    if (lane == 0) {
      sh.group_slots[q] = all;
      sh.group_used[q] = __popc(some);
      sh.group_most[q] = most;
    }
  }
  __syncthreads();
  for (int q = warp; q < groups; q += kThreads / kWarp) {
    const bool before = lane < q;
    const int slots = __reduce_add_sync(0xffffffffu, before ? sh.group_slots[lane] : 0);
    const int used = __reduce_add_sync(0xffffffffu, before ? sh.group_used[lane] : 0);
    const int c = count_of(q * 32 + lane);
    int upto = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const uint32_t some = __ballot_sync(0xffffffffu, c > 0);
    if (c > 0) {
      const int first = slots + upto - c;
      l.used[used + __popc(some & lanemask_lt())] = {(int16_t)(q * 32 + lane), (int16_t)first, (int16_t)c, 0};
      l.start[q * 32 + lane] = (int16_t)first;
    }
    if (q == 0) {
      const int all = __reduce_add_sync(0xffffffffu, lane < groups ? sh.group_used[lane] : 0);
      const int most = __reduce_max_sync(0xffffffffu, lane < groups ? sh.group_most[lane] : 0);
      if (lane == 0) {
        sh.n_used = all;
        sh.most = most;
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int e = l.id[i];
    if (e < 0) continue;
    int at = l.start[e] + __popc(masks[e * words + (i >> 5)] & ((1u << (i & 31)) - 1));
    for (int w = 0; w < (i >> 5); ++w) at += __popc(masks[e * words + w]);
    l.slot[at] = (int16_t)i;
    l.token[at] = (int16_t)(i / p.k);
    l.weight[at] = p.weights[i];
  }
  fence_proxy_async_smem();   // copies will land where the masks are
  __syncthreads();
}

// A CTA's units, one after another: `cols` columns from `col` on of expert e, for
// the tokens s0 .. s0 + m of the lists.
template <bool kIn, int kPass, int kUnitRows>
struct FewWalk {
  const FewUsed* used;
  int n_used;
  int N, left;           // kIn: (expert, column) pairs to come, from `col` of expert d on; kOut: columns from `col` on
  int d, e, col, cols, s0, m, behind;   // behind: the expert's tokens after these
  bool last;             // kOut: last unit of these columns
  int most;              // columns of the widest unit

  __device__ __forceinline__ FewWalk(const FewUsed* list, int count, int n, uint32_t wave) {
    used = list;
    n_used = count;
    N = n;
    const uint32_t all = kIn ? (uint32_t)n_used * (n + kCrossing) : n_used > 0 ? n : 0;   // below 2^32
    // 16 parts a CTA; two for each of kIn's CTAs that come after the first wave
    const uint32_t first = min(gridDim.x, wave), parts = 16 * first + 2 * (gridDim.x - first);
    const uint32_t b = blockIdx.x < first ? 16 * blockIdx.x : 14 * first + 2 * blockIdx.x, size = blockIdx.x < first ? 16 : 2;
    // the first `more` parts have one more, so that in one wave shares are multiples of 16 columns, as copies are, but where
    // widths are not (four tokens, 256 x 128, bf16: 10.8 us by single columns, 9.5 by 8, 9.2 by 16; 16 tokens, 2560 x 1536,
    // E4M3: 81, 79, 79)
    const uint32_t each = all / parts, more = all - each * parts;
    const uint32_t at = each * b + min(b, more);
    left = (int)(each * size + min(b + size, more) - min(b, more));
    most = min(kIn ? kUnitRows / 2 : kUnitRows, left);
    d = kIn ? (int)(at / (uint32_t)(n + kCrossing)) : n_used - 1;
    col = (int)(kIn ? at - (uint32_t)d * (n + kCrossing) : at);
    cols = s0 = m = behind = 0;
  }
  __device__ __forceinline__ bool next() {
    if (behind > 0) {
      s0 += m;
    } else {
      if (kIn) {
        left -= cols;
        col += cols;
        if (col >= N) {
          left -= N + kCrossing - col;
          col = 0;
          ++d;
        }
        if (left <= 0) return false;
        cols = min(min(kUnitRows / 2, N - col), left);
      } else {
        if (++d >= n_used) {
          left -= cols;
          col += cols;
          if (left <= 0) return false;
          cols = min(kUnitRows, left);
          d = 0;
        }
      }
      const FewUsed u = used[d];
      e = u.expert;
      s0 = u.first;
      behind = u.count;
    }
    m = min(kPass, behind);
    behind -= m;
    last = !kIn && behind == 0 && d + 1 == n_used;
    return true;
  }
};

// A bounded wait that looks at the clock (a slow read) only after some tries.
__device__ __forceinline__ bool wait_few(uint64_t* bar, uint32_t parity, uint64_t limit_ns = kWaitNs) {
  bool ok = false;
  for (int i = 0; i < 32 && !ok; ++i) ok = mbar_try_wait(bar, parity);
  return __all_sync(0xffffffffu, ok || mbar_wait_bounded(bar, parity, limit_ns));
}

// The same for a thread by itself.
__device__ __forceinline__ bool wait_alone(uint64_t* bar, uint32_t parity, uint64_t limit_ns = kWaitNs) {
  for (int i = 0; i < 32; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait_bounded(bar, parity, limit_ns);
}

// Where a role is in a ring.
struct RingPosition {
  int s, size;
  uint32_t phase;

  __device__ __forceinline__ RingPosition(int n) : s(0), size(n), phase(0) {}
  __device__ __forceinline__ void advance() {
    if (++s == size) {
      s = 0;
      phase ^= 1;
    }
  }
};

// A half of the layer: kIn or kOut; waves: how many times the CTAs that run at once.
template <typename Params>
int launch_few_half(void (*fn)(Params), int threads, const Params& in, int waves, cudaStream_t s) {
  if (ep_host::ensure_max_smem(reinterpret_cast<const void*>(fn), kFewSmem) != EP_OK) return EP_ERR_CUDA;
  const int grid = ep_host::grid_cap(1);
  Params p = in;
  p.wave = grid;
  if (ep_host::launch_in_budget<Params>(fn, grid * waves, threads, kFewSmem, s, p) != EP_OK) return EP_ERR_CUDA;
  ep_host::count_launch();
  return ep_host::check_launch();
}

int launch_few_bf16(const FewCall& in, const FewCall& out, const void* w_gu, const void* w_down, int act, cudaStream_t s);

}  // namespace ep
