// few.cu -- a whole mixture-of-experts layer for a few tokens, in two kernels.
//
//   k_few<.., kIn>    h = act(Wg x) * (Wu x)   for every slot (a token and one of its experts)
//   k_few<.., kOut>   out = sum over a token's slots of weight * (W_down h)
//
// Both are bound by reading each used expert's weights once.  The first deals
// out (expert, h column) pairs evenly over the CTAs, the second output columns, so
// that every CTA sums its own columns over all experts in a fixed order and
// nothing is added up between CTAs.  A CTA walks its columns in units: 32 columns'
// rows of gate and up, or 64 rows of W_down, whole in the inner index, for the
// tokens of one expert.  The weights' rows are the first operand of tcgen05.mma (64
// of them, those past the unit's being whatever lies there), the tokens
// the second, 16 or 32 of them, so that a product costs what reading its 2 KB of
// weights from shared memory does, a fifth of the time in which they arrive, and no thread
// touches a weight.  (By mma.sync E4M3 weights had to be turned into fp16 first, which bounded the
// kernels at 3.5 to 4.5 TB/s.)  Warps:
//   4 bring the sums out of tensor memory and finish a unit
//   1 issues the products
//   2 copy weights (TMA, 8 rows x 512 bytes a copy), 3 tokens' rows
//   6 put the tokens where the products read them, in three teams, a stage each
// The second kernel comes up as the first one's CTAs leave and fills its ring with
// weights before it waits for h.

#include "expert.cuh"
#include "umma.cuh"

namespace ep {

constexpr int kEpilogues = 4, kWeightWarps = 2, kRowWarps = 3;   // a warp issues a copy in some 80 clocks
constexpr int kTeams = 3, kTeam = 2, kTurners = kTeams * kTeam;   // a stage is one team's: its latency is 500 clocks and more
constexpr int kFewThreads = (kEpilogues + 1 + kRowWarps + kWeightWarps + kTurners) * kWarp;
constexpr int kUnitRows = 64;         // of weights
constexpr int kBlocks = 4;            // 128-byte blocks of a row in a stage
constexpr int kGroupBytes = kBlocks * 1024;   // 8 rows of a stage
constexpr int kWeightBytes = kUnitRows / 8 * kGroupBytes;
constexpr int kSums = 4;              // sums on their way out of tensor memory
constexpr int kScaleRing = 16;        // stages whose tokens' scales are kept: more than are between the copies and the epilogue
constexpr int kCrossing = 16;         // columns: what a narrow unit at an expert's end costs by its products (evenly: 49 us instead of KX)
constexpr int64_t kWaveWork = 1 << 23;
constexpr int kMaxFewStages = 8;
constexpr int kFewSmem = 226 * 1024;
__host__ __device__ constexpr int pass_of(bool fp8) { return fp8 ? 16 : 32; }   // tokens of an expert taken at a time

struct FewParams {
  CUtensorMap whole, tail;     // weights [2 E or E][N][K]: 8 rows of 4 blocks of 128 bytes; of one block, which K may cut
  const uint8_t* scales;
  const __nv_bfloat16* v;      // kIn: x [T, H]; kOut: h [T k, I]
  const int64_t* idx;          // [T, k]
  const float* weights;
  __nv_bfloat16* out;          // kIn: h; kOut: out [T, H]
  int32_t* status;
  int T, k, E, K, N;           // K: inner extent; N: columns of h or out
  uint32_t wave;               // CTAs that run at once
};

struct FewShared {
  uint64_t full[kMaxFewStages], turned[kMaxFewStages], empty[kMaxFewStages];
  uint64_t sums_full[kSums], sums_empty[kSums];
  int group_slots[kMaxE / kWarp], group_used[kMaxE / kWarp], group_most[kMaxE / kWarp];   // of 32 experts
  int n_used, most;                    // used experts; slots of the largest
  uint32_t tmem;
  alignas(16) float scales[kScaleRing][kBlocks][pass_of(true)];   // E4M3: what a token's block was divided by
  float up[2][pass_of(false)][kUnitRows / 2];         // kIn: on its way to its gate
};

// What every CTA works out first: the used experts in rising order, and their
// slots in rising order.
struct FewUsed {
  int16_t expert, first, count, pad;   // slots first .. first + count of the lists
};
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
__device__ __forceinline__ void few_lists(const FewParams& p, FewShared& sh, const FewLists& l, uint32_t* masks, bool report) {
  const int n = p.T * p.k, words = (n + 31) / 32, groups = (p.E + 31) / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (n <= kWarp) {   // one warp by itself, a slot a lane: places by counting the slots before (2.3 us the other way)
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
  for (int i = threadIdx.x; i < p.E * words; i += kFewThreads) masks[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kFewThreads) {
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
  for (int q = warp; q < groups; q += kFewThreads / kWarp) {
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
  for (int q = warp; q < groups; q += kFewThreads / kWarp) {
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
  for (int i = threadIdx.x; i < n; i += kFewThreads) {
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
template <bool kIn, int kPass>
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
    // of kIn's CTAs that come after the first wave, each takes an eighth of a first one's columns
    const uint32_t first = min(gridDim.x, wave), parts = 8 * first + (gridDim.x - first);
    const uint32_t b = blockIdx.x < first ? 8 * blockIdx.x : 7 * first + blockIdx.x, size = blockIdx.x < first ? 8 : 1;
    const uint32_t at = (uint32_t)((uint64_t)all * b / parts);
    left = (int)((uint32_t)((uint64_t)all * (b + size) / parts) - at);
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

// ---------------------------------------------------------------- products

__device__ __forceinline__ void umma_few(bool fp8, uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool add) {
  constexpr uint32_t kWeightsHi = ((uint32_t)kGroupBytes >> 4) | (1u << 14) | (2u << 29);   // 8-row groups 4 KB apart
  if (fp8)
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n"
        " mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %6};\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n}\n" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"((uint32_t)add), "r"(kWeightsHi), "r"(kDescHi)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n"
        " mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %6};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"((uint32_t)add), "r"(kWeightsHi), "r"(kDescHi)
        : "memory");
}
// Instruction descriptor: 64 rows, n tokens; E4M3 or bf16 operands, fp32 sums.  Rows
// 16 w .. 16 w + 15 come out in the first 16 lanes of quarter w of the tensor memory.
__device__ __forceinline__ uint32_t umma_few_idesc(bool fp8, int n) {
  return (1u << 4) | (fp8 ? 0u : (1u << 7) | (1u << 10)) | ((uint32_t)(n >> 3) << 17) | (4u << 24);
}

// A token's bf16 numbers as two E4M3 ones, for E4M3 weights: in a block of 128
// inner elements whose largest is in [2^e, 2^(e+1)), x = 2^(e-7) (hi + lo / 16) with
// hi = E4M3(x 2^(7-e)) and lo = E4M3 of what that leaves, times 16: columns 2 j and
// 2 j + 1 of the products.  bf16 has 8 significant bits and each part 4, so this is x
// itself down to 2^-13 of the largest, and 2^-21 of the largest off below: no more
// than sums in 32 bits lose.  A block with an infinity or NaN gets the scale NaN.
// 8 elements a lane, a block sixteen lanes.
__device__ __forceinline__ void split_e4m3(uint4 v, uint32_t (&hi)[2], uint32_t (&lo)[2], float& scale) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t a = w[0] & 0x7fff7fffu, b = w[1] & 0x7fff7fffu;
  asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(w[2] & 0x7fff7fffu));
  asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(b) : "r"(w[3] & 0x7fff7fffu));
  asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
  uint32_t top = max(a >> 16, a & 0xffffu);
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const uint32_t e = top >> 7;   // biased; up = 2^(134 - e), no more than 2^127
  const float up = __uint_as_float((e <= 7 ? 254u : 261u - min(e, 254u)) << 23);
  scale = e == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(e <= 7 ? 0x00400000u : (e - 7) << 23);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h[2], r[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float x = bf16_lo(w[2 * i + q]) * up, y = bf16_hi(w[2 * i + q]) * up;
      h[q] = cvt_e4m3x2(x, y);
      uint32_t back;
      asm("{\n .reg .b16 t;\n cvt.u16.u32 t, %1;\n cvt.rn.f16x2.e4m3x2 %0, t;\n}" : "=r"(back) : "r"(h[q]));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&back));
      r[q] = cvt_e4m3x2((x - f.x) * 16.0f, (y - f.y) * 16.0f);
    }
    hi[i] = __byte_perm(h[0], h[1], 0x5410);
    lo[i] = __byte_perm(r[0], r[1], 0x5410);
  }
}

__device__ __forceinline__ float ue8m0_value(uint32_t b) {
  return b == 255 ? __uint_as_float(0x7fc00000u) : b == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23);
}

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

// kColumns columns of kCount blocks' sums, all on their way before the first is waited for.
template <int kColumns, int kCount>
__device__ __forceinline__ void few_columns(uint32_t at, int columns, float (&v)[kCount][kColumns]) {
#pragma unroll
  for (int b = 0; b < kCount; ++b)
#pragma unroll
    for (int i = 0; i < kColumns; i += 8) tmem_ld8(at + b * columns + i, &v[b][i]);
#pragma unroll
  for (int b = 0; b < kCount; ++b) tmem_wait_ld(v[b]);
}

// The sums of a unit's rows for the tokens of kColumns columns: y[j] of token j, a
// row a thread; ok: no wait has run out.
template <bool kFp8, int kColumns>
__device__ __forceinline__ void few_sums(FewShared& sh, uint32_t tmem, int columns, int chunks, int K, const uint8_t* scale, RingPosition& sums,
                                         uint32_t& stage, float (&y)[pass_of(false)], bool& ok) {
  if constexpr (kFp8) {
    constexpr int kTokens = kColumns / 2, kCount = kColumns == 32 ? 2 : kBlocks;
    const int blocks = K / kFp8Block;
    uint32_t next[kBlocks];
    auto fetch = [&](int c) {
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) next[b] = c * kBlocks + b < blocks ? __ldg(scale + c * kBlocks + b) : 0u;
    };
    fetch(0);
#pragma unroll
    for (int j = 0; j < kTokens; ++j) y[j] = 0.0f;
    for (int c = 0; c < chunks; ++c) {
      float f[kBlocks];
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) f[b] = ue8m0_value(next[b]);
      fetch(c + 1);
      if (ok) ok = wait_few(&sh.sums_full[sums.s], sums.phase, 4 * kWaitNs);
      tmem_fence_after();
      const uint32_t at = tmem + sums.s * kBlocks * columns;
#pragma unroll
      for (int b0 = 0; b0 < kBlocks; b0 += kCount) {
        float v[kCount][kColumns];
        few_columns(at + b0 * columns, columns, v);
#pragma unroll
        for (int b = 0; b < kCount; ++b) {
          if (c * kBlocks + b0 + b < blocks) {
            const float4* const token = reinterpret_cast<const float4*>(sh.scales[stage % kScaleRing][b0 + b]);
#pragma unroll
            for (int i = 0; i < kTokens / 4; ++i) {
              const float4 t = token[i];
              const float of[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int j = 4 * i + q;
                y[j] = fmaf(fmaf(v[b][2 * j + 1], 0.0625f, v[b][2 * j]) * of[q], f[b0 + b], y[j]);
              }
            }
          }
        }
      }
      tmem_fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.sums_empty[sums.s]);
      sums.advance();
      ++stage;
    }
  } else {
    if (ok) ok = wait_few(&sh.sums_full[sums.s], sums.phase, 4 * kWaitNs);
    tmem_fence_after();
    float v[1][kColumns];
    few_columns(tmem + sums.s * columns, columns, v);
#pragma unroll
    for (int j = 0; j < kColumns; ++j) y[j] = v[0][j];
    tmem_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.sums_empty[sums.s]);
    sums.advance();
  }
}

template <bool kFp8, bool kIn, int kAct>
__global__ void __launch_bounds__(kFewThreads, 1) k_few(const __grid_constant__ FewParams p) {
  constexpr int kOne = kFp8 ? 1 : 2;                 // bytes of a weight
  constexpr int kBlock = 128 / kOne, kChunk = kBlocks * kBlock;   // inner elements of a block, of a stage
  constexpr int kPass = pass_of(kFp8), kColumns = kFp8 ? 2 : 1;   // of the products for a token
  constexpr int kRawBytes = kChunk * 2;              // a token's row in a stage, as it comes
  extern __shared__ __align__(1024) uint8_t raw[];
  FewShared& sh = *reinterpret_cast<FewShared*>(raw);
  uint8_t* const ring = raw + (sizeof(FewShared) + 1023) / 1024 * 1024;
  uint8_t* const lists_at = raw + kFewSmem - FewLists::bytes(p.E, p.T, p.k);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxFewStages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.turned[s], kTeam);
      mbar_init(&sh.empty[s], 1);
    }
    for (int b = 0; b < kSums; ++b) {
      mbar_init(&sh.sums_full[b], 1);
      mbar_init(&sh.sums_empty[b], kEpilogues);
    }
    fence_barrier_init();
  }
  if (warp == kEpilogues) tmem_alloc<1>(&sh.tmem, 512);
  if (kIn) {
    pdl_wait();   // ids and tokens may come from the kernel before
    pdl_launch_dependents();
  }
  const FewLists l(lists_at, p.E, p.T, p.k);
  tmem_fence_before();
  few_lists(p, sh, l, reinterpret_cast<uint32_t*>(ring), kIn && blockIdx.x == 0);
  tmem_fence_after();
  const uint32_t tmem = sh.tmem;
  const int tokens_most = min(sh.most, kPass);
  const int columns = (tokens_most * kColumns + 7) / 8 * 8;   // of products, most
  const int chunks = (p.K + kChunk - 1) / kChunk;
  FewWalk<kIn, kPass> w(l.used, sh.n_used, p.N, p.wave);
  // a stage: weights, tokens for the products, tokens as they came.  Products read 64
  // rows; what W_down's units have no rows for is other stages' memory, or the lists'.
  const int weight_bytes = kIn ? kWeightBytes : (w.most + 7) / 8 * kGroupBytes;
  const int token_block = columns * 128, stage_bytes = (weight_bytes + kBlocks * token_block + tokens_most * kRawBytes + 1023) / 1024 * 1024;
  const int stages = max(1, min(kMaxFewStages, min((int)(lists_at - ring) / stage_bytes, ((int)(raw + kFewSmem - ring) - kWeightBytes) / stage_bytes + 1)));
  RingPosition at(stages);
  bool ok = true;

  if (warp < kEpilogues) {
    // ---------------------------------------------------------------- sums: a row a thread
    RingPosition sums(kSums);
    uint32_t stage = 0, unit = 0;
    const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
    const int row = warp * 16 + (lane & 15), column = kIn ? row % (kUnitRows / 2) : row;   // kIn: gate in two warps, up in the others
    const bool there = lane < 16;
    if (!kIn && there)
      for (int n = 0; n < p.T; ++n) l.sums[n * kUnitRows + row] = 0.0f;
    while (w.next()) {
      const uint8_t* scale = nullptr;
      if (kFp8) {
        const int n = min(w.col + column, p.N - 1);
        scale = p.scales + ((int64_t)(kIn ? w.e * 2 + (warp >> 1) : w.e) * (p.N / kFp8Block) + n / kFp8Block) * (p.K / kFp8Block);
      }
      float y[pass_of(false)];
      if (w.m * kColumns > 16)
        few_sums<kFp8, 32>(sh, lanes, columns, chunks, p.K, scale, sums, stage, y, ok);
      else if (w.m * kColumns > 8)
        few_sums<kFp8, 16>(sh, lanes, columns, chunks, p.K, scale, sums, stage, y, ok);
      else
        few_sums<kFp8, 8>(sh, lanes, columns, chunks, p.K, scale, sums, stage, y, ok);
      if (kIn) {
        float(&up)[pass_of(false)][kUnitRows / 2] = sh.up[unit & 1];
        if (warp >= kEpilogues / 2 && there) {
#pragma unroll
          for (int j = 0; j < kPass; ++j) {
            if (j >= w.m) break;
            up[j][column] = y[j];
          }
        }
        named_barrier_sync(1, kEpilogues * kWarp);
        if (warp < kEpilogues / 2 && there && column < w.cols) {
#pragma unroll
          for (int j = 0; j < kPass; ++j) {   // rounded to bf16: the second kernel's operand
            if (j >= w.m) break;
            p.out[(int64_t)l.slot[w.s0 + j] * p.N + w.col + column] = __float2bfloat16_rn(act_value<kAct>(y[j]) * up[j][column]);
          }
        }
      } else if (there) {
#pragma unroll
        for (int j = 0; j < kPass; ++j) {
          if (j >= w.m) break;
          float* const sum = l.sums + l.token[w.s0 + j] * kUnitRows + row;
          *sum = fmaf(l.weight[w.s0 + j], y[j], *sum);
        }
        if (w.last) {
          for (int n = 0; n < p.T; ++n) {
            if (row < w.cols) p.out[(int64_t)n * p.N + w.col + row] = __float2bfloat16_rn(l.sums[n * kUnitRows + row]);
            l.sums[n * kUnitRows + row] = 0.0f;
          }
        }
      }
      ++unit;
    }
    if (!kIn && sh.n_used == 0) {
      pdl_wait();   // out may be x
      for (int64_t i = (int64_t)blockIdx.x * (kEpilogues * kWarp) + threadIdx.x; i < (int64_t)p.T * p.N; i += (int64_t)gridDim.x * (kEpilogues * kWarp))
        p.out[i] = __float2bfloat16_rn(0.0f);
    }
  } else if (warp == kEpilogues) {
    // ---------------------------------------------------------------- products
    // one thread by itself: votes and the warp's steps cost as much as the products they stand between
    if (elect_one()) {
      const uint32_t weights0 = umma_desc_lo(smem_addr(ring), 16), tokens0 = umma_desc_lo(smem_addr(ring) + weight_bytes, 16);
      RingPosition sums(kSums);
      while (ok && w.next()) {
        const uint32_t idesc = umma_few_idesc(kFp8, (w.m * kColumns + 7) / 8 * 8);
        for (int c = 0; c < chunks; ++c) {
          if (kFp8 || c == 0) ok = wait_alone(&sh.sums_empty[sums.s], sums.phase ^ 1, 4 * kWaitNs);
          ok = ok && wait_alone(&sh.turned[at.s], at.phase);   // by who has seen the weights' copies
          if (!ok) break;
          tmem_fence_after();
          const int blocks = (p.K - c * kChunk + kBlock - 1) / kBlock;
          const uint32_t a = weights0 + (uint32_t)at.s * (stage_bytes >> 4), b = tokens0 + (uint32_t)at.s * (stage_bytes >> 4);
          const uint32_t d = tmem + sums.s * (columns * (kFp8 ? kBlocks : 1));
#pragma unroll
          for (int i = 0; i < kBlocks; ++i) {
            if (i < blocks) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                umma_few(kFp8, kFp8 ? d + i * columns : d, a + (i * 64 + q * 2), b + i * (token_block >> 4) + q * 2, idesc, q > 0 || (!kFp8 && (i > 0 || c > 0)));
            }
          }
          umma_commit(&sh.empty[at.s]);
          at.advance();
          if (kFp8 || c + 1 == chunks) {
            umma_commit(&sh.sums_full[sums.s]);
            sums.advance();
          }
        }
      }
    }
    ok = __all_sync(0xffffffffu, ok);
  } else if (warp < kEpilogues + 1 + kRowWarps) {
    // ---------------------------------------------------------------- tokens, a row a lane
    const int mine = lane * kRowWarps + warp - (kEpilogues + 1);
    if (!kIn) pdl_wait();
    while (ok && w.next()) {
      const int from = mine < w.m ? (kIn ? l.token[w.s0 + mine] : l.slot[w.s0 + mine]) : -1;
      const __nv_bfloat16* row = p.v + (int64_t)from * p.K;
      for (int c = 0; c < chunks; ++c) {
        ok = wait_few(&sh.empty[at.s], at.phase ^ 1);
        if (!ok) break;
        if (from >= 0)
          tma_load_1d(ring + at.s * stage_bytes + weight_bytes + kBlocks * token_block + mine * kRawBytes, row + c * kChunk,
                      min(kChunk, p.K - c * kChunk) * 2, &sh.full[at.s]);
        __syncwarp();
        at.advance();
      }
    }
  } else if (warp < kEpilogues + 1 + kRowWarps + kWeightWarps) {
    // ---------------------------------------------------------------- weights: groups of 8 rows in turn
    // kOut: those of the first stages before h is there
    const int turn = warp - (kEpilogues + 1 + kRowWarps);
    const bool issue = elect_one();
    while (ok && w.next()) {
      const int groups = (w.cols + 7) / 8;   // of W_down, or of gate and of up each
      for (int c = 0; c < chunks; ++c) {
        ok = wait_few(&sh.empty[at.s], at.phase ^ 1);
        if (!ok) break;
        if (issue) {
          const int k = min(kChunk, p.K - c * kChunk);
          const bool cut = k % kBlock != 0;   // K ends inside a block: block by block
          const int blocks = cut ? (k + kBlock - 1) / kBlock : kBlocks;
          if (turn == 0) mbar_arrive_expect_tx(&sh.full[at.s], (kIn ? 2 : 1) * groups * blocks * 1024 + w.m * k * 2);
          const uint32_t to = smem_addr(ring + at.s * stage_bytes), bar = smem_addr(&sh.full[at.s]);
          for (int half = 0; half < (kIn ? 2 : 1); ++half) {
            const int z = kIn ? 2 * w.e + half : w.e;
            for (int g = turn; g < groups; g += kWeightWarps) {
              const uint32_t group = to + (half * (kUnitRows / 16) + g) * kGroupBytes;
              if (!cut)
                tma_load_4d(group, &p.whole, bar, 0, w.col + g * 8, c * kBlocks, z);
              else
                for (int i = 0; i < blocks; ++i) tma_load_3d<false>(group + i * 1024, &p.tail, bar, c * kChunk + i * kBlock, w.col + g * 8, z);
            }
          }
        }
        __syncwarp();
        at.advance();
      }
    }
  } else {
    // ---------------------------------------------------------------- tokens to where the products read them
    const int turn = warp - (kEpilogues + 1 + kRowWarps + kWeightWarps), team = turn / kTeam, member = turn % kTeam;
    uint32_t stage = 0;
    while (w.next()) {
      for (int c = 0; c < chunks; ++c, ++stage, at.advance()) {
        // every stage is waited for, another team's too: they may land out of order, and a wait two phases ahead passes
        if (ok) ok = wait_few(&sh.full[at.s], at.phase);
        if (stage % kTeams != (uint32_t)team) continue;
        const uint32_t to = smem_addr(ring + at.s * stage_bytes + weight_bytes), from = to + kBlocks * token_block;
        const int left = p.K - c * kChunk;
        if constexpr (kFp8) {
          for (int i = member; i < 2 * w.m; i += kTeam) {   // two blocks of a token
            const int j = i >> 1, b = (i & 1) * 2 + (lane >> 4), piece = lane & 15;
            const bool in = b * kBlock < left;
            uint32_t hi[2], lo[2];
            float scale;
            split_e4m3(in ? ld_shared_v4_at(from + j * kRawBytes + (b * kBlock + piece * 8) * 2) : make_uint4(0, 0, 0, 0), hi, lo, scale);
            if (in) {
              const uint32_t row = to + b * token_block + 2 * j * 128, at_hi = row + ((((piece >> 1) ^ (2 * j & 7)) << 4) | ((piece & 1) << 3));
              const uint32_t at_lo = row + 128 + ((((piece >> 1) ^ ((2 * j + 1) & 7)) << 4) | ((piece & 1) << 3));
              asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at_hi), "r"(hi[0]), "r"(hi[1]) : "memory");
              asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at_lo), "r"(lo[0]), "r"(lo[1]) : "memory");
              if (piece == 0) sh.scales[stage % kScaleRing][b][j] = scale;
            }
          }
        } else {
          for (int j = member; j < w.m; j += kTeam) {   // zeros behind the row's end, as the weights have them
            const uint4 v = lane * 8 < left ? ld_shared_v4_at(from + j * kRawBytes + lane * 16) : make_uint4(0, 0, 0, 0);
            st_shared_v4_at(to + (lane >> 3) * token_block + j * 128 + (((lane & 7) ^ (j & 7)) << 4), v);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.turned[at.s]);
      }
    }
  }
  if (!ok) {
    set_status(p.status, EP_ERR_TIMEOUT);
    const uint64_t t0 = globaltimer_ns();   // give the copies in flight time to land before the memory goes
    while (globaltimer_ns() - t0 < 2000000ull) {
    }
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == kEpilogues) tmem_free<1>(tmem, 512);
}

template <bool kFp8, bool kIn, int kAct>
static int launch_few_half(const FewParams& in, cudaStream_t s) {
  auto* fn = k_few<kFp8, kIn, kAct>;
  if (ep_host::ensure_max_smem(reinterpret_cast<const void*>(fn), kFewSmem) != EP_OK) return EP_ERR_CUDA;
  int grid = ep_host::grid_cap(1);
  FewParams p = in;
  p.wave = grid;
  if (kIn && !ep_host::sm_budget_set() && (int64_t)p.T * p.k * p.N * p.K >= kWaveWork * grid) grid *= 1 + 2;
  if (!kIn && ep_host::sm_budget_set()) {   // the second kernel's CTAs do not come up beside the first's
    fn<<<grid, kFewThreads, kFewSmem, s>>>(p);
  } else if (ep_host::launch_dependent<FewParams>(fn, grid, kFewThreads, kFewSmem, s, p) != EP_OK) {
    return EP_ERR_CUDA;
  }
  ep_host::count_launch();
  return ep_host::check_launch();
}

template <bool kFp8>
static int launch_few(const FewParams& in, const FewParams& out, int act, cudaStream_t s) {
  const int rc = act == EP_ACT_RELU   ? launch_few_half<kFp8, true, EP_ACT_RELU>(in, s)
                 : act == EP_ACT_SILU ? launch_few_half<kFp8, true, EP_ACT_SILU>(in, s)
                                      : launch_few_half<kFp8, true, EP_ACT_GELU>(in, s);
  return rc != EP_OK ? rc : launch_few_half<kFp8, false, EP_ACT_NONE>(out, s);
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
  p.scales = w_gu_scales;
  p.v = static_cast<const __nv_bfloat16*>(x);
  p.idx = topk_idx;
  p.weights = topk_weights;
  p.out = static_cast<__nv_bfloat16*>(workspace);
  p.status = status;
  p.T = R * T_r;
  p.k = k;
  p.E = E;
  p.K = H;
  p.N = I;
  FewParams q = p;
  q.scales = w_down_scales;
  q.v = p.out;
  q.out = static_cast<__nv_bfloat16*>(out);
  q.K = I;
  q.N = H;
  auto maps = [&](FewParams& f, const void* w, uint64_t count) {
    const uint64_t one = fp8 ? 1 : 2, block = 128 / one, row = f.K * one, N = f.N, K = f.K;
    const uint64_t dims[4] = {block, N, std::max<uint64_t>(1, K / block), count}, strides[3] = {row, 128, N * row};
    const uint32_t box[4] = {(uint32_t)block, 8, kBlocks, 1};
    // (rows shorter than a block have none that is whole: that map is not used)
    int rc = K >= block ? ep_host::make_map(&f.whole, fp8, 4, w, dims, strides, box) : EP_OK;
    const uint64_t dims3[3] = {K, N, count}, strides3[2] = {row, N * row};
    const uint32_t box3[3] = {(uint32_t)block, 8, 1};
    if (rc == EP_OK) rc = ep_host::make_map(&f.tail, fp8, 3, w, dims3, strides3, box3);
    return rc;
  };
  if (maps(p, w_gu, 2 * E) != EP_OK || maps(q, w_down, E) != EP_OK) return EP_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return fp8 ? launch_few<true>(p, q, act, s) : launch_few<false>(p, q, act, s);
}
