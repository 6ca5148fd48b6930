// few.cu -- a whole mixture-of-experts layer for a few tokens, in two kernels.
//
//   k_few<.., kIn>    h = act(Wg x) * (Wu x)   for every slot (a token and one of its experts)
//   k_few<.., kOut>   out = sum over a token's slots of weight * (W_down h)
//
// Both are bound by reading each used expert's weights once.  The first deals
// out (expert, h column) pairs evenly over the CTAs, the second output columns, so
// that every CTA sums its own columns over all experts in a fixed order and
// nothing is added up between CTAs.  A CTA walks its columns in units: 16 columns'
// rows of gate and up, or 32 rows of W_down, whole in the inner index, for up to 32
// tokens of the expert.  One warp copies 1 KB pieces of those rows and of the
// tokens' rows into a ring of stages (cp.async.bulk); the others take the inner
// index of a stage apart between them, multiply on the tensor cores with the
// weights' rows as the first operand and 8 tokens as the second (m16n8k16, at
// a few tokens an expert the widest form that is not mostly padding: tcgen05
// wants 64 rows or more in tiles of their own, and an SM gets 13 to 110 columns),
// and add their sums up in shared memory once a unit.
//
// The second kernel comes up as the first one's CTAs leave and fills its ring with
// weights before it waits for h.

#include "expert.cuh"
#include "umma.cuh"

namespace ep {

constexpr int kSplit = 8;                           // parts of a stage's inner index
constexpr int kConsumers = 2 * kSplit;              // warps that multiply: 16 of a unit's 32 rows each
constexpr int kTokenWarps = 3;                      // warps that copy tokens' rows
constexpr int kFewThreads = (kConsumers + 1 + kTokenWarps) * kWarp;
constexpr int kPiece = 1024;                        // bytes of a weight row in a stage
constexpr int kUnitRows = 32;
constexpr int kRedPitch = 36;                       // floats: a quarter-warp's sums fall into distinct banks
constexpr int kMaxSlots = EP_MOE_FEW_TOKENS * kMaxK;
constexpr int kMaxFewStages = 8;
constexpr int kFewSmem = 226 * 1024;
__host__ __device__ constexpr int pass_of(bool fp8) { return fp8 ? 16 : 24; }   // tokens of an expert taken at a time: two stages at least

struct FewParams {
  CUtensorMap whole, four, one;   // weights [2 E or E][N][K]: boxes of 1 KB of a unit's rows (kIn: of gate or up), 4 and 1
  const uint8_t* scales;
  const __nv_bfloat16* v;      // kIn: x [T, H]; kOut: h [T k, I]
  const int64_t* idx;          // [T, k]
  const float* weights;
  __nv_bfloat16* out;          // kIn: h; kOut: out [T, H]
  int32_t* status;
  int T, k, E, K, N;           // K: inner extent; N: columns of h or out
};

// What every CTA works out first: the used experts in rising order, and their
// slots in rising order.
struct FewLists {
  int16_t slot[kMaxSlots];
  int16_t id[kMaxSlots];        // expert of a slot, -1: unused
  int16_t rank[kMaxSlots];      // among its expert's slots
  int16_t token[kMaxSlots];     // of slot[i]
  int16_t expert[kMaxE];
  int16_t first[kMaxE + 1];     // of the used expert's slots in `slot`
  int count[kMaxE];
  int used, most;               // used experts; slots of the largest
};

struct FewShared {
  uint64_t full[kMaxFewStages], empty[kMaxFewStages];
  FewLists lists;
  float sums[EP_MOE_FEW_TOKENS * kUnitRows];   // kOut: the columns in hand, [token][column]
};

__device__ __forceinline__ void few_lists(const FewParams& p, FewLists& l, bool report) {
  const int n = p.T * p.k, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < p.E; e += kFewThreads) l.count[e] = 0;
  for (int i = threadIdx.x; i < n; i += kFewThreads) {
    const int64_t e = p.idx[i];
    const bool fits = e >= 0 && e < p.E;
    if (report && !fits && e != -1) set_status(p.status, EP_ERR_INVALID_ARG);
    l.id[i] = fits ? (int16_t)e : (int16_t)-1;
  }
  __syncthreads();
  if (threadIdx.x < kWarp) {
    for (int i0 = 0; i0 < n; i0 += kWarp) {   // 32 slots at a time: their places among the expert's
      const int e = i0 + lane < n ? l.id[i0 + lane] : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, e);
      const int before = e >= 0 ? l.count[e] : 0, at = __popc(same & lanemask_lt());
      __syncwarp();
      if (e >= 0) {
        l.rank[i0 + lane] = (int16_t)(before + at);
        if (at == 0) l.count[e] = before + __popc(same);
      }
      __syncwarp();
    }
    int used = 0, first = 0, most = 0;
    for (int e0 = 0; e0 < p.E; e0 += kWarp) {
      const int c = e0 + lane < p.E ? l.count[e0 + lane] : 0;
      const uint32_t some = __ballot_sync(0xffffffffu, c > 0);
      if (some == 0) continue;
      int upto = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      if (c > 0) {
        const int d = used + __popc(some & lanemask_lt());
        l.expert[d] = (int16_t)(e0 + lane);
        l.first[d] = (int16_t)(first + upto - c);
        l.count[e0 + lane] = first + upto - c;   // from here on: where the expert's slots start
      }
      used += __popc(some);
      first += __shfl_sync(0xffffffffu, upto, 31);
      most = max(most, __reduce_max_sync(0xffffffffu, c));
    }
    if (lane == 0) {
      l.first[used] = (int16_t)first;
      l.used = used;
      l.most = most;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kFewThreads)
    if (l.id[i] >= 0) {
      const int at = l.count[l.id[i]] + l.rank[i];
      l.slot[at] = (int16_t)i;
      l.token[at] = (int16_t)(i / p.k);
    }
  __syncthreads();
}

// A CTA's units, one after another: `cols` columns from `col` on of used expert d,
// for the tokens s0 .. s0 + m of the lists.
template <bool kIn, int kPass>
struct FewWalk {
  const FewLists* l;
  int N, at, end;        // kIn: (expert, column) pairs; kOut: columns
  int d, col, cols, s0, m;
  bool last;             // kOut: of these columns

  __device__ __forceinline__ FewWalk(const FewLists& lists, int n) {
    l = &lists;
    N = n;
    const int64_t all = kIn ? (int64_t)lists.used * n : n;
    at = (int)(all * blockIdx.x / gridDim.x);
    end = (int)(all * (blockIdx.x + 1) / gridDim.x);
    d = -1;
    cols = s0 = m = 0;
  }
  __device__ __forceinline__ bool next() {
    if (d >= 0 && s0 + m < l->first[d + 1]) {   // more tokens of the expert
      s0 += m;
    } else {
      if (kIn) {
        at += cols;
        if (at >= end) return false;
        d = at / N;
        col = at - d * N;
        cols = min(min(kUnitRows / 2, N - col), end - at);
      } else {
        if (d < 0 || d + 1 == l->used) {
          if (d >= 0) at += cols;
          if (at >= end || l->used == 0) return false;
          d = 0;
          col = at;
          cols = min(kUnitRows, end - at);
        } else {
          ++d;
        }
      }
      s0 = l->first[d];
    }
    m = min(kPass, l->first[d + 1] - s0);
    last = d + 1 == l->used && s0 + m == l->first[d + 1];
    return true;
  }
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// E4M3 bytes 0 and 2 (1 and 3) of a word as bf16: the byte's exponent and fraction
// fields set lowest in bf16's give 2^-120 of the value, subnormals too; one exact
// product brings them up.  (The NaN code would read as 480: found apart.)
__device__ __forceinline__ uint32_t times_2_120(uint32_t v) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x7b807b80u));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_even(uint32_t w) { return times_2_120(((w << 4) & 0x07f007f0u) | ((w << 8) & 0x80008000u)); }
__device__ __forceinline__ uint32_t e4m3_odd(uint32_t w) { return times_2_120(((w >> 4) & 0x07f007f0u) | (w & 0x80008000u)); }
// High bits set in the bytes that are NaN.
__device__ __forceinline__ uint32_t e4m3_nan(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

__device__ __forceinline__ float ue8m0_value(uint32_t b) {
  return b == 255 ? __uint_as_float(0x7fc00000u) : b == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23);
}

template <bool kFp8, bool kIn, int kAct>
__global__ void __launch_bounds__(kFewThreads, 1) k_few(const __grid_constant__ FewParams p) {
  constexpr int kOne = kFp8 ? 1 : 2;                 // bytes of a weight
  constexpr int kChunk = kPiece / kOne;              // inner elements of a stage
  constexpr int kTokenPitch = kFp8 ? 2 * kPiece + 16 : kPiece + 64;   // 8 lanes' 16 bytes fall into distinct banks
  constexpr int kPass = pass_of(kFp8), kGroups = kPass / 8;
  constexpr int kStep = kFp8 ? 64 : 32;              // inner elements a warp multiplies at a time: 16 bytes of weights a lane
  extern __shared__ __align__(1024) uint8_t raw[];
  FewShared& sh = *reinterpret_cast<FewShared*>(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxFewStages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], kConsumers);
    }
    fence_barrier_init();
  }
  if (kIn) {
    pdl_wait();   // ids and tokens may come from the kernel before
    pdl_launch_dependents();
  }
  few_lists(p, sh.lists, kIn && blockIdx.x == 0);
  const FewLists& l = sh.lists;
  const int groups_most = (min(l.most, kPass) + 7) / 8;
  const int red_bytes = kSplit * groups_most * 8 * kRedPitch * 4;   // of one unit; the next one's go to a second part
  const int stage_bytes = kUnitRows * kPiece + groups_most * 8 * kTokenPitch;
  uint8_t* const red_base = raw + (sizeof(FewShared) + 127) / 128 * 128;
  uint8_t* const ring = red_base + 2 * red_bytes;
  const int stages = min(kMaxFewStages, (int)((kFewSmem - (int)(ring - raw)) / stage_bytes));
  const int chunks = (p.K + kChunk - 1) / kChunk;
  FewWalk<kIn, kPass> w(l, p.N);
  bool ok = true;
  int s = 0;
  uint32_t phase = 0;

  if (warp >= kConsumers) {
    // ---------------------------------------------------------------- copies
    // one warp the weights, a unit's rows in two copies (kIn) or one: by rows of 1 KB a warp got through 2.4 TB/s; the
    // others tokens' rows, one a lane.  kOut: the weights of the first stages before h is there.
    const bool weights = warp == kConsumers;
    if (!kIn && !weights) pdl_wait();
    while (ok && w.next()) {
      const int e = l.expert[w.d], turn = warp - kConsumers - 1, mine = lane * kTokenWarps + turn;
      const int from = !weights && mine < w.m ? (kIn ? l.token[w.s0 + mine] : l.slot[w.s0 + mine]) : -1;
      const __nv_bfloat16* row = p.v + (int64_t)from * p.K;
      for (int c = 0; c < chunks; ++c) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.empty[s], phase ^ 1));
        if (!ok) break;
        uint8_t* stage = ring + s * stage_bytes;
        const int k = min(kChunk, p.K - c * kChunk);
        if (weights) {
          if (elect_one()) {
            mbar_arrive_expect_tx(&sh.full[s], (kIn ? 2 : 1) * w.cols * kPiece + w.m * k * 2);
            const uint32_t bar = smem_addr(&sh.full[s]);
            constexpr int kWhole = kIn ? kUnitRows / 2 : kUnitRows;
            for (int half = 0; half < (kIn ? 2 : 1); ++half) {
              const uint32_t to = smem_addr(stage) + half * kWhole * kPiece;
              const int z = kIn ? 2 * e + half : e;
              if (w.cols == kWhole) {
                tma_load_3d<false>(to, &p.whole, bar, c * (kPiece / 4), w.col, z);
              } else {
                int n = 0;
                for (; n + 4 <= w.cols; n += 4) tma_load_3d<false>(to + n * kPiece, &p.four, bar, c * (kPiece / 4), w.col + n, z);
                for (; n < w.cols; ++n) tma_load_3d<false>(to + n * kPiece, &p.one, bar, c * (kPiece / 4), w.col + n, z);
              }
            }
          }
        } else if (from >= 0) {
          tma_load_1d(stage + kUnitRows * kPiece + mine * kTokenPitch, row + c * kChunk, k * 2, &sh.full[s]);
        }
        __syncwarp();
        if (++s == stages) {
          s = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok) {   // give the copies in flight time to land before the memory goes
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 2000000ull) {
      }
    }
  } else {
    // ---------------------------------------------------------------- products
    // 16 rows (h: the lower or the upper ones) by a part (part) of a stage's inner index
    const int g = lane >> 2, t = lane & 3, part = warp % kSplit, h = warp / kSplit;
    float* red = reinterpret_cast<float*>(red_base);
    float* red_next = reinterpret_cast<float*>(red_base + red_bytes);
    const int red_part = groups_most * 8 * kRedPitch;
    // this lane's two rows in a stage: kIn gate and up of column 8 h + g; kOut 16 h + g, 16 h + g + 8
    const int row0 = kIn ? 8 * h + g : 16 * h + g, row1 = row0 + (kIn ? 16 : 8);
    if (!kIn)
      for (int i = threadIdx.x; i < p.T * kUnitRows; i += kConsumers * kWarp) sh.sums[i] = 0.0f;
    while (w.next()) {
      const int groups = (w.m + 7) / 8;
      const bool some = w.cols > (kIn ? 8 : 16) * h;   // of these rows
      float acc[kGroups][4] = {};
      const uint8_t *scale0 = nullptr, *scale1 = nullptr;
      uint32_t sc0 = 0, sc1 = 0;
      if (kFp8) {
        const int blocks_n = p.N / kFp8Block, blocks_k = p.K / kFp8Block;
        const int64_t e = l.expert[w.d];
        const int n0 = min(w.col + row0, p.N - 1), n1 = min(w.col + (kIn ? row0 : row1), p.N - 1);
        scale0 = p.scales + ((kIn ? e * 2 : e) * blocks_n + n0 / kFp8Block) * blocks_k;
        scale1 = p.scales + ((kIn ? e * 2 + 1 : e) * blocks_n + n1 / kFp8Block) * blocks_k;
        if (part < blocks_k) {
          sc0 = __ldg(scale0 + part);
          sc1 = __ldg(scale1 + part);
        }
      }
      for (int c = 0; c < chunks; ++c) {
        const int left = p.K - c * kChunk;   // inner elements from this stage on
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.full[s], phase));
        const uint32_t at = smem_addr(ring + s * stage_bytes);
        const uint32_t wa = at + t * 16, va = at + kUnitRows * kPiece + g * kTokenPitch + t * (kFp8 ? 32 : 16);
        if (kFp8) {
          if (some && part * kFp8Block < left) {   // a block of 128 inner elements, whose scale is one a row
            float sum[kGroups][4] = {};
            uint32_t nan0 = 0, nan1 = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int k0 = part * kFp8Block + i * kStep;
              const uint4 r0 = ld_shared_v4_at(wa + row0 * kPiece + k0), r1 = ld_shared_v4_at(wa + row1 * kPiece + k0);
              const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
              uint32_t b[kGroups][8];   // tokens' elements 0, 2 and 1, 3 of every four
#pragma unroll
              for (int j = 0; j < kGroups; ++j) {
                if (j < groups) {
                  const uint4 lo = ld_shared_v4_at(va + j * 8 * kTokenPitch + k0 * 2), hi = ld_shared_v4_at(va + j * 8 * kTokenPitch + k0 * 2 + 16);
                  const uint32_t x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                  for (int f = 0; f < 4; ++f) {
                    b[j][2 * f] = __byte_perm(x[2 * f], x[2 * f + 1], 0x5410);
                    b[j][2 * f + 1] = __byte_perm(x[2 * f], x[2 * f + 1], 0x7632);
                  }
                }
              }
#pragma unroll
              for (int f = 0; f < 4; ++f) {
                nan0 |= e4m3_nan(w0[f]);
                nan1 |= e4m3_nan(w1[f]);
                const uint32_t a0 = e4m3_even(w0[f]), a1 = e4m3_even(w1[f]), a2 = e4m3_odd(w0[f]), a3 = e4m3_odd(w1[f]);
#pragma unroll
                for (int j = 0; j < kGroups; ++j)
                  if (j < groups) mma_bf16(sum[j], a0, a1, a2, a3, b[j][2 * f], b[j][2 * f + 1]);
              }
            }
            float f0 = ue8m0_value(sc0), f1 = ue8m0_value(sc1);
            if (__any_sync(0xffffffffu, (nan0 | nan1) != 0)) {   // a NaN makes its row's sums NaN
              nan0 |= __shfl_xor_sync(0xffffffffu, nan0, 1);
              nan0 |= __shfl_xor_sync(0xffffffffu, nan0, 2);
              nan1 |= __shfl_xor_sync(0xffffffffu, nan1, 1);
              nan1 |= __shfl_xor_sync(0xffffffffu, nan1, 2);
              if (nan0 != 0) f0 = __uint_as_float(0x7fc00000u);
              if (nan1 != 0) f1 = __uint_as_float(0x7fc00000u);
            }
#pragma unroll
            for (int j = 0; j < kGroups; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (j < groups) acc[j][i] = fmaf(sum[j][i], i < 2 ? f0 : f1, acc[j][i]);
          }
          const int next = (c + 1) * kSplit + part;   // the next stage's scales, while this one's products run
          if (next * kFp8Block < p.K) {
            sc0 = __ldg(scale0 + next);
            sc1 = __ldg(scale1 + next);
          }
        } else if (some) {
#pragma unroll
          for (int i = 0; i < kChunk / kStep / kSplit; ++i) {
            const int k0 = (part + i * kSplit) * kStep;
            if (k0 < left) {
              const bool in = k0 + t * 8 < left;          // what lies behind a row is not multiplied
              const uint4 r0 = ld_shared_v4_at(wa + row0 * kPiece + k0 * 2), r1 = ld_shared_v4_at(wa + row1 * kPiece + k0 * 2);
#pragma unroll
              for (int j = 0; j < kGroups; ++j) {
                if (j < groups) {
                  const uint4 b = in ? ld_shared_v4_at(va + j * 8 * kTokenPitch + k0 * 2) : make_uint4(0, 0, 0, 0);
                  mma_bf16(acc[j], r0.x, r1.x, r0.y, r1.y, b.x, b.y);
                  mma_bf16(acc[j], r0.z, r1.z, r0.w, r1.w, b.z, b.w);
                }
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[s]);
        if (++s == stages) {
          s = 0;
          phase ^= 1;
        }
      }
      // ---------------------------------------------------------------- the warps' sums
      if (some) {
#pragma unroll
        for (int j = 0; j < kGroups; ++j)
          if (j < groups)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              red[part * red_part + (j * 8 + 2 * t + (i & 1)) * kRedPitch + h * 16 + (i >> 1) * 8 + g] = acc[j][i];
      }
      named_barrier_sync(1, kConsumers * kWarp);
      auto total = [&](int n, int row) {
        float sum = 0.0f;
#pragma unroll
        for (int q = 0; q < kSplit; ++q) sum += red[q * red_part + n * kRedPitch + row];
        return sum;
      };
      if (kIn) {
        for (int i = threadIdx.x; i < w.m * (kUnitRows / 2); i += kConsumers * kWarp) {
          const int n = i / (kUnitRows / 2), c = i % (kUnitRows / 2), row = (c >> 3) * 16 + (c & 7);
          if (c < w.cols)   // rounded to bf16: the second kernel's operand
            p.out[(int64_t)l.slot[w.s0 + n] * p.N + w.col + c] = __float2bfloat16_rn(act_value<kAct>(total(n, row)) * total(n, row + 8));
        }
      } else {
        for (int i = threadIdx.x; i < w.m * kUnitRows; i += kConsumers * kWarp) {
          const int n = i / kUnitRows, c = i % kUnitRows, token = l.token[w.s0 + n];
          if (c >= w.cols || (n > 0 && l.token[w.s0 + n - 1] == token)) continue;
          float sum = sh.sums[token * kUnitRows + c];
          for (int q = n; q < w.m && l.token[w.s0 + q] == token; ++q)   // one, but for an expert named twice
            sum = fmaf(__ldg(p.weights + l.slot[w.s0 + q]), total(q, c), sum);
          sh.sums[token * kUnitRows + c] = sum;
        }
        if (w.last) {
          named_barrier_sync(1, kConsumers * kWarp);
          for (int i = threadIdx.x; i < p.T * kUnitRows; i += kConsumers * kWarp) {
            const int c = i % kUnitRows;
            if (c < w.cols) p.out[(int64_t)(i / kUnitRows) * p.N + w.col + c] = __float2bfloat16_rn(sh.sums[i]);
            sh.sums[i] = 0.0f;
          }
        }
      }
      float* const was = red;   // the next unit's sums go elsewhere: these may still be read
      red = red_next;
      red_next = was;
    }
    if (!kIn) {
      pdl_wait();   // (the copying warps have; this one writes where the first kernel may still read)
      if (l.used == 0)
        for (int64_t i = (int64_t)blockIdx.x * (kConsumers * kWarp) + threadIdx.x; i < (int64_t)p.T * p.N; i += (int64_t)gridDim.x * (kConsumers * kWarp))
          p.out[i] = __float2bfloat16_rn(0.0f);
    }
  }
  if (!ok) set_status(p.status, EP_ERR_TIMEOUT);
}

template <bool kFp8, bool kIn, int kAct>
static int launch_few_half(const FewParams& p, cudaStream_t s) {
  auto* fn = k_few<kFp8, kIn, kAct>;
  if (ep_host::ensure_max_smem(reinterpret_cast<const void*>(fn), kFewSmem) != EP_OK) return EP_ERR_CUDA;
  const int grid = ep_host::grid_cap(1);
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
  const int one = fp8 ? 1 : 2;
  auto maps = [&](FewParams& f, const void* w, int count, int whole) {
    const uint64_t words = (uint64_t)f.K * one / 4;
    int rc = ep_host::make_row_map(&f.whole, w, words, f.N, count, whole);
    if (rc == EP_OK) rc = ep_host::make_row_map(&f.four, w, words, f.N, count, 4);
    return rc == EP_OK ? ep_host::make_row_map(&f.one, w, words, f.N, count, 1) : rc;
  };
  if (maps(p, w_gu, 2 * E, kUnitRows / 2) != EP_OK || maps(q, w_down, E, kUnitRows) != EP_OK) return EP_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return fp8 ? launch_few<true>(p, q, act, s) : launch_few<false>(p, q, act, s);
}
