// few_bf16.cu -- the layer for few tokens on bf16 weights, by mma.sync.
//
// A unit is 16 columns' rows of gate and up, or 32 rows of W_down.  Warps:
//   8 multiply: each its eighth of a stage's inner index, 32 weight rows as the
//     first operand and 8 tokens as the second (m16n8k16: at a few tokens an expert
//     the widest form that is not mostly padding)
//   4 add the eight sums of a unit up and finish it while the next one's products run
//   1 copies the weights (TMA, 1 KB of each row a stage), 2 tokens' rows
// Registers take the weights as they lie, so rows need no alignment but
// 16 bytes and come in the longest pieces.  The same by tcgen05 (few.cu) wants them in boxes of 128-byte rows, which
// begin off the memory's lines where a row is not a multiple of 128 bytes, and 64 rows a
// product: one token through six experts of 4096 x 1416
// 49 us instead of 39, 18 tokens through 32 of them 176 instead of 151, 64 through eight of 4096 x 2048 92 instead of 75
// (both with h in bf16).

#include <type_traits>

#include "few.cuh"

namespace ep {

constexpr int kParts = 8;             // warps that multiply
constexpr int kAdders = 4;            // warps that add up
constexpr int kTokenWarps = 2;
constexpr int kRowThreads = (kParts + kAdders + 1 + kTokenWarps) * kWarp;
constexpr int kPiece = 1024;          // bytes of a weight row in a stage
constexpr int kChunk = kPiece / 2;    // inner elements of a stage
constexpr int kRowUnit = 32;          // rows of a unit
constexpr int kRedPitch = 36;         // floats: a warp's sums fall into distinct banks
// Tokens of an expert taken at a time: two stages at least.  24 of two words each do not fit the registers (64 tokens
// through eight experts of 4096 x 2048 86 us with 16, 88 with 24, one token 39.2 and 41.0).
__host__ __device__ constexpr int row_pass(bool two) { return two ? 16 : 24; }
constexpr int kRowStages = 8;
constexpr int kTokenPitch = kPiece + 64;   // 8 lanes' 16 bytes fall into distinct banks

struct RowParams : FewCall {
  CUtensorMap whole, four, one;   // weights [2 E or E][N][K]: boxes of 1 KB of a unit's rows (kIn: of gate or up), 4 and 1
};

struct RowShared {
  uint64_t full[kRowStages], empty[kRowStages];
  uint64_t red_full[2], red_empty[2];
  FewCounts counts;
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A warp's eighth of a unit: 32 rows, 8 G columns: of tokens, or (kOut) of the two words of each, whose
// sums come together at the end: the second words lie 4 columns on where all fit 8 (G = 1), else G / 2 times 8.
// Nothing in here branches on what the unit holds (what lies where no row or token
// does is multiplied and not used): with branches around its loads a stage took
// 1500 clocks, most of them waiting for one load after the other.
template <bool kIn, int G>
__device__ __forceinline__ void few_products(int K, RowShared& sh, const uint8_t* ring, int stage_bytes, float* red, int chunks,
                                             RingPosition& at_red, RingPosition& at_stage, bool& ok) {
  constexpr int kStep = 32;   // inner elements a warp multiplies at a time: 16 bytes of weights a lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, odd = g & 1;
  const int k0 = warp * 2 * kStep;        // this warp's first inner element of a stage
  // this lane's rows of a stage: kIn gate and up of column g, then of g + 8; kOut g, g + 8, g + 16, g + 24
  auto row_of = [&](int q) { return kIn ? (q & 1) * 16 + (q >> 1) * 8 + g : q * 8 + g; };
  float acc[2][G][4] = {};
  for (int c = 0; c < chunks; ++c) {
    const int left = K - c * kChunk;   // inner elements from this stage on
    if (ok) ok = wait_few(&sh.full[at_stage.s], at_stage.phase);
    if (k0 < left) {
      const uint32_t at = smem_addr(ring + at_stage.s * stage_bytes), tokens = at + kRowUnit * kPiece;
      const uint32_t wa = at + k0 * 2 + t * 16, va = tokens + g * kTokenPitch + k0 * 2 + t * 16;
      // Rows lie 1 KB apart, in the same banks: lanes of odd rows read the two steps in the other order, so that
      // a quarter-warp's two rows fall into different halves of the banks, and swap.
      uint4 r[4][2];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) r[q][i] = ld_shared_v4_at(wa + row_of(q) * kPiece + (odd ^ i) * 64);
      uint4 b[2][G];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < G; ++j) b[i][j] = ld_shared_v4_at(va + j * 8 * kTokenPitch + i * kStep * 2);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool in = k0 + i * kStep + t * 8 < left;   // what lies behind a token's row is not multiplied (weights are zeros there)
#pragma unroll
        for (int j = 0; j < G; ++j)
          if (!in) b[i][j] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 r0 = odd ? r[2 * h][i ^ 1] : r[2 * h][i], r1 = odd ? r[2 * h + 1][i ^ 1] : r[2 * h + 1][i];
#pragma unroll
          for (int j = 0; j < G; ++j) {
            mma_bf16(acc[h][j], r0.x, r1.x, r0.y, r1.y, b[i][j].x, b[i][j].y);
            mma_bf16(acc[h][j], r0.z, r1.z, r0.w, r1.w, b[i][j].z, b[i][j].w);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.empty[at_stage.s]);
    at_stage.advance();
  }
  constexpr int kSums = !kIn && G > 1 ? G / 2 : G;
  if constexpr (!kIn) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < kSums; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[h][j][i] += G == 1 ? __shfl_xor_sync(0xffffffffu, acc[h][j][i], 2) : acc[h][j + G / 2][i];
  }
  if (ok) ok = wait_few(&sh.red_empty[at_red.s], at_red.phase ^ 1);
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < kSums; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[(j * 8 + 2 * t + (i & 1)) * kRedPitch + h * 16 + (i >> 1) * 8 + g] = acc[h][j][i];
  __syncwarp();
  if (lane == 0) mbar_arrive(&sh.red_full[at_red.s]);
  at_red.advance();
}

// What cutting h to bf16 leaves, off by 2^-16 of h at most (where that is a normal number: above 2^-110).  It has h's sign and is no zero where h is none, so that
// an infinity among the weights comes out as it does from h: of two products with it neither is a NaN, or the other infinity.
__device__ __forceinline__ __nv_bfloat16 second_word(float h) {
  const float hi = __bfloat162float(__float2bfloat16_rz(h));
  float lo = isfinite(hi) ? h - hi : hi;
  if (lo == 0.0f && hi != 0.0f) lo = copysignf(fmaxf(fabsf(hi) * 9.3132257e-10f, 1.1754944e-38f), hi);   // 2^-30 of it, or the least normal number
  return __float2bfloat16_rn(lo);
}

template <bool kIn, int kAct>
__global__ void __launch_bounds__(kRowThreads, 1) k_few_bf16(const __grid_constant__ RowParams p) {
  using Lists = FewLists<kIn ? 0 : kRowUnit>;
  extern __shared__ __align__(1024) uint8_t raw[];
  RowShared& sh = *reinterpret_cast<RowShared*>(raw);
  uint8_t* const lists_at = raw + kFewSmem - Lists::bytes(p.E, p.T, p.k);
  uint8_t* const red_base = raw + (sizeof(RowShared) + 127) / 128 * 128;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kRowStages; ++s) {
      mbar_init(&sh.full[s], 1 + kTokenWarps);   // a token warp without a row of the stage arrives too, or could be left a turn of the ring behind
      mbar_init(&sh.empty[s], kParts);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.red_full[b], kParts);
      mbar_init(&sh.red_empty[b], kAdders);
    }
    fence_barrier_init();
  }
  if (threadIdx.x == kRowThreads - 1) {
    prefetch_map(&p.whole);
    prefetch_map(&p.four);
    prefetch_map(&p.one);
  }
  if (kIn) {
    pdl_wait();   // ids and tokens may come from the kernel before
    pdl_launch_dependents();
  }
  const Lists l(lists_at, p.E, p.T, p.k);
  few_lists<kRowThreads>(p, sh.counts, l, reinterpret_cast<uint32_t*>(red_base), kIn && blockIdx.x == 0);
  constexpr bool kTwo = !kIn;   // token rows of a stage: two for each, as few_products wants them
  constexpr int kPass = row_pass(kTwo);
  const int tokens_most = min(sh.counts.most, kPass);
  const int rows_most = !kTwo ? tokens_most : tokens_most <= 4 ? 8 : (tokens_most + 7) / 8 * 16;
  const int red_part = (tokens_most + 7) / 8 * 8 * kRedPitch;         // floats of one part's sums
  const int red_bytes = kParts * red_part * 4;                        // of one unit
  const int stage_bytes = kRowUnit * kPiece + (rows_most * kTokenPitch + 127) / 128 * 128;
  // products read 8 tokens' rows, there or not: some may lie behind the last stage
  const int behind = kTwo ? 0 : ((tokens_most + 7) / 8 * 8 - tokens_most) * kTokenPitch;
  auto stages_with = [&](int reds) { return min(kRowStages, ((int)(lists_at - red_base) - reds * red_bytes - behind) / stage_bytes); };
  // two units' sums, or one's where that makes a third or fourth stage
  const int reds = stages_with(1) > stages_with(2) && stages_with(1) <= 4 ? 1 : 2, stages = stages_with(reds);
  uint8_t* const ring = red_base + reds * red_bytes;
  const int chunks = (p.K + kChunk - 1) / kChunk;
  FewWalk<kIn, kPass, kRowUnit> w(l.used, sh.counts.n_used, p.N, p.wave);
  bool ok = true;
  RingPosition position(stages), at_red(reds);

  if (warp < kParts) {
    // ---------------------------------------------------------------- products
    while (w.next()) {
      float* const red = reinterpret_cast<float*>(red_base + at_red.s * red_bytes) + warp * red_part;
      auto products = [&](auto g) { few_products<kIn, decltype(g)::value>(p.K, sh, ring, stage_bytes, red, chunks, at_red, position, ok); };
      using std::integral_constant;
      if (kTwo && w.m <= 4)
        products(integral_constant<int, 1>());
      else if (w.m <= 8)
        products(integral_constant<int, kTwo ? 2 : 1>());
      else if (w.m <= 16)
        products(integral_constant<int, kTwo ? 4 : 2>());
      else if constexpr (!kTwo)
        products(integral_constant<int, kPass / 8>());
    }
  } else if (warp < kParts + kAdders) {
    // ---------------------------------------------------------------- sums
    const int q = warp - kParts;
    if (!kIn)
      for (int n = q; n < p.T; n += kAdders) l.sums[n * kRowUnit + lane] = 0.0f;
    while (w.next()) {
      const int b = at_red.s;
      if (ok) ok = wait_few(&sh.red_full[b], at_red.phase, 2 * kWaitNs);
      const float* const red = reinterpret_cast<const float*>(red_base + b * red_bytes);
      auto total = [&](int n, int row) {
        float v[kParts];
#pragma unroll
        for (int i = 0; i < kParts; ++i) v[i] = red[i * red_part + n * kRedPitch + row];
        return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
      };
      if (kIn) {
        const int c = lane & 15, row = (c >> 3) * 16 + (c & 7);
        for (int n = q * 2 + (lane >> 4); n < w.m; n += 2 * kAdders)
          if (c < w.cols) {
            const float h = act_value<kAct>(total(n, row)) * total(n, row + 8);
            __nv_bfloat16* const to = p.out + (int64_t)l.slot[w.s0 + n] * 2 * p.N + w.col + c;   // the second kernel's operand
            to[0] = __float2bfloat16_rz(h);
            to[p.N] = second_word(h);
          }
      } else {
        // a token is one warp's, so its slots are added in the lists' order
        for (int n = 0; n < w.m; ++n) {
          const int token = l.token[w.s0 + n];
          if (token % kAdders == q) {
            float* const sum = l.sums + token * kRowUnit + lane;
            *sum = fmaf(l.weight[w.s0 + n], total(n, lane), *sum);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.red_empty[b]);
      at_red.advance();
      if (!kIn && w.last) {
        for (int n = q; n < p.T; n += kAdders) {
          if (lane < w.cols) p.out[(int64_t)n * p.N + w.col + lane] = __float2bfloat16_rn(l.sums[n * kRowUnit + lane]);
          l.sums[n * kRowUnit + lane] = 0.0f;
        }
      }
    }
    if (!kIn && sh.counts.n_used == 0) {
      pdl_wait();   // out may be x
      for (int64_t i = (int64_t)blockIdx.x * (kAdders * kWarp) + q * kWarp + lane; i < (int64_t)p.T * p.N; i += (int64_t)gridDim.x * (kAdders * kWarp))
        p.out[i] = __float2bfloat16_rn(0.0f);
    }
  } else if (warp == kParts + kAdders) {
    // ---------------------------------------------------------------- weights
    // a unit's rows in two copies (kIn) or one: by rows of 1 KB, a copy each, a warp got through 2.4 TB/s.  kOut: those of
    // the first stages before h is there.
    const bool issue = elect_one();
    while (ok && w.next()) {
      for (int c = 0; c < chunks; ++c) {
        ok = wait_few(&sh.empty[position.s], position.phase ^ 1);
        if (!ok) break;
        if (issue) {
          const int k = min(kChunk, p.K - c * kChunk);
          mbar_arrive_expect_tx(&sh.full[position.s], (kIn ? 2 : 1) * w.cols * kPiece + (kTwo ? 2 : 1) * w.m * k * 2);
          const uint32_t bar = smem_addr(&sh.full[position.s]);
          constexpr int kWhole = kIn ? kRowUnit / 2 : kRowUnit;
          for (int half = 0; half < (kIn ? 2 : 1); ++half) {
            const uint32_t to = smem_addr(ring + position.s * stage_bytes) + half * kWhole * kPiece;
            const int z = kIn ? 2 * w.e + half : w.e;
            if (w.cols == kWhole) {
              tma_load_3d<false>(to, &p.whole, bar, c * (kPiece / 4), w.col, z);
            } else {
              int n = 0;
              for (; n + 4 <= w.cols; n += 4) tma_load_3d<false>(to + n * kPiece, &p.four, bar, c * (kPiece / 4), w.col + n, z);
              for (; n < w.cols; ++n) tma_load_3d<false>(to + n * kPiece, &p.one, bar, c * (kPiece / 4), w.col + n, z);
            }
          }
        }
        __syncwarp();
        position.advance();
      }
    }
  } else {
    // ---------------------------------------------------------------- tokens
    const int turn = warp - (kParts + kAdders + 1);
    if (!kIn) pdl_wait();
    while (ok && w.next()) {   // a row a lane
      const int mine = lane * kTokenWarps + turn, word = kTwo && mine >= w.m ? 1 : 0, n = mine - word * w.m;
      const int from = n < w.m ? (kIn ? l.token[w.s0 + n] : l.slot[w.s0 + n] * (kTwo ? 2 : 1) + word) : -1;
      const int place = n + word * (w.m <= 4 ? 4 : (w.m + 7) / 8 * 8);
      const __nv_bfloat16* row = p.v + (int64_t)from * p.K;
      for (int c = 0; c < chunks; ++c) {
        ok = wait_few(&sh.empty[position.s], position.phase ^ 1);
        if (!ok) break;
        if (from >= 0)
          tma_load_1d(ring + position.s * stage_bytes + kRowUnit * kPiece + place * kTokenPitch, row + c * kChunk, min(kChunk, p.K - c * kChunk) * 2, &sh.full[position.s]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.full[position.s]);
        position.advance();
      }
    }
  }
  if (!ok) {
    set_status(p.status, EP_ERR_TIMEOUT);
    const uint64_t t0 = globaltimer_ns();   // give the copies in flight time to land before the memory goes
    while (globaltimer_ns() - t0 < 2000000ull) {
    }
  }
}

int launch_few_bf16(const FewCall& in, const FewCall& out, const void* w_gu, const void* w_down, int act, cudaStream_t s) {
  RowParams p{in}, q{out};
  auto maps = [&](RowParams& f, const void* w, int count, int whole) {
    const uint64_t words = (uint64_t)f.K / 2;
    int rc = ep_host::make_row_map(&f.whole, w, words, f.N, count, whole);
    if (rc == EP_OK) rc = ep_host::make_row_map(&f.four, w, words, f.N, count, 4);
    return rc == EP_OK ? ep_host::make_row_map(&f.one, w, words, f.N, count, 1) : rc;
  };
  if (maps(p, w_gu, 2 * in.E, kRowUnit / 2) != EP_OK || maps(q, w_down, in.E, kRowUnit) != EP_OK) return EP_ERR_CUDA;
  auto* fn = act == EP_ACT_RELU ? k_few_bf16<true, EP_ACT_RELU> : act == EP_ACT_SILU ? k_few_bf16<true, EP_ACT_SILU> : k_few_bf16<true, EP_ACT_GELU>;
  const int rc = launch_few_half(fn, kRowThreads, p, 1, s);
  return rc != EP_OK ? rc : launch_few_half(k_few_bf16<false, EP_ACT_NONE>, kRowThreads, q, 1, s);
}

}  // namespace ep
