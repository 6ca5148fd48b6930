// few.cu -- a whole mixture-of-experts layer for a few tokens, in two kernels.
//
//   kIn    h = act(Wg x) * (Wu x)   for every slot (a token and one of its experts)
//   kOut   out = sum over a token's slots of weight * (W_down h)
//
// Both are bound by reading each used expert's weights once.  The first deals
// out (expert, h column) pairs over the CTAs, the second output columns, so
// that every CTA sums its own columns over all experts in a fixed order and
// nothing is added up between CTAs.  A CTA walks its columns in units, whole in the
// inner index, for the tokens of one expert.  The second kernel comes up as the first
// one's CTAs leave and fills its ring with weights before it waits for h.
//
// Here for E4M3 weights, by tcgen05: a unit is 32 columns' rows of gate and up, or 64
// rows of W_down.  The weights' rows are the first operand (64
// of them, those past the unit's being whatever lies there), the tokens, split into two E4M3 numbers each,
// the second, 8 to 32 columns, and no thread touches a weight: by mma.sync they had to be turned into fp16 first,
// which took a batch of 32 (128 experts, 7168 x 2048, top-8) 1129 us instead of 767.  bf16 weights need no turning, and
// their rows, of any multiple of 16 bytes, come in 1 KB pieces where this form wants 128-byte ones: few_bf16.cu.
// Warps:
//   8 bring the sums out of tensor memory, in two teams, a stage each; the first finishes a unit
//   1 issues the products
//   2 copy weights (TMA, 8 rows x 512 bytes a copy), 1 tokens' rows
//   4 put the tokens where the products read them, in two teams, a stage each

#include <type_traits>

#include "few.cuh"

namespace ep {

constexpr int kQuarters = 4, kSumTeams = 2, kEpilogues = kQuarters * kSumTeams;   // a unit's stages in turn: one takes a team 1050 clocks
constexpr int kWeightWarps = 2, kRowWarps = 1;   // a warp issues a copy in some 80 clocks; sixteen warps: with one more, 96 registers
constexpr int kTeams = 2, kTeam = 2, kTurners = kTeams * kTeam;   // a stage is one team's: its latency is 500 clocks and more
constexpr int kFewThreads = (kEpilogues + 1 + kRowWarps + kWeightWarps + kTurners) * kWarp;
constexpr int kUnitRows = 64;         // of weights
constexpr int kBlocks = 4;            // 128-byte blocks of a row in a stage
constexpr int kGroupBytes = kBlocks * 1024;   // 8 rows of a stage
constexpr int kWeightBytes = kUnitRows / 8 * kGroupBytes;
constexpr int kSums = 4;              // sums on their way out of tensor memory
constexpr int kScaleRing = 16;        // stages whose tokens' scales are kept: more than are between the copies and the epilogue
constexpr int kMaxFewStages = 8;
constexpr int kPass = 16;             // tokens of an expert taken at a time, two columns of products each

struct FewParams : FewCall {
  CUtensorMap w;               // weights [2 E or E][N][K]: 8 rows of 4 blocks of 128 bytes
};

struct FewShared {
  uint64_t full[kMaxFewStages], turned[kMaxFewStages], empty[kMaxFewStages];
  uint64_t sums_full[kSums], sums_empty[kSums];
  uint64_t part_full[2], part_empty[2];
  FewCounts counts;
  uint32_t tmem;
  alignas(16) float scales[kScaleRing][kBlocks][kPass];   // what a token's block was divided by
  float part[2][kPass][kUnitRows];           // the second team's sums of a unit
  float up[2][kPass][kUnitRows / 2];         // kIn: on its way to its gate
};

// ---------------------------------------------------------------- products

__device__ __forceinline__ void umma_few(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool add) {
  constexpr uint32_t kWeightsHi = ((uint32_t)kGroupBytes >> 4) | (1u << 14) | (2u << 29);   // 8-row groups 4 KB apart
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n"
      " mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %6};\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"((uint32_t)add), "r"(kWeightsHi), "r"(kDescHi)
      : "memory");
}
// Instruction descriptor: 64 rows, n columns; E4M3 operands, fp32 sums.  Rows
// 16 w .. 16 w + 15 come out in the first 16 lanes of quarter w of the tensor memory.
__device__ __forceinline__ uint32_t umma_few_idesc(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | (4u << 24); }

// A token's bf16 numbers as two E4M3 ones, for E4M3 weights: in a block of 128
// inner elements whose largest is in [2^e, 2^(e+1)), x = 2^(e-7) (hi + lo / 16) with
// hi = E4M3(x 2^(7-e)) and lo = E4M3 of what that leaves, times 16: columns 2 j and
// 2 j + 1 of the products.  bf16 has 8 significant bits and each part 4, so this is x
// itself down to 2^-13 of the largest, and 2^-21 of the largest off below: no more
// than sums in 32 bits lose.  A block with an infinity or NaN gets the scale NaN.
// An fp32 number (h) is rounded so to about 2^-9 of itself.  8 elements a lane, a block sixteen lanes.
template <bool kWide>
struct TokenPiece {   // as it lies in memory: bf16 or fp32
  uint4 v[kWide ? 2 : 1];

  // the largest exponent, biased, or 255 with an infinity or NaN among them
  __device__ __forceinline__ uint32_t top() const {
    if constexpr (kWide) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) m = max(max(m, max(v[i].x & 0x7fffffffu, v[i].y & 0x7fffffffu)), max(v[i].z & 0x7fffffffu, v[i].w & 0x7fffffffu));
      return m >> 23;
    } else {
      uint32_t a = v[0].x & 0x7fff7fffu, b = v[0].y & 0x7fff7fffu;
      asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(v[0].z & 0x7fff7fffu));
      asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(b) : "r"(v[0].w & 0x7fff7fffu));
      asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
      return max(a >> 16, a & 0xffffu) >> 7;
    }
  }
  __device__ __forceinline__ float2 pair(int i) const {
    if constexpr (kWide) {
      const uint4 q = v[i >> 1];
      return i & 1 ? make_float2(__uint_as_float(q.z), __uint_as_float(q.w)) : make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
    } else {
      const uint32_t w = i == 0 ? v[0].x : i == 1 ? v[0].y : i == 2 ? v[0].z : v[0].w;
      return make_float2(bf16_lo(w), bf16_hi(w));
    }
  }
  __device__ __forceinline__ void split(uint32_t e, uint32_t (&hi)[2], uint32_t (&lo)[2], float& scale) const {
    const float up = __uint_as_float((e <= 7 ? 254u : 261u - min(e, 254u)) << 23);   // 2^(134 - e), no more than 2^127
    scale = e == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(e <= 7 ? 0x00400000u : (e - 7) << 23);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t h[2], r[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float2 p = pair(2 * i + q);
        const float x = p.x * up, y = p.y * up;
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
};

__device__ __forceinline__ float ue8m0_value(uint32_t b) {
  return b == 255 ? __uint_as_float(0x7fc00000u) : b == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23);
}

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

// A team's sums of a unit's rows, over its stages, for the tokens of kColumns columns:
// y[j] of token j, a row a thread; ok: no wait has run out.
template <int kColumns>
__device__ __forceinline__ void few_sums(FewShared& sh, uint32_t tmem, int team, int columns, int chunks, int K, const uint8_t* scale, RingPosition& sums,
                                         uint32_t& stage, float (&y)[kPass], bool& ok) {
  constexpr int kTokens = kColumns / 2, kCount = kColumns == 32 ? 2 : kBlocks;
  const int blocks = K / kFp8Block;
  uint32_t next[kBlocks];
  auto fetch = [&](int c) {
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) next[b] = c * kBlocks + b < blocks ? __ldg(scale + c * kBlocks + b) : 0u;
  };
  fetch(team);
#pragma unroll
  for (int j = 0; j < kTokens; ++j) y[j] = 0.0f;
  for (int c = 0; c < chunks; ++c, ++stage, sums.advance()) {
    // (the other team's are skipped: a wait for a phase two ahead cannot pass, as the last stage that was this team's
    // lies after the one that had these sums before)
    if (c % kSumTeams != team) continue;
    float f[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) f[b] = ue8m0_value(next[b]);
    fetch(c + kSumTeams);
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
              // (the token's scale first: zeros stay zeros under any weights' scale.  The other way round they would not, and with
              // an order by size, which lifts the limit of 2^111 for tokens, 32 tokens take 783 us instead of 770)
              y[j] = fmaf(fmaf(v[b][2 * j + 1], 0.0625f, v[b][2 * j]) * of[q], f[b0 + b], y[j]);
            }
          }
        }
      }
    }
    tmem_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.sums_empty[sums.s]);
  }
}

template <bool kIn, int kAct>
__global__ void __launch_bounds__(kFewThreads, 1) k_few_e4m3(const __grid_constant__ FewParams p) {
  constexpr int kBlock = 128, kChunk = kBlocks * kBlock;   // inner elements of a block, of a stage
  constexpr bool kWide = !kIn;                       // tokens' rows are fp32
  constexpr int kRawBytes = kChunk * (kWide ? 4 : 2);   // a token's row in a stage, as it comes
  using Lists = FewLists<kIn ? 0 : kUnitRows>;
  using Walk = FewWalk<kIn, kPass, kUnitRows>;
  extern __shared__ __align__(1024) uint8_t raw[];
  FewShared& sh = *reinterpret_cast<FewShared*>(raw);
  uint8_t* const ring = raw + (sizeof(FewShared) + 1023) / 1024 * 1024;
  uint8_t* const lists_at = raw + kFewSmem - Lists::bytes(p.E, p.T, p.k);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    // Everybody who waits for a phase of a barrier takes part in the slot's next one, so that nobody can be left a whole
    // turn of the ring behind: weights' warps without a copy of the stage, and the team of the other stages, arrive too.
    for (int s = 0; s < kMaxFewStages; ++s) {
      mbar_init(&sh.full[s], kWeightWarps);
      mbar_init(&sh.turned[s], kTurners);
      mbar_init(&sh.empty[s], 1);
    }
    for (int b = 0; b < kSums; ++b) {
      mbar_init(&sh.sums_full[b], 1);
      mbar_init(&sh.sums_empty[b], kQuarters);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.part_full[b], kQuarters);
      mbar_init(&sh.part_empty[b], kQuarters);
    }
    fence_barrier_init();
  }
  if (warp == kEpilogues) tmem_alloc<1>(&sh.tmem, 512);
  if (threadIdx.x == kFewThreads - 1) prefetch_map(&p.w);
  if (kIn) {
    pdl_wait();   // ids and tokens may come from the kernel before
    pdl_launch_dependents();
  }
  const Lists l(lists_at, p.E, p.T, p.k);
  tmem_fence_before();
  few_lists<kFewThreads>(p, sh.counts, l, reinterpret_cast<uint32_t*>(ring), kIn && blockIdx.x == 0);
  tmem_fence_after();
  const uint32_t tmem = sh.tmem;
  const int tokens_most = min(sh.counts.most, kPass);
  const int columns = (tokens_most * 2 + 7) / 8 * 8;   // of products, most
  const int chunks = (p.K + kChunk - 1) / kChunk;
  Walk w(l.used, sh.counts.n_used, p.N, p.wave);
  // a stage: weights, tokens for the products, tokens as they came.  Products read 64
  // rows; what W_down's units have no rows for is other stages' memory, or the lists'.
  const int weight_bytes = kIn ? kWeightBytes : (max(w.most, 1) + 7) / 8 * kGroupBytes;
  const int token_block = columns * 128, stage_bytes = (weight_bytes + kBlocks * token_block + tokens_most * kRawBytes + 1023) / 1024 * 1024;
  const int stages = max(1, min(kMaxFewStages, min((int)(lists_at - ring) / stage_bytes, ((int)(raw + kFewSmem - ring) - kWeightBytes) / stage_bytes + 1)));
  RingPosition at(stages);
  bool ok = true;

  if (warp < kEpilogues) {
    // ---------------------------------------------------------------- sums: a row a thread
    RingPosition sums(kSums);
    uint32_t stage = 0, unit = 0;
    const int quarter = warp % kQuarters, team = warp / kQuarters;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const int row = quarter * 16 + (lane & 15), column = kIn ? row % (kUnitRows / 2) : row;   // kIn: gate in two warps, up in the others
    const bool there = lane < 16;
    if (!kIn && there && team == 0)
      for (int n = 0; n < p.T; ++n) l.sums[n * kUnitRows + row] = 0.0f;
    while (w.next()) {
      const int n = min(w.col + column, p.N - 1);
      const uint8_t* const scale = p.scales + ((int64_t)(kIn ? w.e * 2 + (quarter >> 1) : w.e) * (p.N / kFp8Block) + n / kFp8Block) * (p.K / kFp8Block);
      float y[kPass];
      if (w.m * 2 > 16)
        few_sums<32>(sh, lanes, team, columns, chunks, p.K, scale, sums, stage, y, ok);
      else if (w.m * 2 > 8)
        few_sums<16>(sh, lanes, team, columns, chunks, p.K, scale, sums, stage, y, ok);
      else
        few_sums<8>(sh, lanes, team, columns, chunks, p.K, scale, sums, stage, y, ok);
      if (chunks > 1) {   // the teams' sums together
        const int b = unit & 1;
        const uint32_t phase = (unit >> 1) & 1;
        if (ok) ok = team == 0 ? wait_few(&sh.part_full[b], phase, 4 * kWaitNs) : wait_few(&sh.part_empty[b], phase ^ 1, 4 * kWaitNs);
        if (there) {
#pragma unroll
          for (int j = 0; j < kPass; ++j) {
            if (j >= w.m) break;
            if (team == 0)
              y[j] += sh.part[b][j][row];
            else
              sh.part[b][j][row] = y[j];
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(team == 0 ? &sh.part_empty[b] : &sh.part_full[b]);
      }
      ++unit;
      if (team != 0) continue;
      if (kIn) {
        float(&up)[kPass][kUnitRows / 2] = sh.up[unit & 1];
        if (quarter >= kQuarters / 2 && there) {
#pragma unroll
          for (int j = 0; j < kPass; ++j) {
            if (j >= w.m) break;
            up[j][column] = y[j];
          }
        }
        named_barrier_sync(1, kQuarters * kWarp);
        if (quarter < kQuarters / 2 && there && column < w.cols) {
#pragma unroll
          for (int j = 0; j < kPass; ++j) {   // the second kernel's operand
            if (j >= w.m) break;
            reinterpret_cast<float*>(p.out)[(int64_t)l.slot[w.s0 + j] * p.N + w.col + column] = act_value<kAct>(y[j]) * up[j][column];
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
    }
    if (!kIn && sh.counts.n_used == 0) {
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
        const uint32_t idesc = umma_few_idesc((w.m * 2 + 7) / 8 * 8);
        for (int c = 0; c < chunks; ++c) {
          ok = wait_alone(&sh.sums_empty[sums.s], sums.phase ^ 1, 4 * kWaitNs);
          ok = ok && wait_alone(&sh.turned[at.s], at.phase);   // by who has seen the weights' copies
          if (!ok) break;
          tmem_fence_after();
          const int blocks = (p.K - c * kChunk + kBlock - 1) / kBlock;
          const uint32_t a = weights0 + (uint32_t)at.s * (stage_bytes >> 4), b = tokens0 + (uint32_t)at.s * (stage_bytes >> 4);
          const uint32_t d = tmem + sums.s * (columns * kBlocks);
#pragma unroll
          for (int i = 0; i < kBlocks; ++i) {
            if (i < blocks) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                umma_few(d + i * columns, a + (i * 64 + q * 2), b + i * (token_block >> 4) + q * 2, idesc, q > 0);
            }
          }
          umma_commit(&sh.empty[at.s]);
          at.advance();
          umma_commit(&sh.sums_full[sums.s]);
          sums.advance();
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
      const uint8_t* row = reinterpret_cast<const uint8_t*>(p.v) + (int64_t)from * p.K * (kRawBytes / kChunk);
      for (int c = 0; c < chunks; ++c) {
        ok = wait_few(&sh.empty[at.s], at.phase ^ 1);
        if (!ok) break;
        if (from >= 0)
          tma_load_1d(ring + at.s * stage_bytes + weight_bytes + kBlocks * token_block + mine * kRawBytes, row + (int64_t)c * kRawBytes,
                      min(kChunk, p.K - c * kChunk) * (kRawBytes / kChunk), &sh.full[at.s]);
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
          if (turn == 0)
            mbar_arrive_expect_tx(&sh.full[at.s], (kIn ? 2 : 1) * groups * kGroupBytes + w.m * k * (kRawBytes / kChunk));
          else
            mbar_arrive(&sh.full[at.s]);
          const uint32_t to = smem_addr(ring + at.s * stage_bytes), bar = smem_addr(&sh.full[at.s]);
          for (int half = 0; half < (kIn ? 2 : 1); ++half) {
            const int z = kIn ? 2 * w.e + half : w.e;
            for (int g = turn; g < groups; g += kWeightWarps) {
              const uint32_t group = to + (half * (kUnitRows / 16) + g) * kGroupBytes;
              tma_load_4d(group, &p.w, bar, 0, w.col + g * 8, c * kBlocks, z);   // blocks behind the row's end are zeros
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
        // every stage is waited for, another team's too: they may land out of order, and a wait two phases ahead passes;
        // and the products wait until both teams have seen it, or the slot could be filled anew before this team looks
        if (ok) ok = wait_few(&sh.full[at.s], at.phase);
        if (stage % kTeams != (uint32_t)team) {
          if (lane == 0) mbar_arrive(&sh.turned[at.s]);
          continue;
        }
        const uint32_t to = smem_addr(ring + at.s * stage_bytes + weight_bytes), from = to + kBlocks * token_block;
        const int left = p.K - c * kChunk;
        // an item is two blocks of a token, a lane's 8 elements of one: several at a time, each step of all before the next
        // (one after the other they took 440 clocks each: 32 tokens through 32 experts, top-8:
        // 372 us instead of 458)
        auto turn_items = [&](auto items) {
          constexpr int kItems = decltype(items)::value;
          for (int i0 = member; i0 < 2 * w.m; i0 += kTeam * kItems) {
            const int piece = lane & 15;
            TokenPiece<kWide> v[kItems];
            uint32_t top[kItems];
            bool in[kItems];
#pragma unroll
            for (int u = 0; u < kItems; ++u) {
              const int i = i0 + u * kTeam, b = (i & 1) * 2 + (lane >> 4);
              in[u] = i < 2 * w.m && b * kBlock < left;
#pragma unroll
              for (int h = 0; h < (kWide ? 2 : 1); ++h)
                v[u].v[h] = in[u] ? ld_shared_v4_at(from + (i >> 1) * kRawBytes + (b * kBlock + piece * 8) * (kRawBytes / kChunk) + h * 16) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < kItems; ++u) top[u] = v[u].top();
#pragma unroll
            for (int o = 1; o < 16; o <<= 1)
#pragma unroll
              for (int u = 0; u < kItems; ++u) top[u] = max(top[u], __shfl_xor_sync(0xffffffffu, top[u], o));
#pragma unroll
            for (int u = 0; u < kItems; ++u) {
              const int i = i0 + u * kTeam, j = i >> 1, b = (i & 1) * 2 + (lane >> 4);
              uint32_t hi[2], lo[2];
              float scale;
              v[u].split(top[u], hi, lo, scale);
              if (in[u]) {
                const uint32_t row = to + b * token_block + 2 * j * 128, at_hi = row + ((((piece >> 1) ^ (2 * j & 7)) << 4) | ((piece & 1) << 3));
                const uint32_t at_lo = row + 128 + ((((piece >> 1) ^ ((2 * j + 1) & 7)) << 4) | ((piece & 1) << 3));
                asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at_hi), "r"(hi[0]), "r"(hi[1]) : "memory");
                asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at_lo), "r"(lo[0]), "r"(lo[1]) : "memory");
                if (piece == 0) sh.scales[stage % kScaleRing][b][j] = scale;
              }
            }
          }
        };
        if (w.m == 1)
          turn_items(std::integral_constant<int, 2 / kTeam>());
        else
          turn_items(std::integral_constant<int, 4>());
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

static int launch_few_e4m3(const FewCall& in, const FewCall& out, const void* w_gu, const void* w_down, int act, cudaStream_t s) {
  FewParams p{in}, q{out};
  auto map = [&](FewParams& f, const void* w, uint64_t count) {
    const uint64_t N = f.N, K = f.K;
    const uint64_t dims[4] = {kFp8Block, N, K / kFp8Block, count}, strides[3] = {K, kFp8Block, N * K};
    const uint32_t box[4] = {kFp8Block, 8, kBlocks, 1};
    return ep_host::make_map(&f.w, true, 4, w, dims, strides, box);
  };
  if (map(p, w_gu, 2 * (uint64_t)in.E) != EP_OK || map(q, w_down, in.E) != EP_OK) return EP_ERR_CUDA;
  // SMs get through the same work up to a sixth faster or slower than the mean, which a large call
  // pays for at its end: more CTAs with a few columns, which come up where others have left.  0.47 GB of gate and
  // up take 88 us in one wave and 98 so, 0.70 GB 255 and 232, 3.8 GB 842 and 763 (with W_down).  bf16: 0.7 GB 3 % slower
  // so, 2.8 GB 0.3 % faster, so that its kernel keeps to one wave.
  constexpr int64_t kWaveBytes = (int64_t)1 << 29;   // of gate and up, if every slot has its own expert
  const int64_t bytes = 2 * (int64_t)std::min(p.T * p.k, p.E) * p.N * p.K;
  const int waves = bytes >= kWaveBytes && !ep_host::sm_budget_set() ? 3 : 1;
  auto* fn = act == EP_ACT_RELU ? k_few_e4m3<true, EP_ACT_RELU> : act == EP_ACT_SILU ? k_few_e4m3<true, EP_ACT_SILU> : k_few_e4m3<true, EP_ACT_GELU>;
  const int rc = launch_few_half(fn, kFewThreads, p, waves, s);
  return rc != EP_OK ? rc : launch_few_half(k_few_e4m3<false, EP_ACT_NONE>, kFewThreads, q, 1, s);
}

static bool few_sizes(int R, int T_r, int k, int E, int I) {
  return R > 0 && R <= kMaxR && T_r >= 0 && T_r <= EP_MOE_FEW_TOKENS && R * T_r <= EP_MOE_FEW_TOKENS && k > 0 && k <= kMaxK && E > 0 &&
         E <= kMaxE && E % R == 0 && I > 0 && I % 8 == 0 && I <= (1 << 24);
}

}  // namespace ep

extern "C" size_t ep_moe_few_workspace_size(int R, int T_r, int k, int E, int I) {
  if (!ep::few_sizes(R, T_r, k, E, I)) return 0;
  return std::max<size_t>(16, (size_t)R * T_r * k * I * ep::kHiddenBytes);   // (I is a multiple of 8)
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
  if (H % unit != 0 || I % unit != 0 || (int64_t)E * H >= lim || (int64_t)E * (I + kCrossing) >= lim) return EP_ERR_INVALID_ARG;
  if (act <= EP_ACT_NONE || act > EP_ACT_GELU) return EP_ERR_INVALID_ARG;
  if (fp8 != (w_gu_scales != nullptr) || fp8 != (w_down_scales != nullptr)) return EP_ERR_INVALID_ARG;
  if (T_r == 0) return EP_OK;
  for (const void* p : {x, w_gu, w_down, (const void*)out, (const void*)workspace})
    if (p == nullptr || !ep_host::aligned16(p)) return EP_ERR_INVALID_ARG;
  if (topk_idx == nullptr || topk_weights == nullptr || workspace_bytes < ep_moe_few_workspace_size(R, T_r, k, E, I))
    return EP_ERR_INVALID_ARG;
  FewCall p{};
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
  FewCall q = p;
  q.scales = w_down_scales;
  q.v = p.out;
  q.out = static_cast<__nv_bfloat16*>(out);
  q.K = I;
  q.N = H;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return fp8 ? launch_few_e4m3(p, q, w_gu, w_down, act, s) : launch_few_bf16(p, q, w_gu, w_down, act, s);
}
