// few.cu -- a whole mixture-of-experts layer for a few tokens, in two kernels.
//
//   k_few<.., kIn>    h = act(Wg x) * (Wu x)   for every slot (a token and one of its experts)
//   k_few<.., kOut>   out = sum over a token's slots of weight * (W_down h)
//
// Both are bound by reading each used expert's weights once.  The first deals
// out (expert, h column) pairs evenly over the CTAs, the second output columns, so
// that every CTA sums its own columns over all experts in a fixed order and
// nothing is added up between CTAs.  A CTA walks its columns in units: 16 columns'
// rows of gate and up, or 32 rows of W_down, whole in the inner index, for the
// tokens of one expert.  Its warps:
//   8 multiply: each its eighth of a stage's inner index, 32 weight rows as the
//     first operand and 8 tokens as the second (m16n8k16: at a few tokens an expert
//     the widest form that is not mostly padding; tcgen05 wants 64 rows or more in
//     tiles of their own, and an SM gets 13 to 110 columns)
//   4 add the eight sums of a unit up and finish it while the next one's products run
//   1 copies the weights (TMA, 1 KB of each row a stage), the rest tokens' rows
// The second kernel comes up as the first one's CTAs leave and fills its ring with
// weights before it waits for h.

#include "expert.cuh"
#include "umma.cuh"

namespace ep {

constexpr int kParts = 8;             // warps that multiply
constexpr int kAdders = 4;            // warps that add up
constexpr int kPiece = 1024;          // bytes of a weight row in a stage
constexpr int kUnitRows = 32;
constexpr int kRedPitch = 36;         // floats: a warp's sums fall into distinct banks
constexpr int kMaxSlots = EP_MOE_FEW_TOKENS * kMaxK;
constexpr int kMaxFewStages = 8;
constexpr int kFewSmem = 226 * 1024;
__host__ __device__ constexpr int pass_of(bool fp8) { return fp8 ? 16 : 24; }        // tokens of an expert taken at a time: two stages at least
__host__ __device__ constexpr int token_warps_of(bool fp8) { return fp8 ? 3 : 2; }   // fp8: they also turn numbers into fp16
__host__ __device__ constexpr int few_threads(bool fp8) { return (kParts + kAdders + 1 + token_warps_of(fp8)) * kWarp; }

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
struct FewUsed {
  int16_t expert, first, count, pad;   // slots first .. first + count of the lists
};
struct FewLists {
  FewUsed used[kMaxE];
  int16_t slot[kMaxSlots], token[kMaxSlots];
  float weight[kMaxSlots];
  int16_t id[kMaxSlots];               // expert of a slot, -1: unused
  int16_t start[kMaxE];
  int group_slots[kMaxE / kWarp], group_used[kMaxE / kWarp], group_most[kMaxE / kWarp];   // of 32 experts
  int n_used, most;                    // used experts; slots of the largest
};

struct FewShared {
  uint64_t full[kMaxFewStages], empty[kMaxFewStages];
  uint64_t red_full[2], red_empty[2];
  FewLists lists;
  float sums[EP_MOE_FEW_TOKENS * kUnitRows];   // kOut: the columns in hand, [token][column]
};

// masks: a bit a slot for every expert; memory that nothing else uses yet.
template <int kThreads>
__device__ __forceinline__ void few_lists(const FewParams& p, FewLists& l, uint32_t* masks, bool report) {
  const int n = p.T * p.k, words = (n + 31) / 32, groups = (p.E + 31) / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
      l.group_slots[q] = all;
      l.group_used[q] = __popc(some);
      l.group_most[q] = most;
    }
  }
  __syncthreads();
  for (int q = warp; q < groups; q += kThreads / kWarp) {
    const bool before = lane < q;
    const int slots = __reduce_add_sync(0xffffffffu, before ? l.group_slots[lane] : 0);
    const int used = __reduce_add_sync(0xffffffffu, before ? l.group_used[lane] : 0);
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
      const int all = __reduce_add_sync(0xffffffffu, lane < groups ? l.group_used[lane] : 0);
      const int most = __reduce_max_sync(0xffffffffu, lane < groups ? l.group_most[lane] : 0);
      if (lane == 0) {
        l.n_used = all;
        l.most = most;
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

// A CTA's units, one after another: `cols` columns from `col` on of an expert, for
// the tokens s0 .. s0 + m of the lists.
template <bool kIn, int kPass>
struct FewWalk {
  const FewLists* l;
  int N, left;           // kIn: (expert, column) pairs to come, from `col` of expert d on; kOut: columns from `col` on
  int d, e, col, cols, s0, m, behind;   // behind: the expert's tokens after these
  bool last;             // kOut: unit of these columns

  __device__ __forceinline__ FewWalk(const FewLists& lists, int n) {
    l = &lists;
    N = n;
    const int64_t all = kIn ? (int64_t)lists.n_used * n : lists.n_used > 0 ? n : 0;
    const int at = (int)(all * blockIdx.x / gridDim.x);
    left = (int)(all * (blockIdx.x + 1) / gridDim.x) - at;
    d = kIn ? at / n : lists.n_used - 1;
    col = kIn ? at - d * n : at;
    cols = s0 = m = behind = 0;
  }
  __device__ __forceinline__ bool next() {
    if (behind > 0) {
      s0 += m;
    } else {
      if (kIn) {
        left -= cols;
        col += cols;
        if (col == N) {
          col = 0;
          ++d;
        }
        if (left <= 0) return false;
        cols = min(min(kUnitRows / 2, N - col), left);
      } else {
        if (++d >= l->n_used) {
          left -= cols;
          col += cols;
          if (left <= 0) return false;
          cols = min(kUnitRows, left);
          d = 0;
        }
      }
      const FewUsed u = l->used[d];
      e = u.expert;
      s0 = u.first;
      behind = u.count;
    }
    m = min(kPass, behind);
    behind -= m;
    last = !kIn && behind == 0 && d + 1 == l->n_used;
    return true;
  }
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four E4M3 numbers as fp16, exactly (one instruction a pair; a bf16 form of them
// took 12 for the four and bounded the kernels at 3.5-4.0 TB/s of weights).
__device__ __forceinline__ void e4m3_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}" : "=r"(lo), "=r"(hi) : "r"(w));
}

// So tokens' bf16 numbers are multiplied as fp16: a block of 128 inner elements
// whose largest is in [2^e, 2^(e+1)) as x 2^(14-e), which is x itself down to
// 2^-31 of the largest and 2^-39 of the largest off below: far less than sums in 32
// bits lose.  A block with an infinity or NaN gets the scale NaN.
// 32 elements a lane, 128 over four lanes; the scale 2^(e-14) by the first of them.
__device__ __forceinline__ void scaled_f16(const uint4 (&v)[4], uint8_t* to, float* scale, bool first) {
  const uint32_t w[16] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w,
                          v[2].x, v[2].y, v[2].z, v[2].w, v[3].x, v[3].y, v[3].z, v[3].w};
  uint32_t tops[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    tops[i] = w[i] & 0x7fff7fffu;
#pragma unroll
    for (int q = 4; q < 16; q += 4) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(tops[i]) : "r"(w[i + q] & 0x7fff7fffu));
  }
  asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(tops[0]) : "r"(tops[1]));
  asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(tops[2]) : "r"(tops[3]));
  asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(tops[0]) : "r"(tops[2]));
  uint32_t top = max(tops[0] >> 16, tops[0] & 0xffffu);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const uint32_t e = top >> 7;   // biased; up = 2^(141 - e), no more than 2^127
  const float up = __uint_as_float((e <= 14 ? 254u : 268u - min(e, 254u)) << 23);
  if (first) *scale = e == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(e <= 14 ? 0x00400000u : (e - 14) << 23);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t f[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const __half2 h = __floats2half2_rn(bf16_lo(w[4 * i + q]) * up, bf16_hi(w[4 * i + q]) * up);
      f[q] = *reinterpret_cast<const uint32_t*>(&h);
    }
    st_shared_v4(to + 16 * i, make_uint4(f[0], f[1], f[2], f[3]));
  }
}

__device__ __forceinline__ float ue8m0_value(uint32_t b) {
  return b == 255 ? __uint_as_float(0x7fc00000u) : b == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23);
}

// Where a role is in the ring of stages.
struct RingPosition {
  int s;
  uint32_t phase;
  int stages, stage_bytes;

  __device__ __forceinline__ void advance() {
    if (++s == stages) {
      s = 0;
      phase ^= 1;
    }
  }
  __device__ __forceinline__ int offset() const { return s * stage_bytes; }
};

// A token's part of a stage: 8 lanes' 16 bytes (fp8: every second 16) fall into
// distinct banks; fp8: the scales of its 8 blocks lie behind.
__host__ __device__ constexpr int token_bytes(bool fp8) { return fp8 ? 2 * kPiece : kPiece; }
__host__ __device__ constexpr int token_pitch(bool fp8) { return token_bytes(fp8) + (fp8 ? 48 : 64); }

// A warp's eighth of a unit: 32 rows from column col of expert e on, 8 G tokens.
// Nothing in here branches on what the unit holds (what lies where no row or token
// does is multiplied and not used): with branches around its loads a stage took
// 1500 clocks, most of them waiting for one load after the other.
template <bool kFp8, bool kIn, int G>
__device__ __forceinline__ void few_products(const FewParams& p, FewShared& sh, int e, int col, const uint8_t* ring, float* red, int chunks,
                                             uint32_t unit, RingPosition& position, bool& ok) {
  constexpr int kOne = kFp8 ? 1 : 2, kChunk = kPiece / kOne, kTokenPitch = token_pitch(kFp8);
  constexpr int kStep = kFp8 ? 64 : 32;   // inner elements a warp multiplies at a time: 16 bytes of weights a lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, odd = g & 1;
  const int k0 = warp * 2 * kStep;        // this warp's first inner element of a stage
  // this lane's rows of a stage: kIn gate and up of column g, then of g + 8; kOut g, g + 8, g + 16, g + 24
  auto row_of = [&](int q) { return kIn ? (q & 1) * 16 + (q >> 1) * 8 + g : q * 8 + g; };
  float acc[2][G][4] = {};
  const uint8_t* scale[4] = {};
  uint32_t sc[4] = {};
  if (kFp8) {
    const int blocks_n = p.N / kFp8Block, blocks_k = p.K / kFp8Block;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int n = min(col + (kIn ? (q >> 1) * 8 + g : q * 8 + g), p.N - 1);
      scale[q] = p.scales + ((int64_t)(kIn ? e * 2 + (q & 1) : e) * blocks_n + n / kFp8Block) * blocks_k;
      if (warp < blocks_k) sc[q] = __ldg(scale[q] + warp);
    }
  }
  for (int c = 0; c < chunks; ++c) {
    const int left = p.K - c * kChunk;   // inner elements from this stage on
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.full[position.s], position.phase));
    if (k0 < left) {
      const uint32_t at = smem_addr(ring + position.offset()), tokens = at + kUnitRows * kPiece;
      const uint32_t wa = at + k0 * kOne + t * 16, va = tokens + g * kTokenPitch + k0 * 2 + t * (kFp8 ? 32 : 16);
      // Rows lie 1 KB apart, in the same banks: lanes of odd rows read the two steps in the other order, so that
      // a quarter-warp's two rows fall into different halves of the banks, and swap.
      uint4 r[4][2];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) r[q][i] = ld_shared_v4_at(wa + row_of(q) * kPiece + (odd ^ i) * 64);
      if constexpr (kFp8) {   // a block of 128 inner elements, whose scale is one a row and one a token
        uint4 lo[2][G], hi[2][G];
        float token[G][2];   // scales of tokens 2 t and 2 t + 1
        auto tokens_of = [&](int i) {
#pragma unroll
          for (int j = 0; j < G; ++j) {
            lo[i][j] = ld_shared_v4_at(va + j * 8 * kTokenPitch + i * kStep * 2);
            hi[i][j] = ld_shared_v4_at(va + j * 8 * kTokenPitch + i * kStep * 2 + 16);
          }
        };
        tokens_of(0);
        if (G == 1) tokens_of(1);
#pragma unroll
        for (int j = 0; j < G; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            asm volatile("ld.shared.f32 %0, [%1];"
                         : "=f"(token[j][i])
                         : "r"(tokens + (j * 8 + 2 * t + i) * kTokenPitch + token_bytes(true) + warp * 4));
        float sum[2][G][4] = {};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (G > 1 && i == 1) tokens_of(1);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t w0[4], w1[4];
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              w0[f] = odd ? (&r[2 * h][i ^ 1].x)[f] : (&r[2 * h][i].x)[f];
              w1[f] = odd ? (&r[2 * h + 1][i ^ 1].x)[f] : (&r[2 * h + 1][i].x)[f];
            }
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              uint32_t a0, a1, a2, a3;
              e4m3_to_f16(w0[f], a0, a2);
              e4m3_to_f16(w1[f], a1, a3);
#pragma unroll
              for (int j = 0; j < G; ++j)
                mma_f16(sum[h][j], a0, a1, a2, a3, f == 0 ? lo[i][j].x : f == 1 ? lo[i][j].z : f == 2 ? hi[i][j].x : hi[i][j].z,
                        f == 0 ? lo[i][j].y : f == 1 ? lo[i][j].w : f == 2 ? hi[i][j].y : hi[i][j].w);
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float f0 = ue8m0_value(sc[2 * h]), f1 = ue8m0_value(sc[2 * h + 1]);
#pragma unroll
          for (int j = 0; j < G; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[h][j][i] = fmaf(sum[h][j][i] * token[j][i & 1], i < 2 ? f0 : f1, acc[h][j][i]);
        }
      } else {
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
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.empty[position.s]);
    position.advance();
    if (kFp8) {   // the next stage's scales
      const int next = (c + 1) * kParts + warp;
      if (next * kFp8Block < p.K) {
#pragma unroll
        for (int q = 0; q < 4; ++q) sc[q] = __ldg(scale[q] + next);
      }
    }
  }
  if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.red_empty[unit & 1], ((unit >> 1) & 1) ^ 1));
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < G; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[(j * 8 + 2 * t + (i & 1)) * kRedPitch + h * 16 + (i >> 1) * 8 + g] = acc[h][j][i];
  __syncwarp();
  if (lane == 0) mbar_arrive(&sh.red_full[unit & 1]);
}

template <bool kFp8, bool kIn, int kAct>
__global__ void __launch_bounds__(few_threads(kFp8), 1) k_few(const __grid_constant__ FewParams p) {
  constexpr int kOne = kFp8 ? 1 : 2;                 // bytes of a weight
  constexpr int kChunk = kPiece / kOne;              // inner elements of a stage
  constexpr int kPass = pass_of(kFp8), kTokenWarps = token_warps_of(kFp8), kTokenBytes = token_bytes(kFp8), kTokenPitch = token_pitch(kFp8);
  extern __shared__ __align__(1024) uint8_t raw[];
  FewShared& sh = *reinterpret_cast<FewShared*>(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxFewStages; ++s) {
      mbar_init(&sh.full[s], kFp8 ? 1 + kTokenWarps : 1);
      mbar_init(&sh.empty[s], kParts);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.red_full[b], kParts);
      mbar_init(&sh.red_empty[b], kAdders);
    }
    fence_barrier_init();
  }
  if (kIn) {
    pdl_wait();   // ids and tokens may come from the kernel before
    pdl_launch_dependents();
  }
  uint8_t* const red_base = raw + (sizeof(FewShared) + 127) / 128 * 128;
  few_lists<few_threads(kFp8)>(p, sh.lists, reinterpret_cast<uint32_t*>(red_base), kIn && blockIdx.x == 0);
  const FewLists& l = sh.lists;
  const int tokens_most = min(l.most, kPass);
  const int red_part = (tokens_most + 7) / 8 * 8 * kRedPitch;         // floats of one part's sums
  const int red_bytes = kParts * red_part * 4;                        // of one unit; the next one's go to a second part
  const int stage_bytes = kUnitRows * kPiece + (tokens_most * kTokenPitch + 127) / 128 * 128;
  uint8_t* const ring = red_base + 2 * red_bytes;
  // products read 8 tokens' rows, there or not: seven may lie behind the last stage
  const int stages = min(kMaxFewStages, (int)((kFewSmem - (int)(ring - raw) - 7 * kTokenPitch) / stage_bytes));
  const int chunks = (p.K + kChunk - 1) / kChunk;
  FewWalk<kIn, kPass> w(l, p.N);
  bool ok = true;
  RingPosition position = {0, 0, stages, stage_bytes};

  if (warp < kParts) {
    // ---------------------------------------------------------------- products
    uint32_t unit = 0;
    while (w.next()) {
      float* const red = reinterpret_cast<float*>(red_base + (unit & 1) * red_bytes) + warp * red_part;
      if (w.m <= 8)
        few_products<kFp8, kIn, 1>(p, sh, w.e, w.col, ring, red, chunks, unit, position, ok);
      else if (w.m <= 16)
        few_products<kFp8, kIn, 2>(p, sh, w.e, w.col, ring, red, chunks, unit, position, ok);
      else
        few_products<kFp8, kIn, kPass / 8>(p, sh, w.e, w.col, ring, red, chunks, unit, position, ok);
      ++unit;
    }
  } else if (warp < kParts + kAdders) {
    // ---------------------------------------------------------------- sums
    const int q = warp - kParts;
    uint32_t unit = 0;
    if (!kIn)
      for (int n = q; n < p.T; n += kAdders) sh.sums[n * kUnitRows + lane] = 0.0f;
    while (w.next()) {
      const int b = unit & 1;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.red_full[b], (unit >> 1) & 1, 2 * kWaitNs));
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
          if (c < w.cols)   // rounded to bf16: the second kernel's operand
            p.out[(int64_t)l.slot[w.s0 + n] * p.N + w.col + c] = __float2bfloat16_rn(act_value<kAct>(total(n, row)) * total(n, row + 8));
      } else {
        // a token is one warp's, so its slots are added in the lists' order
        for (int n = 0; n < w.m; ++n) {
          const int token = l.token[w.s0 + n];
          if (token % kAdders == q) {
            float* const sum = sh.sums + token * kUnitRows + lane;
            *sum = fmaf(l.weight[w.s0 + n], total(n, lane), *sum);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.red_empty[b]);
      ++unit;
      if (!kIn && w.last) {
        for (int n = q; n < p.T; n += kAdders) {
          if (lane < w.cols) p.out[(int64_t)n * p.N + w.col + lane] = __float2bfloat16_rn(sh.sums[n * kUnitRows + lane]);
          sh.sums[n * kUnitRows + lane] = 0.0f;
        }
      }
    }
    if (!kIn && l.n_used == 0) {
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
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.empty[position.s], position.phase ^ 1));
        if (!ok) break;
        if (issue) {
          const int k = min(kChunk, p.K - c * kChunk);
          mbar_arrive_expect_tx(&sh.full[position.s], (kIn ? 2 : 1) * w.cols * kPiece + (kFp8 ? 0 : w.m * k * 2));
          const uint32_t bar = smem_addr(&sh.full[position.s]);
          constexpr int kWhole = kIn ? kUnitRows / 2 : kUnitRows;
          for (int half = 0; half < (kIn ? 2 : 1); ++half) {
            const uint32_t to = smem_addr(ring + position.offset()) + half * kWhole * kPiece;
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
    if constexpr (kFp8) {
      // a token a warp at a time, the next one's loads before this one is turned into fp16
      FewWalk<kIn, kPass> ahead = w;
      int ahead_c = 0, ahead_i = turn;
      bool go = ahead.next();
      uint4 next[4];
      auto load = [&]() {   // the first token from here on that is this warp's
        while (go && ahead_i >= ahead.m) {
          ahead_i = turn;
          if (++ahead_c == chunks) {
            ahead_c = 0;
            go = ahead.next();
          }
        }
        if (!go || ahead_c * kChunk + lane * 32 >= p.K) return;
        const int from = kIn ? l.token[ahead.s0 + ahead_i] : l.slot[ahead.s0 + ahead_i];
        const __nv_bfloat16* row = p.v + (int64_t)from * p.K + ahead_c * kChunk + lane * 32;
#pragma unroll
        for (int q = 0; q < 4; ++q) next[q] = ld_v4(row + 8 * q);
      };
      load();
      while (ok && w.next()) {
        for (int c = 0; c < chunks; ++c) {
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.empty[position.s], position.phase ^ 1));
          if (!ok) break;
          uint8_t* const tokens = ring + position.offset() + kUnitRows * kPiece;
          for (int i = turn; i < w.m; i += kTokenWarps) {
            const bool in = c * kChunk + lane * 32 < p.K;
            uint4 v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = in ? next[q] : make_uint4(0, 0, 0, 0);
            ahead_i += kTokenWarps;
            load();
            uint8_t* const to = tokens + i * kTokenPitch;
            scaled_f16(v, to + lane * 64, reinterpret_cast<float*>(to + kTokenBytes) + (lane >> 2), (lane & 3) == 0);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.full[position.s]);
          position.advance();
        }
      }
    } else {
      while (ok && w.next()) {   // a row a lane
        const int mine = lane * kTokenWarps + turn;
        const int from = mine < w.m ? (kIn ? l.token[w.s0 + mine] : l.slot[w.s0 + mine]) : -1;
        const __nv_bfloat16* row = p.v + (int64_t)from * p.K;
        for (int c = 0; c < chunks; ++c) {
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.empty[position.s], position.phase ^ 1));
          if (!ok) break;
          if (from >= 0)
            tma_load_1d(ring + position.offset() + kUnitRows * kPiece + mine * kTokenPitch, row + c * kChunk, min(kChunk, p.K - c * kChunk) * 2, &sh.full[position.s]);
          __syncwarp();
          position.advance();
        }
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

template <bool kFp8, bool kIn, int kAct>
static int launch_few_half(const FewParams& p, cudaStream_t s) {
  auto* fn = k_few<kFp8, kIn, kAct>;
  if (ep_host::ensure_max_smem(reinterpret_cast<const void*>(fn), kFewSmem) != EP_OK) return EP_ERR_CUDA;
  const int grid = ep_host::grid_cap(1);
  if (!kIn && ep_host::sm_budget_set()) {   // the second kernel's CTAs do not come up beside the first's
    fn<<<grid, few_threads(kFp8), kFewSmem, s>>>(p);
  } else if (ep_host::launch_dependent<FewParams>(fn, grid, few_threads(kFp8), kFewSmem, s, p) != EP_OK) {
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
