// newton.cu -- orthogonalised update of the experts' weights: momentum, norm,
// Newton-Schulz products, weight update.
//
// Every matrix X [M, N] of a stack goes through steps X <- a X + (b A + c A^2) X
// with A = X X^T (S x S, S the smaller side; X^T X and a product from the right
// where M > N, so that nothing is transposed: an operand that lies the other way
// is read MN-major).  A step is three launches over all matrices:
//   kGram    A = X X^T                 symmetric: tiles on and above the diagonal,
//   kSquare  P = b A + c A^2           the others mirrored (none where c = 0)
//   kApply   X' = a X + P X
// all bound by the tensor cores.  Pairs of SMs compute 256 x 256 tiles as the
// experts' products do (tcgen05.mma.cta_group::2, TMA, sums in tensor memory, the
// epilogue of one tile under the products of the next).
//
// Operands are fp16: X and P stay near 1 in size by construction, so fp16's range
// is enough (they are held 2^8 times as large, which keeps what matters of them above its
// subnormals) and its 11 bits are worth having: bf16's 8 would put the rounding of
// the operands above that of a bf16 result.  a X is the term that lifts small singular values,
// by 3.4 a step; rounding it would lift the rounding too, so X is carried as
// hi + lo, two fp16 words, of which the products take hi alone.
// P's diagonal is kept out of the product: in 32 bits it multiplies both words of X.
// Where singular values are near 1, P is near -2.7 I and all but the diagonal is
// small, and so is what rounding P and leaving out lo costs (256 x 512 normal numbers, five quintic
// steps: 1.7e-3 of the result off without this, 0.8e-3 so).
// The first X is the source times a power of two, exact for a bf16 gradient; the
// rest of the norm, a factor f in (1/2, 1], goes into the first step's epilogues.

#include <cmath>

#include "newton.cuh"

namespace ep {

// ---------------------------------------------------------------- momentum and norm

constexpr int kSourceThreads = 256;
constexpr int kAhead = 4;                 // loads on their way, of 8 elements a thread
// Parts of a matrix's norm, whatever the stack: a matrix comes out as it does alone.
constexpr int kMostParts = 256;

// m <- momentum m + g and the squares' sums of u, a part of a matrix a CTA, in an
// order that only the sizes give.  Memory bounds it: 8 of 4096 x 1416 with momentum at 6.7
// TB/s; 186 MB of bf16 without at 5.2, where one kernel for all types, with the registers of the largest,
// got through 3.4 (k_newton_scale below: 371 MB in 56 us instead of 108).
template <bool kF32, bool kMomentum>
__global__ void __launch_bounds__(kSourceThreads) k_newton_norm(Source s) {
  __shared__ float warps[kSourceThreads / kWarp];
  pdl_wait();
  if (s.early) pdl_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *s.failed = 0;
  for (int64_t item = blockIdx.x; item < (int64_t)s.count * s.parts; item += gridDim.x) {
    const int64_t z = item / s.parts, begin = (item - z * s.parts) * s.part, end = min(begin + s.part, s.each), base = z * s.each;
    float sum[kAhead] = {};
    for (int64_t i0 = begin + threadIdx.x * 8; i0 < end; i0 += kAhead * kSourceThreads * 8) {
      SourceWords g[kAhead] = {}, m[kAhead] = {};
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int64_t i = i0 + k * kSourceThreads * 8;
        if (i >= end) continue;
        g[k] = load_words(s.g, kF32, base + i);
        if (kMomentum) m[k] = load_words(s.m, true, base + i);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int64_t i = i0 + k * kSourceThreads * 8;
        float u[8];
        words_to_floats(g[k], kF32, u);
        if (kMomentum) {
          float v[8];
          words_to_floats(m[k], true, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[e] = fmaf(s.momentum, v[e], u[e]);
            u[e] = s.nesterov ? fmaf(s.momentum, v[e], u[e]) : v[e];
          }
          if (i < end) {
            float4* p = reinterpret_cast<float4*>(s.m + base + i);
            p[0] = make_float4(v[0], v[1], v[2], v[3]);
            p[1] = make_float4(v[4], v[5], v[6], v[7]);
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[k] = fmaf(u[e], u[e], sum[k]);
      }
    }
    float all = (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = all;
    __syncthreads();
    if (threadIdx.x == 0) {
      all = 0.0f;
      for (int w = 0; w < kSourceThreads / kWarp; ++w) all += warps[w];
      s.sums[item] = all;
    }
    __syncthreads();
  }
}

// X = u 2^q, in hi and lo, and the factor that makes it 2^8 u / (|u| + eps).  The
// parts in the other order, as the last ones of the kernel before are still in L2.  m is read past the first-level
// cache, which may hold what it was.
template <bool kF32, bool kMomentum>
__global__ void __launch_bounds__(kSourceThreads) k_newton_scale(Source s) {
  if (s.early) pdl_launch_dependents();
  pdl_wait();
  const int64_t items = (int64_t)s.count * s.parts;
  for (int64_t at = blockIdx.x; at < items; at += gridDim.x) {
    const int64_t item = items - 1 - at;
    const int64_t z = item / s.parts, begin = (item - z * s.parts) * s.part, end = min(begin + s.part, s.each), base = z * s.each;
    float square = 0.0f;   // a warp for itself
#pragma unroll 4
    for (int k = threadIdx.x & 31; k < s.parts; k += kWarp) square += __ldcg(s.sums + z * s.parts + k);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) square += __shfl_xor_sync(0xffffffffu, square, o);
    float up, factor;
    source_scale(square, s.eps, up, factor);
    if (begin == 0 && threadIdx.x == 0) s.factor[z] = factor;
    const int rows_on = kSourceThreads * 8 / s.cols, cols_on = kSourceThreads * 8 % s.cols;
    int64_t row = (begin + threadIdx.x * 8) / s.cols;
    int col = (int)(begin + threadIdx.x * 8 - row * s.cols);
    row += z * s.rows;
    const bool reads_g = !kMomentum || s.nesterov;
    for (int64_t i0 = begin + threadIdx.x * 8; i0 < end; i0 += kAhead * kSourceThreads * 8) {
      SourceWords g[kAhead] = {}, m[kAhead] = {};
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int64_t i = i0 + k * kSourceThreads * 8;
        if (i >= end) continue;
        if (reads_g) g[k] = load_words(s.g, kF32, base + i);
        if (kMomentum) m[k] = load_words(s.m, true, base + i);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int64_t to = row * s.stride + col;
        row += rows_on;
        col += cols_on;
        if (col >= s.cols) {
          col -= s.cols;
          ++row;
        }
        if (i0 + k * kSourceThreads * 8 >= end) continue;
        float u[8];
        words_to_floats(g[k], kF32, u);
        if (kMomentum) {
          float v[8];
          words_to_floats(m[k], true, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] = s.nesterov ? fmaf(s.momentum, v[e], u[e]) : v[e];
        }
        uint32_t h[4], l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split_f16(u[2 * e] * up, u[2 * e + 1] * up, h[e], l[e]);
        st_v4(s.hi + to, make_uint4(h[0], h[1], h[2], h[3]));
        if (s.lo != nullptr) st_v4(s.lo + to, make_uint4(l[0], l[1], l[2], l[3]));
      }
    }
  }
}

// ---------------------------------------------------------------- products

constexpr int kNewtonThreads = 384;
constexpr int kNewtonStages = 5;                      // of a whole tile's operands; more of a narrow one's
constexpr int kMostNewtonStages = 6;
constexpr int kBlock = 256;                           // output rows of a pair's tile, and its columns at most
constexpr int kInner = 64;                            // fp16 elements of one 128-byte row
constexpr int kNewtonOperand = 128 * kInner * 2;      // 16 KB: one CTA's part of an operand
constexpr int kNewtonStage = 2 * kNewtonOperand;
constexpr int kNewtonWarps = 8;                       // of the epilogue: four for the rows, two sides of column chunks
constexpr int kChunkCols = 32;                        // columns that a warp takes at a time, of its 32 rows
constexpr int kPiece = 32 * kChunkCols * 2;           // 2 KB: such a block of 16-bit numbers
constexpr int kWarpBytes = 4 * kPiece;                // a warp's buffers: two of hi and lo, or one and one of w

enum NewtonForm { kGram, kSquare, kApply, kApplyOut, kApplyWeights };
__host__ __device__ constexpr bool reads_tile(int form) { return form != kGram; }
__host__ __device__ constexpr bool symmetric(int form) { return form == kGram || form == kSquare; }

struct NewtonParams {
  CUtensorMap a, b;             // operands
  const __half *in, *in_lo;     // what the epilogue adds: A, or X (in_lo may be nullptr)
  int in_stride;
  CUtensorMap out, out_lo;      // (not kApplyWeights)
  int count, rows, cols, inner; // of a product
  int wide;                     // columns of a tile: 256 or 128
  uint32_t stages, stage_bytes;
  uint32_t tiles_m, tiles_n;    // kSquare, kGram: tiles_m only
  uint32_t each, tiles;         // of a matrix, of all
  uint32_t whole;               // tiles before those that are halved
  bool rows_fast;
  bool backward;                // the last matrix first
  bool a_mn, b_mn;
  bool early;                   // as Source's
  float scale, add;             // epilogue: scale * sums + (add + diagonal_scale * diagonal) * in
  float diagonal_scale;
  const float* factor;          // [count] or nullptr
  float* diagonal;              // [count, S]: P's
  float keep, step;             // kApplyWeights
  float* w;
  __nv_bfloat16* w16;
  int32_t* status;
  int32_t* failed;              // as Source's
};

struct NewtonShared {
  uint64_t full[kMostNewtonStages], empty[kMostNewtonStages];
  uint64_t sums_full[2], sums_empty[2];
  float columns[kNewtonWarps][2][kChunkCols];   // P's diagonal for the columns of a buffer
  uint32_t tmem;
};

struct NewtonTile {
  int z, i0, j0;
  int wide;                     // columns of its products: fewer at the matrix's edge
  bool mirror;
};

template <int kForm>
__device__ __forceinline__ NewtonTile newton_tile(const NewtonParams& p, uint32_t t) {
  NewtonTile out;
  const bool halved = t >= p.whole;
  const uint32_t side = halved ? (t - p.whole) & 1 : 0;
  if (halved) t = p.whole + ((t - p.whole) >> 1);
  const uint32_t z = t / p.each, u = t - z * p.each;
  out.z = p.backward ? p.count - 1 - (int)z : (int)z;
  if (symmetric(kForm)) {
    const uint32_t f = kBlock / p.wide, b = f == 1 ? u : u >> 1;
    uint32_t r = (uint32_t)((sqrtf(8.0f * (float)b + 1.0f) - 1.0f) * 0.5f);
    while ((r + 1) * (r + 2) / 2 <= b) ++r;   // each is below 2^25
    while (r * (r + 1) / 2 > b) --r;
    const uint32_t c = b - r * (r + 1) / 2;
    out.i0 = (int)c * kBlock;
    out.j0 = (int)(r * kBlock + (u - b * f) * p.wide);
    out.mirror = c < r;
  } else {
    const uint32_t fast = p.rows_fast ? p.tiles_m : p.tiles_n, slow = u / fast, rest = u - slow * fast;
    out.i0 = (int)(p.rows_fast ? rest : slow) * kBlock;
    out.j0 = (int)(p.rows_fast ? slow : rest) * p.wide;
    out.mirror = false;
  }
  const int wide = halved ? p.wide / 2 : p.wide;
  out.j0 += (int)side * wide;
  // (an MN-major operand comes 64 columns at a time)
  out.wide = p.b_mn ? wide : min(wide, (p.cols - out.j0 + 31) / 32 * 32);
  return out;
}

// Address of 8 columns (16 bytes) of a row in a piece, 64-byte swizzle.
__device__ __forceinline__ uint32_t piece_address(uint32_t piece, int row, int c) { return piece + row * 64 + ((c ^ ((row >> 1) & 3)) << 4); }

__device__ __forceinline__ void stmatrix4(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// 16 (4) bytes to shared memory when they come; zeros where there is nothing to read.
__device__ __forceinline__ void copy_async16(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_async4(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int kForm>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kNewtonThreads, 1) k_newton(const __grid_constant__ NewtonParams p) {
  extern __shared__ __align__(1024) uint8_t stages[];
  uint8_t* pieces = stages + kNewtonStages * kNewtonStage;   // narrow tiles' stages take no more
  NewtonShared& sh = *reinterpret_cast<NewtonShared*>(pieces + kNewtonWarps * kWarpBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    prefetch_map(&p.a);
    prefetch_map(&p.b);
    for (int s = 0; s < kMostNewtonStages; ++s) {
      mbar_init(&sh.full[s], 1);      // the first CTA's, with the bytes of both
      mbar_init(&sh.empty[s], 1);     // the products' commit
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.sums_full[i], 1);
      mbar_init(&sh.sums_empty[i], 2 * kNewtonWarps);
    }
    fence_barrier_init();
  }
  if (warp == 2) tmem_alloc<2>(&sh.tmem, 512);
  tmem_fence_before();
  __syncwarp();
  cluster_sync();
  tmem_fence_after();
  const uint32_t tmem = sh.tmem;
  bool ok = true;
  const int blocks = (p.inner + kInner - 1) / kInner;
  // a symmetric form's last column tile may lie past the matrix
  auto next = [&](uint32_t& t, NewtonTile& tile) {
    for (; t < p.tiles; t += pairs) {
      tile = newton_tile<kForm>(p, t);
      if (tile.j0 < p.cols) return true;
    }
    return false;
  };
  uint32_t t = pair;
  NewtonTile tile;
  bool more = next(t, tile);
  auto step = [&]() {
    t += pairs;
    more = next(t, tile);
  };
  if (p.early) pdl_launch_dependents();
  pdl_wait();
  if (kForm == kApplyWeights && __ldcg(p.failed) != 0) more = false;   // (no launch of this form sets it)
  if (warp == 0 || warp == 3) {
    // ---------------------------------------------------------------- copies, a warp an operand
    const bool issue = elect_one(), first = warp == 0;
    const bool mn = first ? p.a_mn : p.b_mn;
    const int half = p.wide / 2;   // of the second operand in a CTA
    const uint32_t both = 2 * (kNewtonOperand + half * kInner * 2);
    const CUtensorMap* map = first ? &p.a : &p.b;
    const uint32_t to0 = smem_addr(stages) + (first ? 0 : kNewtonOperand), full0 = map_to_rank(smem_addr(&sh.full[0]), 0);
    uint32_t s = 0, phase = 0;
    for (; ok && more; step()) {
      const int m0 = first ? tile.i0 + (int)rank * 128 : tile.j0 + (int)rank * (tile.wide / 2);
      for (int kb = 0; kb < blocks; ++kb) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.empty[s], phase ^ 1));
        if (!ok) break;
        if (issue) {
          const uint32_t to = to0 + s * p.stage_bytes, bar = full0 + s * (uint32_t)sizeof(uint64_t);
          if (first && rank == 0) mbar_arrive_expect_tx(&sh.full[s], both);
          if (!mn) {
            tma_load_3d<true>(to, map, bar, kb * kInner, m0, tile.z);
          } else {
            for (int i = 0; i < (first ? 2 : half / 64); ++i) tma_load_3d<true>(to + i * (kNewtonOperand / 2), map, bar, m0 + i * 64, kb * kInner, tile.z);
          }
        }
        if (++s == p.stages) {
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
  } else if (warp == 1 && rank == 0) {
    // ---------------------------------------------------------------- products
    const bool issue = elect_one();
    const uint32_t a0 = umma_desc_lo(smem_addr(stages), p.a_mn ? kNewtonOperand / 2 : 16);
    const uint32_t b0 = umma_desc_lo(smem_addr(stages) + kNewtonOperand, p.b_mn ? kNewtonOperand / 2 : 16);
    const uint32_t step_a = (p.a_mn ? 2048 : 32) >> 4, step_b = (p.b_mn ? 2048 : 32) >> 4;
    uint32_t s = 0, phase = 0, n = 0;
    while (ok && more) {
      const uint32_t idesc = umma_idesc_f16(kBlock, tile.wide, p.a_mn, p.b_mn);
      step();   // looked up while this tile's products run
      const uint32_t half = n & 1, d = tmem + half * kBlock;
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.sums_empty[half], ((n >> 1) & 1) ^ 1, 4 * kWaitNs));
      if (!ok) break;
      tmem_fence_after();
      for (int kb = 0; kb < blocks; ++kb) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.full[s], phase));
        if (!ok) break;
        tmem_fence_after();
        if (issue) {
          const uint32_t a = a0 + s * (p.stage_bytes >> 4), b = b0 + s * (p.stage_bytes >> 4);
#pragma unroll
          for (uint32_t i = 0; i < kInner / 16; ++i) umma_bf16_pair(d, a + i * step_a, b + i * step_b, idesc, kb > 0 || i > 0);
          umma_commit_pair(&sh.empty[s]);
        }
        if (++s == p.stages) {
          s = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
      if (issue) umma_commit_pair(&sh.sums_full[half]);
      ++n;
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- epilogue
    // A warp takes its 32 rows, 32 columns at a time, on its own.  What is added is copied into a buffer (cp.async:
    // whole 64-byte rows side by side) while the last chunk leaves the other, read from it a row a thread, replaced
    // there by the result, which leaves by TMA.  (Copied in by TMA, it stood behind the operands in the copy engine's
    // queue, 2000 to 5000 clocks; loaded a chunk ahead into registers, a chunk's arithmetic took 2500 clocks instead
    // of 900, waiting for those loads with its own.)
    const int q = warp & 3, side = (warp - 4) >> 2;
    constexpr int kBuffers = kForm == kApplyWeights ? 1 : 2;
    constexpr bool kAheadOfChunk = reads_tile(kForm) && kBuffers == 2;
    const uint32_t buffers = smem_addr(pieces) + (warp - 4) * kWarpBytes, at_w = buffers + 2 * kPiece;
    const uint32_t columns = smem_addr(&sh.columns[warp - 4][0][0]);
    const int row0 = (int)rank * 128 + q * 32;
    const bool lo = kForm != kSquare && p.in_lo != nullptr, by_column = kForm != kSquare && !p.rows_fast;
    auto live = [&](const NewtonTile& x, int ch) { return ch < x.wide / kChunkCols && x.j0 + ch * kChunkCols < p.cols && x.i0 + row0 < p.rows; };
    // the chunk that is copied next: (t_ahead, ch_ahead), number k_ahead
    uint32_t t_ahead = t, k_ahead = 0;
    int ch_ahead = side;
    NewtonTile ahead = tile;
    bool more_ahead = more;
    auto seek = [&]() {
      while (more_ahead && !live(ahead, ch_ahead)) {
        t_ahead += pairs;
        ch_ahead = side;
        more_ahead = next(t_ahead, ahead);
      }
    };
    auto fetch = [&]() {
      seek();
      if (more_ahead) {
        const uint32_t to = buffers + k_ahead % kBuffers * 2 * kPiece;
        const int col0 = ahead.j0 + ch_ahead * kChunkCols, c = lane & 3;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i * 8 + (lane >> 2);
          const bool in = ahead.i0 + row0 + r < p.rows && col0 + c * 8 < p.cols;
          const int64_t at = in ? ((int64_t)ahead.z * p.rows + ahead.i0 + row0 + r) * p.in_stride + col0 + c * 8 : 0;
          copy_async16(piece_address(to, r, c), p.in + at, in);
          if (kForm != kSquare) copy_async16(piece_address(to + kPiece, r, c), lo ? p.in_lo + at : p.in, in && lo);
        }
        if (by_column) {
          const bool in = col0 + lane < p.cols;
          copy_async4(columns + k_ahead % 2 * (kChunkCols * 4) + lane * 4, p.diagonal + (in ? (int64_t)ahead.z * p.cols + col0 + lane : 0), in);
        }
        if (kForm == kApplyWeights) {   // 8 pieces of 4 a row, 128-byte swizzle
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3), e = lane & 7;
            const bool in = ahead.i0 + row0 + r < p.rows && col0 + e * 4 < p.cols;
            copy_async16(at_w + r * 128 + ((e ^ (r & 7)) << 4), p.w + (in ? ((int64_t)ahead.z * p.rows + ahead.i0 + row0 + r) * p.cols + col0 + e * 4 : 0), in);
          }
        }
        ch_ahead += 2;
        ++k_ahead;
      }
      copy_async_commit();
    };
    if (reads_tile(kForm)) fetch();
    if (kAheadOfChunk) fetch();
    uint32_t n = 0, k = 0;   // tiles, chunks
    for (; more; step(), ++n) {
      const uint32_t half = n & 1;
      const float f = p.factor != nullptr ? __ldcg(p.factor + tile.z) : 1.0f;
      const float scale = kForm == kGram ? p.scale * f * f : p.scale;
      const int row = tile.i0 + row0 + lane;
      const bool there = row < p.rows;
      const int64_t line = (int64_t)tile.z * p.rows + row;
      const float row_add =
          reads_tile(kForm) && kForm != kSquare && p.rows_fast && there ? fmaf(__ldcg(p.diagonal + line), p.diagonal_scale, p.add) : p.add;
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.sums_full[half], (n >> 1) & 1, kWaitNs + (uint64_t)blocks * 4000));
      if (!ok) break;
      tmem_fence_after();
      const uint32_t d = tmem + half * kBlock + ((uint32_t)(q * 32) << 16);
#pragma unroll 1
      for (int ch = side; live(tile, ch); ch += 2, ++k) {
        const uint32_t at = buffers + k % kBuffers * 2 * kPiece, at_lo = at + kPiece;
        const int col0 = tile.j0 + ch * kChunkCols;
        if (reads_tile(kForm)) copy_async_wait<0>();
        __syncwarp();
        float v[32];
        tmem_ld32(d + ch * kChunkCols, v);
        if (kAheadOfChunk && k > 0) {   // the next chunk's, into the other buffer, once the last one's copy has left it
          if (lane == 0) tma_wait_read<0>();
          __syncwarp();
          fetch();
        }
        tmem_wait_ld(v);
#pragma unroll
        for (int c = 0; c < 4; ++c) {   // 8 columns
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = v[c * 8 + e] * scale;
          if (reads_tile(kForm)) {
            const uint4 hi = ld_shared_v4_at(piece_address(at, lane, c));
            uint4 low = make_uint4(0, 0, 0, 0);
            if (kForm != kSquare) low = ld_shared_v4_at(piece_address(at_lo, lane, c));
            const uint32_t wh[4] = {hi.x, hi.y, hi.z, hi.w}, wl[4] = {low.x, low.y, low.z, low.w};
            float add[8];   // a, and P's diagonal for the row, or for the column where P stands to the right
#pragma unroll
            for (int e = 0; e < 8; ++e) add[e] = row_add;
            if (by_column) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint4 y = ld_shared_v4_at(columns + k % 2 * (kChunkCols * 4) + (c * 2 + e) * 16);
                add[4 * e] = fmaf(__uint_as_float(y.x), p.diagonal_scale, row_add), add[4 * e + 1] = fmaf(__uint_as_float(y.y), p.diagonal_scale, row_add);
                add[4 * e + 2] = fmaf(__uint_as_float(y.z), p.diagonal_scale, row_add), add[4 * e + 3] = fmaf(__uint_as_float(y.w), p.diagonal_scale, row_add);
              }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float2 y = floats_of(wh[e]);
              if (kForm != kSquare) {
                const float2 l = floats_of(wl[e]);
                y.x += l.x;
                y.y += l.y;
              }
              x[2 * e] = fmaf(add[2 * e], y.x, x[2 * e]);
              x[2 * e + 1] = fmaf(add[2 * e + 1], y.y, x[2 * e + 1]);
              if (kForm != kSquare) {
                x[2 * e] *= f;
                x[2 * e + 1] *= f;
              }
            }
          }
          if (symmetric(kForm) && p.diagonal != nullptr && !tile.mirror) {
            const int at_diagonal = row - (col0 + c * 8);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if (at_diagonal == e) {
                if (there) p.diagonal[line] = x[e] * (1.0f / kHeld);
                x[e] = 0.0f;
              }
            }
          }
          uint32_t h[4], l[4];
          if (kForm == kApplyWeights) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {   // a row of w is 8 pieces of 4, 128-byte swizzle
              const uint32_t to = at_w + lane * 128 + (((2 * c + e) ^ (lane & 7)) << 4);
              const uint4 w = ld_shared_v4_at(to);
              const float w0 = fmaf(-p.step, x[4 * e], p.keep * __uint_as_float(w.x)), w1 = fmaf(-p.step, x[4 * e + 1], p.keep * __uint_as_float(w.y));
              const float w2 = fmaf(-p.step, x[4 * e + 2], p.keep * __uint_as_float(w.z)), w3 = fmaf(-p.step, x[4 * e + 3], p.keep * __uint_as_float(w.w));
              st_shared_v4_at(to, make_uint4(__float_as_uint(w0), __float_as_uint(w1), __float_as_uint(w2), __float_as_uint(w3)));
              h[2 * e] = pack_bf16x2(w0, w1);
              h[2 * e + 1] = pack_bf16x2(w2, w3);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (kForm == kApplyOut) {
                h[e] = pack_bf16x2(x[2 * e], x[2 * e + 1]);
              } else {
                split_f16(x[2 * e], x[2 * e + 1], h[e], l[e]);   // l: kApply
              }
            }
          }
          st_shared_v4_at(piece_address(at, lane, c), make_uint4(h[0], h[1], h[2], h[3]));
          if (kForm == kApply) st_shared_v4_at(piece_address(at_lo, lane, c), make_uint4(l[0], l[1], l[2], l[3]));
        }
        if (symmetric(kForm) && tile.mirror) {   // the block turned around: rows j, columns i
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t x[4];
            ldmatrix4_trans(piece_address(at, lane, j), x);
            stmatrix4(piece_address(at_lo, j * 8 + (lane & 7), lane >> 3), x);
          }
        }
        if (kForm == kApplyWeights) {   // by whole rows, so that the buffers are free at once
          __syncwarp();
          const int64_t base = ((int64_t)tile.z * p.rows + tile.i0 + row0) * p.cols + col0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3), c = lane & 7;
            if (tile.i0 + row0 + r < p.rows && col0 + c * 4 < p.cols)
              st_v4(p.w + base + (int64_t)r * p.cols + c * 4, ld_shared_v4_at(at_w + r * 128 + ((c ^ (r & 7)) << 4)));
          }
          if (p.w16 != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = i * 8 + (lane >> 2), c = lane & 3;
              if (tile.i0 + row0 + r < p.rows && col0 + c * 8 < p.cols)
                st_v4(p.w16 + base + (int64_t)r * p.cols + c * 8, ld_shared_v4_at(piece_address(at, r, c)));
            }
          }
          __syncwarp();
        } else {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (!kAheadOfChunk) tma_wait_read<0>();   // the last chunk's copy, out of the other buffer
            tma_store_3d(&p.out, at, col0, tile.i0 + row0, tile.z);
            if (kForm == kApply) tma_store_3d(&p.out_lo, at_lo, col0, tile.i0 + row0, tile.z);
            if (symmetric(kForm) && tile.mirror) tma_store_3d(&p.out, at_lo, tile.i0 + row0, col0, tile.z);
            tma_commit();
          }
          __syncwarp();
        }
        if (kForm == kApplyWeights) fetch();
      }
      tmem_fence_before();   // the next tile's products may have this half
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(map_to_rank(smem_addr(&sh.sums_empty[half]), 0));
    }
    copy_async_wait<0>();
    if (lane == 0) tma_wait_all();
  }
  if (!ok) {
    set_status(p.status, EP_ERR_TIMEOUT);
    if (kForm != kApplyWeights) *p.failed = 1;
  }
  __syncwarp();
  tmem_fence_before();
  cluster_sync();
  tmem_fence_after();
  if (warp == 2) tmem_free<2>(tmem, 512);
}

// ---------------------------------------------------------------- host

struct NewtonSpace {
  float *sums, *factor, *diagonal;
  __half *x[2], *lo[2], *A, *P;
  int32_t* failed;
  size_t bytes;
};

// Row stride of A and P, and of X where it adds no more than an eighth: whole 128-byte lines, which a copied row of 64
// elements then is one of (A and P, S = 1416, without: 870 clocks a stage instead of 610).  X without and with it, five quintic
// steps: 8 of 4096 x 1416 1247 us, 1057; 8 of 2048 x 2056 1214, 1070; 16 of 2048 x 520 500, 470; 16 of 520 x 584 266.5, 266.
// Narrower ones gain too (16 of 1024 x 504 273, 258; 32 of 1024 x 264 313, 290) but would need up to 8 times the room.
static int64_t padded(int n) { return (int64_t)(n + 63) / 64 * 64; }
static int64_t padded_x(int N) { return N >= 512 ? padded(N) : N; }

static NewtonSpace newton_space(int count, int M, int N, void* base) {
  NewtonSpace s;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* const p = static_cast<uint8_t*>(base) + at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  const size_t each = (size_t)M * padded_x(N), S = std::min(M, N);
  s.sums = reinterpret_cast<float*>(take((size_t)count * kMostParts * 4));
  s.factor = reinterpret_cast<float*>(take((size_t)count * 4));
  s.diagonal = reinterpret_cast<float*>(take((size_t)count * S * 4));
  for (int i = 0; i < 2; ++i) {
    s.x[i] = reinterpret_cast<__half*>(take(count * each * 2));
    s.lo[i] = reinterpret_cast<__half*>(take(count * each * 2));
  }
  s.A = reinterpret_cast<__half*>(take(count * S * padded((int)S) * 2));
  s.P = reinterpret_cast<__half*>(take(count * S * padded((int)S) * 2));
  s.failed = reinterpret_cast<int32_t*>(take(4));
  s.bytes = at;
  return s;
}

static bool newton_sizes(int count, int M, int N) {
  if (count < 0 || count > 65535 || M <= 0 || N <= 0 || N % 8 != 0 || M > (1 << 20) || N > (1 << 20)) return false;
  const int64_t lim = (int64_t)1 << 31, square = (std::min(M, N) + kBlock - 1) / kBlock;
  const int64_t tiles = (int64_t)((M + kBlock - 1) / kBlock) * ((N + kBlock / 2 - 1) / (kBlock / 2));
  return (int64_t)count * M < lim && count * tiles < lim && count * square * (square + 1) < lim;   // tiles are numbered in 32 bits
}

// Rows of `cols` 16-bit elements at `stride` elements; boxes of 64 columns, or an epilogue's of 32 x 32 (box_rows 0).
static int newton_map(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t count, int64_t stride, int box_rows) {
  const uint64_t dims[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)count}, strides[2] = {(uint64_t)stride * 2, (uint64_t)(stride * rows) * 2};
  const uint32_t box[3] = {box_rows > 0 ? 64u : (uint32_t)kChunkCols, box_rows > 0 ? (uint32_t)box_rows : 32u, 1};
  return ep_host::make_map(m, false, 3, base, dims, strides, box, box_rows == 0);
}

template <int kForm>
static int launch_newton(NewtonParams& p, cudaStream_t s) {
  constexpr int kSmem = kNewtonStages * kNewtonStage + kNewtonWarps * kWarpBytes + (int)sizeof(NewtonShared);
  const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(p.tiles, ep_host::grid_cap(1) / 2));
  if (ep_host::ensure_max_smem(reinterpret_cast<const void*>(k_newton<kForm>), kSmem) != EP_OK) return EP_ERR_CUDA;
  if (ep_host::launch_in_budget(k_newton<kForm>, (int)pairs * 2, kNewtonThreads, kSmem, s, p) != EP_OK) return EP_ERR_CUDA;
  ep_host::count_launch();
  return ep_host::check_launch();
}

// What all steps share, and the launches.
struct Newton {
  int count, M, N, S;
  NewtonSpace space;
  int32_t* status;
  cudaStream_t stream;

  // Tiles of 256 columns, or of 128 where twice as many still come at once (five quintic steps, us with 256 and with 128:
  // 2048 x 1000 187.5, 181; two of them 219.6, 212.4; 1024 x 1024 147.5, 145.3; eight of 512 x 512 132.7, 130; where they come in
  // two waves 20 of 512 x 512 195.7, 204.5; two of 1416 x 1416 244.6, 261.5).
  void tiles(NewtonParams& p, bool sym) const {
    auto of = [&](int wide) {
      p.wide = wide;
      p.tiles_m = (p.rows + kBlock - 1) / kBlock;
      p.tiles_n = (p.cols + wide - 1) / wide;
      p.stage_bytes = kNewtonOperand + wide / 2 * kInner * 2;
      p.stages = std::min<uint32_t>(kMostNewtonStages, kNewtonStages * kNewtonStage / p.stage_bytes);
      const int64_t each = sym ? (int64_t)p.tiles_m * (p.tiles_m + 1) / 2 * (kBlock / wide) : (int64_t)p.tiles_m * p.tiles_n;
      p.each = (uint32_t)each;
      p.tiles = (uint32_t)(each * count);
    };
    of(kBlock);
    // whatever the SM budget: results go by the sizes alone
    const uint32_t pairs = std::max(1, ep_host::num_sms() / 2), left = p.tiles % pairs;
    p.whole = p.tiles;
    if (2 * p.tiles <= pairs) {
      of(kBlock / 2);
      p.whole = p.tiles;
    } else if (2 * left <= pairs) {   // a last wave of halves (16 of 1416 x 4096: X X^T in 94 us instead of 99, its square in 47 instead of 49)
      p.whole -= left;
      p.tiles += left;
    }
  }
  NewtonParams start(int rows, int cols, int inner, bool sym) const {
    NewtonParams p{};
    p.count = count;
    p.rows = rows;
    p.cols = cols;
    p.inner = inner;
    p.status = status;
    p.failed = space.failed;
    p.early = !ep_host::sm_budget_set();
    tiles(p, sym);
    return p;
  }
  int square_map(CUtensorMap* m, const __half* base, int box_rows) const { return newton_map(m, base, S, S, count, padded(S), box_rows); }
  int x_map(CUtensorMap* m, const __half* base, int box_rows) const { return newton_map(m, base, N, M, count, padded_x(N), box_rows); }

  // A = X X^T (or b A where that is the whole polynomial) from x.
  int gram(const __half* x, __half* to, float b, const float* factor) const {
    NewtonParams p = start(S, S, std::max(M, N), true);
    p.a_mn = p.b_mn = M > N;
    p.scale = b / kHeld;
    p.factor = factor;
    p.diagonal = to == space.P ? space.diagonal : nullptr;
    int rc = x_map(&p.a, x, M > N ? 64 : 128);
    if (rc == EP_OK) rc = x_map(&p.b, x, M > N ? 64 : p.wide / 2);
    if (rc == EP_OK) rc = square_map(&p.out, to, 0);
    return rc != EP_OK ? rc : launch_newton<kGram>(p, stream);
  }
  int square(float b, float c) const {
    NewtonParams p = start(S, S, S, true);
    p.scale = c / kHeld;
    p.add = b;
    p.diagonal = space.diagonal;
    int rc = square_map(&p.a, space.A, 128);
    if (rc == EP_OK) rc = square_map(&p.b, space.A, p.wide / 2);
    p.in = space.A;
    p.in_stride = (int)padded(S);
    if (rc == EP_OK) rc = square_map(&p.out, space.P, 0);
    return rc != EP_OK ? rc : launch_newton<kSquare>(p, stream);
  }
  // X' = a X + P X, into buffer `to`; the last one into out or w.
  int apply(int from, bool has_lo, float a, const float* factor, bool last, __nv_bfloat16* out, float* w, __nv_bfloat16* w16, float keep,
            float step) const {
    NewtonParams p = start(M, N, S, false);
    const bool tall = M > N;
    p.rows_fast = !tall;
    p.backward = true;   // what the product before read last is still in L2, and what this one writes last for the next
    p.b_mn = !tall;
    p.in = space.x[from];
    p.in_lo = has_lo ? space.lo[from] : nullptr;
    p.in_stride = (int)padded_x(N);
    p.factor = factor;
    p.scale = (last ? 1.0f / kHeld : 1.0f) / kHeld;
    p.diagonal_scale = last ? 1.0f / kHeld : 1.0f;
    p.add = a * p.diagonal_scale;
    p.diagonal = space.diagonal;
    int rc = tall ? x_map(&p.a, space.x[from], 128) : square_map(&p.a, space.P, 128);
    if (rc == EP_OK) rc = tall ? square_map(&p.b, space.P, p.wide / 2) : x_map(&p.b, space.x[from], 64);
    if (rc != EP_OK) return rc;
    if (!last) {
      rc = x_map(&p.out, space.x[1 - from], 0);
      if (rc == EP_OK) rc = x_map(&p.out_lo, space.lo[1 - from], 0);
      return rc != EP_OK ? rc : launch_newton<kApply>(p, stream);
    }
    if (out != nullptr) {
      rc = newton_map(&p.out, out, N, M, count, N, 0);
      return rc != EP_OK ? rc : launch_newton<kApplyOut>(p, stream);
    }
    p.w = w;
    p.w16 = w16;
    p.keep = keep;
    p.step = step;
    return launch_newton<kApplyWeights>(p, stream);
  }
};

static int newton(Source src, int count, int M, int N, int steps, const float* abc, float eps, __nv_bfloat16* out, float* w,
                  __nv_bfloat16* w16, float keep, float step, void* workspace, int32_t* status, cudaStream_t s) {
  src.eps = eps;
  src.early = !ep_host::sm_budget_set();
  if (std::min(M, N) <= kSmallSide && std::max(M, N) <= kSmallLength) {
    SmallNewton p{};
    p.src = src;
    p.src.count = count;
    p.M = M;
    p.N = N;
    p.steps = steps;
    std::copy(abc, abc + 3 * steps, p.abc);
    p.out = out;
    p.w = w;
    p.w16 = w16;
    p.keep = keep;
    p.step = step;
    p.status = status;
    return launch_newton_small(p, s);
  }
  Newton n = {count, M, N, std::min(M, N), newton_space(count, M, N, workspace), status, s};
  src.each = (int64_t)M * N;
  const int64_t unit = 8 * kSourceThreads;
  src.part = std::max<int64_t>(2 * unit, ((src.each + kMostParts - 1) / kMostParts + unit - 1) / unit * unit);
  src.parts = (int)((src.each + src.part - 1) / src.part);
  src.count = count;
  src.sums = n.space.sums;
  src.factor = n.space.factor;
  src.failed = n.space.failed;
  src.rows = M;
  src.cols = N;
  src.stride = (int)padded_x(N);
  src.hi = n.space.x[0];
  const bool exact = !src.f32 && src.m == nullptr;   // bf16 times a power of two is fp16, but for what is 2^-24 of the norm and smaller
  src.lo = exact ? nullptr : n.space.lo[0];
  const int grid = (int)std::min<int64_t>((int64_t)count * src.parts, ep_host::grid_cap(16));
  auto* norm = src.m != nullptr ? (src.f32 ? k_newton_norm<true, true> : k_newton_norm<false, true>) : src.f32 ? k_newton_norm<true, false> : k_newton_norm<false, false>;
  auto* scale = src.m != nullptr ? (src.f32 ? k_newton_scale<true, true> : k_newton_scale<false, true>) : src.f32 ? k_newton_scale<true, false> : k_newton_scale<false, false>;
  for (auto* kernel : {norm, scale}) {
    if (ep_host::launch_in_budget(kernel, grid, kSourceThreads, 0, s, src) != EP_OK) return EP_ERR_CUDA;
    ep_host::count_launch();
  }
  for (int t = 0; t < steps; ++t) {
    const float a = abc[3 * t], b = abc[3 * t + 1], c = abc[3 * t + 2];
    const float* factor = t == 0 ? n.space.factor : nullptr;
    int rc = n.gram(n.space.x[t & 1], c != 0.0f ? n.space.A : n.space.P, c != 0.0f ? 1.0f : b, factor);
    if (rc == EP_OK && c != 0.0f) rc = n.square(b, c);
    if (rc == EP_OK) rc = n.apply(t & 1, t > 0 || !exact, a, factor, t + 1 == steps, out, w, w16, keep, step);
    if (rc != EP_OK) return rc;
  }
  return EP_OK;
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
  return ep::newton_space(count, M, N, nullptr).bytes;
}

extern "C" int ep_orthogonalize(const void* g, int dtype, int count, int M, int N, int steps, const float* coefficients, float eps, void* out,
                                void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
  using namespace ep;
  const int rc = check_newton(g, dtype, count, M, N, steps, coefficients, eps, workspace, workspace_bytes);
  if (rc != EP_OK) return rc;
  if (count == 0) return EP_OK;
  if (out == nullptr || !ep_host::aligned16(out)) return EP_ERR_INVALID_ARG;
  Source src{};
  src.g = g;
  src.f32 = dtype == EP_DTYPE_F32;
  return newton(src, count, M, N, steps, coefficients, eps, static_cast<__nv_bfloat16*>(out), nullptr, nullptr, 0.0f, 0.0f, workspace, status,
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
  Source src{};
  src.g = g;
  src.f32 = dtype == EP_DTYPE_F32;
  src.m = m;
  src.momentum = momentum;
  src.nesterov = nesterov != 0;
  return newton(src, count, M, N, steps, coefficients, eps, nullptr, w, static_cast<__nv_bfloat16*>(w16),
                (float)(1.0 - (double)lr * weight_decay), (float)((double)lr * scale), workspace, status, static_cast<cudaStream_t>(stream));
}
