// expert_gemm.cu -- the experts' bf16 products on the tensor cores.
//
//   kGlu     h = act(x Wg^T) * (x Wu^T)        per expert, rows of its segment
//   kLinear  y = act(x W^T + b) + r
//   kDx      dx = d W
//   kDw      dw = d^T x                        contraction over the segment's rows
//
// A pair of CTAs (one cluster, two SMs) computes a tile of 256 output columns by
// up to 256 output rows with tcgen05.mma.cta_group::2: each CTA stages 128
// columns of the first operand (the weights; kDw: x) and half the rows of the
// second (the segment's; kDw: d) and holds its 128 columns of the sums in tensor
// memory.  Per 64 inner elements a CTA reads 32 KB for 512 clocks of products,
// where a single CTA with the same tile would read 48 KB: the L2 is what a 1-CTA
// form waits for.
//
// The output's rows are the product's second extent because that is any multiple
// of 16: an expert with 40 rows, or the last rows of one with 2088, cost what they
// are and not a tile of 256 (65536 rows over 32 experts of about 2048: 2737 us
// with the rows as the first operand).  Sums then come out column by column;
// stmatrix turns them around on their way to a 32-row buffer from which one TMA
// store writes whole lines (turned by shuffles and stored by every thread, the
// weights' gradient of 32 experts with 12288 rows took 440 us, 278 us of them
// without any epilogue).  kGlu's first operand alternates 8 rows of Wg with the
// same 8 of Wu (one copy through a 5-d tensor map), which brings both halves of
// an output into one thread.
//
// Roles: warps 0 and 3 copy (TMA, 5 or 6 stages), warp 1 of the first CTA issues
// products, warp 2 owns the tensor memory and walks the list of tiles, in kDw,
// whose inner index is the row, warp 3 clears the rows past a segment's end
// instead and warp 0 copies both operands, warps 4-11 read
// the sums back and run the epilogue while the products of the next tile fill the
// other half of the tensor memory.

#include "expert_gemm.cuh"
#include "umma.cuh"

namespace ep {

constexpr int kGemmThreads = 384;
constexpr int kMaxStages = 10;
constexpr int kTileM = 256, kTileN = 256, kHalf = 128;   // columns, rows of the output; a CTA's columns
constexpr int kTileK = 64;                       // bf16 elements of one 128-byte row
constexpr int kOperandBytes = kHalf * kTileK * 2;   // 16 KB: one CTA's part of an operand
constexpr int kStageBytes = 2 * kOperandBytes;      // of a whole tile
constexpr int kBox = 32;                         // rows of a small copy
constexpr int kEpilogueWarps = 8;                // two groups of four
constexpr int kChunk = 32;                       // rows a group takes at a time
constexpr int kPieceBytes = kChunk * 128;        // 32 rows of 64 columns
constexpr int kBufferBytes = 2 * kPieceBytes;

// Stages of copies and output buffers of a group (one a warp) share 224 KB.  kGlu,
// in calls that the power limit bounds, does better with fewer stages (65536 x
// 7168 x 4096: 2326 us against 2413), the others with more (4096 x 8192 x 4864:
// 172 us against 176; zeros, which the power limit leaves alone, 148 against 158).
__host__ __device__ constexpr int stages_of(int form) { return form == kGlu ? 5 : 6; }
__host__ __device__ constexpr int buffers_of(int form) { return form == kGlu ? 4 : 2; }

struct GemmParams {
  CUtensorMap a, b, b_small, out, keep;
  ProductParams p;
  int tile_rows, tiles_n;
  int stages, stage_bytes;   // small tiles' stages hold fewer rows, and there are more of them
  bool a_whole, b_whole;   // an MN-major operand's 128 columns in one copy (4-d map)
};

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t landed[kMaxStages], cleared[kMaxStages];   // kDw: the block that a segment ends in
  uint64_t sums_full[2], sums_empty[2];
  TileRing ring;
  uint32_t tmem;
};

// A group's way out: four warps fill a buffer (32 rows x 128 columns of bf16, two
// pieces of 64 columns in the 128-byte swizzle), lane 0 of the buffer's own warp
// copies it out while the next ones are filled.  One barrier a buffer: before it,
// the next buffer's warp has seen that buffer's last copy read.
template <int kBuffers>
struct OutBuffers {
  uint8_t* base;
  int barrier;       // named barrier of the group's 128 threads
  int q, lane;
  uint32_t used;

  __device__ __forceinline__ uint8_t* next() { return base + (used % kBuffers) * kBufferBytes; }
  // The group's writes to next() are done; true in the thread that copies.
  __device__ __forceinline__ bool filled() {
    const int mine = used++ % kBuffers;
    fence_proxy_async_smem();
    if (lane == 0 && q == (int)(used % kBuffers)) tma_wait_read<0>();
    named_barrier_sync(barrier, 128);
    return lane == 0 && q == mine;
  }
};

// Address of 8 columns (16 bytes) of a row in a buffer: piece number 0-15.
__device__ __forceinline__ uint32_t out_address(const uint8_t* buffer, int row, int piece) {
  return smem_addr(buffer) + (piece >> 3) * kPieceBytes + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
}

template <int kForm, int kAct>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
    k_expert_gemm(const __grid_constant__ GemmParams g) {
  extern __shared__ uint8_t raw[];
  uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  constexpr int kBuffers = buffers_of(kForm);
  const int n_stages = g.stages, stage_bytes = g.stage_bytes;
  uint8_t* out_buffers = stages + stages_of(kForm) * kStageBytes;
  Shared& sh = *reinterpret_cast<Shared*>(out_buffers + 2 * kBuffers * kBufferBytes);
  constexpr bool kAMn = kForm == kDw || kForm == kDx, kBMn = kForm == kDw;
  constexpr int kCols = kForm == kGlu ? kHalf : 256;   // output columns of a tile

  const ProductParams& p = g.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    prefetch_map(&g.a);
    prefetch_map(&g.b);
    prefetch_map(&g.b_small);
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&sh.full[s], 1);      // the first CTA's, with the bytes of both
      mbar_init(&sh.empty[s], 1);     // the products' commit
      mbar_init(&sh.landed[s], 1);
      mbar_init(&sh.cleared[s], 2);   // one arrival of each CTA
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.sums_full[i], 1);
      mbar_init(&sh.sums_empty[i], 2 * kEpilogueWarps);
    }
    for (int i = 0; i < kTiles; ++i) {
      mbar_init(&sh.ring.full[i], 1);
      mbar_init(&sh.ring.empty[i], 2 + (rank == 0 ? 1 : 0) + kEpilogueWarps);   // warps 0, 3, 1 and the epilogue's
    }
    fence_barrier_init();
  }
  if (warp == 2) tmem_alloc<2>(&sh.tmem, 512);
  tmem_fence_before();
  __syncwarp();
  cluster_arrive();
  if (p.early) pdl_launch_dependents();
  pdl_wait();   // all that follows reads what kernels before this one may have written
  TileWalk walk;
  Tile first = {};
  if (warp == 2) {
    walk.begin(p.seg, kForm == kDw ? p.K : -1, g.tile_rows, g.tiles_n, kCols, blockIdx.x == 0, lane);
    first = walk.at(pair, lane);
  }
  __syncwarp();
  cluster_wait();
  tmem_fence_after();
  const uint32_t tmem = sh.tmem;

  bool ok = true;
  uint32_t taken = 0;
  Tile t = {};
  auto inner_blocks = [&]() { return ((kForm == kDw ? t.count : p.K) + kTileK - 1) / kTileK; };

  if (warp == 0 || (kForm != kDw && warp == 3)) {
    // ---------------------------------------------------------------- copies
    // warp 0 the first operand and kDw's second, else warp 3 the second: one warp issues a stage's copies in
    // about 300 ns, as long as the products of a whole tile's stage take.  Converged, one lane issues.
    const bool issue = elect_one();
    const uint32_t stage0 = smem_addr(stages), full0 = map_to_rank(smem_addr(&sh.full[0]), 0);
    uint32_t s = 0, phase = 0;
    while (next_tile(sh.ring, taken, t, ok, lane)) {
      const int blocks = inner_blocks();
      const int half = (t.rows + 15) / 16 * 8;   // rows of the second operand in a CTA
      // copied 32 at a time, or all 128; kDw: 64 columns of d at a time
      const int boxes = kForm == kDw ? (half + 63) / 64 : (half + kBox - 1) / kBox;
      const uint32_t mine = kOperandBytes + boxes * (kForm == kDw ? kOperandBytes / 2 : kOperandBytes / 4);
      const int n0 = t.n0 + (int)rank * (kForm == kGlu ? 64 : kHalf);                        // of the first operand
      const int m0 = t.m0 + (int)rank * half + (kForm == kDw ? 0 : t.start);                 // of the second
      for (int kb = 0; kb < blocks; ++kb) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.empty[s], phase ^ 1));
        if (!ok) break;
        if (issue) {
          const uint32_t sa = stage0 + s * stage_bytes, sb = sa + kOperandBytes;
          uint32_t bar = full0 + s * (uint32_t)sizeof(uint64_t);
          if (kForm == kDw) {
            // the segment's last rows first; where they end inside a product's 16, warp 3 clears the others
            if (kb == 0 && t.count % 16 != 0) {
              bar = smem_addr(&sh.landed[s]);
              mbar_arrive_expect_tx(&sh.landed[s], mine);
            } else if (rank == 0) {
              mbar_arrive_expect_tx(&sh.full[s], 2 * mine);
            }
            const int row = t.start + (blocks - 1 - kb) * kTileK;
            if (g.a_whole)
              tma_load_4d_pair(sa, &g.a, bar, 0, row, n0 / 64, 0);
            else
              for (int i = 0; i < 2; ++i)
                tma_load_3d<true>(sa + i * (kOperandBytes / 2), &g.a, bar, n0 + i * 64, row, 0);
            if (g.b_whole && half == kHalf && m0 % 64 == 0)
              tma_load_4d_pair(sb, &g.b, bar, 0, row, m0 / 64, 0);
            else
              for (int i = 0; i < boxes; ++i)
                tma_load_3d<true>(sb + i * (kOperandBytes / 2), &g.b_small, bar, m0 + i * 64, row, 0);
          } else if (warp == 0) {
            if (rank == 0) mbar_arrive_expect_tx(&sh.full[s], 2 * mine);
            const int k0 = kb * kTileK;
            if (kForm == kGlu)
              tma_load_5d_pair(sa, &g.a, bar, k0, 0, 0, n0 / 8, t.e);
            else if (kForm == kLinear)
              tma_load_3d<true>(sa, &g.a, bar, k0, n0, t.e);
            else if (g.a_whole)
              tma_load_4d_pair(sa, &g.a, bar, 0, k0, n0 / 64, t.e);
            else
              for (int i = 0; i < 2; ++i)
                tma_load_3d<true>(sa + i * (kOperandBytes / 2), &g.a, bar, n0 + i * 64, k0, t.e);
          } else {
            const int k0 = kb * kTileK;
            if (boxes == 4)
              tma_load_3d<true>(sb, &g.b, bar, k0, m0, 0);
            else
              for (int i = 0; i < boxes; ++i)
                tma_load_3d<true>(sb + i * (kOperandBytes / 4), &g.b_small, bar, k0, m0 + i * kBox, 0);
          }
        }
        if (++s == (uint32_t)n_stages) {
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
    // the whole warp walks along, so that addresses stay uniform; one lane issues
    const bool issue = elect_one();
    // MN-major: 64-element columns 8 KB apart, 16 inner rows of 128 bytes a product
    const uint32_t a0 = umma_desc_lo(smem_addr(stages), kAMn ? kOperandBytes / 2 : 16);
    const uint32_t b0 = umma_desc_lo(smem_addr(stages) + kOperandBytes, kBMn ? kOperandBytes / 2 : 16);
    constexpr uint32_t kStepA = (kAMn ? 2048 : 32) >> 4, kStepB = (kBMn ? 2048 : 32) >> 4;
    uint32_t s = 0, n = 0, full = 0, cleared = 0;   // parities: a bit per stage
    while (next_tile(sh.ring, taken, t, ok, lane)) {
      const int blocks = inner_blocks();
      if (blocks == 0) continue;
      const uint32_t idesc = umma_idesc_bf16(kTileM, (t.rows + 15) / 16 * 16, kAMn, kBMn);
      const uint32_t half = n & 1, d = tmem + half * kTileN;
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.sums_empty[half], ((n >> 1) & 1) ^ 1));
      if (!ok) break;
      tmem_fence_after();
      int kb = 0;
      if (kForm == kDw) {   // the segment's end first: as many products of 16 inner rows as it leaves
        if (t.count % 16 != 0) {
          ok = __all_sync(0xffffffffu, mbar_wait_cluster(&sh.cleared[s], (cleared >> s) & 1));
          cleared ^= 1u << s;
        } else {
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.full[s], (full >> s) & 1));
          full ^= 1u << s;
        }
        if (!ok) break;
        tmem_fence_after();
        if (issue) {
          const int steps = (t.count - (blocks - 1) * kTileK + 15) / 16;
          for (int i = 0; i < steps; ++i)
            umma_bf16_pair(d, a0 + s * (stage_bytes >> 4) + i * kStepA, b0 + s * (stage_bytes >> 4) + i * kStepB, idesc, i > 0);
          umma_commit_pair(&sh.empty[s]);
        }
        if (++s == n_stages) s = 0;
        kb = 1;
      }
      for (; kb < blocks; ++kb) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.full[s], (full >> s) & 1));
        if (!ok) break;
        full ^= 1u << s;
        tmem_fence_after();
        if (issue) {
          const uint32_t a = a0 + s * (stage_bytes >> 4), b = b0 + s * (stage_bytes >> 4);
          umma_bf16_pair(d, a, b, idesc, kForm == kDw || kb > 0);
#pragma unroll
          for (uint32_t i = 1; i < kTileK / 16; ++i) umma_bf16_pair(d, a + i * kStepA, b + i * kStepB, idesc, true);
          umma_commit_pair(&sh.empty[s]);
        }
        if (++s == n_stages) s = 0;
      }
      if (!ok) break;
      if (issue) umma_commit_pair(&sh.sums_full[half]);
      ++n;
    }
  } else if (warp == 2) {
    ok = feed_tiles(sh.ring, walk, first, pair, pairs, lane);
  } else if (kForm == kDw && warp == 3) {
    // ---------------------------------------------------------------- rows past a segment's end
    int s = 0;
    uint32_t parity = 0;   // bit per stage
    while (next_tile(sh.ring, taken, t, ok, lane)) {
      const int blocks = inner_blocks();
      if (t.count % 16 != 0) {
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(&sh.landed[s], (parity >> s) & 1, 2 * kWaitNs));
        if (ok) {
          uint8_t* base = stages + s * stage_bytes;
          // boxes of 64 x 64 (two of x, one or two of d), rows of 8 16-byte pieces: a lane a piece of one box
          const int boxes = 2 + ((t.rows + 15) / 16 * 8 + 63) / 64;
          if (lane >> 3 < boxes)
            for (int r = t.count - (blocks - 1) * kTileK; r % 16 != 0; ++r)
              st_shared_v4(base + (lane >> 3) * (kOperandBytes / 2) + r * 128 + (lane & 7) * 16, make_uint4(0, 0, 0, 0));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_addr(&sh.cleared[s]), 0));
          parity ^= 1u << s;
        }
      }
      s = (s + blocks) % n_stages;
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3, side = (warp - 4) >> 2;   // 32 lanes of the tensor memory; even or odd chunks of rows
    OutBuffers<kBuffers> buffers = {out_buffers + side * kBuffers * kBufferBytes, 1 + side, q, lane, 0};
    const int mrow = lane & 7, mat = lane >> 3;   // this lane's address in the four 8 x 8 matrices of a store
    // columns of this thread's sums: 16 hh + lane / 4 (+ 8); kGlu: gate and up of column 8 hh + lane / 4
    uint32_t n = 0;
    while (next_tile(sh.ring, taken, t, ok, lane)) {
      const int blocks = inner_blocks();
      const uint32_t half = n & 1;
      if (blocks > 0) {
        // a group's threads wait for one another below, so they give up together
        ok = named_barrier_and(1 + side, 128, mbar_wait_bounded(&sh.sums_full[half], (n >> 1) & 1,
                                                                kWaitNs + (uint64_t)blocks * 2000));
        if (!ok) break;
        tmem_fence_after();
        ++n;
      }
      const uint32_t d = tmem + half * kTileN + ((uint32_t)(q * 32) << 16);
      const int col0 = t.n0 + (int)rank * (kCols / 2);   // first output column of this CTA
      const int64_t row0 = kForm == kDw ? (int64_t)t.e * p.K + t.m0 : (int64_t)t.start + t.m0;
      const int y0 = kForm == kDw ? t.m0 : t.start + t.m0, z0 = kForm == kDw ? t.e : 0;
      float bias[4] = {};
      if (kForm == kLinear && p.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int col = col0 + q * 32 + i * 8 + (lane >> 2);
          if (col < p.N) bias[i] = __bfloat162float(p.bias[(int64_t)t.e * p.N + col]);
        }
      }
      auto sums_read = [&]() {   // the next tile's products may have this half
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(map_to_rank(smem_addr(&sh.sums_empty[half]), 0));
      };
      if (blocks > 0 && side * kChunk >= t.rows) sums_read();
#pragma unroll 1
      for (int r0 = side * kChunk; r0 < t.rows; r0 += 2 * kChunk) {
        const int rows = min(kChunk, t.rows - r0);
        float v[2][16];
        if (blocks > 0) {
          tmem_ld_16x32(d + r0, v[0]);
          tmem_ld_16x32(d + (16u << 16) + r0, v[1]);
          tmem_wait_ld(v[0], v[1]);
          if (r0 + 2 * kChunk >= t.rows) sums_read();
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[0][i] = v[1][i] = 0.0f;
        }
        // a filled buffer's pieces of 64 columns, at column x of `dst` (kept gate and up: both at x)
        auto copy_out = [&](const uint8_t* buf, const CUtensorMap* map, __nv_bfloat16* dst, int pieces, bool gate_up) {
          const bool copies = buffers.filled();
          if (rows == kChunk) {
            if (copies) {
              for (int i = 0; i < pieces; ++i) {
                const int col = col0 + (gate_up ? 0 : i * 64);
                if (col < p.N)
                  tma_store_3d(map, smem_addr(buf) + i * kPieceBytes, col, gate_up ? i : y0 + r0, gate_up ? y0 + r0 : z0);
              }
            }
          } else {   // the segment ends inside the chunk
            for (int i = q * 32 + lane; i < rows * pieces * 8; i += 128) {
              const int r = i / (pieces * 8), c = i % (pieces * 8);
              const int col = col0 + (gate_up ? (c & 7) * 8 : c * 8);
              const int64_t row = gate_up ? (row0 + r0 + r) * 2 + (c >> 3) : row0 + r0 + r;
              if (col < p.N) st_v4(dst + row * p.N + col, ld_shared_v4_at(out_address(buf, r, c)));
            }
          }
          if (copies) tma_commit();
        };
        if (kForm == kGlu) {
          if (p.keep != nullptr) {
            uint8_t* buf = buffers.next();
#pragma unroll
            for (int i = 0; i < 4; ++i)   // gate of both column groups, then up
              stmatrix4_trans(out_address(buf, 8 * i + mrow, (mat >> 1) * 8 + q * 2 + (mat & 1)),
                              pack_bf16x2(v[0][4 * i], v[0][4 * i + 1]), pack_bf16x2(v[1][4 * i], v[1][4 * i + 1]),
                              pack_bf16x2(v[0][4 * i + 2], v[0][4 * i + 3]), pack_bf16x2(v[1][4 * i + 2], v[1][4 * i + 3]));
            copy_out(buf, &g.keep, p.keep, 2, true);
          }
          uint32_t w[2][4];
#pragma unroll
          for (int hh = 0; hh < 2; ++hh)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[hh][i] = pack_bf16x2(act_value<kAct>(v[hh][4 * i]) * v[hh][4 * i + 2],
                                     act_value<kAct>(v[hh][4 * i + 1]) * v[hh][4 * i + 3]);
          uint8_t* buf = buffers.next();
#pragma unroll
          for (int i = 0; i < 4; i += 2)   // both column groups of 8 rows, then of the next 8
            stmatrix4_trans(out_address(buf, 8 * i + 8 * (mat >> 1) + mrow, q * 2 + (mat & 1)), w[0][i], w[1][i],
                            w[0][i + 1], w[1][i + 1]);
          copy_out(buf, &g.out, static_cast<__nv_bfloat16*>(p.out), 1, false);
        } else {
          const int piece = q * 4 + mat;   // 8 columns a matrix
          uint8_t* buf;
          if (kForm == kLinear) {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
              for (int i = 0; i < 16; ++i) v[hh][i] += bias[2 * hh + ((i >> 1) & 1)];
            if (p.keep != nullptr) {
              buf = buffers.next();
#pragma unroll
              for (int i = 0; i < 4; ++i)
                stmatrix4_trans(out_address(buf, 8 * i + mrow, piece), pack_bf16x2(v[0][4 * i], v[0][4 * i + 1]),
                                pack_bf16x2(v[0][4 * i + 2], v[0][4 * i + 3]), pack_bf16x2(v[1][4 * i], v[1][4 * i + 1]),
                                pack_bf16x2(v[1][4 * i + 2], v[1][4 * i + 3]));
              copy_out(buf, &g.keep, p.keep, 2, false);
            }
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
              for (int i = 0; i < 16; ++i) v[hh][i] = act_value<kAct>(v[hh][i]);
          }
          buf = buffers.next();
          if (kForm == kLinear && p.residual != nullptr) {
            // this warp's 32 rows x 32 columns through its own part of the buffer
#pragma unroll
            for (int i = lane; i < kChunk * 4; i += 32) {
              const int r = i >> 2, c = q * 4 + (i & 3);
              uint4 x = make_uint4(0, 0, 0, 0);
              if (r < rows && col0 + c * 8 < p.N) x = ld_v4(p.residual + (row0 + r0 + r) * p.N + col0 + c * 8);
              st_shared_v4_at(out_address(buf, r, c), x);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t x[4];
              ldmatrix4_trans(out_address(buf, 8 * i + mrow, piece), x);
#pragma unroll
              for (int m = 0; m < 4; ++m) {
                v[m >> 1][4 * i + 2 * (m & 1)] += bf16_lo(x[m]);
                v[m >> 1][4 * i + 2 * (m & 1) + 1] += bf16_hi(x[m]);
              }
            }
            __syncwarp();
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            stmatrix4_trans(out_address(buf, 8 * i + mrow, piece), pack_bf16x2(v[0][4 * i], v[0][4 * i + 1]),
                            pack_bf16x2(v[0][4 * i + 2], v[0][4 * i + 3]), pack_bf16x2(v[1][4 * i], v[1][4 * i + 1]),
                            pack_bf16x2(v[1][4 * i + 2], v[1][4 * i + 3]));
          copy_out(buf, &g.out, static_cast<__nv_bfloat16*>(p.out), 2, false);
        }
      }
    }
    if (lane == 0) tma_wait_all();
  }
  if (!ok) set_status(p.seg.status, EP_ERR_TIMEOUT);
  __syncwarp();
  tmem_fence_before();
  cluster_sync();
  tmem_fence_after();
  if (warp == 2) tmem_free<2>(tmem, 512);
}

template <int kForm, int kAct>
static int launch_gemm_t(const GemmParams& g, int64_t tiles, cudaStream_t stream) {
  const int smem = stages_of(kForm) * kStageBytes + 2 * buffers_of(kForm) * kBufferBytes + (int)sizeof(Shared) + 1024;
  const void* fn = reinterpret_cast<const void*>(k_expert_gemm<kForm, kAct>);
  if (ep_host::ensure_max_smem(fn, smem) != EP_OK) return EP_ERR_CUDA;
  const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(tiles, ep_host::grid_cap(1) / 2));
  if (ep_host::launch_dependent(k_expert_gemm<kForm, kAct>, (int)pairs * 2, kGemmThreads, smem, stream, g) != EP_OK)
    return EP_ERR_CUDA;
  ep_host::count_launch();
  return ep_host::check_launch();
}

template <int kForm>
static int launch_gemm_act(const GemmParams& g, int64_t tiles, int act, cudaStream_t s) {
  switch (act) {
    case EP_ACT_RELU: return launch_gemm_t<kForm, EP_ACT_RELU>(g, tiles, s);
    case EP_ACT_SILU: return launch_gemm_t<kForm, EP_ACT_SILU>(g, tiles, s);
    default: return launch_gemm_t<kForm, EP_ACT_GELU>(g, tiles, s);
  }
}

int launch_gemm_bf16(Form form, const ProductParams& p, int act, cudaStream_t stream) {
  GemmParams g;
  g.p = p;
  const uint64_t rows = (uint64_t)p.rows, E = (uint64_t)p.seg.E, N = (uint64_t)p.N, K = (uint64_t)p.K;
  int rc = EP_OK;
  auto map = [&](CUtensorMap* m, const void* base, uint64_t d0, uint64_t d1, uint64_t d2, uint32_t b0, uint32_t b1) {
    const uint64_t dims[3] = {d0, d1, d2}, strides[2] = {d0 * 2, d0 * d1 * 2};
    const uint32_t box[3] = {b0, b1, 1};
    if (rc == EP_OK) rc = ep_host::make_map(m, false, 3, base, dims, strides, box);
  };
  // An MN-major operand of `wide` columns whose 64-column pieces end with the row: both pieces of a
  // CTA's 128 columns in one copy.
  auto map_whole = [&](CUtensorMap* m, const void* base, uint64_t wide, uint64_t deep, uint64_t count) {
    const uint64_t dims[4] = {64, deep, wide / 64, count}, strides[3] = {wide * 2, 128, wide * deep * 2};
    const uint32_t box[4] = {64, kTileK, 2, 1};
    if (rc == EP_OK) rc = ep_host::make_map(m, false, 4, base, dims, strides, box);
  };
  g.a_whole = (form == kDw || form == kDx) && p.N % 64 == 0;
  g.b_whole = form == kDw && p.K % 64 == 0;
  if (form == kDw) {
    if (g.a_whole)
      map_whole(&g.a, p.b, N, rows, 1);
    else
      map(&g.a, p.b, N, rows, 1, 64, kTileK);
    map(&g.b_small, p.a, K, rows, 1, 64, kTileK);
    if (g.b_whole)
      map_whole(&g.b, p.a, K, rows, 1);
    else
      g.b = g.b_small;
  } else {
    if (form == kGlu) {   // (inner, row of 8, gate / up, 8-row group, expert)
      const uint64_t dims[5] = {K, 8, 2, N / 8, E}, strides[4] = {K * 2, N * K * 2, 8 * K * 2, 2 * N * K * 2};
      const uint32_t box[5] = {kTileK, 8, 2, 8, 1};
      rc = ep_host::make_map(&g.a, false, 5, p.b, dims, strides, box);
    } else if (form == kLinear) {
      map(&g.a, p.b, K, N, E, kTileK, kHalf);
    } else if (g.a_whole) {
      map_whole(&g.a, p.b, N, K, E);
    } else {
      map(&g.a, p.b, N, K, E, 64, kTileK);
    }
    map(&g.b, p.a, K, rows, 1, kTileK, kHalf);
    map(&g.b_small, p.a, K, rows, 1, kTileK, kBox);
  }
  auto map_out = [&](CUtensorMap* m, const void* base, uint64_t d1, uint64_t d2, uint32_t b1, uint32_t b2) {
    const uint64_t dims[3] = {N, d1, d2}, strides[2] = {N * 2, N * d1 * 2};
    const uint32_t box[3] = {64, b1, b2};
    if (rc == EP_OK) rc = ep_host::make_map(m, false, 3, base, dims, strides, box);
  };
  if (form == kDw)
    map_out(&g.out, p.out, K, E, kChunk, 1);
  else
    map_out(&g.out, p.out, rows, 1, kChunk, 1);
  g.keep = g.out;
  if (p.keep != nullptr) {
    if (form == kGlu)
      map_out(&g.keep, p.keep, 2, rows, 1, kChunk);
    else
      map_out(&g.keep, p.keep, rows, 1, kChunk, 1);
  }
  if (rc != EP_OK) return rc;
  const int cols = form == kGlu ? kHalf : kTileN;
  g.tiles_n = (p.N + cols - 1) / cols;
  // Row tiles: whole ones and at most one ragged one an expert.  Where that leaves pairs without a tile they
  // are made smaller (777 x 2048 x 1000, dx: 21.7 us with 16 tiles of 256 rows).
  auto tiles_of = [&](int64_t tile) {
    const int64_t each = (p.K + tile - 1) / tile;
    const int64_t m = form == kDw ? p.seg.E * each : p.seg.E == 1 ? (p.rows + tile - 1) / tile : p.rows / tile + p.seg.E;
    return m * g.tiles_n;
  };
  const int64_t pairs = std::max(1, ep_host::grid_cap(1) / 2);
  g.tile_rows = kTileN;
  while (g.tile_rows > 32 && tiles_of(g.tile_rows / 2) <= pairs) g.tile_rows /= 2;
  const int64_t tiles = tiles_of(g.tile_rows);
  const int b_bytes = form == kDw ? (g.tile_rows / 2 + 63) / 64 * (kOperandBytes / 2) : (g.tile_rows / 2 + kBox - 1) / kBox * (kOperandBytes / 4);
  g.stage_bytes = kOperandBytes + b_bytes;
  g.stages = std::min(kMaxStages, stages_of(form) * kStageBytes / g.stage_bytes);
  if (tiles / g.tiles_n >= (int64_t)1 << 31) return EP_ERR_INVALID_ARG;
  switch (form) {
    case kGlu: return launch_gemm_act<kGlu>(g, tiles, act, stream);
    case kLinear:
      return act == EP_ACT_NONE ? launch_gemm_t<kLinear, EP_ACT_NONE>(g, tiles, stream)
                                : launch_gemm_act<kLinear>(g, tiles, act, stream);
    case kDx: return launch_gemm_t<kDx, EP_ACT_NONE>(g, tiles, stream);
    default: return launch_gemm_t<kDw, EP_ACT_NONE>(g, tiles, stream);
  }
}

}  // namespace ep

namespace ep_host {

typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                           const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                           CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static Encode encoder() {
  static const Encode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<Encode>(f);
  }();
  return encode;
}

int make_map(CUtensorMap* m, bool bytes, int rank, const void* base, const uint64_t* dims, const uint64_t* strides,
             const uint32_t* box, bool half_swizzle) {
  const Encode encode = encoder();
  if (encode == nullptr) return EP_ERR_CUDA;
  const cuuint32_t steps[5] = {1, 1, 1, 1, 1};
  const CUresult r = encode(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                            (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, steps,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, half_swizzle ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? EP_OK : EP_ERR_CUDA;
}

int make_row_map(CUtensorMap* m, const void* base, uint64_t words, uint64_t rows, uint64_t count, uint32_t box_rows) {
  const Encode encode = encoder();
  if (encode == nullptr) return EP_ERR_CUDA;
  const cuuint64_t dims[3] = {words, rows, count}, strides[2] = {words * 4, words * rows * 4};
  const cuuint32_t box[3] = {256, box_rows, 1}, steps[3] = {1, 1, 1};
  const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(base), dims, strides, box, steps,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? EP_OK : EP_ERR_CUDA;
}

}  // namespace ep_host
