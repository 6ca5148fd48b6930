// expert_gemm.cu -- the experts' bf16 products on the tensor cores.
//
//   kGlu     h = act(x Wg^T) * (x Wu^T)        per expert, rows of its segment
//   kLinear  y = act(x W^T + b) + r
//   kDx      dx = d W
//   kDw      dw = d^T x                        contraction over the segment's rows
//
// A pair of CTAs (one cluster, two SMs) computes a tile of 256 x up to 256 with
// tcgen05.mma.cta_group::2: each CTA stages 128 rows of the first operand and half
// of the second and holds its 128 rows of the sums in tensor memory.  Per 64 inner
// elements a CTA reads 32 KB for 512 clocks of products, where a single CTA with
// the same tile would read 48 KB: the L2 is what a 1-CTA form waits for.
//
// In kGlu, kLinear and kDx the weights are the first operand and the segment's
// rows the second: the product's second extent is any multiple of 16, so that an
// expert with 40 rows, or the last rows of one with 2088, cost what they are and
// not a tile of 256 (65536 rows over 32 experts of about 2048 rows: 2737 us with
// the rows as the first operand, 2248 us where every segment was a multiple of
// 256).  Sums then lie column by column; the epilogue turns 32 rows at a time
// around in shared memory.  kGlu's first operand alternates 8 rows of Wg with the
// same 8 of Wu (one copy through a 5-d tensor map), which puts both halves of an
// output next to each other.
//
// Roles: warp 0 copies (TMA, 6 stages), warp 1 of the first CTA issues products,
// warp 2 owns the tensor memory and looks the tiles up, warp 3 clears the rows past a segment's end
// (kDw, whose inner index is the row), warps 4-11 read the sums back and run the
// epilogue while the products of the next tile fill the other half of the tensor
// memory.  Tiles of all experts form one list that the pairs walk with a fixed
// stride; inside an expert 8 row tiles are taken together, so that the tiles in
// flight share operands in L2.

#include "expert_gemm.cuh"
#include "umma.cuh"

namespace ep {

constexpr int kGemmThreads = 384;
constexpr int kStages = 6;
constexpr int kTileM = 256, kTileN = 256, kHalf = 128;
constexpr int kTileK = 64;                       // bf16 elements of one 128-byte row
constexpr int kOperandBytes = kHalf * kTileK * 2;   // 16 KB: one CTA's part of an operand
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kBox = 32;                         // rows of a small copy
constexpr int kEpilogueWarps = 8;
constexpr int kTiles = 4;                        // tiles looked up ahead
constexpr int kChunk = 32;                       // rows turned around at a time
constexpr int kTurnBytes = kChunk * kHalf * 4;

struct GemmParams {
  CUtensorMap a, b, b_small;
  ProductParams p;
  int tiles_n;
};

struct Shared {
  uint64_t full[kStages], empty[kStages];
  uint64_t landed[kStages], cleared[kStages];   // kDw: the block that a segment ends in
  uint64_t sums_full[2], sums_empty[2];
  uint64_t tile_full[kTiles], tile_empty[kTiles];
  Tile tiles[kTiles];
  uint32_t tmem;
  TileTable table;
};

template <int kForm, int kAct>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
    k_expert_gemm(const __grid_constant__ GemmParams g) {
  extern __shared__ uint8_t raw[];
  uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  float* turn = reinterpret_cast<float*>(stages + kStages * kStageBytes);   // [kChunk][kHalf]
  Shared& sh = *reinterpret_cast<Shared*>(stages + kStages * kStageBytes + (kForm == kDw ? 0 : kTurnBytes));
  constexpr bool kAMn = kForm == kDw || kForm == kDx, kBMn = kForm == kDw;
  constexpr int kCols = kForm == kGlu ? kHalf : 256;   // output columns of a tile

  const ProductParams& p = g.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int E = p.seg.E, fixed_rows = kForm == kDw ? p.K : -1;

  if (threadIdx.x == 0) {
    prefetch_map(&g.a);
    prefetch_map(&g.b);
    if (kForm != kDw) prefetch_map(&g.b_small);
    for (int s = 0; s < kStages; ++s) {
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
      mbar_init(&sh.tile_full[i], 1);
      mbar_init(&sh.tile_empty[i], 1 + (rank == 0 ? 1 : 0) + (kForm == kDw ? 1 : 0) + kEpilogueWarps);
    }
    fence_barrier_init();
  }
  if (warp == 2) tmem_alloc<2>(&sh.tmem, 512);
  build_table<kTileM, kGemmThreads>(sh.table, p.seg, fixed_rows, blockIdx.x == 0);
  tmem_fence_before();
  cluster_sync();
  tmem_fence_after();
  const uint32_t tmem = sh.tmem;

  bool ok = true;
  Tile t;
  uint32_t taken = 0;
  // the pair's next tile, as warp 2 looked it up; e < 0 past the last.  One
  // arrival a consumer frees its place: `first` in a single thread, or in lane 0
  // of a converged warp.
  auto next_tile = [&](bool first) {
    if (!ok) return false;
    const uint32_t i = taken % kTiles;
    ok = mbar_wait_bounded(&sh.tile_full[i], (taken / kTiles) & 1, 30 * kWaitNs);
    if (!ok) return false;
    t = sh.tiles[i];
    ++taken;
    if (first) mbar_arrive(&sh.tile_empty[i]);
    return t.e >= 0;
  };
  auto next_tile_warp = [&]() {
    const bool more = next_tile(false);
    ok = __all_sync(0xffffffffu, ok);
    if (ok && lane == 0) mbar_arrive(&sh.tile_empty[(taken - 1) % kTiles]);
    return ok && more;
  };
  auto inner_blocks = [&]() { return ((kForm == kDw ? t.count : p.K) + kTileK - 1) / kTileK; };

  if (warp == 0 && lane == 0) {
    // ---------------------------------------------------------------- copies
    int s = 0;
    uint32_t phase = 0;
    while (next_tile(true)) {
      const int blocks = inner_blocks();
      const int half = kForm == kDw ? kHalf : (t.rows + 15) / 16 * 8;   // rows of the second operand in a CTA
      const int boxes = (half + kBox - 1) / kBox;
      const uint32_t bytes = 2 * kOperandBytes + 2 * (kForm == kDw ? kOperandBytes : boxes * (kOperandBytes / 4));
      for (int kb = 0; kb < blocks; ++kb) {
        if (!mbar_wait_bounded(&sh.empty[s], phase ^ 1)) {
          ok = false;
          break;
        }
        const uint32_t sa = smem_addr(stages + s * kStageBytes), sb = sa + kOperandBytes;
        // kDw takes the segment's last rows first; where they end inside a product's 16, warp 3 clears the others
        const bool tail = kForm == kDw && kb == 0 && t.count % 16 != 0;
        uint32_t bar = map_to_rank(smem_addr(&sh.full[s]), 0);
        if (tail) {
          bar = smem_addr(&sh.landed[s]);
          mbar_arrive_expect_tx(&sh.landed[s], kStageBytes);
        } else if (rank == 0) {
          mbar_arrive_expect_tx(&sh.full[s], bytes);
        }
        const int k0 = (kForm == kDw ? blocks - 1 - kb : kb) * kTileK;
        if (kForm == kDw) {
          for (int i = 0; i < 2; ++i) {
            const int at_box = (int)rank * kHalf + i * 64;
            tma_load_3d<true>(sa + i * (kOperandBytes / 2), &g.a, bar, t.m0 + at_box, t.start + k0, 0);
            tma_load_3d<true>(sb + i * (kOperandBytes / 2), &g.b, bar, t.n0 + at_box, t.start + k0, 0);
          }
        } else {
          if (kForm == kGlu)
            tma_load_5d_pair(sa, &g.a, bar, k0, 0, 0, t.n0 / 8 + (int)rank * 8, t.e);
          else if (kForm == kLinear)
            tma_load_3d<true>(sa, &g.a, bar, k0, t.n0 + (int)rank * kHalf, t.e);
          else
            for (int i = 0; i < 2; ++i)
              tma_load_3d<true>(sa + i * (kOperandBytes / 2), &g.a, bar, t.n0 + (int)rank * kHalf + i * 64, k0, t.e);
          const int row = t.start + t.m0 + (int)rank * half;
          if (boxes == 4)
            tma_load_3d<true>(sb, &g.b, bar, k0, row, 0);
          else
            for (int i = 0; i < boxes; ++i)
              tma_load_3d<true>(sb + i * (kOperandBytes / 4), &g.b_small, bar, k0, row + i * kBox, 0);
        }
        if (++s == kStages) {
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
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ---------------------------------------------------------------- products
    int s = 0;
    uint32_t n = 0, full = 0, cleared = 0;   // parities, a bit per stage
    while (next_tile(true)) {
      const int blocks = inner_blocks();
      if (blocks == 0) continue;
      const uint32_t idesc = umma_idesc_bf16(kTileM, kForm == kDw ? kTileN : (t.rows + 15) / 16 * 16, kAMn, kBMn);
      const uint32_t half = n & 1, d = tmem + half * kTileN;
      if (!mbar_wait_cluster(&sh.sums_empty[half], ((n >> 1) & 1) ^ 1)) {
        ok = false;
        break;
      }
      tmem_fence_after();
      for (int kb = 0; kb < blocks; ++kb) {
        const bool tail = kForm == kDw && kb == 0 && t.count % 16 != 0;
        if (tail) {
          ok = mbar_wait_cluster(&sh.cleared[s], (cleared >> s) & 1);
          cleared ^= 1u << s;
        } else {
          ok = mbar_wait_bounded(&sh.full[s], (full >> s) & 1);
          full ^= 1u << s;
        }
        if (!ok) break;
        tmem_fence_after();
        // products of 16 inner rows: as many as the segment's end leaves
        const int steps = kForm == kDw && kb == 0 ? (t.count - (blocks - 1) * kTileK + 15) / 16 : kTileK / 16;
        const uint32_t sa = smem_addr(stages + s * kStageBytes), sb = sa + kOperandBytes;
        // MN-major: 64-element columns 8 KB apart, 16 inner rows of 128 bytes a product
        const uint64_t da = umma_desc(sa, kAMn ? kOperandBytes / 2 : 16), db = umma_desc(sb, kBMn ? kOperandBytes / 2 : 16);
#pragma unroll
        for (int i = 0; i < kTileK / 16; ++i)
          if (i < steps)
            umma_bf16_pair(d, da + i * (kAMn ? 2048 >> 4 : 32 >> 4), db + i * (kBMn ? 2048 >> 4 : 32 >> 4), idesc,
                           kb > 0 || i > 0);
        umma_commit_pair(&sh.empty[s]);
        if (++s == kStages) s = 0;
      }
      umma_commit_pair(&sh.sums_full[half]);
      ++n;
    }
  } else if (warp == 2 && lane == 0) {
    // ---------------------------------------------------------------- tiles
    int64_t at = pair;
    for (uint32_t n = 0; ok; ++n, at += pairs) {
      const uint32_t i = n % kTiles;
      const bool more = tile_at<kTileM, kForm != kDw>(sh.table, E, fixed_rows, g.tiles_n, kCols, at, t);
      // a place is free when the slowest reader is done with a tile: as long as the epilogue's wait
      ok = mbar_wait_bounded(&sh.tile_empty[i], ((n / kTiles) & 1) ^ 1, 30 * kWaitNs);
      if (!ok) break;
      if (!more) t.e = -1;
      sh.tiles[i] = t;
      mbar_arrive(&sh.tile_full[i]);
      if (!more) break;
    }
  } else if (kForm == kDw && warp == 3) {
    // ---------------------------------------------------------------- rows past a segment's end
    int s = 0;
    uint32_t parity = 0;   // bit per stage
    while (next_tile_warp()) {
      const int blocks = inner_blocks();
      if (t.count % 16 != 0) {
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(&sh.landed[s], (parity >> s) & 1, 2 * kWaitNs));
        if (ok) {
          uint8_t* base = stages + s * kStageBytes;
          const int last = t.count - (blocks - 1) * kTileK, rows = 16 - last % 16;
          for (int i = lane; i < 4 * 8 * rows; i += 32)   // 4 boxes of 64 x 64, rows of 8 16-byte pieces
            st_shared_v4(base + (i / (8 * rows)) * (kOperandBytes / 2) + (last + i / 8 % rows) * 128 + (i % 8) * 16,
                         make_uint4(0, 0, 0, 0));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_addr(&sh.cleared[s]), 0));
          parity ^= 1u << s;
        }
      }
      s = (s + blocks) % kStages;
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3, side = (warp - 4) >> 2;   // 32 lanes of the tensor memory; which columns of them
    const int tid = threadIdx.x - 128;
    uint32_t n = 0;
    while (next_tile_warp()) {
      const int blocks = inner_blocks();
      const uint32_t half = n & 1;
      if (blocks > 0) {
        ok = mbar_wait_cluster(&sh.sums_full[half], (n >> 1) & 1, kWaitNs + (uint64_t)blocks * 2000);
        // a thread that gives up takes its group along: the barriers below are for all of them
        ok = __all_sync(0xffffffffu, ok);
        if (kForm != kDw) ok = named_barrier_and(1, 32 * kEpilogueWarps, ok);
        if (!ok) break;
        tmem_fence_after();
        ++n;
      }
      const uint32_t d = tmem + half * kTileN + ((uint32_t)(q * 32) << 16);
      auto sums_read = [&]() {   // the next tile's products may have this half
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_addr(&sh.sums_empty[half]), 0));
      };
      if (kForm == kDw) {
        const int m = t.m0 + (int)rank * kHalf + q * 32 + lane;
#pragma unroll 1
        for (int c0 = side * kHalf; c0 < side * kHalf + kHalf; c0 += 32) {
          float v[32];
          if (blocks > 0) {
            tmem_ld32(d + c0, v);
            tmem_wait_ld();
            if (c0 + 32 == side * kHalf + kHalf) sums_read();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.0f;
          }
          if (m < p.K) store32<kForm, kAct>(p, t.e, (int64_t)t.e * p.K + m, t.n0 + c0, v, v);
          __syncwarp();
        }
      } else {
        constexpr int kGroups = kForm == kGlu ? 8 : 16;   // of 8 output columns in this CTA
#pragma unroll 1
        for (int r0 = 0; r0 < t.rows; r0 += kChunk) {
          float v[16];
          tmem_ld16(d + r0 + side * 16, v);
          tmem_wait_ld();
          if (r0 + kChunk >= t.rows) sums_read();
#pragma unroll
          for (int i = 0; i < 16; ++i) turn[(side * 16 + i) * kHalf + q * 32 + lane] = v[i];
          named_barrier_sync(1, 32 * kEpilogueWarps);
#pragma unroll
          for (int i = tid; i < kChunk * kGroups; i += 32 * kEpilogueWarps) {
            const int r = r0 + i / kGroups, c = i % kGroups;
            const int col = t.n0 + (int)rank * (kGroups * 8) + c * 8;
            if (r < t.rows && col < p.N) {
              float z[8], u[8];
              const float* src = turn + (i / kGroups) * kHalf + c * (kForm == kGlu ? 16 : 8);
#pragma unroll
              for (int j = 0; j < 8; ++j) z[j] = src[j];
#pragma unroll
              for (int j = 0; j < 8; ++j) u[j] = kForm == kGlu ? src[8 + j] : 0.0f;
              store8<kForm, kAct>(p, t.e, (int64_t)t.start + t.m0 + r, col, z, u);
            }
          }
          named_barrier_sync(1, 32 * kEpilogueWarps);
        }
      }
    }
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
  const int smem = kStages * kStageBytes + (kForm == kDw ? 0 : kTurnBytes) + (int)sizeof(Shared) + 1024;
  const void* fn = reinterpret_cast<const void*>(k_expert_gemm<kForm, kAct>);
  if (ep_host::ensure_max_smem(fn, smem) != EP_OK) return EP_ERR_CUDA;
  const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(tiles, ep_host::grid_cap(1) / 2));
  k_expert_gemm<kForm, kAct><<<(int)pairs * 2, kGemmThreads, smem, stream>>>(g);
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
  if (form == kDw) {
    map(&g.a, p.a, K, rows, 1, 64, kTileK);
    map(&g.b, p.b, N, rows, 1, 64, kTileK);
    g.b_small = g.b;
  } else {
    if (form == kGlu) {   // (inner, row of 8, gate / up, 8-row group, expert)
      const uint64_t dims[5] = {K, 8, 2, N / 8, E}, strides[4] = {K * 2, N * K * 2, 8 * K * 2, 2 * N * K * 2};
      const uint32_t box[5] = {kTileK, 8, 2, 8, 1};
      rc = ep_host::make_map(&g.a, false, 5, p.b, dims, strides, box);
    } else if (form == kLinear) {
      map(&g.a, p.b, K, N, E, kTileK, kHalf);
    } else {
      map(&g.a, p.b, N, K, E, 64, kTileK);
    }
    map(&g.b, p.a, K, rows, 1, kTileK, kHalf);
    map(&g.b_small, p.a, K, rows, 1, kTileK, kBox);
  }
  if (rc != EP_OK) return rc;
  const int cols = form == kGlu ? kHalf : kTileN;
  g.tiles_n = (p.N + cols - 1) / cols;
  // at most one ragged row tile an expert
  const int64_t tiles_m = form == kDw ? (int64_t)p.seg.E * ((p.K + kTileM - 1) / kTileM) : p.rows / kTileM + p.seg.E;
  if (tiles_m >= (int64_t)1 << 31) return EP_ERR_INVALID_ARG;
  const int64_t tiles = tiles_m * g.tiles_n;
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

int make_map(CUtensorMap* m, bool bytes, int rank, const void* base, const uint64_t* dims, const uint64_t* strides,
             const uint32_t* box) {
  typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
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
  if (encode == nullptr) return EP_ERR_CUDA;
  const cuuint32_t steps[5] = {1, 1, 1, 1, 1};
  const CUresult r = encode(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                            (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, steps,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? EP_OK : EP_ERR_CUDA;
}

}  // namespace ep_host
