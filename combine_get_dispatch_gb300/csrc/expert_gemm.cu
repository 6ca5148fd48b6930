// expert_gemm.cu -- the experts' bf16 products on the tensor cores.
//
//   kGlu     h = act(x Wg^T) * (x Wu^T)        per expert, rows of its segment
//   kLinear  y = act(x W^T + b) + r
//   kDx      dx = d W
//   kDw      dw = d^T x                        contraction over the segment's rows
//
// A pair of CTAs (one cluster, two SMs) computes a 256 x 256 tile with
// tcgen05.mma.cta_group::2: each CTA stages its 128 rows of A and half of B
// (kGlu: CTA 0 the gate's 128 columns, CTA 1 the up projection's, so that both
// halves of an output meet in one accumulator row) and holds its 128 rows of
// the sums in tensor memory.  Per 64 inner elements a CTA reads 32 KB for
// 512 clocks of products, where a single CTA with the same tile would read
// 48 KB: the L2 is what a 1-CTA form waits for.
//
// Roles: warp 0 copies (TMA, 6 stages), warp 1 of the first CTA issues products,
// warp 2 owns the tensor memory, warp 3 clears the rows past a segment's end
// (kDw, whose inner index is the row), warps 4-7 read the sums back and run the
// epilogue while the products of the next tile fill the other half of the
// tensor memory.  Tiles of all experts form one list that the pairs walk with a
// fixed stride; inside an expert 8 row tiles are taken together, so that the
// tiles in flight share operands in L2.

#include "expert_gemm.cuh"
#include "umma.cuh"

namespace ep {

constexpr int kGemmThreads = 256;
constexpr int kStages = 6;
constexpr int kTileM = 256, kTileN = 256, kHalf = 128;
constexpr int kTileK = 64;                       // bf16 elements of one 128-byte row
constexpr int kOperandBytes = kHalf * kTileK * 2;   // 16 KB: one CTA's half of an operand
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kBox = 32;                         // rows of a small A copy
constexpr int kEpilogueWarps = 4;

struct GemmParams {
  CUtensorMap a, a_small, b;
  ProductParams p;
  int tiles_n;
};

struct Shared {
  uint64_t full[kStages], empty[kStages];
  uint64_t landed[kStages], cleared[kStages];   // kDw: a segment's last block
  uint64_t sums_full[2], sums_empty[2];
  uint32_t tmem;
  TileTable table;
};

template <int kForm, int kAct>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
    k_expert_gemm(const __grid_constant__ GemmParams g) {
  extern __shared__ uint8_t raw[];
  uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  Shared& sh = *reinterpret_cast<Shared*>(stages + kStages * kStageBytes);
  constexpr bool kAMn = kForm == kDw, kBMn = kForm == kDw || kForm == kDx;
  constexpr int kCols = kForm == kGlu ? kHalf : kTileN;   // output columns of a tile
  constexpr uint32_t kIdesc = umma_idesc_bf16(kTileM, kTileN, kAMn, kBMn);

  const ProductParams& p = g.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    prefetch_map(&g.a);
    prefetch_map(&g.b);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sh.full[s], 1);      // the first CTA's, with the bytes of both
      mbar_init(&sh.empty[s], 1);     // the products' commit
      mbar_init(&sh.landed[s], 1);
      mbar_init(&sh.cleared[s], 1);   // the second CTA's
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.sums_full[i], 1);
      mbar_init(&sh.sums_empty[i], 2 * kEpilogueWarps);
    }
    fence_barrier_init();
  }
  if (warp == 2) tmem_alloc<2>(&sh.tmem, 512);
  build_table<kTileM, kGemmThreads>(sh.table, p.seg, kForm == kDw ? p.K : -1, blockIdx.x == 0);
  tmem_fence_before();
  cluster_sync();
  tmem_fence_after();
  const uint32_t tmem = sh.tmem;
  const int E = p.seg.E;

  bool ok = true;
  if (warp == 0 && lane == 0) {
    // ---------------------------------------------------------------- copies
    int s = 0;
    uint32_t phase = 0;
    Tile t;
    for (int64_t at = pair; ok && tile_at<kTileM>(sh.table, E, g.tiles_n, kCols, at, t); at += pairs) {
      const int inner = kForm == kDw ? t.count : p.K;
      const int blocks = (inner + kTileK - 1) / kTileK;
      // rows of A that each CTA has to read: all 128 of them in one copy, or 32 at a time
      int boxes[2] = {4, 4};
      if (kForm != kDw)
        for (int r = 0; r < 2; ++r) boxes[r] = max(0, min(4, (t.count - t.m0 - r * kHalf + kBox - 1) / kBox));
      const int mine = boxes[rank];
      const uint32_t bytes = 2 * kOperandBytes + (uint32_t)(boxes[0] + boxes[1]) * (kOperandBytes / 4);
      for (int kb = 0; kb < blocks; ++kb) {
        if (!mbar_wait_bounded(&sh.empty[s], phase ^ 1)) {
          ok = false;
          break;
        }
        const uint32_t sa = smem_addr(stages + s * kStageBytes), sb = sa + kOperandBytes;
        // a block that the segment ends in is cleared past its end first (warp 3)
        const bool tail = kForm == kDw && t.count - kb * kTileK < kTileK;
        uint32_t bar = map_to_rank(smem_addr(&sh.full[s]), 0);
        if (tail) {
          bar = smem_addr(&sh.landed[s]);
          mbar_arrive_expect_tx(&sh.landed[s], kStageBytes);
        } else if (rank == 0) {
          mbar_arrive_expect_tx(&sh.full[s], bytes);
        }
        const int k0 = kb * kTileK, am = t.m0 + (int)rank * kHalf;
        if (kAMn) {
          for (int i = 0; i < 2; ++i)
            tma_load_3d<true>(sa + i * (kOperandBytes / 2), &g.a, bar, am + i * 64, t.start + k0, 0);
        } else if (mine == 4) {
          tma_load_3d<true>(sa, &g.a, bar, k0, t.start + am, 0);
        } else {
          for (int i = 0; i < mine; ++i)
            tma_load_3d<true>(sa + i * (kOperandBytes / 4), &g.a_small, bar, k0, t.start + am + i * kBox, 0);
        }
        const int bn = t.n0 + (kForm == kGlu ? 0 : (int)rank * kHalf);
        if (kForm == kDw) {
          for (int i = 0; i < 2; ++i)
            tma_load_3d<true>(sb + i * (kOperandBytes / 2), &g.b, bar, bn + i * 64, t.start + k0, 0);
        } else if (kForm == kDx) {
          for (int i = 0; i < 2; ++i)
            tma_load_3d<true>(sb + i * (kOperandBytes / 2), &g.b, bar, bn + i * 64, k0, t.e);
        } else {
          tma_load_3d<true>(sb, &g.b, bar, k0, bn, kForm == kGlu ? 2 * t.e + (int)rank : t.e);
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
    uint32_t phase = 0, n = 0;
    Tile t;
    for (int64_t at = pair; ok && tile_at<kTileM>(sh.table, E, g.tiles_n, kCols, at, t); at += pairs) {
      const int blocks = ((kForm == kDw ? t.count : p.K) + kTileK - 1) / kTileK;
      if (blocks == 0) continue;
      const uint32_t half = n & 1, d = tmem + half * kTileN;
      if (!mbar_wait_cluster(&sh.sums_empty[half], ((n >> 1) & 1) ^ 1)) {
        ok = false;
        break;
      }
      tmem_fence_after();
      for (int kb = 0; kb < blocks; ++kb) {
        if (!mbar_wait_bounded(&sh.full[s], phase)) {
          ok = false;
          break;
        }
        tmem_fence_after();
        const uint32_t sa = smem_addr(stages + s * kStageBytes), sb = sa + kOperandBytes;
        // MN-major: 64-element columns 8 KB apart, 16 inner rows of 128 bytes a product
        const uint64_t da = umma_desc(sa, kAMn ? kOperandBytes / 2 : 16), db = umma_desc(sb, kBMn ? kOperandBytes / 2 : 16);
#pragma unroll
        for (int i = 0; i < kTileK / 16; ++i)
          umma_bf16_pair(d, da + i * (kAMn ? 2048 >> 4 : 32 >> 4), db + i * (kBMn ? 2048 >> 4 : 32 >> 4), kIdesc,
                         kb > 0 || i > 0);
        umma_commit_pair(&sh.empty[s]);
        if (++s == kStages) {
          s = 0;
          phase ^= 1;
        }
      }
      umma_commit_pair(&sh.sums_full[half]);
      ++n;
    }
  } else if (kForm == kDw && warp == 3) {
    // ---------------------------------------------------------------- rows past a segment's end
    int s = 0;
    uint32_t parity = 0;   // bit per stage
    Tile t;
    for (int64_t at = pair; ok && tile_at<kTileM>(sh.table, E, g.tiles_n, kCols, at, t); at += pairs) {
      const int blocks = (t.count + kTileK - 1) / kTileK;
      const int left = t.count % kTileK;
      if (left != 0) {
        const int st = (s + blocks - 1) % kStages;
        // a whole tile's copies may lie before this block
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(&sh.landed[st], (parity >> st) & 1,
                                                       kWaitNs + (uint64_t)blocks * 2000));
        if (ok) {
          uint8_t* base = stages + st * kStageBytes;
          for (int i = lane; i < 4 * (kTileK - left) * 8; i += 32) {   // 4 boxes, rows, 16-byte pieces
            const int box = i / ((kTileK - left) * 8), r = i % ((kTileK - left) * 8);
            st_shared_v4(base + box * (kOperandBytes / 2) + (left + r / 8) * 128 + (r % 8) * 16, make_uint4(0, 0, 0, 0));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (rank == 0) {
            ok = __all_sync(0xffffffffu, mbar_wait_cluster(&sh.cleared[st], (parity >> st) & 1));
            if (ok && lane == 0) mbar_arrive(&sh.full[st]);
          } else if (lane == 0) {
            mbar_arrive_cluster(map_to_rank(smem_addr(&sh.cleared[st]), 0));
          }
          parity ^= 1u << st;
        }
      }
      s = (s + blocks) % kStages;
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3;   // this warp's 32 lanes of the tensor memory
    uint32_t n = 0;
    Tile t;
    for (int64_t at = pair; ok && tile_at<kTileM>(sh.table, E, g.tiles_n, kCols, at, t); at += pairs) {
      const int blocks = ((kForm == kDw ? t.count : p.K) + kTileK - 1) / kTileK;
      const int m = t.m0 + (int)rank * kHalf + q * 32 + lane;
      const bool in = m < (kForm == kDw ? p.K : t.count);
      const uint32_t half = n & 1;
      if (blocks > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(&sh.sums_full[half], (n >> 1) & 1,
                                                       kWaitNs + (uint64_t)blocks * 2000));
        if (!ok) break;
        tmem_fence_after();
        ++n;
      }
      const uint32_t d = tmem + half * kTileN + ((uint32_t)(q * 32) << 16);
#pragma unroll 1
      for (int c0 = 0; c0 < kCols; c0 += 32) {
        float v[32], u[32];
        if (blocks > 0) {
          tmem_ld32(d + c0, v);
          if (kForm == kGlu) tmem_ld32(d + kHalf + c0, u);
          tmem_wait_ld();
          if (c0 + 32 == kCols) {   // the sums are read: the next tile's products may have them
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_addr(&sh.sums_empty[half]), 0));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = u[i] = 0.0f;
        }
        if (in) store_row<kForm, kAct>(p, t, m, c0, v, u);
        __syncwarp();
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
  const int smem = kStages * kStageBytes + (int)sizeof(Shared) + 1024;
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
  const uint64_t rows = (uint64_t)p.rows, E = (uint64_t)p.seg.E;
  int rc = EP_OK;
  auto map = [&](CUtensorMap* m, const void* base, uint64_t d0, uint64_t d1, uint64_t d2, uint32_t b0, uint32_t b1) {
    const uint64_t dims[3] = {d0, d1, d2}, strides[2] = {d0 * 2, d0 * d1 * 2};
    const uint32_t box[3] = {b0, b1, 1};
    if (rc == EP_OK) rc = ep_host::make_map(m, false, base, dims, strides, box);
  };
  const uint64_t N = (uint64_t)p.N, K = (uint64_t)p.K;
  if (form == kDw) {
    map(&g.a, p.a, K, rows, 1, 64, kTileK);
    map(&g.b, p.b, N, rows, 1, 64, kTileK);
    g.a_small = g.a;
  } else {
    map(&g.a, p.a, K, rows, 1, kTileK, kHalf);
    map(&g.a_small, p.a, K, rows, 1, kTileK, kBox);
    if (form == kDx)
      map(&g.b, p.b, N, K, E, 64, kTileK);
    else
      map(&g.b, p.b, K, N, form == kGlu ? 2 * E : E, kTileK, kHalf);
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

int make_map(CUtensorMap* m, bool bytes, const void* base, const uint64_t dims[3], const uint64_t strides[2],
             const uint32_t box[3]) {
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
  const cuuint32_t steps[3] = {1, 1, 1};
  const CUresult r = encode(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                            const_cast<void*>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? EP_OK : EP_ERR_CUDA;
}

}  // namespace ep_host
