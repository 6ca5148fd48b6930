// expert_gemm_e4m3.cu -- the experts' forward products on E4M3 rows and weights
// with power-of-two scales, as the FP8 dispatch lays them out.
//
//   sum over 128-blocks b of  2^(sx[row][b] - 127) 2^(sw[col/128][b] - 127)
//                             sum_{k in b} qx[row][k] qw[col][k]
//
// tcgen05.mma kind::mxf8f6f4 applies ue8m0 scales from tensor memory inside the
// product (one per row and 32 inner elements: the same byte for the four of a
// 128-block), so the sums need no second pass.  Serving batches give an expert
// some tens of rows and the time is that of reading its weights once: one CTA per
// SM computes 128 x 256 tiles, so that two thirds of the bytes in flight (4 stages
// of 48 KB, fewer rows of A where the segment has fewer) are weights: 64 experts
// with 64 rows of 7168, gated, in 278-285 us (1.0 of the copy rate), 2048 ->
// 7168 in 148-151 us (0.98-1.0).  65536 rows over 32 experts, gated, take 1303 us
// (2950 TFLOP/s; 1549 us while one warp issued all copies); pairs of CTAs as for
// bf16 took 1343 us there, and 361 and 193 us on the two decode products, whose
// few rows leave most of a 256-row tile empty.
//
// Roles: warps 0 and 3 copy, warp 1 issues products, warp 2 owns the tensor memory,
// warps 4-7 and 12-15 run the epilogue, warps 8-11 move the scales of a stage from global
// memory (read a few blocks ahead) to tensor memory, each to its own 32 lanes.

#include "expert_gemm.cuh"
#include "umma.cuh"

namespace ep {

constexpr int kMxThreads = 512;
constexpr int kMxStages = 4;
constexpr int kMxTileM = 128, kMxTileN = 256;
constexpr int kMxABytes = kMxTileM * kFp8Block, kMxBBytes = kMxTileN * kFp8Block;
constexpr int kMxStageBytes = kMxABytes + kMxBBytes;
constexpr int kMxBox = 32;
// tensor memory: sums in columns 0-255, then 16 columns of scales a stage
constexpr int kMxScaleCol = 256, kMxScaleCols = 16, kMxScaleB = 8;
constexpr int kMxAhead = 4;   // blocks whose scales are read ahead

struct MxParams {
  CUtensorMap a, a_small, b;
  ProductParams p;
  int tiles_n;
};

struct MxShared {
  uint64_t full[kMxStages], scaled[kMxStages], empty[kMxStages];
  uint64_t sums_full, sums_empty;
  TileRing ring;
  uint32_t tmem;
  float amax[2][kMxTileM];   // of the halves of a row's outputs (E4M3 output)
};

// One block's scale bytes as a lane of a scale warp reads them: rows lane + 32 j
// of A, and the two 128-column halves of B.
struct MxScales {
  uint8_t a[4], b[2];
};

// Eight fp32 sums -> 16 bytes of bf16.
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

__device__ __forceinline__ void add8(float* z, uint4 b) {
  const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    z[2 * i] += bf16_lo(w[i]);
    z[2 * i + 1] += bf16_hi(w[i]);
  }
}

// The epilogue of 32 columns from n0 on of output row `row` of expert e: v the
// sums (kGlu: of the gate), u those of the up projection.
template <int kForm, int kAct>
__device__ __forceinline__ void store32(const ProductParams& p, int e, int64_t row, int n0, float (&v)[32],
                                        const float (&u)[32]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int n = n0 + q * 8;
    if (n >= p.N) break;
    float* z = v + q * 8;
    if (kForm == kGlu) {
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = act_value<kAct>(z[i]) * u[q * 8 + i];
    } else {
      if (p.bias != nullptr) add8(z, __ldg(reinterpret_cast<const uint4*>(p.bias + (int64_t)e * p.N + n)));
      if (p.keep != nullptr) st_v4(p.keep + row * p.N + n, pack8(z));
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = act_value<kAct>(z[i]);
      if (p.residual != nullptr) add8(z, ld_v4(p.residual + row * p.N + n));   // may be the output itself
    }
    st_v4(static_cast<__nv_bfloat16*>(p.out) + row * p.N + n, pack8(z));
  }
}

template <int kForm, int kAct>
__global__ void __launch_bounds__(kMxThreads, 1) k_expert_gemm_e4m3(const __grid_constant__ MxParams g) {
  extern __shared__ uint8_t raw[];
  uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  MxShared& sh = *reinterpret_cast<MxShared*>(stages + kMxStages * kMxStageBytes);
  constexpr int kCols = kForm == kGlu ? 128 : 256;
  constexpr uint32_t kIdesc = umma_idesc_mx8(kMxTileM, kMxTileN);

  const ProductParams& p = g.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blocks = p.K / kFp8Block;

  if (warp == 2) tmem_alloc<1>(&sh.tmem, 512);
  if (threadIdx.x == 0) {
    prefetch_map(&g.a);
    prefetch_map(&g.a_small);
    prefetch_map(&g.b);
    for (int s = 0; s < kMxStages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.scaled[s], 4);
      mbar_init(&sh.empty[s], 1);
    }
    mbar_init(&sh.sums_full, 1);
    mbar_init(&sh.sums_empty, 8);
    for (int i = 0; i < kTiles; ++i) {
      mbar_init(&sh.ring.full[i], 1);
      mbar_init(&sh.ring.empty[i], 3 + 4 + 8);   // copies (two), products, scale warps, epilogue warps
    }
    fence_barrier_init();
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (p.early) pdl_launch_dependents();
  pdl_wait();   // all that follows reads what kernels before this one may have written
  const uint32_t tmem = sh.tmem;

  bool ok = true;
  uint32_t taken = 0;
  Tile t = {};
  if (warp == 0 || warp == 3) {   // the weights; the rows: converged warps, one lane issues
    const bool issue = elect_one();
    const uint32_t stage0 = smem_addr(stages);
    uint32_t s = 0, phase = 0;
    while (next_tile(sh.ring, taken, t, ok, lane)) {
      const int boxes = (t.rows + kMxBox - 1) / kMxBox, row = t.start + t.m0;
      for (int kb = 0; kb < blocks; ++kb) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.empty[s], phase ^ 1));
        if (!ok) break;
        if (issue) {
          const uint32_t sa = stage0 + s * kMxStageBytes, sb = sa + kMxABytes, bar = smem_addr(&sh.full[s]);
          const int k0 = kb * kFp8Block;
          if (warp == 0) {
            mbar_arrive_expect_tx(&sh.full[s], kMxBBytes + boxes * (kMxABytes / 4));
            if (kForm == kGlu)
              tma_load_4d(sb, &g.b, bar, k0, t.n0, 0, t.e);
            else
              tma_load_3d<false>(sb, &g.b, bar, k0, t.n0, t.e);
          } else if (boxes == 4) {
            tma_load_3d<false>(sa, &g.a, bar, k0, row, 0);
          } else {
            for (int i = 0; i < boxes; ++i)
              tma_load_3d<false>(sa + i * (kMxABytes / 4), &g.a_small, bar, k0, row + i * kMxBox, 0);
          }
        }
        if (++s == kMxStages) {
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
  } else if (warp == 1) {
    // the whole warp walks along, so that addresses stay uniform; one lane issues
    const bool issue = elect_one();
    const uint32_t a0 = umma_desc_lo(smem_addr(stages), 16), b0 = umma_desc_lo(smem_addr(stages) + kMxABytes, 16);
    uint32_t s = 0, phase = 0, n = 0;
    while (next_tile(sh.ring, taken, t, ok, lane)) {
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.sums_empty, (n & 1) ^ 1));
      if (!ok) break;
      ++n;
      tmem_fence_after();
      for (int kb = 0; kb < blocks; ++kb) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.full[s], phase) && mbar_wait_bounded(&sh.scaled[s], phase));
        if (!ok) break;
        tmem_fence_after();
        if (issue) {
          const uint32_t a = a0 + s * (kMxStageBytes >> 4), b = b0 + s * (kMxStageBytes >> 4);
          const uint32_t sc = tmem + kMxScaleCol + s * kMxScaleCols;
#pragma unroll
          for (uint32_t i = 0; i < kFp8Block / 32; ++i)
            umma_mx8(tmem, a + i * (32 >> 4), b + i * (32 >> 4), kIdesc, sc, sc + kMxScaleB, kb > 0 || i > 0);
          umma_commit(&sh.empty[s]);
        }
        if (++s == kMxStages) {
          s = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
      if (issue) umma_commit(&sh.sums_full);
    }
  } else if (warp == 2) {
    TileWalk walk;
    walk.begin(p.seg, -1, kMxTileM, g.tiles_n, kCols, blockIdx.x == 0, lane);
    ok = feed_tiles(sh.ring, walk, walk.at(blockIdx.x, lane), blockIdx.x, gridDim.x, lane);
  } else if (warp >= 8 && warp < 12) {
    // ---------------------------------------------------------------- scales
    int s = 0;
    uint32_t phase = 0;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    while (next_tile(sh.ring, taken, t, ok, lane)) {
      const int64_t owner = t.start / p.seg.cap;
      const uint8_t* xs = p.a_scales + owner * blocks * p.seg.cap + (t.start - owner * p.seg.cap) + t.m0 + lane;
      const uint8_t* ws[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t col = kForm == kGlu ? (int64_t)(2 * t.e + i) * (p.N / kFp8Block) + t.n0 / kFp8Block
                                          : (int64_t)t.e * (p.N / kFp8Block) + t.n0 / kFp8Block + i;
        ws[i] = p.b_scales + col * blocks;
      }
      const bool second = kForm == kGlu || t.n0 + 128 < p.N;
      auto read = [&](int kb) {
        MxScales v;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v.a[j] = kb < blocks && 32 * j + lane < t.rows ? __ldg(xs + (int64_t)kb * p.seg.cap + 32 * j) : (uint8_t)0;
        v.b[0] = kb < blocks ? __ldg(ws[0] + kb) : (uint8_t)0;
        v.b[1] = kb < blocks && second ? __ldg(ws[1] + kb) : (uint8_t)0;
        return v;
      };
      MxScales now[kMxAhead];
#pragma unroll
      for (int i = 0; i < kMxAhead; ++i) now[i] = read(i);
      for (int k0 = 0; ok && k0 < blocks; k0 += kMxAhead) {
        MxScales next[kMxAhead];
#pragma unroll
        for (int i = 0; i < kMxAhead; ++i) next[i] = read(k0 + kMxAhead + i);
#pragma unroll
        for (int i = 0; i < kMxAhead; ++i) {
          if (ok && k0 + i < blocks) {
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.empty[s], phase ^ 1));
            if (ok) {
              const uint32_t sc = lanes + kMxScaleCol + s * kMxScaleCols;
              const uint32_t b0 = now[i].b[0] * 0x01010101u, b1 = now[i].b[1] * 0x01010101u;
              tmem_st4(sc, now[i].a[0] * 0x01010101u, now[i].a[1] * 0x01010101u, now[i].a[2] * 0x01010101u,
                       now[i].a[3] * 0x01010101u);
              tmem_st4(sc + kMxScaleB, b0, b0, b0, b0);
              tmem_st4(sc + kMxScaleB + 4, b1, b1, b1, b1);
              tmem_wait_st();
              tmem_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&sh.scaled[s]);
              if (++s == kMxStages) {
                s = 0;
                phase ^= 1;
              }
            }
          }
          now[i] = next[i];
        }
      }
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3, side = warp >= 12 ? 1 : 0;   // 32 rows; which half of the columns
    const int first = side * (kCols / 2);
    uint32_t n = 0;
    const uint32_t d = tmem + ((uint32_t)(q * 32) << 16);
    while (next_tile(sh.ring, taken, t, ok, lane)) {
      const int r = q * 32 + lane;
      const bool in = r < t.rows, quantised = kForm == kGlu && p.out_scales != nullptr;
      // with scales the two warps of a row meet below, so they give up together
      ok = mbar_wait_bounded(&sh.sums_full, n & 1, kWaitNs + (uint64_t)blocks * 2000);
      ok = quantised ? named_barrier_and(1 + q, 64, ok) : __all_sync(0xffffffffu, ok);
      if (!ok) break;
      ++n;
      tmem_fence_after();
      auto sums_read = [&]() {   // the next tile's products may have them
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.sums_empty);
      };
      if (q * 32 >= t.rows) {   // none of this warp's rows
        sums_read();
        continue;
      }
      const int64_t row = (int64_t)t.start + t.m0 + r;
      float v[32], u[32];
      float mul = 1.0f;
      if (quantised) {   // the row's largest output first: its 128 columns are one scale block
        float amax = 0.0f;
#pragma unroll 1
        for (int c0 = first; c0 < first + kCols / 2; c0 += 32) {
          tmem_ld32(d + c0, v);
          tmem_ld32(d + 128 + c0, u);
          tmem_wait_ld(v, u);
#pragma unroll
          for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(act_value<kAct>(v[i]) * u[i]));
        }
        sh.amax[side][r] = amax;
        named_barrier_sync(1 + q, 64);
        const uint32_t byte = ue8m0_of(fmaxf(amax, sh.amax[side ^ 1][r]));
        mul = __uint_as_float((254u - byte) << 23);
        if (in && side == 0) {
          const int64_t owner = row / p.seg.cap;
          p.out_scales[(owner * (p.N / kFp8Block) + t.n0 / kFp8Block) * p.seg.cap + (row - owner * p.seg.cap)] = (uint8_t)byte;
        }
      }
#pragma unroll 1
      for (int c0 = first; c0 < first + kCols / 2; c0 += 32) {
        tmem_ld32(d + c0, v);
        if constexpr (kForm == kGlu) {
          tmem_ld32(d + 128 + c0, u);
          tmem_wait_ld(v, u);
        } else {
          tmem_wait_ld(v);
        }
        if (c0 + 32 == first + kCols / 2) sums_read();
        if (in) {
          if (quantised) {
            uint8_t* out = static_cast<uint8_t*>(p.out) + row * p.N + t.n0 + c0;
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float z[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) z[j] = __fmul_rn(act_value<kAct>(v[4 * i + j]) * u[4 * i + j], mul);
              w[i] = cvt_e4m3x2(z[0], z[1]) | (cvt_e4m3x2(z[2], z[3]) << 16);
            }
            st_v4(out, make_uint4(w[0], w[1], w[2], w[3]));
            st_v4(out + 16, make_uint4(w[4], w[5], w[6], w[7]));
          } else {
            store32<kForm, kAct>(p, t.e, row, t.n0 + c0, v, u);
          }
        }
        __syncwarp();
      }
    }
  }
  if (!ok) set_status(p.seg.status, EP_ERR_TIMEOUT);
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == 2) tmem_free<1>(tmem, 512);
}

template <int kForm, int kAct>
static int launch_mx_t(const MxParams& g, int64_t tiles, cudaStream_t stream) {
  const int smem = kMxStages * kMxStageBytes + (int)sizeof(MxShared) + 1024;
  const void* fn = reinterpret_cast<const void*>(k_expert_gemm_e4m3<kForm, kAct>);
  if (ep_host::ensure_max_smem(fn, smem) != EP_OK) return EP_ERR_CUDA;
  const int grid = (int)std::min<int64_t>(tiles, ep_host::grid_cap(1));
  if (ep_host::launch_dependent(k_expert_gemm_e4m3<kForm, kAct>, grid, kMxThreads, smem, stream, g) != EP_OK)
    return EP_ERR_CUDA;
  ep_host::count_launch();
  return ep_host::check_launch();
}

template <int kForm>
static int launch_mx_act(const MxParams& g, int64_t tiles, int act, cudaStream_t s) {
  switch (act) {
    case EP_ACT_RELU: return launch_mx_t<kForm, EP_ACT_RELU>(g, tiles, s);
    case EP_ACT_SILU: return launch_mx_t<kForm, EP_ACT_SILU>(g, tiles, s);
    default: return launch_mx_t<kForm, EP_ACT_GELU>(g, tiles, s);
  }
}

int launch_gemm_e4m3(Form form, const ProductParams& p, int act, cudaStream_t stream) {
  MxParams g;
  g.p = p;
  const uint64_t K = (uint64_t)p.K, N = (uint64_t)p.N, rows = (uint64_t)p.rows, E = (uint64_t)p.seg.E;
  const uint64_t ad[3] = {K, rows, 1}, as[2] = {K, K * rows};
  const uint32_t big[3] = {kFp8Block, kMxTileM, 1}, small[3] = {kFp8Block, kMxBox, 1};
  int rc = ep_host::make_map(&g.a, true, 3, p.a, ad, as, big);
  if (rc == EP_OK) rc = ep_host::make_map(&g.a_small, true, 3, p.a, ad, as, small);
  if (form == kGlu) {   // 128 columns of gate and the same of up
    const uint64_t bd[4] = {K, N, 2, E}, bs[3] = {K, K * N, 2 * K * N};
    const uint32_t box[4] = {kFp8Block, kMxTileN / 2, 2, 1};
    if (rc == EP_OK) rc = ep_host::make_map(&g.b, true, 4, p.b, bd, bs, box);
  } else {
    const uint64_t bd[3] = {K, N, E}, bs[2] = {K, K * N};
    const uint32_t box[3] = {kFp8Block, kMxTileN, 1};
    if (rc == EP_OK) rc = ep_host::make_map(&g.b, true, 3, p.b, bd, bs, box);
  }
  if (rc != EP_OK) return rc;
  const int cols = form == kGlu ? 128 : 256;
  g.tiles_n = (p.N + cols - 1) / cols;
  const int64_t tiles = (p.rows / kMxTileM + p.seg.E) * g.tiles_n;   // at most one ragged row tile an expert
  if (form == kGlu) return launch_mx_act<kGlu>(g, tiles, act, stream);
  return act == EP_ACT_NONE ? launch_mx_t<kLinear, EP_ACT_NONE>(g, tiles, stream)
                            : launch_mx_act<kLinear>(g, tiles, act, stream);
}

}  // namespace ep
