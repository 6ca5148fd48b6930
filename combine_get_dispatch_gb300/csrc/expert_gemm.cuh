// expert_gemm.cuh -- what the product kernels share: arguments, the list of
// tiles over the experts' segments, the epilogue of a row.
#pragma once

#include "expert.cuh"

namespace ep {

enum Form { kGlu, kLinear, kDx, kDw };

struct ProductParams {
  Segments seg;
  int64_t rows;              // of the whole layout
  const void* a;             // rows operand
  const uint8_t* a_scales;
  const void* b;             // weights, or the second rows operand (kDw)
  const uint8_t* b_scales;
  int N, K;                  // output columns, inner extent (kDw: output rows K)
  const __nv_bfloat16* bias;
  const __nv_bfloat16* residual;
  void* out;
  uint8_t* out_scales;
  __nv_bfloat16* keep;       // gu / pre
};

// One tile of the list: output rows m0 .. m0 + rows of expert e (numbered inside
// its segment; kDw: inside its weights) and output columns from n0 on.
struct Tile {
  int e, m0, rows, n0;
  int start, count;   // segment
};

constexpr int kGroupM = 8;   // row tiles taken together

struct TileTable {
  int32_t warp_total[32];
  int32_t first_tile[kMaxE + 1];   // row tiles of the experts before e
  int32_t start[kMaxE], count[kMaxE];
};

// Row tiles before each expert, and the segments, in shared memory.
// fixed_rows: the output's rows where they are not the segment's (kDw), else -1.
template <int kTileM, int kThreads>
__device__ __forceinline__ void build_table(TileTable& sh, Segments seg, int fixed_rows, bool report) {
  const int E = seg.E, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int base = 0;
  if (!report) seg.status = nullptr;   // one CTA reports a segment that was cut
  for (int e0 = 0; e0 < E; e0 += kThreads) {
    const int e = e0 + tid;
    int tiles = 0;
    if (e < E) {
      const Segment s = segment_of(seg, e);
      sh.start[e] = (int)s.start;
      sh.count[e] = s.count;
      tiles = ((fixed_rows >= 0 ? fixed_rows : s.count) + kTileM - 1) / kTileM;
    }
    int incl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sh.warp_total[warp] = incl;
    __syncthreads();
    int before = base, all = base;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += sh.warp_total[w];
      all += sh.warp_total[w];
    }
    if (e < E) sh.first_tile[e] = before + incl - tiles;
    base = all;
    __syncthreads();
  }
  if (tid == 0) sh.first_tile[E] = base;
  __syncthreads();
}

// Tile number t of the list, false past its end.
template <int kTileM, bool kEven>
__device__ __forceinline__ bool tile_at(const TileTable& sh, int E, int fixed_rows, int tiles_n, int cols, int64_t t,
                                        Tile& out) {
  const int64_t total = (int64_t)sh.first_tile[E] * tiles_n;
  if (t >= total) return false;
  int lo = 0, hi = E;   // last expert whose first tile is at or before t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)sh.first_tile[mid] * tiles_n <= t)
      lo = mid;
    else
      hi = mid;
  }
  // experts without tiles share a first tile with the next: lo is the last of them, the one that has it
  const int tiles_m = sh.first_tile[lo + 1] - sh.first_tile[lo];
  const int64_t in = t - (int64_t)sh.first_tile[lo] * tiles_n;
  const int64_t group = in / ((int64_t)kGroupM * tiles_n);
  const int gm = min(kGroupM, tiles_m - (int)group * kGroupM);
  const int64_t r = in - group * kGroupM * tiles_n;
  out.e = lo;
  out.start = sh.start[lo];
  out.count = sh.count[lo];
  out.n0 = (int)(r / gm) * cols;
  const int of = fixed_rows >= 0 ? fixed_rows : out.count;
  const int i = (int)group * kGroupM + (int)(r % gm);
  if (kEven) {   // an expert's rows are spread over its row tiles in units of 16
    const int64_t units = (of + 15) / 16;
    out.m0 = (int)(units * i / tiles_m) * 16;
    out.rows = min(of, (int)(units * (i + 1) / tiles_m) * 16) - out.m0;
  } else {
    out.m0 = i * kTileM;
    out.rows = min(kTileM, of - out.m0);
  }
  return true;
}

// Eight fp32 sums -> 16 bytes of bf16.
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// The epilogue of 8 columns from n on of output row `row` of expert e: z the sums
// (kGlu: of the gate), u those of the up projection.
template <int kForm, int kAct>
__device__ __forceinline__ void store8(const ProductParams& p, int e, int64_t row, int n, float (&z)[8],
                                       const float* u) {
  if (kForm == kGlu) {
    if (p.keep != nullptr) {
      st_v4(p.keep + row * 2 * p.N + n, pack8(z));
      st_v4(p.keep + (row * 2 + 1) * p.N + n, pack8(u));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = act_value<kAct>(z[i]) * u[i];
  } else if (kForm == kLinear) {
    if (p.bias != nullptr) {
      const uint4 b = __ldg(reinterpret_cast<const uint4*>(p.bias + (int64_t)e * p.N + n));
      const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        z[2 * i] += bf16_lo(w[i]);
        z[2 * i + 1] += bf16_hi(w[i]);
      }
    }
    if (p.keep != nullptr) st_v4(p.keep + row * p.N + n, pack8(z));
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = act_value<kAct>(z[i]);
    if (p.residual != nullptr) {   // may be the output itself: a plain load
      const uint4 r = ld_v4(p.residual + row * p.N + n);
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        z[2 * i] += bf16_lo(w[i]);
        z[2 * i + 1] += bf16_hi(w[i]);
      }
    }
  }
  st_v4(static_cast<__nv_bfloat16*>(p.out) + row * p.N + n, pack8(z));
}

// As store8 for 32 columns that one thread holds, up to the output's last.
template <int kForm, int kAct>
__device__ __forceinline__ void store32(const ProductParams& p, int e, int64_t row, int n0, float (&v)[32],
                                        const float* u) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (n0 + q * 8 >= p.N) break;
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = v[q * 8 + i];
    store8<kForm, kAct>(p, e, row, n0 + q * 8, z, u + q * 8);
  }
}

int launch_gemm_bf16(Form form, const ProductParams& p, int act, cudaStream_t stream);
int launch_gemm_e4m3(Form form, const ProductParams& p, int act, cudaStream_t stream);

}  // namespace ep
