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
  bool early;                // the next kernel of the stream may come up while this one runs
};

// One tile of the list: output rows m0 .. m0 + rows of expert e (numbered inside
// its segment; kDw: inside its weights) and output columns from n0 on.  e < 0:
// past the last.
struct Tile {
  int e, m0, rows, n0;
  int start, count;   // segment
};

constexpr int kGroupM = 16;   // row tiles taken together

// Walks the list of all experts' tiles; one warp, converged.  An expert has
// ceil(rows / tile_rows) row tiles, its rows spread over them in units of 32, and
// tiles_n column tiles of `cols`; 16 row tiles are taken together, column after
// column.  Looks at 32 experts at a time, so that nothing has to be kept for
// all of them.
struct TileWalk {
  Segments seg;
  int fixed_rows;   // output rows where they are not the segment's (kDw), else -1
  int tile_rows, tiles_n, cols;
  int e0;           // first of the 32 experts looked at
  int64_t before;   // tiles of the experts below e0
  Segment s;        // this lane's expert
  int rows, upto;   // its output rows; row tiles of the lanes up to it

  __device__ __forceinline__ void look(int at, int lane) {
    e0 = at;
    s = {0, 0};
    rows = 0;
    if (e0 + lane < seg.E) {
      s = segment_of(seg, e0 + lane);
      rows = fixed_rows >= 0 ? fixed_rows : s.count;
    }
    upto = (rows + tile_rows - 1) / tile_rows;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
  }

  // report: this warp records a segment that was cut.
  __device__ __forceinline__ void begin(const Segments& segments, int fixed, int tile, int n, int c, bool report, int lane) {
    seg = segments;
    if (!report) seg.status = nullptr;
    fixed_rows = fixed;
    tile_rows = tile;
    tiles_n = n;
    cols = c;
    before = 0;
    look(0, lane);
  }

  // Tile number t (not below the last one asked for).
  __device__ __forceinline__ Tile at(int64_t t, int lane) {
    Tile out = {-1, 0, 0, 0, 0, 0};
    for (;;) {
      const int64_t all = (int64_t)__shfl_sync(0xffffffffu, upto, 31) * tiles_n;
      if (t < before + all) break;
      if (e0 + 32 >= seg.E) return out;
      before += all;
      look(e0 + 32, lane);
    }
    const int who = __ffs(__ballot_sync(0xffffffffu, t < before + (int64_t)upto * tiles_n)) - 1;
    const int tiles_m = __shfl_sync(0xffffffffu, (rows + tile_rows - 1) / tile_rows, who);
    // 32-bit divisions: the tiles of one expert's output are far below 2^31 (each is 64 KB or more of it)
    const uint32_t in = (uint32_t)(t - before - (int64_t)(__shfl_sync(0xffffffffu, upto, who) - tiles_m) * tiles_n);
    const int of = __shfl_sync(0xffffffffu, rows, who);
    out.e = e0 + who;
    out.start = __shfl_sync(0xffffffffu, (int)s.start, who);
    out.count = __shfl_sync(0xffffffffu, s.count, who);
    const uint32_t group = in / (uint32_t)(kGroupM * tiles_n);
    const uint32_t r = in - group * (uint32_t)(kGroupM * tiles_n);
    const uint32_t gm = (uint32_t)min(kGroupM, tiles_m - (int)group * kGroupM);
    const uint32_t column = r / gm;
    const int i = (int)(group * kGroupM + r - column * gm);
    const int units = (int)((uint32_t)(of + 31) / 32u);
    const int each = (int)((uint32_t)units / (uint32_t)tiles_m), more = units - each * tiles_m;
    out.n0 = (int)column * cols;
    out.m0 = (i * each + min(i, more)) * 32;
    out.rows = min(of, out.m0 + (each + (i < more ? 1 : 0)) * 32) - out.m0;
    return out;
  }
};

// The looked-up tiles on their way from the warp that walks the list to the
// other warps of the CTA.
constexpr int kTiles = 4;
constexpr uint64_t kTileWaitNs = 30 * kWaitNs;   // a reader may be as far behind as a tile takes
struct TileRing {
  uint64_t full[kTiles], empty[kTiles];
  Tile tiles[kTiles];
};

// The next tile for a converged warp; false past the last one, or (ok false) when
// the wait ran out.
__device__ __forceinline__ bool next_tile(TileRing& ring, uint32_t& taken, Tile& t, bool& ok, int lane) {
  if (!ok) return false;
  const uint32_t i = taken % kTiles;
  ok = __all_sync(0xffffffffu, mbar_wait_bounded(&ring.full[i], (taken / kTiles) & 1, kTileWaitNs));
  if (!ok) return false;
  t = ring.tiles[i];
  ++taken;
  __syncwarp();
  if (lane == 0) mbar_arrive(&ring.empty[i]);
  return t.e >= 0;
}
// The walking warp: tiles first (which is t), first + step, ... until the list
// ends.
__device__ __forceinline__ bool feed_tiles(TileRing& ring, TileWalk& walk, Tile t, int64_t first, int64_t step, int lane) {
  for (uint32_t n = 0;; ++n) {
    const uint32_t i = n % kTiles;
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(&ring.empty[i], ((n / kTiles) & 1) ^ 1, kTileWaitNs))) return false;
    if (lane == 0) {
      ring.tiles[i] = t;
      mbar_arrive(&ring.full[i]);
    }
    if (t.e < 0) return true;
    first += step;
    t = walk.at(first, lane);
  }
}

int launch_gemm_bf16(Form form, const ProductParams& p, int act, cudaStream_t stream);
int launch_gemm_e4m3(Form form, const ProductParams& p, int act, cudaStream_t stream);

}  // namespace ep
