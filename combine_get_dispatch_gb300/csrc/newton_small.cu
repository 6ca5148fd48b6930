// newton_small.cu -- the orthogonalised update of matrices that fit one SM: all
// steps in one launch, a matrix a CTA.
//
// X (S x L, S the smaller side, turned around on the way in and out where M > N)
// stays in registers, in 32 bits, a thread a row of 64 columns; in shared memory it
// and the polynomial lie as fp16 in the layout that the tensor cores read (128-byte
// swizzle, 64 columns a block), which serves X both as a K-major operand (X X^T) and
// as an MN-major one (P X).  A step is three
// products, tcgen05.mma of one SM, with the epilogue of each by sixteen warps, a row
// a thread.  Bound by latency: a launch a product took 7 us each, 125 us for 32
// matrices of 128 x 256 and five steps; so it is 37 us.

#include "newton.cuh"

namespace ep {

constexpr int kSmallThreads = 512;
constexpr int kSides = kSmallThreads / 128;             // of an epilogue's columns
constexpr int kHeldChunks = kSmallLength / kSides / 32; // of X in a thread's registers, 32 columns each
constexpr int kPart = kSmallThreads;                    // vectors of 8 elements that come in at a time, one a thread
constexpr int kPartBytes = 2 * kPart * 32;              // of gradient and momentum
constexpr int kParts = 3;                               // on their way at a time, where X and the polynomial will be
constexpr int kSmallBlock = 128 * 128;                  // bytes of 128 rows x 64 columns
constexpr int kSmallBytes = kSmallSide * kSmallLength * 4 + (kSmallLength / 64 + kSmallSide / 64) * kSmallBlock;

struct SmallShared {
  uint64_t done, part[kParts];
  uint32_t tmem;
  float sums[kSmallThreads / kWarp];
  float diagonal[kSmallSide];
};

__device__ __forceinline__ void umma_f16(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n"
      " mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"((uint32_t)add), "r"(kDescHi)
      : "memory");
}

// Address of 8 columns from column c on of a row of X or P.
__device__ __forceinline__ uint32_t small_address(uint32_t base, int row, int c) {
  return base + (c >> 6) * kSmallBlock + row * 128 + ((((c >> 3) & 7) ^ (row & 7)) << 4);
}

// Address of element (row, column c) of the 32-bit matrix that is on its way in or out.
__device__ __forceinline__ uint32_t wide_address(uint32_t base, int row, int c) {
  return base + row * (kSmallLength * 4) + ((((c >> 2) ^ (row & 7)) << 4) | ((c & 3) << 2));
}

__global__ void __launch_bounds__(kSmallThreads, 1) k_newton_small(const __grid_constant__ SmallNewton p) {
  extern __shared__ __align__(1024) uint8_t raw[];
  const bool tall = p.M > p.N;
  const int S = tall ? p.N : p.M, L = tall ? p.M : p.N;
  const int blocks = (L + 63) / 64;
  const uint32_t wide = smem_addr(raw), hi = wide + kSmallSide * kSmallLength * 4, poly = hi + kSmallLength / 64 * kSmallBlock;
  SmallShared& sh = *reinterpret_cast<SmallShared*>(raw + kSmallBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = warp & 3, side = warp >> 2, row = q * 32 + lane;   // of the epilogues
  if (threadIdx.x == 0) {
    mbar_init(&sh.done, 1);
    for (int i = 0; i < kParts; ++i) mbar_init(&sh.part[i], 1);
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc<1>(&sh.tmem, 512);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = sh.tmem, t_square = tmem, t_apply = tmem + 128;
  const uint32_t lanes = (uint32_t)(q * 32) << 16;
  if (p.src.early) pdl_launch_dependents();
  pdl_wait();
  bool ok = true;
  uint32_t phase = 0;
  // all threads: what was written here is multiplied by one thread, then everybody goes on
  auto products = [&](auto issue) {
    fence_proxy_async_smem();
    tmem_fence_before();
    __syncthreads();
    bool done = true;
    if (warp == 0) {
      if (elect_one()) {
        tmem_fence_after();
        issue();
        umma_commit(&sh.done);
      }
      __syncwarp();
      done = mbar_wait_bounded(&sh.done, phase);   // one warp; the others wait at the barrier
    }
    ok = __syncthreads_and(done) != 0;
    phase ^= 1;
    tmem_fence_after();
  };
  const int vectors = p.M * p.N / 8, per_row = p.N / 8, parts = (vectors + kPart - 1) / kPart;
  uint32_t parts_seen = 0;
  // part k of up to two arrays of `bytes` a vector, by one thread
  auto bring = [&](int k, const void* a, int a_bytes, const void* b) {
    if (threadIdx.x != 0 || k >= parts) return;
    const uint32_t slot = (parts_seen + k) % kParts;
    const int n = min(kPart, vectors - k * kPart);
    uint8_t* const to = raw + (hi - wide) + slot * kPartBytes;
    mbar_arrive_expect_tx(&sh.part[slot], n * (a_bytes + (b != nullptr ? 32 : 0)));
    tma_load_1d(to, static_cast<const uint8_t*>(a) + (int64_t)k * kPart * a_bytes, n * a_bytes, &sh.part[slot]);
    if (b != nullptr) tma_load_1d(to + kPartBytes / 2, static_cast<const uint8_t*>(b) + (int64_t)k * kPart * 32, n * 32, &sh.part[slot]);
  };
  // part k's momentum or weights, replaced in place, go out by one copy (16 bytes a thread are half sectors, and
  // took three times as long), and the part after next comes in where the last one went out
  auto send = [&](int k, float* to, int offset, const void* a, int a_bytes, const void* b) {
    fence_proxy_async_smem();
    __syncthreads();
    if (threadIdx.x != 0 || !ok) return;
    const int n = min(kPart, vectors - k * kPart);
    if (to != nullptr) {
      tma_store_1d(to + (int64_t)k * kPart * 8, raw + (hi - wide) + (parts_seen + k) % kParts * kPartBytes + offset, n * 32);
      tma_commit();
      tma_wait_read<1>();
    }
    if (k > 0) bring(k - 1 + kParts, a, a_bytes, b);
  };
  // wait for part k; where it is.  A warp whose wait ran out leaves its share there as it comes, so that it goes out as it was
  auto part = [&](int k) {
    const uint32_t at = parts_seen + k;
    ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.part[at % kParts], (at / kParts) & 1, ok ? kWaitNs : 0)) && ok;
    return hi + at % kParts * kPartBytes;
  };

  for (int z = blockIdx.x; ok && z < p.src.count; z += gridDim.x) {
    const int64_t base = (int64_t)z * p.M * p.N;
    // ---------------------------------------------------------------- momentum, norm
    const int g_bytes = p.src.f32 ? 32 : 16;
    const uint8_t* const g = static_cast<const uint8_t*>(p.src.g) + base / 8 * g_bytes;
    const float* const momentum = p.src.m != nullptr ? p.src.m + base : nullptr;
    fence_proxy_async_smem();
    if (threadIdx.x == 0) tma_wait_read<0>();
    __syncthreads();   // nobody uses X and the polynomial of the matrix before
    for (int k = 0; k < kParts; ++k) bring(k, g, g_bytes, momentum);
    // everything is zero where the matrix is not: rows past S, columns past L
    if (S < kSmallSide || L < blocks * 64) {
      for (int i = threadIdx.x; i < kSmallSide * kSmallLength / 4; i += kSmallThreads) st_shared_v4_at(wide + i * 16, make_uint4(0, 0, 0, 0));
      __syncthreads();
    }
    float square = 0.0f;
#pragma unroll 1
    for (int k = 0; k < parts; ++k) {
      const uint32_t at = part(k);
      const int i = k * kPart + threadIdx.x;
      float u[8], m[8];
      auto read8 = [&](uint32_t from, float (&y)[8]) {
        const uint4 v0 = ld_shared_v4_at(from), v1 = ld_shared_v4_at(from + 16);
        y[0] = __uint_as_float(v0.x), y[1] = __uint_as_float(v0.y), y[2] = __uint_as_float(v0.z), y[3] = __uint_as_float(v0.w);
        y[4] = __uint_as_float(v1.x), y[5] = __uint_as_float(v1.y), y[6] = __uint_as_float(v1.z), y[7] = __uint_as_float(v1.w);
      };
      if (p.src.f32) {
        read8(at + threadIdx.x * 32, u);
      } else {
        const uint4 v = ld_shared_v4_at(at + threadIdx.x * 16);
        u[0] = bf16_lo(v.x), u[1] = bf16_hi(v.x), u[2] = bf16_lo(v.y), u[3] = bf16_hi(v.y);
        u[4] = bf16_lo(v.z), u[5] = bf16_hi(v.z), u[6] = bf16_lo(v.w), u[7] = bf16_hi(v.w);
      }
      if (momentum != nullptr) {
        const uint32_t at_m = at + kPartBytes / 2 + threadIdx.x * 32;
        read8(at_m, m);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          m[e] = fmaf(p.src.momentum, m[e], u[e]);
          u[e] = p.src.nesterov ? fmaf(p.src.momentum, m[e], u[e]) : m[e];
        }
        if (ok) st_shared_v4_at(at_m, make_uint4(__float_as_uint(m[0]), __float_as_uint(m[1]), __float_as_uint(m[2]), __float_as_uint(m[3])));
        if (ok) st_shared_v4_at(at_m + 16, make_uint4(__float_as_uint(m[4]), __float_as_uint(m[5]), __float_as_uint(m[6]), __float_as_uint(m[7])));
      }
      send(k, p.src.m != nullptr ? p.src.m + base : nullptr, kPartBytes / 2, g, g_bytes, momentum);
      if (i >= vectors) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) square = fmaf(u[e], u[e], square);
      const int r = i / per_row, c = (i - r * per_row) * 8;
      if (!tall) {
#pragma unroll
        for (int e = 0; e < 8; e += 4)
          st_shared_v4_at(wide_address(wide, r, c + e),
                          make_uint4(__float_as_uint(u[e]), __float_as_uint(u[e + 1]), __float_as_uint(u[e + 2]), __float_as_uint(u[e + 3])));
      } else {   // 8 rows of column r
#pragma unroll
        for (int e = 0; e < 8; ++e) asm volatile("st.shared.f32 [%0], %1;" ::"r"(wide_address(wide, c + e, r)), "f"(u[e]) : "memory");
      }
    }
    parts_seen += parts;
    if (threadIdx.x == 0) tma_wait_read<0>();   // X goes where the momentum comes from
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) square += __shfl_xor_sync(0xffffffffu, square, o);
    if (lane == 0) sh.sums[warp] = square;
    ok = __syncthreads_and(ok) != 0;
    square = 0.0f;
    for (int w = 0; w < kSmallThreads / kWarp; ++w) square += sh.sums[w];
    float up, factor;
    source_scale(square, p.src.eps, up, factor);
    // X: into registers, and as fp16 for the products
    float x[kHeldChunks][32];
    auto store_x = [&](int col, const float* y) {   // 8 columns
      uint32_t h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __half2 v = __floats2half2_rn(y[2 * e], y[2 * e + 1]);
        h[e] = *reinterpret_cast<const uint32_t*>(&v);
      }
      st_shared_v4_at(small_address(hi, row, col), make_uint4(h[0], h[1], h[2], h[3]));
    };
#pragma unroll
    for (int n = 0; n < kHeldChunks; ++n) {
      const int j = (n * kSides + side) * 32;
      if (j < blocks * 64) {
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const uint4 y = ld_shared_v4_at(wide_address(wide, row, j + e));
          x[n][e] = __uint_as_float(y.x) * up, x[n][e + 1] = __uint_as_float(y.y) * up;
          x[n][e + 2] = __uint_as_float(y.z) * up, x[n][e + 3] = __uint_as_float(y.w) * up;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) store_x(j + 8 * k, &x[n][8 * k]);
      }
    }
    // ---------------------------------------------------------------- steps
#pragma unroll 1
    for (int t = 0; ok && t < p.steps; ++t) {
      const float a = p.abc[3 * t], b = p.abc[3 * t + 1], c = p.abc[3 * t + 2];
      const float f = t == 0 ? factor : 1.0f;
      const uint32_t k_major = umma_idesc_f16(128, 128, false, false);
      products([&] {
        const uint32_t at0 = umma_desc_lo(hi, 16);
        for (int k = 0; k < (L + 15) / 16; ++k) {
          const uint32_t at = at0 + (((k >> 2) * kSmallBlock + (k & 3) * 32) >> 4);
          umma_f16(tmem, at, at, k_major, k > 0);
        }
      });
      if (!ok) break;
      // 8 columns of A, or of the polynomial, whose diagonal is kept apart
      auto store_poly = [&](int col, float (&y)[8], bool last) {
        if (last && (row & ~7) == col) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (col + e == row) {
              sh.diagonal[row] = y[e] * (1.0f / kHeld);
              y[e] = 0.0f;
            }
        }
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __half2 v = __floats2half2_rn(y[2 * e], y[2 * e + 1]);
          h[e] = *reinterpret_cast<const uint32_t*>(&v);
        }
        st_shared_v4_at(small_address(poly, row, col), make_uint4(h[0], h[1], h[2], h[3]));
      };
      const float gram_scale = f * f / kHeld * (c != 0.0f ? 1.0f : b), square_scale = c / kHeld;
#pragma unroll 1
      for (int j = side * 32; j < side * 32 + 32; j += 16) {
        float v[16];
        tmem_ld16(tmem + lanes + j, v);
        tmem_wait_ld(v);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = v[8 * k + e] * gram_scale;
          store_poly(j + 8 * k, y, c == 0.0f);
        }
      }
      if (c != 0.0f) {
        products([&] {
          const uint32_t at0 = umma_desc_lo(poly, 16);
          for (int k = 0; k < (S + 15) / 16; ++k) {
            const uint32_t at = at0 + (((k >> 2) * kSmallBlock + (k & 3) * 32) >> 4);
            umma_f16(t_square, at, at, k_major, k > 0);
          }
        });
        if (!ok) break;
#pragma unroll 1
        for (int j = side * 32; j < side * 32 + 32; j += 16) {
          float v[16];
          tmem_ld16(t_square + lanes + j, v);
          tmem_wait_ld(v);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint4 r = ld_shared_v4_at(small_address(poly, row, j + 8 * k));
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
            float y[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 A = floats_of(w[e]);
              y[2 * e] = fmaf(b, A.x, v[8 * k + 2 * e] * square_scale);
              y[2 * e + 1] = fmaf(b, A.y, v[8 * k + 2 * e + 1] * square_scale);
            }
            store_poly(j + 8 * k, y, true);
          }
        }
      }
      products([&] {
        // X's rows are the inner index: MN-major, 64 columns a block
        const uint32_t pa = umma_desc_lo(poly, 16), at0 = umma_desc_lo(hi, kSmallBlock), idesc = umma_idesc_f16(128, blocks * 64, false, true);
        for (int k = 0; k < (S + 15) / 16; ++k)
          umma_f16(t_apply, pa + (((k >> 2) * kSmallBlock + (k & 3) * 32) >> 4), at0 + (k * 2048 >> 4), idesc, k > 0);
      });
      if (!ok) break;
      const float add = (a + sh.diagonal[row]) * f, scale = f / kHeld;
#pragma unroll
      for (int n = 0; n < kHeldChunks; ++n) {
        const int j = (n * kSides + side) * 32;
        if (j < blocks * 64) {
#pragma unroll
          for (int i = 0; i < 32; i += 16) {
            float v[16];
            tmem_ld16(t_apply + lanes + j + i, v);
            tmem_wait_ld(v);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[n][i + e] = fmaf(add, x[n][i + e], v[e] * scale);
            if (t + 1 < p.steps) {
              store_x(j + i, &x[n][i]);
              store_x(j + i + 8, &x[n][i + 8]);
            }
          }
        }
      }
    }
    if (!ok) break;
    // ---------------------------------------------------------------- out
    float* const w = p.out == nullptr ? p.w + base : nullptr;
    if (w != nullptr) {
      fence_proxy_async_smem();
      __syncthreads();
      for (int k = 0; k < kParts; ++k) bring(k, w, 32, nullptr);
    }
#pragma unroll
    for (int n = 0; n < kHeldChunks; ++n) {
      const int j = (n * kSides + side) * 32;
      if (j < blocks * 64) {
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          st_shared_v4_at(wide_address(wide, row, j + e),
                          make_uint4(__float_as_uint(x[n][e] * (1.0f / kHeld)), __float_as_uint(x[n][e + 1] * (1.0f / kHeld)),
                                     __float_as_uint(x[n][e + 2] * (1.0f / kHeld)), __float_as_uint(x[n][e + 3] * (1.0f / kHeld))));
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int k = 0; k < parts; ++k) {
      const int i = k * kPart + threadIdx.x;
      const int r = i / per_row, c = (i - r * per_row) * 8;
      const bool in = i < vectors;
      float y[8] = {};
      if (in && !tall) {
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const uint4 v = ld_shared_v4_at(wide_address(wide, r, c + e));
          y[e] = __uint_as_float(v.x), y[e + 1] = __uint_as_float(v.y), y[e + 2] = __uint_as_float(v.z), y[e + 3] = __uint_as_float(v.w);
        }
      } else if (in) {
#pragma unroll
        for (int e = 0; e < 8; ++e) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(y[e]) : "r"(wide_address(wide, c + e, r)) : "memory");
      }
      __nv_bfloat16* to = p.out;
      if (w != nullptr) {
        const uint32_t at = part(k) + threadIdx.x * 32;
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const uint4 v = ld_shared_v4_at(at + e * 4);
          y[e] = fmaf(-p.step, y[e], p.keep * __uint_as_float(v.x)), y[e + 1] = fmaf(-p.step, y[e + 1], p.keep * __uint_as_float(v.y));
          y[e + 2] = fmaf(-p.step, y[e + 2], p.keep * __uint_as_float(v.z)), y[e + 3] = fmaf(-p.step, y[e + 3], p.keep * __uint_as_float(v.w));
          if (ok) st_shared_v4_at(at + e * 4, make_uint4(__float_as_uint(y[e]), __float_as_uint(y[e + 1]), __float_as_uint(y[e + 2]), __float_as_uint(y[e + 3])));
        }
        send(k, w, 0, w, 32, nullptr);
        to = p.w16;
      }
      if (in && ok && to != nullptr)
        st_v4(to + base + (int64_t)i * 8, make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7])));
    }
    if (w != nullptr) parts_seen += parts;
    ok = __syncthreads_and(ok) != 0;   // the next matrix comes in
  }
  if (threadIdx.x == 0) tma_wait_all();
  if (!ok) {
    set_status(p.status, EP_ERR_TIMEOUT);
    const uint64_t t0 = globaltimer_ns();   // give the copies in flight time to land before the memory goes
    while (globaltimer_ns() - t0 < 2000000ull) {
    }
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == 0) tmem_free<1>(tmem, 512);
}

int launch_newton_small(const SmallNewton& p, cudaStream_t stream) {
  constexpr int kSmem = kSmallBytes + (int)sizeof(SmallShared);
  if (ep_host::ensure_max_smem(reinterpret_cast<const void*>(k_newton_small), kSmem) != EP_OK) return EP_ERR_CUDA;
  if (ep_host::launch_in_budget(k_newton_small, std::min(p.src.count, ep_host::grid_cap(1)), kSmallThreads, kSmem, stream, p) != EP_OK) return EP_ERR_CUDA;
  ep_host::count_launch();
  return ep_host::check_launch();
}

}  // namespace ep
