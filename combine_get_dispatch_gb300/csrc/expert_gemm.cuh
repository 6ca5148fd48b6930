// expert_gemm.cuh -- what expert.cu asks of the product kernels.
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

int launch_gemm_bf16(Form form, const ProductParams& p, int act, cudaStream_t stream);

}  // namespace ep
