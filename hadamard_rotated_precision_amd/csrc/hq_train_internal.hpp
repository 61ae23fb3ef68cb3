// hq_train_internal.hpp — launchers shared between the kernel files of include/hq_train.h and
// their C-ABI layer (plain host C++).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/hq_train.h"
#include "hq_internal.hpp"

namespace hq {

// Block quantizer (hq_block.hip). codes or codes_t may be null, not both.
struct BlockQuantPass {
  const void* src = nullptr;
  int in_dt = 0;
  int64_t rows = 0, cols = 0;
  bool tiles = false, pow2 = false;
  uint8_t* codes = nullptr;
  int64_t ld = 0;
  uint8_t* codes_t = nullptr;
  int64_t ld_t = 0;
  float* scales = nullptr;
  int64_t lds = 0;
  float* scales_t = nullptr;
  int64_t lds_t = 0;
};
hipError_t block_quant_pass(const BlockQuantPass& p, hipStream_t st);

// One operand of a block-scaled product: rows x K code bytes, and the scale of (row, kb) at
// scales[(tiles ? row / 128 : row) * sg + kb * sk].
struct BlockOperand {
  const uint8_t* codes = nullptr;
  int64_t ld = 0;
  const float* scales = nullptr;
  int64_t sg = 0, sk = 0;
  bool tiles = false, pow2 = false;
};

// c[m][n] (+)= sum_kb sa sb sum_k a[m][k] b[n][k] (hq_block_gemm.hip); c contiguous M x N.
struct BlockGemmPass {
  BlockOperand a, b;
  int64_t M = 0, N = 0, K = 0;
  void* c = nullptr;
  int out_dt = 0;
  bool accumulate = false;
  void* ws = nullptr;
};
size_t block_gemm_ws(int64_t M, int64_t N, int64_t K);
hipError_t block_gemm_pass(const BlockGemmPass& p, hipStream_t st);

// The product for few rows of a (hq_block_gemv.hip; block_gemm_pass uses it where block_gemv_ok).
// x given: a is the M x K matrix x of type x_dt, quantized within (ROWS blocks, scale kind pow2);
// block_gemv_fused_ok has to hold.
bool block_gemv_ok(int64_t M, int64_t N, int64_t K);
bool block_gemv_fused_ok(int64_t M, int64_t K);
hipError_t block_gemv_pass(const BlockGemmPass& p, const void* x, int x_dt, bool pow2, hipStream_t st);

// AdamW over tensors (hq_adamw.hip): pointers and lengths are checked, lengths above zero.
hipError_t adamw_pass(const hq_adamw_tensor* t, int count, const hq_adamw_config& cfg,
                      const hq_adamw_scalars& host, const hq_adamw_scalars* device,
                      hipStream_t st);

}  // namespace hq
