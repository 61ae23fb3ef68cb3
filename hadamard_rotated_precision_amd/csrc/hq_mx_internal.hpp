// hq_mx_internal.hpp — launchers shared between the kernel files of include/hq_mx.h and their C-ABI
// layer (plain host C++).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/hq_mx.h"
#include "hq_internal.hpp"

namespace hq {

inline int64_t mx_blocks(int64_t n) { return (n + HQ_MX_BLOCK - 1) / HQ_MX_BLOCK; }

// Quantizer (hq_mx.hip). codes or codes_t may be null, not both.
struct MxQuantPass {
  const void* src = nullptr;
  int in_dt = 0;
  int64_t rows = 0, cols = 0;
  int rot = 1;
  const uint32_t* seed = nullptr;
  uint8_t *codes = nullptr, *codes_t = nullptr;
  uint8_t *scales = nullptr, *scales_t = nullptr;
  int64_t ld = 0, ld_t = 0, lds = 0, lds_t = 0;
};
hipError_t mx_quant_pass(const MxQuantPass& p, hipStream_t st);

// One layout of a tensor: rows x K codes and their scale bytes.
struct MxOperand {
  const uint8_t* codes = nullptr;
  int64_t ld = 0;
  const uint8_t* scales = nullptr;
  int64_t lds = 0;
};
hipError_t mx_dequant_pass(const MxOperand& q, int64_t rows, int64_t cols, int rot, void* dst,
                           int out_dt, hipStream_t st);

// c[m][n] (+)= alpha sum_k a[m][k] b[n][k] (hq_mx_gemm.hip); c contiguous M x N.
struct MxGemmPass {
  MxOperand a, b;
  int64_t M = 0, N = 0, K = 0;
  float alpha = 1.0f;
  void* c = nullptr;
  int out_dt = 0;
  bool accumulate = false;
  void* ws = nullptr;
};
size_t mx_gemm_ws(int64_t M, int64_t N, int64_t K);
hipError_t mx_gemm_pass(const MxGemmPass& p, hipStream_t st);

// The product for few rows of a (hq_mx_gemv.hip; mx_gemm_pass uses it where mx_gemv_ok). x given: a
// is the M x K matrix x of type x_dt, rotated and quantized within (to nearest); mx_gemv_fused_ok
// has to hold.
bool mx_gemv_ok(int64_t M, int64_t N, int64_t K);
bool mx_gemv_fused_ok(int64_t M, int64_t K);
hipError_t mx_gemv_pass(const MxGemmPass& p, const void* x, int x_dt, int rot, hipStream_t st);

// The cache (hq_kv.hip).
struct KvAppendPass {
  const void *k = nullptr, *v = nullptr;
  int dt = 0;
  int64_t tokens = 0;
  int64_t k_token = 0, k_head = 0, v_token = 0, v_head = 0;
  const int64_t* slots = nullptr;
  hq_kv_cache cache = {};
};
hipError_t kv_append_pass(const KvAppendPass& p, hipStream_t st);
struct KvReadPass {
  const int64_t* slots = nullptr;
  int64_t n = 0;
  void *k = nullptr, *v = nullptr;
  int dt = 0;
  hq_kv_cache cache = {};
};
hipError_t kv_read_pass(const KvReadPass& p, hipStream_t st);

// Attention over it (hq_kv_attention.hip).
struct KvAttentionPass {
  const void* q = nullptr;
  int q_dt = 0;
  int64_t tokens = 0, q_token = 0, q_head = 0;
  hq_kv_cache cache = {};
  hq_kv_batch batch = {};
  void* out = nullptr;
  int out_dt = 0;
  float* lse = nullptr;
  void* ws = nullptr;
};
size_t kv_attention_ws(const hq_kv_cache& cache, const hq_kv_batch& batch);
hipError_t kv_attention_pass(const KvAttentionPass& p, hipStream_t st);

}  // namespace hq
