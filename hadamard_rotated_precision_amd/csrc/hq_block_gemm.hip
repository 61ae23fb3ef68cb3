// hq_block_gemm.hip — product of block-scaled FP8 matrices on the matrix cores:
//   c[m][n] (+)= sum_kb sa(m,kb) sb(n,kb) sum_{k in kb} a[m][k] b[n][k],  kb = blocks of 128.
//
// Per block the codes are multiplied into fresh accumulators, and acc += t (sa sb) follows in fp32.
#include "hq_device.hpp"
#include "hq_launch.hpp"
#include "hq_train_internal.hpp"

namespace hq {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

struct BlockGemmArgs {
  BlockOperand a, b;
  int64_t M, N, K;
  void* c;
  int accumulate;
};

// Eight E4M3 codes as fp16 values (exact: E4M3 is a subset of fp16).
__device__ inline v8h f8_to_h8(uint2 q) {
  const v2h a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(q.x, 1.0f, false);
  const v2h b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(q.x, 1.0f, true);
  const v2h c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(q.y, 1.0f, false);
  const v2h d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(q.y, 1.0f, true);
  return v8h{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// One wave per 32 x 32 tile, fragments straight from memory: v_mfma_f32_32x32x16_f16 with b's rows
// along the accumulator's registers (row 8 (r/4) + 4 (lane/32) + r%4) and a's rows along the lanes.
template <class Out>
__global__ __launch_bounds__(64) void block_gemm_plain_kernel(BlockGemmArgs g) {
  const int lane = threadIdx.x, half = lane >> 5;
  const int64_t tiles_n = (g.N + 31) / 32;
  const int64_t m = blockIdx.x / tiles_n * 32 + (lane & 31), n0 = blockIdx.x % tiles_n * 32;
  const int64_t n = n0 + (lane & 31);
  const uint8_t* pa = g.a.codes + m * g.a.ld;
  const uint8_t* pb = g.b.codes + n * g.b.ld;
  v16f acc = {};
  const int64_t K16 = (g.K + 15) / 16 * 16;
  for (int64_t kb = 0; kb * 128 < g.K; ++kb) {
    v16f t = {};
    for (int kk = 0; kk < 128; kk += 16) {
      const int64_t k = kb * 128 + kk + 8 * half;
      uint2 qa = {0u, 0u}, qb = {0u, 0u};
      if (k < K16 && m < g.M) qa = *reinterpret_cast<const uint2*>(pa + k);
      if (k < K16 && n < g.N) qb = *reinterpret_cast<const uint2*>(pb + k);
      t = __builtin_amdgcn_mfma_f32_32x32x16_f16(f8_to_h8(qb), f8_to_h8(qa), t, 0, 0, 0);
    }
    const float sa = m < g.M ? g.a.scales[(g.a.tiles ? m / 128 : m) * g.a.sg + kb * g.a.sk] : 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int64_t nr = n0 + 8 * (r >> 2) + 4 * half + (r & 3);
      const float sb = nr < g.N ? g.b.scales[(g.b.tiles ? nr / 128 : nr) * g.b.sg + kb * g.b.sk] : 0.0f;
      acc[r] = __builtin_fmaf(t[r], sa * sb, acc[r]);
    }
  }
  if (m >= g.M) return;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int64_t nr = n0 + 8 * (r >> 2) + 4 * half + (r & 3);
    if (nr < g.N) {
      const float old = g.accumulate ? Out::load(g.c, m * g.N + nr) : 0.0f;
      Out::store(g.c, m * g.N + nr, acc[r] + old);
    }
  }
}

size_t block_gemm_ws(int64_t, int64_t, int64_t) { return 0; }

hipError_t block_gemm_pass(const BlockGemmPass& p, hipStream_t st) {
  BlockGemmArgs a{p.a, p.b, p.M, p.N, p.K, p.c, p.accumulate};
  const int tok = prof_open(K_GEMM, 2.0 * p.M * p.N * p.K);
  const dim3 grid(static_cast<unsigned>(((p.M + 31) / 32) * ((p.N + 31) / 32)));
  switch (p.out_dt) {
    case DT_F32: return launch_k(block_gemm_plain_kernel<F32>, grid, dim3(64), st, tok, a);
    case DT_F16: return launch_k(block_gemm_plain_kernel<F16>, grid, dim3(64), st, tok, a);
    case DT_BF16: return launch_k(block_gemm_plain_kernel<BF16>, grid, dim3(64), st, tok, a);
  }
  return hipErrorInvalidValue;
}

}  // namespace hq
