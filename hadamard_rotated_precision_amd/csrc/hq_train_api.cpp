// hq_train_api.cpp — the C ABI of include/hq_train.h: argument checks, workspace layout and the
// order of the kernel passes. Every argument check runs before the first HIP call, so invalid
// calls launch nothing (and need no GPU).
#include "../../include/hq_train.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "hq_checks.hpp"
#include "hq_train_internal.hpp"

namespace {

using hq::BlockGemmPass;
using hq::BlockOperand;
using hq::BlockQuantPass;

using hq::align256;
using hq::aligned;
using hq::check_ws;
using hq::dims_ok;
using hq::element_aligned;
using hq::kMaxDim;
using hq::pitch16;
using hq::stream_ok;
using hq::valid_dt;

int64_t blocks(int64_t n) { return (n + HQ_BLOCK - 1) / HQ_BLOCK; }

// Buffers of a tensor that a call writes: layouts it asks for, pitches and alignment.
hq_status check_out(const hq_block_tensor* q, int64_t rows, int64_t cols, int32_t shape,
                    bool need_codes) {
  if (!q) return HQ_ERR_NULL;
  if (rows * cols == 0) return HQ_OK;
  if (need_codes ? !q->codes : (!q->codes && !q->codes_t)) return HQ_ERR_NULL;
  const bool tiles = shape == HQ_BLOCK_TILES;
  if ((tiles || q->codes) && !q->scales) return HQ_ERR_NULL;
  if (!tiles && q->codes_t && !q->scales_t) return HQ_ERR_NULL;
  if (q->codes) {
    if (!aligned(q->codes, 16) || q->ld % 16) return HQ_ERR_ALIGN;
    if (q->ld < cols || q->ld >= 2 * kMaxDim) return HQ_ERR_SHAPE;
  }
  if (q->codes_t) {
    if (!aligned(q->codes_t, 16) || q->ld_t % 16) return HQ_ERR_ALIGN;
    if (q->ld_t < rows || q->ld_t >= 2 * kMaxDim) return HQ_ERR_SHAPE;
  }
  if (q->scales && !aligned(q->scales, 4)) return HQ_ERR_ALIGN;
  if (q->scales_t && !aligned(q->scales_t, 4)) return HQ_ERR_ALIGN;
  if (tiles ? q->lds < blocks(cols) : (q->codes && q->lds < rows)) return HQ_ERR_SHAPE;
  if (!tiles && q->codes_t && q->lds_t < cols) return HQ_ERR_SHAPE;
  return HQ_OK;
}

// A tensor that a product reads through one of its layouts. rows, cols < 0: not prescribed.
hq_status check_operand(const hq_block_tensor* q, int32_t side, int64_t rows, int64_t cols) {
  if (!q) return HQ_ERR_NULL;
  if (side != HQ_SIDE_ROWS && side != HQ_SIDE_COLS) return HQ_ERR_MODE;
  if (q->shape != HQ_BLOCK_ROWS && q->shape != HQ_BLOCK_TILES) return HQ_ERR_MODE;
  if (q->scale != HQ_BSCALE_F32 && q->scale != HQ_BSCALE_POW2) return HQ_ERR_MODE;
  if (!dims_ok(q->rows, q->cols)) return HQ_ERR_SHAPE;
  if ((rows >= 0 && q->rows != rows) || (cols >= 0 && q->cols != cols)) return HQ_ERR_MISMATCH;
  if (q->rows * q->cols == 0) return HQ_OK;
  const bool t = side == HQ_SIDE_COLS, tiles = q->shape == HQ_BLOCK_TILES;
  const uint8_t* codes = t ? q->codes_t : q->codes;
  const float* scales = (t && !tiles) ? q->scales_t : q->scales;
  if (!codes || !scales) return HQ_ERR_NULL;
  const int64_t ld = t ? q->ld_t : q->ld, len = t ? q->rows : q->cols;
  if (!aligned(codes, 16) || ld % 16 || !aligned(scales, 4)) return HQ_ERR_ALIGN;
  if (ld < len || ld >= 2 * kMaxDim) return HQ_ERR_SHAPE;
  const int64_t lds = (t && !tiles) ? q->lds_t : q->lds;
  const int64_t need = tiles ? blocks(q->cols) : (t ? q->cols : q->rows);
  if (lds < need) return HQ_ERR_SHAPE;
  return HQ_OK;
}

BlockOperand operand(const hq_block_tensor& q, int32_t side) {
  BlockOperand o;
  const bool t = side == HQ_SIDE_COLS;
  o.codes = t ? q.codes_t : q.codes;
  o.ld = t ? q.ld_t : q.ld;
  o.tiles = q.shape == HQ_BLOCK_TILES;
  o.pow2 = q.scale == HQ_BSCALE_POW2;
  o.scales = (t && !o.tiles) ? q.scales_t : q.scales;
  if (o.tiles) {   // RB x CB: a row group of `codes` is a row of it, of `codes_t` a column
    o.sg = t ? 1 : q.lds;
    o.sk = t ? q.lds : 1;
  } else {         // block-of-K x rows
    o.sg = 1;
    o.sk = t ? q.lds_t : q.lds;
  }
  return o;
}

BlockQuantPass quant_pass(const void* src, int32_t dt, int64_t rows, int64_t cols, int32_t shape,
                          int32_t scale, const hq_block_tensor& q) {
  BlockQuantPass p;
  p.src = src;
  p.in_dt = dt;
  p.rows = rows;
  p.cols = cols;
  p.tiles = shape == HQ_BLOCK_TILES;
  p.pow2 = scale == HQ_BSCALE_POW2;
  p.codes = q.codes;
  p.ld = q.ld;
  p.codes_t = q.codes_t;
  p.ld_t = q.ld_t;
  p.scales = q.scales;
  p.lds = q.lds;
  p.scales_t = q.scales_t;
  p.lds_t = q.lds_t;
  return p;
}

void fill_meta(hq_block_tensor* q, int64_t rows, int64_t cols, int32_t shape, int32_t scale) {
  q->rows = rows;
  q->cols = cols;
  q->shape = shape;
  q->scale = scale;
}

// Codes and scales of a rows x cols ROWS tensor (row-major layout) in a workspace.
size_t scratch_bytes(int64_t rows, int64_t cols) {
  return align256(static_cast<size_t>(rows * pitch16(cols))) +
         align256(static_cast<size_t>(blocks(cols) * rows) * sizeof(float));
}
hq_block_tensor scratch_tensor(void* ws, int64_t rows, int64_t cols) {
  hq_block_tensor q = {};
  q.codes = static_cast<uint8_t*>(ws);
  q.ld = pitch16(cols);
  q.scales = reinterpret_cast<float*>(static_cast<char*>(ws) +
                                      align256(static_cast<size_t>(rows * q.ld)));
  q.lds = rows;
  return q;
}

// The product of a validated call.
hq_status product(const BlockOperand& a, const BlockOperand& b, int64_t M, int64_t N, int64_t K,
                  void* c, int32_t dt, bool accumulate, void* ws, void* stream) {
  if (M == 0 || N == 0 || (K == 0 && accumulate)) return HQ_OK;
  BlockGemmPass g;
  g.a = a;
  g.b = b;
  g.M = M;
  g.N = N;
  g.K = K;
  g.c = c;
  g.out_dt = dt;
  g.accumulate = accumulate;
  g.ws = ws;
  HQ_TRY(hq::block_gemm_pass(g, static_cast<hipStream_t>(stream)));
  return HQ_OK;
}

// out = Q(in) * w^T with `in` rows x K and `out` rows x n: the forward and the input gradient.
hq_status quantized_product(const void* in, int32_t in_dt, int64_t rows, int64_t K, int64_t n,
                            const hq_block_tensor* w, int32_t w_side, int32_t scale, void* out,
                            int32_t out_dt, hq_block_tensor* save, void* ws, size_t ws_bytes,
                            void* stream) {
  if (scale != HQ_BSCALE_F32 && scale != HQ_BSCALE_POW2) return HQ_ERR_MODE;
  if ((rows * K > 0 && !in) || (rows * n > 0 && !out)) return HQ_ERR_NULL;
  if (!element_aligned(in, in_dt) || !element_aligned(out, out_dt)) return HQ_ERR_ALIGN;
  if (save) HQ_CHECK(check_out(save, rows, K, HQ_BLOCK_ROWS, true));
  const size_t own = save ? 0 : scratch_bytes(rows, K);
  HQ_CHECK(check_ws(ws, ws_bytes, own + hq::block_gemm_ws(rows, n, K)));
  HQ_CHECK(stream_ok(stream));
  if (!save && n > 0 && hq::block_gemv_fused_ok(rows, K)) {
    BlockGemmPass g;
    g.b = operand(*w, w_side);
    g.M = rows;
    g.N = n;
    g.K = K;
    g.c = out;
    g.out_dt = out_dt;
    HQ_TRY(hq::block_gemv_pass(g, in, in_dt, scale == HQ_BSCALE_POW2, static_cast<hipStream_t>(stream)));
    return HQ_OK;
  }
  hq_block_tensor q = save ? *save : scratch_tensor(ws, rows, K);
  if (rows * K > 0)
    HQ_TRY(hq::block_quant_pass(quant_pass(in, in_dt, rows, K, HQ_BLOCK_ROWS, scale, q),
                                static_cast<hipStream_t>(stream)));
  fill_meta(&q, rows, K, HQ_BLOCK_ROWS, scale);
  if (save) fill_meta(save, rows, K, HQ_BLOCK_ROWS, scale);
  return product(operand(q, HQ_SIDE_ROWS), operand(*w, w_side), rows, n, K, out, out_dt, false,
                 static_cast<char*>(ws) + own, stream);
}

}  // namespace

extern "C" {

int32_t hq_train_abi_version(void) { return HQ_TRAIN_ABI_VERSION; }

hq_status hq_block_quantize(const void* src, int32_t src_dtype, int64_t rows, int64_t cols,
                            int32_t shape, int32_t scale, hq_block_tensor* out, void* stream) {
  if (!valid_dt(src_dtype)) return HQ_ERR_DTYPE;
  if (shape != HQ_BLOCK_ROWS && shape != HQ_BLOCK_TILES) return HQ_ERR_MODE;
  if (scale != HQ_BSCALE_F32 && scale != HQ_BSCALE_POW2) return HQ_ERR_MODE;
  if (!dims_ok(rows, cols)) return HQ_ERR_SHAPE;
  if (rows * cols > 0 && !src) return HQ_ERR_NULL;
  if (!element_aligned(src, src_dtype)) return HQ_ERR_ALIGN;
  HQ_CHECK(check_out(out, rows, cols, shape, false));
  HQ_CHECK(stream_ok(stream));
  if (rows * cols > 0)
    HQ_TRY(hq::block_quant_pass(quant_pass(src, src_dtype, rows, cols, shape, scale, *out),
                                static_cast<hipStream_t>(stream)));
  fill_meta(out, rows, cols, shape, scale);
  return HQ_OK;
}

size_t hq_block_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (!dims_ok(M, N) || !dims_ok(M, K) || !dims_ok(N, K)) return 0;
  return hq::block_gemm_ws(M, N, K);
}

hq_status hq_block_gemm(const hq_block_tensor* a, int32_t a_side, const hq_block_tensor* b,
                        int32_t b_side, void* c, int32_t c_dtype, int32_t accumulate, void* ws,
                        size_t ws_bytes, void* stream) {
  HQ_CHECK(check_operand(a, a_side, -1, -1));
  HQ_CHECK(check_operand(b, b_side, -1, -1));
  if (!valid_dt(c_dtype)) return HQ_ERR_DTYPE;
  const int64_t M = a_side == HQ_SIDE_ROWS ? a->rows : a->cols;
  const int64_t K = a_side == HQ_SIDE_ROWS ? a->cols : a->rows;
  const int64_t N = b_side == HQ_SIDE_ROWS ? b->rows : b->cols;
  if ((b_side == HQ_SIDE_ROWS ? b->cols : b->rows) != K) return HQ_ERR_MISMATCH;
  if (!dims_ok(M, N)) return HQ_ERR_SHAPE;
  if (M * N > 0 && !c) return HQ_ERR_NULL;
  if (!element_aligned(c, c_dtype)) return HQ_ERR_ALIGN;
  HQ_CHECK(check_ws(ws, ws_bytes, hq::block_gemm_ws(M, N, K)));
  HQ_CHECK(stream_ok(stream));
  return product(operand(*a, a_side), operand(*b, b_side), M, N, K, c, c_dtype, accumulate != 0,
                 ws, stream);
}

size_t hq_block_workspace_bytes(int64_t N, int64_t C, int64_t D) {
  if (!dims_ok(N, C) || !dims_ok(N, D) || !dims_ok(D, C)) return 0;
  const size_t fwd = scratch_bytes(N, C) + hq::block_gemm_ws(N, D, C);
  const size_t bwd = scratch_bytes(N, D) + hq::block_gemm_ws(N, C, D);
  const size_t dw = hq::block_gemm_ws(D, C, N);
  return fwd > bwd ? (fwd > dw ? fwd : dw) : (bwd > dw ? bwd : dw);
}

hq_status hq_block_linear_fwd(const void* x, int32_t x_dtype, int64_t N, int64_t C, int64_t D,
                              const hq_block_tensor* w, int32_t scale, void* y, int32_t y_dtype,
                              hq_block_tensor* save_x, void* ws, size_t ws_bytes, void* stream) {
  if (!valid_dt(x_dtype) || !valid_dt(y_dtype)) return HQ_ERR_DTYPE;
  if (!dims_ok(N, C) || !dims_ok(N, D) || !dims_ok(D, C)) return HQ_ERR_SHAPE;
  HQ_CHECK(check_operand(w, HQ_SIDE_ROWS, D, C));
  return quantized_product(x, x_dtype, N, C, D, w, HQ_SIDE_ROWS, scale, y, y_dtype, save_x, ws,
                           ws_bytes, stream);
}

hq_status hq_block_linear_bwd_input(const void* dy, int32_t dy_dtype, int64_t N, int64_t C,
                                    int64_t D, const hq_block_tensor* w, int32_t scale, void* dx,
                                    int32_t dx_dtype, hq_block_tensor* save_g, void* ws,
                                    size_t ws_bytes, void* stream) {
  if (!valid_dt(dy_dtype) || !valid_dt(dx_dtype)) return HQ_ERR_DTYPE;
  if (!dims_ok(N, C) || !dims_ok(N, D) || !dims_ok(D, C)) return HQ_ERR_SHAPE;
  HQ_CHECK(check_operand(w, HQ_SIDE_COLS, D, C));
  return quantized_product(dy, dy_dtype, N, D, C, w, HQ_SIDE_COLS, scale, dx, dx_dtype, save_g,
                           ws, ws_bytes, stream);
}

hq_status hq_block_linear_bwd_weight(const hq_block_tensor* saved_g,
                                     const hq_block_tensor* saved_x, int64_t N, int64_t C,
                                     int64_t D, void* dw, int32_t dw_dtype, int32_t accumulate,
                                     void* ws, size_t ws_bytes, void* stream) {
  if (!valid_dt(dw_dtype)) return HQ_ERR_DTYPE;
  if (!dims_ok(N, C) || !dims_ok(N, D) || !dims_ok(D, C)) return HQ_ERR_SHAPE;
  HQ_CHECK(check_operand(saved_g, HQ_SIDE_COLS, N, D));
  HQ_CHECK(check_operand(saved_x, HQ_SIDE_COLS, N, C));
  if (D * C > 0 && !dw) return HQ_ERR_NULL;
  if (!element_aligned(dw, dw_dtype)) return HQ_ERR_ALIGN;
  HQ_CHECK(check_ws(ws, ws_bytes, hq::block_gemm_ws(D, C, N)));
  HQ_CHECK(stream_ok(stream));
  return product(operand(*saved_g, HQ_SIDE_COLS), operand(*saved_x, HQ_SIDE_COLS), D, C, N, dw,
                 dw_dtype, accumulate != 0, ws, stream);
}

}  // extern "C"

namespace {

uint32_t mix32(uint32_t h) {
  h ^= h >> 16;
  h *= 2654435761u;
  h ^= h >> 15;
  h *= 2891336453u;
  return h ^ (h >> 16);
}

hq_status check_adamw(const hq_adamw_config* cfg) {
  if (!cfg) return HQ_ERR_NULL;
  if (!valid_dt(cfg->param_dtype) || !valid_dt(cfg->grad_dtype) || !valid_dt(cfg->copy_dtype))
    return HQ_ERR_DTYPE;
  if (cfg->state_bits != 32 && cfg->state_bits != 8) return HQ_ERR_BITS;
  // written so that a NaN fails too
  if (!(cfg->lr >= 0.0 && cfg->lr <= 1e30) || !(cfg->beta1 >= 0.0 && cfg->beta1 < 1.0) ||
      !(cfg->beta2 >= 0.0 && cfg->beta2 < 1.0) || !(cfg->eps >= 1.2e-38 && cfg->eps <= 1e30))
    return HQ_ERR_MODE;
  return HQ_OK;
}

}  // namespace

extern "C" {

hq_status hq_adamw_scalars_at(const hq_adamw_config* cfg, int64_t step, double grad_scale,
                              hq_adamw_scalars* out) {
  HQ_CHECK(check_adamw(cfg));
  if (!out) return HQ_ERR_NULL;
  if (step < 1) return HQ_ERR_SHAPE;
  const double t = static_cast<double>(step);
  out->lr = static_cast<float>(cfg->lr);
  out->step_size = static_cast<float>(cfg->lr / (1.0 - std::pow(cfg->beta1, t)));
  out->inv_sqrt_bias2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(cfg->beta2, t)));
  out->grad_scale = static_cast<float>(grad_scale);
  out->key = mix32(cfg->seed + 2654435761u * static_cast<uint32_t>(step));
  return HQ_OK;
}

hq_status hq_adamw_step(const hq_adamw_tensor* tensors, int32_t count, const hq_adamw_config* cfg,
                        const hq_adamw_scalars* host_scalars,
                        const hq_adamw_scalars* device_scalars, void* stream) {
  HQ_CHECK(check_adamw(cfg));
  if (count < 0) return HQ_ERR_SHAPE;
  if (count > 0 && !tensors) return HQ_ERR_NULL;
  if (!host_scalars && !device_scalars) return HQ_ERR_NULL;
  if (!aligned(device_scalars, 4)) return HQ_ERR_ALIGN;
  for (int32_t i = 0; i < count; ++i) {
    const hq_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n > (int64_t{1} << 34)) return HQ_ERR_SHAPE;
    if (!(t.weight_decay >= 0.0f && t.weight_decay <= 1e30f)) return HQ_ERR_MODE;
    if (t.n == 0) continue;
    if (!t.p || !t.grad || !t.m || !t.v) return HQ_ERR_NULL;
    if (cfg->state_bits == 8 && (!t.m_scales || !t.v_scales)) return HQ_ERR_NULL;
    const unsigned state = cfg->state_bits == 8 ? 1 : 4;
    if (!element_aligned(t.p, cfg->param_dtype) || !element_aligned(t.grad, cfg->grad_dtype) ||
        !element_aligned(t.copy, cfg->copy_dtype) || !aligned(t.m, state) || !aligned(t.v, state) ||
        !aligned(t.m_scales, 4) || !aligned(t.v_scales, 4))
      return HQ_ERR_ALIGN;
  }
  HQ_CHECK(stream_ok(stream));
  const hq_adamw_scalars none = {};
  HQ_TRY(hq::adamw_pass(tensors, count, *cfg, host_scalars ? *host_scalars : none, device_scalars,
                        static_cast<hipStream_t>(stream)));
  return HQ_OK;
}

}  // extern "C"
