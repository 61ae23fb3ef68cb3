// hq_mx_api.cpp — the C ABI of include/hq_mx.h: argument checks, workspace layout and the order of
// the kernel passes. Every argument check runs before the first HIP call, so invalid calls launch
// nothing (and need no GPU).
#include "../../include/hq_mx.h"

#include <hip/hip_runtime.h>

#include "hq_checks.hpp"
#include "hq_mx_internal.hpp"

namespace {

using namespace hq;

// As the other libraries', and 2^34 elements in all: a kernel's threads, of eight elements each, stay
// countable in 32 bits.
bool mx_dims_ok(int64_t a, int64_t b) {
  return dims_ok(a, b) && ((a + 127) / 128) * ((b + 127) / 128) <= (int64_t{1} << 20);
}
bool valid_rot(int32_t rot) { return rot == 1 || rot == HQ_MX_BLOCK; }

// One layout's buffers: rows of n codes.
hq_status check_layout(const uint8_t* codes, int64_t ld, const uint8_t* scales, int64_t lds, int64_t n) {
  if (!codes || !scales) return HQ_ERR_NULL;
  if (!aligned(codes, 16) || ld % 16 || !aligned(scales, 16) || lds % 16) return HQ_ERR_ALIGN;
  if (ld < 16 * mx_blocks(n) || ld >= kMaxDim || lds < mx_blocks(n) || lds >= kMaxDim) return HQ_ERR_SHAPE;
  return HQ_OK;
}

// Buffers of a tensor that a call writes.
hq_status check_out(const hq_mx_tensor* q, int64_t rows, int64_t cols, bool need_codes) {
  if (!q) return HQ_ERR_NULL;
  if (rows * cols == 0) return HQ_OK;
  if (need_codes ? !q->codes : (!q->codes && !q->codes_t)) return HQ_ERR_NULL;
  if (q->codes) HQ_CHECK(check_layout(q->codes, q->ld, q->scales, q->lds, cols));
  if (q->codes_t) HQ_CHECK(check_layout(q->codes_t, q->ld_t, q->scales_t, q->lds_t, rows));
  return HQ_OK;
}

// A tensor that a call reads through one of its layouts. rows, cols < 0: not prescribed.
hq_status check_operand(const hq_mx_tensor* q, int32_t side, int64_t rows, int64_t cols) {
  if (!q) return HQ_ERR_NULL;
  if (side != HQ_SIDE_ROWS && side != HQ_SIDE_COLS) return HQ_ERR_MODE;
  if (!valid_rot(q->rot)) return HQ_ERR_K;
  if (!mx_dims_ok(q->rows, q->cols)) return HQ_ERR_SHAPE;
  if ((rows >= 0 && q->rows != rows) || (cols >= 0 && q->cols != cols)) return HQ_ERR_MISMATCH;
  if (q->rows * q->cols == 0) return HQ_OK;
  return side == HQ_SIDE_COLS ? check_layout(q->codes_t, q->ld_t, q->scales_t, q->lds_t, q->rows)
                              : check_layout(q->codes, q->ld, q->scales, q->lds, q->cols);
}

MxOperand operand(const hq_mx_tensor& q, int32_t side) {
  return side == HQ_SIDE_COLS ? MxOperand{q.codes_t, q.ld_t, q.scales_t, q.lds_t}
                              : MxOperand{q.codes, q.ld, q.scales, q.lds};
}

hq_status quantize(const void* src, int32_t dt, int64_t rows, int64_t cols, int32_t rot,
                   const uint32_t* seed, hq_mx_tensor* q, void* stream) {
  if (rows * cols > 0) {
    const MxQuantPass p{src, dt, rows, cols, rot, seed, q->codes, q->codes_t, q->scales, q->scales_t,
                        q->ld, q->ld_t, q->lds, q->lds_t};
    HQ_TRY(mx_quant_pass(p, static_cast<hipStream_t>(stream)));
  }
  q->rows = rows;
  q->cols = cols;
  q->rot = rot;
  return HQ_OK;
}

// Codes and scales of a rows x cols matrix (row-major layout) in a workspace.
size_t scratch_codes(int64_t rows, int64_t cols) {
  return align256(static_cast<size_t>(rows) * 16 * mx_blocks(cols));
}
size_t scratch_bytes(int64_t rows, int64_t cols) {
  return scratch_codes(rows, cols) + align256(static_cast<size_t>(rows) * pitch16(mx_blocks(cols)));
}
hq_mx_tensor scratch_tensor(void* ws, int64_t rows, int64_t cols) {
  hq_mx_tensor q = {};
  q.codes = static_cast<uint8_t*>(ws);
  q.ld = 16 * mx_blocks(cols);
  q.scales = static_cast<uint8_t*>(ws) + scratch_codes(rows, cols);
  q.lds = pitch16(mx_blocks(cols));
  return q;
}

MxGemmPass pass(int64_t M, int64_t N, int64_t K, int32_t rot, void* c, int32_t dt) {
  MxGemmPass g;
  g.M = M;
  g.N = N;
  g.K = K;
  g.alpha = 1.0f / static_cast<float>(rot);
  g.c = c;
  g.out_dt = dt;
  return g;
}

// The product of a validated call.
hq_status product(const MxOperand& a, const MxOperand& b, MxGemmPass g, bool accumulate, void* ws,
                  void* stream) {
  if (g.M == 0 || g.N == 0 || (g.K == 0 && accumulate)) return HQ_OK;
  g.a = a;
  g.b = b;
  g.accumulate = accumulate;
  g.ws = ws;
  HQ_TRY(mx_gemm_pass(g, static_cast<hipStream_t>(stream)));
  return HQ_OK;
}

// out = Q(in) w^T with `in` rows x K and `out` rows x n: the forward and the input gradient.
hq_status quantized_product(const void* in, int32_t in_dt, int64_t rows, int64_t K, int64_t n,
                            const hq_mx_tensor* w, int32_t w_side, const uint32_t* seed, void* out,
                            int32_t out_dt, hq_mx_tensor* save, void* ws, size_t ws_bytes,
                            void* stream) {
  if ((rows * K > 0 && !in) || (rows * n > 0 && !out)) return HQ_ERR_NULL;
  if (!element_aligned(in, in_dt) || !element_aligned(out, out_dt) || !aligned(seed, 4)) return HQ_ERR_ALIGN;
  if (save) HQ_CHECK(check_out(save, rows, K, true));
  const size_t own = save ? 0 : scratch_bytes(rows, K);
  HQ_CHECK(check_ws(ws, ws_bytes, own + mx_gemm_ws(rows, n, K)));
  HQ_CHECK(stream_ok(stream));
  const MxGemmPass g = pass(rows, n, K, w->rot, out, out_dt);
  if (!save && !seed && n > 0 && mx_gemv_fused_ok(rows, K)) {
    MxGemmPass f = g;
    f.b = operand(*w, w_side);
    HQ_TRY(mx_gemv_pass(f, in, in_dt, w->rot, static_cast<hipStream_t>(stream)));
    return HQ_OK;
  }
  hq_mx_tensor scratch = {};
  if (!save) scratch = scratch_tensor(ws, rows, K);
  hq_mx_tensor* q = save ? save : &scratch;
  HQ_CHECK(quantize(in, in_dt, rows, K, w->rot, seed, q, stream));
  return product(operand(*q, HQ_SIDE_ROWS), operand(*w, w_side), g, false,
                 own ? static_cast<char*>(ws) + own : ws, stream);
}

bool shapes_ok(int64_t N, int64_t C, int64_t D) { return mx_dims_ok(N, C) && mx_dims_ok(N, D) && mx_dims_ok(D, C); }

// ---------------------------------------------------------------- the cache
constexpr int64_t kMaxSlots = int64_t{1} << 31;

// Tokens of a call: two vectors of head_dim / 8 threads for each head, in whole workgroups of 256, are fewer
// than 2^32 threads, the most that a launch takes.
bool tokens_ok(int64_t n, const hq_kv_cache& c) {
  return n >= 0 && n <= ((int64_t{1} << 31) - 128) / (static_cast<int64_t>(c.heads) * (c.head_dim / 8));
}

hq_status check_cache(const hq_kv_cache* c) {
  if (!c) return HQ_ERR_NULL;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return HQ_ERR_SHAPE;
  if (c->heads < 1 || c->heads > 1024 || c->pages < 0) return HQ_ERR_SHAPE;
  if (c->page < 16 || c->page > (1 << 20) || (c->page & (c->page - 1))) return HQ_ERR_SHAPE;
  if (c->pages > kMaxSlots / c->page) return HQ_ERR_SHAPE;
  if (c->rot != 1 && c->rot != c->head_dim) return HQ_ERR_K;
  if (c->pages == 0) return HQ_OK;
  if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales) return HQ_ERR_NULL;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 16) ||
      !aligned(c->v_scales, 16))
    return HQ_ERR_ALIGN;
  return HQ_OK;
}

bool stride_ok(int64_t s) { return s >= 0 && s <= (int64_t{1} << 40); }

hq_status check_batch(const hq_kv_cache& c, const hq_kv_batch* b) {
  if (!b) return HQ_ERR_NULL;
  if (b->seqs < 0 || b->max_q < 0 || b->max_len < 0 || b->table_ld < 0 || b->window < 0) return HQ_ERR_SHAPE;
  if (b->table_ld > (int64_t{1} << 31) || b->max_len > (1 << 30)) return HQ_ERR_SHAPE;
  if (b->q_heads < 1 || b->q_heads % c.heads || b->q_heads / c.heads > 1024) return HQ_ERR_MISMATCH;
  // workgroups and partial results of a call stay countable
  if (static_cast<int64_t>(b->max_q) * (b->q_heads / c.heads) > (int64_t{1} << 27) ||
      static_cast<int64_t>(b->seqs) * c.heads > (int64_t{1} << 24))
    return HQ_ERR_SHAPE;
  const int64_t tiles = (static_cast<int64_t>(b->max_q) * (b->q_heads / c.heads) + 15) / 16;
  if (static_cast<int64_t>(b->seqs) * c.heads * tiles > (int64_t{1} << 22)) return HQ_ERR_SHAPE;
  if (!(b->scale >= -1e30f && b->scale <= 1e30f)) return HQ_ERR_MODE;   // a NaN fails too
  return HQ_OK;
}

}  // namespace

extern "C" {

int32_t hq_mx_abi_version(void) { return HQ_MX_ABI_VERSION; }

hq_status hq_mx_quantize(const void* src, int32_t src_dtype, int64_t rows, int64_t cols, int32_t rot,
                         const uint32_t* seed, hq_mx_tensor* out, void* stream) {
  if (!valid_dt(src_dtype)) return HQ_ERR_DTYPE;
  if (!valid_rot(rot)) return HQ_ERR_K;
  if (!mx_dims_ok(rows, cols)) return HQ_ERR_SHAPE;
  if (rows * cols > 0 && !src) return HQ_ERR_NULL;
  if (!element_aligned(src, src_dtype) || !aligned(seed, 4)) return HQ_ERR_ALIGN;
  HQ_CHECK(check_out(out, rows, cols, false));
  HQ_CHECK(stream_ok(stream));
  return quantize(src, src_dtype, rows, cols, rot, seed, out, stream);
}

hq_status hq_mx_dequantize(const hq_mx_tensor* q, int32_t side, void* dst, int32_t dst_dtype,
                           void* stream) {
  HQ_CHECK(check_operand(q, side, -1, -1));
  if (!valid_dt(dst_dtype)) return HQ_ERR_DTYPE;
  const bool t = side == HQ_SIDE_COLS;
  if (q->rows * q->cols > 0 && !dst) return HQ_ERR_NULL;
  if (!element_aligned(dst, dst_dtype)) return HQ_ERR_ALIGN;
  HQ_CHECK(stream_ok(stream));
  if (q->rows * q->cols > 0)
    HQ_TRY(mx_dequant_pass(operand(*q, side), t ? q->cols : q->rows, t ? q->rows : q->cols, q->rot, dst,
                           dst_dtype, static_cast<hipStream_t>(stream)));
  return HQ_OK;
}

size_t hq_mx_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (!mx_dims_ok(M, N) || !mx_dims_ok(M, K) || !mx_dims_ok(N, K)) return 0;
  return mx_gemm_ws(M, N, K);
}

hq_status hq_mx_gemm(const hq_mx_tensor* a, int32_t a_side, const hq_mx_tensor* b, int32_t b_side,
                     void* c, int32_t c_dtype, int32_t accumulate, void* ws, size_t ws_bytes,
                     void* stream) {
  HQ_CHECK(check_operand(a, a_side, -1, -1));
  HQ_CHECK(check_operand(b, b_side, -1, -1));
  if (!valid_dt(c_dtype)) return HQ_ERR_DTYPE;
  const int64_t M = a_side == HQ_SIDE_ROWS ? a->rows : a->cols;
  const int64_t K = a_side == HQ_SIDE_ROWS ? a->cols : a->rows;
  const int64_t N = b_side == HQ_SIDE_ROWS ? b->rows : b->cols;
  if ((b_side == HQ_SIDE_ROWS ? b->cols : b->rows) != K || a->rot != b->rot) return HQ_ERR_MISMATCH;
  if (!mx_dims_ok(M, N)) return HQ_ERR_SHAPE;
  if (M * N > 0 && !c) return HQ_ERR_NULL;
  if (!element_aligned(c, c_dtype)) return HQ_ERR_ALIGN;
  HQ_CHECK(check_ws(ws, ws_bytes, mx_gemm_ws(M, N, K)));
  HQ_CHECK(stream_ok(stream));
  return product(operand(*a, a_side), operand(*b, b_side), pass(M, N, K, a->rot, c, c_dtype),
                 accumulate != 0, ws, stream);
}

size_t hq_mx_workspace_bytes(int64_t N, int64_t C, int64_t D) {
  if (!shapes_ok(N, C, D)) return 0;
  const size_t fwd = scratch_bytes(N, C) + mx_gemm_ws(N, D, C);
  const size_t bwd = scratch_bytes(N, D) + mx_gemm_ws(N, C, D);
  const size_t dw = mx_gemm_ws(D, C, N);
  return fwd > bwd ? (fwd > dw ? fwd : dw) : (bwd > dw ? bwd : dw);
}

hq_status hq_mx_linear_fwd(const void* x, int32_t x_dtype, int64_t N, int64_t C, int64_t D,
                           const hq_mx_tensor* w, const uint32_t* seed, void* y, int32_t y_dtype,
                           hq_mx_tensor* save_x, void* ws, size_t ws_bytes, void* stream) {
  if (!valid_dt(x_dtype) || !valid_dt(y_dtype)) return HQ_ERR_DTYPE;
  if (!shapes_ok(N, C, D)) return HQ_ERR_SHAPE;
  HQ_CHECK(check_operand(w, HQ_SIDE_ROWS, D, C));
  return quantized_product(x, x_dtype, N, C, D, w, HQ_SIDE_ROWS, seed, y, y_dtype, save_x, ws, ws_bytes,
                           stream);
}

hq_status hq_mx_linear_bwd_input(const void* dy, int32_t dy_dtype, int64_t N, int64_t C, int64_t D,
                                 const hq_mx_tensor* w, const uint32_t* seed, void* dx,
                                 int32_t dx_dtype, hq_mx_tensor* save_g, void* ws, size_t ws_bytes,
                                 void* stream) {
  if (!valid_dt(dy_dtype) || !valid_dt(dx_dtype)) return HQ_ERR_DTYPE;
  if (!shapes_ok(N, C, D)) return HQ_ERR_SHAPE;
  HQ_CHECK(check_operand(w, HQ_SIDE_COLS, D, C));
  return quantized_product(dy, dy_dtype, N, D, C, w, HQ_SIDE_COLS, seed, dx, dx_dtype, save_g, ws,
                           ws_bytes, stream);
}

hq_status hq_mx_linear_bwd_weight(const hq_mx_tensor* saved_g, const hq_mx_tensor* saved_x, int64_t N,
                                  int64_t C, int64_t D, void* dw, int32_t dw_dtype,
                                  int32_t accumulate, void* ws, size_t ws_bytes, void* stream) {
  if (!valid_dt(dw_dtype)) return HQ_ERR_DTYPE;
  if (!shapes_ok(N, C, D)) return HQ_ERR_SHAPE;
  HQ_CHECK(check_operand(saved_g, HQ_SIDE_COLS, N, D));
  HQ_CHECK(check_operand(saved_x, HQ_SIDE_COLS, N, C));
  if (saved_g->rot != saved_x->rot) return HQ_ERR_MISMATCH;
  if (D * C > 0 && !dw) return HQ_ERR_NULL;
  if (!element_aligned(dw, dw_dtype)) return HQ_ERR_ALIGN;
  HQ_CHECK(check_ws(ws, ws_bytes, mx_gemm_ws(D, C, N)));
  HQ_CHECK(stream_ok(stream));
  return product(operand(*saved_g, HQ_SIDE_COLS), operand(*saved_x, HQ_SIDE_COLS),
                 pass(D, C, N, saved_g->rot, dw, dw_dtype), accumulate != 0, ws, stream);
}

hq_status hq_kv_append(const void* k, const void* v, int32_t dtype, int64_t tokens, int64_t k_token,
                       int64_t k_head, int64_t v_token, int64_t v_head, const int64_t* slots,
                       const hq_kv_cache* cache, void* stream) {
  HQ_CHECK(check_cache(cache));
  if (!valid_dt(dtype)) return HQ_ERR_DTYPE;
  if (!tokens_ok(tokens, *cache)) return HQ_ERR_SHAPE;
  if (!stride_ok(k_token) || !stride_ok(k_head) || !stride_ok(v_token) || !stride_ok(v_head)) return HQ_ERR_SHAPE;
  if (tokens > 0 && (!k || !v || !slots)) return HQ_ERR_NULL;
  if (!element_aligned(k, dtype) || !element_aligned(v, dtype) || !aligned(slots, 8)) return HQ_ERR_ALIGN;
  HQ_CHECK(stream_ok(stream));
  if (tokens > 0 && cache->pages > 0) {
    const KvAppendPass p{k, v, dtype, tokens, k_token, k_head, v_token, v_head, slots, *cache};
    HQ_TRY(kv_append_pass(p, static_cast<hipStream_t>(stream)));
  }
  return HQ_OK;
}

hq_status hq_kv_read(const hq_kv_cache* cache, const int64_t* slots, int64_t n, void* k_out,
                     void* v_out, int32_t dtype, void* stream) {
  HQ_CHECK(check_cache(cache));
  if (!valid_dt(dtype)) return HQ_ERR_DTYPE;
  if (!tokens_ok(n, *cache)) return HQ_ERR_SHAPE;
  if (n > 0 && (!slots || (!k_out && !v_out))) return HQ_ERR_NULL;
  if (!element_aligned(k_out, dtype) || !element_aligned(v_out, dtype) || !aligned(slots, 8)) return HQ_ERR_ALIGN;
  HQ_CHECK(stream_ok(stream));
  if (n > 0) {
    const KvReadPass p{slots, n, k_out, v_out, dtype, *cache};
    HQ_TRY(kv_read_pass(p, static_cast<hipStream_t>(stream)));
  }
  return HQ_OK;
}

size_t hq_kv_attention_workspace_bytes(const hq_kv_cache* cache, const hq_kv_batch* batch) {
  if (check_cache(cache) != HQ_OK || check_batch(*cache, batch) != HQ_OK) return 0;
  return kv_attention_ws(*cache, *batch);
}

hq_status hq_kv_attention(const void* q, int32_t q_dtype, int64_t tokens, int64_t q_token,
                          int64_t q_head, const hq_kv_cache* cache, const hq_kv_batch* batch, void* out,
                          int32_t out_dtype, float* lse, void* ws, size_t ws_bytes, void* stream) {
  HQ_CHECK(check_cache(cache));
  HQ_CHECK(check_batch(*cache, batch));
  if (!valid_dt(q_dtype) || !valid_dt(out_dtype)) return HQ_ERR_DTYPE;
  if (tokens < 0 || tokens > kMaxSlots || !stride_ok(q_token) || !stride_ok(q_head)) return HQ_ERR_SHAPE;
  const bool any = tokens > 0 && batch->seqs > 0 && batch->max_q > 0;
  if (any && (!q || !out || !batch->q_starts || !batch->lens)) return HQ_ERR_NULL;
  if (any && batch->max_len > 0 && batch->table_ld > 0 && !batch->table) return HQ_ERR_NULL;
  if (!element_aligned(q, q_dtype) || !element_aligned(out, out_dtype) || !aligned(lse, 4) ||
      !aligned(batch->q_starts, 4) || !aligned(batch->lens, 4) || !aligned(batch->table, 4))
    return HQ_ERR_ALIGN;
  HQ_CHECK(check_ws(ws, ws_bytes, kv_attention_ws(*cache, *batch)));
  HQ_CHECK(stream_ok(stream));
  if (any) {
    const KvAttentionPass p{q, q_dtype, tokens, q_token, q_head, *cache, *batch, out, out_dtype, lse, ws};
    HQ_TRY(kv_attention_pass(p, static_cast<hipStream_t>(stream)));
  }
  return HQ_OK;
}

}  // extern "C"
