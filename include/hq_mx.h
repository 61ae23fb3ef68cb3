/*
 * hq_mx.h — C ABI of libhq_mx.so (MI355X, gfx950): operators in microscaled 4-bit floating point,
 * beside the tensor-wise layer of hq.h and the block-scaled FP8 one of hq_train.h, with their
 * statuses (hq_status), element types (hq_dtype), sides of a matrix (hq_block_side), launch
 * instrumentation and conventions.
 *
 * A layer's products, and what a server keeps of the past, in one format:
 *   hq_mx_quantize            a matrix to 4-bit codes, rotated on the way if asked for
 *   hq_mx_dequantize          the values that codes stand for
 *   hq_mx_gemm                the product of two such matrices
 *   hq_mx_linear_fwd          Y = X W^T        (any N: single tokens to whole batches)
 *   hq_mx_linear_bwd_input    dX = dY W
 *   hq_mx_linear_bwd_weight   dW = dY^T X
 *   hq_kv_append              keys and values of new tokens into a paged cache of such codes
 *   hq_kv_read                keys and values of tokens out of it
 *   hq_kv_attention           attention of queries over it, from one token to pieces of prompts
 *
 * Conventions (those of hq.h; where this header adds to them it says so):
 *   - Pointers are DEVICE pointers unless a comment says otherwise. Codes, scales and workspaces
 *     are 16-byte aligned and the pitches of codes and scales multiples of 16 bytes; everything
 *     else needs only the alignment of its elements (HQ_ERR_ALIGN otherwise).
 *   - Every call is asynchronous on `stream`, whose device must be the current one
 *     (HQ_ERR_DEVICE otherwise). No call synchronizes, allocates or records a memset, so all of
 *     them can be captured into a HIP graph.
 *   - The caller owns every buffer; nothing is kept after a call returns. Calls that may run at
 *     the same time need workspaces and outputs of their own (two captured graphs too). Outputs
 *     overlap neither inputs nor each other.
 *   - All argument checks run before any launch; on error nothing is launched or written.
 *   - Results do not depend on the order in which workgroups run: the same call on the same data
 *     gives the same bits. They do depend on the shapes: another number of rows, another bound on
 *     the lengths, or other lengths of the sequences beside it, may take another order of summation.
 *   - hq_profile_start's kinds: products and attention HQ_KIND_GEMM, quantizing and appending
 *     HQ_KIND_ROT_QUANT, reading back HQ_KIND_ROT_STORE, the joining of split sums HQ_KIND_MISC.
 */
#ifndef HQ_MX_H
#define HQ_MX_H

#include "hq_train.h"

#ifdef __cplusplus
extern "C" {
#endif

#define HQ_MX_ABI_VERSION 1

/* Version of the ABI of this header. */
int32_t hq_mx_abi_version(void);

/* ---------------------------------------------------------------- codes
 * A code is an E2M1 number: 0, 0.5, 1, 1.5, 2, 3, 4, 6 (codes 0 to 7) or, with bit 3 set, its
 * negative. HQ_MX_BLOCK consecutive elements along the contraction share a scale 2^(b - 127), kept
 * as the byte b (E8M0; 255 stands for NaN). Blocks at the end of an axis are cut short.
 *
 * Rotation k: before quantizing, every k consecutive elements along the contraction (zeros past its
 * end) are multiplied by the Walsh-Hadamard matrix H_k, unnormalised, in fp32 butterflies: stages of
 * strides 1, 2, .. k / 2, in each of which (x_i, x_{i+stride}) becomes (x_i + x_{i+stride},
 * x_i - x_{i+stride}). H_k H_k = k I, so a product of two such operands is k times the product and
 * is divided by k, which is exact. k = 1 is none.
 *
 * The scale of a block with largest magnitude a: the smallest power of two s with a <= 6 s, at least
 * 2^-126 (so nothing saturates, also where rounding is at random). A code is the value nearest to
 * v / s, ties to the even code. A block that holds a NaN or an infinity (or a rotated sum past fp32)
 * gets b = 255 and zero codes, so every product that reads it is NaN.
 *
 * Rounding at random (for gradients: the mean of a code is v / s, less at most 2^-16 of the step between
 * its neighbours, toward zero, since u has 16 bits; below 2^-17 s it is 0): with x = |v| / s and 16
 * random bits u, x >= 1: the bit pattern of fp32 x plus 64 u, cut to one bit of fraction; x < 1:
 * floor(fp32(2 x + u / 65536)) halves. The bits of row r and column c come from a seed alone:
 *   mix(h): h ^= h >> 16; h *= 2654435761; h ^= h >> 15; h *= 2891336453; h ^= h >> 16
 *   h = mix(mix(seed + 2654435761 r) ^ (c / 2));  u = the low 16 bits of h for even c, else the high
 * (all mod 2^32). For transposed codes r is the column of the matrix, c its row, and the seed is
 * seed + 0x9E3779B9. */
#define HQ_MX_BLOCK 32

/* A rows x cols matrix. With RB = ceil(rows / 32), CB = ceil(cols / 32):
 * codes    rows x ld bytes (ld >= 16 CB, a multiple of 16): element c of a row in byte c / 2, in its
 *          low half for even c; or NULL
 * codes_t  the same of the transpose, cols x ld_t (ld_t >= 16 RB), or NULL
 * scales   rows x lds bytes (lds >= CB, a multiple of 16): of `codes`, block by block
 * scales_t cols x lds_t (lds_t >= RB): of `codes_t`
 * Codes from a row's length to the end of its last block are zero, unless that block is rotated (its
 * zeros take part in the sums then, and all 32 codes count). Scale bytes from CB (RB) to the next
 * multiple of 16 are zero. The producer writes both; a caller that brings codes of its own keeps
 * these rules.
 * rows, cols and rot are written by hq_mx_quantize and checked by every consumer; rot: 1 or 32. */
typedef struct {
  uint8_t *codes;
  uint8_t *codes_t;
  uint8_t *scales;
  uint8_t *scales_t;
  int64_t rows, cols;
  int64_t ld, ld_t;
  int64_t lds, lds_t;
  int32_t rot;
  int32_t reserved; /* 0 */
} hq_mx_tensor;

/* Quantize a rows x cols matrix (row-major, contiguous, dtype src_dtype) into out->codes and/or
 * out->codes_t (at least one non-NULL) with their scales, from one read of src. Each layout is
 * rotated along its own rows. seed: NULL for rounding to nearest, or a device pointer to the seed of
 * a rounding at random (read when the kernel runs, so a captured call follows what it holds).
 * The call fills rows, cols and rot of *out (host struct). */
hq_status hq_mx_quantize(const void *src, int32_t src_dtype, int64_t rows, int64_t cols,
                         int32_t rot, const uint32_t *seed, hq_mx_tensor *out, void *stream);

/* What one layout stands for: HQ_SIDE_ROWS writes rows x cols values from codes, HQ_SIDE_COLS
 * cols x rows values from codes_t (contiguous, dtype dst_dtype), rotated back (H_k / k) and rounded
 * once. */
hq_status hq_mx_dequantize(const hq_mx_tensor *q, int32_t side, void *dst, int32_t dst_dtype,
                           void *stream);

/* c[m][n] (+)= sum_k A[m][k] B[n][k] for the values A, B that a layout of each tensor stands for:
 *   1 / rot  sum over blocks kb of 32 of 2^(ea + eb - 254)  sum_{k in kb} a[m][k] b[n][k]
 * a_side, b_side: HQ_SIDE_ROWS = codes (rows x cols) or HQ_SIDE_COLS = codes_t (cols x rows); the
 * contracted lengths and the rotations must agree (HQ_ERR_MISMATCH). c is M x N, contiguous, dtype
 * c_dtype; accumulate != 0 adds to what c holds (the sum is formed in fp32 and rounded once).
 * Sums: products of codes and their sum over a block are exact; blocks are added in fp32 by the
 * matrix instruction, whose sum of 128 products is within 2^-24 of the sum of their magnitudes. The
 * sum is rot times the result: where rot sum |A B| reaches 2^128 the result may be infinite or NaN.
 * Workspace: hq_mx_gemm_workspace_bytes(M, N, K) bytes; 0 (and NULL) for many shapes. */
size_t hq_mx_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);
hq_status hq_mx_gemm(const hq_mx_tensor *a, int32_t a_side, const hq_mx_tensor *b, int32_t b_side,
                     void *c, int32_t c_dtype, int32_t accumulate, void *ws, size_t ws_bytes,
                     void *stream);

/* Shapes as in hq.h: X is N x C, W is D x C, dY is N x D, row-major and contiguous. What a call
 * quantizes is rotated as its weight tensor w is.
 * Workspace bytes that the three layer calls below need at most for these shapes. */
size_t hq_mx_workspace_bytes(int64_t N, int64_t C, int64_t D);

/* Forward Y = X W^T; w is the D x C weight tensor (codes). y: N x D, dtype y_dtype. seed: of the
 * rounding of X (NULL: to nearest). save_x: NULL, or receives Q(X) as hq_mx_quantize writes it:
 * codes (required when save_x is given) and, if codes_t is set, the transposed codes that the weight
 * gradient reads. */
hq_status hq_mx_linear_fwd(const void *x, int32_t x_dtype, int64_t N, int64_t C, int64_t D,
                           const hq_mx_tensor *w, const uint32_t *seed, void *y, int32_t y_dtype,
                           hq_mx_tensor *save_x, void *ws, size_t ws_bytes, void *stream);

/* Input gradient dX = dY W; w needs codes_t. dx: N x C. save_g: NULL, or receives Q(dY) (codes
 * required when given, codes_t for the weight gradient). */
hq_status hq_mx_linear_bwd_input(const void *dy, int32_t dy_dtype, int64_t N, int64_t C, int64_t D,
                                 const hq_mx_tensor *w, const uint32_t *seed, void *dx,
                                 int32_t dx_dtype, hq_mx_tensor *save_g, void *ws, size_t ws_bytes,
                                 void *stream);

/* Weight gradient dW = dY^T X from the transposed codes of the saved tensors (saved_g: N x D,
 * saved_x: N x C, of one rotation). dw: D x C, dtype dw_dtype; accumulate != 0 adds to it. */
hq_status hq_mx_linear_bwd_weight(const hq_mx_tensor *saved_g, const hq_mx_tensor *saved_x,
                                  int64_t N, int64_t C, int64_t D, void *dw, int32_t dw_dtype,
                                  int32_t accumulate, void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------- the cache
 * Keys and values of `heads` heads of head_dim elements (64, 128 or 256) each, in pages of `page`
 * tokens (a power of two from 16 to 2^20):
 *   k_codes, v_codes    pages x heads x page x head_dim / 2 bytes
 *   k_scales, v_scales  pages x heads x page x head_dim / 32 bytes
 * contiguous, codes and scales as above with blocks along head_dim. rot: 1, or head_dim for keys and
 * values rotated over the whole head (the dot products of a query rotated likewise are head_dim
 * times the unrotated ones, and a weighted sum of rotated values is the rotated sum). A slot is
 * page_index * page + row; slots need no order. Slots that nothing was written to may hold
 * anything. */
typedef struct {
  uint8_t *k_codes, *v_codes;
  uint8_t *k_scales, *v_scales;
  int64_t pages; /* pages * page at most 2^31 */
  int32_t page, heads, head_dim, rot;
} hq_kv_cache;

/* Write the keys and values of `tokens` tokens to their slots (int64 device array): element d of
 * head h of token t is at k[t * k_token + h * k_head + d], v likewise (strides in elements). A token
 * whose slot lies outside [0, pages * page) is left out (padding of a batch). Slots within must
 * differ: of two tokens for the same slot a mixture may stay. */
hq_status hq_kv_append(const void *k, const void *v, int32_t dtype, int64_t tokens, int64_t k_token,
                       int64_t k_head, int64_t v_token, int64_t v_head, const int64_t *slots,
                       const hq_kv_cache *cache, void *stream);

/* Read keys and/or values of n slots back: k_out, v_out (either may be NULL) n x heads x head_dim,
 * contiguous, rotated back and rounded once. A slot outside [0, pages * page) reads as zeros. */
hq_status hq_kv_read(const hq_kv_cache *cache, const int64_t *slots, int64_t n, void *k_out,
                     void *v_out, int32_t dtype, void *stream);

/* A batch of `seqs` sequences. Device arrays:
 *   q_starts  seqs + 1: the query rows of sequence s are q_starts[s] .. q_starts[s + 1]
 *   lens      seqs: tokens of the sequence in the cache, its new ones (already appended) among them
 *   table     seqs x table_ld: the page of its tokens [p * page, (p + 1) * page)
 * max_q, max_len: bounds on the numbers of query rows and on the lengths (at most 2^30), known on the
 * host; rows and tokens beyond them are not computed and not seen. A page outside [0, pages), or past
 * table_ld, is not seen either; query rows outside the tensor are not touched. (A server's own mistake
 * in these arrays gives wrong answers, but no access outside the buffers.) */
typedef struct {
  const int32_t *q_starts, *lens, *table;
  int64_t table_ld;
  int32_t seqs, max_q, max_len;
  int32_t q_heads; /* a multiple of the cache's heads: head h reads head h / (q_heads / heads) */
  int32_t window;  /* 0: none */
  float scale;     /* of the dot products, before the softmax */
} hq_kv_batch;

/* Bytes of hq_kv_attention's workspace for these bounds (0 where there is nothing to split). A window
 * needs no more than none. */
size_t hq_kv_attention_workspace_bytes(const hq_kv_cache *cache, const hq_kv_batch *batch);

/* out = softmax(scale q K^T) V. Query row i of a sequence with n rows and length len stands at
 * position p = len - n + i and sees the positions j <= p, with a window w those with j > p - w. A row
 * that sees nothing gets zeros (lse: -infinity). q: element d of head h of token t at
 * q[t * q_token + h * q_head + d]; out: tokens x q_heads x head_dim, contiguous, dtype out_dtype. Rows
 * of `tokens` that belong to no sequence are left as they are. lse: NULL, or tokens x q_heads fp32
 * logarithms of the sums of exp(scale q k).
 * Sums, maxima and accumulators are fp32. Queries enter the matrix instruction beside the keys' codes,
 * in parts of 6 bits with a scale for each block of 32: four parts (their sum is within 2^-18 of the
 * block's largest magnitude, or 2^-125 where that is more), six (2^-28) where q or out is fp32. lse has
 * the scores' precision: an fp32 lse of 16-bit q and out is no more precise for being fp32. An infinity
 * or a NaN in a query, or a rotated sum of it past fp32, makes its row NaN. Probabilities enter it as two bf16
 * numbers (their sum is within 2^-17 of the value) or three (2^-25) beside the values, which are exact
 * in bf16.
 * A token changes no row that does not see it, whatever its codes and scales hold; one whose scale is
 * NaN makes the rows that see it NaN (of values: in that block, or all of it if rotated). Accumulators are
 * sums of exp(s - m) v with m the largest score so far: where such a sum of magnitudes reaches 2^128, and in
 * elements where a token that a row sees has a value of 2^128 or more (scale bytes 253 and 254 allow
 * them), the result may be infinite or NaN.
 * Sequences' query rows must not overlap (their results would). */
hq_status hq_kv_attention(const void *q, int32_t q_dtype, int64_t tokens, int64_t q_token,
                          int64_t q_head, const hq_kv_cache *cache, const hq_kv_batch *batch,
                          void *out, int32_t out_dtype, float *lse, void *ws, size_t ws_bytes,
                          void *stream);

#ifdef __cplusplus
}
#endif

#endif /* HQ_MX_H */
