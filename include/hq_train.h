/*
 * hq_train.h — C ABI of libhq_train.so (MI355X, gfx950): block-scaled FP8 operators and the AdamW
 * step, beside the tensor-wise layer of hq.h (libhq.so, which this library links): the same
 * statuses (hq_status), element types (hq_dtype), launch instrumentation and conventions.
 *
 * What a training step of a linear layer in 8-bit floating point needs around its three products:
 *   hq_block_quantize            a matrix to FP8 E4M3 codes with one scale for each block of 128
 *   hq_block_gemm                the product of two such matrices
 *   hq_block_linear_fwd          Y = X W^T        (any N: single tokens to whole batches)
 *   hq_block_linear_bwd_input    dX = dY W
 *   hq_block_linear_bwd_weight   dW = dY^T X
 *   hq_adamw_step                the update of many tensors at once, states in 32 or 8 bits
 *
 * Shapes as in hq.h: X is N x C, W is D x C, dY is N x D, row-major and contiguous.
 *
 * Conventions (those of hq.h; where this header adds to them it says so):
 *   - Pointers are DEVICE pointers unless a comment says otherwise. Code matrices and workspaces
 *     are 16-byte aligned and code pitches multiples of 16 bytes; everything else (inputs, outputs,
 *     scales, parameters, gradients, states) needs only the alignment of its elements
 *     (HQ_ERR_ALIGN otherwise).
 *   - Every call is asynchronous on `stream`, whose device must be the current one
 *     (HQ_ERR_DEVICE otherwise). No call synchronizes, allocates or records a memset, so all of
 *     them can be captured into a HIP graph.
 *   - The caller owns every buffer; nothing is kept after a call returns. Calls that may run at
 *     the same time need workspaces and outputs of their own (two captured graphs too).
 *   - All argument checks run before any launch; on error nothing is launched or written.
 *   - Results do not depend on the order in which workgroups run: the same call on the same data
 *     gives the same bits. They do depend on the shapes: another number of rows may take another
 *     order of summation.
 *   - hq_profile_start's kinds: products HQ_KIND_GEMM, quantizing HQ_KIND_ROT_QUANT, the joining of
 *     a split contraction and AdamW HQ_KIND_MISC.
 */
#ifndef HQ_TRAIN_H
#define HQ_TRAIN_H

#include "hq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define HQ_TRAIN_ABI_VERSION 1

/* Version of the ABI of this header. */
int32_t hq_train_abi_version(void);

/* ---------------------------------------------------------------- block-scaled FP8 tensors
 * Elements that share a scale:
 * ROWS:  1 x 128 along the axis that the product contracts (activations, gradients): for the
 *        row-major codes 128 columns of one row, for the transposed codes 128 rows of one column;
 * TILES: 128 x 128 (weights); the row-major and the transposed codes are the same numbers.
 * Blocks at the end of an axis are cut short. */
#define HQ_BLOCK 128
typedef enum { HQ_BLOCK_ROWS = 0, HQ_BLOCK_TILES = 1 } hq_block_shape;

/* The scale of a block with largest magnitude a:
 * F32:  s = fp32(a / 448), the E4M3 format's largest value being 448;
 * POW2: the smallest power of two not below fp32(a / 448).
 * Both: at least 2^-126 when a > 0; s = 0 and all codes 0 when a = 0. A code is the E4M3 value
 * nearest to fp32(v * fp32(1/s)), ties to even, saturating at +-448. A block that holds a NaN or
 * an infinity gets s = NaN and zero codes, so every product that reads it is NaN. */
typedef enum { HQ_BSCALE_F32 = 0, HQ_BSCALE_POW2 = 1 } hq_block_scale;

/* A rows x cols matrix in block-scaled FP8. RB = ceil(rows / 128), CB = ceil(cols / 128).
 * codes    rows x cols E4M3 bytes, row pitch ld (>= cols, a multiple of 16), or NULL
 * codes_t  the transpose, cols x rows, row pitch ld_t (>= rows, a multiple of 16), or NULL
 * scales   ROWS:  scales of `codes`: CB x rows, row pitch lds (>= rows);
 *          TILES: of both layouts: RB x CB, row pitch lds (>= CB)
 * scales_t ROWS:  scales of `codes_t`: RB x cols, row pitch lds_t (>= cols); TILES: not used
 * Pitches of scales count floats.
 * Bytes of a code row from its length to the next multiple of 16 are zero (the producer writes
 * them; a caller that brings codes of its own keeps this rule).
 * rows, cols, shape and scale are written by hq_block_quantize and checked by every consumer.
 * A tensor with scale = POW2 promises that every scale is a power of two from 2^-126 up, NaN, or 0
 * with zero codes, as the quantizer writes them: the products may read its exponent alone. */
typedef struct {
  uint8_t *codes;
  uint8_t *codes_t;
  float *scales;
  float *scales_t;
  int64_t rows, cols;
  int64_t ld, ld_t;
  int64_t lds, lds_t;
  int32_t shape; /* hq_block_shape */
  int32_t scale; /* hq_block_scale */
} hq_block_tensor;

/* Quantize a rows x cols matrix (row-major, contiguous, dtype src_dtype) into out->codes and/or
 * out->codes_t (at least one non-NULL) with their scales, from one read of src. The call fills
 * rows, cols, shape and scale of *out (host struct). */
hq_status hq_block_quantize(const void *src, int32_t src_dtype, int64_t rows, int64_t cols,
                            int32_t shape, int32_t scale, hq_block_tensor *out, void *stream);

/* Product of block-scaled matrices, both contiguous along the contraction:
 *   c[m][n] (+)= sum over blocks kb of 128 of sa(m,kb) sb(n,kb) sum_{k in kb} a[m][k] b[n][k]
 * a_side, b_side: which layout of the tensor is the operand, HQ_SIDE_ROWS = codes (rows x cols)
 * or HQ_SIDE_COLS = codes_t (cols x rows); the contracted lengths must agree (HQ_ERR_MISMATCH).
 * c is M x N, contiguous, dtype c_dtype; accumulate != 0 adds to what c holds (the sum is formed
 * in fp32 and rounded once). Any mix of shapes and scale kinds.
 * Sums: products of codes are exact. fp32 outputs are summed by the 16-bit matrix instruction
 * (E4M3 is a subset of fp16), which is as exact as a sum in fp32. 16-bit outputs are summed by the
 * FP8 instruction: of each group of eight consecutive products it cuts every one, towards zero, 13
 * bits below the largest 2^(ea + eb) of the group (2^e <= |code| < 2^(e + 1)), and adds the groups
 * in fp32. Against the root mean square of the results that is an error of 2e-5 on normally
 * distributed data, 7e-5 to 9e-5 with columns 50 times larger than the others or with heavy-tailed
 * gradients, and 1.1e-4 with columns 1000 times larger, where an fp16 output's own rounding is 2e-4
 * and a bf16 one's 1.7e-3. Who needs the exact sum takes an fp32 output.
 * Scales: sa sb is formed in fp32 before it meets the block's sum. While it is at least 2^-126 the
 * above holds. A smaller one has a step of 2^-149: an error of at most 2^-150 times the sum of the
 * block's |a b|, so below 2^-125. From 2^128 on it is infinite, and the outputs that read the block
 * are infinite or NaN. (Two POW2 tensors with 16-bit outputs may escape either limit: the
 * instruction then adds their exponents.)
 * Workspace: hq_block_gemm_workspace_bytes(M, N, K) bytes; 0 (and NULL) for many shapes. */
typedef enum { HQ_SIDE_ROWS = 0, HQ_SIDE_COLS = 1 } hq_block_side;

size_t hq_block_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);
hq_status hq_block_gemm(const hq_block_tensor *a, int32_t a_side, const hq_block_tensor *b,
                        int32_t b_side, void *c, int32_t c_dtype, int32_t accumulate, void *ws,
                        size_t ws_bytes, void *stream);

/* Workspace bytes that the three layer calls below need at most for these shapes. */
size_t hq_block_workspace_bytes(int64_t N, int64_t C, int64_t D);

/* Forward Y = X W^T. X (N x C, dtype x_dtype) is quantized in ROWS blocks with scale kind
 * `scale`; w is the D x C weight tensor (codes; TILES or ROWS) that hq_block_quantize wrote.
 * y: N x D, dtype y_dtype. save_x: NULL, or receives Q(X) as hq_block_quantize writes it: codes
 * (required when save_x is given) and, if codes_t is set, the transposed codes in blocks of 128
 * tokens that the weight gradient reads. */
hq_status hq_block_linear_fwd(const void *x, int32_t x_dtype, int64_t N, int64_t C, int64_t D,
                              const hq_block_tensor *w, int32_t scale, void *y, int32_t y_dtype,
                              hq_block_tensor *save_x, void *ws, size_t ws_bytes, void *stream);

/* Input gradient dX = dY W. dY (N x D) is quantized in ROWS blocks; w needs codes_t. dx: N x C.
 * save_g: NULL, or receives Q(dY) (codes required when given, codes_t for the weight gradient). */
hq_status hq_block_linear_bwd_input(const void *dy, int32_t dy_dtype, int64_t N, int64_t C,
                                    int64_t D, const hq_block_tensor *w, int32_t scale, void *dx,
                                    int32_t dx_dtype, hq_block_tensor *save_g, void *ws,
                                    size_t ws_bytes, void *stream);

/* Weight gradient dW = dY^T X from the transposed codes of the saved tensors (saved_g: N x D,
 * saved_x: N x C). dw: D x C, dtype dw_dtype; accumulate != 0 adds to it (gradients summed over
 * micro-batches). */
hq_status hq_block_linear_bwd_weight(const hq_block_tensor *saved_g,
                                     const hq_block_tensor *saved_x, int64_t N, int64_t C,
                                     int64_t D, void *dw, int32_t dw_dtype, int32_t accumulate,
                                     void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------- AdamW
 * One step of AdamW (decoupled weight decay) over many tensors:
 *   g = grad_scale * grad          m = beta1 m + (1 - beta1) g      v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * in fp32, p rounded to nearest to its dtype; `copy` (optional) receives the new p in copy_dtype.
 * States of 32 bits: m and v are fp32. States of 8 bits: m and v are E4M3 codes with one scale
 * for each 128 consecutive elements (m_scales, v_scales: ceil(n / 128) floats); m stands for
 * code * s and v for (code * s)^2. New states are rounded at random to one of the two
 * neighbouring codes so that the mean is m and v themselves (a rounding to nearest would keep v
 * from ever decaying: a step moves it by 1 - beta2 of itself, a code by an eighth); a v above
 * zero keeps a code above zero. p is updated with m and v before that rounding. A block that
 * holds a NaN or an infinity gets a NaN scale.
 * The random numbers come from (seed, step, index of the tensor, index of the element) alone:
 *   mix(h):  h ^= h >> 16; h *= 2654435761; h ^= h >> 15; h *= 2891336453; h ^= h >> 16
 *   key   =  mix(seed + 2654435761 step);   k = key + 0x9E3779B9 (tensor + 1)
 *   u     =  mix((low 32 bits of element) ^ (k + 0x632BE5AB (element >> 32)))    (all mod 2^32)
 * m rounds up where its fraction between the two codes plus (u mod 2^16) / 2^16 reaches 1, v where
 * (u >> 16) / 2^16 is below (v - low^2) / (high^2 - low^2). The multipliers are Knuth's
 * multiplicative hash and one of L'Ecuyer's tables for modulus 2^32 (Math. Comp. 68, 1999). */
typedef struct {
  void *p;           /* n parameters, param_dtype */
  const void *grad;  /* n gradients, grad_dtype */
  void *m, *v;       /* n states: fp32, or E4M3 bytes */
  float *m_scales;   /* 8-bit states: ceil(n / 128) floats each; NULL for 32 bits */
  float *v_scales;
  void *copy;        /* NULL, or n elements of copy_dtype */
  int64_t n;         /* at most 2^34; 0 is skipped */
  float weight_decay;
  int32_t reserved;  /* 0 */
} hq_adamw_tensor;

typedef struct {
  double lr, beta1, beta2, eps; /* 0 <= beta < 1, eps >= 1.2e-38 (fp32 normal), lr >= 0 */
  int32_t param_dtype, grad_dtype, copy_dtype; /* hq_dtype */
  int32_t state_bits;                          /* 32 or 8 */
  uint32_t seed;                               /* of the rounding of 8-bit states */
  int32_t reserved;                            /* 0 */
} hq_adamw_config;

/* What changes from step to step. */
typedef struct {
  float lr;
  float step_size;       /* lr / (1 - beta1^t) */
  float inv_sqrt_bias2;  /* 1 / sqrt(1 - beta2^t) */
  float grad_scale;
  uint32_t key;          /* of the step's random numbers */
} hq_adamw_scalars;

/* The scalars of step t = 1, 2, ... (host memory; no GPU needed). */
hq_status hq_adamw_scalars_at(const hq_adamw_config *cfg, int64_t step, double grad_scale,
                              hq_adamw_scalars *out);

/* One step over `count` tensors (host array, read before the call returns). The step's scalars
 * are those in device memory when device_scalars is given (a captured step reads what it holds at
 * each replay; grad_scale may be written there by a kernel), else those of host_scalars.
 * p, m, v, copy and the scales of all tensors must overlap neither each other nor a gradient; a
 * copy of the parameters' type may be its own p.
 * No workspace. */
hq_status hq_adamw_step(const hq_adamw_tensor *tensors, int32_t count, const hq_adamw_config *cfg,
                        const hq_adamw_scalars *host_scalars,
                        const hq_adamw_scalars *device_scalars, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* HQ_TRAIN_H */
