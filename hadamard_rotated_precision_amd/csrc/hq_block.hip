// hq_block.hip — block-scaled FP8 quantizer: E4M3 codes with one scale for each 1 x 128 (ROWS) or
// 128 x 128 (TILES) block, row-major and transposed codes from one read of the source.
//
// For a block with largest magnitude a: s = fp32(a / 448), at least 2^-126 (POW2: rounded up to a
// power of two), r = fp32(1 / s), code = E4M3(v r) to nearest even. 448 is the format's largest
// value. The maxima are taken on the bit patterns of |v| as integers: they order like the
// magnitudes, and an infinity or a NaN comes out on top instead of being skipped.
//
// What bounds it: bytes. R x C elements of e bytes are read once, R C bytes of codes are written
// for each layout.
//
// One workgroup of 256 threads takes a 128 x 128 tile, which holds whole blocks of either
// direction: thread t has columns 8 (t % 16) + [0, 8) of rows 8 (t / 16) + [0, 8) in registers, so
// the source is read once (16 lanes cover 256 contiguous bytes of a 16-bit row), the row maxima
// are a reduction over 16 lanes, the column maxima over the eight rows in registers, four lanes
// and four waves (LDS), and a column's eight codes of a thread pack into two dwords. Those go to
// LDS and leave as 16-byte pieces of the transposed rows.
#include "hq_device.hpp"
#include "hq_launch.hpp"
#include "hq_train_device.hpp"
#include "hq_train_internal.hpp"

namespace hq {

struct BlockQuantArgs {
  const void* src;
  int64_t rows, cols;
  uint8_t* codes;
  int64_t ld;
  uint8_t* codes_t;
  int64_t ld_t;
  float* scales;
  int64_t lds;
  float* scales_t;
  int64_t lds_t;
  int tiles_c;
  int pow2;
  int vec;   // rows start on 16-byte boundaries and hold whole groups of eight elements
};

template <class T, bool TILES>
__global__ __launch_bounds__(256) void block_quant_kernel(BlockQuantArgs g) {
  constexpr int TP = 144;   // LDS pitch of a transposed code row
  __shared__ uint32_t cmax[4][128];
  __shared__ __attribute__((aligned(16))) uint8_t turned[128 * TP];
  const int t = threadIdx.x, cg = t & 15, rg = t >> 4, wave = t >> 6;
  const int tr = blockIdx.x / g.tiles_c, tc = blockIdx.x % g.tiles_c;
  const int64_t r0 = static_cast<int64_t>(tr) * 128, c0 = static_cast<int64_t>(tc) * 128;
  const int64_t row0 = r0 + 8 * rg, col0 = c0 + 8 * cg;
  const int ncol = static_cast<int>(min<int64_t>(max<int64_t>(g.cols - col0, 0), 8));

  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    load8<T>(g.src, (row0 + i) * g.cols + col0, row0 + i < g.rows ? ncol : 0, g.vec, v[i]);

  uint32_t rm[8], cm[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) rm[i] = mag8(v[i]);
  float sr[8], rr[8];
  if constexpr (TILES) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, rm[i]);
    a = shfl_max(shfl_max(max16(a), 16), 32);
    if ((t & 63) == 0) cmax[wave][0] = a;
    __syncthreads();
    a = max(max(cmax[0][0], cmax[1][0]), max(cmax[2][0], cmax[3][0]));
    float s, r;
    block_scale(a, g.pow2, s, r);
    if (t == 0) g.scales[tr * g.lds + tc] = s;
#pragma unroll
    for (int i = 0; i < 8; ++i) sr[i] = s, rr[i] = r;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      block_scale(max16(rm[i]), g.pow2, sr[i], rr[i]);
    }
  }

  if (g.codes) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint2 q = e4m3_codes8(v[i], sr[i], rr[i]);
      // zeros up to the next multiple of 16 columns, which the pitch covers
      if (row0 + i < g.rows && col0 < ((g.cols + 15) & ~int64_t{15}))
        *reinterpret_cast<uint2*>(g.codes + (row0 + i) * g.ld + col0) = q;
      if (!TILES && cg == 0 && row0 + i < g.rows) g.scales[tc * g.lds + row0 + i] = sr[i];
    }
  }
  if (!g.codes_t) return;

  float sc[8], rc[8];
  if constexpr (TILES) {
#pragma unroll
    for (int j = 0; j < 8; ++j) sc[j] = sr[0], rc[j] = rr[0];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      cm[j] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) cm[j] = max(cm[j], mag(v[i][j]));
      cm[j] = shfl_max(shfl_max(cm[j], 16), 32);
      if ((t & 48) == 0) cmax[wave][8 * cg + j] = cm[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = 8 * cg + j;
      block_scale(max(max(cmax[0][c], cmax[1][c]), max(cmax[2][c], cmax[3][c])), g.pow2, sc[j], rc[j]);
      if (rg == 0 && j < ncol) g.scales_t[tr * g.lds_t + col0 + j] = sc[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float u[8] = {v[0][j], v[1][j], v[2][j], v[3][j], v[4][j], v[5][j], v[6][j], v[7][j]};
    *reinterpret_cast<uint2*>(&turned[(8 * cg + j) * TP + 8 * rg]) = e4m3_codes8(u, sc[j], rc[j]);
  }
  __syncthreads();
  // 8 lanes cover the 128 codes of a transposed row
  const int64_t rows16 = (g.rows + 15) & ~int64_t{15};
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int c = (t >> 3) + 32 * p, part = 16 * (t & 7);
    if (c0 + c < g.cols && r0 + part < rows16)
      *reinterpret_cast<uint4*>(g.codes_t + (c0 + c) * g.ld_t + r0 + part) =
          *reinterpret_cast<const uint4*>(&turned[c * TP + part]);
  }
}

// ROWS blocks in the row-major layout alone: sixteen lanes take the 128 columns of a block, a
// thread the same eight columns of R rows (R loads in flight; one where there are few rows).
template <class T, int R>
__global__ __launch_bounds__(256) void block_quant_rows_kernel(BlockQuantArgs g) {
  const int t = threadIdx.x;
  const int span = (g.tiles_c + 15) >> 4;               // workgroups along a row: 16 blocks each
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / span) * R;
  const int64_t col0 = static_cast<int64_t>(blockIdx.x % span) * 2048 + 8 * t;
  const int64_t n = g.cols - col0;
  float v[R][8];
#pragma unroll
  for (int i = 0; i < R; ++i)
    load8<T>(g.src, (row0 + i) * g.cols + col0, row0 + i < g.rows ? n : 0, g.vec, v[i]);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float s, r;
    block_scale(max16(mag8(v[i])), g.pow2, s, r);
    if (row0 + i >= g.rows) continue;
    if (col0 < ((g.cols + 15) & ~int64_t{15}))
      *reinterpret_cast<uint2*>(g.codes + (row0 + i) * g.ld + col0) = e4m3_codes8(v[i], s, r);
    if ((t & 15) == 0 && n > 0) g.scales[(col0 >> 7) * g.lds + row0 + i] = s;
  }
}

hipError_t block_quant_pass(const BlockQuantPass& p, hipStream_t st) {
  const int64_t tiles_r = (p.rows + 127) / 128, tiles_c = (p.cols + 127) / 128;
  BlockQuantArgs a{p.src, p.rows, p.cols, p.codes, p.ld, p.codes_t, p.ld_t, p.scales, p.lds,
                   p.scales_t, p.lds_t, static_cast<int>(tiles_c), p.pow2, p.cols % 8 == 0};
  const int bytes = p.in_dt == DT_F32 ? 4 : 2;
  const double units = static_cast<double>(p.rows) * p.cols * (bytes + (p.codes != nullptr) + (p.codes_t != nullptr));
  const int tok = prof_open(K_ROT_QUANT, units);
  const dim3 grid(static_cast<unsigned>(tiles_r * tiles_c)), block(256);
  if (!p.tiles && !p.codes_t) {
    // four rows a thread once one row a thread would fill the chip twice over
    const int64_t span = (tiles_c + 15) / 16;
    const bool many = p.rows * span >= 4096;
    const dim3 rgrid(static_cast<unsigned>((many ? (p.rows + 3) / 4 : p.rows) * span));
#define HQ_R(T) \
  return many ? launch_k(block_quant_rows_kernel<T, 4>, rgrid, block, st, tok, a) \
              : launch_k(block_quant_rows_kernel<T, 1>, rgrid, block, st, tok, a)
    switch (p.in_dt) {
      case DT_F32: HQ_R(F32);
      case DT_F16: HQ_R(F16);
      case DT_BF16: HQ_R(BF16);
    }
#undef HQ_R
    return hipErrorInvalidValue;
  }
#define HQ_Q(T) \
  return p.tiles ? launch_k(block_quant_kernel<T, true>, grid, block, st, tok, a) \
                 : launch_k(block_quant_kernel<T, false>, grid, block, st, tok, a)
  switch (p.in_dt) {
    case DT_F32: HQ_Q(F32);
    case DT_F16: HQ_Q(F16);
    case DT_BF16: HQ_Q(BF16);
  }
#undef HQ_Q
  return hipErrorInvalidValue;
}

}  // namespace hq
