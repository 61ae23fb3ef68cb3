// hq_block.hip — block-scaled FP8 quantizer: E4M3 codes with one scale for each 1 x 128 (ROWS) or
// 128 x 128 (TILES) block, row-major and transposed codes from one read of the source.
//
// For a block with largest magnitude a: s = fp32(a / 448), at least 2^-126 (POW2: rounded up to a
// power of two), r = fp32(1 / s), code = E4M3(v r) to nearest even. 448 is the format's largest
// value. The maxima are taken on the bit patterns of |v| as integers: they order like the
// magnitudes, and an infinity or a NaN comes out on top instead of being skipped.
//
// What bounds it: bytes. R x C elements of e bytes are read once, R C bytes of codes are written
// for each layout: 8192 x 13824 bf16 into both layouts takes 86 to 96 us (4.8 to 5.3 TB/s; a large
// copy reaches 4.8), 11008 x 4096 fp32 into tiles 55 us (4.9 TB/s).
//
// One workgroup of 256 threads takes a 128 x 128 tile, which holds whole blocks of either
// direction: thread t has columns 8 (t % 16) + [0, 8) of rows 8 (t / 16) + [0, 8) in registers, so
// the source is read once (16 lanes cover 256 contiguous bytes of a 16-bit row), the row maxima
// are a reduction over 16 lanes, the column maxima over the eight rows in registers, four lanes
// and four waves (LDS), and a column's eight codes of a thread pack into two dwords. Those go to
// LDS and leave as 16-byte pieces of the transposed rows. With elements widened in registers and
// a scale computed by every lane the same pass took 166 us: two workgroups per compute unit and
// two divisions per row and column in all 16 lanes.
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
};

// Lane l of each 16 gets the largest of the sixteen lanes' m[l % 8]: each step halves the values a
// lane still carries, so 8 x 16 maxima take 8 exchanges instead of 32.
__device__ inline uint32_t max16_of8(const uint32_t (&m)[8], int lane) {
  uint32_t a[4], b[2], c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t keep = (lane & 1) ? m[2 * i + 1] : m[2 * i], give = (lane & 1) ? m[2 * i] : m[2 * i + 1];
    a[i] = max(keep, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(give), 0xB1, 0xF, 0xF, false)));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t keep = (lane & 2) ? a[2 * i + 1] : a[2 * i], give = (lane & 2) ? a[2 * i] : a[2 * i + 1];
    b[i] = max(keep, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(give), 0x4E, 0xF, 0xF, false)));
  }
  {
    const uint32_t keep = (lane & 4) ? b[1] : b[0], give = (lane & 4) ? b[0] : b[1];
    c = max(keep, static_cast<uint32_t>(__shfl_xor(static_cast<int>(give), 4, 64)));
  }
  return max(c, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(c), 0x128, 0xF, 0xF, false)));   // lane ^ 8
}

// Lane K of each 16 lanes, in all of them.
template <int K>
__device__ inline float bcast16(float x) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x150 + K, 0xF, 0xF, false));
}
__device__ inline void bcast16_first8(float x, float (&r)[8]) {
  r[0] = bcast16<0>(x); r[1] = bcast16<1>(x); r[2] = bcast16<2>(x); r[3] = bcast16<3>(x);
  r[4] = bcast16<4>(x); r[5] = bcast16<5>(x); r[6] = bcast16<6>(x); r[7] = bcast16<7>(x);
}

template <class T, bool TILES>
__global__ __launch_bounds__(256) void block_quant_kernel(BlockQuantArgs g) {
  __shared__ uint32_t cmax[4][128];
  __shared__ __attribute__((aligned(16))) float rcol[128];
  // transposed codes: 128 bytes per column; the 8-byte slot of a thread's eight rows is XORed with
  // twice the column's group of eight, so that a wave's writes spread over the banks and 16-byte
  // pieces stay whole
  __shared__ __attribute__((aligned(16))) uint8_t turned[128 * 128];
  const int t = threadIdx.x, cg = t & 15, rg = t >> 4, wave = t >> 6;
  const int tr = blockIdx.x / g.tiles_c, tc = blockIdx.x % g.tiles_c;
  const int64_t r0 = static_cast<int64_t>(tr) * 128, c0 = static_cast<int64_t>(tc) * 128;
  const int64_t row0 = r0 + 8 * rg, col0 = c0 + 8 * cg;
  const int ncol = static_cast<int>(min<int64_t>(max<int64_t>(g.cols - col0, 0), 8));

  Tile8<T> x;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    x.load(i, g.src, (row0 + i) * g.cols + col0, row0 + i < g.rows ? ncol : 0);

  float rr[8];
  if constexpr (TILES) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, x.row_mag(i));
    a = shfl_max(shfl_max(max16(a), 16), 32);
    if ((t & 63) == 0) cmax[wave][0] = a;
    __syncthreads();
    a = max(max(cmax[0][0], cmax[1][0]), max(cmax[2][0], cmax[3][0]));
    float s, r;
    block_scale(Tile8<T>::widen(a), g.pow2, s, r);
    if (t == 0) g.scales[tr * g.lds + tc] = s;
#pragma unroll
    for (int i = 0; i < 8; ++i) rr[i] = r;
  } else if (g.codes) {
    uint32_t m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = x.row_mag(i);
    float s, r;     // of row t % 8 of the thread's eight
    block_scale(Tile8<T>::widen(max16_of8(m, t)), g.pow2, s, r);
    if (cg < 8 && row0 + cg < g.rows) g.scales[tc * g.lds + row0 + cg] = s;
    bcast16_first8(r, rr);
  }

  if (g.codes) {
    const bool in = col0 < ((g.cols + 15) & ~int64_t{15});   // zeros up to the next multiple of 16
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = x.value(i, j);
      const uint2 q = e4m3_codes8(v, rr[i]);
      if (row0 + i < g.rows && in) *reinterpret_cast<uint2*>(g.codes + (row0 + i) * g.ld + col0) = q;
    }
  }
  if (!g.codes_t) return;

  float rc[8];
  if constexpr (TILES) {
#pragma unroll
    for (int j = 0; j < 8; ++j) rc[j] = rr[0];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t m = shfl_max(shfl_max(x.col_mag(j), 16), 32);
      if ((t & 48) == 0) cmax[wave][8 * cg + j] = m;
    }
    __syncthreads();
    if (t < 128) {    // one thread per column
      float s, r;
      block_scale(Tile8<T>::widen(max(max(cmax[0][t], cmax[1][t]), max(cmax[2][t], cmax[3][t]))), g.pow2, s, r);
      rcol[t] = r;
      if (c0 + t < g.cols) g.scales_t[tr * g.lds_t + c0 + t] = s;
    }
    __syncthreads();
    const float4 a = *reinterpret_cast<const float4*>(&rcol[8 * cg]), b = *reinterpret_cast<const float4*>(&rcol[8 * cg + 4]);
    rc[0] = a.x; rc[1] = a.y; rc[2] = a.z; rc[3] = a.w;
    rc[4] = b.x; rc[5] = b.y; rc[6] = b.z; rc[7] = b.w;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x.value(i, j);
    *reinterpret_cast<uint2*>(&turned[(8 * cg + j) * 128 + 8 * (rg ^ (2 * (cg & 7)))]) = e4m3_codes8(v, rc[j]);
  }
  __syncthreads();
  // 8 lanes cover the 128 codes of a transposed row
  const int64_t rows16 = (g.rows + 15) & ~int64_t{15};
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int c = (t >> 3) + 32 * p, part = t & 7;
    if (c0 + c < g.cols && r0 + 16 * part < rows16)
      *reinterpret_cast<uint4*>(g.codes_t + (c0 + c) * g.ld_t + r0 + 16 * part) =
          *reinterpret_cast<const uint4*>(&turned[c * 128 + 8 * ((2 * part) ^ (2 * ((c >> 3) & 7)))]);
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
    load8<T>(g.src, (row0 + i) * g.cols + col0, row0 + i < g.rows ? n : 0, v[i]);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float s, r;
    block_scale(max16(mag8(v[i])), g.pow2, s, r);
    if (row0 + i >= g.rows) continue;
    if (col0 < ((g.cols + 15) & ~int64_t{15}))
      *reinterpret_cast<uint2*>(g.codes + (row0 + i) * g.ld + col0) = e4m3_codes8(v[i], r);
    if ((t & 15) == 0 && n > 0) g.scales[(col0 >> 7) * g.lds + row0 + i] = s;
  }
}

hipError_t block_quant_pass(const BlockQuantPass& p, hipStream_t st) {
  const int64_t tiles_r = (p.rows + 127) / 128, tiles_c = (p.cols + 127) / 128;
  BlockQuantArgs a{p.src, p.rows, p.cols, p.codes, p.ld, p.codes_t, p.ld_t, p.scales, p.lds,
                   p.scales_t, p.lds_t, static_cast<int>(tiles_c), p.pow2};
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
