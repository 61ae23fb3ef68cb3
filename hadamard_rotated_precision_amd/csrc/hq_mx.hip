// hq_mx.hip — microscaled 4-bit quantizer: E2M1 codes with one power-of-two scale for each 32
// elements along a row, of the matrix and/or of its transpose from one read of the source, rotated
// by H_32 within each block if asked for; and the way back.
//
// The scale is the smallest power of two s with a <= 6 s (a: the block's largest magnitude, taken on
// bit patterns so that an infinity or a NaN comes out on top); v / s is exact, so a code is the value
// nearest to v / s without an intermediate rounding.
//
// What bounds it: R x C elements of e bytes are read once, 17/32 R C bytes are written for each layout.
// One layout goes at the rate of its bytes (1000 x 5120: 5.8 us, launch included), the way back too (from
// 8192 x 13824 45 us: 286 MB, 6.4 TB/s, in part out of caches). Both layouts from 8192 x 13824 bf16, rotated,
// take 100 us to nearest (347 MB, 3.5 TB/s; a copy 72), the vector pipe busy for 78 % of the time and LDS
// conflicts for 17 % of the cycles, and 180 to 192 rounded at random, where the vector pipe is the bound (95 %: the
// two hashes' multiplications at a quarter of its rate, for each pair and layout).
#include "hq_device.hpp"
#include "hq_launch.hpp"
#include "hq_mx_device.hpp"
#include "hq_mx_internal.hpp"

namespace hq {

struct MxQuantArgs {
  const void* src;
  int64_t rows, cols;
  const uint32_t* seed;
  uint8_t* codes;
  int64_t ld;
  uint8_t* codes_t;
  int64_t ld_t;
  uint8_t* scales;
  int64_t lds;
  uint8_t* scales_t;
  int64_t lds_t;
  int tiles_c;
};

__device__ inline int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// The row-major layout alone: four lanes take a block, a thread the same eight columns of R rows
// (R loads in flight; one where there are few rows).
template <class T, int ROT, bool RANDOM, int R>
__global__ __launch_bounds__(256) void mx_quant_rows_kernel(MxQuantArgs g) {
  const int t = threadIdx.x;
  const int span = static_cast<int>((g.cols + 2047) >> 11);     // workgroups along a row
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / span) * R;
  const int64_t col0 = static_cast<int64_t>(blockIdx.x % span) * 2048 + 8 * t;
  const int64_t n = g.cols - col0;
  uint32_t seed = 0;
  if constexpr (RANDOM) seed = *g.seed;
  float v[R][8];
#pragma unroll
  for (int i = 0; i < R; ++i)
    load8<T>(g.src, (row0 + i) * g.cols + col0, row0 + i < g.rows ? n : 0, v[i]);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if constexpr (ROT > 1) rotate_lanes<ROT>(v[i], t);
    const int byte = mx_scale_byte(quad_max(mag8(v[i])));
    const uint32_t key = RANDOM ? mx_row_key(seed, row0 + i) : 0u;
    const uint32_t w = mx_codes8<RANDOM>(v[i], byte, key, static_cast<uint32_t>(col0 >> 1));
    if (row0 + i >= g.rows) continue;
    const int64_t b = col0 >> 5, nb = (g.cols + 31) >> 5;
    if (b < nb) *reinterpret_cast<uint32_t*>(g.codes + (row0 + i) * g.ld + (col0 >> 1)) = w;
    if ((t & 3) == 0 && b < up(nb, 16)) g.scales[(row0 + i) * g.lds + b] = b < nb ? byte : 0;
  }
}

// Both layouts, or the transposed one: a workgroup takes a 128 x 128 tile, which holds whole blocks
// of either direction; thread t has columns 8 (t % 16) + [0, 8) of rows 8 (t / 16) + [0, 8), so a
// wave has a band of 32 rows, whole blocks of the transpose: strides 1, 2, 4 are in registers in
// either direction, 8 and 16 across lanes.
template <class T, int ROT, bool RANDOM>
__global__ __launch_bounds__(256) void mx_quant_kernel(MxQuantArgs g) {
  // 64 code bytes of a row and of a column, at a pitch of 80 (16-byte pieces): a wave's dwords of its rows
  // spread over the banks, those of its columns (neighbouring lanes 8 x 80 bytes apart) meet eight of them
  __shared__ __attribute__((aligned(16))) uint8_t straight[128 * 80], turned[128 * 80];
  __shared__ __attribute__((aligned(4))) uint8_t rs[128][4], cs[128][4];
  const int t = threadIdx.x, cg = t & 15, rg = t >> 4, wave = t >> 6;
  const int tr = blockIdx.x / g.tiles_c, tc = blockIdx.x % g.tiles_c;
  const int64_t r0 = static_cast<int64_t>(tr) * 128, c0 = static_cast<int64_t>(tc) * 128;
  const int64_t row0 = r0 + 8 * rg, col0 = c0 + 8 * cg;
  const int ncol = static_cast<int>(min<int64_t>(max<int64_t>(g.cols - col0, 0), 8));
  uint32_t seed = 0;
  if constexpr (RANDOM) seed = *g.seed;

  Tile8<T> x;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    x.load(i, g.src, (row0 + i) * g.cols + col0, row0 + i < g.rows ? ncol : 0);

  if (g.codes) {
    const bool in = col0 < up(g.cols, 32);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = x.value(i, j);
      if constexpr (ROT > 1) rotate_lanes<ROT>(v, t);
      const int byte = mx_scale_byte(quad_max(mag8(v)));
      const uint32_t key = RANDOM ? mx_row_key(seed, row0 + i) : 0u;
      const uint32_t w = mx_codes8<RANDOM>(v, byte, key, static_cast<uint32_t>(col0 >> 1));
      *reinterpret_cast<uint32_t*>(&straight[(8 * rg + i) * 80 + 4 * cg]) = w;
      if ((t & 3) == 0) rs[8 * rg + i][cg >> 2] = in ? byte : 0;
    }
  }
  if (g.codes_t) {
    const bool in = row0 < up(g.rows, 32);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      float a[8], b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = x.value(i, j), b[i] = x.value(i, j + 1);
      if constexpr (ROT > 1) {
        fwht_inreg<8, 8>(a);
        fwht_inreg<8, 8>(b);
#pragma unroll
        for (int i = 0; i < 8; ++i) fwht_swap<16>(a[i], b[i]);
#pragma unroll
        for (int i = 0; i < 8; ++i) fwht_swap<32>(a[i], b[i]);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float (&v)[8] = e ? b : a;
        const int byte = mx_scale_byte(swap_max<32>(swap_max<16>(mag8(v))));
        const uint32_t key = RANDOM ? mx_row_key(seed + 0x9E3779B9u, col0 + j + e) : 0u;
        const uint32_t w = mx_codes8<RANDOM>(v, byte, key, static_cast<uint32_t>(row0 >> 1));
        const int c = 8 * cg + j + e;
        *reinterpret_cast<uint32_t*>(&turned[c * 80 + 4 * rg]) = w;
        if ((t & 48) == 0) cs[c][wave] = in ? byte : 0;
      }
    }
  }
  __syncthreads();
  if (t < 128) {
    // four scales of a row; the last tile also clears them up to the next multiple of 16
    if (g.codes && r0 + t < g.rows) {
      uint32_t* s = reinterpret_cast<uint32_t*>(g.scales + (r0 + t) * g.lds + 4 * static_cast<int64_t>(tc));
      *s = *reinterpret_cast<const uint32_t*>(rs[t]);
      if (tc == g.tiles_c - 1)
        for (int64_t b = 4 * (tc + 1); b < up((g.cols + 31) >> 5, 16); b += 4) *++s = 0;
    }
  } else if (g.codes_t && c0 + t - 128 < g.cols) {
    uint32_t* s = reinterpret_cast<uint32_t*>(g.scales_t + (c0 + t - 128) * g.lds_t + 4 * static_cast<int64_t>(tr));
    *s = *reinterpret_cast<const uint32_t*>(cs[t - 128]);
    if (r0 + 128 >= g.rows)
      for (int64_t b = 4 * (tr + 1); b < up((g.rows + 31) >> 5, 16); b += 4) *++s = 0;
  }
  // four lanes cover the 64 bytes of a row
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int c = (t >> 2) + 64 * p, part = t & 3;
    if (g.codes && r0 + c < g.rows && c0 + 32 * part < g.cols)
      *reinterpret_cast<uint4*>(g.codes + (r0 + c) * g.ld + (c0 >> 1) + 16 * part) =
          *reinterpret_cast<const uint4*>(&straight[c * 80 + 16 * part]);
    if (g.codes_t && c0 + c < g.cols && r0 + 32 * part < g.rows)
      *reinterpret_cast<uint4*>(g.codes_t + (c0 + c) * g.ld_t + (r0 >> 1) + 16 * part) =
          *reinterpret_cast<const uint4*>(&turned[c * 80 + 16 * part]);
  }
}

// rows x cols values of codes: a thread takes eight of each of R rows, four lanes a block.
template <class Out, int ROT, int R>
__global__ __launch_bounds__(256) void mx_dequant_kernel(MxOperand q, int64_t rows, int64_t cols, void* dst) {
  const int t = threadIdx.x;
  const int span = static_cast<int>((cols + 2047) >> 11);
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / span) * R;
  const int64_t col0 = static_cast<int64_t>(blockIdx.x % span) * 2048 + 8 * t;
  const bool in = col0 < up(cols, 32);
  uint32_t w[R];
  int byte[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t row = min(row0 + i, rows - 1);
    w[i] = in ? *reinterpret_cast<const uint32_t*>(q.codes + row * q.ld + (col0 >> 1)) : 0u;
    byte[i] = in ? q.scales[row * q.lds + (col0 >> 5)] : 0;
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float v[8];
    mx_values8(w[i], v);
    // sums of 32 codes are exact; byte 0 stands for 2^-127, byte 255 for NaN
    if constexpr (ROT > 1) rotate_lanes<ROT>(v, t);
    const float s = byte[i] == 255 ? __uint_as_float(0x7FC00000u) : byte[i] ? mx_scale(byte[i]) : 5.87747175e-39f;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] * (1.0f / ROT) * s;
    if (col0 < cols && row0 + i < rows) store8_stream<Out>(dst, (row0 + i) * cols + col0, cols - col0, v);
  }
}

template <class T, int ROT, bool RANDOM>
static hipError_t launch_quant(const MxQuantPass& p, const MxQuantArgs& a, hipStream_t st, int tok) {
  const int64_t tiles_r = (p.rows + 127) / 128;
  const dim3 block(256);
  if (p.codes_t)
    return launch_k(mx_quant_kernel<T, ROT, RANDOM>, dim3(static_cast<unsigned>(tiles_r * a.tiles_c)), block, st, tok, a);
  // four rows a thread once one row a thread would fill the chip twice over: on the way back from
  // 8192 x 13824 one took 80 us, four 45
  const int64_t span = (p.cols + 2047) / 2048;
  if (p.rows * span >= 4096)
    return launch_k(mx_quant_rows_kernel<T, ROT, RANDOM, 4>, dim3(static_cast<unsigned>((p.rows + 3) / 4 * span)), block, st, tok, a);
  return launch_k(mx_quant_rows_kernel<T, ROT, RANDOM, 1>, dim3(static_cast<unsigned>(p.rows * span)), block, st, tok, a);
}

template <class T>
static hipError_t launch_type(const MxQuantPass& p, const MxQuantArgs& a, hipStream_t st, int tok) {
  if (p.rot == 1) return p.seed ? launch_quant<T, 1, true>(p, a, st, tok) : launch_quant<T, 1, false>(p, a, st, tok);
  return p.seed ? launch_quant<T, 32, true>(p, a, st, tok) : launch_quant<T, 32, false>(p, a, st, tok);
}

hipError_t mx_quant_pass(const MxQuantPass& p, hipStream_t st) {
  const MxQuantArgs a{p.src, p.rows, p.cols, p.seed, p.codes, p.ld, p.codes_t, p.ld_t, p.scales, p.lds,
                      p.scales_t, p.lds_t, static_cast<int>((p.cols + 127) / 128)};
  const int layouts = (p.codes != nullptr) + (p.codes_t != nullptr);
  const double units = static_cast<double>(p.rows) * p.cols * ((p.in_dt == DT_F32 ? 4 : 2) + layouts * 17.0 / 32.0);
  const int tok = prof_open(K_ROT_QUANT, units);
  switch (p.in_dt) {
    case DT_F32: return launch_type<F32>(p, a, st, tok);
    case DT_F16: return launch_type<F16>(p, a, st, tok);
    case DT_BF16: return launch_type<BF16>(p, a, st, tok);
  }
  return hipErrorInvalidValue;
}

hipError_t mx_dequant_pass(const MxOperand& q, int64_t rows, int64_t cols, int rot, void* dst, int out_dt, hipStream_t st) {
  const double units = static_cast<double>(rows) * cols * ((out_dt == DT_F32 ? 4 : 2) + 17.0 / 32.0);
  const int tok = prof_open(K_ROT_STORE, units);
  const int64_t span = (cols + 2047) / 2048;
  const bool many = rows * span >= 4096;
  const dim3 grid(static_cast<unsigned>((many ? (rows + 3) / 4 : rows) * span)), block(256);
#define HQ_R(T, ROT)                                                                               \
  (many ? launch_k(mx_dequant_kernel<T, ROT, 4>, grid, block, st, tok, q, rows, cols, dst)         \
        : launch_k(mx_dequant_kernel<T, ROT, 1>, grid, block, st, tok, q, rows, cols, dst))
#define HQ_D(T) return rot == 1 ? HQ_R(T, 1) : HQ_R(T, 32)
  switch (out_dt) {
    case DT_F32: HQ_D(F32);
    case DT_F16: HQ_D(F16);
    case DT_BF16: HQ_D(BF16);
  }
#undef HQ_D
#undef HQ_R
  return hipErrorInvalidValue;
}

}  // namespace hq
