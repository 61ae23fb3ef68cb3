// hq_mx_device.hpp — device helpers shared by the kernels of include/hq_mx.h: scales and codes of a
// block of 32, and the rotation of values that lie eight to a lane.
#pragma once

#include "hq_device.hpp"
#include "hq_train_device.hpp"

namespace hq {

// The scale byte of a block whose largest magnitude has the bit pattern `a`: the smallest e with
// a <= 1.5 * 2^(e + 2). Adding all but the top bit of the fraction carries into the exponent exactly
// where the significand is above 1.5.
__device__ inline int mx_scale_byte(uint32_t a) {
  const int b = static_cast<int>((a + 0x3FFFFFu) >> 23) - 2;
  return a >= 0x7F800000u ? 255 : max(b, 1);
}
// The scale itself; byte 255 gives an infinity's pattern, which the conversions below read as NaN.
__device__ inline float mx_scale(int byte) { return __uint_as_float(static_cast<uint32_t>(byte) << 23); }

// The 32-bit mixing steps of the random rounding (the multipliers: Knuth's multiplicative hash and
// one of L'Ecuyer's tables for modulus 2^32, Math. Comp. 68, 1999).
__device__ inline uint32_t mix32(uint32_t h) {
  h ^= h >> 16;
  h *= 2654435761u;
  h ^= h >> 15;
  h *= 2891336453u;
  return h ^ (h >> 16);
}
__device__ inline uint32_t mx_row_key(uint32_t seed, int64_t row) {
  return mix32(seed + 2654435761u * static_cast<uint32_t>(row));
}

// y = 2 v / s, rounded at random with the 16 bits u to twice a value that E2M1 has, toward zero after u
// is added to the magnitude: from |y| = 2 on to the significand's dropped 22 bits, 64 u of their
// 2^22 carrying into the kept one, below it to the fraction, for the step is uniform there.
__device__ inline float mx_random(float y, uint32_t u) {
  const float high = __uint_as_float((__float_as_uint(y) + (u << 6)) & 0xFFC00000u);
  const float low = __builtin_truncf(__builtin_fmaf(static_cast<float>(u), copysignf(1.0f / 65536.0f, y), y));
  return fabsf(y) >= 2.0f ? high : low;
}

// Eight codes, packed low first. key, pair: the row's key and half the first column's index.
template <bool RANDOM>
__device__ inline uint32_t mx_codes8(const float (&v)[8], int byte, uint32_t key, uint32_t pair) {
  uint32_t w = 0;
  if constexpr (RANDOM) {
    const float r = __uint_as_float(static_cast<uint32_t>(255 - byte) << 23);   // 2 / s, exact
    float y[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t h = mix32(key ^ (pair + j));
      y[2 * j] = mx_random(v[2 * j] * r, h & 0xFFFFu);
      y[2 * j + 1] = mx_random(v[2 * j + 1] * r, h >> 16);
    }
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[0], y[1], 2.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[2], y[3], 2.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[4], y[5], 2.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[6], y[7], 2.0f, 3);
  } else {
    const float s = mx_scale(byte);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
  }
  return byte == 255 ? 0u : w;
}

// The values of eight codes (without their scale).
__device__ inline void mx_values8(uint32_t w, float (&v)[8]) {
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
  const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
  const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
  v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1];
  v[4] = c[0]; v[5] = c[1]; v[6] = d[0]; v[7] = d[1];
}

// H_K on K values that lie eight to a lane in K / 8 consecutive lanes, strides in rising order.
template <int K>
__device__ inline void rotate_lanes(float (&v)[8], int lane) {
  fwht_inreg<K, 8>(v);
#pragma unroll
  for (int m = 1; 8 * m < K; m <<= 1) fwht_xlane(v, lane, m);
}

// A butterfly stage over lanes l and l ^ M (M = 16 or 32) of two values at once: swapping a's upper lanes with
// b's lower ones puts the halves of a into the lower lanes and those of b into the upper ones, so one sum and one
// difference serve both; a second swap puts them back. The same sums as fwht_xlane_c, without the LDS permute.
template <int M>
__device__ inline void swap_lanes(uint32_t& a, uint32_t& b) {
  const auto r = M == 16 ? __builtin_amdgcn_permlane16_swap(a, b, false, false) : __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
template <int M>
__device__ inline void fwht_swap(float& a, float& b) {
  uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
  swap_lanes<M>(x, y);
  const float s = __uint_as_float(x) + __uint_as_float(y), d = __uint_as_float(x) - __uint_as_float(y);
  x = __float_as_uint(s), y = __float_as_uint(d);
  swap_lanes<M>(x, y);
  a = __uint_as_float(x);
  b = __uint_as_float(y);
}
// The larger of lanes l and l ^ M, in both.
template <int M>
__device__ inline uint32_t swap_max(uint32_t x) {
  uint32_t y = x;
  swap_lanes<M>(x, y);
  return max(x, y);
}

// Largest of the four lanes of a quad, in all of them.
__device__ inline uint32_t quad_max(uint32_t x) {
  x = max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0xB1, 0xF, 0xF, false)));
  return max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x4E, 0xF, 0xF, false)));
}

}  // namespace hq
