// hq_train_device.hpp — device helpers shared by the kernels of include/hq_train.h: groups of eight
// consecutive elements (whole ones with wide accesses, at any alignment; stores keep NaN, where the
// bf16 store of hq_device.hpp takes finite values only), block scales and codes, and the products
// of one block of K.
#pragma once

#include "hq_device.hpp"

namespace hq {

__device__ inline void unpack8(uint4 q, bool bf16, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint16_t lo = static_cast<uint16_t>(w[j] & 0xFFFFu), hi = static_cast<uint16_t>(w[j] >> 16);
    v[2 * j] = bf16 ? BF16::from_bits(lo) : F16::from_bits(lo);
    v[2 * j + 1] = bf16 ? BF16::from_bits(hi) : F16::from_bits(hi);
  }
}

// Elements [i, i + 8) of base, those past the first n as 0. A whole group is one or two 16-byte
// loads whatever its alignment: rows of an odd length start anywhere, and the hardware takes such
// loads (a 1000 x 1030 fp32 matrix, element by element at the odd rows: 12 us, so: 6).
template <class T>
__device__ inline void load8(const void* base, int64_t i, int64_t n, float (&v)[8]) {
  if (n >= 8) {
    const char* p = static_cast<const char*>(base) + i * T::bytes;
    if constexpr (T::bytes == 4) {
      __builtin_memcpy(v, p, 32);
    } else {
      uint4 q;
      __builtin_memcpy(&q, p, 16);
      unpack8(q, T::is_bf16, v);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? T::load(base, i + j) : 0.0f;
  }
}

template <class T>
__device__ inline void put_one(void* base, int64_t i, float v) {
  if constexpr (T::is_bf16) static_cast<uint16_t*>(base)[i] = static_cast<uint16_t>(T::pack2(v, 0.0f));
  else T::store(base, i, v);
}

// The first n of eight elements from element i on, a whole group with 16-byte stores.
template <class T>
__device__ inline void store8(void* base, int64_t i, int64_t n, const float (&v)[8]) {
  if (n >= 8) {
    char* p = static_cast<char*>(base) + i * T::bytes;
    if constexpr (T::bytes == 4) {
      __builtin_memcpy(p, v, 32);
    } else {
      uint4 q;
      q.x = T::pack2(v[0], v[1]);
      q.y = T::pack2(v[2], v[3]);
      q.z = T::pack2(v[4], v[5]);
      q.w = T::pack2(v[6], v[7]);
      __builtin_memcpy(p, &q, 16);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) put_one<T>(base, i + j, v[j]);
  }
}

// store8 with the non-temporal hint on whole groups (one element aligned, as store8).
template <class T>
__device__ inline void store8_stream(void* base, int64_t i, int64_t n, const float (&v)[8]) {
  typedef uint32_t u4 __attribute__((ext_vector_type(4), aligned(2)));
  if (n < 8) return store8<T>(base, i, n, v);
  char* p = static_cast<char*>(base) + i * T::bytes;
  if constexpr (T::bytes == 4) {
    __builtin_nontemporal_store(u4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])},
                                reinterpret_cast<u4*>(p));
    __builtin_nontemporal_store(u4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])},
                                reinterpret_cast<u4*>(p) + 1);
  } else {
    __builtin_nontemporal_store(u4{T::pack2(v[0], v[1]), T::pack2(v[2], v[3]), T::pack2(v[4], v[5]), T::pack2(v[6], v[7])},
                                reinterpret_cast<u4*>(p));
  }
}

// ---------------------------------------------------------------- block scales and codes
// Magnitudes are compared as bit patterns: they order like the values, and an infinity or a NaN
// comes out on top instead of being skipped.
__device__ inline uint32_t mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ inline uint32_t mag8(const float (&v)[8]) {
  uint32_t a = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) a = max(a, mag(v[j]));
  return a;
}
__device__ inline uint32_t shfl_max(uint32_t x, int m) {
  return max(x, static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), m, 64)));
}
// Largest of 16 neighbouring lanes, in all of them: quad permutes (lanes ^ 1, ^ 2), then the
// mirrored half row and row, whose other half or row holds one value already.
__device__ inline uint32_t max16(uint32_t x) {
  x = max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0xB1, 0xF, 0xF, false)));
  x = max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x4E, 0xF, 0xF, false)));
  x = max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x141, 0xF, 0xF, false)));
  return max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x140, 0xF, 0xF, false)));
}

// x / 448 and 1 / x, correctly rounded, in three operations each instead of the dozen of a
// division: an estimate within one unit, its exact remainder by one fma, and a correction. Both are
// tested on the GPU for every significand (the exponent does not matter to the quotient above
// 2^-117, where the remainder is a normal or an exact subnormal number).
__device__ inline float div448(float x) {
  constexpr float c = 1.0f / 448.0f;
  const float q = x * c;
  return __builtin_fmaf(__builtin_fmaf(-448.0f, q, x), c, q);
}
__device__ inline float reciprocal(float x) {
  const float r = __builtin_amdgcn_rcpf(x);
  return __builtin_fmaf(__builtin_fmaf(-x, r, 1.0f), r, r);
}

// The scale of a block whose largest magnitude has the bit pattern `a`, and r = 1 / s. A NaN or
// infinity: s = NaN, r = 0.
__device__ inline void block_scale(uint32_t a, bool pow2, float& s, float& r) {
  s = div448(__uint_as_float(a));
  if (pow2) s = __uint_as_float((__float_as_uint(s) + 0x7FFFFFu) & 0x7F800000u);
  s = fmaxf(s, 1.17549435e-38f);     // 2^-126: 1 / s stays finite
  r = reciprocal(s);
  if (a == 0u) s = 0.0f, r = 0.0f;
  if (a >= 0x7F800000u) s = __uint_as_float(0x7FC00000u), r = 0.0f;
}

// Four E4M3 codes of v r. |v r| is at most 448 (1 + 2^-22), because s is at least the correctly
// rounded a / 448, so the hardware conversion (to nearest even, no saturation below 464) needs no
// clamp.
__device__ inline uint32_t e4m3_codes4(float a, float b, float c, float d, float r) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * r, b * r, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c * r, d * r, w, true);
  return static_cast<uint32_t>(w);
}
// Eight codes. r = 0 stands for a block of zeros (of either sign) or one that is not finite: zero
// bytes.
__device__ inline uint2 e4m3_codes8(const float (&v)[8], float r) {
  const uint2 q = {e4m3_codes4(v[0], v[1], v[2], v[3], r), e4m3_codes4(v[4], v[5], v[6], v[7], r)};
  return r != 0.0f ? q : uint2{0u, 0u};
}

// ---------------------------------------------------------------- products of one block of K
// Eight E4M3 codes as fp16 values (exact: E4M3 is a subset of fp16).
__device__ inline auto f8_to_h8(uint32_t lo, uint32_t hi) {
  typedef _Float16 h2 __attribute__((ext_vector_type(2)));
  typedef _Float16 h8 __attribute__((ext_vector_type(8)));
  const h2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
  const h2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
  const h2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
  const h2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
  return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// 16 x 16 products over 128 K. A lane holds 32 of a row's bytes; which ones does not matter as
// long as both operands agree. EXACT: four fp16 instructions on the codes' values, eight bytes a
// lane each; else one FP8 instruction.
template <bool EXACT, class V>
__device__ inline auto multiply_block(const V& p, const V& q) {
  typedef float f4 __attribute__((ext_vector_type(4)));
  f4 u = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (EXACT) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      u = __builtin_amdgcn_mfma_f32_16x16x32_f16(f8_to_h8(p[2 * i], p[2 * i + 1]),
                                                 f8_to_h8(q[2 * i], q[2 * i + 1]), u, 0, 0, 0);
  } else {
    u = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(p, q, u, 0, 0, 0, 0, 0, 0);
  }
  return u;
}

}  // namespace hq
