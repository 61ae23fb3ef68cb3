// hq_train_device.hpp — element access shared by the kernels of include/hq_train.h: groups of
// eight consecutive elements, whole and aligned ones with wide accesses. Stores keep NaN (the
// shared bf16 store of hq_device.hpp takes finite values only).
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

// Elements [i, i + 8) of base, those past the first n as 0. `wide`: the eight are aligned to 16
// bytes, so a whole group is one or two wide loads.
template <class T>
__device__ inline void load8(const void* base, int64_t i, int64_t n, bool wide, float (&v)[8]) {
  if (wide && n >= 8) {
    const char* p = static_cast<const char*>(base) + i * T::bytes;
    if constexpr (T::bytes == 4) {
      const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      unpack8(*reinterpret_cast<const uint4*>(p), T::is_bf16, v);
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

template <class T>
__device__ inline void store8(void* base, int64_t i, int64_t n, bool wide, const float (&v)[8]) {
  if (wide && n >= 8) {
    char* p = static_cast<char*>(base) + i * T::bytes;
    if constexpr (T::bytes == 4) {
      reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint4 q;
      q.x = T::pack2(v[0], v[1]);
      q.y = T::pack2(v[2], v[3]);
      q.z = T::pack2(v[4], v[5]);
      q.w = T::pack2(v[6], v[7]);
      *reinterpret_cast<uint4*>(p) = q;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) put_one<T>(base, i + j, v[j]);
  }
}

// The same where the alignment is found at run time.
template <class T>
__device__ inline bool aligned8(const void* base, int64_t i) {
  return ((reinterpret_cast<uintptr_t>(base) + static_cast<uintptr_t>(i) * T::bytes) & 15u) == 0;
}
template <class T>
__device__ inline void load_run(const void* base, int64_t i, int64_t n, float (&v)[8]) {
  load8<T>(base, i, n, aligned8<T>(base, i), v);
}
template <class T>
__device__ inline void put_run(void* base, int64_t i, int64_t n, const float (&v)[8]) {
  store8<T>(base, i, n, aligned8<T>(base, i), v);
}

}  // namespace hq
