// hq_kv.hip — keys and values into a paged cache of microscaled 4-bit codes, and back.
//
// A head's vector of D elements is rotated by H_D (if the cache is), split into blocks of 32, and
// each block quantized as hq_mx.hip does: D / 8 lanes hold eight elements each, so strides 1, 2, 4
// are in registers, the others across lanes, and a block's largest magnitude is that of a quad.
//
// What bounds it: the vector pipe, busy for 80 to 90 % of the time (16384 tokens of 8 heads of 128, bf16: 85 MB
// in 25.7 us to the cache and 23.7 back, where a copy of as many bytes takes 18): the index of a vector and its
// addresses, 64-bit numbers, serve eight elements only. For a decode batch, the launch (48 tokens: 3 us).
#include "hq_device.hpp"
#include "hq_kv_index.hpp"
#include "hq_launch.hpp"
#include "hq_mx_device.hpp"
#include "hq_mx_internal.hpp"

namespace hq {

struct KvArgs {
  const void *k, *v;              // append: sources
  int64_t k_token, k_head, v_token, v_head;
  void *k_out, *v_out;            // read: destinations
  const int64_t* slots;
  int64_t tokens;
  int64_t pages;
  int shift, heads;
  uint8_t *k_codes, *v_codes, *k_scales, *v_scales;
};

// Vector `vec` of the call: keys and values of a token's heads lie side by side.
struct KvPlace {
  int64_t token;
  int head, value;
  __device__ KvPlace(int64_t vec, int heads) {
    const int64_t group = vec / heads;
    head = static_cast<int>(vec - group * heads);
    token = group >> 1;
    value = static_cast<int>(group & 1);
  }
};

template <class T, int D, bool ROT>
__global__ __launch_bounds__(256) void kv_append_kernel(KvArgs g) {
  constexpr int LPV = D / 8;
  const int t = threadIdx.x, l = t % LPV;
  const int64_t vec = (static_cast<int64_t>(blockIdx.x) * 256 + t) / LPV;
  const bool in = vec < 2 * g.tokens * g.heads;
  const KvPlace at(in ? vec : 0, g.heads);
  const int64_t row = in ? kv_row_of_slot(g.slots[at.token], g.pages, g.shift, g.heads, at.head) : -1;
  float v[8];
  const int64_t src = at.value ? at.token * g.v_token + at.head * g.v_head : at.token * g.k_token + at.head * g.k_head;
  load8<T>(at.value ? g.v : g.k, src + 8 * l, row >= 0 ? 8 : 0, v);
  if constexpr (ROT) rotate_lanes<D>(v, t & 63);
  const int byte = mx_scale_byte(quad_max(mag8(v)));
  const uint32_t w = mx_codes8<false>(v, byte, 0, 0);
  if (row < 0) return;
  uint8_t* const codes = at.value ? g.v_codes : g.k_codes;
  uint8_t* const scales = at.value ? g.v_scales : g.k_scales;
  *reinterpret_cast<uint32_t*>(codes + row * (D / 2) + 4 * l) = w;
  if ((l & 3) == 0) scales[row * (D / 32) + (l >> 2)] = static_cast<uint8_t>(byte);
}

template <class T, int D, bool ROT>
__global__ __launch_bounds__(256) void kv_read_kernel(KvArgs g) {
  constexpr int LPV = D / 8;
  const int t = threadIdx.x, l = t % LPV;
  const int64_t vec = (static_cast<int64_t>(blockIdx.x) * 256 + t) / LPV;
  const bool in = vec < 2 * g.tokens * g.heads;
  const KvPlace at(in ? vec : 0, g.heads);
  void* const out = at.value ? g.v_out : g.k_out;
  const bool wanted = in && out != nullptr;
  const int64_t row = wanted ? kv_row_of_slot(g.slots[at.token], g.pages, g.shift, g.heads, at.head) : -1;
  uint32_t w = 0;
  int byte = 0;
  if (row >= 0) {
    w = *reinterpret_cast<const uint32_t*>((at.value ? g.v_codes : g.k_codes) + row * (D / 2) + 4 * l);
    byte = (at.value ? g.v_scales : g.k_scales)[row * (D / 32) + (l >> 2)];
  }
  float v[8];
  mx_values8(w, v);
  // divided by D first (exact: codes times at least 2^-135), so that the sums stay below the largest value
  const float s = byte == 255 ? __uint_as_float(0x7FC00000u) : byte ? mx_scale(byte) : 5.87747175e-39f;
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= ROT ? s * (1.0f / D) : s;
  if constexpr (ROT) rotate_lanes<D>(v, t & 63);
  if (wanted) store8<T>(out, (at.token * g.heads + at.head) * D + 8 * l, 8, v);
}

static KvArgs cache_args(const hq_kv_cache& c) {
  KvArgs a = {};
  a.pages = c.pages;
  a.shift = __builtin_ctz(static_cast<unsigned>(c.page));
  a.heads = c.heads;
  a.k_codes = c.k_codes;
  a.v_codes = c.v_codes;
  a.k_scales = c.k_scales;
  a.v_scales = c.v_scales;
  return a;
}

static dim3 kv_grid(const hq_kv_cache& c, int64_t tokens) {
  const int64_t threads = 2 * tokens * c.heads * (c.head_dim / 8);
  return dim3(static_cast<unsigned>((threads + 255) / 256));
}

template <class T>
static hipError_t launch_append(const hq_kv_cache& c, const KvArgs& a, hipStream_t st, int tok) {
  const dim3 grid = kv_grid(c, a.tokens), block(256);
  switch (c.head_dim) {
#define HQ_D(D)                                                                              \
  case D:                                                                                    \
    return c.rot > 1 ? launch_k(kv_append_kernel<T, D, true>, grid, block, st, tok, a)       \
                     : launch_k(kv_append_kernel<T, D, false>, grid, block, st, tok, a);
    HQ_D(64) HQ_D(128) HQ_D(256)
#undef HQ_D
  }
  return hipErrorInvalidValue;
}

template <class T>
static hipError_t launch_read(const hq_kv_cache& c, const KvArgs& a, hipStream_t st, int tok) {
  const dim3 grid = kv_grid(c, a.tokens), block(256);
  switch (c.head_dim) {
#define HQ_D(D)                                                                            \
  case D:                                                                                  \
    return c.rot > 1 ? launch_k(kv_read_kernel<T, D, true>, grid, block, st, tok, a)       \
                     : launch_k(kv_read_kernel<T, D, false>, grid, block, st, tok, a);
    HQ_D(64) HQ_D(128) HQ_D(256)
#undef HQ_D
  }
  return hipErrorInvalidValue;
}

static double kv_units(const hq_kv_cache& c, int64_t tokens, int dt) {
  return 2.0 * tokens * c.heads * c.head_dim * ((dt == DT_F32 ? 4 : 2) + 17.0 / 32.0);
}

hipError_t kv_append_pass(const KvAppendPass& p, hipStream_t st) {
  KvArgs a = cache_args(p.cache);
  a.k = p.k;
  a.v = p.v;
  a.k_token = p.k_token;
  a.k_head = p.k_head;
  a.v_token = p.v_token;
  a.v_head = p.v_head;
  a.slots = p.slots;
  a.tokens = p.tokens;
  const int tok = prof_open(K_ROT_QUANT, kv_units(p.cache, p.tokens, p.dt));
  switch (p.dt) {
    case DT_F32: return launch_append<F32>(p.cache, a, st, tok);
    case DT_F16: return launch_append<F16>(p.cache, a, st, tok);
    case DT_BF16: return launch_append<BF16>(p.cache, a, st, tok);
  }
  return hipErrorInvalidValue;
}

hipError_t kv_read_pass(const KvReadPass& p, hipStream_t st) {
  KvArgs a = cache_args(p.cache);
  a.k_out = p.k;
  a.v_out = p.v;
  a.slots = p.slots;
  a.tokens = p.n;
  const int tok = prof_open(K_ROT_STORE, kv_units(p.cache, p.n, p.dt));
  switch (p.dt) {
    case DT_F32: return launch_read<F32>(p.cache, a, st, tok);
    case DT_F16: return launch_read<F16>(p.cache, a, st, tok);
    case DT_BF16: return launch_read<BF16>(p.cache, a, st, tok);
  }
  return hipErrorInvalidValue;
}

}  // namespace hq
