// hq_adamw.hip — one AdamW step over many tensors, states in fp32 or in 8-bit codes.
//
// The formulas stand in include/hq_train.h. What bounds it: bytes; per element the parameter and
// the states are read and written once and the gradient is read once. 88 M elements with fp32
// parameters, bf16 gradients and a bf16 copy: 457 us with 32-bit states (5.4 TB/s), 265 with 8-bit
// ones (5.4 TB/s; 304 before one square root and a three-operation reciprocal took the place of two
// and a division: the vector work of 8-bit states is close behind the bytes). Stores past the
// caches changed nothing.
//
// The tensors' pointers travel in the kernel's arguments (a table of up to kTable tensors, within
// the 4 KB an argument block holds), so a call needs no copy to the device and can be captured; a
// longer list takes several launches. Each workgroup takes a run of kChunk elements of one tensor
// and finds its tensor by a search over the table's first-workgroup numbers. A thread holds eight
// consecutive elements, so the 128 elements that share an 8-bit state's scale are sixteen
// neighbouring lanes.
#include "hq_device.hpp"
#include "hq_launch.hpp"
#include "hq_train_device.hpp"
#include "hq_train_internal.hpp"

namespace hq {

constexpr int kTable = 40;
constexpr int kThreads = 256;
constexpr int kChunk = kThreads * 8;

struct AdamwEntry {
  void* p;
  const void* grad;
  void* m;
  void* v;
  float* ms;
  float* vs;
  void* copy;
  int64_t n;
  float wd;
  uint32_t key_add;      // 0x9E3779B9 (index of the tensor + 1)
};

struct AdamwArgs {
  AdamwEntry t[kTable];
  uint32_t first[kTable + 1];   // first workgroup of each tensor, and the grid's size
  int count;
  float beta1, rest1, beta2, rest2, eps;
  hq_adamw_scalars host;
  const hq_adamw_scalars* device;
};
static_assert(sizeof(AdamwArgs) <= 4096, "the table must fit a kernel's argument block");

__device__ inline uint32_t mix32(uint32_t h) {
  h ^= h >> 16;
  h *= 2654435761u;
  h ^= h >> 15;
  h *= 2891336453u;
  return h ^ (h >> 16);
}

// Eight code bytes from element i on (bytes past n read as 0 and are not written).
__device__ inline uint2 get_codes(const void* base, int64_t i, int n) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + i;
  if (n >= 8) {
    uint2 q;
    __builtin_memcpy(&q, p, 8);
    return q;
  }
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) w[j >> 2] |= static_cast<uint32_t>(p[j]) << (8 * (j & 3));
  return {w[0], w[1]};
}

__device__ inline void put_codes(void* base, int64_t i, int n, uint2 q) {
  uint8_t* p = static_cast<uint8_t*>(base) + i;
  if (n >= 8) {
    __builtin_memcpy(p, &q, 8);
    return;
  }
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) p[j] = static_cast<uint8_t>(w[j >> 2] >> (8 * (j & 3)));
}

__device__ inline void e4m3_values(uint2 q, float (&v)[8]) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8(q.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(q.x, true);
  const f2 c = __builtin_amdgcn_cvt_pk_f32_fp8(q.y, false), d = __builtin_amdgcn_cvt_pk_f32_fp8(q.y, true);
  v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1];
  v[4] = c[0]; v[5] = c[1]; v[6] = d[0]; v[7] = d[1];
}

// The E4M3 code of x in [0, 448] below or at it: from the bits for the normal values (x >= 2^-6),
// in steps of 2^-9 below.
// m: up when the 20 dropped bits plus 16 random ones (above 4 zeros) carry.
__device__ inline uint32_t round_m(float x, uint32_t u16) {
  if (x >= 0.015625f) return ((__float_as_uint(x) + (u16 << 4)) >> 20) - 960u;
  return static_cast<uint32_t>(x * 512.0f + static_cast<float>(u16) * 0x1p-16f);
}

// sqrt(v): up with the probability (x^2 - low^2) / (high^2 - low^2), so that the mean of the
// square is v.
__device__ inline uint32_t round_v(float x, uint32_t u16) {
#pragma clang fp contract(off)
  const uint32_t b = __float_as_uint(x);
  const bool normal = x >= 0.015625f;
  uint32_t code = normal ? (b >> 20) - 960u : static_cast<uint32_t>(x * 512.0f);
  const float low = normal ? __uint_as_float(b & 0xFFF00000u) : static_cast<float>(code) * 0x1p-9f;
  const float step = normal ? __uint_as_float(((b >> 23) - 3u) << 23) : 0x1p-9f;
  const float f = static_cast<float>(u16) * 0x1p-16f;
  if (f * (step * (2.0f * low + step)) < (x - low) * (x + low)) ++code;
  return code;
}

// The products and sums are rounded one by one (no fused multiply-add): the codes of 8-bit states
// then hang on the stated fp32 formulas alone, not on what a compiler fuses.
template <class P, class G, class C, bool EIGHT>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamwArgs g) {
#pragma clang fp contract(off)
  int k = 0;
  for (int lo = 0, hi = g.count; hi - lo > 1;) {
    const int mid = (lo + hi) >> 1;
    if (g.first[mid] <= blockIdx.x) lo = mid; else hi = mid;
    k = lo;
  }
  const AdamwEntry& t = g.t[k];
  hq_adamw_scalars s = g.host;
  if (g.device) s = *g.device;
  const int64_t i = static_cast<int64_t>(blockIdx.x - g.first[k]) * kChunk + threadIdx.x * 8;
  const int n = static_cast<int>(min<int64_t>(max<int64_t>(t.n - i, 0), 8));
  if (!EIGHT && n == 0) return;

  float p[8], gr[8], m[8], v[8];
  load8<P>(t.p, i, n, p);
  load8<G>(t.grad, i, n, gr);
  if constexpr (EIGHT) {
    const float ms = n > 0 ? t.ms[i >> 7] : 0.0f, vs = n > 0 ? t.vs[i >> 7] : 0.0f;
    e4m3_values(get_codes(t.m, i, n), m);
    e4m3_values(get_codes(t.v, i, n), v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] *= ms;
      v[j] *= vs;
      v[j] *= v[j];
    }
  } else {
    load8<F32>(t.m, i, n, m);
    load8<F32>(t.v, i, n, v);
  }
  const float keep = 1.0f - s.lr * t.wd;
  float y[8];     // sqrt(v): the update's, and what 8-bit states store
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float gj = gr[j] * s.grad_scale;
    m[j] = g.beta1 * m[j] + g.rest1 * gj;
    v[j] = g.beta2 * v[j] + (g.rest2 * gj) * gj;
    y[j] = sqrtf(v[j]);
    const float den = y[j] * s.inv_sqrt_bias2 + g.eps;
    // 1 / den to the nearest fp32 (den is at least eps, a normal number); an infinite den keeps 0
    const float r = den < __builtin_inff() ? reciprocal(den) : __builtin_amdgcn_rcpf(den);
    p[j] = p[j] * keep - s.step_size * (m[j] * r);
  }
  store8<P>(t.p, i, n, p);
  if (t.copy) store8<C>(t.copy, i, n, p);
  if constexpr (!EIGHT) {
    store8<F32>(t.m, i, n, m);
    store8<F32>(t.v, i, n, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j >= n) m[j] = y[j] = 0.0f;   // elements behind the tensor take no part in the maxima
    float ms, mr, vs, vr;
    block_scale(max16(mag8(m)), false, ms, mr);
    block_scale(max16(mag8(y)), false, vs, vr);
    if (n == 0) return;
    const uint32_t key = s.key + t.key_add + 0x632BE5ABu * static_cast<uint32_t>(i >> 32);
    uint32_t qm[2] = {0u, 0u}, qv[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t u = mix32(static_cast<uint32_t>(i + j) ^ key);
      uint32_t cm = round_m(fminf(fabsf(m[j]) * mr, 448.0f), u & 0xFFFFu);
      if (m[j] < 0.0f) cm |= 0x80u;
      uint32_t cv = round_v(fminf(y[j] * vr, 448.0f), u >> 16);
      if (v[j] > 0.0f) cv = max(cv, 1u);
      qm[j >> 2] |= cm << (8 * (j & 3));
      qv[j >> 2] |= cv << (8 * (j & 3));
    }
    put_codes(t.m, i, n, uint2{qm[0], qm[1]});
    put_codes(t.v, i, n, uint2{qv[0], qv[1]});
    if ((threadIdx.x & 15) == 0) {
      t.ms[i >> 7] = ms;
      t.vs[i >> 7] = vs;
    }
  }
}

template <class P, class G, class C>
static hipError_t launch_adamw(bool eight, unsigned grid, hipStream_t st, int tok, const AdamwArgs& a) {
  return eight ? launch_k(adamw_kernel<P, G, C, true>, dim3(grid), dim3(kThreads), st, tok, a)
               : launch_k(adamw_kernel<P, G, C, false>, dim3(grid), dim3(kThreads), st, tok, a);
}

template <class P, class G>
static hipError_t launch_copy(int cdt, bool eight, unsigned grid, hipStream_t st, int tok, const AdamwArgs& a) {
  switch (cdt) {
    case DT_F32: return launch_adamw<P, G, F32>(eight, grid, st, tok, a);
    case DT_F16: return launch_adamw<P, G, F16>(eight, grid, st, tok, a);
    case DT_BF16: return launch_adamw<P, G, BF16>(eight, grid, st, tok, a);
  }
  return hipErrorInvalidValue;
}

template <class P>
static hipError_t launch_grad(int gdt, int cdt, bool eight, unsigned grid, hipStream_t st, int tok, const AdamwArgs& a) {
  switch (gdt) {
    case DT_F32: return launch_copy<P, F32>(cdt, eight, grid, st, tok, a);
    case DT_F16: return launch_copy<P, F16>(cdt, eight, grid, st, tok, a);
    case DT_BF16: return launch_copy<P, BF16>(cdt, eight, grid, st, tok, a);
  }
  return hipErrorInvalidValue;
}

hipError_t adamw_pass(const hq_adamw_tensor* t, int count, const hq_adamw_config& cfg,
                      const hq_adamw_scalars& host, const hq_adamw_scalars* device,
                      hipStream_t st) {
  const bool eight = cfg.state_bits == 8;
  const double state = eight ? 4.0 : 16.0;
  const int pb = cfg.param_dtype == HQ_F32 ? 4 : 2, gb = cfg.grad_dtype == HQ_F32 ? 4 : 2,
            cb = cfg.copy_dtype == HQ_F32 ? 4 : 2;
  AdamwArgs a;
  a.beta1 = static_cast<float>(cfg.beta1);
  a.rest1 = static_cast<float>(1.0 - cfg.beta1);
  a.beta2 = static_cast<float>(cfg.beta2);
  a.rest2 = static_cast<float>(1.0 - cfg.beta2);
  a.eps = static_cast<float>(cfg.eps);
  a.host = host;
  a.device = device;
  int i = 0;
  constexpr int64_t kMaxGrid = ((int64_t{1} << 32) - 1) / kThreads;   // a grid has less than 2^32 threads
  while (i < count) {
    // a table of tensors whose workgroups fit one grid
    a.count = 0;
    int64_t grid = 0;
    double units = 0.0;
    for (; i < count && a.count < kTable; ++i) {
      const hq_adamw_tensor& x = t[i];
      if (x.n == 0) continue;
      const int64_t chunks = (x.n + kChunk - 1) / kChunk;
      if (grid + chunks > kMaxGrid) break;
      AdamwEntry& e = a.t[a.count];
      e = AdamwEntry{x.p, x.grad, x.m, x.v, x.m_scales, x.v_scales, x.copy, x.n, x.weight_decay,
                     0x9E3779B9u * static_cast<uint32_t>(i + 1)};
      a.first[a.count++] = static_cast<uint32_t>(grid);
      grid += chunks;
      units += static_cast<double>(x.n) * (2 * pb + gb + state + (x.copy ? cb : 0));
    }
    if (a.count == 0) return i < count ? hipErrorInvalidValue : hipSuccess;
    a.first[a.count] = static_cast<uint32_t>(grid);
    const int tok = prof_open(K_MISC, units);
    hipError_t e = hipErrorInvalidValue;
    switch (cfg.param_dtype) {
      case HQ_F32: e = launch_grad<F32>(cfg.grad_dtype, cfg.copy_dtype, eight, static_cast<unsigned>(grid), st, tok, a); break;
      case HQ_F16: e = launch_grad<F16>(cfg.grad_dtype, cfg.copy_dtype, eight, static_cast<unsigned>(grid), st, tok, a); break;
      case HQ_BF16: e = launch_grad<BF16>(cfg.grad_dtype, cfg.copy_dtype, eight, static_cast<unsigned>(grid), st, tok, a); break;
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace hq
