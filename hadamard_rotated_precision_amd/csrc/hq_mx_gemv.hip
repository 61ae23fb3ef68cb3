// hq_mx_gemv.hip — microscaled 4-bit product for a few output rows (at most 32 tokens):
//   c[m][n] (+)= alpha sum_kb 2^(ea(m,kb) + eb(n,kb)) sum_{k in kb} a[m][k] b[n][k]
//
// What bounds it: the bytes of b, read once, and the launch, first loads and joining (one token at
// 11008 x 4096, fused: 24 MB in 8.7 us, 2.8 TB/s, launch included). A workgroup
// takes 16 RT rows of b and the whole contraction; its eight waves take every eighth step of 256 K
// each. A wave's fragments come straight from memory into the operand registers, kMvAhead steps ahead
// of their use; the tokens are the lanes' side of v_mfma_scale_f32_16x16x128_f8f6f4, padded to 16 or
// 32 with zeros. The eight partial sums meet in LDS and are added in the order of the waves.
//
// The tokens come as codes, or (fused, for few enough elements) as the caller's own values: then
// every workgroup rotates and quantizes them into LDS while its first rows of b are on their way.
#include "hq_device.hpp"
#include "hq_launch.hpp"
#include "hq_mx_device.hpp"
#include "hq_mx_internal.hpp"

namespace hq {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kMvWaves = 8;
constexpr int kMvAhead = 2;              // steps of K in flight per wave
constexpr int kMvCodes = 16384;          // LDS bytes of the tokens' codes (fused)
constexpr int kMvFar = 0x7FFFFFF0;

struct MxGemvArgs {
  MxOperand p, q;       // b, and a's codes (not fused)
  const void* x;        // a's values (fused): M x K, contiguous
  int M;
  int64_t N;
  int K;
  int x_dt, rot;        // fused: type and rotation
  float alpha;
  void* c;
  int accumulate;
};

// Fused: codes of the tokens in LDS, a thread per eight elements, four lanes per block, four tokens'
// loads in flight. kb16: a row's code bytes, kpad / 2, kpad being K up to the next multiple of 256.
template <class T, int ROT>
__device__ inline void quantize_tokens(const MxGemvArgs& g, int kpad, uint8_t* codes, uint8_t* scales) {
  constexpr int U = 4;
  auto put = [&](int m, int c, float (&v)[8]) {
    if constexpr (ROT > 1) rotate_lanes<ROT>(v, threadIdx.x);
    const int byte = mx_scale_byte(quad_max(mag8(v)));
    *reinterpret_cast<uint32_t*>(codes + m * (kpad >> 1) + (c >> 1)) = mx_codes8<false>(v, byte, 0, 0);
    if ((threadIdx.x & 3) == 0) scales[m * (kpad >> 5) + (c >> 5)] = byte;
  };
  for (int c = 8 * threadIdx.x; c < kpad; c += 8 * 64 * kMvWaves) {
    const int n = max(g.K - c, 0);
    int m = 0;
    for (; m + U <= g.M; m += U) {
      float v[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) load8<T>(g.x, static_cast<int64_t>(m + u) * g.K + c, n, v[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) put(m + u, c, v[u]);
    }
    for (; m < g.M; ++m) {
      float v[8];
      load8<T>(g.x, static_cast<int64_t>(m) * g.K + c, n, v);
      put(m, c, v);
    }
  }
}

template <int ROT>
__device__ inline void quantize_tokens_of(const MxGemvArgs& g, int kpad, uint8_t* codes, uint8_t* scales) {
  switch (g.x_dt) {
    case DT_F32: quantize_tokens<F32, ROT>(g, kpad, codes, scales); break;
    case DT_F16: quantize_tokens<F16, ROT>(g, kpad, codes, scales); break;
    default: quantize_tokens<BF16, ROT>(g, kpad, codes, scales); break;
  }
}

template <class Out, int RT, int QT, bool FUSED>
__global__ __launch_bounds__(64 * kMvWaves) void mx_gemv_kernel(MxGemvArgs g) {
  static_assert(!FUSED || QT == 1, "");
  __shared__ float part[kMvWaves][RT][QT][64][4];
  __shared__ __attribute__((aligned(16))) uint8_t xc[FUSED ? kMvCodes : 16];
  __shared__ __attribute__((aligned(16))) uint8_t xs[FUSED ? kMvCodes / 16 : 16];
  const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * RT);
  const int rows = static_cast<int>(min<int64_t>(16 * RT, g.N - n0));
  const int ldp = static_cast<int>(g.p.ld), lsp = static_cast<int>(g.p.lds);
  const int KB = (g.K + 31) >> 5, KT = (KB + 7) >> 3, kpad = KT * 256;
  const __amdgpu_buffer_rsrc_t rsp = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(g.p.codes + n0 * g.p.ld), 0, rows * ldp, kBufferFlags);
  const __amdgpu_buffer_rsrc_t ssp = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(g.p.scales + n0 * g.p.lds), 0, rows * lsp, kBufferFlags);
  const int rows_q = min(16 * QT, g.M);
  const int ldq = static_cast<int>(g.q.ld), lsq = static_cast<int>(g.q.lds);
  const __amdgpu_buffer_rsrc_t rsq = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(g.q.codes), 0, FUSED ? 0 : rows_q * ldq, kBufferFlags);
  const __amdgpu_buffer_rsrc_t ssq = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(g.q.scales), 0, FUSED ? 0 : rows_q * lsq, kBufferFlags);

  // Blocks lg and lg + 4 of a step's eight (for both operands), so that four lanes read 64
  // consecutive bytes; and the eight scale bytes of the row, whose byte lg of each dword is the
  // lane's. A scale row is padded to 16 bytes.
  struct Step {
    v4i x[2];
    v2i s;
  };
  auto load = [&](const __amdgpu_buffer_rsrc_t& rs, const __amdgpu_buffer_rsrc_t& ss, int ld, int lds, int row, int kt) {
    Step f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int b = 8 * kt + 4 * h + lg;
      f.x[h] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rs, b < KB ? row * ld + 16 * b : kMvFar, 0, 0));
    }
    f.s = __builtin_bit_cast(v2i, __builtin_amdgcn_raw_buffer_load_b64(ss, kt < KT ? row * lds + 8 * kt : kMvFar, 0, 0));
    return f;
  };
  Step wf[kMvAhead][RT], xf[kMvAhead][QT];
  auto fetch = [&](int slot, int kt) {
#pragma unroll
    for (int i = 0; i < RT; ++i) wf[slot][i] = load(rsp, ssp, ldp, lsp, 16 * i + lr, kt);
    if constexpr (!FUSED) {
#pragma unroll
      for (int j = 0; j < QT; ++j) xf[slot][j] = load(rsq, ssq, ldq, lsq, 16 * j + lr, kt);
    }
  };
#pragma unroll
  for (int s = 0; s < kMvAhead; ++s) fetch(s, w + kMvWaves * s);

  if constexpr (FUSED) {
    if (g.rot == 1) quantize_tokens_of<1>(g, kpad, xc, xs);
    else quantize_tokens_of<32>(g, kpad, xc, xs);
    __syncthreads();
  }

  v4f acc[RT][QT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < QT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  auto wide = [](v4i a) { return v8i{a[0], a[1], a[2], a[3], 0, 0, 0, 0}; };
  auto block = [&](int slot, int kt) {
    if constexpr (FUSED) {
      Step f = {{v4i{0, 0, 0, 0}, v4i{0, 0, 0, 0}}, v2i{0, 0}};
      if (lr < g.M) {
        const uint8_t* row = xc + lr * (kpad >> 1) + kt * 128 + 16 * lg;
        f.x[0] = *reinterpret_cast<const v4i*>(row);
        f.x[1] = *reinterpret_cast<const v4i*>(row + 64);
        f.s = *reinterpret_cast<const v2i*>(xs + lr * (kpad >> 5) + 8 * kt);
      }
      xf[slot][0] = f;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < QT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              wide(wf[slot][i].x[h]), wide(xf[slot][j].x[h]), acc[i][j], 4, 4, 0, wf[slot][i].s[h] >> (8 * lg), 0,
              xf[slot][j].s[h] >> (8 * lg));
  };
  for (int kt = w; kt < KT; kt += kMvWaves * kMvAhead) {
#pragma unroll
    for (int s = 0; s < kMvAhead; ++s) {
      const int k = kt + kMvWaves * s;
      if (k < KT) {
        block(s, k);
        fetch(s, k + kMvWaves * kMvAhead);   // past the end: zeros, never used
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < QT; ++j) *reinterpret_cast<v4f*>(part[w][i][j][lane]) = acc[i][j];
  __syncthreads();
  for (int e = t; e < rows_q * 16 * RT; e += 64 * kMvWaves) {
    const int m = e / (16 * RT), n = e % (16 * RT);
    if (n0 + n >= g.N) continue;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kMvWaves; ++i) sum += part[i][n >> 4][m >> 4][((n & 15) >> 2) * 16 + (m & 15)][n & 3];
    sum *= g.alpha;
    const int64_t at = static_cast<int64_t>(m) * g.N + n0 + n;
    if (g.accumulate) sum += Out::load(g.c, at);
    put_one<Out>(g.c, at, sum);
  }
}

// Where this kernel is faster than the tiles of hq_mx_gemm.hip: up to 16 tokens while every compute
// unit gets one workgroup of 32 rows at most (N <= 32 x 256; 16 x 5120 x 5120 7.4 against 10.3 us,
// 16 x 11008 x 4096 13.8 against 10.8, 1 x 32000 x 4096 20.6 against 17.4), 17 to 32 while that holds
// with 16 rows and the tokens are few and short enough, for each workgroup reads all of their codes
// (32 x 4096 x 4096 7.9 against 9.2 us, 24 x 4096 x 11008 13.1 against 12.7).
bool mx_gemv_ok(int64_t M, int64_t N, int64_t K) {
  return M >= 1 && K >= 1 &&
         ((M <= 16 && N <= 32 * 256) || (M <= 32 && N <= 16 * 256 && M * K <= int64_t{3} << 16));
}

// Fused when the tokens' codes fit their LDS.
bool mx_gemv_fused_ok(int64_t M, int64_t K) {
  return M >= 1 && M <= 16 && K >= 1 && M * ((K + 255) / 256 * 128) <= kMvCodes;
}

template <class Out, int RT, int QT>
static hipError_t launch_gemv(const MxGemvArgs& a, bool fused, hipStream_t st, int tok) {
  const dim3 grid(static_cast<unsigned>((a.N + 16 * RT - 1) / (16 * RT)));
  const dim3 block(64 * kMvWaves);
  if constexpr (QT == 1) {
    if (fused) return launch_k(mx_gemv_kernel<Out, RT, QT, true>, grid, block, st, tok, a);
  }
  return launch_k(mx_gemv_kernel<Out, RT, QT, false>, grid, block, st, tok, a);
}

template <class Out>
static hipError_t launch_rows(const MxGemvArgs& a, bool fused, hipStream_t st, int tok) {
  // 16 rows of b per workgroup while every compute unit gets one at most, else 32: one token at
  // 4096 x 11008 9.0 and 11.3 us, 16 at 5120 x 5120 9.2 and 7.4
  if (a.M > 16) return launch_gemv<Out, 1, 2>(a, fused, st, tok);
  return a.N > 16 * 256 ? launch_gemv<Out, 2, 1>(a, fused, st, tok) : launch_gemv<Out, 1, 1>(a, fused, st, tok);
}

hipError_t mx_gemv_pass(const MxGemmPass& p, const void* x, int x_dt, int rot, hipStream_t st) {
  if (x ? !mx_gemv_fused_ok(p.M, p.K) : !mx_gemv_ok(p.M, p.N, p.K)) return hipErrorInvalidValue;
  const MxGemvArgs a{p.b, p.a, x, static_cast<int>(p.M), p.N, static_cast<int>(p.K), x_dt, rot, p.alpha, p.c, p.accumulate};
  const int tok = prof_open(K_GEMM, 2.0 * p.M * p.N * p.K);
  switch (p.out_dt) {
    case DT_F32: return launch_rows<F32>(a, x != nullptr, st, tok);
    case DT_F16: return launch_rows<F16>(a, x != nullptr, st, tok);
    case DT_BF16: return launch_rows<BF16>(a, x != nullptr, st, tok);
  }
  return hipErrorInvalidValue;
}

}  // namespace hq
