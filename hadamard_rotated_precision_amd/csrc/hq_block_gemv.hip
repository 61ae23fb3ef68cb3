// hq_block_gemv.hip — block-scaled FP8 product for a few output rows (at most 32 tokens):
//   c[m][n] (+)= sum_kb sa(m,kb) sb(n,kb) sum_{k in kb} a[m][k] b[n][k]
//
// What bounds it: the bytes of b, read once, and about 3 us of launch, first loads and joining. One
// token takes 11.5 us at 4096 x 11008 with the weights in the 256 MB cache before the memory (45 MB:
// 3.9 TB/s, 5.3 TB/s past those 3 us) and 12.4 us from memory, 6.2 and 7.4 at 4096 x 4096, 13.4 and
// 16 at 5120 x 13824 (5.3 and 4.4 TB/s). Four blocks ahead instead of two, four or sixteen waves
// instead of eight: equal or slower. A workgroup takes 16 RT rows of b and the whole
// contraction; its eight waves take every eighth block of 128 K each, so that together they read
// 1 KB of every row at a time. A wave's fragments come straight from memory into the operand
// registers (16 rows x 64 contiguous bytes per load), two blocks ahead of their use; the tokens
// are the lanes' side of v_mfma_f32_16x16x128_f8f6f4, padded to 16 or 32 with zeros. The eight partial
// sums meet in LDS and are added in the order of the waves. 16-bit outputs take the FP8 instruction
// here too (its error: hq_block_gemm.hip); the exact sums of fp32 outputs cost up to 2 % with one
// token and 1 to 5 % with 13 to 16 (16 tokens at 5120 x 13824: 23.4 against 22.3 us).
//
// The tokens come as codes, or (fused, for few enough elements) as the caller's own values:
// then every workgroup quantizes them into LDS while its first rows of b are on their way.
// Quantizing again in each workgroup costs less than a launch of its own as long as a thread has
// few elements to do.
#include "hq_device.hpp"
#include "hq_launch.hpp"
#include "hq_train_device.hpp"
#include "hq_train_internal.hpp"

namespace hq {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kGvWaves = 8;
constexpr int kGvAhead = 2;              // blocks of K in flight per wave
constexpr int kGvCodes = 16384;          // LDS bytes of the tokens' codes (fused)
constexpr int kGvFar = 0x7FFFFFF0;

struct GemvArgs {
  BlockOperand p, q;    // b, and a's codes (not fused)
  const void* x;        // a's values (fused): M x K, contiguous
  int M;
  int64_t N;
  int K;
  int x_dt, pow2;       // fused: type and scale kind
  void* c;
  int accumulate;
};

// Fused: codes of the tokens in LDS, a thread per eight elements, sixteen lanes per block, four
// tokens' loads in flight.
template <class T>
__device__ inline void quantize_tokens(const GemvArgs& g, int kpad, uint8_t* codes, float* scales) {
  constexpr int U = 4;
  auto put = [&](int m, int c, const float (&v)[8]) {
    float s, r;
    block_scale(max16(mag8(v)), g.pow2, s, r);
    *reinterpret_cast<uint2*>(codes + m * kpad + c) = e4m3_codes8(v, r);
    if ((threadIdx.x & 15) == 0) scales[m * (kpad >> 7) + (c >> 7)] = s;
  };
  for (int c = 8 * threadIdx.x; c < kpad; c += 8 * 64 * kGvWaves) {
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

// EXACT: the fp16 instruction on the codes' values (fp32 outputs); else the FP8 one.
template <class Out, int RT, int QT, bool P_ROWS, bool EXACT, bool FUSED>
__global__ __launch_bounds__(64 * kGvWaves) void block_gemv_kernel(GemvArgs g) {
  static_assert(!FUSED || QT == 1, "");
  __shared__ float part[kGvWaves][RT][QT][64][4];
  __shared__ __attribute__((aligned(16))) uint8_t xc[FUSED ? kGvCodes : 16];
  __shared__ float xs[FUSED ? kGvCodes / 128 : 4];
  const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * RT);
  const int rows = static_cast<int>(min<int64_t>(16 * RT, g.N - n0));
  const int ldp = static_cast<int>(g.p.ld), KB = (g.K + 127) / 128, K16 = (g.K + 15) & ~15, kpad = KB * 128;
  const __amdgpu_buffer_rsrc_t rsp = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(g.p.codes + n0 * g.p.ld), 0, rows * ldp, kBufferFlags);
  const int rows_q = min(16 * QT, g.M);
  const int ldq = static_cast<int>(g.q.ld);
  const __amdgpu_buffer_rsrc_t rsq = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(g.q.codes), 0, FUSED ? 0 : rows_q * ldq, kBufferFlags);

  // chunks lg and lg + 4 of a row's 128 bytes (for both operands: products pair equal K)
  auto chunks = [&](const __amdgpu_buffer_rsrc_t& rs, int row_off, int kb) {
    const int k = kb * 128 + 16 * lg;
    const v4i a = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rs, k < K16 ? row_off + k : kGvFar, 0, 0));
    const v4i b = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rs, k + 64 < K16 ? row_off + k + 64 : kGvFar, 0, 0));
    return v8i{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  };
  v8i wf[kGvAhead][RT], xf[kGvAhead][QT];
  float sx[kGvAhead][QT];
  v4f sw[kGvAhead][RT];
  auto fetch = [&](int slot, int kb) {
#pragma unroll
    for (int i = 0; i < RT; ++i) wf[slot][i] = chunks(rsp, (16 * i + lr) * ldp, kb);
    const int kc = min(kb, KB - 1);
    if constexpr (P_ROWS) {
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int64_t n = n0 + 16 * i + 4 * lg + r;
          sw[slot][i][r] = n < g.N ? g.p.scales[n + kc * g.p.sk] : 0.0f;
        }
    } else {
      sw[slot][0][0] = g.p.scales[(n0 >> 7) * g.p.sg + kc * g.p.sk];
    }
    if constexpr (!FUSED) {
#pragma unroll
      for (int j = 0; j < QT; ++j) {
        const int m = 16 * j + lr;
        xf[slot][j] = chunks(rsq, (16 * j + lr) * ldq, kb);
        sx[slot][j] = m < g.M ? g.q.scales[(g.q.tiles ? m >> 7 : m) * g.q.sg + kc * g.q.sk] : 0.0f;
      }
    }
  };
#pragma unroll
  for (int s = 0; s < kGvAhead; ++s) fetch(s, w + kGvWaves * s);

  if constexpr (FUSED) {
    switch (g.x_dt) {
      case DT_F32: quantize_tokens<F32>(g, kpad, xc, xs); break;
      case DT_F16: quantize_tokens<F16>(g, kpad, xc, xs); break;
      default: quantize_tokens<BF16>(g, kpad, xc, xs); break;
    }
    __syncthreads();
  }

  v4f acc[RT][QT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < QT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  auto block = [&](int slot, int kb) {
    if constexpr (FUSED) {
      v4i a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
      sx[slot][0] = 0.0f;
      if (lr < g.M) {
        const uint8_t* row = xc + lr * kpad + kb * 128 + 16 * lg;
        a = *reinterpret_cast<const v4i*>(row);
        b = *reinterpret_cast<const v4i*>(row + 64);
        sx[slot][0] = xs[lr * KB + kb];
      }
      xf[slot][0] = v8i{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < QT; ++j) {
        const v4f u = multiply_block<EXACT>(wf[slot][i], xf[slot][j]);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[i][j][r] = __builtin_fmaf(u[r], sx[slot][j] * (P_ROWS ? sw[slot][i][r] : sw[slot][0][0]), acc[i][j][r]);
      }
  };
  for (int kb = w; kb < KB; kb += kGvWaves * kGvAhead) {
#pragma unroll
    for (int s = 0; s < kGvAhead; ++s) {
      const int k = kb + kGvWaves * s;
      if (k < KB) {
        block(s, k);
        fetch(s, k + kGvWaves * kGvAhead);   // past the end: zeros, never used
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < QT; ++j) *reinterpret_cast<v4f*>(part[w][i][j][lane]) = acc[i][j];
  __syncthreads();
  for (int e = t; e < rows_q * 16 * RT; e += 64 * kGvWaves) {
    const int m = e / (16 * RT), n = e % (16 * RT);
    if (n0 + n >= g.N) continue;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kGvWaves; ++i) sum += part[i][n >> 4][m >> 4][((n & 15) >> 2) * 16 + (m & 15)][n & 3];
    const int64_t at = static_cast<int64_t>(m) * g.N + n0 + n;
    if (g.accumulate) sum += Out::load(g.c, at);
    put_one<Out>(g.c, at, sum);
  }
}

// Up to 16 tokens; 17 to 32 while every compute unit gets one workgroup at most (N <= 16 x 256) and
// the tokens are few and short enough, for each workgroup reads all of their codes: M K up to 3 2^16.
// Against 64 x 64 tiles with K split, us at 17 / 24 / 32 tokens, this form first (N x K):
//   4096 x 4096: 8.0 8.7 9.3 / 10.9 11.1 11.2       1024 x 4096: 7.2 7.9 8.5 / 11.5 12.0 12.4
//   4096 x 6400: 9.8 11.1 12.2 / 13.3 13.6 13.7     2048 x 6400: 9.4 10.6 11.8 / 11.5 11.5 11.7
//   4096 x 8192: 11.3 12.7 14.4 / 13.3 13.6 13.5    1024 x 8192: 11.2 12.6 14.6 / 12.0 12.9 13.0
//   1024 x 16384: 19.2 21.8 24.9 / 14.2 14.8 14.6   (M K at 32 tokens: 3.1 2^16 for K = 6400)
// and with two rounds of workgroups: 4112 x 4096: 12.2 13.4 14.7 / 11.9 12.0 12.1,
//   4112 x 11008: 25.2 28.7 32.2 / 16.7 17.0 17.4,  16384 x 1024: 8.5 8.9 9.3 / 7.5 7.5 7.5.
bool block_gemv_ok(int64_t M, int64_t N, int64_t K) {
  return M >= 1 && K >= 1 && (M <= 16 || (M <= 32 && N <= 16 * 256 && M * K <= int64_t{3} << 16));
}

// Fused when the tokens' codes fit their LDS. Every workgroup repeats the quantizing: past that a
// launch of its own is cheaper (eight tokens of 4096 for 11008 rows: 15.3 us on their own launch,
// 16.9 fused).
bool block_gemv_fused_ok(int64_t M, int64_t K) {
  return M >= 1 && M <= 16 && K >= 1 && M * ((K + 127) / 128 * 128) <= kGvCodes;
}

template <class Out, int RT, int QT, bool P_ROWS, bool EXACT>
static hipError_t launch_gemv(const GemvArgs& a, bool fused, hipStream_t st, int tok) {
  const dim3 grid(static_cast<unsigned>((a.N + 16 * RT - 1) / (16 * RT)));
  const dim3 block(64 * kGvWaves);
  if constexpr (QT == 1) {
    if (fused) return launch_k(block_gemv_kernel<Out, RT, QT, P_ROWS, EXACT, true>, grid, block, st, tok, a);
  }
  return launch_k(block_gemv_kernel<Out, RT, QT, P_ROWS, EXACT, false>, grid, block, st, tok, a);
}

template <class Out, bool P_ROWS, bool EXACT>
static hipError_t launch_rows(const GemvArgs& a, bool fused, hipStream_t st, int tok) {
  // 16 rows of b per workgroup while all workgroups are on the chip at once (three to a compute
  // unit), else 32. One token, weights from memory, 16 / 32 rows (N x K): 1024 x 4096 6.5 / 8.6 us,
  // 11008 x 4096 13.8 / 14.0, 4096 x 11008 14.9 / 16.9; 13824 x 5120 17.6 / 15.7, 16384 x 1024
  // 7.8 / 6.6, 32000 x 4096 32.5 / 29.8. (Against the rule: 5120 x 13824 20.1 / 18.4, 20000 x 2048
  // 11.4 / 12.3.)
  if (a.M > 16) return launch_gemv<Out, 1, 2, P_ROWS, EXACT>(a, fused, st, tok);
  return a.N > 16 * 3 * 256 ? launch_gemv<Out, 2, 1, P_ROWS, EXACT>(a, fused, st, tok)
                            : launch_gemv<Out, 1, 1, P_ROWS, EXACT>(a, fused, st, tok);
}

template <class Out, bool EXACT>
static hipError_t launch_out(const GemvArgs& a, bool fused, hipStream_t st, int tok) {
  return a.p.tiles ? launch_rows<Out, false, EXACT>(a, fused, st, tok) : launch_rows<Out, true, EXACT>(a, fused, st, tok);
}

hipError_t block_gemv_pass(const BlockGemmPass& p, const void* x, int x_dt, bool pow2, hipStream_t st) {
  if (!block_gemv_ok(p.M, p.N, p.K) || (x && !block_gemv_fused_ok(p.M, p.K)))
    return hipErrorInvalidValue;
  GemvArgs a{p.b, p.a, x, static_cast<int>(p.M), p.N, static_cast<int>(p.K), x_dt, pow2, p.c, p.accumulate};
  const int tok = prof_open(K_GEMM, 2.0 * p.M * p.N * p.K);
  switch (p.out_dt) {
    case DT_F32: return launch_out<F32, true>(a, x != nullptr, st, tok);
    case DT_F16: return launch_out<F16, false>(a, x != nullptr, st, tok);
    case DT_BF16: return launch_out<BF16, false>(a, x != nullptr, st, tok);
  }
  return hipErrorInvalidValue;
}

}  // namespace hq
