// hq_kv_attention.hip — attention over the paged cache of microscaled 4-bit codes:
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j - m_i),
// in one pass over the cache with running maxima m and sums.
//
// A workgroup takes 16 query rows of one sequence and one head of the cache (a group of query heads
// times a few tokens) and a part of the tokens; its four waves take every fourth chunk of 64 tokens
// each. The products are transposed, S^T = K Q^T and O^T = V^T P^T, so that a lane keeps one query
// row throughout (lane % 16): the statistics of a row are a lane's own, and the probabilities leave the
// first product in the very registers that the second one reads them from (the tokens of a chunk in
// another order, the same for P and V).
//   K: a lane holds D / 4 consecutive elements of a token, straight from memory, inside one or two
//      blocks, and widens them with their scale: E2M1 times a power of two is a bf16 number.
//   V: the contraction runs over tokens, the codes lie along D: the chunk goes through LDS and is read
//      transposed, 16 tokens of a column a lane. A value's scale belongs to a token, so it multiplies
//      the probability, once for each block of D.
// Rotated caches: (H q) . (H k) = D q . k, and the sum of rotated values is the rotated sum, so queries
// are rotated in the prologue and outputs in the epilogue.
//
// Precision: fp32 statistics, scores and accumulators. Queries and probabilities are split into NS bf16
// numbers (2: within 2^-17, 3: 2^-25), each a matrix instruction of its own; codes are exact.
#include "hq_device.hpp"
#include "hq_kv_index.hpp"
#include "hq_launch.hpp"
#include "hq_mx_device.hpp"
#include "hq_mx_internal.hpp"

namespace hq {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kRows = 16;          // query rows of a workgroup
constexpr int kChunk = 64;         // tokens of a wave's step
constexpr int kWaves = 4;
constexpr float kLn2 = 0.693147180559945309f;

struct KvAttnArgs {
  const void* q;
  int q_dt;
  int64_t tokens, q_token, q_head;
  const uint8_t *k_codes, *v_codes, *k_scales, *v_scales;
  int64_t pages;
  int shift, heads, rot;
  const int32_t *q_starts, *lens, *table;
  int64_t table_ld;
  int max_q, max_len, group, window;
  float scale2;                    // scale log2(e) (/ D if rotated): scores are powers of two
  void* out;
  int out_dt;
  float* lse;
  int tiles, splits;
  float* part;                     // several splits: their sums and statistics
  float* stats;
};

__device__ inline float load_any(const void* p, int dt, int64_t i) {
  return dt == DT_F32 ? F32::load(p, i) : dt == DT_F16 ? F16::load(p, i) : BF16::load(p, i);
}
__device__ inline void load8_any(const void* p, int dt, int64_t i, int n, float (&v)[8]) {
  if (dt == DT_F32) load8<F32>(p, i, n, v);
  else if (dt == DT_F16) load8<F16>(p, i, n, v);
  else load8<BF16>(p, i, n, v);
}
__device__ inline void store8_any(void* p, int dt, int64_t i, const float (&v)[8]) {
  if (dt == DT_F32) store8<F32>(p, i, 8, v);
  else if (dt == DT_F16) store8<F16>(p, i, 8, v);
  else store8<BF16>(p, i, 8, v);
}

// What a workgroup works on: 16 rows from row r0 of a sequence's n x group (token by token).
struct KvTile {
  KvSequence s;
  int head, r0, rows;      // rows: of the sequence
  int64_t index;           // of the tile, for the partial results
  __device__ KvTile(const KvAttnArgs& g, int64_t work) {
    index = work;
    const int tile = static_cast<int>(work % g.tiles);
    const int64_t sh = work / g.tiles;
    head = static_cast<int>(sh % g.heads);
    seq = static_cast<int>(sh / g.heads);
    s = kv_sequence(g.q_starts[seq], g.q_starts[seq + 1], g.lens[seq], g.tokens, g.max_q, g.max_len);
    r0 = tile * kRows;
    rows = s.n * g.group;
  }
  int seq;
  __device__ int64_t token(const KvAttnArgs& g, int r) const { return s.first + r / g.group; }
  __device__ int q_head(const KvAttnArgs& g, int r) const { return head * g.group + r % g.group; }
};

// x as NS bf16 numbers that add up to it, eight at a time.
template <int NS>
__device__ inline void split8(const float (&x)[8], v8b (&out)[NS]) {
  float rest[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) rest[j] = x[j];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    v4u w;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = BF16::pack2(rest[2 * j], rest[2 * j + 1]);
      if (s + 1 < NS) {
        rest[2 * j] -= __uint_as_float(w[j] << 16);
        rest[2 * j + 1] -= __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
    out[s] = __builtin_bit_cast(v8b, w);
  }
}

// Eight codes times their scale as bf16 numbers (exact).
__device__ inline v8b widen8(uint32_t w, float s) {
  const v2b a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
  const v2b b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
  const v2b c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
  const v2b d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
  return v8b{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// x y, but 0 where either is 0, whatever the other: v_mul_legacy_f32, by the compiler's own name (as
// inline assembly it would have to wait for a transcendental result by itself).
extern "C" __device__ float hq_fmul_legacy(float, float) __asm("llvm.amdgcn.fmul.legacy");
// p s: a token that a row does not see may have a scale that is not a number.
__device__ inline float times_scale(float p, float s) { return hq_fmul_legacy(p, s); }

__device__ inline float shfl_fmax(float x, int m) { return fmaxf(x, __shfl_xor(x, m, 64)); }

// Rotated back, divided and stored: eight elements of a row.
template <int D>
__device__ inline void finish_row(const KvAttnArgs& g, const KvTile& tile, int row, int l, float total, float m, bool in,
                                  float (&v)[8]) {
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;     // a row that sees nothing: zeros
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= inv;
  if (g.rot > 1) {
    rotate_lanes<D>(v, threadIdx.x & 63);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= 1.0f / D;
  }
  if (!in) return;
  const int64_t at = tile.token(g, row) * (g.heads * g.group) + tile.q_head(g, row);
  store8_any(g.out, g.out_dt, at * D + 8 * l, v);
  if (g.lse && l == 0) g.lse[at] = total == 0.0f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(total)) * kLn2;
}

template <int D, int NS>
__global__ __launch_bounds__(64 * kWaves) void kv_attention_kernel(KvAttnArgs g) {
  constexpr int NB = D / 32;                 // blocks of a head, and 32-wide steps of the first product
  constexpr int DT = D / 16;                 // 16-wide tiles of the output
  constexpr int VP = D / 2 + 8;              // bytes of a V row in LDS: 16 rows at a column on all banks
  constexpr int QP = D + 4;                  // floats of a row in LDS
  constexpr int V_BYTES = kWaves * kChunk * VP, O_BYTES = kWaves * kRows * QP * 4;
  __shared__ __attribute__((aligned(16))) uint8_t mem[V_BYTES > O_BYTES ? V_BYTES : O_BYTES];
  __shared__ float wave_m[kWaves][kRows], wave_l[kWaves][kRows];

  const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int split = static_cast<int>(blockIdx.x % g.splits);
  const KvTile tile(g, blockIdx.x / g.splits);
  if (tile.r0 >= tile.rows) return;
  const KvSequence& s = tile.s;

  // queries: rotated and scaled in fp32, through LDS to the lanes of the second operand
  float* const rows = reinterpret_cast<float*>(mem);
  for (int e = t; e < kRows * D / 8; e += 64 * kWaves) {
    const int row = tile.r0 + e / (D / 8), l = e % (D / 8);
    float v[8];
    const bool in = row < tile.rows;
    load8_any(g.q, g.q_dt, in ? tile.token(g, row) * g.q_token + tile.q_head(g, row) * g.q_head + 8 * l : 0, in ? 8 : 0, v);
    if (g.rot > 1) rotate_lanes<D>(v, lane);
#pragma unroll
    for (int j = 0; j < 8; ++j) rows[(e / (D / 8)) * QP + 8 * l + j] = v[j] * g.scale2;
  }
  __syncthreads();
  v8b qf[NB][NS];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = rows[lr * QP + (D / 4) * lg + 8 * b + j];
    split8<NS>(x, qf[b]);
  }
  __syncthreads();

  // tokens that this lane's row sees: [from, to); and those of all rows, and of any
  const int q0 = tile.r0 / g.group, q1 = min(tile.r0 + kRows - 1, tile.rows - 1) / g.group;
  auto end_of = [&](int i) { return static_cast<int>(max<int64_t>(0, min<int64_t>(s.len, s.pos0 + i + 1))); };
  auto start_of = [&](int i) { return g.window ? static_cast<int>(max<int64_t>(0, s.pos0 + i + 1 - g.window)) : 0; };
  const int my = (tile.r0 + lr) / g.group;
  const int from = start_of(my), to = tile.r0 + lr < tile.rows ? end_of(my) : 0;
  const int any_to = end_of(q1), any_from = start_of(q0), all_to = end_of(q0), all_from = start_of(q1);
  const int first = any_from / kChunk, chunks = max(0, (any_to + kChunk - 1) / kChunk - first);
  const int per = (chunks + g.splits - 1) / g.splits;
  const int begin = first + min(chunks, split * per), end = first + min(chunks, (split + 1) * per);

  v4f o[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) o[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  float m = -__builtin_inff(), l = 0.0f;     // l: of this lane's tokens
  uint8_t* const vs_lds = mem + w * kChunk * VP;
  const int32_t* const table = g.table + tile.seq * g.table_ld;

  for (int c = begin + w; c < end; c += kWaves) {
    const int t0 = c * kChunk;
    uint32_t kx[4][NB], vx[4][NB], vs[4][NB];   // codes of K and V, scale bytes of four tokens
    float ks[4][D == 256 ? 2 : 1];
    bool ok[4];
    bool all_ok = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = t0 + 16 * i < any_to ? kv_row_of_token(t0 + 16 * i, table, g.table_ld, g.pages, g.shift, g.heads, tile.head) : -1;
      ok[i] = row >= 0;
      all_ok &= ok[i];
      if (ok[i]) {
        __builtin_memcpy(kx[i], g.k_codes + (row + lr) * (D / 2) + lg * (D / 8), D / 8);
        __builtin_memcpy(vx[i], g.v_codes + row * (D / 2) + lane * (D / 8), D / 8);
        __builtin_memcpy(vs[i], g.v_scales + (row + 4 * lg) * NB, 4 * NB);
        const uint8_t* const kp = g.k_scales + (row + lr) * NB;
        if constexpr (D == 64) ks[i][0] = mx_scale(kp[lg >> 1]);
        else if constexpr (D == 128) ks[i][0] = mx_scale(kp[lg]);
        else ks[i][0] = mx_scale(kp[2 * lg]), ks[i][1] = mx_scale(kp[2 * lg + 1]);
      } else {
#pragma unroll
        for (int b = 0; b < NB; ++b) kx[i][b] = vx[i][b] = vs[i][b] = 0u;
        ks[i][0] = 0.0f;
        if constexpr (D == 256) ks[i][1] = 0.0f;
      }
    }
    // V into LDS: a lane's D / 8 bytes are a quarter of token 16 i + lane / 4
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int b = 0; b < NB; b += 2)
        *reinterpret_cast<uint2*>(vs_lds + (16 * i + (lane >> 2)) * VP + (lane & 3) * (D / 8) + 4 * b) = uint2{vx[i][b], vx[i][b + 1]};

    // scores of tokens 16 i + 4 lg + r
    float p[4][4];
    float top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v4f a = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const v8b k = widen8(kx[i][b], ks[i][D == 256 ? b / 4 : 0]);
#pragma unroll
        for (int e = NS - 1; e >= 0; --e) a = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, qf[b][e], a, 0, 0, 0);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) p[i][r] = a[r];
    }
    if (!all_ok || t0 + kChunk > all_to || t0 < all_from) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int at = t0 + 16 * i + 4 * lg + r;
          p[i][r] = ok[i] && at < to && at >= from ? p[i][r] : -__builtin_inff();
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) top = fmaxf(top, p[i][r]);
    top = fmaxf(m, shfl_fmax(shfl_fmax(top, 16), 32));
    const float base = top == -__builtin_inff() ? 0.0f : top;
    if (__any(top > m)) {
      const float f = __builtin_amdgcn_exp2f(m - base);
      l *= f;
#pragma unroll
      for (int i = 0; i < DT; ++i) o[i] *= f;
    }
    m = top;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        p[i][r] = __builtin_amdgcn_exp2f(p[i][r] - base);
        l += p[i][r];
      }
    __builtin_amdgcn_wave_barrier();

    // O^T += V^T P^T, block by block of D
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      v8b pf[2][NS];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = 2 * h + j / 4, r = j % 4, at = r * NB + b;
          x[j] = times_scale(p[i][r], mx_scale((vs[i][at / 4] >> (8 * (at % 4))) & 0xFF));
        }
        split8<NS>(x, pf[h]);
      }
#pragma unroll
      for (int dt = 2 * b; dt < 2 * b + 2; ++dt) {
        // 16 x 16 codes transposed: from row 16 i + 4 lg + r of lane 4 i + r, columns 16 dt + lane % 16
        const v2i y = __builtin_amdgcn_ds_read_tr4_b64_v2i32(
            (__attribute__((address_space(3))) v2i*)(vs_lds + (16 * (lr >> 2) + 4 * lg + (lr & 3)) * VP + 8 * dt));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const v8b v = widen8(static_cast<uint32_t>(y[h]), 1.0f);
#pragma unroll
          for (int e = NS - 1; e >= 0; --e) o[dt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, pf[h][e], o[dt], 0, 0, 0);
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }

  // the waves' sums, to a common maximum
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);
  if (lane < kRows) wave_m[w][lane] = m, wave_l[w][lane] = l;
  __syncthreads();
  float top = wave_m[0][lr];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) top = fmaxf(top, wave_m[i][lr]);
  const float f = __builtin_amdgcn_exp2f(m - (top == -__builtin_inff() ? 0.0f : top));
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
    *reinterpret_cast<v4f*>(rows + (w * kRows + lr) * QP + 16 * dt + 4 * lg) = o[dt] * f;
  __syncthreads();
  for (int e = t; e < kRows * D / 8; e += 64 * kWaves) {
    const int r = e / (D / 8), i = e % (D / 8);
    float big = wave_m[0][r];
#pragma unroll
    for (int k = 1; k < kWaves; ++k) big = fmaxf(big, wave_m[k][r]);
    const float base = big == -__builtin_inff() ? 0.0f : big;
    float total = 0.0f, v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kWaves; ++k) {
      total += wave_l[k][r] * __builtin_amdgcn_exp2f(wave_m[k][r] - base);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += rows[(k * kRows + r) * QP + 8 * i + j];
    }
    if (g.splits == 1) {
      finish_row<D>(g, tile, tile.r0 + r, i, total, base, tile.r0 + r < tile.rows, v);
    } else {
      const int64_t at = (tile.index * g.splits + split) * kRows + r;
      store8<F32>(g.part, at * D + 8 * i, 8, v);
      if (i == 0) {
        g.stats[2 * at] = big;
        g.stats[2 * at + 1] = total;
      }
    }
  }
}

// The splits' sums of a tile's rows, to a common maximum, in their order.
template <int D>
__global__ __launch_bounds__(256) void kv_join_kernel(KvAttnArgs g) {
  const KvTile tile(g, blockIdx.x);
  if (tile.r0 >= tile.rows) return;
  for (int e = threadIdx.x; e < kRows * D / 8; e += 256) {
    const int r = e / (D / 8), i = e % (D / 8);
    const int64_t at = tile.index * g.splits * kRows + r;
    float big = -__builtin_inff();
    for (int k = 0; k < g.splits; ++k) big = fmaxf(big, g.stats[2 * (at + k * kRows)]);
    const float base = big == -__builtin_inff() ? 0.0f : big;
    float total = 0.0f, v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int k = 0; k < g.splits; ++k) {
      const float f = __builtin_amdgcn_exp2f(g.stats[2 * (at + k * kRows)] - base);
      total += g.stats[2 * (at + k * kRows) + 1] * f;
      float x[8];
      load8<F32>(g.part, (at + k * kRows) * D + 8 * i, 8, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __builtin_fmaf(x[j], f, v[j]);
    }
    finish_row<D>(g, tile, tile.r0 + r, i, total, base, tile.r0 + r < tile.rows, v);
  }
}

// Parts of the tokens over workgroups, while the rows alone leave the chip idle: four workgroups to a
// compute unit, and at least a chunk for each wave.
struct KvPlan {
  int64_t tiles;      // of a sequence and head
  int64_t work;       // of the batch
  int splits;
};
static KvPlan kv_plan(const hq_kv_cache& c, const hq_kv_batch& b) {
  KvPlan p;
  p.tiles = (static_cast<int64_t>(b.max_q) * (b.q_heads / c.heads) + kRows - 1) / kRows;
  p.work = static_cast<int64_t>(b.seqs) * c.heads * p.tiles;
  const int64_t most = (static_cast<int64_t>(b.max_len) + kWaves * kChunk - 1) / (kWaves * kChunk);
  int64_t s = p.work > 0 ? (1024 + p.work - 1) / p.work : 1;
  s = s < most ? s : most;
  p.splits = static_cast<int>(s < 1 ? 1 : s > 256 ? 256 : s);
  return p;
}

static size_t part_bytes(const KvPlan& p, int D) {
  return static_cast<size_t>(p.work) * p.splits * kRows * D * sizeof(float);
}

size_t kv_attention_ws(const hq_kv_cache& c, const hq_kv_batch& b) {
  const KvPlan p = kv_plan(c, b);
  if (p.splits == 1 || p.work == 0) return 0;
  return part_bytes(p, c.head_dim) + static_cast<size_t>(p.work) * p.splits * kRows * 2 * sizeof(float);
}

template <int D>
static hipError_t launch_dim(const KvAttnArgs& a, const KvPlan& p, bool wide, hipStream_t st, int tok) {
  const dim3 grid(static_cast<unsigned>(p.work * p.splits)), block(64 * kWaves);
  const hipError_t e = wide ? launch_k(kv_attention_kernel<D, 3>, grid, block, st, tok, a)
                            : launch_k(kv_attention_kernel<D, 2>, grid, block, st, tok, a);
  if (e != hipSuccess || p.splits == 1) return e;
  return launch_k(kv_join_kernel<D>, dim3(static_cast<unsigned>(p.work)), dim3(256), st,
                  prof_open(K_MISC, static_cast<double>(part_bytes(p, D))), a);
}

hipError_t kv_attention_pass(const KvAttentionPass& p, hipStream_t st) {
  const hq_kv_cache& c = p.cache;
  const hq_kv_batch& b = p.batch;
  const KvPlan plan = kv_plan(c, b);
  if (plan.work == 0) return hipSuccess;
  if (plan.splits > 1 && !p.ws) return hipErrorInvalidValue;
  KvAttnArgs a = {};
  a.q = p.q;
  a.q_dt = p.q_dt;
  a.tokens = p.tokens;
  a.q_token = p.q_token;
  a.q_head = p.q_head;
  a.k_codes = c.k_codes;
  a.v_codes = c.v_codes;
  a.k_scales = c.k_scales;
  a.v_scales = c.v_scales;
  a.pages = c.pages;
  a.shift = __builtin_ctz(static_cast<unsigned>(c.page));
  a.heads = c.heads;
  a.rot = c.rot;
  a.q_starts = b.q_starts;
  a.lens = b.lens;
  a.table = b.table;
  a.table_ld = b.table_ld;
  a.max_q = b.max_q;
  a.max_len = b.max_len;
  a.group = b.q_heads / c.heads;
  a.window = b.window;
  a.scale2 = static_cast<float>(static_cast<double>(b.scale) * 1.4426950408889634 / c.rot);
  a.out = p.out;
  a.out_dt = p.out_dt;
  a.lse = p.lse;
  a.tiles = static_cast<int>(plan.tiles);
  a.splits = plan.splits;
  a.part = static_cast<float*>(p.ws);
  if (plan.splits > 1) a.stats = a.part + part_bytes(plan, c.head_dim) / sizeof(float);
  const bool wide = p.q_dt == DT_F32 || p.out_dt == DT_F32;
  const double units = 4.0 * c.head_dim * b.q_heads * static_cast<double>(p.tokens) * b.max_len;
  const int tok = prof_open(K_GEMM, units);
  switch (c.head_dim) {
    case 64: return launch_dim<64>(a, plan, wide, st, tok);
    case 128: return launch_dim<128>(a, plan, wide, st, tok);
    case 256: return launch_dim<256>(a, plan, wide, st, tok);
  }
  return hipErrorInvalidValue;
}

}  // namespace hq
