// hq_kv_attention.hip — attention over the paged cache of microscaled 4-bit codes:
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j - m_i),
// in one pass over the cache with running maxima m and sums.
//
// A wave takes 16 RT (RT = 1 or 2) query rows of one sequence and one head of the cache (a group of query heads
// times a few tokens) through chunks of 64 tokens. The products are transposed, S^T = K Q^T and
// O^T = V^T P^T, so that a lane keeps one query row throughout (lane % 16): the statistics of a row
// are a lane's own, and the probabilities leave the first product in the very registers that the
// second one reads them from (the tokens of a chunk in another order, the same for P and V).
//   K: the codes and their scale bytes go from memory into v_mfma_scale_f32_16x16x128_f8f6f4 as they
//      are: a lane's 32 elements are one block. The other operand, Q, is a sum of QN parts in 6 bits
//      (E2M3), each with a scale for 32 elements: each part takes the rest of the ones before, so its
//      scale is 2^-4, then 2^-5 of the last. At 16 cycles an instruction that costs as much as two
//      bf16 parts would, without the widening of K.
//   V: the contraction runs over tokens, the scales lie along D, so codes are widened to bf16 with
//      their scales (exact). A lane reads the same D / 16 elements of each of its tokens and pairs
//      tokens by byte permutes.
// Codes and scales go straight from memory into LDS, a chunk ahead of their use.
// Rotated caches: (H q) . (H k) = D q . k, and the sum of rotated values is the rotated sum, so queries
// are rotated in the prologue and outputs in the epilogue.
//
// Few rows and many tokens: all chunks of a call form a line, of which each wave takes an even piece; a second
// kernel joins the parts of rows whose tokens lay in several pieces. Few rows and tokens: the waves of a
// workgroup share the rows, and their sums meet in LDS. Many rows: each wave has rows of its own.
//
// Precision: fp32 statistics, scores and accumulators. Of the largest in its block of 32, a query is
// kept to 2^-18 (QN = 4) or 2^-28 (6; fp32 in or out). Probabilities are split into PN bf16 numbers:
// to 2^-17 (2) or 2^-25 (3). Four and two leave less than outputs of 16 bits round away (2^-8, 2^-11), and
// six and three cost a prompt 37 % more.
//
// What bounds it: single tokens of many long sequences the bytes of the cache (32 of up to 16384 tokens, 8 heads
// of 128: 364 MB in 78 us, 4.7 TB/s, and 7.5 us of joining); of few a memory round trip for each step of 64 tokens
// (one of 777: 12.4 us, of 32768: 34.5); prompts the vector and the matrix pipe in turns (2 x 1500 rows over
// 9000, 40 heads on 8 of 128: 454 us, 0.74 PFLOP/s, the pipes busy for 47 and 33 % of the time; fp32 620, where
// 37 registers spill, 152 bytes a lane; 700 rows of 256 elements 602 and 718).
#include <algorithm>

#include "hq_device.hpp"
#include "hq_kv_index.hpp"
#include "hq_launch.hpp"
#include "hq_mx_device.hpp"
#include "hq_mx_internal.hpp"

namespace hq {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef uint32_t v6u __attribute__((ext_vector_type(6)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v32f __attribute__((ext_vector_type(32)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

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
  float scale2;                    // |scale| log2(e) (/ D if rotated): scores become powers of two
  float sign;                      // of scale, taken by the queries
  void* out;
  int out_dt;
  float* lse;
  int seqs, tiles, splits, tile_rows;
  int least;                       // chunks of a wave's piece of the line at least; 0: no line
  float* part;                     // parts of rows' tokens: their sums and statistics
  float* stats;
};

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

// Memory that no kernel of a call writes, read through the scalar cache where the address is uniform.
typedef const __attribute__((address_space(4))) int32_t* ConstInts;
__device__ inline ConstInts constant(const int32_t* p) { return (ConstInts)(reinterpret_cast<uintptr_t>(p)); }

// Rows from row r0 of a sequence's n x group (token by token), and a head of the cache. Inlined by force: a call
// puts it into scratch memory.
struct KvTile {
  KvSequence s;
  int seq, head, r0, rows;      // rows: of the sequence
  __device__ __forceinline__ KvTile(const KvAttnArgs& g, int seq_, int tile, int head_) : seq(seq_), head(head_) {
    s = kv_sequence(constant(g.q_starts)[seq], constant(g.q_starts)[seq + 1], constant(g.lens)[seq], g.tokens, g.max_q, g.max_len);
    r0 = tile * g.tile_rows;
    rows = s.n * g.group;
  }
  __device__ __forceinline__ int64_t token(const KvAttnArgs& g, int r) const { return s.first + r / g.group; }
  __device__ __forceinline__ int q_head(const KvAttnArgs& g, int r) const { return head * g.group + r % g.group; }
  // tokens [from, to) that query row i of the sequence sees, and the chunks that a row of the tile sees
  __device__ __forceinline__ int end_of(int i) const { return kv_end_of(s, i); }
  __device__ __forceinline__ int start_of(const KvAttnArgs& g, int i) const { return kv_start_of(s, i, g.window); }
  __device__ __forceinline__ int last_row(const KvAttnArgs& g) const { return (min(r0 + g.tile_rows, rows) - 1) / g.group; }
  __device__ __forceinline__ int first_chunk(const KvAttnArgs& g) const { return start_of(g, r0 / g.group) / kChunk; }
  __device__ __forceinline__ int end_token(const KvAttnArgs& g) const { return end_of(last_row(g)); }
  __device__ __forceinline__ int chunks(const KvAttnArgs& g) const {
    return r0 < rows ? kv_chunks(s, r0 / g.group, last_row(g), g.window, kChunk).count : 0;
  }
};

// The chunks of all rows in a line (sequence by sequence, tile by tile, head by head), cut into even
// pieces, one for each wave of a call. A prefix sum over the sequences' tiles by all threads of a
// workgroup; every workgroup of a call comes to the same numbers.
struct KvLine {
  int64_t total;      // chunks of the batch
  int64_t piece;      // of a wave
  int tile;           // that this wave's piece begins in (or the wanted one); -1: none
  int64_t before;     // chunks that lie before this tile
};
__device__ inline int tile_chunks(const KvAttnArgs& g, int tile) { return KvTile(g, tile / g.tiles, tile % g.tiles, 0).chunks(g); }

// wanted < 0: for the pieces of this workgroup's waves; else for a tile. waves: of the call.
__device__ inline KvLine kv_line(const KvAttnArgs& g, int waves, int wanted) {
  __shared__ int64_t sums[kWaves];
  __shared__ int tile_of[kWaves];
  __shared__ int64_t before_of[kWaves];
  const int n = g.seqs * g.tiles, t = threadIdx.x, lane = t & 63, w = t >> 6;
  const int strip = (n + 64 * kWaves - 1) / (64 * kWaves);
  int64_t mine = 0;
  for (int i = t * strip; i < min(n, (t + 1) * strip); ++i) mine += tile_chunks(g, i);
  mine *= g.heads;
  int64_t up_to = mine;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const int64_t x = __shfl_up(up_to, m, 64);
    if (lane >= m) up_to += x;
  }
  if (lane == 63) sums[w] = up_to;
  if (t < kWaves) tile_of[t] = -1;
  __syncthreads();
  int64_t base = 0;
  KvLine line = {0, 0, -1, 0};
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    if (i < w) base += sums[i];
    line.total += sums[i];
  }
  line.piece = max<int64_t>(g.least, (line.total + waves - 1) / waves);
  const int64_t from = base + up_to - mine;
#pragma unroll
  for (int k = 0; k < kWaves; ++k) {
    const int64_t at = (static_cast<int64_t>(blockIdx.x) * kWaves + k) * line.piece;
    const bool here = wanted >= 0 ? k == 0 && wanted >= t * strip && wanted < min(n, (t + 1) * strip) : at >= from && at < from + mine;
    if (here) {
      int64_t before = from;
      int i = t * strip;
      for (; i + 1 < min(n, (t + 1) * strip); ++i) {
        if (wanted >= 0 && i == wanted) break;
        const int64_t c = static_cast<int64_t>(tile_chunks(g, i)) * g.heads;
        if (wanted < 0 && at < before + c) break;
        before += c;
      }
      tile_of[k] = i;
      before_of[k] = before;
    }
  }
  __syncthreads();
  const int k = wanted >= 0 ? 0 : w;
  line.tile = tile_of[k];
  line.before = line.tile >= 0 ? before_of[k] : 0;
  return line;
}

// x as PN bf16 numbers that add up to it, eight at a time.
template <int PN>
__device__ inline void split8(const float (&x)[8], v8b (&out)[PN]) {
  float rest[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) rest[j] = x[j];
#pragma unroll
  for (int s = 0; s < PN; ++s) {
    v4u w;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = BF16::pack2(rest[2 * j], rest[2 * j + 1]);
      if (s + 1 < PN) {
        rest[2 * j] -= __uint_as_float(w[j] << 16);
        rest[2 * j + 1] -= __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
    out[s] = __builtin_bit_cast(v8b, w);
  }
}

// 32 values divided by s in 6 bits (E2M3, to nearest even), element j in bits 6 j of the result, and
// back. The conversion takes even and odd elements apart. Both write before they have read everything,
// which the builtins do not tell the register allocator (it has given v[32:37] as the result of
// v[2:17] and v[18:33]): hence the assembly, with outputs of their own.
__device__ inline v6u to_e2m3(const float (&x)[32], float s) {
  v16f even, odd;
#pragma unroll
  for (int j = 0; j < 16; ++j) even[j] = x[2 * j], odd[j] = x[2 * j + 1];
  v6u y;
  asm("s_nop 1\n\tv_cvt_scalef32_2xpk16_fp6_f32 %0, %1, %2, %3" : "=&v"(y) : "v"(even), "v"(odd), "v"(s));
  return y;
}
__device__ inline void subtract_e2m3(v6u y, float s, float (&x)[32]) {
  v32f z;
  asm("s_nop 1\n\tv_cvt_scalef32_pk32_f32_fp6 %0, %1, %2\n\ts_nop 1" : "=&v"(z) : "v"(y), "v"(s));
#pragma unroll
  for (int j = 0; j < 32; ++j) x[j] -= z[j];
}

// 32 consecutive elements of a query as QN parts and their scale bytes. An infinity or a NaN makes
// the row's scores NaN. Parts whose scale would fall below 2^-127 (blocks below 2^-100) are left out.
template <int QN>
__device__ inline void split_query(float (&x)[32], v6u (&part)[QN], int (&byte)[QN]) {
  uint32_t a = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) a = max(a, mag(x[j]));
  const int b0 = a >= 0x7F800000u ? 255 : max(static_cast<int>((a + 0xFFFFFu) >> 23) - 2, 1);   // a <= 7.5 2^(b0 - 127)
#pragma unroll
  for (int i = 0; i < QN; ++i) {
    const int b = i == 0 ? b0 : b0 + 1 - 5 * i;
    const bool use = b0 != 255 && b > 0;
    const float s = __uint_as_float(static_cast<uint32_t>(use ? b : 127) << 23);
    part[i] = to_e2m3(x, s);
    if (!use) part[i] = v6u{0u, 0u, 0u, 0u, 0u, 0u};
    if (i + 1 < QN) subtract_e2m3(part[i], s, x);
    byte[i] = b0 == 255 ? 255 : max(b, 0);
  }
}

// Stages of H_D on D elements of a row of which this lane holds N consecutive ones from N (lane / 16 %
// LANES) on, in rising strides: in registers, then across lanes 16 and 32 apart.
template <int N, int LANES>
__device__ inline void rotate_row(float (&v)[N], int lane) {
  fwht_inreg<N, N>(v);
  if constexpr (LANES > 1) fwht_xlane_c<16>(v, lane);
  if constexpr (LANES > 2) fwht_xlane_c<32>(v, lane);
}

// c + K Q over 128 (64) elements: codes times 6-bit numbers. e: the byte of qb (a constant once unrolled).
__device__ __forceinline__ v4f multiply_part(int e, v4i k, int kb, v8i q, int qb, v4f c) {
  const v8i x = {k[0], k[1], k[2], k[3], 0, 0, 0, 0};
  switch (e & 3) {
    case 0: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, q, c, 4, 2, 0, kb, 0, qb);
    case 1: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, q, c, 4, 2, 0, kb, 1, qb);
    case 2: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, q, c, 4, 2, 0, kb, 2, qb);
    default: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, q, c, 4, 2, 0, kb, 3, qb);
  }
}

__device__ inline float shfl_fmax(float x, int m) { return fmaxf(x, __shfl_xor(x, m, 64)); }

// Rotated back, divided and stored: eight elements of a row.
template <int D>
__device__ inline void finish_row(const KvAttnArgs& g, const KvTile& tile, int row, int l, float total, float m, bool in,
                                  float (&v)[8]) {
  // a row that sees nothing: zeros. The rotation's 1 / D comes before its sums, which then stay in range
  const float inv = total == 0.0f ? 0.0f : 1.0f / total * (g.rot > 1 ? 1.0f / D : 1.0f);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= inv;
  if (g.rot > 1) rotate_lanes<D>(v, threadIdx.x & 63);
  if (!in) return;
  const int64_t at = tile.token(g, row) * (g.heads * g.group) + tile.q_head(g, row);
  store8_any(g.out, g.out_dt, at * D + 8 * l, v);
  if (g.lse && l == 0) g.lse[at] = total == 0.0f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(total)) * kLn2;
}

// 16 or 4 bytes a lane from a scalar address and the lane's offset straight into LDS (lane l at to + l * BYTES).
template <int BYTES>
__device__ __forceinline__ void load_to_lds(const uint8_t* base, uint32_t offset, int8_t* to) {
  const auto from = (const __attribute__((address_space(1))) void*)(base + offset);
  const auto lds = (__attribute__((address_space(3))) void*)to;
  if constexpr (BYTES == 16) __builtin_amdgcn_global_load_lds(from, lds, 16, 0, 0);
  else __builtin_amdgcn_global_load_lds(from, lds, 4, 0, 0);
}

// A chunk's codes and scales in LDS. Token u = 4 a + b of a tile of 16 is row 4 b + a of the score's tile
// and so element (a, lane / 16 = b) of the second product's: four lane groups then read four neighbouring
// tokens of V. The 16-byte pieces of a token are XORed with a few of its bits, so that reads of
// a piece of many tokens (K) spread over the banks.
template <int D>
struct KvStage {
  static constexpr int NB = D / 32;              // scale bytes, and 16-byte pieces, of a token
  static constexpr int KU = D == 256 ? 2 : 1;    // instructions of a tile of scores along D
  static constexpr int VD = D == 256 ? 2 : 1;    // dwords of V that a lane reads of a token (half of one for D = 64)
  static constexpr int CODES = kChunk * D / 2, SCALES = kChunk * NB;
  static constexpr int BYTES = 2 * CODES + 2 * SCALES;
  __device__ static int piece(int u, int c) { return c ^ (D == 64 ? (u >> 3) & 1 : (u >> 2) & 3); }
  __device__ static int turned(int u) { return 4 * (u & 3) + (u >> 2); }

  // Codes of N tiles of 16 tokens from `row` on (a scalar base and the lane's offset).
  template <int N>
  __device__ static void load_codes(const uint8_t* pool, int64_t row, int8_t* to, int lane) {
    constexpr int PIECES = 16 * NB;              // of a tile
    const uint8_t* const base = pool + row * (D / 2);
#pragma unroll
    for (int q = 0; q < (N * PIECES + 63) / 64; ++q) {
      const int at = 64 * q + lane, tok = at / NB, c = at % NB;
      if (N * PIECES >= 64 || lane < PIECES)
        load_to_lds<16>(base, static_cast<uint32_t>(tok * (D / 2) + 16 * piece(tok & 15, c)), to + 1024 * q);
    }
  }
  // The scale bytes of a chunk in four tiles; for D = 128 the tokens of a tile in turned order.
  __device__ static void load_scales(const uint8_t* pool, const int64_t (&row)[4], int8_t* to, int lane) {
    constexpr int DWORDS = 4 * NB;               // of a tile
    const int64_t r0 = row[0], r1 = row[1], r2 = row[2], r3 = row[3];
#pragma unroll
    for (int q = 0; q < (4 * DWORDS + 63) / 64; ++q) {
      const int at = 64 * q + lane, i = at / DWORDS, d = at % DWORDS;
      const int64_t r = i < 2 ? (i == 0 ? r0 : r1) : (i == 2 ? r2 : r3);
      if (at < 4 * DWORDS && r >= 0)
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(pool + r * NB + 4 * (D == 128 ? turned(d) : d)),
                                         (__attribute__((address_space(3))) void*)(to + 256 * q), 4, 0, 0);
    }
  }
  // The same of 64 tokens from `row` on.
  __device__ static void load_scales(const uint8_t* pool, int64_t row, int8_t* to, int lane) {
    constexpr int DWORDS = 4 * NB;
    const uint8_t* const base = pool + row * NB;
#pragma unroll
    for (int q = 0; q < (4 * DWORDS + 63) / 64; ++q) {
      const int at = 64 * q + lane, i = at / DWORDS, d = at % DWORDS;
      if (4 * DWORDS >= 64 || at < 4 * DWORDS)
        load_to_lds<4>(base, static_cast<uint32_t>(4 * (DWORDS * i + (D == 128 ? turned(d) : d))), to + 256 * q);
    }
  }
  __device__ static int8_t* k_codes(int8_t* s, int i) { return s + i * (16 * D / 2); }
  __device__ static int8_t* v_codes(int8_t* s, int i) { return s + CODES + i * (16 * D / 2); }
  __device__ static int8_t* k_scales(int8_t* s) { return s + 2 * CODES; }
  __device__ static int8_t* v_scales(int8_t* s) { return s + 2 * CODES + SCALES; }

  // What a lane reads: 16 bytes and the scale byte of its token of a tile of K (D = 64: lanes 32 on read
  // the same again, for other parts of Q),
  __device__ static v4i k(const int8_t* s, int i, int u, int lr, int lg) {
    const int tok = turned(lr);
    return *reinterpret_cast<const v4i*>(s + (16 * i + tok) * (D / 2) + 16 * piece(tok, 4 * u + (D == 64 ? lg & 1 : lg)));
  }
  __device__ static int k_scale(const int8_t* s, int i, int u, int lr, int lg) {
    const int slot = D == 128 ? lr : turned(lr);
    return static_cast<uint8_t>(s[2 * CODES + (16 * i + slot) * NB + 4 * u + (D == 64 ? lg & 1 : lg)]);
  }
  // its D / 16 codes of token (r, lg) of a tile of V,
  __device__ static void v(const int8_t* s, int i, int r, int lr, int lg, uint32_t (&x)[VD]) {
    const int tok = 4 * r + lg;
    const int8_t* const at = s + CODES + (16 * i + tok) * (D / 2);
    if constexpr (D == 64) {
      x[0] = *reinterpret_cast<const uint16_t*>(at + 16 * piece(tok, lr >> 3) + 2 * (lr & 7));
    } else if constexpr (D == 128) {
      x[0] = *reinterpret_cast<const uint32_t*>(at + 16 * piece(tok, lr >> 2) + 4 * (lr & 3));
    } else {
      const uint2 y = *reinterpret_cast<const uint2*>(at + 16 * piece(tok, lr >> 1) + 8 * (lr & 1));
      x[0] = y.x, x[1] = y.y;
    }
  }
  // and patterns whose bits 23 to 30 are the scale bytes of its block of V for the four tokens (r, lg);
  // the conversions read nothing else of them.
  __device__ static void v_scale(const int8_t* s, int i, int lr, int lg, uint32_t (&x)[4]) {
    const int8_t* const at = s + 2 * CODES + SCALES;
    if constexpr (D == 128) {
      const uint4 y = *reinterpret_cast<const uint4*>(at + (16 * i + 4 * lg) * NB);
      const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] = __builtin_amdgcn_alignbit(w[r], w[r], (8 * (lr >> 2) + 9) & 31);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        x[r] = static_cast<uint32_t>(static_cast<uint8_t>(at[(16 * i + 4 * r + lg) * NB + (D == 64 ? lr >> 3 : lr >> 1)])) << 23;
    }
  }
};

// The pages of a sequence, 64 entries of its table at a time in the lanes: an entry is a lane's, read
// without a wait. (A load for each chunk would be waited for behind the chunk's own loads, or, through the
// scalar cache, took a third of an iteration.) Nothing is read before a token is asked for: a wave without
// a chunk reads no table, and there may be none.
struct KvPages {
  const int32_t* table;
  int64_t ld, pages;
  int shift, heads, head;
  int from;          // first entry held; at first far below any
  int32_t held;      // entry from + lane; -1 past the table's end
  __device__ KvPages(const KvAttnArgs& g, const KvTile& tile)
      : table(g.table + tile.seq * g.table_ld), ld(g.table_ld), pages(g.pages), shift(g.shift), heads(g.heads), head(tile.head),
        from(-(1 << 30)), held(-1) {}
  __device__ void fetch(int entry) {
    from = entry;
    const int64_t mine = static_cast<int64_t>(entry) + (threadIdx.x & 63);
    held = kv_entry_in_table(mine, ld) ? table[mine] : -1;
  }
  // Row of token `at` >= 0, or -1; `at` is the same in all lanes.
  __device__ int64_t row(int at) {
    const int entry = at >> shift;
    if (static_cast<unsigned>(entry - from) >= 64u) fetch(entry);
    return kv_row_in_page(at, __builtin_amdgcn_readlane(held, entry - from), pages, shift, heads, head);
  }
  // Rows of the four tiles of the chunk from token t0 on; -1: behind `end` or in no page. What LDS holds of
  // such a tile does not matter: codes are numbers whatever their bits, and its tokens count as masked. With
  // pages of 64 tokens and more all four lie in one, and are loaded whole.
  __device__ void chunk(int t0, int end, int64_t (&r)[4]) {
    if (shift >= 6) {
      r[0] = t0 < end ? row(t0) : -1;
#pragma unroll
      for (int i = 1; i < 4; ++i) r[i] = r[0] >= 0 ? r[0] + 16 * i : -1;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = t0 + 16 * i < end ? row(t0 + 16 * i) : -1;
    }
  }
};

template <int N>
struct Const {
  static constexpr int value = N;
};

// The two codes of a byte times the scale in bits 23 to 30 of s, as bf16 numbers (exact).
template <int BYTE>
__device__ __forceinline__ uint32_t widen2(uint32_t w, uint32_t s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, __uint_as_float(s), BYTE));
}

// How the waves of a workgroup divide the work:
//   OWN_ROWS  each has 16 RT rows of its own; all read the same chunk, of which each loads a tile
//   MERGED    they share 16 RT rows and take every fourth chunk each; their sums meet in LDS
//   MERGED8   the same with eight waves, where no compute unit has more than one workgroup
//   ALONE     each has a piece of the line of chunks for itself
// All but OWN_ROWS have a part of each stage for every wave.
enum KvMode { OWN_ROWS = 0, MERGED = 1, ALONE = 2, MERGED8 = 3 };
constexpr int waves_of(int mode) { return mode == MERGED8 ? 2 * kWaves : kWaves; }

template <int D, int RT>
struct KvShared {
  static constexpr int QP = D + 4;           // floats of a row
  static_assert(16 * QP * 4 <= KvStage<D>::BYTES, "a wave's sums of 16 rows must fit its part of a stage");
  static_assert(RT <= kWaves, "the queries' rows must fit a stage");
  int8_t *st0, *st1;                         // the stages
  float (*wave_m)[16 * RT], (*wave_l)[16 * RT];
};

// Chunks [begin, end) of a tile's; part < 0: these are all of them and the rows are finished, else their sums
// go to that part of the workspace.
template <int D, int RT, int QN, int PN, int MODE>
__device__ __forceinline__ void attend(const KvAttnArgs& g, const KvTile& tile, int begin, int end, int64_t part_at, const KvShared<D, RT>& sh) {
  constexpr int NW = waves_of(MODE);
  constexpr bool MERGE = MODE == MERGED || MODE == MERGED8;
  constexpr int DT = D / 16;                        // 16-wide tiles of the output; elements a lane reads of a token of V
  using Stage = KvStage<D>;
  constexpr int KU = Stage::KU;
  constexpr int QI = D == 64 ? QN / 2 : QN;         // instructions for a tile of scores and KU
  constexpr int QP = KvShared<D, RT>::QP;
  constexpr int ROWS = 16 * RT;
  static_assert(QN % 2 == 0, "");
  int8_t *const st0 = sh.st0, *const st1 = sh.st1;
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));        // what follows from it is formed here, not kept over a workgroup's tiles
  const int lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int r0 = tile.r0 + (MODE == OWN_ROWS ? w * ROWS : 0);     // of this wave
  const KvSequence& s = tile.s;
  const int wg_to = tile.end_token(g);
  KvPages pages(g, tile);

  // One chunk: its loads have landed (and, where the waves share it, everybody's), those of the next go
  // out into the other stage, whose last reads are done.
  constexpr int STEP = MERGE ? NW : 1;
  const int part_of_stage = MODE == OWN_ROWS ? 0 : w * Stage::BYTES;
  int8_t *const s0 = st0 + part_of_stage, *const s1 = st1 + part_of_stage;
  int64_t row[4] = {-1, -1, -1, -1}, next[4] = {-1, -1, -1, -1};
  auto issue = [&](const int64_t (&r)[4], int8_t* to) {
    if (MODE != OWN_ROWS && g.shift >= 6) {
      if (r[0] >= 0) {
        Stage::template load_codes<4>(g.k_codes, r[0], Stage::k_codes(to, 0), lane);
        Stage::template load_codes<4>(g.v_codes, r[0], Stage::v_codes(to, 0), lane);
        Stage::load_scales(g.k_scales, r[0], Stage::k_scales(to), lane);
        Stage::load_scales(g.v_scales, r[0], Stage::v_scales(to), lane);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((MODE != OWN_ROWS || i == w) && r[i] >= 0) {
        Stage::template load_codes<1>(g.k_codes, r[i], Stage::k_codes(to, i), lane);
        Stage::template load_codes<1>(g.v_codes, r[i], Stage::v_codes(to, i), lane);
      }
    }
    if (MODE != OWN_ROWS || w == 0) Stage::load_scales(g.k_scales, r, Stage::k_scales(to), lane);
    if (MODE != OWN_ROWS || w == 1) Stage::load_scales(g.v_scales, r, Stage::v_scales(to), lane);
  };
  int c = begin + (MERGE ? w : 0);
  if (c < end) {       // on their way while the queries are prepared
    pages.chunk(c * kChunk, wg_to, row);
    issue(row, s0);
  }

  // queries: rotated in fp32, split into parts
  v6u qp[RT][KU][QI];
  int qb[RT][KU][(QI + 3) / 4] = {};                        // the parts' scale bytes, four to a dword
  // eight elements a lane, through the second stage to the lanes of the second operand; `count` rows from row
  // `first` of the tile by lanes at, at + step, ..
  auto bring_rows = [&](float* rows, int first, int count, int at, int by) {
    for (int e = at; e < count * D / 8; e += by) {
      const int r = tile.r0 + first + e / (D / 8), i = e % (D / 8);
      float v[8];
      const bool in = r < tile.rows;
      load8_any(g.q, g.q_dt, in ? tile.token(g, r) * g.q_token + tile.q_head(g, r) * g.q_head + 8 * i : 0, in ? 8 : 0, v);
      if (g.rot > 1) rotate_lanes<D>(v, lane);
      float* const to = rows + (e / (D / 8)) * QP + 8 * i;
#pragma unroll
      for (int j = 0; j < 8; ++j) to[j] = v[j] * g.sign;
    }
  };
  if constexpr (MERGE) {
    bring_rows(reinterpret_cast<float*>(st1), 0, ROWS, t, 64 * NW);
    __syncthreads();
  }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    float x[KU][32];
    if constexpr (MODE != OWN_ROWS) {
      if constexpr (MODE == ALONE) {
        bring_rows(reinterpret_cast<float*>(s1), 16 * rt, 16, lane, 64);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");      // the wave's own writes
      }
      const float* const rows = reinterpret_cast<const float*>(MODE == ALONE ? s1 : st1) + ((MODE == ALONE ? 0 : 16 * rt) + lr) * QP +
                                32 * (D == 64 ? lg & 1 : lg);
#pragma unroll
      for (int u = 0; u < KU; ++u)
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const v4f y = *reinterpret_cast<const v4f*>(rows + 128 * u + j);
          x[u][j] = y[0], x[u][j + 1] = y[1], x[u][j + 2] = y[2], x[u][j + 3] = y[3];
        }
    } else {
      const int r = r0 + 16 * rt + lr;
      const bool in = r < tile.rows;
      const int64_t from = in ? tile.token(g, r) * g.q_token + tile.q_head(g, r) * g.q_head : 0;
#pragma unroll
      for (int u = 0; u < KU; ++u)
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          float y[8];
          load8_any(g.q, g.q_dt, from + 128 * u + 32 * (D == 64 ? lg & 1 : lg) + j, in ? 8 : 0, y);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[u][j + e] = y[e] * g.sign;
        }
      if (g.rot > 1) {
#pragma unroll
        for (int u = 0; u < KU; ++u) rotate_row<32, (D == 64 ? 2 : 4)>(x[u], lane);
        if constexpr (KU == 2) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float a = x[0][j], b = x[1][j];
            x[0][j] = a + b;
            x[1][j] = a - b;
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      v6u part[QN];
      int byte[QN];
      split_query<QN>(x[u], part, byte);
#pragma unroll
      for (int i = 0; i < QI; ++i) {
        int by = byte[D == 64 ? 2 * i : i];
        qp[rt][u][i] = part[D == 64 ? 2 * i : i];
        if constexpr (D == 64) {
          const v6u other = part[2 * i + 1];
          const int other_by = byte[2 * i + 1];
          if (lg >= 2) qp[rt][u][i] = other, by = other_by;
        }
        qb[rt][u][i / 4] |= by << (8 * (i % 4));
      }
    }
  }

  // the second stage is free again
  if constexpr (MERGE) __syncthreads();

  // tokens that this lane's rows see: [from, to); and those of all rows, and of any (of the wave: one whose
  // rows lie behind the last sees nothing)
  const int q0 = r0 / g.group, q1 = min(r0 + ROWS - 1, tile.rows - 1) / g.group;
  int from[RT], to[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int r = r0 + 16 * rt + lr;
    from[rt] = tile.start_of(g, r / g.group);
    to[rt] = r < tile.rows ? tile.end_of(r / g.group) : 0;
  }
  const int any_to = r0 < tile.rows ? tile.end_of(q1) : 0, any_from = tile.start_of(g, q0);
  const int all_to = tile.end_of(q0), all_from = tile.start_of(g, q1);

  v4f o[RT][DT];
  float m[RT], base[RT], l[RT];     // maximum (in the scores' own unit) and in powers of two; l: of this lane's tokens
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    m[rt] = -__builtin_inff(), base[rt] = 0.0f, l[rt] = 0.0f;
#pragma unroll
    for (int i = 0; i < DT; ++i) o[rt][i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  }
  uint32_t bad = 0;      // largest scale byte (bits 24 to 31) of V's tokens that not every row sees
  // masked: not every row of the wave sees every token of the chunk.
  auto compute = [&](bool masked, const int8_t* x, const bool (&ok)[4], int t0) {
    // scores of tokens 16 i + 4 r + lg
    float p[RT][4][4];
    v4i kc[4][KU];
    int ks[4][KU];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int u = 0; u < KU; ++u) kc[i][u] = Stage::k(x, i, u, lr, lg), ks[i][u] = Stage::k_scale(x, i, u, lr, lg);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      v4f a[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < KU; ++u)
#pragma unroll
        for (int e = 0; e < QI; ++e) {
          const v6u& y = qp[rt][u][e];
          const v8i qv = {static_cast<int>(y[0]), static_cast<int>(y[1]), static_cast<int>(y[2]), static_cast<int>(y[3]),
                          static_cast<int>(y[4]), static_cast<int>(y[5]), 0, 0};
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] = multiply_part(e, kc[i][u], ks[i][u], qv, qb[rt][u][e / 4], a[i]);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) p[rt][i][r] = a[i][r];
    }
    if (masked) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        // tokens 16 i + 4 r of the chunk from `low` on and below `high`; formed here, where the compiler would
        // compare before the branch
        int low = from[rt] - t0 - lg, high = to[rt] - t0 - lg;
        asm volatile("" : "+v"(low), "+v"(high));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int top_of_tile = ok[i] ? high : 0;
#pragma unroll
          for (int r = 0; r < 4; ++r)
            p[rt][i][r] = 16 * i + 4 * r < top_of_tile && 16 * i + 4 * r >= low ? p[rt][i][r] : -__builtin_inff();
        }
      }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float top = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) top = fmaxf(top, p[rt][i][r]);
      top = fmaxf(m[rt], shfl_fmax(shfl_fmax(top, 16), 32));
      if (__any(top > m[rt])) {
        const float b = top == -__builtin_inff() ? 0.0f : top * g.scale2;
        const float f = m[rt] == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(base[rt] - b);
        l[rt] *= f;
#pragma unroll
        for (int i = 0; i < DT; ++i) o[rt][i] *= f;
        m[rt] = top;
        base[rt] = b;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(p[rt][i][r], g.scale2, -base[rt]));   // 0 if masked
          p[rt][i][r] = e;
          l[rt] += e;
        }
    }

    // Where not every row sees every token: what lies in LDS for a token that no row sees may be
    // anything (times a large scale infinite, and 0 times that is NaN), so its scale becomes a small one.
    // A scale that is not a number, or of 2^126 and more (4 times it is past bf16), must not reach the rows
    // that do not see its token: its values become nothing here, and the rows that see it get them by themselves
    // below.
    // O^T += V^T P^T: 32 tokens an instruction, tokens (2 h + j / 4, j % 4) at a lane's element j
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v8b pf[RT][PN];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = p[rt][2 * h + j / 4][j % 4];
        split8<PN>(y, pf[rt]);
      }
      uint32_t sv[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) Stage::v_scale(x, 2 * h + i, lr, lg, sv[i]);
      if (masked) {
        int low = any_from - t0 - lg, high = any_to - t0 - lg;
        asm volatile("" : "+v"(low), "+v"(high));
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int at = 16 * (2 * h + i) + 4 * r;
            const bool any = ok[2 * h + i] && at < high && at >= low, past = (sv[i][r] << 1) >= 0xFD000000u;
            bad = max(bad, any ? sv[i][r] << 1 : 0u);
            if (past || !any) sv[i][r] = 0u;
          }
      }
      uint32_t y[4][2][Stage::VD];      // of tokens (i, r), (i, r + 1), four such pairs
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) Stage::v(x, 2 * h + c / 2, 2 * (c % 2) + e, lr, lg, y[c][e]);
      // byte by byte: two elements of each token, so two of the output's tiles
      auto two_tiles = [&](auto WORD, auto BYTE) {
        constexpr int wd = decltype(WORD)::value, by = decltype(BYTE)::value, d = 8 * wd + 2 * by;
        v4u v0, v1;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t a = widen2<by>(y[c][0][wd], sv[c / 2][2 * (c % 2)]), b = widen2<by>(y[c][1][wd], sv[c / 2][2 * (c % 2) + 1]);
          v0[c] = __builtin_amdgcn_perm(b, a, 0x05040100u);
          v1[c] = __builtin_amdgcn_perm(b, a, 0x07060302u);
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int e = PN - 1; e >= 0; --e) {
            o[rt][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, v0), pf[rt][e], o[rt][d], 0, 0, 0);
            o[rt][d + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, v1), pf[rt][e], o[rt][d + 1], 0, 0, 0);
          }
      };
      two_tiles(Const<0>{}, Const<0>{});
      two_tiles(Const<0>{}, Const<1>{});
      if constexpr (D > 64) {
        two_tiles(Const<0>{}, Const<2>{});
        two_tiles(Const<0>{}, Const<3>{});
      }
      if constexpr (D > 128) {
        two_tiles(Const<1>{}, Const<0>{});
        two_tiles(Const<1>{}, Const<1>{});
        two_tiles(Const<1>{}, Const<2>{});
        two_tiles(Const<1>{}, Const<3>{});
      }
    }
  };

  // whether not every row of the wave sees every token of a chunk
  auto cut = [&](const int64_t (&r)[4], int t0) {
    return !(r[0] >= 0 && r[1] >= 0 && r[2] >= 0 && r[3] >= 0) || t0 + kChunk > all_to || t0 < all_from;
  };
  auto seen = [&](int t0) { return MODE != OWN_ROWS || (t0 < any_to && t0 + kChunk > any_from); };
  auto step = [&](int c, int8_t* cur, int8_t* other) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    if constexpr (MODE == OWN_ROWS) __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    if (c + STEP < end) {
      pages.chunk((c + STEP) * kChunk, wg_to, next);
      issue(next, other);
    }
    __builtin_amdgcn_sched_barrier(0);
    const int t0 = c * kChunk;
    if (seen(t0)) {
      const bool ok[4] = {row[0] >= 0, row[1] >= 0, row[2] >= 0, row[3] >= 0};
      compute(cut(row, t0), cur, ok, t0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) row[i] = next[i];
  };
  // unrolled over the two stages, each an LDS object of its own: the compiler then waits only
  // for the loads that a read depends on
  for (; c < end; c += 2 * STEP) {
    step(c, s0, s1);
    if (c + STEP < end) step(c + STEP, s1, s0);
  }

  // The values that were left out, token by token from memory: the scores of its tile of 16 once more (token u
  // of it in register u % 4 of the lanes u / 4), and what the token adds to the rows that see it. It stands here,
  // behind the loop, because any more code for such scales in the loop itself spilled registers (prompts of
  // 128 elements took 11 % longer with fp32, so none; with bf16 1 to 3 either way).
  if (__any(bad >= 0xFD000000u)) {
    constexpr int NB = D / 32;
    // copies that the compiler takes for other values: what it would keep for this over the loop is formed here
    const uint8_t *kc = g.k_codes, *vc = g.v_codes, *ks = g.k_scales, *vs = g.v_scales;
    const int32_t* tb = g.table + tile.seq * g.table_ld;
    asm volatile("" : "+s"(kc), "+s"(vc), "+s"(ks), "+s"(vs), "+s"(tb));
    for (int c = begin + (MERGE ? w : 0); c < end; c += STEP) {
      const int t0 = c * kChunk;
      int64_t rows[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        rows[i] = t0 + 16 * i < wg_to
                      ? kv_row_of_token(t0 + 16 * i, tb, g.table_ld, g.pages, g.shift, g.heads, tile.head)
                      : -1;
      if (!seen(t0) || !cut(rows, t0)) continue;
      for (int i = 0; i < 4; ++i) {
        const int64_t tile_row = i < 2 ? (i == 0 ? rows[0] : rows[1]) : (i == 2 ? rows[2] : rows[3]);
        if (tile_row < 0) continue;
        v4f a[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) a[rt] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < KU; ++u) {
          const int block = 4 * u + (D == 64 ? lg & 1 : lg);
          const v4i k = *reinterpret_cast<const v4i*>(kc + (tile_row + lr) * (D / 2) + 16 * block);
          const int scale = ks[(tile_row + lr) * NB + block];
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int e = 0; e < QI; ++e) {
              const v6u& y = qp[rt][u][e];
              const v8i qv = {static_cast<int>(y[0]), static_cast<int>(y[1]), static_cast<int>(y[2]), static_cast<int>(y[3]),
                              static_cast<int>(y[4]), static_cast<int>(y[5]), 0, 0};
              a[rt] = multiply_part(e, k, scale, qv, qb[rt][u][e / 4], a[rt]);
            }
        }
        for (int u = 0; u < 16; ++u) {
          const int at = t0 + 16 * i + u, from_lane = 16 * (u >> 2) + lr;
          const uint8_t* const scales = vs + (tile_row + u) * NB;
          const uint8_t* const codes = vc + (tile_row + u) * (D / 2);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const float s0 = (u & 1) ? a[rt][1] : a[rt][0], s1 = (u & 1) ? a[rt][3] : a[rt][2];
            const float score = __shfl((u & 2) ? s1 : s0, from_lane, 64);
            if (at >= to[rt] || at < from[rt]) continue;
            const float weight = __builtin_amdgcn_exp2f(__builtin_fmaf(score, g.scale2, -base[rt]));
#pragma unroll
            for (int r = 0; r < 4; ++r) {                 // element r of o's tiles lies in block DT (4 lg + r) / 32
              const int first = DT * (4 * lg + r), byte = scales[first / 32];
              if (byte < 253) continue;
#pragma unroll
              for (int d = 0; d < DT; ++d) {
                const uint32_t code = codes[(first + d) / 2] >> (4 * (d & 1));
                const float x = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 0)[0];
                o[rt][d][r] = byte == 255 ? __uint_as_float(0x7FC00000u) : __builtin_fmaf(weight * x, mx_scale(byte), o[rt][d][r]);
              }
            }
          }
        }
      }
    }
  }

#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    l[rt] += __shfl_xor(l[rt], 16, 64);
    l[rt] += __shfl_xor(l[rt], 32, 64);
  }

  if constexpr (!MERGE) {
    // a lane holds D / 4 consecutive elements of a row, from D / 4 lg on
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int row = r0 + 16 * rt + lr;
      const bool in = row < tile.rows;
      if (r0 >= tile.rows) return;                // the whole wave
      float v[D / 4];
      const float inv = part_at >= 0 ? 1.0f : l[rt] == 0.0f ? 0.0f : 1.0f / l[rt] * (g.rot > 1 ? 1.0f / D : 1.0f);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int d = 0; d < DT; ++d) v[DT * r + d] = o[rt][d][r] * inv;
      if (part_at >= 0) {
        const int64_t at = part_at * g.tile_rows + (row - tile.r0);
#pragma unroll
        for (int j = 0; j < D / 4; j += 4)
          *reinterpret_cast<v4f*>(g.part + at * D + D / 4 * lg + j) = v4f{v[j], v[j + 1], v[j + 2], v[j + 3]};
        if (lg == 0) g.stats[2 * at] = m[rt] == -__builtin_inff() ? m[rt] : base[rt], g.stats[2 * at + 1] = l[rt];
        continue;
      }
      if (g.rot > 1) rotate_row<D / 4, 4>(v, lane);
      if (!in) continue;
      const int64_t at = tile.token(g, row) * (g.heads * g.group) + tile.q_head(g, row);
#pragma unroll
      for (int j = 0; j < D / 4; j += 8) {
        const float y[8] = {v[j], v[j + 1], v[j + 2], v[j + 3], v[j + 4], v[j + 5], v[j + 6], v[j + 7]};
        store8_any(g.out, g.out_dt, at * D + D / 4 * lg + j, y);
      }
      if (g.lse && lg == 0) g.lse[at] = l[rt] == 0.0f ? -__builtin_inff() : (base[rt] + __builtin_amdgcn_logf(l[rt])) * kLn2;
    }
  } else {
    // the waves' sums, to a common maximum (in powers of two), 16 rows at a time through the first stage
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
      if (lane < 16) sh.wave_m[w][16 * rt + lr] = m[rt] == -__builtin_inff() ? m[rt] : base[rt], sh.wave_l[w][16 * rt + lr] = l[rt];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      __syncthreads();
      float top = sh.wave_m[0][16 * rt + lr];
#pragma unroll
      for (int i = 1; i < NW; ++i) top = fmaxf(top, sh.wave_m[i][16 * rt + lr]);
      const float f = __builtin_amdgcn_exp2f(sh.wave_m[w][16 * rt + lr] - (top == -__builtin_inff() ? 0.0f : top));
      float* const mine = reinterpret_cast<float*>(s0) + lr * QP;
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int d = 0; d < DT; d += 4)
          *reinterpret_cast<v4f*>(mine + DT * (4 * lg + e) + d) =
              v4f{o[rt][d][e] * f, o[rt][d + 1][e] * f, o[rt][d + 2][e] * f, o[rt][d + 3][e] * f};
      __syncthreads();
      for (int e = t; e < 16 * D / 8; e += 64 * NW) {
        const int r = 16 * rt + e / (D / 8), i = e % (D / 8);
        float big = sh.wave_m[0][r];
#pragma unroll
        for (int k = 1; k < NW; ++k) big = fmaxf(big, sh.wave_m[k][r]);
        const float low = big == -__builtin_inff() ? 0.0f : big;
        float total = 0.0f, v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < NW; ++k) {
          total += sh.wave_l[k][r] * __builtin_amdgcn_exp2f(sh.wave_m[k][r] - low);
          const float* const from_wave = reinterpret_cast<const float*>(st0 + k * Stage::BYTES) + (r - 16 * rt) * QP + 8 * i;
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] += from_wave[j];
        }
        finish_row<D>(g, tile, tile.r0 + r, i, total, low, tile.r0 + r < tile.rows, v);
      }
    }
  }
}

template <int D, int RT, int QN, int PN, int MODE>
__global__ __launch_bounds__(64 * waves_of(MODE), 2) void kv_attention_kernel(KvAttnArgs g) {
  constexpr int NW = waves_of(MODE), PARTS = MODE == OWN_ROWS ? 1 : NW, HELD = MODE == MERGED || MODE == MERGED8 ? NW : 1;
  __shared__ __attribute__((aligned(16))) int8_t st0[PARTS * KvStage<D>::BYTES];
  __shared__ __attribute__((aligned(16))) int8_t st1[PARTS * KvStage<D>::BYTES];
  __shared__ float wave_m[HELD][16 * RT], wave_l[HELD][16 * RT];
  const KvShared<D, RT> sh{st0, st1, wave_m, wave_l};
  if constexpr (MODE != ALONE) {
    // one tile's tokens, or a split of them
    const int split = static_cast<int>(blockIdx.x % g.splits), work = static_cast<int>(blockIdx.x / g.splits);
    const int at = work % g.tiles, sh_at = work / g.tiles;
    const KvTile tile(g, sh_at / g.heads, at, sh_at % g.heads);
    if (tile.r0 >= tile.rows) return;
    const int first = tile.first_chunk(g), chunks = tile.chunks(g), per = (chunks + g.splits - 1) / g.splits;
    attend<D, RT, QN, PN, MODE>(g, tile, first + min(chunks, split * per), first + min(chunks, (split + 1) * per),
                                g.splits > 1 ? static_cast<int64_t>(blockIdx.x) : -1, sh);
  } else {
    const int wave = static_cast<int>(blockIdx.x) * NW + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const KvLine line = kv_line(g, gridDim.x * NW, -1);
    // the same in all lanes: addresses and loops stay scalar
    int at = __builtin_amdgcn_readfirstlane(line.tile);
    if (at < 0) return;
    const int64_t start = wave * line.piece, off = start - line.before;
    const int in_tile = max(tile_chunks(g, at), 1);
    int left = __builtin_amdgcn_readfirstlane(static_cast<int>(min(line.piece, line.total - start)));   // chunks of the piece
    int head = __builtin_amdgcn_readfirstlane(static_cast<int>(off / in_tile));
    int skip = __builtin_amdgcn_readfirstlane(static_cast<int>(off % in_tile));                            // of the tile's, before it
    while (left > 0 && at < g.seqs * g.tiles) {
      const KvTile tile(g, at / g.tiles, at % g.tiles, head);
      const int n = tile.chunks(g), first = tile.first_chunk(g), take = min(left, n - skip);
      // a wave has two parts: of a tile that it goes on with, and of one that it begins
      if (take > 0)
        attend<D, RT, QN, PN, MODE>(g, tile, first + skip, first + skip + take, take == n ? -1 : 2 * static_cast<int64_t>(wave) + (skip == 0), sh);
      left -= take;
      skip = 0;
      if (n == 0 || ++head == g.heads) head = 0, ++at;
    }
  }
}

// The parts of a tile's rows to a common maximum: a wave's lanes hold 512 / D rows, eight elements each;
// the waves take every fourth part, four in flight, and their sums meet in LDS. Parts: first, then second,
// second + stride, .. (count of them).
template <int D>
__device__ inline void join_parts(const KvAttnArgs& g, const KvTile& tile, int row0, int64_t first, int64_t second, int64_t stride, int count) {
  constexpr int U = 4;
  __shared__ float sums[kWaves][64][12];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const int r = row0 + lane / (D / 8), i = lane % (D / 8);
  const bool in = r < g.tile_rows && tile.r0 + r < tile.rows;      // rows behind the last have no parts
  float m = -__builtin_inff(), l = 0.0f, v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  for (int k = w; k < count; k += kWaves * U) {
    float pm[U], pl[U], x[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = k + kWaves * u;
      pm[u] = -__builtin_inff(), pl[u] = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[u][e] = 0.0f;
      if (in && j < count) {
        const int64_t at = (j == 0 ? first : second + (j - 1) * stride) * g.tile_rows + r;
        pm[u] = g.stats[2 * at];
        pl[u] = g.stats[2 * at + 1];
        load8<F32>(g.part, at * D + 8 * i, 8, x[u]);
      }
    }
    float top = m;
#pragma unroll
    for (int u = 0; u < U; ++u) top = fmaxf(top, pm[u]);
    const float base = top == -__builtin_inff() ? 0.0f : top, f = __builtin_amdgcn_exp2f(m - base);
    l *= f;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float h = __builtin_amdgcn_exp2f(pm[u] - base);
      l = __builtin_fmaf(pl[u], h, l);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(x[u][e], h, v[e]);
    }
    m = top;
  }
  float* const mine = sums[w][lane];
#pragma unroll
  for (int e = 0; e < 8; ++e) mine[e] = v[e];
  mine[8] = m;
  mine[9] = l;
  __syncthreads();
  if (w > 0) return;
  float big = sums[0][lane][8];
#pragma unroll
  for (int k = 1; k < kWaves; ++k) big = fmaxf(big, sums[k][lane][8]);
  const float base = big == -__builtin_inff() ? 0.0f : big;
  float total = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.0f;
#pragma unroll
  for (int k = 0; k < kWaves; ++k) {
    const float f = __builtin_amdgcn_exp2f(sums[k][lane][8] - base);
    total = __builtin_fmaf(sums[k][lane][9], f, total);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(sums[k][lane][e], f, v[e]);
  }
  finish_row<D>(g, tile, tile.r0 + r, i, total, base, in, v);
}

// The splits' sums (least = 0), or the parts of a tile that lay in several waves' pieces of the line; and
// the rows that see nothing, which lie in none. `groups` workgroups to a tile.
template <int D>
__global__ __launch_bounds__(64 * kWaves) void kv_join_kernel(KvAttnArgs g, int waves, int groups) {
  const int row0 = static_cast<int>(blockIdx.x % groups) * (512 / D), work = static_cast<int>(blockIdx.x / groups);
  if (g.least == 0) {
    const int at = work % g.tiles, sh_at = work / g.tiles;
    const KvTile tile(g, sh_at / g.heads, at, sh_at % g.heads);
    if (tile.r0 + row0 < tile.rows)
      join_parts<D>(g, tile, row0, static_cast<int64_t>(work) * g.splits, static_cast<int64_t>(work) * g.splits + 1, 1, g.splits);
    return;
  }
  const int at = work / g.heads, head = work % g.heads;
  const KvTile tile(g, at / g.tiles, at % g.tiles, head);
  if (tile.r0 + row0 >= tile.rows) return;
  const KvLine line = kv_line(g, waves, at);
  const int n = tile.chunks(g);
  const int64_t off = line.before + static_cast<int64_t>(head) * n;
  const int64_t w0 = off / line.piece, w1 = (off + max(n, 1) - 1) / line.piece;
  if (n == 0) join_parts<D>(g, tile, row0, 0, 0, 0, 0);
  else if (w0 != w1) join_parts<D>(g, tile, row0, 2 * w0 + 1, 2 * (w0 + 1), 2, static_cast<int>(w1 - w0 + 1));
}

// How a call is cut up. Rows of a sequence and head: up to 64 (32 with 256 elements) a workgroup or wave
// takes 16 of them with all their tokens or a part of them; more: each wave of a workgroup has 32 (16) of
// its own, and the tokens may be split. Measured, in us, sequences of lengths up to L, 8 heads of the
// cache, groups of 4, D = 128, bf16:
//   single tokens; four waves that share the rows, eight (a workgroup to a compute unit), the line (which
//     costs a joining kernel and a walk over the sequences, but fills the chip): 1 sequence, L = 1000 15.5,
//     14.1, 23, 4096 30, 26, 25, 8192 53, 40, 24; 8 sequences, 4096 30, 24, 30, 8192 57, 45, 39; 32, 4096
//     38, 31, 46, 8192 66, 50, 64, 16384 125, 96, 90; 64, 2000 30, 40, 50, 16384 165, -, 165; 128, 8192
//     160, -, 193, 16384 300, -, 306
//   the least piece of the line 2, 4, 8, 16 chunks: 1 sequence, 4096 21, 23, 29, -, 32768 45, 34, 35, 45
//   8 tokens (32 rows); the same three, and own rows: 1 sequence, 1000 14.4, 14.6, 24, 23, 4096 31, 26, 25,
//     25; 8 sequences, 4096 35, 28, 40, 39; 32, 4096 50, 55, 65, 103, 16384 157, 171, 163, 325. Tiles of 32
//     rows for the first three spill registers with fp32 and took, for 8 sequences of 4096, 45, 37, 46, for
//     32 of 16384 169, 131, 142.
//   own rows, split to 256, 512, 1024 workgroups: 500 tokens behind 7500, 171, 140, 154; 4 x 64 tokens of
//     16000, 167, 106, 129
struct KvPlan {
  int mode;
  int tile_rows;
  int64_t tiles;      // of a sequence and head
  int64_t work;       // of the batch
  int splits;
  int least;          // ALONE: chunks of a wave's piece at least
  int64_t grid, parts;
};
static KvPlan kv_plan(const hq_kv_cache& c, const hq_kv_batch& b) {
  KvPlan p = {};
  const int64_t rows = static_cast<int64_t>(b.max_q) * (b.q_heads / c.heads);
  const bool few = rows <= (c.head_dim == 256 ? 32 : 64);
  const int64_t seen = b.window ? std::min<int64_t>(b.max_len, static_cast<int64_t>(b.window) + b.max_q) : b.max_len;
  const int64_t chunks = (seen + kChunk - 1) / kChunk + 1, unwindowed = (static_cast<int64_t>(b.max_len) + kChunk - 1) / kChunk + 1;
  const int64_t fit = 256 * (c.head_dim == 64 ? 3 : c.head_dim == 128 ? 2 : 1);   // workgroups on the chip
  auto shape = [&](int mode) {
    p.mode = mode;
    p.tile_rows = mode != OWN_ROWS ? 16 : 16 * kWaves * (c.head_dim < 256 ? 2 : 1);
    p.tiles = (rows + p.tile_rows - 1) / p.tile_rows;
    p.work = static_cast<int64_t>(b.seqs) * c.heads * p.tiles;
    p.grid = p.work;
    p.splits = 1;
  };
  shape(few ? MERGED : OWN_ROWS);
  if (few && c.head_dim < 256 && p.work <= 256 && chunks > kWaves) shape(MERGED8);
  // (a wave counts its chunks in 32 bits; asked without the window, so that one never brings the line, and a
  // workspace, where none has neither)
  if (few && chunks > (p.mode == MERGED8 ? 52 + 7 * p.work / 10 : 48 + p.work / 4) &&
      p.work * unwindowed < int64_t{1} << 40)
    shape(ALONE);
  if (p.mode == ALONE) {
    p.least = 4;
    const int64_t most = (p.work * chunks + p.least * kWaves - 1) / (p.least * kWaves);
    p.grid = most < fit ? most : fit;
    p.parts = 2 * kWaves * p.grid;
  }
  if (p.mode == OWN_ROWS) {
    const int64_t most = (chunks + 3) / 4;
    int64_t s = p.work > 0 ? 512 / p.work : 1;      // two workgroups to a compute unit
    s = s < most ? s : most;
    p.splits = static_cast<int>(s < 1 ? 1 : s > 256 ? 256 : s);
    p.grid = p.work * p.splits;
    p.parts = p.splits > 1 ? p.grid : 0;
  }
  return p;
}

static size_t part_bytes(const KvPlan& p, int D) { return static_cast<size_t>(p.parts) * p.tile_rows * D * sizeof(float); }

size_t kv_attention_ws(const hq_kv_cache& c, const hq_kv_batch& b) {
  const KvPlan p = kv_plan(c, b);
  if (p.work == 0) return 0;
  return part_bytes(p, c.head_dim) + static_cast<size_t>(p.parts) * p.tile_rows * 2 * sizeof(float);
}

template <int D, int RT, int MODE>
static hipError_t launch_shape(const KvAttnArgs& a, const KvPlan& p, hipStream_t st, int tok) {
  const dim3 grid(static_cast<unsigned>(p.grid)), block(64 * waves_of(MODE));
  if (a.q_dt == DT_F32 || a.out_dt == DT_F32) return launch_k(kv_attention_kernel<D, RT, 6, 3, MODE>, grid, block, st, tok, a);
  return launch_k(kv_attention_kernel<D, RT, 4, 2, MODE>, grid, block, st, tok, a);
}

template <int D>
static hipError_t launch_mode(const KvAttnArgs& a, const KvPlan& p, hipStream_t st, int tok) {
  if (p.mode == OWN_ROWS) return launch_shape<D, D < 256 ? 2 : 1, OWN_ROWS>(a, p, st, tok);
  if (p.mode == ALONE) return launch_shape<D, 1, ALONE>(a, p, st, tok);
  if constexpr (D < 256) {
    if (p.mode == MERGED8) return launch_shape<D, 1, MERGED8>(a, p, st, tok);
  }
  return launch_shape<D, 1, MERGED>(a, p, st, tok);
}

template <int D>
static hipError_t launch_dim(const KvAttnArgs& a, const KvPlan& p, hipStream_t st, int tok) {
  const hipError_t e = launch_mode<D>(a, p, st, tok);
  if (e != hipSuccess || p.parts == 0) return e;
  const int groups = (p.tile_rows * D + 511) / 512;
  return launch_k(kv_join_kernel<D>, dim3(static_cast<unsigned>(p.work * groups)), dim3(64 * kWaves), st,
                  prof_open(K_MISC, static_cast<double>(part_bytes(p, D))), a, static_cast<int>(p.grid) * kWaves, groups);
}

hipError_t kv_attention_pass(const KvAttentionPass& p, hipStream_t st) {
  const hq_kv_cache& c = p.cache;
  const hq_kv_batch& b = p.batch;
  const KvPlan plan = kv_plan(c, b);
  if (plan.work == 0) return hipSuccess;
  if (plan.parts > 0 && !p.ws) return hipErrorInvalidValue;
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
  // a scale of 0 as a tiny one: a score of -infinity (a token that a row does not see) stays one
  const double scale2 = __builtin_fabs(static_cast<double>(b.scale)) * 1.4426950408889634 / c.rot;
  a.scale2 = static_cast<float>(scale2 < 1e-37 ? 1e-37 : scale2);
  a.sign = b.scale < 0.0f ? -1.0f : 1.0f;
  a.out = p.out;
  a.out_dt = p.out_dt;
  a.lse = p.lse;
  a.tiles = static_cast<int>(plan.tiles);
  a.tile_rows = plan.tile_rows;
  a.seqs = b.seqs;
  a.splits = plan.splits;
  a.least = plan.least;
  a.part = static_cast<float*>(p.ws);
  if (plan.parts > 0) a.stats = a.part + part_bytes(plan, c.head_dim) / sizeof(float);
  const double units = 4.0 * c.head_dim * b.q_heads * static_cast<double>(p.tokens) * b.max_len;
  const int tok = prof_open(K_GEMM, units);
  switch (c.head_dim) {
    case 64: return launch_dim<64>(a, plan, st, tok);
    case 128: return launch_dim<128>(a, plan, st, tok);
    case 256: return launch_dim<256>(a, plan, st, tok);
  }
  return hipErrorInvalidValue;
}

}  // namespace hq
