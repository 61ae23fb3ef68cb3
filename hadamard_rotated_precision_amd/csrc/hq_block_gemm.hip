// hq_block_gemm.hip — product of block-scaled FP8 matrices on the matrix cores:
//   c[m][n] (+)= sum_kb sa(m,kb) sb(n,kb) sum_{k in kb} a[m][k] b[n][k],  kb = blocks of 128.
//
// One v_mfma_f32_16x16x128_f8f6f4 multiplies a whole block of K, so a block's products come out of
// fresh accumulators and meet their scales in one fp32 fma per value, beside the next instruction;
// power-of-two scales go into the instruction itself (its scale operands are the exponents).
// P is the operand along the accumulator's registers (b: output columns, four consecutive ones per
// lane), Q the one along the lanes (a: output rows): a tile-scaled P then has one scale for a whole
// wave, and Q's is one number per lane.
//
// Precision. Products of E4M3 codes are exact. The FP8 instruction cuts every product of a group of
// eight, towards zero, 13 bits below the largest 2^(ea + eb) of the group (e: a code's exponent;
// measured on sums whose large products cancel: equal to this rule to the last bit). Computed by
// it, the error is 2e-5 of the results' root mean square on normal data, 7e-5 to 9e-5 with outlier
// columns of 50 times or heavy-tailed gradients, 1.1e-4 with columns of 1000 times: up to half of an
// fp16 output's own rounding (2e-4) and a fifteenth of a bf16 one's (1.7e-3), so 16-bit outputs
// take it. fp32 outputs take v_mfma_f32_16x16x32_f16 on the codes' fp16 values (E4M3 is a subset),
// whose sums are fp32's, at half the rate and the cost of widening the codes. Scales, their products
// and the sums over blocks are fp32 throughout; the output is rounded once.
//
// What bounds it: power and the matrix pipe. Back to back, 8192 x 5120 x 13824 takes 480 to 500 us
// by the card (2.3 to 2.4 PFLOP/s) at a shader clock of 1.83 GHz, the pipe busy two thirds of the
// time that a workgroup is resident; 8192^3 runs at 2.55 PFLOP/s with fp32 scales and 2.75 with
// powers of two (a library FP8 product without block scales: 2.9). A scale for each row of both
// operands (the weight gradient) doubles the vector work to eight instructions per matrix
// instruction: 590 us, 1.96 PFLOP/s, at 5120 x 13824 x 8192. There the matrix pipe is busy for 45 %
// of the launch and the vector pipe for at most 55 % (137 instructions of four cycles in 1000), with
// a sixth of the slots of its five rounds of workgroups empty: neither pipe is full, the two waves
// of a SIMD mostly take turns with it. fp32 outputs: 1.1 PFLOP/s at 4096^3. From registers alone the
// matrix pipe hides four vector instructions behind each of its own (33 of 32 cycles), and of eight
// what does not wait for one another.
// Tried and slower or equal: 32 x 32 x 64 instructions (8192^3, powers of two: 416 us against 400),
// waves of 128 x 128 with accumulators in AGPRs (spills), fragments two rows ahead, double-buffered
// fragments and four stages for the small tiles, a tail of half tiles for a partly filled last
// round (5 % alone, nothing within a training step: the clock rises when units idle).
#include "hq_device.hpp"
#include "hq_launch.hpp"
#include "hq_train_device.hpp"
#include "hq_train_internal.hpp"

namespace hq {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int kFar = 0x7FFFFFF0;   // an offset past any descriptor: the load reads 0

struct BlockGemmArgs {
  BlockOperand p, q;       // b and a
  int64_t M, N, K;         // q rows, p rows, contraction
  void* c;
  int accumulate;
  int k_blocks;            // blocks of K per split (grid.y): all of them for one
  float* part;             // several splits: their sums, M x N each, joined by join_kernel
};

// ------------------------------------------------------------------ tiled kernel
// How the scales come in:
//   S_TILES: p's scale is one number per wave and K step (a wave's P rows lie inside one 128-row
//            block), q's one per lane: f = sp sq, then acc = t f + acc, one fma per value;
//   S_ROWS:  p has a scale for each row: acc = t (sp sq) + acc, a multiplication and an fma;
//   S_POW2:  both are powers of two: the instruction takes their exponents and adds to acc itself.
enum ScaleMode { S_TILES = 0, S_ROWS = 1, S_POW2 = 2 };

// LDS rows of 128 bytes (one block of K); the 16-byte chunk index is XORed with (row / 2) % 8, so
// the 128-bit reads of 16 consecutive rows at one chunk meet 16 different bank groups.
__device__ inline int lds_at(int row, int chunk) { return row * 128 + ((chunk ^ ((row >> 1) & 7)) << 4); }

__device__ inline v8i join(v4i a, v4i b) { return v8i{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}; }

// y[r] = f times x of lane k + r of each 16 (k a constant once loops are unrolled): the
// multiplications read the other lane themselves, where the builtin's moves would be instructions
// of their own. The two wait states are those between a vector write of x and such a read.
__device__ __forceinline__ void times_lanes16(float x, int k, float f, float (&y)[4]) {
  asm("s_nop 1\n\t"
      "v_mul_f32_dpp %0, %4, %5 row_newbcast:%6 row_mask:0xf bank_mask:0xf\n\t"
      "v_mul_f32_dpp %1, %4, %5 row_newbcast:%7 row_mask:0xf bank_mask:0xf\n\t"
      "v_mul_f32_dpp %2, %4, %5 row_newbcast:%8 row_mask:0xf bank_mask:0xf\n\t"
      "v_mul_f32_dpp %3, %4, %5 row_newbcast:%9 row_mask:0xf bank_mask:0xf"
      : "=&v"(y[0]), "=&v"(y[1]), "=&v"(y[2]), "=&v"(y[3])
      : "v"(x), "v"(f), "i"(k), "i"(k + 1), "i"(k + 2), "i"(k + 3));
}

// One dword per lane straight into LDS (lane l at lds + 4 l).
__device__ inline void lds_dma4(__amdgpu_buffer_rsrc_t rs, float* lds, int voffset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)lds, 4, voffset, 0, 0, 0);
}

// A workgroup of NWP x NWQ waves (times KS groups over K) computes (16 TP NWP) x (16 TQ NWQ)
// outputs, a wave 16 TP x 16 TQ of them. The large tile is 256 x 256 from eight waves of 128 x 64:
// two waves per SIMD whose 128 fp32 accumulators each stay in vector registers, where the scaling
// fma's can reach them.
template <class Out, int MODE, bool EXACT, int NWP, int NWQ, int TP, int TQ, int HOLD, int KS>
__global__ __launch_bounds__(64 * NWP * NWQ * KS, 2) void block_gemm_kernel(BlockGemmArgs g) {
  constexpr int NW = NWP * NWQ;
  constexpr int BP = NWP * TP * 16, BQ = NWQ * TQ * 16;    // workgroup tile
  constexpr int P_BYTES = BP * 128, Q_BYTES = BQ * 128;
  constexpr int STAGE = P_BYTES + Q_BYTES + (BP + BQ) * 4;
  constexpr int PL = BP / 8 / NW, QL = BQ / 8 / NW;        // 1 KB direct-to-LDS loads per wave
  constexpr int SL = (BP + BQ) / 64;                       // 64-row scale loads of the workgroup
  static_assert(BP % (8 * NW) == 0 && BQ % (8 * NW) == 0 && SL <= NW && BP % 64 == 0 && BQ % 64 == 0, "");
  static_assert(HOLD < TP && HOLD <= TQ, "");
  static_assert(!EXACT || MODE != S_POW2, "the fp16 instruction takes no scales");
  __shared__ __attribute__((aligned(16))) int8_t st0[KS * STAGE];
  __shared__ __attribute__((aligned(16))) int8_t st1[KS * STAGE];

  // XCD-contiguous order: workgroup b runs on XCD b % 8; each XCD gets consecutive tiles, in
  // groups of 8 q tiles that share p rows in its L2
  const int tiles_q = static_cast<int>((g.M + BQ - 1) / BQ), tiles_p = static_cast<int>((g.N + BP - 1) / BP);
  const int ntiles = tiles_q * tiles_p;
  const int xcd = blockIdx.x & 7, q8 = ntiles >> 3, r8 = ntiles & 7;
  const int pid = xcd * q8 + min(xcd, r8) + (blockIdx.x >> 3);
  constexpr int kGroup = 8;
  const int group = pid / (kGroup * tiles_p), first = group * kGroup;
  const int gsize = min(tiles_q - first, kGroup);
  const int tq = first + (pid % (kGroup * tiles_p)) % gsize;
  const int tp = (pid % (kGroup * tiles_p)) / gsize;
  const int64_t p0 = static_cast<int64_t>(tp) * BP, q0 = static_cast<int64_t>(tq) * BQ;

  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  // KS > 1: groups of waves take every KS-th block of K, in a part of each stage of their own
  const int kg = KS > 1 ? wave / NW : 0, w = KS > 1 ? wave % NW : wave;
  const int wp = w / NWQ, wq = w % NWQ, lr = lane & 15, lg = lane >> 4;

  // operand descriptors from the tile's first row: rows past the end read as zero
  const int rows_p = static_cast<int>(min<int64_t>(BP, g.N - p0)), rows_q = static_cast<int>(min<int64_t>(BQ, g.M - q0));
  const int ldp = static_cast<int>(g.p.ld), ldq = static_cast<int>(g.q.ld);
  const __amdgpu_buffer_rsrc_t rsp = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(g.p.codes + p0 * g.p.ld), 0, rows_p * ldp, kBufferFlags);
  const __amdgpu_buffer_rsrc_t rsq = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(g.q.codes + q0 * g.q.ld), 0, rows_q * ldq, kBufferFlags);
  // lane's place in a 1 KB load: 8 rows of 128 bytes; it fetches the chunk its swizzled slot holds
  // (the same for every load: rows advance by multiples of 16)
  const int dr = 8 * w + (lane >> 3), dc = ((lane & 7) ^ ((dr >> 1) & 7)) << 4;
  const int vp = dr * ldp + dc, vq = dr * ldq + dc;
  const int K16 = static_cast<int>((g.K + 15) & ~int64_t{15});
  // this split's blocks of K
  const int k_first = blockIdx.y * g.k_blocks, KT = min(static_cast<int>((g.K + 127) / 128), k_first + g.k_blocks);

  // scales: each wave fetches those of 64 rows (q's first) for each K step; with more waves than
  // such pieces some are fetched twice, to the same place
  const int ws = w % SL;
  const bool s_is_q = ws < BQ / 64;
  const BlockOperand& so = s_is_q ? g.q : g.p;
  const int64_t s_row0 = s_is_q ? q0 + 64 * ws : p0 + 64 * (ws - BQ / 64);
  const int64_t s_rows = s_is_q ? g.M : g.N;
  const int64_t s_first = so.tiles ? s_row0 >> 7 : s_row0;                      // group of the first row
  const int64_t s_last = so.tiles ? (s_rows - 1) >> 7 : s_rows - 1;             // of the last valid row
  const int s_voff = so.tiles ? 0 : lane * 4;
  const bool s_in = (so.tiles ? s_row0 + lane < s_rows : s_first + lane <= s_last);
  const float* s_base = so.scales + s_first * so.sg;

  // one of the PL + QL + 1 loads that a wave makes of a stage; bp, bq: its offsets at this K step
  auto load_piece = [&](int kt, int8_t* stg, int l, unsigned bp, unsigned bq) {
    if (l == 0) {
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<float*>(s_base + static_cast<int64_t>(min(kt, KT - 1)) * so.sk), 0, 256, kBufferFlags);
      lds_dma4(rs, reinterpret_cast<float*>(stg + P_BYTES + Q_BYTES) + 64 * ws, s_in ? s_voff : kFar);
    } else if (l <= QL) {
      lds_dma16(rsq, stg + P_BYTES + (w + NW * (l - 1)) * 1024, bq + (l - 1) * NW * 8 * ldq);
    } else {
      lds_dma16(rsp, stg + (w + NW * (l - 1 - QL)) * 1024, bp + (l - 1 - QL) * NW * 8 * ldp);
    }
  };
  auto dma = [&](int step, int8_t* stg) {
    const int kt = k_first + step * KS + kg, k0 = kt * 128;
    const bool in = kt < KT && k0 + dc < K16;
    const unsigned bp = in ? vp + k0 : kFar, bq = in ? vq + k0 : kFar;
#pragma unroll
    for (int l = 0; l < PL + QL + 1; ++l) load_piece(kt, stg, l, bp, bq);
  };
  // fragments of v_mfma_f32_16x16x128_f8f6f4: lane group lg holds 32 of the 128 K bytes of row lr;
  // chunks lg and lg + 4, the same for both operands, so products pair equal K whatever the
  // instruction's own order of bytes
  auto frag = [&](const int8_t* base, int row) {
    return join(*reinterpret_cast<const v4i*>(base + lds_at(row, lg)),
                *reinterpret_cast<const v4i*>(base + lds_at(row, lg + 4)));
  };
  auto q_frag = [&](const int8_t* stg, int j) { return frag(stg + P_BYTES, wq * TQ * 16 + j * 16 + lr); };
  auto q_scale = [&](const int8_t* stg, int j) {
    return reinterpret_cast<const float*>(stg + P_BYTES + Q_BYTES)[wq * TQ * 16 + j * 16 + lr];
  };
  auto p_scales = [&](const int8_t* stg) { return reinterpret_cast<const float*>(stg + P_BYTES + Q_BYTES) + BQ + wp * TP * 16; };

  v4f acc[TP][TQ];
#pragma unroll
  for (int i = 0; i < TP; ++i)
#pragma unroll
    for (int j = 0; j < TQ; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  // One K step is TP TQ slots, one instruction of 16 x 16 x 128 each, in a fixed order that keeps
  // the matrix pipe fed: the fma's of a slot follow LAG slots later, when its result is there.
  // First the rows of tiles 0 .. TP-HOLD-1, reading the fragments of the rows to come; then the
  // barrier, when every wave's loads of the next stage have landed and its reads of this one are
  // done; then the HOLD last rows from registers, column by column of tiles: a column's q fragment
  // is read for the next step as soon as it is free, and the loads of the step after the next go
  // into this stage's buffer. So nothing of the next step is waited for right after the barrier.
  constexpr int N = TP * TQ;
  constexpr int LAG = MODE == S_TILES && N > 8 ? 3 : 2;
  constexpr int FRONT = (TP - HOLD) * TQ, NDMA = PL + QL + 1;
  v8i qf[TQ], pf[TP];
  v8h qh[TQ][EXACT ? 4 : 1], ph[TP][EXACT ? 4 : 1];   // EXACT: the codes' values as fp16
  float f[TQ], fn[TQ], spn = 0.0f;    // S_TILES: sp sq of this step and what the next needs; S_ROWS: sq
  int qe[TQ];                         // S_POW2: exponent bytes
  // S_ROWS: lane 16 lg + x has p's scale of row 16 (4 h + x / 4) + 4 lg + x % 4 in sp[h], so the
  // four of tile i that its 16 lanes need are those of lanes 4 (i % 4) + r in sp[i / 4]: two
  // registers and small reads instead of four registers a tile and a 16-byte read each (the same
  // product: 583 against 574 us)
  constexpr int SH = (TP + 3) / 4;
  float sp[SH], spr[SH];
  int pe[TP];
  auto read_p = [&](const int8_t* stg, int i) {
    pf[i] = frag(stg, wp * TP * 16 + i * 16 + lr);
    if constexpr (MODE == S_POW2) pe[i] = __float_as_int(p_scales(stg)[i * 16 + lr]);
  };
  auto read_scales = [&](const int8_t* stg) {
#pragma unroll
    for (int j = 0; j < TQ; ++j) fn[j] = q_scale(stg, j);
    if constexpr (MODE == S_TILES) spn = p_scales(stg)[0];
    if constexpr (MODE == S_ROWS) {
#pragma unroll
      for (int h = 0; h < SH; ++h) spr[h] = p_scales(stg)[(4 * h + (lr >> 2)) % TP * 16 + 4 * lg + (lr & 3)];
    }
  };
  auto halves = [&](const v8i& x, v8h (&h)[EXACT ? 4 : 1]) {
#pragma unroll
    for (int e = 0; e < (EXACT ? 4 : 1); ++e) h[e] = f8_to_h8(x[2 * e], x[2 * e + 1]);
  };
  auto take_scales = [&]() {
    if constexpr (MODE == S_ROWS) {
#pragma unroll
      for (int h = 0; h < SH; ++h) sp[h] = spr[h];
    }
#pragma unroll
    for (int j = 0; j < TQ; ++j) {
      if constexpr (MODE == S_POW2) qe[j] = __float_as_int(fn[j]) >> 23;
      else f[j] = MODE == S_TILES ? fn[j] * spn : fn[j];
      if constexpr (EXACT) halves(qf[j], qh[j]);
    }
  };
  auto slot_i = [](int n) { return n < FRONT ? n / TQ : TP - HOLD + (n - FRONT) % HOLD; };
  auto slot_j = [](int n) { return n < FRONT ? n % TQ : (n - FRONT) / HOLD; };
  auto step = [&](int kt, int8_t* cur_, int8_t* nxt_) {
    int8_t *const cur = cur_ + kg * STAGE, *const nxt = nxt_ + kg * STAGE;
    v4f u[N];
    auto finish = [&](int n) {
      if constexpr (MODE != S_POW2) {
        const int i = slot_i(n), j = slot_j(n);
        // the four products before the four fma's: each fma right behind its own product waits for
        // it (5120 x 13824 x 8192: 602 against 583 us)
        float s[4] = {f[j], f[j], f[j], f[j]};
        if constexpr (MODE == S_ROWS) {
          times_lanes16(sp[i / 4], 4 * (i % 4), f[j], s);
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(u[n][r], s[r], acc[i][j][r]);
      }
    };
    const int ktn = k_first + (kt + 2) * KS + kg, k0 = ktn * 128;
    const bool in = ktn < KT && k0 + dc < K16;
    const unsigned bp = in ? vp + k0 : kFar, bq = in ? vq + k0 : kFar;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int i = slot_i(n), j = slot_j(n);
      if (n == FRONT) {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (EXACT) {
        if (n < FRONT ? j == 0 : n < FRONT + HOLD) halves(pf[i], ph[i]);
        u[n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < 4; ++e) u[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ph[i][e], qh[j][e], u[n], 0, 0, 0);
      } else if constexpr (MODE == S_POW2) {
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(pf[i], qf[j], acc[i][j], 0, 0, 0, pe[i] >> 23, 0, qe[j]);
      } else {
        const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
        u[n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(pf[i], qf[j], zero, 0, 0, 0, 0, 0, 0);
      }
      if (n >= LAG) finish(n - LAG);
      if (n < FRONT) {
        // the next row's fragment, and in the last of the front's rows those of the held rows
        if (n % TQ == 0) read_p(cur, n / TQ + 1);
        if (n >= FRONT - TQ && n % TQ > 0 && n % TQ < HOLD) read_p(cur, TP - HOLD + n % TQ);
      } else {
        const int s = n - FRONT;
        constexpr int PER = (NDMA + N - FRONT - 1) / (N - FRONT);
#pragma unroll
        for (int l = s * PER; l < (s + 1) * PER && l < NDMA; ++l) load_piece(ktn, cur, l, bp, bq);
        if (s == 0) read_p(nxt, 0);
        if (s == 1) read_scales(nxt);
        if ((s + 1) % HOLD == 0) qf[j] = q_frag(nxt, j);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int n = N - LAG; n < N; ++n) finish(n);
    take_scales();
  };

  const int steps = (KT - k_first + KS - 1) / KS;
  if (steps > 0) {
    int8_t* const first = st0 + kg * STAGE;
    dma(0, first);
    dma(1, st1 + kg * STAGE);
    // the loads of stage 0 have landed: those of stage 1 stay in flight
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(NDMA) : "memory");
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int j = 0; j < TQ; ++j) qf[j] = q_frag(first, j);
    read_p(first, 0);
    read_scales(first);
    take_scales();
    // unrolled over the two stages, each an LDS object of its own: the compiler then waits only
    // for the loads that a read depends on
    int kt = 0;
    for (; kt + 1 < steps; kt += 2) {
      step(kt, st0, st1);
      step(kt + 1, st1, st0);
    }
    if (kt < steps) step(kt, st0, st1);
  }
  // loads past K (zeros) have landed before the stages are used again
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __syncthreads();

  // the groups' sums, added in their order by the first
  if constexpr (KS > 1) {
    static_assert((KS - 1) * NW * TP * TQ * 1024 <= 2 * KS * STAGE, "");
    auto at = [&](int group, int i, int j) {
      const int o = (((group - 1) * NW + w) * TP * TQ + i * TQ + j) * 1024 + lane * 16;
      return reinterpret_cast<v4f*>(o < KS * STAGE / 1024 * 1024 ? st0 + o : st1 + o - KS * STAGE / 1024 * 1024);
    };
#pragma unroll
    for (int i = 0; i < TP; ++i)
#pragma unroll
      for (int j = 0; j < TQ; ++j)
        if (kg > 0) *at(kg, i, j) = acc[i][j];
    __syncthreads();
    if (kg == 0) {
#pragma unroll
      for (int e = 1; e < KS; ++e)
#pragma unroll
        for (int i = 0; i < TP; ++i)
#pragma unroll
          for (int j = 0; j < TQ; ++j) acc[i][j] += *at(e, i, j);
    }
    __syncthreads();
    if (kg > 0) return;
  }

  // Epilogue, a wave alone: a strip of 16 output rows goes through the wave's part of a stage, so
  // that lanes hold eight consecutive outputs of a row and neighbouring lanes continue it.
  constexpr int W = TP * 16, PITCH = W + 4;
  static_assert(16 * PITCH * 4 * ((NW + 1) / 2) <= KS * STAGE, "the strips of half the waves must fit a stage");
  float* const strip = reinterpret_cast<float*>((w & 1) ? st1 : st0) + (w >> 1) * 16 * PITCH;
  constexpr int LPR = W / 8, RPI = 64 / LPR;     // lanes per output row, rows per pass
#pragma unroll
  for (int j = 0; j < TQ; ++j) {
#pragma unroll
    for (int i = 0; i < TP; ++i) *reinterpret_cast<v4f*>(strip + lr * PITCH + i * 16 + 4 * lg) = acc[i][j];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int h = 0; h < 16 / RPI; ++h) {
      const int sr = h * RPI + lane / LPR, sc = 8 * (lane % LPR);
      const v4f a = *reinterpret_cast<const v4f*>(strip + sr * PITCH + sc);
      const v4f b = *reinterpret_cast<const v4f*>(strip + sr * PITCH + sc + 4);
      float u[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      const int64_t m = q0 + wq * TQ * 16 + j * 16 + sr, n = p0 + wp * W + sc;
      if (m < g.M && n < g.N) {
        const int64_t off = m * g.N + n;
        if (KS > 1 && g.part) {
          store8<F32>(g.part + blockIdx.y * g.M * g.N, off, g.N - n, u);
          continue;
        }
        if (g.accumulate) {
          float old[8];
          load8<Out>(g.c, off, g.N - n, old);
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] += old[e];
        }
        // past the caches: nothing of the call reads it again, and its lines would displace
        // operands (1000 tokens at 5120 x 13824: 77 -> 70 us; the 8192 training step: -1.5 %)
        store8_stream<Out>(g.c, off, g.N - n, u);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

// c (+)= the splits' sums, added in their order.
template <class Out>
__global__ __launch_bounds__(256) void join_kernel(const float* part, int splits, int64_t n, void* c, int accumulate) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (i >= n) return;
  float sum[8];
  load8<F32>(part, i, n - i, sum);
  for (int s = 1; s < splits; ++s) {
    float x[8];
    load8<F32>(part + s * n, i, n - i, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] += x[e];
  }
  if (accumulate) {
    float old[8];
    load8<Out>(c, i, n - i, old);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] += old[e];
  }
  store8<Out>(c, i, n - i, sum);
}


template <class Out, int MODE, bool EXACT, int NWP, int NWQ, int TP, int TQ, int HOLD, int KS>
static hipError_t launch_tiled(const BlockGemmArgs& a, hipStream_t st, int tok, int splits = 1) {
  constexpr int BP = NWP * TP * 16, BQ = NWQ * TQ * 16;
  const int64_t tiles = ((a.M + BQ - 1) / BQ) * ((a.N + BP - 1) / BP);
  return launch_k(block_gemm_kernel<Out, MODE, EXACT, NWP, NWQ, TP, TQ, HOLD, KS>, dim3(static_cast<unsigned>(tiles), splits),
                  dim3(64 * NWP * NWQ * KS), st, tok, a);
}

// Tile size by the time it would take, in microseconds per 128 of K as measured on whole rounds
// and on ones with fewer workgroups per compute unit (256 x 256: one fits; 128 x 128: two;
// 64 x 64: four). Large tiles read less from LDS and L2 per product, small ones fill the chip when
// the output is small: at K = 4096 (us, tiles of 64 / 128 / 256) 256 x 4096 outputs take
// 11 / 20 / 46, 1000 x 4096 28 / 26 / 48, and 1000 x 13824 at K = 5120 - / 91 / 65.
static int pick_tile(int64_t M, int64_t N, bool exact) {
  constexpr int kCus = 256;
  struct Shape { int size, fit; double us[4]; };
  static const Shape shapes[] = {{256, 1, {1.65}}, {128, 2, {0.75, 1.13}}, {64, 4, {0.32, 0.55, 0.72, 0.9}}};
  int best = 0;
  double best_us = 0.0;
  for (const Shape& s : shapes) {
    if (exact && s.size == 256) continue;   // its fp16 fragments and accumulators do not fit a wave
    const int64_t tiles = ((M + s.size - 1) / s.size) * ((N + s.size - 1) / s.size);
    const int64_t full = tiles / (kCus * s.fit), rest = (tiles % (kCus * s.fit) + kCus - 1) / kCus;
    const double us = static_cast<double>(full) * s.us[s.fit - 1] + (rest ? s.us[rest - 1] : 0.0);
    if (best_us == 0.0 || us < best_us) best = s.size, best_us = us;
  }
  return best;
}

// Splits of K over workgroups where 64 x 64 tiles leave most of the chip idle and K is long. With
// the tiles' two groups of waves a step takes 256 of K: 0.55 us with one workgroup to a compute
// unit, 1.0 with two; joining costs a launch and the splits' sums, written and read in fp32.
static int pick_splits(int64_t M, int64_t N, int64_t K) {
  const int64_t tiles = ((M + 63) / 64) * ((N + 63) / 64), steps = (K + 255) / 256;
  if (tiles > 256 || steps < 2) return 1;
  int best = 1;
  double best_us = 0.0;
  for (int s = 1; s <= 16 && tiles * s <= 512; ++s) {
    const double us = static_cast<double>((steps + s - 1) / s) * (tiles * s <= 256 ? 0.55 : 1.0) +
                      (s > 1 ? 3.0 + static_cast<double>(s) * M * N * 8.0 / 4e6 : 0.0);
    if (s == 1 || us < best_us) best = s, best_us = us;
  }
  // no split without work
  return static_cast<int>((steps + (steps + best - 1) / best - 1) / ((steps + best - 1) / best));
}

template <class Out, int MODE, bool EXACT>
static hipError_t launch_mode(BlockGemmArgs a, hipStream_t st, int tok) {
  a.k_blocks = static_cast<int>((a.K + 127) / 128);
  switch (pick_tile(a.M, a.N, EXACT)) {
    case 64: {
      // two groups of waves over K while no more than two workgroups of eight waves come to a
      // compute unit (64 x 4096, K = 4096: 9.6 against 10.8 us; 300 x 8192, K = 1024, five tiles
      // for two units: 10.4 against 8.8)
      const int64_t tiles = ((a.M + 63) / 64) * ((a.N + 63) / 64);
      if (tiles > 512) return launch_tiled<Out, MODE, EXACT, 2, 2, 2, 2, 1, 1>(a, st, tok);
      const int splits = pick_splits(a.M, a.N, a.K);
      if (splits == 1) {
        a.part = nullptr;
        return launch_tiled<Out, MODE, EXACT, 2, 2, 2, 2, 1, 2>(a, st, tok);
      }
      const int64_t steps = (a.K + 255) / 256;
      a.k_blocks = 2 * static_cast<int>((steps + splits - 1) / splits);
      const hipError_t e = launch_tiled<Out, MODE, EXACT, 2, 2, 2, 2, 1, 2>(a, st, tok, splits);
      if (e != hipSuccess) return e;
      const int64_t n = a.M * a.N;
      return launch_k(join_kernel<Out>, dim3(static_cast<unsigned>((n + 2047) / 2048)), dim3(256), st,
                      prof_open(K_MISC, 4.0 * splits * n), static_cast<const float*>(a.part), splits, n, a.c,
                      a.accumulate);
    }
    case 128: return launch_tiled<Out, MODE, EXACT, 2, 2, 4, 4, 2, 1>(a, st, tok);
    default:
      if constexpr (!EXACT) {
        // rows held over the barrier: more of them lengthen the stretch in which the next loads are
        // issued one by one. Three against two, tile scales, M x N x K outputs and contraction:
        // 8192 x 5120 x 13824 480 / 484 us, 4096 x 11008 x 4096 162 / 164, 4096^3 58.2 / 59.3,
        // 3500 x 4096 x 11008 134 / 135; of ten shapes of a single round of workgroups with their
        // tokens' quantization eight gain up to 2 % and 1792 x 8960 x 2000 loses 1.5 %; of twenty that
        // leave compute units idle seven gain up to 1.6 %, eight are equal and five lose up to 1.7 %
        // (1000 x 13824 x 5120: between -1 and +3 % by the card)
        return launch_tiled<Out, MODE, EXACT, 2, 4, 8, 4, MODE == S_POW2 ? 4 : 3, 1>(a, st, tok);
      }
  }
  return hipErrorInvalidValue;
}

// The splits' sums. The same for every output type: a caller sizes a workspace before it knows.
size_t block_gemm_ws(int64_t M, int64_t N, int64_t K) {
  if (M == 0 || N == 0 || K == 0 || block_gemv_ok(M, N, K) || (pick_tile(M, N, false) != 64 && pick_tile(M, N, true) != 64)) return 0;
  const int splits = pick_splits(M, N, K);
  return splits > 1 ? static_cast<size_t>(splits) * M * N * sizeof(float) : 0;
}

template <class Out>
static hipError_t launch_16bit(const BlockGemmPass& p, const BlockGemmArgs& a, hipStream_t st, int tok) {
  if (p.a.pow2 && p.b.pow2) return launch_mode<Out, S_POW2, false>(a, st, tok);
  if (p.b.tiles) return launch_mode<Out, S_TILES, false>(a, st, tok);
  return launch_mode<Out, S_ROWS, false>(a, st, tok);
}

hipError_t block_gemm_pass(const BlockGemmPass& p, hipStream_t st) {
  if (block_gemv_ok(p.M, p.N, p.K)) return block_gemv_pass(p, nullptr, 0, false, st);
  BlockGemmArgs a{p.b, p.a, p.M, p.N, p.K, p.c, p.accumulate, 0, static_cast<float*>(p.ws)};
  if (block_gemm_ws(p.M, p.N, p.K) > 0 && !p.ws) return hipErrorInvalidValue;
  const int tok = prof_open(K_GEMM, 2.0 * p.M * p.N * p.K);
  switch (p.out_dt) {
    case DT_F32:   // fp32 results: summed by the fp16 instruction
      return p.b.tiles ? launch_mode<F32, S_TILES, true>(a, st, tok) : launch_mode<F32, S_ROWS, true>(a, st, tok);
    case DT_F16: return launch_16bit<F16>(p, a, st, tok);
    case DT_BF16: return launch_16bit<BF16>(p, a, st, tok);
  }
  return hipErrorInvalidValue;
}

}  // namespace hq
