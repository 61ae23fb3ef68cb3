// hq_mx_gemm.hip — product of microscaled 4-bit matrices on the matrix cores:
//   c[m][n] (+)= alpha sum_kb 2^(ea(m,kb) + eb(n,kb)) sum_{k in kb} a[m][k] b[n][k],  kb = blocks of 32.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes a block of 32 codes (16 bytes) and its scale byte from each
// lane: row lane % 16, the block of group lane / 16. It scales and adds by itself, so nothing but the
// loads stands beside it. Products and the sums of a block are exact (multiples of 1/4 below 2^11);
// its sum of 128 products was within 2^-25 of the sum of their magnitudes on random codes and scales.
// P is the operand along the accumulator's registers (b: output columns, four consecutive ones per
// lane), Q the one along the lanes (a: output rows).
//
// What bounds it: no single unit. At 8192^3 (286 us, 3.84 PFLOP/s; 16384^3 4.6) a step of 256 of K takes a
// compute unit about 4900 cycles, in which the matrix pipes are busy for 2050, LDS serves fragments for
// 1540, and 64 KB arrive, 7.5 TB/s over the chip.
#include "hq_device.hpp"
#include "hq_launch.hpp"
#include "hq_mx_device.hpp"
#include "hq_mx_internal.hpp"

namespace hq {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));

constexpr int kFar = 0x7FFFFFF0;   // an offset past any descriptor: the load reads 0

struct MxGemmArgs {
  MxOperand p, q;          // b and a
  int64_t M, N, K;         // q rows, p rows, contraction
  float alpha;
  void* c;
  int accumulate;
  int k_steps;             // steps of 256 of K per split (grid.y): all of them for one
  float* part;             // several splits: their sums, M x N each, joined by mx_join_kernel
};

// LDS rows of 128 bytes (256 of K); the place of a 16-byte chunk is XORed with (row / 2) % 8, so the
// 128-bit reads of 16 lanes served at once, of consecutive rows at one place or of some at the next,
// meet 16 different bank groups (with the chunks in order a sixth of the time went into conflicts:
// 8192^3 292 us, so 286, 3.84 PFLOP/s).
__device__ inline int lds_at(int row, int place) { return row * 128 + ((place ^ ((row >> 1) & 7)) << 4); }

// One dword per lane straight into LDS (lane l at lds + 4 l).
__device__ inline void lds_dma4(__amdgpu_buffer_rsrc_t rs, int8_t* lds, int voffset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)lds, 4, voffset, 0, 0, 0);
}

// The two blocks of a lane in a step: 16 bytes of codes each, and their scale bytes in the two low
// bytes of s.
struct Fragment {
  v4i x[2];
  int s;
};

__device__ inline v8i wide(v4i a) { return v8i{a[0], a[1], a[2], a[3], 0, 0, 0, 0}; }

__device__ inline v4f multiply(const Fragment& p, const Fragment& q, v4f c) {
  c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(p.x[0]), wide(q.x[0]), c, 4, 4, 0, p.s, 0, q.s);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(p.x[1]), wide(q.x[1]), c, 4, 4, 1, p.s, 1, q.s);
}

// A workgroup of NWP x NWQ waves (times KS groups over K) computes (16 TP NWP) x (16 TQ NWQ)
// outputs, a wave 16 TP x 16 TQ of them.
template <class Out, int NWP, int NWQ, int TP, int TQ, int HOLD, int KS>
__global__ __launch_bounds__(64 * NWP * NWQ * KS, 2) void mx_gemm_kernel(MxGemmArgs g) {
  constexpr int NW = NWP * NWQ;
  constexpr int BP = NWP * TP * 16, BQ = NWQ * TQ * 16;    // workgroup tile
  constexpr int P_BYTES = BP * 128, Q_BYTES = BQ * 128;
  constexpr int STAGE = P_BYTES + Q_BYTES + (BP + BQ) * 8;
  constexpr int PL = BP / 8 / NW, QL = BQ / 8 / NW;        // 1 KB direct-to-LDS loads per wave
  constexpr int SL = (BP + BQ) / 32;                       // 32-row scale loads of the workgroup
  constexpr int SLW = (SL + NW - 1) / NW;                  // of a wave (some twice, to the same place)
  static_assert(BP % (8 * NW) == 0 && BQ % (8 * NW) == 0 && BP % 32 == 0 && BQ % 32 == 0, "");
  static_assert(HOLD < TP && HOLD <= TQ, "");
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
  // KS > 1: groups of waves take every KS-th step, in a part of each stage of their own
  const int kg = KS > 1 ? wave / NW : 0, w = KS > 1 ? wave % NW : wave;
  const int wp = w / NWQ, wq = w % NWQ, lr = lane & 15, lg = lane >> 4;

  // operand descriptors from the tile's first row: rows past the end read as zero
  const int rows_p = static_cast<int>(min<int64_t>(BP, g.N - p0)), rows_q = static_cast<int>(min<int64_t>(BQ, g.M - q0));
  const int ldp = static_cast<int>(g.p.ld), ldq = static_cast<int>(g.q.ld);
  const int lsp = static_cast<int>(g.p.lds), lsq = static_cast<int>(g.q.lds);
  const __amdgpu_buffer_rsrc_t rsp = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(g.p.codes + p0 * g.p.ld), 0, rows_p * ldp, kBufferFlags);
  const __amdgpu_buffer_rsrc_t rsq = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(g.q.codes + q0 * g.q.ld), 0, rows_q * ldq, kBufferFlags);
  const __amdgpu_buffer_rsrc_t ssp = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(g.p.scales + p0 * g.p.lds), 0, rows_p * lsp, kBufferFlags);
  const __amdgpu_buffer_rsrc_t ssq = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(g.q.scales + q0 * g.q.lds), 0, rows_q * lsq, kBufferFlags);
  // lane's place in a 1 KB load: 8 rows of 128 bytes; it fetches the chunk its swizzled slot holds
  // (the same for every load: rows advance by multiples of 16). Place i of a row holds chunk 2 i, place
  // 4 + i chunk 2 i + 1.
  const int dr = 8 * w + (lane >> 3), place = (lane & 7) ^ ((dr >> 1) & 7), dc = ((place << 1 | place >> 2) & 7) << 4;
  const int vp = dr * ldp + dc, vq = dr * ldq + dc;
  const int KB = static_cast<int>((g.K + 31) >> 5);        // blocks: 16 bytes and a scale each
  // this split's steps
  const int k_first = blockIdx.y * g.k_steps, KT = min((KB + 7) >> 3, k_first + g.k_steps);

  // one of the SLW + PL + QL loads that a wave makes of a stage
  auto load_piece = [&](int kt, int8_t* stg, int l, unsigned bp, unsigned bq) {
    if (l < SLW) {
      const int piece = (w + NW * l) % SL;                 // q's rows first, 32 of them a piece
      const bool is_q = piece < BQ / 32;
      const int row = (is_q ? 32 * piece : 32 * piece - BQ) + (lane >> 1);
      const int b = 8 * kt + 4 * (lane & 1);               // first of four blocks; rows are padded to 16
      const int off = kt < KT && b < KB ? row * (is_q ? lsq : lsp) + b : kFar;
      if (is_q) lds_dma4(ssq, stg + P_BYTES + Q_BYTES + 256 * piece, off);
      else lds_dma4(ssp, stg + P_BYTES + Q_BYTES + 256 * piece, off);
    } else if (l < SLW + QL) {
      lds_dma16(rsq, stg + P_BYTES + (w + NW * (l - SLW)) * 1024, bq + (l - SLW) * NW * 8 * ldq);
    } else {
      lds_dma16(rsp, stg + (w + NW * (l - SLW - QL)) * 1024, bp + (l - SLW - QL) * NW * 8 * ldp);
    }
  };
  constexpr int NDMA = SLW + PL + QL;
  auto dma = [&](int step, int8_t* stg) {
    const int kt = k_first + step * KS + kg, k0 = kt * 128;
    const bool in = kt < KT && k0 + dc < 16 * KB;
    const unsigned bp = in ? vp + k0 : kFar, bq = in ? vq + k0 : kFar;
#pragma unroll
    for (int l = 0; l < NDMA; ++l) load_piece(kt, stg, l, bp, bq);
  };
  // a lane's blocks are 2 lg and 2 lg + 1 of the step's eight, the same for both operands. The swizzle is
  // that of row lr for every tile of 16 rows, so a lane has two offsets and a tile adds a constant (with
  // an address for each tile the registers ran out and the loop read scratch memory: 8192^3 took 364 us,
  // without 293)
  const int at0 = lds_at(lr, lg), at1 = lds_at(lr, lg + 4), at_s = lr * 8 + 2 * lg;
  auto frag = [&](const int8_t* base, const int8_t* scales, int tile) {
    Fragment f;
    f.x[0] = *reinterpret_cast<const v4i*>(base + at0 + tile * 2048);
    f.x[1] = *reinterpret_cast<const v4i*>(base + at1 + tile * 2048);
    f.s = *reinterpret_cast<const uint16_t*>(scales + at_s + tile * 128);
    return f;
  };
  auto q_frag = [&](const int8_t* stg, int j) {
    return frag(stg + P_BYTES + wq * TQ * 2048, stg + P_BYTES + Q_BYTES + wq * TQ * 128, j);
  };
  auto p_frag = [&](const int8_t* stg, int i) {
    return frag(stg + wp * TP * 2048, stg + P_BYTES + Q_BYTES + BQ * 8 + wp * TP * 128, i);
  };

  v4f acc[TP][TQ];
#pragma unroll
  for (int i = 0; i < TP; ++i)
#pragma unroll
    for (int j = 0; j < TQ; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  // One step is TP TQ slots of two instructions each, in a fixed order that keeps the matrix pipe
  // fed: first the rows of tiles 0 .. TP-HOLD-1, reading the fragments of the rows to come; then
  // the barrier, when every wave's loads of the next stage have landed and its reads of this one are
  // done; then the HOLD last rows from registers, column by column of tiles: a column's q fragment
  // is read for the next step as soon as it is free, and the loads of the step after the next go
  // into this stage's buffer. So nothing of the next step is waited for right after the barrier.
  constexpr int N = TP * TQ;
  constexpr int FRONT = (TP - HOLD) * TQ;
  Fragment qf[TQ], pf[TP];
  auto slot_i = [](int n) { return n < FRONT ? n / TQ : TP - HOLD + (n - FRONT) % HOLD; };
  auto slot_j = [](int n) { return n < FRONT ? n % TQ : (n - FRONT) / HOLD; };
  auto step = [&](int kt, int8_t* cur_, int8_t* nxt_) {
    int8_t *const cur = cur_ + kg * STAGE, *const nxt = nxt_ + kg * STAGE;
    const int ktn = k_first + (kt + 2) * KS + kg, k0 = ktn * 128;
    const bool in = ktn < KT && k0 + dc < 16 * KB;
    const unsigned bp = in ? vp + k0 : kFar, bq = in ? vq + k0 : kFar;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int i = slot_i(n), j = slot_j(n);
      if (n == FRONT) {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
      }
      acc[i][j] = multiply(pf[i], qf[j], acc[i][j]);
      if (n < FRONT) {
        // the next row's fragment, and in the last of the front's rows those of the held rows
        if (n % TQ == 0) pf[n / TQ + 1] = p_frag(cur, n / TQ + 1);
        if (n >= FRONT - TQ && n % TQ > 0 && n % TQ < HOLD) pf[TP - HOLD + n % TQ] = p_frag(cur, TP - HOLD + n % TQ);
      } else {
        const int s = n - FRONT;
        constexpr int PER = (NDMA + N - FRONT - 1) / (N - FRONT);
#pragma unroll
        for (int l = s * PER; l < (s + 1) * PER && l < NDMA; ++l) load_piece(ktn, cur, l, bp, bq);
        if (s == 0) pf[0] = p_frag(nxt, 0);
        if ((s + 1) % HOLD == 0) qf[j] = q_frag(nxt, j);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
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
    pf[0] = p_frag(first, 0);
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
    static_assert((KS - 1) * NW * TP * TQ * 1024 <= 2 * KS * (STAGE / 1024 * 1024), "");
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
      const v4f a = *reinterpret_cast<const v4f*>(strip + sr * PITCH + sc) * g.alpha;
      const v4f b = *reinterpret_cast<const v4f*>(strip + sr * PITCH + sc + 4) * g.alpha;
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
        // past the caches: nothing of the call reads it again
        store8_stream<Out>(g.c, off, g.N - n, u);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

// c (+)= the splits' sums, added in their order.
template <class Out>
__global__ __launch_bounds__(256) void mx_join_kernel(const float* part, int splits, int64_t n, void* c, int accumulate) {
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

template <class Out, int NWP, int NWQ, int TP, int TQ, int HOLD, int KS>
static hipError_t launch_tiled(const MxGemmArgs& a, hipStream_t st, int tok, int splits = 1) {
  constexpr int BP = NWP * TP * 16, BQ = NWQ * TQ * 16;
  const int64_t tiles = ((a.M + BQ - 1) / BQ) * ((a.N + BP - 1) / BP);
  return launch_k(mx_gemm_kernel<Out, NWP, NWQ, TP, TQ, HOLD, KS>, dim3(static_cast<unsigned>(tiles), splits),
                  dim3(64 * NWP * NWQ * KS), st, tok, a);
}

// Tile size by the time it would take, in microseconds per 256 of K on whole rounds and on ones with
// fewer workgroups per compute unit (256 x 256: one fits; 128 x 128: two; 64 x 64: four): the rest's
// from one round as K grows from 8192 to 16384, the whole rounds' from products of several. Tiles of
// 64, 128 and 256 take 13.7, 16.5 and 30 us at 512 x 4096 x 4096, 24, 18 and 31 at 1000 x 4096 x 4096,
// 97, 60 and 42 at 1000 x 13824 x 5120; those of 128 and 256 445 and 294 us at 8192 x 5120 x 13824.
static int pick_tile(int64_t M, int64_t N) {
  constexpr int kCus = 256;
  struct Shape { int size, fit; double us[4]; };
  static const Shape shapes[] = {{256, 1, {2.1}}, {128, 2, {0.8, 1.6}}, {64, 4, {0.45, 0.6, 0.85, 1.4}}};
  int best = 0;
  double best_us = 0.0;
  for (const Shape& s : shapes) {
    const int64_t tiles = ((M + s.size - 1) / s.size) * ((N + s.size - 1) / s.size);
    const int64_t full = tiles / (kCus * s.fit), rest = (tiles % (kCus * s.fit) + kCus - 1) / kCus;
    const double us = static_cast<double>(full) * s.us[s.fit - 1] + (rest ? s.us[rest - 1] : 0.0);
    if (best_us == 0.0 || us < best_us) best = s.size, best_us = us;
  }
  return best;
}

// Splits of K over workgroups where 64 x 64 tiles leave most of the chip idle and K is long. With
// the tiles' two groups of waves a step takes 512 of K: 0.85 us with one workgroup to a compute
// unit, 1.2 with two; joining costs a launch (4 us beside a short product) and the splits' sums,
// written and read in fp32. 1, 2, 4, 8 and 16 splits of 64 x 1024 x 16384 take 26, 17, 12.5, 11.6 and
// 13.2 us, of 64 x 4096 x 4096 9.3, 10.4, 10.9, 13.5 and 21.
static int pick_splits(int64_t M, int64_t N, int64_t K) {
  const int64_t tiles = ((M + 63) / 64) * ((N + 63) / 64), steps = (K + 511) / 512;
  if (tiles > 256 || steps < 2) return 1;
  int best = 1;
  double best_us = 0.0;
  for (int s = 1; s <= 16 && tiles * s <= 512; ++s) {
    const double us = static_cast<double>((steps + s - 1) / s) * (tiles * s <= 256 ? 0.85 : 1.2) +
                      (s > 1 ? 4.0 + static_cast<double>(s) * M * N * 8.0 / 1.5e6 : 0.0);
    if (s == 1 || us < best_us) best = s, best_us = us;
  }
  // no split without work
  return static_cast<int>((steps + (steps + best - 1) / best - 1) / ((steps + best - 1) / best));
}

template <class Out>
static hipError_t launch_out(MxGemmArgs a, hipStream_t st, int tok) {
  a.k_steps = static_cast<int>((a.K + 255) / 256);
  switch (pick_tile(a.M, a.N)) {
    case 64: {
      // two groups of waves over K while no more than two workgroups of eight waves come to a
      // compute unit
      const int64_t tiles = ((a.M + 63) / 64) * ((a.N + 63) / 64);
      if (tiles > 512) return launch_tiled<Out, 2, 2, 2, 2, 1, 1>(a, st, tok);
      const int splits = pick_splits(a.M, a.N, a.K);
      if (splits == 1) {
        a.part = nullptr;
        return launch_tiled<Out, 2, 2, 2, 2, 1, 2>(a, st, tok);
      }
      const int64_t steps = (a.K + 511) / 512;
      a.k_steps = 2 * static_cast<int>((steps + splits - 1) / splits);
      const hipError_t e = launch_tiled<Out, 2, 2, 2, 2, 1, 2>(a, st, tok, splits);
      if (e != hipSuccess) return e;
      const int64_t n = a.M * a.N;
      return launch_k(mx_join_kernel<Out>, dim3(static_cast<unsigned>((n + 2047) / 2048)), dim3(256), st,
                      prof_open(K_MISC, 4.0 * splits * n), static_cast<const float*>(a.part), splits, n, a.c,
                      a.accumulate);
    }
    case 128: return launch_tiled<Out, 2, 2, 4, 4, 2, 1>(a, st, tok);
    default: return launch_tiled<Out, 2, 4, 8, 4, 4, 1>(a, st, tok);
  }
}

// The splits' sums.
size_t mx_gemm_ws(int64_t M, int64_t N, int64_t K) {
  if (M == 0 || N == 0 || K == 0 || mx_gemv_ok(M, N, K) || pick_tile(M, N) != 64) return 0;
  if (((M + 63) / 64) * ((N + 63) / 64) > 512) return 0;
  const int splits = pick_splits(M, N, K);
  return splits > 1 ? static_cast<size_t>(splits) * M * N * sizeof(float) : 0;
}

hipError_t mx_gemm_pass(const MxGemmPass& p, hipStream_t st) {
  if (mx_gemv_ok(p.M, p.N, p.K)) return mx_gemv_pass(p, nullptr, 0, 1, st);
  const MxGemmArgs a{p.b, p.a, p.M, p.N, p.K, p.alpha, p.c, p.accumulate, 0, static_cast<float*>(p.ws)};
  if (mx_gemm_ws(p.M, p.N, p.K) > 0 && !p.ws) return hipErrorInvalidValue;
  const int tok = prof_open(K_GEMM, 2.0 * p.M * p.N * p.K);
  switch (p.out_dt) {
    case DT_F32: return launch_out<F32>(a, st, tok);
    case DT_F16: return launch_out<F16>(a, st, tok);
    case DT_BF16: return launch_out<BF16>(a, st, tok);
  }
  return hipErrorInvalidValue;
}

}  // namespace hq
