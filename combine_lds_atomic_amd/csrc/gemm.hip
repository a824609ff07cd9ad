// Expert products over the expert-major rows that dispatch writes: block-128
// scaled e4m3 activations times block-128x128 scaled e4m3 weights, grouped
// over the experts by exp_off.
//
//   y[i][f] = sum_b x_s[i][b] * w_s[e][f/128][b] * sum_{c in block b} x_q[i][c] * w_q[e][f][c]
//
// with e the expert of row i.  k_grouped_gemm<..., false> rounds y to bf16;
// k_grouped_gemm<..., true> takes features f and I + f as gate and up,
// forms silu(gate) * up and quantises it per 128 features.
#include <type_traits>

#include "gemm_dev.h"
#include "moe_internal.h"
#include "quant_dev.h"

namespace moe {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

struct GemmArgs {
  const uint8_t* x_q;
  const float* x_s;
  const uint8_t* w_q;
  const float* w_s;
  const int* exp_off;
  uint16_t* y;      // plain form: [rows][F]
  uint8_t* a_q;     // SwiGLU form: [rows][F]
  float* a_s;       // SwiGLU form: [rows][F/128]
  int N, L, E, R;   // ranks, experts per rank, experts, fixed region rows (0 = packed)
  int rows;         // rows of the arrays
  int K, F;         // input features, output features
  int bn;           // rows of a tile at most (a multiple of 16, no more than the kernel's BN)
};

// One lane's 32 bytes of a 16-row tile and K step: as they are in LDS, and as
// the operand of a 16x16 product over the step's 128 columns, which is the
// e4m3 bytes themselves (Wide = false) or those widened to bf16 (exactly).
struct Raw {
  v4u lo, hi;
  __device__ __forceinline__ void load(const unsigned char* p, int o0, int o1) {
    lo = *reinterpret_cast<const v4u*>(p + o0);
    hi = *reinterpret_cast<const v4u*>(p + o1);
  }
};
template <bool Wide>
struct Operand;
template <>
struct Operand<false> {
  v8i v;
  __device__ __forceinline__ void load(const unsigned char* p, int o0, int o1) {
    Raw r;
    r.load(p, o0, o1);
    set(r);
  }
  __device__ __forceinline__ void set(const Raw& r) {
    v = __builtin_shufflevector(__builtin_bit_cast(v4i, r.lo), __builtin_bit_cast(v4i, r.hi), 0, 1, 2, 3, 4, 5, 6, 7);
  }
};
template <>
struct Operand<true> {
  v8bf v[4];
  __device__ __forceinline__ void load(const unsigned char* p, int o0, int o1) {
    Raw r;
    r.load(p, o0, o1);
    set(r);
  }
  __device__ __forceinline__ void set(const Raw& r) {
    v[0] = widen8(r.lo[0], r.lo[1]);
    v[1] = widen8(r.lo[2], r.lo[3]);
    v[2] = widen8(r.hi[0], r.hi[1]);
    v[3] = widen8(r.hi[2], r.hi[3]);
  }
};

template <int NT>
__device__ __forceinline__ void multiply(const Operand<false>& a, const Operand<false> (&b)[NT], v4f (&p)[NT]) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
    p[n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b[n].v, v4f{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
}
template <int NT>
__device__ __forceinline__ void multiply(const Operand<true>& a, const Operand<true> (&b)[NT], v4f (&p)[NT]) {
#pragma unroll
  for (int n = 0; n < NT; ++n) p[n] = v4f{0, 0, 0, 0};
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int n = 0; n < NT; ++n) p[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[c], b[n].v[c], p[n], 0, 0, 0);
}

constexpr int kBK = kScaleBlock;   // one K step = one scale block = one 16x16x128 product
constexpr int kXsChunk = 8;        // K steps whose scales are staged together
static_assert(2 * kXsChunk <= kWave, "one lane a weight scale");

// One workgroup forms BM weight rows x up to BN tokens of one expert: WM x WN
// waves, each MT x NT matrix tiles of 16 x 16 with the weights as the left
// operand, so a lane holds four neighbouring features of one token.  A K step
// is one scale block: the step's products start from zero and join the
// float32 sums with one fused multiply-add by x_s * w_s.  S stages of both
// operands sit in LDS, filled by loads that bypass the registers.
//
// Two kinds of products:
//   - plain form: e4m3 matrix instructions.  They add the products of eight
//     consecutive columns on a grid of 2^-13 of the largest one's power of two,
//     towards zero (measured with single products, for both e4m3 forms of the
//     instruction); everything behind that is float32.  That leaves 1.3e-5 of a
//     row's norm on normal data, where y's bf16 rounding leaves 1.7e-3, and
//     what the largest of eight hides from its neighbours is less than the 8-bit
//     rounding of that largest one.  Widened operands, as in the SwiGLU form,
//     are exact and were measured for it: 15.7 ms against 9.9 (2048 rows an
//     expert, K = 2048 -> 7168), 28.6 against 17.4 (7168 -> 4096), 1.32 ms
//     against 1.04 (128 rows), 105 us against 63 (1337 rows of one expert), 102
//     against 99 (5 rows), one run.  So this form keeps the grid.
//   - SwiGLU form: its scales are float32 outputs, on which those 1.3e-5 would
//     be seen, so the bytes are widened to bf16 (exactly) behind LDS and
//     multiplied there, at half the instruction's rate and 1.5 to 2
//     conversions per instruction (2e-7 against 64-bit sums).
//
// What bounds it on MI355X (ranges are over machines and runs).  Plain form,
// 256 x 256, 2048 rows an expert: 9.3 to 10.0 ms for K = 2048 -> 7168 (1.54 to
// 1.66 PFLOP/s), 16.5 to 17.4 ms for 7168 -> 4096 (1.77 to 1.86); a large
// library e4m3 product without block scales reaches 3.06.  No unit is full: the
// matrix pipes are busy 36% of the cycles, LDS 16% (a counter that may leave out
// the loads' writes), and waves wait for 37% of theirs.  A timing copy of an
// earlier step without the loads of the K loop took 7.7 ms against 9.8 (12.3
// against 17.1 for K = 7168), one with a quarter of the scaled additions 9.3.
// Weights loaded straight to registers, prefetches into L2, smaller tiles with a
// third stage, and non-temporal stores of y (11.4 ms) were slower.
// SwiGLU form: 26.3 to 29.0 ms for 2048 rows an expert, K = 7168, I = 2048
// (1.06 to 1.17 PFLOP/s; with 160-row tiles 29.3 where this took 27.0); a large
// library bf16 product reaches 1.5 to 1.6.  A wave's 128 x 64 tile fills the 256
// registers that vector instructions can address, which rules out larger ones;
// the clock falls to 2.2 GHz under it, and the matrix pipes are busy 50% of the
// cycles.  Waves in two groups that convert and multiply in turn were no faster.
template <int BM, int BN, int WM, int WN, int S, int EPL, bool SW>
__global__ __launch_bounds__(WM* WN* kWave) void k_grouped_gemm(GemmArgs A) {
  constexpr int NW = WM * WN, THREADS = NW * kWave;
  constexpr int MT = BM / WM / 16, NT = BN / WN / 16;     // 16x16 tiles of a wave
  constexpr int kRowsPerLoad = kWave / 8;                  // 8 lanes of 16 bytes per row
  constexpr int BNL = (BN + kRowsPerLoad * NW - 1) / (kRowsPerLoad * NW) * (kRowsPerLoad * NW);   // rows loaded
  constexpr int LPS = (BM + BNL) / kRowsPerLoad / NW;      // loads per wave and stage
  static_assert(BM % (kRowsPerLoad * NW) == 0, "rows split evenly over the waves");
  static_assert(!SW || BM == 2 * kScaleBlock, "a gate and an up half of one scale block");
  constexpr int kStage = (BM + BNL) * kBK;
  __shared__ __align__(1024) unsigned char lds[S * kStage];
  constexpr int XG = (BN + kWave - 1) / kWave, XI = kXsChunk * XG / NW;   // scale loads of a chunk, and of a wave
  static_assert(kXsChunk * XG % NW == 0, "scale loads split evenly over the waves");
  __shared__ float sx[2][kXsChunk][XG * kWave];
  __shared__ float sw[2][kWave];   // [block][K step of the chunk], 16 of the 64

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN;

  constexpr int BF = SW ? BM / 2 : BM;      // output features of a tile
  const Tile T = find_tile<EPL>(A, (A.F + BF - 1) / BF);
  if (T.n <= 0) return;
  const int ft = T.f;

  const int KB = A.K / kBK;
  const int wrows = SW ? 2 * A.F : A.F;     // weight rows of an expert
  const uint8_t* wbase = A.w_q + (int64_t)T.e * wrows * A.K;
  const uint8_t* xbase = A.x_q + (int64_t)T.row * A.K;

  // ---- this lane's source of each of its loads: LDS row R (weights first,
  // then tokens), 16-byte position p of the row holds chunk p ^ (R & 7), so
  // that the 8 lanes of a ds_read_b128 phase hit 8 different bank groups.
  constexpr int kWLoads = BM / kRowsPerLoad / NW, kStep = NW * kRowsPerLoad;
  const uint32_t r0 = wave * kRowsPerLoad + (lane >> 3), c0 = ((lane & 7) ^ (r0 & 7)) * 16;
  // Offsets of the weight loads: one for all where rows are whole blocks,
  // else each with its row held below F (F * K <= 2^30).
  uint32_t woff[SW ? 1 : kWLoads];
  if constexpr (SW) {
    woff[0] = r0 * (uint32_t)A.K + c0;
  } else {
#pragma unroll
    for (int i = 0; i < kWLoads; ++i) woff[i] = min(ft * BF + r0 + i * kStep, (uint32_t)A.F - 1u) * (uint32_t)A.K + c0;
  }
  // Loads [i0, i1) of step kb.
  auto issue = [&](int kb, int i0, int i1) {
    unsigned char* dst = lds + (kb % S) * kStage + wave * 1024;
#pragma unroll
    for (int i = 0; i < LPS; ++i) {
      if (i < i0 || i >= i1) continue;
      if (i < kWLoads) {
        const int64_t row = !SW ? 0 : ft * BF + (i < kWLoads / 2 ? i * kStep : A.F + (i - kWLoads / 2) * kStep);
        load_lds16(wbase + row * A.K + kb * kBK, woff[SW ? 0 : i], dst + i * NW * 1024);
      } else {   // the rows behind the tile's last are that row again
        const uint32_t row = min(r0 + (i - kWLoads) * kStep, (uint32_t)T.n - 1u);
        load_lds16(xbase + kb * kBK, __umul24(row, (uint32_t)A.K) + c0, dst + i * NW * 1024);
      }
    }
  };

  // ---- scales, kXsChunk K steps at a time, by the same kind of loads: a
  // scale loaded into a register where it is needed would wait for every load
  // in front of it, the next stage's among them.  A tile has two blocks of
  // weight rows: gate and up, or the lower and the upper 128 features.
  const int nfb = (A.F + kScaleBlock - 1) / kScaleBlock;
  const int wb0 = SW ? ft : min(ft * 2, nfb - 1), wb1 = SW ? nfb + ft : min(ft * 2 + 1, nfb - 1);
  const float* wsp = A.w_s + ((int64_t)T.e * (SW ? 2 : 1) * nfb + wb0) * KB;
  const float* xsp = A.x_s + (int64_t)T.row * KB;
  auto scales = [&](int kb0) {
    const int buf = (kb0 / kXsChunk) & 1;
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const int j = i * NW + wave, kk = j / XG, g = j - kk * XG;
      const uint32_t tok = min(g * kWave + lane, T.n - 1);
      load_lds4(xsp + min(kb0 + kk, KB - 1), __umul24(tok, (uint32_t)KB * 4u), &sx[buf][kk][g * kWave]);
    }
    if (wave == 0) {
      const int kk = min(kb0 + (lane & (kXsChunk - 1)), KB - 1), blk = lane / kXsChunk & 1;
      load_lds4(wsp, (uint32_t)(blk * (wb1 - wb0) * KB + kk) * 4u, &sw[buf][0]);
    }
  };

  v4f acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = v4f{0, 0, 0, 0};

  scales(0);
#pragma unroll
  for (int s = 0; s < S - 1; ++s)
    if (s < KB) issue(s, 0, LPS);

  // Byte offset of this lane's 16 bytes (chunk lane/16, second chunk 4 on) in
  // a 16-row tile; row & 7 = lane & 7 in every tile.
  const int lr = (lane & 15) * kBK;
  const int o0 = lr + (((lane >> 4) ^ (lane & 7)) << 4), o1 = lr + (((4 + (lane >> 4)) ^ (lane & 7)) << 4);
  // The wave's n-th tile of tokens is tile n * WN + wn, so that the waves of a
  // short tile have the same number of them to one; those behind the last row
  // are left out.
  const int tok0 = wn * 16 + (lane & 15);
  const int live = min(max(((T.n + 15) / 16 - wn + WN - 1) / WN, 0), NT);
  // First LDS row of the wave's m-th tile of weight rows.
  auto wrow = [&](int m) {
    return SW ? (m < MT / 2 ? wm * (BF / WM) + m * 16 : BF + wm * (BF / WM) + (m - MT / 2) * 16)
              : wm * (BM / WM) + m * 16;
  };
  const int wblk = SW ? 0 : wm * (BM / WM) / kScaleBlock;

  auto steps = [&](auto nl) {
    constexpr int NL = decltype(nl)::value;
    for (int kb = 0; kb < KB; ++kb) {
      if (S > 2 && kb + S - 1 <= KB) wait_and_barrier<(S - 2) * LPS>();
      else wait_and_barrier<0>();
      const int ph = kb % kXsChunk, buf = (kb / kXsChunk) & 1;
      // Asked for early enough that the wait of a step before theirs covers them, with any S.
      if (ph == 1 && kb - ph + kXsChunk < KB) scales(kb - ph + kXsChunk);
      if constexpr (NL == 0) {
        if (kb + S - 1 < KB) issue(kb + S - 1, 0, LPS);
      } else {
        // The next stage is asked for behind this step's first LDS reads: in
        // front of them they would wait until all loads are issued.
        const unsigned char* st = lds + (kb % S) * kStage;
        const bool more = kb + S - 1 < KB;
        Operand<SW> b[NL];
        if constexpr (SW) {
          // Registers are short (64 hold the tokens' operands), so one tile of
          // weight rows after the other; the SIMD's other wave fills the gaps.
#pragma unroll
          for (int n = 0; n < NL; ++n) {
            b[n].load(st + (BM + (n * WN + wn) * 16) * kBK, o0, o1);
            if (n == 1) __builtin_amdgcn_sched_barrier(0);   // no more than two tiles' bytes beside their operands
          }
          Raw ra;
          ra.load(st + wrow(0) * kBK, o0, o1);
          float sc[NL];
#pragma unroll
          for (int n = 0; n < NL; ++n) sc[n] = sx[buf][ph][tok0 + n * WN * 16];
          const float w0 = sw[buf][ph], w1 = sw[buf][kXsChunk + ph];
          if (more) issue(kb + S - 1, 0, LPS / 2);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            __builtin_amdgcn_sched_barrier(0);
            Operand<SW> a;
            a.set(ra);
            if (m + 1 < MT) ra.load(st + wrow(m + 1) * kBK, o0, o1);
            if (m == 0 && more) issue(kb + S - 1, LPS / 2, LPS);
            v4f pr[NL];
            multiply(a, b, pr);
#pragma unroll
            for (int n = 0; n < NL; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                acc[m][n][i] = __builtin_fmaf(pr[n][i], sc[n] * (m < MT / 2 ? w0 : w1), acc[m][n][i]);
          }
        } else {
          // Tile m's products run while the sums take tile m - 1's and tile
          // m + 1's operand is read.
          Operand<SW> a[2];
#pragma unroll
          for (int n = 0; n < NL; ++n) b[n].load(st + (BM + (n * WN + wn) * 16) * kBK, o0, o1);
          a[0].load(st + wrow(0) * kBK, o0, o1);
          __builtin_amdgcn_sched_barrier(0);
          if (more) issue(kb + S - 1, 0, LPS);
          __builtin_amdgcn_sched_barrier(0);
          float sc[NL];
#pragma unroll
          for (int n = 0; n < NL; ++n) sc[n] = sx[buf][ph][tok0 + n * WN * 16] * sw[buf][wblk * kXsChunk + ph];
          v4f pr[2][NL];
#pragma unroll
          for (int m = 0; m <= MT; ++m) {
            if (m + 1 < MT) a[(m + 1) & 1].load(st + wrow(m + 1) * kBK, o0, o1);
            if (m < MT) multiply(a[m & 1], b, pr[m & 1]);
            if (m > 0)
#pragma unroll
              for (int n = 0; n < NL; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  acc[m - 1][n][i] = __builtin_fmaf(pr[(m - 1) & 1][n][i], sc[n], acc[m - 1][n][i]);
          }
        }
      }
    }
  };
  static_assert(NT <= 5, "a loop for each number of live tiles");
  if (live == NT) steps(std::integral_constant<int, NT>());
  else if (NT > 4 && live == 4) steps(std::integral_constant<int, NT < 4 ? NT : 4>());
  else if (NT > 3 && live == 3) steps(std::integral_constant<int, NT < 3 ? NT : 3>());
  else if (NT > 2 && live == 2) steps(std::integral_constant<int, NT < 2 ? NT : 2>());
  else if (NT > 1 && live == 1) steps(std::integral_constant<int, 1>());
  else steps(std::integral_constant<int, 0>());

  // No load may be on its way to LDS that the epilogue, or another workgroup, uses.
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  // ---- epilogue: lane holds features row + 4*(lane/16) + i of token tok0 + 16n
  if constexpr (!SW) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int tok = tok0 + n * WN * 16;
      if (tok >= T.n) continue;
      uint16_t* yr = A.y + (int64_t)(T.row + tok) * A.F;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int f = ft * BM + wm * (BM / WM) + m * 16 + (lane >> 4) * 4;
        if (f < A.F)
          *reinterpret_cast<uint2*>(yr + f) =
              uint2{pack_bf16(acc[m][n][0], acc[m][n][1]), pack_bf16(acc[m][n][2], acc[m][n][3])};
      }
    }
  } else {
    __syncthreads();
    int* red = reinterpret_cast<int*>(lds);            // [WM][BN] block maxima of each wave's features
    unsigned char* stage = lds + WM * BN * 4;          // [BN][128] bytes
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      int am = 0;
#pragma unroll
      for (int m = 0; m < MT / 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float gt = acc[m][n][i], up = acc[m + MT / 2][n][i];
          const float v = gt / (1.0f + __expf(-gt)) * up;
          acc[m][n][i] = v;
          am = max(am, abs_bits(v));
        }
      am = max(am, __shfl_xor(am, 16));
      am = max(am, __shfl_xor(am, 32));
      if (lane < 16) red[wm * BN + tok0 + n * WN * 16] = am;
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int tok = tok0 + n * WN * 16;
      int am = 0;
#pragma unroll
      for (int w = 0; w < WM; ++w) am = max(am, red[w * BN + tok]);
      const float scale = block_scale(am);
      if (wm == 0 && lane < 16 && tok < T.n) A.a_s[(int64_t)(T.row + tok) * nfb + ft] = scale;
#pragma unroll
      for (int m = 0; m < MT / 2; ++m) {
        float v[4] = {acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]};
        const int col = wm * (BF / WM) + m * 16 + (lane >> 4) * 4;
        *reinterpret_cast<uint32_t*>(stage + tok * kBK + (((col >> 4) ^ (tok & 7)) << 4) + (col & 15)) =
            quant4_scaled(v, scale);
      }
    }
    __syncthreads();
    for (int u = threadIdx.x; u < BN * 8; u += THREADS) {
      const int tok = u >> 3, c = u & 7;
      if (tok < T.n)
        *reinterpret_cast<v4u*>(A.a_q + (int64_t)(T.row + tok) * A.F + ft * kScaleBlock + c * 16) =
            *reinterpret_cast<const v4u*>(stage + tok * kBK + ((c ^ (tok & 7)) << 4));
    }
  }
}

template <int BM, int BN, int WM, int WN, int S, bool SW>
int launch_tile(GemmArgs A, int64_t slots, int cus, hipStream_t st) {
  constexpr int BF = SW ? BM / 2 : BM, kThreadsHere = WM * WN * kWave;
  const int64_t active = slots < A.E ? slots : A.E;
  const int nf = (A.F + BF - 1) / BF;
  A.bn = tile_rows(slots / active, active, nf, BN, cus);
  const int64_t tiles = (slots / A.bn + active) * nf;   // no fewer than the rows can need
  const int64_t grid = (tiles + 7) / 8 * 8;
  if (grid * kThreadsHere > UINT32_MAX) return MOE_ERANGE;
  const auto k = A.E <= 4 * kWave ? k_grouped_gemm<BM, BN, WM, WN, S, 4, SW>
                                  : k_grouped_gemm<BM, BN, WM, WN, S, 16, SW>;
  return launch("k_grouped_gemm", k, dim3((uint32_t)grid), dim3(kThreadsHere), 0, st, A);
}

// The tile goes by the rows that an active expert has on average, all that the
// host knows of the load.  us of each tile, even load but where noted; plain
// form K = 2048 -> 7168, SwiGLU K = 7168, I = 2048, 64 experts; "Zipf": 256
// experts, a few with most of the rows.
//   - narrow, 32 rows in workgroups of 4 waves, two on a compute unit: the
//     weights' stream is the bound.  Middle, 128 rows and three stages for the
//     plain form (128 rows an expert, 256 experts: 1.03 ms against 1.05 with
//     160 rows and two stages), 160 rows for SwiGLU (2.32 ms against 2.65 with
//     128 rows, which half of the experts exceed, and 2.51 with 256).
//       plain            8    16    24    32   Zipf 8   16   32
//       narrow         171   176   179   202      282  409  581
//       middle         169   174   179   185      295  388  493
//       (128 experts, 2048 -> 2048: 2 rows 87 against 95, 12 rows 103 against
//       107, 16 rows 104 against 107, 24 rows 119 against 110.)
//       SwiGLU           8    24    32    40    48    56    64   Zipf 16   32   64
//       narrow         313   344   342   415   428   479   498       727 1159 1868
//       middle         377   401   406   427   430   433   440       875 1209 1754
//   - large, 256 rows, above 256 rows where there are enough tiles.
//       plain          128   160   224   256   320   512  1024   Zipf 128  256  400
//       middle         269   321   379   420   514   768  1371      1026 1751 2481
//       large          269   291   338   406   481   681  1244      1106 1719 2371
//       SwiGLU         128   160   224   256   288   320   512  1024   Zipf 160  256  400
//       middle         620   778   953  1031  1188  1325  1980  3802      3315 4823 7063
//       large          632   706   899  1074  1247  1267  1818  3403      3531 4815 7159
//     From 144 to 224 rows an even load would gain from it and an uneven one
//     lose as much, so those stay with the middle tile.
template <bool SW>
int launch_any(const GemmArgs& A, int64_t slots, int cus, hipStream_t st) {
  constexpr int BF = SW ? 128 : 256, kNarrowRows = SW ? 48 : 12;
  const int64_t active = slots < A.E ? slots : A.E, avg = slots / active;
  const int64_t big = active * ((avg + 255) / 256) * ((A.F + BF - 1) / BF);   // tiles of 256 rows
  if (avg > 256 && big >= 2 * cus) return launch_tile<256, 256, 2, 4, 2, SW>(A, slots, cus, st);
  if (avg > kNarrowRows) return launch_tile<256, SW ? 160 : 128, 4, 2, SW ? 2 : 3, SW>(A, slots, cus, st);
  return launch_tile<256, 32, 4, 1, 2, SW>(A, slots, cus, st);
}

}  // namespace

int launch_grouped_gemm(const Dims& D, const uint8_t* x_q, const float* x_s, const uint8_t* w_q, const float* w_s,
                        const int* exp_off, int K, int F, uint16_t* y, int cus, hipStream_t st) {
  GemmArgs A = {x_q, x_s, w_q, w_s, exp_off, y, nullptr, nullptr, D.N, D.L, D.E, D.R, D.rows, K, F, 0};
  return launch_any<false>(A, (int64_t)D.N * D.TK, cus, st);
}

int launch_grouped_gemm_swiglu(const Dims& D, const uint8_t* x_q, const float* x_s, const uint8_t* w_q,
                               const float* w_s, const int* exp_off, int K, int I, uint8_t* a_q, float* a_s, int cus,
                               hipStream_t st) {
  GemmArgs A = {x_q, x_s, w_q, w_s, exp_off, nullptr, a_q, a_s, D.N, D.L, D.E, D.R, D.rows, K, I, 0};
  return launch_any<true>(A, (int64_t)D.N * D.TK, cus, st);
}

}  // namespace moe
