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
};

// Rows of expert e (rank d, l-th of the rank), and in *off its offset inside
// the rank's region.
__device__ __forceinline__ int expert_rows(const GemmArgs& A, int e, int* off) {
  const int d = e / A.L, l = e - d * A.L;
  const int* eo = A.exp_off + d * (A.L + 1) + l;
  const int cap = A.R ? A.R : A.rows;
  const int a = min(max(eo[0], 0), cap), b = min(max(eo[1], a), cap);
  *off = a;
  return b - a;
}

// A workgroup's tile: up to BN rows of one expert and one block of features.
struct Tile {
  int e;      // expert, -1 for none
  int row;    // first row
  int n;      // rows, at most BN
  int f;      // feature tile
};

// Tiles are numbered expert after expert; those of one expert token tile
// fastest, in groups of up to 10 token tiles.  Each of the 8 XCDs takes one
// contiguous share of the numbers (workgroup b runs on XCD b % 8), so the 32
// compute units of an XCD work on some 3 x 10 tiles of one expert at a time
// and most of their loads meet in its L2.  An expert's rows are split evenly
// over its token tiles, in steps of 16.
//
// Every wave finds its tile by itself: lane i takes EPL consecutive experts,
// so there is no barrier and no table in memory.
template <int BN, int EPL>
__device__ __forceinline__ Tile find_tile(const GemmArgs& A, int nf) {
  const int lane = threadIdx.x & (kWave - 1);
  int n[EPL], off[EPL];
  int rows = 0, tiles = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * EPL + i;
    n[i] = expert_rows(A, min(e, A.E - 1), &off[i]);
    if (e >= A.E) n[i] = 0;
    rows += n[i];
    tiles += (n[i] + BN - 1) / BN;
  }
  int ri = rows, ti = tiles;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int a = __shfl_up(ri, d), b = __shfl_up(ti, d);
    if (lane >= d) {
      ri += a;
      ti += b;
    }
  }
  Tile T = {-1, 0, 0, 0};
  const int64_t total = (int64_t)__builtin_amdgcn_readlane(ti, kWave - 1) * nf;
  const int64_t per = (total + 7) / 8;
  const int64_t t = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((int64_t)(blockIdx.x >> 3) >= per || t >= total) return T;
  const int tt = (int)(t / nf);   // some token tile of the same expert
  int r = ri - rows, first = ti - tiles, e = -1, row = 0, m = 0, c = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int ci = (n[i] + BN - 1) / BN;
    if (tt >= first && tt < first + ci) {
      e = lane * EPL + i;
      row = A.R ? A.R * (e / A.L) + off[i] : r;
      m = n[i];
      c = ci;
      break;
    }
    first += ci;
    r += n[i];
  }
  const unsigned long long who = __ballot(e >= 0);
  if (!who) return T;
  const int src = __builtin_ctzll(who);
  e = __builtin_amdgcn_readlane(e, src);
  row = __builtin_amdgcn_readlane(row, src);
  m = __builtin_amdgcn_readlane(m, src);
  c = __builtin_amdgcn_readlane(c, src);
  first = __builtin_amdgcn_readlane(first, src);
  constexpr int kGroup = 10;
  const int groups = (c + kGroup - 1) / kGroup, size = (c + groups - 1) / groups;
  int x = (int)(t - (int64_t)first * nf);      // number among the expert's tiles
  const int g = x / (size * nf), g0 = g * size, gs = min(size, c - g0);
  x -= g0 * nf;
  const int tile = g0 + x % gs, share = min((m + c - 1) / c + 15 & ~15, BN);
  const int cap = A.R ? A.R * (e / A.L + 1) : A.rows;
  T.e = e;
  T.f = x / gs;
  T.row = min(max(row + tile * share, 0), cap);
  T.n = min(min(m - tile * share, share), cap - T.row);
  return T;
}

// 16 bytes per lane straight from global memory into LDS: lane i's bytes land
// at dst + 16*i (dst wave-uniform).
__device__ __forceinline__ void load_lds16(const uint8_t* src, unsigned char* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

// Wait until at most `Left` of this wave's LDS loads are on their way and all
// its LDS reads are done, then for the other waves.
template <int Left>
__device__ __forceinline__ void wait_and_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(Left) : "memory");
}

// One lane's 32 bytes of a 16-row tile and K step, as the operand of a
// 16x16 product over the step's 128 columns: the e4m3 bytes themselves
// (Wide = false) or widened to bf16, which is exact.
template <bool Wide>
struct Operand;
template <>
struct Operand<false> {
  v8i v;
  __device__ __forceinline__ void load(const unsigned char* p, int o0, int o1) {
    const v4i lo = *reinterpret_cast<const v4i*>(p + o0), hi = *reinterpret_cast<const v4i*>(p + o1);
    v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};
template <>
struct Operand<true> {
  v8bf v[4];
  __device__ __forceinline__ void load(const unsigned char* p, int o0, int o1) {
    const v4u lo = *reinterpret_cast<const v4u*>(p + o0), hi = *reinterpret_cast<const v4u*>(p + o1);
    v[0] = widen8(lo[0], lo[1]);
    v[1] = widen8(lo[2], lo[3]);
    v[2] = widen8(hi[0], hi[1]);
    v[3] = widen8(hi[2], hi[3]);
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
constexpr int kXsChunk = 8;        // K steps whose token scales are staged together

template <int BM, int BN, int WM, int WN, int S, int EPL, bool SW>
__global__ __launch_bounds__(WM* WN* kWave) void k_grouped_gemm(GemmArgs A) {
  constexpr int NW = WM * WN, THREADS = NW * kWave;
  constexpr int MT = BM / WM / 16, NT = BN / WN / 16;     // 16x16 tiles of a wave
  constexpr int kRowsPerLoad = kWave / 8;                  // 8 lanes of 16 bytes per row
  constexpr int LPS = (BM + BN) / kRowsPerLoad / NW;       // loads per wave and stage
  static_assert(BM % (kRowsPerLoad * NW) == 0 && BN % (kRowsPerLoad * NW) == 0, "rows split evenly over the waves");
  static_assert(!SW || BM == 2 * kScaleBlock, "a gate and an up half of one scale block");
  constexpr int kStage = (BM + BN) * kBK;
  __shared__ __align__(1024) unsigned char lds[S * kStage];
  __shared__ float sx[2][kXsChunk][BN];
  __shared__ float sw[2][2][kXsChunk];

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN;

  constexpr int BF = SW ? BM / 2 : BM;      // output features of a tile
  const Tile T = find_tile<BN, EPL>(A, (A.F + BF - 1) / BF);
  if (T.n <= 0) return;
  const int ft = T.f;

  const int KB = A.K / kBK;
  const int wrows = SW ? 2 * A.F : A.F;     // weight rows of an expert
  const uint8_t* wbase = A.w_q + (int64_t)T.e * wrows * A.K;
  const uint8_t* xbase = A.x_q + (int64_t)T.row * A.K;

  // ---- this lane's source of each of its loads: LDS row R (weights first,
  // then tokens), 16-byte position p of the row holds chunk p ^ (R & 7), so
  // that the 8 lanes of a ds_read_b128 phase hit 8 different bank groups.
  constexpr int kWLoads = BM / kRowsPerLoad / NW;
  uint32_t src[LPS];   // F * K <= 2^30, and twice that with gate and up
#pragma unroll
  for (int i = 0; i < LPS; ++i) {
    const int R = (i * NW + wave) * kRowsPerLoad + (lane >> 3);
    const int f = SW ? (R < BF ? ft * BF + R : A.F + ft * BF + R - BF) : min(ft * BF + R, A.F - 1);
    const int row = i < kWLoads ? f : min(R - BM, T.n - 1);
    src[i] = (uint32_t)row * (uint32_t)A.K + ((lane & 7) ^ (R & 7)) * 16;
  }
  auto issue = [&](int kb) {
    unsigned char* dst = lds + (kb % S) * kStage + wave * 1024;
    const uint8_t *wk = wbase + kb * kBK, *xk = xbase + kb * kBK;
#pragma unroll
    for (int i = 0; i < LPS; ++i) load_lds16((i < kWLoads ? wk : xk) + src[i], dst + i * NW * 1024);
  };

  // ---- scales, kXsChunk K steps at a time through registers into LDS: a
  // scale loaded where it is needed would wait for every load in front of it,
  // the next stage's among them.  A tile has two blocks of weight rows: gate
  // and up, or (BM = 256) the lower and the upper 128 features.
  constexpr int kXsPer = BN * kXsChunk / THREADS > 0 ? BN * kXsChunk / THREADS : 1;   // token scales of a thread
  constexpr int kXsThreads = BN * kXsChunk / kXsPer;
  constexpr int kXsGroups = kXsChunk / kXsPer;
  static_assert(kXsPer <= kXsChunk && THREADS >= 2 * kXsChunk, "");
  const int nfb = (A.F + kScaleBlock - 1) / kScaleBlock;
  float xs[kXsPer], wsc;
  const int xtok = threadIdx.x / kXsGroups, xk = (threadIdx.x % kXsGroups) * kXsPer;
  const int wk = threadIdx.x % kXsChunk, wb = threadIdx.x / kXsChunk;   // the first 16 threads
  const float* wsp = A.w_s + (SW ? ((int64_t)T.e * 2 + (wb & 1)) * nfb + ft
                                 : (int64_t)T.e * nfb + min(ft * (BM / kScaleBlock) + (wb & 1), nfb - 1)) * KB;
  const float* xsp = A.x_s + (int64_t)(T.row + min(xtok, T.n - 1)) * KB;
  auto scales_load = [&](int kb0) {
    if (kXsThreads == THREADS || threadIdx.x < kXsThreads)
#pragma unroll
      for (int i = 0; i < kXsPer; ++i) xs[i] = xsp[min(kb0 + xk + i, KB - 1)];
    if (threadIdx.x < 2 * kXsChunk) wsc = wsp[min(kb0 + wk, KB - 1)];
  };
  auto scales_store = [&](int kb0) {
    const int buf = (kb0 / kXsChunk) & 1;
    if (kXsThreads == THREADS || threadIdx.x < kXsThreads)
#pragma unroll
      for (int i = 0; i < kXsPer; ++i) sx[buf][xk + i][xtok] = xs[i];
    if (threadIdx.x < 2 * kXsChunk) sw[buf][wb][wk] = wsc;
  };

  v4f acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = v4f{0, 0, 0, 0};

  scales_load(0);
  scales_store(0);
#pragma unroll
  for (int s = 0; s < S - 1; ++s)
    if (s < KB) issue(s);

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
      if (ph == kXsChunk - 1 && kb + 1 < KB) scales_store(kb + 1);
      if (kb + S - 1 < KB) issue(kb + S - 1);
      if (ph == 2 && kb - ph + kXsChunk < KB) scales_load(kb - ph + kXsChunk);
      if constexpr (NL > 0) {
        const unsigned char* st = lds + (kb % S) * kStage;
        Operand<SW> b[NL], a[2];
#pragma unroll
        for (int n = 0; n < NL; ++n) b[n].load(st + (BM + (n * WN + wn) * 16) * kBK, o0, o1);
        a[0].load(st + wrow(0) * kBK, o0, o1);
        float s0[NL], s1[NL];
#pragma unroll
        for (int n = 0; n < NL; ++n) {
          const float x = sx[buf][ph][tok0 + n * WN * 16];
          s0[n] = x * sw[buf][wblk][ph];
          s1[n] = SW ? x * sw[buf][1][ph] : s0[n];
        }
        // Tile m's products run while the sums take tile m - 1's and tile
        // m + 1's operand is read.
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
                acc[m - 1][n][i] =
                    __builtin_fmaf(pr[(m - 1) & 1][n][i], m - 1 < MT / 2 ? s0[n] : s1[n], acc[m - 1][n][i]);
        }
      }
    }
  };
  static_assert(NT <= 4, "a loop for each number of live tiles");
  if (live == NT) steps(std::integral_constant<int, NT>());
  else if (NT > 3 && live == 3) steps(std::integral_constant<int, NT < 3 ? NT : 3>());
  else if (NT > 2 && live == 2) steps(std::integral_constant<int, NT < 2 ? NT : 2>());
  else if (NT > 1 && live == 1) steps(std::integral_constant<int, 1>());
  else steps(std::integral_constant<int, 0>());

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
          *reinterpret_cast<uint2*>(yr + f) = uint2{pack_bf16(acc[m][n][0], acc[m][n][1]), pack_bf16(acc[m][n][2], acc[m][n][3])};
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
int launch_tile(const GemmArgs& A, int64_t slots, hipStream_t st) {
  constexpr int BF = SW ? BM / 2 : BM;
  const int64_t active = slots < A.E ? slots : A.E;
  const int64_t tiles = (slots / BN + active) * ((A.F + BF - 1) / BF);   // no fewer than the rows can need
  const int64_t grid = (tiles + 7) / 8 * 8;
  if (grid > INT32_MAX) return MOE_ERANGE;
  if (A.E <= 4 * kWave)
    return launch("k_grouped_gemm", k_grouped_gemm<BM, BN, WM, WN, S, 4, SW>, dim3((uint32_t)grid), dim3(WM * WN * kWave),
                  0, st, A);
  return launch("k_grouped_gemm", k_grouped_gemm<BM, BN, WM, WN, S, 16, SW>, dim3((uint32_t)grid), dim3(WM * WN * kWave),
                0, st, A);
}

template <bool SW>
int launch_any(const GemmArgs& A, int64_t slots, int cus, hipStream_t st) {
  const int64_t active = slots < A.E ? slots : A.E;
  const int64_t avg = slots / active;
  if (avg > 256) return launch_tile<256, 256, 2, 4, 2, SW>(A, slots, st);
  if (avg > 32) return launch_tile<256, 128, 4, 2, 3, SW>(A, slots, st);
  return launch_tile<256, 32, 4, 1, 4, SW>(A, slots, st);
}

}  // namespace

int launch_grouped_gemm(const Dims& D, const uint8_t* x_q, const float* x_s, const uint8_t* w_q, const float* w_s,
                        const int* exp_off, int K, int F, uint16_t* y, int cus, hipStream_t st) {
  GemmArgs A = {x_q, x_s, w_q, w_s, exp_off, y, nullptr, nullptr, D.N, D.L, D.E, D.R, D.rows, K, F};
  return launch_any<false>(A, (int64_t)D.N * D.TK, cus, st);
}

int launch_grouped_gemm_swiglu(const Dims& D, const uint8_t* x_q, const float* x_s, const uint8_t* w_q,
                               const float* w_s, const int* exp_off, int K, int I, uint8_t* a_q, float* a_s, int cus,
                               hipStream_t st) {
  GemmArgs A = {x_q, x_s, w_q, w_s, exp_off, nullptr, a_q, a_s, D.N, D.L, D.E, D.R, D.rows, K, I};
  return launch_any<true>(A, (int64_t)D.N * D.TK, cus, st);
}

}  // namespace moe
