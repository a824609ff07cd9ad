// Expert products in bfloat16, for training: the gated feed-forward block of
// the experts over expert-major rows, its gradients, and an 8-bit checkpoint of
// the gate and up rows between the two.  With e the expert of row i:
//
//   up        [g u] = W13[e] x,  a = g / (1 + exp(-g)) * u,  h_q, h_s = e4m3 blocks of [g u]
//   product   y = W[e] x   or   y = W[e]^T x
//   up grad   da = W2[e]^T dy;  with s = 1 / (1 + exp(-g)) and [g u] from h_q, h_s:
//             dh = [da u s (1 + g (1 - s)),  da g s],  a = g s u
//   wgrad     dW[e] = sum over its rows i of d[i] x[i]^T
//
// All of them are one kernel: a left operand (features, the matrix
// instruction's rows) times a right one (tokens; for wgrad the other side's
// features), with float32 sums, each output rounded once.
//
// a and dh are rounded to bf16 where a call ends, because they are operands of
// the next call's matrix instructions: keeping them in 32 bits would take two
// bf16 parts, so twice the products.  What follows them is then two roundings
// away from the formula: y, dx and the weight gradients are off by 0.00235 of
// their norm, 0.00166 with one rounding (E = 16, 64 rows each, H = I = 2048).
#include <type_traits>

#include "gemm_dev.h"
#include "moe_internal.h"
#include "quant_dev.h"

namespace moe {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));

// What a product does with its sums.
enum class Epi { kPlain, kUp, kUpGrad, kWgrad };

struct ProductArgs {
  const uint16_t* left;    // weights of all experts; wgrad: x [rows][F]
  const uint16_t* right;   // rows [rows][K]; wgrad: d [rows][G]
  const int* exp_off;
  void* y;                 // plain: bf16 [rows][F]; up: a [rows][F]; up grad: dh [rows][2F]; wgrad: [E][G][F]
  uint16_t* a;             // up grad: a [rows][F], may be null
  uint8_t* h_q;            // up (out, may be null) and up grad (in): [rows][2F]
  float* h_s;              //                                          [rows][2F/128]
  int N, L, E, R;          // ranks, experts per rank, experts, fixed region rows (0 = packed)
  int rows;                // rows of the arrays
  int K;                   // length of the sums (wgrad: 0, it is the expert's rows)
  int F;                   // output features (of up: gate features)
  int G;                   // wgrad: features of d
  int bn;                  // rows of a tile at most
  int f32, add;            // wgrad: float32 output; added to what is there
};

constexpr int kBK = 64;                // columns of a K step
constexpr int kStepBytes = kBK * 2;    // of one row
static_assert(kStepBytes == 128, "eight 16-byte units a row and step");

// First row and number of rows of expert e.
__device__ __forceinline__ int expert_first(const ProductArgs& A, int e, int* n) {
  const int lane = threadIdx.x & (kWave - 1), d = e / A.L;
  int off;
  *n = 0;
  if (A.rows == 0) return 0;   // no tokens: neither exp_off nor d and x are there
  *n = __builtin_amdgcn_readfirstlane(expert_rows(A, e, &off));
  if (A.R) return __builtin_amdgcn_readfirstlane(A.R * d + off);
  int before = 0;      // rows of the ranks in front
  for (int i = lane; i < d; i += kWave) before += min(max(A.exp_off[i * (A.L + 1) + A.L], 0), A.rows);
#pragma unroll
  for (int s = 1; s < kWave; s <<= 1) before += __shfl_xor(before, s);
  const int row = min(max(before + off, 0), A.rows);
  *n = __builtin_amdgcn_readfirstlane(min(*n, A.rows - row));
  return __builtin_amdgcn_readfirstlane(row);
}

// The two ways an operand lies in memory and in LDS.
//
// Rows (COL = false): one row per feature or token, the sum's index fastest.
// LDS row r holds its 128 bytes of the step, unit u (16 bytes) at position
// u ^ (r & 7), so that the 8 lanes of a ds_read_b128 phase hit 8 bank groups.
//
// Columns (COL = true): one row per index of the sum, features fastest.  LDS
// row k holds W features, the 32-byte chunk c at c ^ swizzle(k).  A transposing
// read (ds_read_b64_tr_b16: 16 lanes read 4 rows of 16 features, each lane
// gets one feature's four) then turns them into the same registers: the 16
// chunks that the four lane groups read fall on all bank groups alike.
__device__ __forceinline__ int swizzle(int k) { return (k & 3) | ((k >> 1) & 4); }

// 16x16x32 operand of tile `t` (16 rows or features) and half `kh` of the step.
template <bool COL, int W>
struct Reader {
  int o[COL ? 1 : 2];
  int f;
  __device__ __forceinline__ void set(int lane) {
    if constexpr (COL) {
      const int k = (lane >> 4) * 8 + ((lane & 15) >> 2);
      o[0] = k * (W * 2) + (lane & 3) * 8;
      f = swizzle(k) * 32;
    } else {
      o[0] = (lane & 15) * kStepBytes + (((lane >> 4) ^ (lane & 7)) << 4);
      o[1] = (lane & 15) * kStepBytes + (((4 + (lane >> 4)) ^ (lane & 7)) << 4);
    }
  }
  __device__ __forceinline__ v8bf load(const unsigned char* p, int t, int kh) const {
    if constexpr (COL) {
      const unsigned char* q = p + o[0] + ((t * 32) ^ f) + kh * 32 * (W * 2);
      typedef __attribute__((address_space(3))) v4s* lds4;
      const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(q));
      const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(q + 4 * (W * 2)));
      return __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      return *reinterpret_cast<const v8bf*>(p + t * 16 * kStepBytes + o[kh]);
    }
  }
};

// 4 / (1 + exp(-g)), with the reciprocal instruction: off by at most one unit in
// the last place.  That instruction gives 0 where the quotient is subnormal,
// which 1 / (1 + exp(-g)) is for g from -87.3 down to -88.7, where exp(-g) leaves
// float32; a quarter of the sum has a normal one, and scaling by 4 is exact.
// With a division instead (correctly rounded), up and down of 2048 rows for each
// of 32 experts took 4.97 to 5.02 ms against 4.94 to 4.95, all gradients 10.03
// against 9.99.
__device__ __forceinline__ float sigmoid4(float g) {
  return __builtin_amdgcn_rcpf(__builtin_fmaf(__expf(-g), 0.25f, 0.25f));
}

// One workgroup forms BM left features x up to BN right rows of one expert:
// WM x WN waves of MT x NT matrix tiles of 16 x 16, so a lane holds four
// neighbouring features of one row.  Steps of 64 columns; SL and SR stages of
// the operands sit in LDS, filled by loads that bypass the registers.
//
// What bounds it on MI355X (2048 rows for each of 32 experts, H = 7168, I =
// 2048; ranges are over machines and runs): up 3.25 to 3.43 ms (1.12 to 1.18
// PFLOP/s), down 1.65 to 1.73, the transposed product 3.11 to 3.24 (1.19 to 1.24), up
// gradient 1.87 to 1.95 (0.99 to 1.03), weight gradients 3.21 to 3.33 and 1.55 to
// 1.61 (1.16 to 1.24; added 3.57 and 1.77, in float32 3.50 and 1.74, added there
// 4.28 and 2.11); large library products of the three layouts reach 1.60 (rows
// x rows), 1.38 and 1.18.  The matrix pipes are busy 51% to 64% of the cycles
// at a clock that falls to 1.77 to 1.9 GHz; LDS reads have no bank conflicts.
// Timing copies: with loads that stay on two steps (so in L2) 3.00 ms for up and 3.02
// transposed, against 3.57 and 3.33 then; without the loop's loads 2.68 and 2.66;
// without the epilogue 3.05, 1.42, 2.94, 1.58, 2.82 and 1.43 (so the 128 to 512 KiB
// that all compute units write at about the same time cost 7% to 16%).  Deeper
// stages are what helped most: a 256 x 128 tile with three stages against two took
// 3.99 ms against 4.85.
// Tried and slower: four waves of 128 x 128 (up 3.9 to 4.4 ms, whatever the order of
// its reads); steps of 32 columns with four or five stages (3.70); 32 x 32 matrix
// instructions (3% to 5%); groups of 2 to 6 token tiles (up to 9%); non-temporal
// stores of y (down 1.72 against 1.65) and of weight gradients (3.46 against 3.32);
// workgroups that take tile after tile and load the next one's first stages before
// they store (down 1.75 against 1.65; weight gradients of 5 rows an expert 747 us
// against 520: finding the next tile is in the way of a short one).
template <Epi EPI, bool LC, int BM, int BN, int WM, int WN, int SL, int SR, int EPL>
__global__ __launch_bounds__(WM* WN* kWave) void k_ffn_product(ProductArgs A) {
  constexpr bool RC = EPI == Epi::kWgrad;
  constexpr int NW = WM * WN, THREADS = NW * kWave;
  constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
  constexpr int LL = BM * kStepBytes / 1024 / NW, LR = BN * kStepBytes / 1024 / NW;   // loads of a wave and stage
  static_assert(LL * NW * 1024 == BM * kStepBytes && LR * NW * 1024 == BN * kStepBytes, "loads split evenly");
  static_assert(MT % (EPI == Epi::kUp ? 4 : 2) == 0, "the epilogue takes tiles in pairs");
  static_assert(EPI != Epi::kUp || (BM == 2 * kScaleBlock && LL % 2 == 0), "a gate and an up half of one scale block");
  static_assert(SR == SL || SR == SL + 1, "the right operand's loads are a step's last");
  constexpr int kLeft = BM * kStepBytes, kRight = BN * kStepBytes;   // bytes of a stage
  static_assert(EPI != Epi::kUp || 2 * WM * BN * 4 + BN * 256 <= SL * kLeft + SR * kRight, "the epilogue's rows fit");
  __shared__ __align__(1024) unsigned char lds[SL * kLeft + SR * kRight];
  unsigned char* const lds_r = lds + SL * kLeft;

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN;

  constexpr int BF = EPI == Epi::kUp ? BM / 2 : BM;     // output features of a tile
  const int nf = (A.F + BF - 1) / BF;
  int e, row, n, ft, gt = 0, KB;     // expert, first right row, right rows, left tile, right tile, K steps
  int rem = kBK;                     // wgrad: rows of the last step
  if constexpr (RC) {
    // Expert after expert; each XCD (workgroup b runs on XCD b % 8) takes an
    // eighth of every expert's tiles, so that an expert with many rows keeps all of
    // them busy.  Within an expert groups of 4 right tiles, those fastest.
    const int ng = (A.G + BN - 1) / BN, per = nf * ng, share = (per + 7) / 8;
    e = (int)((blockIdx.x >> 3) / (uint32_t)share);
    int x = (int)(blockIdx.x & 7) * share + (int)((blockIdx.x >> 3) - (uint32_t)e * (uint32_t)share);
    if (x >= per) return;
    const int g0 = x / (4 * nf) * 4, gs = min(4, ng - g0);
    x -= g0 * nf;
    gt = g0 + x % gs;
    ft = x / gs;
    row = expert_first(A, e, &n);
    KB = (n + kBK - 1) / kBK;
    rem = n - (KB - 1) * kBK;
  } else {
    const Tile T = find_tile<EPL>(A, nf);
    if (T.n <= 0) return;
    e = T.e;
    row = T.row;
    n = T.n;
    ft = T.f;
    KB = A.K / kBK;
  }

  // ---- loads: each fills 1 KiB of LDS, 64 lanes of 16 bytes in LDS order, and
  // takes them from where the layout above has them.  What lies behind the last
  // feature or row is the last one again.
  const int64_t wrows = EPI == Epi::kUp ? 2 * A.F : A.F;
  const uint16_t* lbase = A.left + (RC ? (int64_t)row * A.F : (int64_t)e * wrows * A.K + (LC ? 0 : (int64_t)ft * BF * A.K));
  const uint16_t* rbase = A.right + (int64_t)row * (RC ? A.G : A.K);
  const uint32_t r0 = wave * 8 + (lane >> 3), c0 = ((lane & 7) ^ (r0 & 7)) * 16;
  // Byte offset in its row of this lane's 16 bytes of the i-th load of a column
  // operand W features wide, `first` and `last` the tile's first feature and
  // all there are, and the load's row in the step.
  auto col_row = [&](int W, int i) { return (i * NW + wave) * (512 / W) + lane / (W / 8); };
  auto col_off = [&](int W, int i, int first, int last) {
    const int u = lane % (W / 8), c = (((u >> 1) ^ swizzle(col_row(W, i))) << 1) | (u & 1);
    return (uint32_t)min(first + c * 8, last - 8) * 2u;
  };
  uint32_t loff[LL], roff[RC ? LR : 1];
#pragma unroll
  for (int i = 0; i < LL; ++i) {
    if constexpr (LC) {
      loff[i] = col_off(BM, i, ft * BM, A.F) + (RC ? 0u : (uint32_t)col_row(BM, i) * (uint32_t)A.F * 2u);
    } else if constexpr (EPI == Epi::kUp) {   // the second half of the loads: up rows, F rows on
      loff[i] = (uint32_t)((i % (LL / 2)) * NW * 8 + r0) * (uint32_t)A.K * 2u + c0;
    } else {
      loff[i] = min(i * NW * 8 + r0, (uint32_t)(A.F - ft * BF) - 1u) * (uint32_t)A.K * 2u + c0;
    }
  }
  if constexpr (RC) {
#pragma unroll
    for (int i = 0; i < LR; ++i) roff[i] = col_off(BN, i, gt * BN, A.G);
  }
  // The i-th of the wave's loads of the left operand's stage kb, and of the right one's.
  auto issue_left = [&](int kb, int i) {
    unsigned char* dst = lds + (kb % SL) * kLeft + (i * NW + wave) * 1024;
    if constexpr (RC) {
      const int r = min(col_row(BM, i), n - 1 - kb * kBK);
      load_lds16(lbase + (int64_t)kb * kBK * A.F, loff[i] + (uint32_t)r * (uint32_t)A.F * 2u, dst);
    } else if constexpr (LC) {
      load_lds16(lbase + (int64_t)kb * kBK * A.F, loff[i], dst);
    } else {
      const int64_t up = EPI == Epi::kUp && i >= LL / 2 ? (int64_t)A.F * A.K : 0;
      load_lds16(lbase + up + kb * kBK, loff[i], dst);
    }
  };
  auto issue_right = [&](int kb, int i) {
    unsigned char* dst = lds_r + (kb % SR) * kRight + (i * NW + wave) * 1024;
    if constexpr (RC) {
      const int r = min(col_row(BN, i), n - 1 - kb * kBK);
      load_lds16(rbase + (int64_t)kb * kBK * A.G, roff[i] + (uint32_t)r * (uint32_t)A.G * 2u, dst);
    } else {
      const uint32_t r = min(i * NW * 8 + r0, (uint32_t)n - 1u);
      load_lds16(rbase + kb * kBK, r * (uint32_t)A.K * 2u + c0, dst);
    }
  };

  v4f acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[m][j] = v4f{0, 0, 0, 0};

#pragma unroll
  for (int s = 0; s < SR; ++s) {
    if (s >= KB) break;
    if (s < SL)
#pragma unroll
      for (int i = 0; i < LL; ++i) issue_left(s, i);
#pragma unroll
    for (int i = 0; i < LR; ++i) issue_right(s, i);
  }

  Reader<LC, BM> rl;
  Reader<RC, BN> rr;
  rl.set(lane);
  rr.set(lane);
  // The wave's j-th tile of right rows is tile j * WN + wn, so that the waves of
  // a short tile have the same number of them to one; those behind the last
  // row are left out.
  const int live = RC ? NT : min(max(((n + 15) / 16 - wn + WN - 1) / WN, 0), NT);
  // The wave's m-th tile of left features.
  auto ltile = [&](int m) {
    return EPI == Epi::kUp ? (m < MT / 2 ? wm * (MT / 2) + m : BF / 16 + wm * (MT / 2) + m - MT / 2) : wm * MT + m;
  };

  // Stage kb is in LDS for all waves, with zeros behind the expert's last row;
  // what was asked for after it may be on its way: SL - 2 stages of the left
  // operand and SR - 2 of the right one.
  auto arrived = [&](int kb) {
    constexpr int kLater = (SL - 2) * LL + (SR - 2) * LR;
    if (kLater > 0 && kb + SR - 2 < KB) wait_and_barrier<kLater>();
    else wait_and_barrier<0>();
    if constexpr (RC) {
      if (kb == KB - 1 && rem < kBK) {
        unsigned char *l = lds + (kb % SL) * kLeft, *r = lds_r + (kb % SR) * kRight;
        for (int u = rem * (BM / 8) + threadIdx.x; u < kBK * (BM / 8); u += THREADS)
          reinterpret_cast<v4u*>(l)[u] = v4u{0, 0, 0, 0};
        for (int u = rem * (BN / 8) + threadIdx.x; u < kBK * (BN / 8); u += THREADS)
          reinterpret_cast<v4u*>(r)[u] = v4u{0, 0, 0, 0};
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      }
    }
  };

  // Two halves of 32 columns a step.  While one half's products run, the
  // operands of the next are read: those of the step's second half during the
  // first, those of the next step's first half during the second.  So the one
  // barrier of a step stands in its middle, where every wave has read all of the
  // stage, and the loads of step kb + SL (SR) go into it from there on.
  auto steps = [&](auto nl) {
    constexpr int NL = decltype(nl)::value;
    constexpr int kReads = NL + MT, kProducts = MT * NL;
    // The checkpoint's scales are float32 outputs, and a long chain of joins shows
    // in them (K = 2048: 2.5e-7 of a value against a library product's 1.1e-7).
    // So the sums of 128 columns (narrow tile, bound by the weights' stream) or
    // 512 (middle tile) join a total; the large tile has no registers for one.
    // Of the scales' norm at K = 7168: middle tile 8.5e-8, large tile 4.7e-7, a
    // float32 product of the library 8.9e-7; at K = 32768 large tile 9.9e-7, library
    // 2.3e-6.  Float32 weight gradients have no total either: their error grows as the
    // root of the rows, 1.6e-6 of the norm at 65536 (library 1.9e-6).
    constexpr int kJoin = EPI != Epi::kUp ? 0 : BN <= 32 ? 2 : BN <= 128 ? 8 : 0;   // steps
    v4f total[kJoin ? MT : 1][kJoin && NL > 0 ? NL : 1] = {};
    v8bf a[2][MT], b[2][NL > 0 ? NL : 1];
    auto read = [&](int kb, int kh, int i) {   // the i-th operand of a half
      if (i < NL) b[kh][i] = rr.load(lds_r + (kb % SR) * kRight, i * WN + wn, kh);
      else a[kh][i - NL] = rl.load(lds + (kb % SL) * kLeft, ltile(i - NL), kh);
    };
    // A half's products with `ops` reads and loads spread evenly between them, in
    // this order: a wave issues in order, and a row of reads would leave its
    // matrix pipe without work.
    auto half = [&](auto kh, auto ops, auto op) {
      constexpr int H = decltype(kh)::value, N = decltype(ops)::value;
      if constexpr (NL == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) op(i);
      } else {
#pragma unroll
        for (int q = 0; q < kProducts; ++q) {
#pragma unroll
          for (int i = q * N / kProducts; i < (q + 1) * N / kProducts; ++i) op(i);
          const int m = q / NL, j = q % NL;
          acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[H][m], b[H][j], acc[m][j], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    };
    constexpr std::integral_constant<int, 0> first{};
    constexpr std::integral_constant<int, 1> second{};
    auto step = [&](int kb, auto next, auto left, auto right) {   // which of the later stages there are
      constexpr int R = NL > 0 ? kReads : 0, LD = (left ? LL : 0) + (right ? LR : 0);
      half(first, std::integral_constant<int, R>(), [&](int i) { read(kb, 1, i); });
      if constexpr (next) arrived(kb + 1);
      // reads and loads in turn, the loads of the left operand first
      half(second, std::integral_constant<int, (next ? R : 0) + LD>(), [&](int i) {
        constexpr int Rn = next ? R : 0, N = Rn + LD;
        const int r0 = i * Rn / N, r1 = (i + 1) * Rn / N;
        if (r1 > r0) read(kb + 1, 0, r0);
        else if (i - r0 < LL && left) issue_left(kb + SL, i - r0);
        else issue_right(kb + SR, i - r0 - (left ? LL : 0));
      });
      if constexpr (kJoin && NL > 0) {
        if ((kb + 1) % kJoin == 0) {
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < NL; ++j) {
              total[m][j] += acc[m][j];
              acc[m][j] = v4f{0, 0, 0, 0};
            }
        }
      }
    };
    if (KB == 0) return;
    arrived(0);
    if constexpr (NL > 0) {
#pragma unroll
      for (int i = 0; i < kReads; ++i) read(0, 0, i);
    }
    int kb = 0;
    for (; kb + SR < KB; ++kb) step(kb, std::true_type(), std::true_type(), std::true_type());
    for (; kb + SL < KB; ++kb) step(kb, std::true_type(), std::true_type(), std::false_type());
    for (; kb + 1 < KB; ++kb) step(kb, std::true_type(), std::false_type(), std::false_type());
    step(kb, std::false_type(), std::false_type(), std::false_type());
    if constexpr (kJoin && NL > 0) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NL; ++j) acc[m][j] += total[m][j];
    }
  };
  // A loop for each number of live tiles.
  auto pick = [&](auto self, auto nl) -> void {
    constexpr int NL = decltype(nl)::value;
    if (live >= NL) steps(nl);
    else if constexpr (NL > 0) self(self, std::integral_constant<int, NL - 1>());
  };
  pick(pick, std::integral_constant<int, NT>());

  // No load may be on its way to LDS that the epilogue, or another workgroup, uses.
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  // ---- epilogue: acc[m][j] holds features 16 ltile(m) + 4 (lane / 16) + i of
  // right row tok0 + 16 WN j.  Lanes 16 apart trade halves of two neighbouring
  // tiles, so that a lane has eight consecutive features (f8 on from the first
  // tile's) and four lanes 64 consecutive bytes of a bf16 row: eight[0..7] of
  // the pair m, m + 1.
  const int tok0 = wn * 16 + (lane & 15), f8 = ((lane >> 4) & 1) * 16 + (lane >> 5) * 8;
  auto pair = [&](int m, int j, float (&eight)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const auto w = __builtin_amdgcn_permlane16_swap(__float_as_uint(acc[m][j][i]), __float_as_uint(acc[m + 1][j][i]),
                                                      false, false);
      eight[i] = __uint_as_float(w[0]);
      eight[4 + i] = __uint_as_float(w[1]);
    }
  };
  auto rounded = [](const float (&v)[8]) {
    return v4u{cvt_bf16(v[0], v[1]), cvt_bf16(v[2], v[3]), cvt_bf16(v[4], v[5]), cvt_bf16(v[6], v[7])};
  };
  if constexpr (EPI == Epi::kPlain) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int tok = tok0 + j * WN * 16;
      uint16_t* yr = static_cast<uint16_t*>(A.y) + (int64_t)(row + tok) * A.F;
#pragma unroll
      for (int m = 0; m < MT; m += 2) {
        const int f = ft * BM + ltile(m) * 16 + f8;
        float v[8];
        pair(m, j, v);
        if (tok < n && f < A.F) *reinterpret_cast<v4u*>(yr + f) = rounded(v);
      }
    }
  } else if constexpr (EPI == Epi::kWgrad) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int g = gt * BN + tok0 + j * WN * 16;
      const int64_t at = ((int64_t)e * A.G + g) * A.F;
      if (A.f32) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int f = ft * BM + ltile(m) * 16 + (lane >> 4) * 4;
          if (g >= A.G || f >= A.F) continue;
          v4f* p = reinterpret_cast<v4f*>(static_cast<float*>(A.y) + at + f);
          v4f v = acc[m][j];
          if (A.add) v += *p;
          *p = v;
        }
      } else {
#pragma unroll
        for (int m = 0; m < MT; m += 2) {
          const int f = ft * BM + ltile(m) * 16 + f8;
          float v[8];
          pair(m, j, v);
          if (g >= A.G || f >= A.F) continue;
          v4u* p = reinterpret_cast<v4u*>(static_cast<uint16_t*>(A.y) + at + f);
          if (A.add) {
            const v4u o = *p;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v[2 * i] += bf16_lo(o[i]);
              v[2 * i + 1] += bf16_hi(o[i]);
            }
          }
          *p = rounded(v);
        }
      }
    }
  } else if constexpr (EPI == Epi::kUpGrad) {
    // All of a column's checkpoint is asked for before the first of it is used.
    typedef unsigned int v2u __attribute__((ext_vector_type(2)));
    const int nfb = A.F / kScaleBlock;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int tok = tok0 + j * WN * 16;
      const int64_t r = row + min(tok, n - 1);
      const uint8_t* hq = A.h_q + r * 2 * A.F;
      const float* hs = A.h_s + r * 2 * nfb;
      uint16_t* dh = static_cast<uint16_t*>(A.y) + r * 2 * A.F;
      v2u gq[MT / 2], uq[MT / 2];
      float gs[MT / 2], us[MT / 2];
#pragma unroll
      for (int p = 0; p < MT / 2; ++p) {
        const int f = min(ft * BM + ltile(2 * p) * 16 + f8, A.F - 8);
        gq[p] = *reinterpret_cast<const v2u*>(hq + f);
        uq[p] = *reinterpret_cast<const v2u*>(hq + A.F + f);
        gs[p] = hs[f / kScaleBlock];
        us[p] = hs[nfb + f / kScaleBlock];
      }
#pragma unroll
      for (int p = 0; p < MT / 2; ++p) {
        const int f = ft * BM + ltile(2 * p) * 16 + f8;
        float da[8], dg[8], du[8], av[8];
        pair(2 * p, j, da);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float g = fp8_value(gq[p][i / 4], i & 3) * gs[p], u = fp8_value(uq[p][i / 4], i & 3) * us[p];
          const float q = sigmoid4(g), s = 0.25f * q, y = 0.25f * g * q;
          du[i] = da[i] * y;
          dg[i] = da[i] * u * (q * (0.25f + 0.25f * g * (1.0f - s)));
          av[i] = y * u;
        }
        if (tok < n && f < A.F) {
          *reinterpret_cast<v4u*>(dh + f) = rounded(dg);
          *reinterpret_cast<v4u*>(dh + A.F + f) = rounded(du);
          if (A.a) *reinterpret_cast<v4u*>(A.a + r * A.F + f) = rounded(av);
        }
      }
    }
  } else {
    __syncthreads();
    // gate and up are rounded to 8 bits per 128 features, so block maxima go over the WM waves of a row
    int* red = reinterpret_cast<int*>(lds);            // [2][WM][BN]
    unsigned char* stage = lds + 2 * WM * BN * 4;      // [BN][256] bytes: gate, up
    const int nfb = A.F / kScaleBlock;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int tok = tok0 + j * WN * 16;
      int mg = 0, mu = 0;
#pragma unroll
      for (int m = 0; m < MT / 2; m += 2) {
        float g[8], u[8], v[8];
        pair(m, j, g);
        pair(m + MT / 2, j, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = 0.25f * g[i] * sigmoid4(g[i]) * u[i];
          mg = max(mg, abs_bits(g[i]));
          mu = max(mu, abs_bits(u[i]));
          // kept in the new order
          acc[m + i / 4][j][i & 3] = g[i];
          acc[m + MT / 2 + i / 4][j][i & 3] = u[i];
        }
        if (tok < n)
          *reinterpret_cast<v4u*>(static_cast<uint16_t*>(A.y) + (int64_t)(row + tok) * A.F + ft * BF + ltile(m) * 16 +
                                  f8) = rounded(v);
      }
      mg = max(mg, __shfl_xor(mg, 16));
      mg = max(mg, __shfl_xor(mg, 32));
      mu = max(mu, __shfl_xor(mu, 16));
      mu = max(mu, __shfl_xor(mu, 32));
      if (lane < 16) {
        red[wm * BN + tok] = mg;
        red[(WM + wm) * BN + tok] = mu;
      }
    }
    if (!A.h_q) return;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int tok = tok0 + j * WN * 16;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        int am = 0;
#pragma unroll
        for (int w = 0; w < WM; ++w) am = max(am, red[(half * WM + w) * BN + tok]);
        const float scale = block_scale(am);
        if (wm == 0 && lane < 16 && tok < n) A.h_s[((int64_t)(row + tok) * 2 + half) * nfb + ft] = scale;
#pragma unroll
        for (int m = 0; m < MT / 2; m += 2) {
          const v4f &c = acc[m + half * (MT / 2)][j], &d = acc[m + 1 + half * (MT / 2)][j];
          const float v[8] = {c[0], c[1], c[2], c[3], d[0], d[1], d[2], d[3]};
          const int col = ltile(m) * 16 + f8;
          *reinterpret_cast<uint2*>(stage + tok * 256 + half * 128 + (((col >> 4) ^ (tok & 7)) << 4) + (col & 15)) =
              uint2{quant4_scaled(v, scale), quant4_scaled(v + 4, scale)};
        }
      }
    }
    __syncthreads();
    for (int u = threadIdx.x; u < BN * 16; u += THREADS) {
      const int tok = u >> 4, half = (u >> 3) & 1, c = u & 7;
      if (tok < n)
        *reinterpret_cast<v4u*>(A.h_q + ((int64_t)(row + tok) * 2 + half) * A.F + ft * BF + c * 16) =
            *reinterpret_cast<const v4u*>(stage + tok * 256 + half * 128 + ((c ^ (tok & 7)) << 4));
    }
  }
}

template <Epi EPI, bool LC, int BM, int BN, int WM, int WN, int SL, int SR>
int launch_rows(ProductArgs A, int64_t slots, int cus, hipStream_t st) {
  constexpr int BF = EPI == Epi::kUp ? BM / 2 : BM, kThreadsHere = WM * WN * kWave;
  const int64_t active = slots < A.E ? slots : A.E;
  const int nf = (A.F + BF - 1) / BF;
  A.bn = tile_rows(slots / active, active, nf, BN, cus);
  const int64_t tiles = (slots / A.bn + active) * nf;   // no fewer than the rows can need
  const int64_t grid = (tiles + 7) / 8 * 8;
  if (grid * kThreadsHere > UINT32_MAX) return MOE_ERANGE;
  auto k = k_ffn_product<EPI, LC, BM, BN, WM, WN, SL, SR, 4>;   // the small tile: at most 256 experts
  if constexpr (BM > 128)
    if (A.E > 4 * kWave) k = k_ffn_product<EPI, LC, BM, BN, WM, WN, SL, SR, 16>;
  return launch("k_ffn_product", k, dim3((uint32_t)grid), dim3(kThreadsHere), 0, st, A);
}

// The tile goes by the rows that an active expert has on average, all that the
// host knows of the load.  us of each tile; "even": 32 experts, "Zipf": 64 experts,
// a few with most of the rows; H = 7168, I = 2048; up / down / up gradient /
// transposed.
//   - narrow, 32 rows in workgroups of 4 waves, up to 24 rows an expert:
//       even    24                    32                    48
//       narrow  314 179 165 330       340 194 200 378       390 226 192 394
//       middle  316 181 173 334       319 173 219 338       324 216 221 344
//       Zipf    16                    32                    64
//       narrow  583 323 322 615       732 389 393 755       1037 528 527 1030
//       middle  584 320 323 589       687 343 410 664       708 395 414 719
//   - middle, 128 rows and three stages of both operands;
//   - small, 128 features x 128 rows, where the middle tile would leave half of the
//     compute units without one (one expert; up gradient, down):
//       rows    200        500        1000       1337       2000
//       small   41 14      43 19      48         53         63
//       middle  67 19      68 22      70         76         80
//     (down with 1000 rows, 224 middle tiles: 34 against 29.)  Up's tile cannot
//     shrink, it holds a gate and an up block of 128 features;
//   - large, 256 rows, above 150 rows an expert where there are two tiles for every
//     compute unit at least (200 rows, up gradient with one: 377 against 283):
//       even    128           160           200           256
//       middle  429 248 455   483 273 493   516 266 526   631 317 634   (up, down, transposed)
//       large   394 259 425   410 266 441   445 242 472   566 302 619
//       Zipf    128               170                 256                 400
//       middle  904 452 533 894   1071 512 578 1009   1340 653 756 1307   1878 916 1046 1825
//       large   991 458 557 918   1038 517 574 1026   1248 619 745 1259   1666 820  976 1670
//     A single expert's rows are known to the host, so its tile is chosen by the
//     rounds that tiles of up to 128 and up to 256 rows need (up, down, up gradient,
//     transposed):
//       rows    1000              1337              2000               2300              4000
//       middle  75 31  70  60     85 50  76  97     107 62 81  117     159 64 87  124    212 122 115 232
//       large   90 32 100  63     95 40 101  75     111 49 104  92     125 53 110  98    172  98 123 182
template <Epi EPI, bool LC>
int launch_any(const ProductArgs& A, int64_t slots, int cus, hipStream_t st) {
  constexpr int BF = EPI == Epi::kUp ? 128 : 256;
  const int64_t active = slots < A.E ? slots : A.E, avg = slots / active, nf = (A.F + BF - 1) / BF;
  // The third stage of the right operand pays where both lie in rows (up: 3.39
  // ms against 3.55, the transposed product 3.32 against 3.24).
  auto cost = [&](int BN) {   // rounds of tiles, as tile_rows prices them
    const int bn = tile_rows(avg, active, (int)nf, BN, cus);
    return (active * ((avg + bn - 1) / bn) * nf + cus - 1) / cus * (bn + 48);
  };
  if ((avg > 150 && active * ((avg + 255) / 256) * nf >= 2 * cus) ||
      (A.E == 1 && avg > 24 && 9 * cost(256) < 8 * cost(128)))
    return launch_rows<EPI, LC, 256, 256, 2, 4, 2, LC ? 2 : 3>(A, slots, cus, st);
  if (avg > 24) {
    if constexpr (EPI != Epi::kUp) {
      if (2 * active * ((avg + 127) / 128) * nf <= cus && A.E <= 4 * kWave)
        return launch_rows<EPI, LC, 128, 128, 2, 4, 4, 4>(A, slots, cus, st);
    }
    return launch_rows<EPI, LC, 256, 128, 4, 2, 3, 3>(A, slots, cus, st);
  }
  return launch_rows<EPI, LC, 256, 32, 4, 1, 3, 3>(A, slots, cus, st);
}

// One tile of 256 x 256 for every load: with tiles of 128 x 128, two workgroups on a
// compute unit, 5 rows an expert took 628 us against 507, 2048 rows 5.05 ms against
// 3.56.
int launch_wgrad(const ProductArgs& A, hipStream_t st) {
  constexpr int BM = 256, BN = 256, WM = 2, WN = 4, kThreadsHere = WM * WN * kWave;
  const int64_t per = (int64_t)((A.F + BM - 1) / BM) * ((A.G + BN - 1) / BN), grid = (per + 7) / 8 * 8 * A.E;
  if (grid * kThreadsHere > UINT32_MAX) return MOE_ERANGE;
  return launch("k_ffn_product", k_ffn_product<Epi::kWgrad, true, BM, BN, WM, WN, 2, 2, 1>, dim3((uint32_t)grid),
                dim3(kThreadsHere), 0, st, A);
}

ProductArgs base_args(const Dims& D, const uint16_t* left, const uint16_t* right, const int* exp_off, void* y, int K,
                      int F) {
  ProductArgs A = {};
  A.left = left;
  A.right = right;
  A.exp_off = exp_off;
  A.y = y;
  A.N = D.N;
  A.L = D.L;
  A.E = D.E;
  A.R = D.R;
  A.rows = D.T ? D.rows : 0;   // an empty batch has no rows, whatever its regions would hold
  A.K = K;
  A.F = F;
  return A;
}

}  // namespace

int launch_ffn_up(const Dims& D, const uint16_t* x, const uint16_t* w13, const int* exp_off, int K, int I, uint16_t* a,
                  uint8_t* h_q, float* h_s, int cus, hipStream_t st) {
  ProductArgs A = base_args(D, w13, x, exp_off, a, K, I);
  A.h_q = h_q;
  A.h_s = h_s;
  return launch_any<Epi::kUp, false>(A, (int64_t)D.N * D.TK, cus, st);
}

int launch_grouped_gemm_bf16(const Dims& D, const uint16_t* x, const uint16_t* w, const int* exp_off, int K, int F,
                             bool w_t, uint16_t* y, int cus, hipStream_t st) {
  const ProductArgs A = base_args(D, w, x, exp_off, y, K, F);
  return w_t ? launch_any<Epi::kPlain, true>(A, (int64_t)D.N * D.TK, cus, st)
             : launch_any<Epi::kPlain, false>(A, (int64_t)D.N * D.TK, cus, st);
}

int launch_ffn_up_grad(const Dims& D, const uint16_t* dy, const uint16_t* w2, const uint8_t* h_q, const float* h_s,
                       const int* exp_off, int K, int I, uint16_t* dh, uint16_t* a, int cus, hipStream_t st) {
  ProductArgs A = base_args(D, w2, dy, exp_off, dh, K, I);
  A.a = a;
  A.h_q = const_cast<uint8_t*>(h_q);
  A.h_s = const_cast<float*>(h_s);
  return launch_any<Epi::kUpGrad, true>(A, (int64_t)D.N * D.TK, cus, st);
}

int launch_grouped_wgrad(const Dims& D, const uint16_t* d, const uint16_t* x, const int* exp_off, int F, int K,
                         void* dw, bool f32, bool add, hipStream_t st) {
  ProductArgs A = base_args(D, x, d, exp_off, dw, 0, K);
  A.G = F;
  A.f32 = f32;
  A.add = add;
  return launch_wgrad(A, st);
}

}  // namespace moe
