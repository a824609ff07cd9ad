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
  if (A.rows == 0) return 0;   // no tokens: exp_off is not there
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

// One workgroup: BM left features x up to BN right rows, WM x WN waves of
// MT x NT matrix tiles; S stages of both operands in LDS.
template <Epi EPI, bool LC, int BM, int BN, int WM, int WN, int S, int EPL>
__global__ __launch_bounds__(WM* WN* kWave) void k_ffn_product(ProductArgs A) {
  constexpr bool RC = EPI == Epi::kWgrad;
  constexpr int NW = WM * WN, THREADS = NW * kWave;
  constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
  constexpr int LL = BM * kStepBytes / 1024 / NW, LR = BN * kStepBytes / 1024 / NW;   // loads of a wave and stage
  static_assert(LL * NW * 1024 == BM * kStepBytes && LR * NW * 1024 == BN * kStepBytes, "loads split evenly");
  static_assert(EPI != Epi::kUp || BM == 2 * kScaleBlock, "a gate and an up half of one scale block");
  constexpr int kLeft = BM * kStepBytes, kStage = (BM + BN) * kStepBytes;
  __shared__ __align__(1024) unsigned char lds[S * kStage];

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN;

  constexpr int BF = EPI == Epi::kUp ? BM / 2 : BM;     // output features of a tile
  const int nf = (A.F + BF - 1) / BF;
  int e, row, n, ft, gt = 0, KB;     // expert, first right row, right rows, left tile, right tile, K steps
  int rem = kBK;                     // wgrad: rows of the last step
  if constexpr (RC) {
    // Tiles expert after expert; within one, groups of 4 right tiles, those fastest.
    const int ng = (A.G + BN - 1) / BN, per = nf * ng;
    const int64_t total = (int64_t)A.E * per, share = (total + 7) / 8;
    const int64_t t = (int64_t)(blockIdx.x & 7) * share + (blockIdx.x >> 3);
    if ((int64_t)(blockIdx.x >> 3) >= share || t >= total) return;
    e = (int)(t / per);
    int x = (int)(t - (int64_t)e * per);
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
    } else if constexpr (EPI == Epi::kUp) {
      const int r = i * NW * 8 + (int)r0;
      loff[i] = (uint32_t)(r < BF ? r : A.F + r - BF) * (uint32_t)A.K * 2u + c0;   // F * K <= 2^30
    } else {
      loff[i] = min(i * NW * 8 + r0, (uint32_t)(A.F - ft * BF) - 1u) * (uint32_t)A.K * 2u + c0;
    }
  }
  if constexpr (RC) {
#pragma unroll
    for (int i = 0; i < LR; ++i) roff[i] = col_off(BN, i, gt * BN, A.G);
  }
  auto issue = [&](int kb) {
    unsigned char* dst = lds + (kb % S) * kStage + wave * 1024;
#pragma unroll
    for (int i = 0; i < LL; ++i) {
      if constexpr (RC) {
        const int r = min(col_row(BM, i), n - 1 - kb * kBK);
        load_lds16(lbase + (int64_t)kb * kBK * A.F, loff[i] + (uint32_t)r * (uint32_t)A.F * 2u, dst + i * NW * 1024);
      } else if constexpr (LC) {
        load_lds16(lbase + (int64_t)kb * kBK * A.F, loff[i], dst + i * NW * 1024);
      } else {
        load_lds16(lbase + kb * kBK, loff[i], dst + i * NW * 1024);
      }
    }
#pragma unroll
    for (int i = 0; i < LR; ++i) {
      if constexpr (RC) {
        const int r = min(col_row(BN, i), n - 1 - kb * kBK);
        load_lds16(rbase + (int64_t)kb * kBK * A.G, roff[i] + (uint32_t)r * (uint32_t)A.G * 2u,
                   dst + kLeft + i * NW * 1024);
      } else {
        const uint32_t r = min(i * NW * 8 + r0, (uint32_t)n - 1u);
        load_lds16(rbase + kb * kBK, r * (uint32_t)A.K * 2u + c0, dst + kLeft + i * NW * 1024);
      }
    }
  };

  v4f acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[m][j] = v4f{0, 0, 0, 0};

#pragma unroll
  for (int s = 0; s < S - 1; ++s)
    if (s < KB) issue(s);

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

  auto steps = [&](auto nl) {
    constexpr int NL = decltype(nl)::value;
    for (int kb = 0; kb < KB; ++kb) {
      if (S > 2 && kb + S - 1 <= KB) wait_and_barrier<(S - 2) * (LL + LR)>();
      else wait_and_barrier<0>();
      unsigned char* st = lds + (kb % S) * kStage;
      if constexpr (RC) {
        if (kb == KB - 1 && rem < kBK) {   // rows behind the expert's last count as zeros
          for (int u = rem * (BM / 8) + threadIdx.x; u < kBK * (BM / 8); u += THREADS)
            reinterpret_cast<v4u*>(st)[u] = v4u{0, 0, 0, 0};
          for (int u = rem * (BN / 8) + threadIdx.x; u < kBK * (BN / 8); u += THREADS)
            reinterpret_cast<v4u*>(st + kLeft)[u] = v4u{0, 0, 0, 0};
          wait_and_barrier<0>();
        }
      }
      const bool more = kb + S - 1 < KB;
      if constexpr (NL == 0) {
        if (more) issue(kb + S - 1);
      } else {
        // The next stage is asked for behind this step's first LDS reads.
        v8bf b[2][NL], a[2];
#pragma unroll
        for (int j = 0; j < NL; ++j) b[0][j] = rr.load(st + kLeft, j * WN + wn, 0);
        a[0] = rl.load(st, ltile(0), 0);
        __builtin_amdgcn_sched_barrier(0);
        if (more) issue(kb + S - 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int kh = 0; kh < 2; ++kh) {
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const int i = kh * MT + m;
            if (i + 1 < 2 * MT) a[(i + 1) & 1] = rl.load(st, ltile((i + 1) % MT), (i + 1) / MT);
            if (kh == 0 && m == MT / 2) {
#pragma unroll
              for (int j = 0; j < NL; ++j) b[1][j] = rr.load(st + kLeft, j * WN + wn, 1);
            }
#pragma unroll
            for (int j = 0; j < NL; ++j)
              acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i & 1], b[kh][j], acc[m][j], 0, 0, 0);
          }
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

  // No load may be on its way to LDS that the epilogue, or another workgroup, uses.
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  // ---- epilogue: lane holds features 16 ltile(m) + 4 (lane/16) + i of right row tok
  const int tok0 = wn * 16 + (lane & 15), f4 = (lane >> 4) * 4;
  if constexpr (EPI == Epi::kPlain) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int tok = tok0 + j * WN * 16;
      if (tok >= n) continue;
      uint16_t* yr = static_cast<uint16_t*>(A.y) + (int64_t)(row + tok) * A.F;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int f = ft * BM + ltile(m) * 16 + f4;
        if (f < A.F)
          *reinterpret_cast<uint2*>(yr + f) =
              uint2{pack_bf16(acc[m][j][0], acc[m][j][1]), pack_bf16(acc[m][j][2], acc[m][j][3])};
      }
    }
  } else if constexpr (EPI == Epi::kWgrad) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int g = gt * BN + tok0 + j * WN * 16;
      if (g >= A.G) continue;
      const int64_t at = ((int64_t)e * A.G + g) * A.F;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int f = ft * BM + ltile(m) * 16 + f4;
        if (f >= A.F) continue;
        if (A.f32) {
          v4f* p = reinterpret_cast<v4f*>(static_cast<float*>(A.y) + at + f);
          v4f v = acc[m][j];
          if (A.add) v += *p;
          *p = v;
        } else {
          uint2* p = reinterpret_cast<uint2*>(static_cast<uint16_t*>(A.y) + at + f);
          v4f v = acc[m][j];
          if (A.add) {
            const uint2 o = *p;
            v += v4f{bf16_lo(o.x), bf16_hi(o.x), bf16_lo(o.y), bf16_hi(o.y)};
          }
          *p = uint2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        }
      }
    }
  } else if constexpr (EPI == Epi::kUpGrad) {
    const int nfb = A.F / kScaleBlock;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int tok = tok0 + j * WN * 16;
      if (tok >= n) continue;
      const int64_t r = row + tok;
      const uint8_t* hq = A.h_q + r * 2 * A.F;
      const float* hs = A.h_s + r * 2 * nfb;
      uint16_t* dh = static_cast<uint16_t*>(A.y) + r * 2 * A.F;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int f = ft * BM + ltile(m) * 16 + f4;
        if (f >= A.F) continue;
        const uint32_t gq = *reinterpret_cast<const uint32_t*>(hq + f);
        const uint32_t uq = *reinterpret_cast<const uint32_t*>(hq + A.F + f);
        const float gs = hs[f / kScaleBlock], us = hs[nfb + f / kScaleBlock];
        float dg[4], du[4], av[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float g = fp8_value(gq, i) * gs, u = fp8_value(uq, i) * us, da = acc[m][j][i];
          const float s = 1.0f / (1.0f + __expf(-g)), gs1 = g * s;
          du[i] = da * gs1;
          dg[i] = da * u * (s * (1.0f + g * (1.0f - s)));
          av[i] = gs1 * u;
        }
        *reinterpret_cast<uint2*>(dh + f) = uint2{pack_bf16(dg[0], dg[1]), pack_bf16(dg[2], dg[3])};
        *reinterpret_cast<uint2*>(dh + A.F + f) = uint2{pack_bf16(du[0], du[1]), pack_bf16(du[2], du[3])};
        if (A.a)
          *reinterpret_cast<uint2*>(A.a + r * A.F + f) = uint2{pack_bf16(av[0], av[1]), pack_bf16(av[2], av[3])};
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
      for (int m = 0; m < MT / 2; ++m) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float g = acc[m][j][i], u = acc[m + MT / 2][j][i];
          v[i] = g / (1.0f + __expf(-g)) * u;
          mg = max(mg, abs_bits(g));
          mu = max(mu, abs_bits(u));
        }
        if (tok < n)
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(A.y) + (int64_t)(row + tok) * A.F + ft * BF +
                                    ltile(m) * 16 + f4) = uint2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
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
        for (int m = 0; m < MT / 2; ++m) {
          const v4f& c = acc[m + half * (MT / 2)][j];
          float v[4] = {c[0], c[1], c[2], c[3]};
          const int col = ltile(m) * 16 + f4;
          *reinterpret_cast<uint32_t*>(stage + tok * 256 + half * 128 + (((col >> 4) ^ (tok & 7)) << 4) + (col & 15)) =
              quant4_scaled(v, scale);
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

template <Epi EPI, bool LC, int BM, int BN, int WM, int WN, int S>
int launch_rows(ProductArgs A, int64_t slots, int cus, hipStream_t st) {
  constexpr int BF = EPI == Epi::kUp ? BM / 2 : BM, kThreadsHere = WM * WN * kWave;
  const int64_t active = slots < A.E ? slots : A.E;
  const int nf = (A.F + BF - 1) / BF;
  A.bn = tile_rows(slots / active, active, nf, BN, cus);
  const int64_t tiles = (slots / A.bn + active) * nf;   // no fewer than the rows can need
  const int64_t grid = (tiles + 7) / 8 * 8;
  if (grid * kThreadsHere > UINT32_MAX) return MOE_ERANGE;
  const auto k = A.E <= 4 * kWave ? k_ffn_product<EPI, LC, BM, BN, WM, WN, S, 4>
                                  : k_ffn_product<EPI, LC, BM, BN, WM, WN, S, 16>;
  return launch("k_ffn_product", k, dim3((uint32_t)grid), dim3(kThreadsHere), 0, st, A);
}

template <Epi EPI, bool LC>
int launch_any(const ProductArgs& A, int64_t slots, int cus, hipStream_t st) {
  constexpr int BF = EPI == Epi::kUp ? 128 : 256;
  const int64_t active = slots < A.E ? slots : A.E, avg = slots / active;
  const int64_t big = active * ((avg + 255) / 256) * ((A.F + BF - 1) / BF);   // tiles of 256 rows
  if (avg > 256 && big >= 2 * cus) return launch_rows<EPI, LC, 256, 256, 2, 4, 2>(A, slots, cus, st);
  if (avg > 48) return launch_rows<EPI, LC, 256, 128, 4, 2, 2>(A, slots, cus, st);
  return launch_rows<EPI, LC, 256, 32, 4, 1, 2>(A, slots, cus, st);
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
  A.rows = D.rows;
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
  const int64_t tiles = (int64_t)A.E * ((A.F + 255) / 256) * ((A.G + 255) / 256);
  const int64_t grid = (tiles + 7) / 8 * 8;
  if (grid * 512 > UINT32_MAX) return MOE_ERANGE;
  return launch("k_ffn_product", k_ffn_product<Epi::kWgrad, true, 256, 256, 2, 4, 2, 1>, dim3((uint32_t)grid),
                dim3(512), 0, st, A);
}

}  // namespace moe
