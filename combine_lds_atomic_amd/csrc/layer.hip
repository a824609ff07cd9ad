// The experts' part of a whole MoE layer for a few tokens, in two kernels:
//
//   out[t] = bf16( sum_j w[t][j] * W2[e] ( silu(Wg[e] x_t) * (Wu[e] x_t) ) ),  e = topk_idx[t][j]
//
// with e4m3 weights and a scale for each 128x128 block, and the tokens in
// bf16.  The weights' stream is what counts at these sizes: every weight that
// some token needs is read once for each pass of 16, 32 or 64 of its expert's
// tokens, so once where they fit one pass.  e4m3 converts to bf16 exactly, so
// the products run on bf16 matrix instructions and nothing but the output is
// rounded to 8 bits.
//
// The activation between the two products is held as the sum of two bf16 (16
// significand bits), multiplied one after the other: a relative 2^-16 of each
// value at most, 3e-6 of a row's norm, beside the 1.7e-3 of the output's rounding.  A
// third bf16 would hold float32's 24 bits; it took 90 us against 81 for one
// token, 750 against 709 for 13, 588 against 525 for 16 members an expert and
// 1385 against 1167 for 64.
#include "moe_internal.h"
#include "quant_dev.h"

namespace moe {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

struct LayerArgs {
  const uint16_t* x;
  const int* idx;
  const float* w;
  const uint8_t* w13_q;
  const float* w13_s;
  const uint8_t* w2_q;
  const float* w2_s;
  uint16_t* out;
  uint32_t* flags;
  uint16_t* a_hi;   // [slots][I]: the weighted activation's upper bf16
  uint16_t* a_lo;   // [slots][I]: what is left of it
  float* part;      // [splits][H/32][tokens][32] sums of the down product's splits (splits > 1)
  int* ticket;      // [H/32] splits of the tile that are done
  int splits;
  int tokens, slots, k, E, H, I;
};

constexpr int kLayerUpWaves = 4;
constexpr int kLayerDownWaves = 4;
constexpr int kLayerDownRows = 32;                       // output rows of a workgroup
constexpr int kLayerMaxSplits = 16;
constexpr int kLayerMaxTiles = kMaxH / kLayerDownRows;   // tickets
constexpr int kLayerMaxSlots = kLayerMaxTokens * kMaxK;
static_assert(kLayerMaxTokens <= kWave, "a lane for each token");

// The call's distinct experts, ascending, and every slot's expert (-1 for an
// id outside [0, E)).
struct LayerRoutes {
  int16_t id[kLayerMaxSlots];
  int16_t experts[kMaxE];
  uint32_t mask[kMaxE / 32];
  int before[kMaxE / 32];   // experts in front of each word of the mask
  int count;
};

// Fills R; returns whether this thread saw a bad id.  Ends with a barrier.
__device__ __forceinline__ bool layer_routes(const LayerArgs& A, LayerRoutes& R) {
  constexpr int kWords = kMaxE / 32;
  static_assert(kWords <= kWave, "one lane a word");
  bool bad = false;
  if (threadIdx.x < kWords) R.mask[threadIdx.x] = 0u;
  __syncthreads();
  for (int s = threadIdx.x; s < A.slots; s += blockDim.x) {
    int e = A.idx[s];
    if (e < 0 || e >= A.E) {
      bad = true;
      e = -1;
    } else {
      atomicOr(&R.mask[e >> 5], 1u << (e & 31));
    }
    R.id[s] = (int16_t)e;
  }
  __syncthreads();
  if (threadIdx.x < kWave) {
    const int lane = threadIdx.x, n = lane < kWords ? __popc(R.mask[lane]) : 0;
    int x = n;
#pragma unroll
    for (int d = 1; d < kWords; d <<= 1) {
      const int y = __shfl_up(x, d);
      if (lane >= d) x += y;
    }
    if (lane < kWords) R.before[lane] = x - n;
    if (lane == kWords - 1) R.count = x;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < A.E; e += blockDim.x) {
    const uint32_t m = R.mask[e >> 5];
    if (m >> (e & 31) & 1u) R.experts[R.before[e >> 5] + __popc(m & ((1u << (e & 31)) - 1u))] = (int16_t)e;
  }
  __syncthreads();
  return bad;
}

// The tokens that chose expert e, ascending: lane c < n has the c-th one's
// number and the first of its slots of e, which names its row of the
// activation.
struct LayerMembers {
  int n, token, slot;
};

__device__ __forceinline__ LayerMembers layer_members(const LayerArgs& A, const LayerRoutes& R, int e) {
  const int lane = threadIdx.x & (kWave - 1);
  int slot = -1;
  if (lane < A.tokens)
    for (int j = A.k - 1; j >= 0; --j)
      if (R.id[lane * A.k + j] == e) slot = lane * A.k + j;
  const unsigned long long in = __ballot(slot >= 0), below = (1ull << lane) - 1ull;
  LayerMembers M;
  M.n = __popcll(in);
  const int to = (slot >= 0 ? __popcll(in & below) : M.n + __popcll(~in & below)) * 4;
  M.token = __builtin_amdgcn_ds_permute(to, lane);
  M.slot = __builtin_amdgcn_ds_permute(to, slot);
  return M;
}

// The weight of expert e for token `slot / k`, whose first slot of e is
// `slot`: the sum over its slots of e, in slot order.
__device__ __forceinline__ float layer_weight(const LayerArgs& A, const LayerRoutes& R, int e, int slot) {
  const int end = (slot / A.k + 1) * A.k;
  float w = 0.0f;
  for (int s = slot; s < end; ++s)
    if (R.id[s] == e) w += A.w[s];
  return w;
}

__device__ __forceinline__ v8bf as_bf(const v4u& a) { return __builtin_bit_cast(v8bf, a); }
__device__ __forceinline__ v4u ld16_cached(const void* p) { return *static_cast<const v4u*>(p); }

// One 128-column block of a 16-row weight tile: lane l holds, of row l % 16,
// columns h*64 + (l/16)*16 .. + 15 for h = 0, 1.  Product (h, s) takes the
// 8 columns from h*64 + (l/16)*16 + s*8 of both operands: a permutation of
// the block's columns, the same on both sides.
//
// Plain loads: a row's 128-byte line is read by two instructions, and
// non-temporal ones took 502 us instead of 431 for the up product of 13
// tokens (2.5 GB of weights).
struct WBlock {
  v4u q[2];
};
__device__ __forceinline__ WBlock load_w(const uint8_t* p) {
  WBlock b;
  b.q[0] = ld16_cached(p);
  b.q[1] = ld16_cached(p + 64);
  return b;
}
// The same block of one token's bf16 row.
struct XBlock {
  v4u v[4];
};
__device__ __forceinline__ XBlock load_x(const uint16_t* p) {
  XBlock b;
#pragma unroll
  for (int i = 0; i < 4; ++i) b.v[i] = ld16_cached(p + (i >> 1) * 64 + (i & 1) * 8);
  return b;
}
__device__ __forceinline__ v8bf w_part(const WBlock& b, int i) {
  return widen8(b.q[i >> 1][(i & 1) * 2], b.q[i >> 1][(i & 1) * 2 + 1]);
}

// Gate and up rows of expert e, 16 of each a tile, for the tiles first,
// first + stride, ..., times the NT*16 members from c0 on.  Wave w takes
// blocks w, w + 4, ... of a tile; then the waves' sums are joined in LDS.
template <int NT>
__device__ __forceinline__ void layer_up_tiles(const LayerArgs& A, const LayerRoutes& R, int e, int first, int stride,
                                               float (*red)[2][NT * 16][17]) {
  constexpr int kXBufs = NT <= 2 ? 2 : 1;   // with more columns the tokens' blocks are loaded when needed
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int KB = A.H / kScaleBlock, IB = A.I / kScaleBlock, tiles = A.I / 16;
  const uint8_t* wexp = A.w13_q + ((int64_t)e * 2 * A.I + (lane & 15)) * A.H + (lane >> 4) * 16;
  const int64_t up = (int64_t)A.I * A.H;
  WBlock g[2], u[2];
  XBlock x[kXBufs][NT];
  auto fetch_w = [&](int slot, int tile, int kb) {
    if (kb < KB) {
      const uint8_t* p = wexp + (int64_t)tile * 16 * A.H + kb * kScaleBlock;
      g[slot] = load_w(p);
      u[slot] = load_w(p + up);
    }
  };
  // Two blocks of weights are on their way while one is multiplied, the first
  // of them before it is known which tokens they are for.
  fetch_w(0, first, wave);
  fetch_w(1, first, wave + kLayerUpWaves);
  const LayerMembers M = layer_members(A, R, e);
  for (int c0 = 0; c0 < M.n; c0 += NT * 16) {
    const uint16_t* xp[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int c = c0 + n * 16 + (lane & 15);
      xp[n] = A.x + (int64_t)__shfl(M.token, c < M.n ? c : 0) * A.H + (lane >> 4) * 16;
    }
    auto fetch_x = [&](int slot, int kb) {
      if (kb < KB)
#pragma unroll
        for (int n = 0; n < NT; ++n) x[slot][n] = load_x(xp[n] + kb * kScaleBlock);
    };
    if (c0) {
      fetch_w(0, first, wave);
      fetch_w(1, first, wave + kLayerUpWaves);
    }
    if (kXBufs == 2) {
      fetch_x(0, wave);
      fetch_x(kXBufs - 1, wave + kLayerUpWaves);
    }
    for (int tile = first; tile < tiles; tile += stride) {
      const float* sg = A.w13_s + ((int64_t)e * 2 * IB + tile / (kScaleBlock / 16)) * KB;
      const float* su = sg + (int64_t)IB * KB;
      v4f ag[NT], au[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) ag[n] = au[n] = v4f{0, 0, 0, 0};
      auto step = [&](int slot, int kb) {
        const float s0 = sg[kb], s1 = su[kb];
        if (kXBufs == 1) fetch_x(0, kb);
        const XBlock* xs = x[slot % kXBufs];
        v4f pg[NT], pu[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) pg[n] = pu[n] = v4f{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const v8bf a = w_part(g[slot], i), b = w_part(u[slot], i);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            pg[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, as_bf(xs[n].v[i]), pg[n], 0, 0, 0);
            pu[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, as_bf(xs[n].v[i]), pu[n], 0, 0, 0);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            ag[n][i] = __builtin_fmaf(pg[n][i], s0, ag[n][i]);
            au[n][i] = __builtin_fmaf(pu[n][i], s1, au[n][i]);
          }
      };
      // The block two steps on, in this tile or at the start of the next.
      auto fetch = [&](int slot, int kb) {
        const bool here = kb < KB;
        const int t = here ? tile : tile + stride, b = here ? kb : wave + slot * kLayerUpWaves;
        if (t < tiles) {
          fetch_w(slot, t, b);
          if (kXBufs == 2) fetch_x(slot % kXBufs, b);
        }
      };
      for (int kb = wave; kb < KB; kb += 2 * kLayerUpWaves) {
        step(0, kb);
        fetch(0, kb + 2 * kLayerUpWaves);
        if (kb + kLayerUpWaves < KB) step(1, kb + kLayerUpWaves);
        if (kb + kLayerUpWaves < KB || kb + 2 * kLayerUpWaves >= KB) fetch(1, kb + 3 * kLayerUpWaves);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          red[wave][0][n * 16 + (lane & 15)][(lane >> 4) * 4 + i] = ag[n][i];
          red[wave][1][n * 16 + (lane & 15)][(lane >> 4) * 4 + i] = au[n][i];
        }
      __syncthreads();
      const int r = threadIdx.x & 15;
#pragma unroll
      for (int n = 0; n < NT; ++n) {   // 256 threads: 16 members x 16 rows
        const int cl = n * 16 + threadIdx.x / 16, c = c0 + cl;
        float gt = 0.0f, upv = 0.0f;
#pragma unroll
        for (int v = 0; v < kLayerUpWaves; ++v) {
          gt += red[v][0][cl][r];
          upv += red[v][1][cl][r];
        }
        const int slot = __shfl(M.slot, c);
        if (c < M.n) {
          const float v = gt / (1.0f + __expf(-gt)) * upv * layer_weight(A, R, e, slot);
          const uint32_t hi = f32_to_bf16_rne(v);
          const float left = v - __uint_as_float(hi << 16);
          const int64_t at = (int64_t)slot * A.I + tile * 16 + r;
          A.a_hi[at] = (uint16_t)hi;
          // Infinity and NaN are in the upper part alone.
          A.a_lo[at] = (hi & 0x7F80u) == 0x7F80u ? (uint16_t)0 : (uint16_t)f32_to_bf16_rne(left);
        }
      }
      __syncthreads();   // red is read until here
    }
  }
}

// Four workgroups a compute unit (128 registers a thread): one token of 8
// experts is 1024 workgroups, which are then all resident (47 us for 235 MB
// of weights at H = 7168, I = 2048, 5.0 TB/s; 60 us with three).  13 tokens
// (104 experts at most, 2.5 GB) take 421 us, 6.0 TB/s.
template <int NT>
__global__ __launch_bounds__(kLayerUpWaves* kWave, NT == 1 ? 4 : 1) void k_layer_up(LayerArgs A) {
  __shared__ LayerRoutes R;
  __shared__ float red[kLayerUpWaves][2][NT * 16][17];
  const bool bad = layer_routes(A, R);
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    const int any = __syncthreads_or(bad);
    if (threadIdx.x == 0) *A.flags = any ? MOE_FLAG_BADID : 0u;
    for (int i = threadIdx.x; i < A.H / kLayerDownRows; i += blockDim.x) A.ticket[i] = 0;
  }
  if ((int)blockIdx.y >= R.count) return;
  const int e = __builtin_amdgcn_readfirstlane(R.experts[blockIdx.y]);
  layer_up_tiles<NT>(A, R, e, blockIdx.x, gridDim.x, red);
}

// Output rows [h0, h0 + 16*RT) of expert e over blocks [k0, k1), of the NT*16
// members from c0 on, added to the wave's own sums acc[token][16*RT].
template <int RT, int NT>
__device__ __forceinline__ void layer_down_part(const LayerArgs& A, const LayerMembers& M, int e, int h0, int k0,
                                                int k1, int c0, float* acc) {
  constexpr int kXBufs = NT == 1 ? 2 : 1;
  const int lane = threadIdx.x & (kWave - 1);
  const int IB = A.I / kScaleBlock, HB = A.H / kScaleBlock;
  const uint8_t* wp[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
    wp[r] = A.w2_q + ((int64_t)e * A.H + h0 + r * 16 + (lane & 15)) * A.I + (lane >> 4) * 16;
  const float* sp = A.w2_s + ((int64_t)e * HB + h0 / kScaleBlock) * IB;
  int64_t ap[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int c = c0 + n * 16 + (lane & 15);
    ap[n] = (int64_t)__shfl(M.slot, c < M.n ? c : 0) * A.I + (lane >> 4) * 16;
  }
  v4f o[RT][NT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n) o[r][n] = v4f{0, 0, 0, 0};
  WBlock w[2][RT];
  XBlock hi[kXBufs], lo[kXBufs];
  auto fetch = [&](int slot, int kb) {
    if (kb < k1) {
#pragma unroll
      for (int r = 0; r < RT; ++r) w[slot][r] = load_w(wp[r] + kb * kScaleBlock);
      if (kXBufs == 2) {
        hi[slot % kXBufs] = load_x(A.a_hi + ap[0] + kb * kScaleBlock);
        lo[slot % kXBufs] = load_x(A.a_lo + ap[0] + kb * kScaleBlock);
      }
    }
  };
  auto step = [&](int slot, int kb) {
    const float s = sp[kb];
    v4f p[RT][NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (kXBufs == 1) {
        hi[0] = load_x(A.a_hi + ap[n] + kb * kScaleBlock);
        lo[0] = load_x(A.a_lo + ap[n] + kb * kScaleBlock);
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        p[r][n] = v4f{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const v8bf a = w_part(w[slot][r], i);
          p[r][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, as_bf(hi[slot % kXBufs].v[i]), p[r][n], 0, 0, 0);
          p[r][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, as_bf(lo[slot % kXBufs].v[i]), p[r][n], 0, 0, 0);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[r][n][i] = __builtin_fmaf(p[r][n][i], s, o[r][n][i]);
  };
  fetch(0, k0);
  fetch(1, k0 + 1);
  for (int kb = k0; kb < k1; kb += 2) {
    step(0, kb);
    fetch(0, kb + 2);
    if (kb + 1 < k1) {
      step(1, kb + 1);
      fetch(1, kb + 3);
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int c = c0 + n * 16 + (lane & 15);
    const int token = __shfl(M.token, c);
    if (c < M.n)
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        v4f* p = reinterpret_cast<v4f*>(acc + (token * RT + r) * 16 + (lane >> 4) * 4);
        *p = *p + o[r][n];
      }
  }
}

// Workgroup (b, z) forms output rows [32 b, 32 b + 32) of every token from
// the z-th share of the weights.  The blocks of all distinct experts, expert
// after expert, are split evenly over the splits and their waves; each wave
// adds its products into LDS sums of its own, which are joined in wave order.
// With several splits the sums go to memory and the tile's last workgroup (by
// ticket) joins them in split order, so the result does not depend on timing.
//
// 31 us for one token of 8 experts (117 MB of weights), 261 us for 13 tokens
// (1.26 GB, 4.8 TB/s).  With H = 2048 there are 64 tiles, and the splits count:
// 64 tokens on 128 experts (0.53 GB) take 128 us, against 442 us with one
// workgroup of 8 waves a tile.  The activation's two halves cost 12% (232 us
// without their loads); 64 rows a workgroup gain nothing (259 us).
template <int NT>
__global__ __launch_bounds__(kLayerDownWaves* kWave) void k_layer_down(LayerArgs A) {
  constexpr int RT = kLayerDownRows / 16, kRows = kLayerDownRows;
  __shared__ LayerRoutes R;
  __shared__ int last;
  extern __shared__ __align__(16) float sums[];   // [waves][tokens][32]
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x & (kWave - 1);
  const int per = A.tokens * kRows;
  float* mine = sums + wave * per;
  for (int i = lane; i < per; i += kWave) mine[i] = 0.0f;
  layer_routes(A, R);
  const int h0 = blockIdx.x * kRows;
  const int IB = A.I / kScaleBlock;
  const int64_t all = (int64_t)R.count * IB;
  const int share = blockIdx.y * kLayerDownWaves + wave, shares = A.splits * kLayerDownWaves;
  int64_t b = all * share / shares;
  const int64_t end = all * (share + 1) / shares;
  while (b < end) {
    const int d = (int)(b / IB), k0 = (int)(b - (int64_t)d * IB);
    const int k1 = (int)min((int64_t)IB, end - (int64_t)d * IB);
    const int e = __builtin_amdgcn_readfirstlane(R.experts[d]);
    const LayerMembers M = layer_members(A, R, e);
    for (int c0 = 0; c0 < M.n; c0 += NT * 16) layer_down_part<RT, NT>(A, M, e, h0, k0, k1, c0, mine);
    b = (int64_t)d * IB + k1;
  }
  __syncthreads();
  const int64_t stride = (int64_t)gridDim.x * per;
  float* part = A.part + (int64_t)blockIdx.x * per;
  if (A.splits > 1) {
    for (int i = threadIdx.x; i < per; i += kLayerDownWaves * kWave) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kLayerDownWaves; ++w) v += sums[w * per + i];
      __hip_atomic_store(part + blockIdx.y * stride + i, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    // The stores above go through to memory (agent scope); once they are
    // acknowledged the ticket may be taken.  A fence would write back the
    // whole L2 besides.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(&A.ticket[blockIdx.x], 1) == A.splits - 1;
    __syncthreads();
    if (!last) return;
  }
  for (int i = threadIdx.x; i < per / 2; i += kLayerDownWaves * kWave) {
    float v0 = 0.0f, v1 = 0.0f;
    if (A.splits > 1) {
      for (int z = 0; z < A.splits; ++z) {
        v0 += __hip_atomic_load(part + z * stride + 2 * i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        v1 += __hip_atomic_load(part + z * stride + 2 * i + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    } else {
#pragma unroll
      for (int w = 0; w < kLayerDownWaves; ++w) {
        v0 += sums[w * per + 2 * i];
        v1 += sums[w * per + 2 * i + 1];
      }
    }
    const int t = i / (kRows / 2), c = (i - t * (kRows / 2)) * 2;
    *reinterpret_cast<uint32_t*>(A.out + (int64_t)t * A.H + h0 + c) = pack_bf16(v0, v1);
  }
}

// Workspace: tickets, the activation's two halves, the splits' sums.
struct LayerWs {
  int64_t a, part, bytes;
};
LayerWs layer_ws(int64_t tokens, int64_t slots, int H, int I, int splits) {
  auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
  LayerWs w;
  w.a = up((int64_t)sizeof(int) * kLayerMaxTiles);
  w.part = w.a + up(2 * slots * I * (int64_t)sizeof(uint16_t));
  w.bytes = w.part + up(splits > 1 ? splits * tokens * H * (int64_t)sizeof(float) : 0);
  return w;
}

// Splits of the down product: enough workgroups of 4 waves for 12 waves a
// compute unit, but at least 8 blocks of weights a wave.
int layer_splits(int64_t active, int H, int I) {
  const int64_t tiles = H / kLayerDownRows;
  const int64_t want = (768 + tiles - 1) / tiles, most = active * (I / kScaleBlock) / (8 * kLayerDownWaves);
  const int64_t s = want < most ? want : most;
  return (int)(s < 1 ? 1 : s < kLayerMaxSplits ? s : kLayerMaxSplits);
}

}  // namespace

int64_t layer_ll_workspace(const Dims& D, int I) {
  const int64_t tokens = (int64_t)D.N * D.T, slots = tokens * D.k, active = slots < D.E ? slots : D.E;
  return layer_ws(tokens, slots, D.H, I, layer_splits(active, D.H, I)).bytes;
}

int launch_layer_ll(const Dims& D, const uint16_t* x, const int* idx, const float* w, const uint8_t* w13_q,
                    const float* w13_s, const uint8_t* w2_q, const float* w2_s, int I, uint16_t* out, uint32_t* flags,
                    void* ws, hipStream_t st) {
  const int tokens = D.N * D.T, slots = tokens * D.k, active = slots < D.E ? slots : D.E;
  const int splits = layer_splits(active, D.H, I);
  const LayerWs L = layer_ws(tokens, slots, D.H, I, splits);
  char* b = static_cast<char*>(ws);
  uint16_t* a = reinterpret_cast<uint16_t*>(b + L.a);
  const LayerArgs A = {x, idx, w, w13_q, w13_s, w2_q, w2_s, out, flags, a, a + (int64_t)slots * I,
                       reinterpret_cast<float*>(b + L.part), reinterpret_cast<int*>(b), splits,
                       tokens, slots, D.k, D.E, D.H, I};
  // Columns of a pass over the weights, in tiles of 16 members, by the members
  // that an active expert has on average (at most 64).  64 tokens on 32 experts,
  // H = 7168, I = 2048 (1.4 GB of weights), the whole call in us:
  //   members                       8    12    16    24    32    48    64
  //   up of 1 tile, down of 1      346   421   545   714   914  1297  1528
  //   up of 2                      396   458   522   634   849  1198  1406
  //   up of 4                      498   562   628   744   875  1120  1317
  //   up of 1, down of 2           467   524   609   753   946  1276  1460
  //   up of 1, down of 4           489   540   632   758   910  1193  1371
  // The average decides because the host does not know the load: an expert with
  // more members than its pass has columns is read again for the rest.
  const int members = slots / active;
  const auto up = members > 32 ? k_layer_up<4> : members > 12 ? k_layer_up<2> : k_layer_up<1>;
  const auto down = members > 32 ? k_layer_down<4> : k_layer_down<1>;
  // Tiles of one expert that a workgroup takes one after the other: about 256
  // KiB of weights, as long as that leaves 2048 workgroups.
  const int tiles = I / 16;
  const int64_t most = (int64_t)tiles * active / 2048, want = (256 << 10) / (32 * D.H);
  const int turns = (int)(want < 1 || most < 1 ? 1 : want < most ? want : most);
  int rc = launch("k_layer_up", up, dim3((tiles + turns - 1) / turns, active),
                  dim3(kLayerUpWaves * kWave), 0, st, A);
  if (rc) return rc;
  return launch("k_layer_down", down, dim3(D.H / kLayerDownRows, splits),
                dim3(kLayerDownWaves * kWave), (size_t)kLayerDownWaves * tokens * kLayerDownRows * sizeof(float), st, A);
}

}  // namespace moe
