// The norms around a block, fused with the block's gate and the residual's
// scale, and their gradients.  With x the block's output and rms(v) =
// sqrt(mean(v^2) + eps):
//
//   r = alpha * residual + gate * (x / rms(x) * gamma_post),  y = r / rms(r) * gamma_next
//
// and backwards, from dy and the gradient dr that reaches r from behind, with
// i1 = 1 / rms(x), i2 = 1 / rms(r), t = dy * gamma_next:
//
//   d = dr + i2 * (t - r * i2^2 * mean(t * r)),      dresidual = alpha * d
//   dgate = sum(d * gamma_post * x * i1),            dx = i1 * (gate * d * gamma_post - x * i1 * gate * dgate / H)
//   dgamma_next = sum over rows of dy * r * i2,      dgamma_post = sum over rows of gate * d * x * i1
//
// in float32, each output rounded once.
#include <algorithm>

#include "moe_internal.h"
#include "quant_dev.h"

namespace moe {

namespace {

constexpr int kMaxThreads = 1024, kMaxWaves = kMaxThreads / kWave;
constexpr int64_t kLaunchRows = 1 << 21;   // rows of a launch: keeps grid.x * 1024 below 2^32

struct BlockArgs {
  const uint16_t* dy;          // backwards: null without a next norm
  const uint16_t* dr;          // backwards: may be null
  const uint16_t* x;
  const uint16_t* residual;
  const uint16_t* gamma_post;
  const float* gate;           // may be null (1)
  const uint16_t* gamma_next;  // null without a next norm
  uint16_t* o0;                // res_out; backwards dx
  uint16_t* o1;                // y (may be null); backwards dresidual
  float* dgate;                // may be null
  float* part;                 // [workgroups][2][H] sums of dgamma_post, dgamma_next
  float alpha, eps;
  int64_t rows;
  int H;
};

__device__ __forceinline__ void unpack8(const v4u& a, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(a[i]);
    f[2 * i + 1] = bf16_hi(a[i]);
  }
}
// Elements 4h .. 4h + 3 of a unit.
__device__ __forceinline__ void unpack4(const v4u& a, int h, float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[2 * i] = bf16_lo(a[2 * h + i]);
    f[2 * i + 1] = bf16_hi(a[2 * h + i]);
  }
}
__device__ __forceinline__ v4u pack8(const float* f) {
  v4u o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = cvt_bf16(f[2 * i], f[2 * i + 1]);
  return o;
}
__device__ __forceinline__ v4u unit(const uint16_t* p, int64_t at, int c) {
  return ld16(reinterpret_cast<const v4u*>(p + at) + c);
}

// Keeps the compiler from holding what it unpacked from `v` for the next use.
__device__ __forceinline__ void forget(v4u& v) { asm volatile("" : "+v"(v)); }

// v's sum over the threads of a row, the same in all of them.  A barrier lies
// between one use of `part` and the next.
template <bool WAVE>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d);
  if constexpr (!WAVE) {
    if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = v;
    __syncthreads();
    v = 0.0f;
    for (int w = 0; w < (int)blockDim.x / kWave; ++w) v += part[w];
  }
  return v;
}

// v's value from the lane that DPP control `Ctrl` names, added.
template <int Ctrl>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float(dpp_mov<Ctrl>(__float_as_uint(v)));
}
// Over each aligned group of 8 lanes.
__device__ __forceinline__ float sum8_lanes(float v) {
  return dpp_add<kDppHalfMirror>(dpp_add<kDppQuadXor2>(dpp_add<kDppQuadXor1>(v)));
}

// Sums of eight values over the threads of a workgroup of at most 16 waves,
// as scalars.  Each of the first three steps adds halves of the wave and halves
// the values that a lane carries; from then on lane i has value i / 8.  All
// moves between lanes are register moves: through LDS the same chain took 3%
// of the gradient's time.
__device__ __forceinline__ void row_sum8(float (&v)[8], float (*part)[8]) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave, waves = blockDim.x / kWave;
  constexpr int kRowRor8 = 0x128;   // lane i <-> i ^ 8 inside 16 lanes
  float a[4], b[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[i]), __float_as_uint(v[i + 4]), false, false);
    a[i] = __uint_as_float(w[0]) + __uint_as_float(w[1]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto w = __builtin_amdgcn_permlane16_swap(__float_as_uint(a[i]), __float_as_uint(a[i + 2]), false, false);
    b[i] = __uint_as_float(w[0]) + __uint_as_float(w[1]);
  }
  const float keep = lane & 8 ? b[1] : b[0], give = lane & 8 ? b[0] : b[1];
  float s = sum8_lanes(keep + __uint_as_float(dpp_mov<kRowRor8>(__float_as_uint(give))));
  if ((lane & 7) == 0) part[wave][lane >> 3] = s;
  __syncthreads();
  s = (lane & 7) < waves ? part[lane & 7][lane >> 3] : 0.0f;
  if ((lane & 7) + 8 < waves) s += part[(lane & 7) + 8][lane >> 3];
  s = sum8_lanes(s);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(s), i * 8));
}

// A unit is 8 elements: 16 bytes.  Thread i of a row's threads takes units i,
// i + threads, ... (U of them, the last ones past the row's end idle).  One
// wave per row if WAVE (no barrier), otherwise a workgroup.  Every read of a
// row comes before the first write to it, so outputs may be the inputs' own
// memory.
//
// Bound by HBM: 8 H bytes a row, 622 to 651 us for 65536 rows of 7168 (5.8 to
// 6.0 TB/s, where a plain copy reaches 6.7); one token takes 4 us.
template <int U, bool WAVE>
__global__ __launch_bounds__(WAVE ? 4 * kWave : kMaxThreads) void k_block_norm(BlockArgs A) {
  __shared__ float p1[kMaxWaves], p2[kMaxWaves];
  const int threads = WAVE ? kWave : blockDim.x;
  const int tid = WAVE ? (threadIdx.x & (kWave - 1)) : threadIdx.x;
  const int64_t row = WAVE ? (int64_t)blockIdx.x * 4 + threadIdx.x / kWave : blockIdx.x;
  if (WAVE && row >= A.rows) return;
  const int units = A.H / 8;
  const int64_t at = row * A.H;
  const float gate = A.gate ? A.gate[row] : 1.0f;
  float x[U][8], r[U][8], s1 = 0.0f, s2 = 0.0f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = tid + u * threads;
    v4u a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
    if (c < units) {
      a = unit(A.x, at, c);
      b = unit(A.residual, at, c);
    }
    unpack8(a, x[u]);
    unpack8(b, r[u]);
#pragma unroll
    for (int i = 0; i < 8; ++i) s1 = __builtin_fmaf(x[u][i], x[u][i], s1);
  }
  s1 = row_sum<WAVE>(s1, p1);
  const float i1 = 1.0f / sqrtf(s1 / (float)A.H + A.eps);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = tid + u * threads;
    float g[8];
    unpack8(c < units ? *(reinterpret_cast<const v4u*>(A.gamma_post) + c) : v4u{0, 0, 0, 0}, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      r[u][i] = A.alpha * r[u][i] + gate * (x[u][i] * i1 * g[i]);
      s2 = __builtin_fmaf(r[u][i], r[u][i], s2);
    }
    if (c < units) st16(reinterpret_cast<v4u*>(A.o0 + at) + c, pack8(r[u]));
  }
  if (!A.o1) return;
  s2 = row_sum<WAVE>(s2, p2);
  const float i2 = 1.0f / sqrtf(s2 / (float)A.H + A.eps);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = tid + u * threads;
    if (c >= units) continue;
    float g[8];
    unpack8(*(reinterpret_cast<const v4u*>(A.gamma_next) + c), g);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[u][i] = r[u][i] * i2 * g[i];
    st16(reinterpret_cast<v4u*>(A.o1 + at) + c, pack8(r[u]));
  }
}

// Backwards: a workgroup takes rows blockIdx.x, + gridDim.x, ... and keeps its
// columns' sums of the two dgammas in registers until the last of them.  With
// KEEP a row stays in registers between its reduction and its outputs, and the
// next row's loads are issued before this one is worked on; without, both are
// too large for the registers and the row is read again.
//
// r is linear in 1 / rms(x), so one reduction of seven sums gives both roots,
// the part of t along r and dgate, where a reduction after each of them would
// be three.  The sum of r^2 comes out of its three parts.  That asks two things
// of a row: the residual and the block's term do not cancel to less than an
// eighth of the parts, and the squares of x * gamma_post, which the formula has
// only after the division by rms(x), neither leave float32 nor lose digits that
// count beside eps.  For a row that fails either, the five sums that follow the
// first root are formed from r and x / rms(x) themselves in a second reduction.
//
// Bound by HBM and, nearly as much, by its 350 vector instructions a wave and
// row: 991 to 1097 us for 65536 rows of 7168 (12 H bytes a row, 5.1 to 5.7
// TB/s).  One unit a thread leaves registers for the next row's loads; two
// units took 1146, three reductions a row 1184, and 2 workgroups a compute
// unit without loads ahead 2.4 ms, since registers went to scratch.  Rows above 8192
// are read twice: 869 to 925 us at 32768 rows of 8320 (484 at a copy's rate with one
// reading), 1270 with all of it in registers and scratch.  Both of their forms
// still send some registers to scratch, 10 with two units a thread and 80 with
// four (8192 rows of 32768: 1.51 to 1.56 ms, 2.1 TB/s; 1.3 before one of the
// sums went to LDS).
template <int U, bool KEEP>
__global__ __launch_bounds__(kMaxThreads) void k_block_norm_grad(BlockArgs A) {
  __shared__ float part[2][kMaxWaves][8], again[kMaxWaves][8];
  const int threads = blockDim.x, units = A.H / 8;
  const v4u zero = {0, 0, 0, 0};
  const float h = 1.0f / (float)A.H;
  // With four units one of the two sums is in LDS, each thread's own, else in registers.
  constexpr bool kLds = U > 2;
  __shared__ float4 lds_sum[kLds ? U * kMaxThreads * 2 : 1];
  float dgp[kLds ? 1 : U][8], dgn[U][8];
  v4u gp[KEEP ? U : 1], gn[KEEP ? U : 1];
  auto gammas = [&](int u) {
    const int c = threadIdx.x + u * threads;
    gp[KEEP ? u : 0] = c < units ? *(reinterpret_cast<const v4u*>(A.gamma_post) + c) : zero;
    gn[KEEP ? u : 0] = c < units && A.gamma_next ? *(reinterpret_cast<const v4u*>(A.gamma_next) + c) : zero;
  };
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if constexpr (KEEP) gammas(u);
#pragma unroll
    for (int i = 0; i < 8; ++i) dgp[kLds ? 0 : u][i] = dgn[u][i] = 0.0f;
    if constexpr (kLds)
#pragma unroll
      for (int i = 0; i < 2; ++i) lds_sum[(u * kMaxThreads + threadIdx.x) * 2 + i] = float4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  struct Row {
    v4u x[KEEP ? U : 1], r[KEEP ? U : 1], t[KEEP ? U : 1], d[KEEP ? U : 1];
  };
  auto read = [&](int64_t row, int u, Row& q) {
    const int c = threadIdx.x + u * threads, i = KEEP ? u : 0;
    const bool in = c < units;
    auto get = [&](const uint16_t* p) {   // what is read twice may stay in the caches
      return KEEP ? unit(p, row * A.H, c) : *(reinterpret_cast<const v4u*>(p + row * A.H) + c);
    };
    q.x[i] = in ? get(A.x) : zero;
    q.r[i] = in ? get(A.residual) : zero;
    q.t[i] = in && A.dy ? get(A.dy) : zero;
    q.d[i] = in && A.dr ? get(A.dr) : zero;
  };
  Row next;
  if (KEEP && blockIdx.x < A.rows)
#pragma unroll
    for (int u = 0; u < U; ++u) read(blockIdx.x, u, next);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x, turn ^= 1) {
    const int64_t at = row * A.H;
    const float gate = A.gate ? A.gate[row] : 1.0f;
    Row q;
    if constexpr (KEEP) {
      q = next;
      if (row + gridDim.x < A.rows)
#pragma unroll
        for (int u = 0; u < U; ++u) read(row + gridDim.x, u, next);
    }
    // What a unit needs, from the registers or again from memory.
    auto bring = [&](int u) {
      if constexpr (KEEP) {
        forget(q.x[u]);
        forget(q.r[u]);
        forget(q.t[u]);
        forget(q.d[u]);
        forget(gp[u]);
        forget(gn[u]);
      } else {
        read(row, u, q);
        gammas(u);
      }
    };
    // sums of: x x, (x gp)^2, res res, res x gp, t res, t x gp, dr x gp
    float m[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      bring(u);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float x[4], r[4], g[4], n[4], t[4], d[4];
        unpack4(q.x[KEEP ? u : 0], half, x);
        unpack4(q.r[KEEP ? u : 0], half, r);
        unpack4(gp[KEEP ? u : 0], half, g);
        unpack4(gn[KEEP ? u : 0], half, n);
        unpack4(q.t[KEEP ? u : 0], half, t);
        unpack4(q.d[KEEP ? u : 0], half, d);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float xg = x[i] * g[i], tn = t[i] * n[i];
          m[0] = __builtin_fmaf(x[i], x[i], m[0]);
          m[1] = __builtin_fmaf(xg, xg, m[1]);
          m[2] = __builtin_fmaf(r[i], r[i], m[2]);
          m[3] = __builtin_fmaf(r[i], xg, m[3]);
          m[4] = __builtin_fmaf(tn, r[i], m[4]);
          m[5] = __builtin_fmaf(tn, xg, m[5]);
          m[6] = __builtin_fmaf(d[i], xg, m[6]);
        }
        __builtin_amdgcn_sched_barrier(0);   // few numbers unpacked at a time
      }
    }
    row_sum8(m, part[turn]);
    const float i1 = rsqrtf(m[0] * h + A.eps), b = gate * i1;
    const float apart = A.alpha * A.alpha * m[2] + b * b * m[1];
    float rr = apart + 2.0f * A.alpha * b * m[3];                  // r r
    float tr = A.alpha * m[4] + b * m[5];                          // t r
    float rx = A.alpha * m[3] + b * m[1];                          // r x gp
    float lack = i1;                                               // what the sums with x gp lack of x / rms(x)
    // 2^-149 is the least step of a square, 2^-24 what counts beside eps
    const bool apart_ok = apart < __builtin_inff() && b * b * 0x1p-125f < A.eps;
    if (__builtin_expect(!(rr >= 0.125f * apart && apart_ok), 0)) {
      float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
      for (int u = 0; u < U; ++u) {   // not unrolled: what the rest keeps in registers stays there
        bring(u);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float x[4], r[4], g[4], n[4], t[4], d[4];
          unpack4(q.x[KEEP ? u : 0], half, x);
          unpack4(q.r[KEEP ? u : 0], half, r);
          unpack4(gp[KEEP ? u : 0], half, g);
          unpack4(gn[KEEP ? u : 0], half, n);
          unpack4(q.t[KEEP ? u : 0], half, t);
          unpack4(q.d[KEEP ? u : 0], half, d);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float xg = x[i] * i1 * g[i], w = A.alpha * r[i] + gate * xg, tn = t[i] * n[i];
            v[0] = __builtin_fmaf(w, w, v[0]);
            v[1] = __builtin_fmaf(tn, w, v[1]);
            v[2] = __builtin_fmaf(w, xg, v[2]);
            v[3] = __builtin_fmaf(tn, xg, v[3]);
            v[4] = __builtin_fmaf(d[i], xg, v[4]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      row_sum8(v, again);
      rr = v[0];
      tr = v[1];
      rx = v[2];
      m[5] = v[3];
      m[6] = v[4];
      lack = 1.0f;
    }
    const float i2 = rsqrtf(rr * h + A.eps);
    const float along = tr * h * i2 * i2;
    const float dg = lack * (m[6] + i2 * (m[5] - along * rx));
    if (threadIdx.x == 0 && A.dgate) A.dgate[row] = dg;
    const float k0 = i1 * i1 * gate * dg * h, k1 = i2 * along;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = threadIdx.x + u * threads;
      bring(u);
      v4u dx, dres;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float x[4], r[4], g[4], n[4], t[4], d[4];
        unpack4(q.x[KEEP ? u : 0], half, x);
        unpack4(q.r[KEEP ? u : 0], half, r);
        unpack4(gp[KEEP ? u : 0], half, g);
        unpack4(gn[KEEP ? u : 0], half, n);
        unpack4(q.t[KEEP ? u : 0], half, t);
        unpack4(q.d[KEEP ? u : 0], half, d);
        float sum[4];
        float4* mine = &lds_sum[kLds ? (u * kMaxThreads + threadIdx.x) * 2 + half : 0];
        if constexpr (kLds) *reinterpret_cast<float4*>(sum) = *mine;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          r[i] = A.alpha * r[i] + b * (x[i] * g[i]);
          d[i] = d[i] + i2 * (t[i] * n[i]) - k1 * r[i];
          float& gn_sum = dgn[u][half * 4 + i];
          float& gp_sum = kLds ? sum[i] : dgp[kLds ? 0 : u][half * 4 + i];
          gn_sum = __builtin_fmaf(t[i], r[i] * i2, gn_sum);
          const float e = b * d[i];
          gp_sum = __builtin_fmaf(e, x[i], gp_sum);
          x[i] = e * g[i] - x[i] * k0;
          d[i] *= A.alpha;
        }
        if constexpr (kLds) *mine = *reinterpret_cast<float4*>(sum);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          dx[2 * half + i] = cvt_bf16(x[2 * i], x[2 * i + 1]);
          dres[2 * half + i] = cvt_bf16(d[2 * i], d[2 * i + 1]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (c < units) {
        st16(reinterpret_cast<v4u*>(A.o0 + at) + c, dx);
        st16(reinterpret_cast<v4u*>(A.o1 + at) + c, dres);
      }
    }
  }
  float* out = A.part + (int64_t)blockIdx.x * 2 * A.H;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = threadIdx.x + u * threads;
    if (c >= units) continue;
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      if constexpr (kLds)
        *reinterpret_cast<float4*>(out + c * 8 + i) = lds_sum[(u * kMaxThreads + threadIdx.x) * 2 + i / 4];
      else
        *reinterpret_cast<float4*>(out + c * 8 + i) = float4{dgp[u][i], dgp[u][i + 1], dgp[u][i + 2], dgp[u][i + 3]};
      *reinterpret_cast<float4*>(out + A.H + c * 8 + i) =
          float4{dgn[u][i], dgn[u][i + 1], dgn[u][i + 2], dgn[u][i + 3]};
    }
  }
}

// The workgroups' sums added up, in their order: 64 columns a workgroup, its
// waves taking an equal share of the parts each, eight loads on their way.
constexpr int kJoinWaves = 16;
__global__ __launch_bounds__(kJoinWaves* kWave) void k_block_norm_join(const float* __restrict__ part, int parts,
                                                                      int H, float* __restrict__ dgamma_post,
                                                                      float* __restrict__ dgamma_next) {
  __shared__ float sum[kJoinWaves][kWave];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave, c = blockIdx.x * kWave + lane;   // c < 2H
  const int end = (int)((int64_t)parts * (wave + 1) / kJoinWaves);
  const float* at = part + c;
  float s = 0.0f;
  int p = (int)((int64_t)parts * wave / kJoinWaves);
  for (; p + 8 <= end; p += 8) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = at[(int64_t)(p + i) * 2 * H];
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[i];
  }
  for (; p < end; ++p) s += at[(int64_t)p * 2 * H];
  sum[wave][lane] = s;
  __syncthreads();
  if (wave) return;
  s = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinWaves; ++w) s += sum[w][lane];
  float* out = c < H ? dgamma_post : dgamma_next;
  if (out) out[c < H ? c : c - H] = s;
}

// Units of a thread backwards: the fewest that leave a workgroup of at most 1024
// threads.
inline int grad_units(int H) { return H <= 8 * kMaxThreads ? 1 : H <= 16 * kMaxThreads ? 2 : 4; }
inline int grad_threads(int H) {
  const int u = grad_units(H);
  return (H / 8 + u * kWave - 1) / (u * kWave) * kWave;
}

// Workgroups of the gradient's first kernel: what 256 compute units hold at
// once, but not above the larger of 256 and a quarter of the rows (so from 1024
// rows on at least four rows each, below that one to four), since the sums that
// a workgroup leaves, written and read, are as many bytes as one row and a third.
inline int64_t grad_groups(const Dims& D) {
  const int64_t rows = (int64_t)D.N * D.T, most = 256 * (1024 / grad_threads(D.H));
  if (rows <= 256) return rows;
  return std::min(std::max<int64_t>(rows / 4, 256), most);
}

}  // namespace

int64_t block_norm_grad_workspace(const Dims& D) {
  const int64_t b = grad_groups(D) * 2 * D.H * (int64_t)sizeof(float);
  return b > 256 ? b : 256;
}

int launch_block_norm(const Dims& D, const uint16_t* x, const uint16_t* residual, const uint16_t* gamma_post,
                      const float* gate, float alpha, const uint16_t* gamma_next, float eps, uint16_t* res_out,
                      uint16_t* y, hipStream_t st) {
  const int64_t rows = (int64_t)D.N * D.T;
  const int units = D.H / 8;
  const char* name = "k_block_norm";
  auto threads = [&](int u) { return dim3((units + u * kWave - 1) / (u * kWave) * kWave); };
  for (int64_t r0 = 0; r0 < rows; r0 += kLaunchRows) {
    const int64_t n = rows - r0 < kLaunchRows ? rows - r0 : kLaunchRows, at = r0 * D.H;
    BlockArgs A = {};
    A.x = x + at;
    A.residual = residual + at;
    A.gamma_post = gamma_post;
    A.gate = gate ? gate + r0 : nullptr;
    A.gamma_next = gamma_next;
    A.o0 = res_out + at;
    A.o1 = y ? y + at : nullptr;
    A.alpha = alpha;
    A.eps = eps;
    A.rows = n;
    A.H = D.H;
    const dim3 some((uint32_t)((n + 3) / 4)), all((uint32_t)n);
    int rc;
    if (units <= kWave) rc = launch(name, k_block_norm<1, true>, some, dim3(4 * kWave), 0, st, A);
    else if (units <= 2 * kWave) rc = launch(name, k_block_norm<2, true>, some, dim3(4 * kWave), 0, st, A);
    else if (units <= 2 * kMaxThreads) rc = launch(name, k_block_norm<2, false>, all, threads(2), 0, st, A);
    else rc = launch(name, k_block_norm<4, false>, all, threads(4), 0, st, A);
    if (rc != MOE_OK) return rc;
  }
  return MOE_OK;
}

int launch_block_norm_grad(const Dims& D, const uint16_t* dy, const uint16_t* dres, const uint16_t* x,
                           const uint16_t* residual, const uint16_t* gamma_post, const float* gate, float alpha,
                           const uint16_t* gamma_next, float eps, uint16_t* dx, uint16_t* dresidual, float* dgate,
                           float* dgamma_post, float* dgamma_next, void* ws, hipStream_t st) {
  BlockArgs A = {};
  A.dy = dy;
  A.dr = dres;
  A.x = x;
  A.residual = residual;
  A.gamma_post = gamma_post;
  A.gate = gate;
  A.gamma_next = gamma_next;
  A.o0 = dx;
  A.o1 = dresidual;
  A.dgate = dgate;
  A.part = static_cast<float*>(ws);
  A.alpha = alpha;
  A.eps = eps;
  A.rows = (int64_t)D.N * D.T;
  A.H = D.H;
  const int64_t groups = grad_groups(D);
  const dim3 threads(grad_threads(D.H));
  if (groups) {
    const int u = grad_units(D.H);
    const auto k = u == 1   ? k_block_norm_grad<1, true>
                   : u == 2 ? k_block_norm_grad<2, false>
                            : k_block_norm_grad<4, false>;
    const int rc = launch("k_block_norm_grad", k, dim3((uint32_t)groups), threads, 0, st, A);
    if (rc != MOE_OK) return rc;
  }
  return launch("k_block_norm_join", k_block_norm_join, dim3(2 * D.H / kWave), dim3(kJoinWaves * kWave), 0, st, A.part,
                (int)groups, D.H, dgamma_post, dgamma_next);
}

}  // namespace moe
