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
__device__ __forceinline__ v4u pack8(const float* f) {
  v4u o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
  return o;
}
__device__ __forceinline__ v4u unit(const uint16_t* p, int64_t at, int c) {
  return ld16(reinterpret_cast<const v4u*>(p + at) + c);
}

// Sums of V values over the threads of a row, the same in all of them.  `part`
// is used by one sum of a row only.
template <int V, bool WAVE>
__device__ __forceinline__ void row_sum(float (&v)[V], float (*part)[V]) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1)
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += __shfl_xor(v[i], d);
  if constexpr (!WAVE) {
    if ((threadIdx.x & (kWave - 1)) == 0)
#pragma unroll
      for (int i = 0; i < V; ++i) part[threadIdx.x / kWave][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.0f;
    for (int w = 0; w < (int)blockDim.x / kWave; ++w)
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += part[w][i];
  }
}

// A unit is 8 elements: 16 bytes.  Thread i of a row's threads takes units i,
// i + threads, ... (U of them, the last ones past the row's end idle).  One
// wave per row if WAVE (no barrier), otherwise a workgroup.  Every read of a
// row comes before the first write to it, so outputs may be the inputs' own
// memory.
template <int U, bool WAVE>
__global__ __launch_bounds__(WAVE ? 4 * kWave : kMaxThreads) void k_block_norm(BlockArgs A) {
  __shared__ float p1[kMaxWaves][1], p2[kMaxWaves][1];
  const int threads = WAVE ? kWave : blockDim.x;
  const int tid = WAVE ? (threadIdx.x & (kWave - 1)) : threadIdx.x;
  const int64_t row = WAVE ? (int64_t)blockIdx.x * 4 + threadIdx.x / kWave : blockIdx.x;
  if (WAVE && row >= A.rows) return;
  const int units = A.H / 8;
  const int64_t at = row * A.H;
  const float gate = A.gate ? A.gate[row] : 1.0f;
  float x[U][8], r[U][8], s1[1] = {0.0f}, s2[1] = {0.0f};
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
    for (int i = 0; i < 8; ++i) s1[0] = __builtin_fmaf(x[u][i], x[u][i], s1[0]);
  }
  row_sum<1, WAVE>(s1, p1);
  const float i1 = 1.0f / sqrtf(s1[0] / (float)A.H + A.eps);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = tid + u * threads;
    float g[8];
    unpack8(c < units ? *(reinterpret_cast<const v4u*>(A.gamma_post) + c) : v4u{0, 0, 0, 0}, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      r[u][i] = A.alpha * r[u][i] + gate * (x[u][i] * i1 * g[i]);
      s2[0] = __builtin_fmaf(r[u][i], r[u][i], s2[0]);
    }
    if (c < units) st16(reinterpret_cast<v4u*>(A.o0 + at) + c, pack8(r[u]));
  }
  if (!A.o1) return;
  row_sum<1, WAVE>(s2, p2);
  const float i2 = 1.0f / sqrtf(s2[0] / (float)A.H + A.eps);
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
// columns' sums of the two dgammas in registers until the last of them.
template <int U>
__global__ __launch_bounds__(kMaxThreads) void k_block_norm_grad(BlockArgs A) {
  __shared__ float p1[kMaxWaves][1], p2[kMaxWaves][2], p3[kMaxWaves][1];
  const int threads = blockDim.x, units = A.H / 8;
  float dgp[U][8], dgn[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) dgp[u][i] = dgn[u][i] = 0.0f;
  for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x) {
    const int64_t at = row * A.H;
    const float gate = A.gate ? A.gate[row] : 1.0f;
    float x[U][8], r[U][8], t[U][8], d[U][8], s1[1] = {0.0f}, s2[2] = {0.0f, 0.0f}, s3[1] = {0.0f};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = threadIdx.x + u * threads;
      const v4u zero = {0, 0, 0, 0};
      unpack8(c < units ? unit(A.x, at, c) : zero, x[u]);
      unpack8(c < units ? unit(A.residual, at, c) : zero, r[u]);
      unpack8(c < units && A.dy ? unit(A.dy, at, c) : zero, t[u]);
      unpack8(c < units && A.dr ? unit(A.dr, at, c) : zero, d[u]);
#pragma unroll
      for (int i = 0; i < 8; ++i) s1[0] = __builtin_fmaf(x[u][i], x[u][i], s1[0]);
    }
    row_sum<1, false>(s1, p1);
    const float i1 = 1.0f / sqrtf(s1[0] / (float)A.H + A.eps);
    float gp[U][8], gn[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = threadIdx.x + u * threads;
      const v4u zero = {0, 0, 0, 0};
      unpack8(c < units ? *(reinterpret_cast<const v4u*>(A.gamma_post) + c) : zero, gp[u]);
      unpack8(c < units && A.gamma_next ? *(reinterpret_cast<const v4u*>(A.gamma_next) + c) : zero, gn[u]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[u][i] *= i1;
        r[u][i] = A.alpha * r[u][i] + gate * (x[u][i] * gp[u][i]);
        s2[0] = __builtin_fmaf(r[u][i], r[u][i], s2[0]);
        s2[1] = __builtin_fmaf(t[u][i] * gn[u][i], r[u][i], s2[1]);
      }
    }
    row_sum<2, false>(s2, p2);
    const float i2 = 1.0f / sqrtf(s2[0] / (float)A.H + A.eps), along = s2[1] / (float)A.H * i2 * i2;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[u][i] += i2 * (t[u][i] * gn[u][i] - r[u][i] * along);
        s3[0] = __builtin_fmaf(d[u][i] * gp[u][i], x[u][i], s3[0]);
        dgn[u][i] = __builtin_fmaf(t[u][i], r[u][i] * i2, dgn[u][i]);
        dgp[u][i] = __builtin_fmaf(gate * d[u][i], x[u][i], dgp[u][i]);
      }
    row_sum<1, false>(s3, p3);
    if (threadIdx.x == 0 && A.dgate) A.dgate[row] = s3[0];
    const float part = gate * s3[0] / (float)A.H;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = threadIdx.x + u * threads;
      if (c >= units) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[u][i] = i1 * (gate * d[u][i] * gp[u][i] - x[u][i] * part);
        d[u][i] *= A.alpha;
      }
      st16(reinterpret_cast<v4u*>(A.o0 + at) + c, pack8(x[u]));
      st16(reinterpret_cast<v4u*>(A.o1 + at) + c, pack8(d[u]));
    }
  }
  float* out = A.part + (int64_t)blockIdx.x * 2 * A.H;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = threadIdx.x + u * threads;
    if (c >= units) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      out[c * 8 + i] = dgp[u][i];
      out[A.H + c * 8 + i] = dgn[u][i];
    }
  }
}

// The workgroups' sums added up, in their order: 64 columns a workgroup, its
// four waves taking a quarter of the parts each.
__global__ __launch_bounds__(256) void k_block_norm_join(const float* __restrict__ part, int parts, int H,
                                                        float* __restrict__ dgamma_post,
                                                        float* __restrict__ dgamma_next) {
  __shared__ float sum[4][kWave];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave, c = blockIdx.x * kWave + lane;   // c < 2H
  float s = 0.0f;
  for (int p = parts * wave / 4; p < parts * (wave + 1) / 4; ++p) s += part[(int64_t)p * 2 * H + c];
  sum[wave][lane] = s;
  __syncthreads();
  if (wave) return;
  s = sum[0][lane] + sum[1][lane] + sum[2][lane] + sum[3][lane];
  float* out = c < H ? dgamma_post : dgamma_next;
  if (out) out[c < H ? c : c - H] = s;
}

inline int grad_threads(int H) {
  const int units = H / 8, u = units <= 2 * kMaxThreads ? 2 : 4;
  return (units + u * kWave - 1) / (u * kWave) * kWave;
}

// Workgroups of the gradient's first kernel: what 256 compute units hold at once.
inline int64_t grad_groups(const Dims& D) {
  const int64_t rows = (int64_t)D.N * D.T, most = 256 * (2048 / grad_threads(D.H));
  return rows < most ? rows : most;
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
    const int rc = D.H / 8 <= 2 * kMaxThreads
                       ? launch("k_block_norm_grad", k_block_norm_grad<2>, dim3((uint32_t)groups), threads, 0, st, A)
                       : launch("k_block_norm_grad", k_block_norm_grad<4>, dim3((uint32_t)groups), threads, 0, st, A);
    if (rc != MOE_OK) return rc;
  }
  return launch("k_block_norm_join", k_block_norm_join, dim3(2 * D.H / kWave), dim3(256), 0, st, A.part, (int)groups,
                D.H, dgamma_post, dgamma_next);
}

}  // namespace moe
