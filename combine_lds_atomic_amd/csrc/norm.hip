// Root-mean-square norm of token rows with the residual's addition in front
// and an 8-bit output behind:
//
//   r = x + residual,  n = r / sqrt(mean(r^2) + eps) * gamma,
//   res_out = bf16(r),  y = bf16(n),  y_q, y_s = block-128 e4m3 of n
//
// in float32, each output rounded once.
#include "moe_internal.h"
#include "quant_dev.h"

namespace moe {

namespace {

constexpr int kNormWaves = 4;          // rows of a workgroup when one wave takes a row
constexpr int kNormMaxThreads = 1024;
constexpr int64_t kNormLaunchRows = 1 << 21;   // rows of a launch: keeps grid.x * 1024 below 2^32

struct NormArgs {
  const uint16_t* x;
  const uint16_t* residual;   // may be null
  const uint16_t* gamma;
  uint16_t* res_out;          // may be null
  uint16_t* y;                // may be null
  uint8_t* q;                 // null together with s
  float* s;
  float eps;
  int64_t rows;
  int H;
};

constexpr int kDppRowMirror = 0x140;   // lane i <-> 15-i inside 16 lanes

// Max over each aligned group of 16 lanes.
__device__ __forceinline__ int max16_lanes(int v) {
  v = max8_lanes(v);
  return max(v, dpp_mov<kDppRowMirror>(v));
}

__device__ __forceinline__ void unpack8(const v4u& a, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(a[i]);
    f[2 * i + 1] = bf16_hi(a[i]);
  }
}

// A unit is 8 elements: 16 bytes of x.  Thread i of a row's threads takes
// units i, i + threads, ... (U of them, the last ones past the row's end
// idle).  One wave per row if WAVE (no barrier), otherwise a workgroup.
// Every read of a row comes before the first write to it, so outputs may be
// the inputs' own memory.
//
// Bound by HBM: 4 H bytes in and 5 H + H/32 out per row.  Two units a thread
// (448 threads at H = 7168) measured 679 us on 65536 rows, 6.25 TB/s, against
// a plain copy's 6.6; one unit 815 us, four 677, a wave per row (14 units)
// 790 (709 to 760 us for the first on other days).  On 4096 rows 53, 59, 56
// and 70 us.  Several rows a workgroup, one after the other with gamma kept
// and the next row's loads in flight, were slower: 744 us for one row, 784
// for four, 866 for sixteen, in one run.
template <int U, bool WAVE>
__global__ __launch_bounds__(WAVE ? kNormWaves* kWave : kNormMaxThreads) void k_rmsnorm_quant(NormArgs A) {
  __shared__ float part[kNormMaxThreads / kWave];
  const int threads = WAVE ? kWave : blockDim.x;
  const int tid = WAVE ? (threadIdx.x & (kWave - 1)) : threadIdx.x;
  const int64_t row = WAVE ? (int64_t)blockIdx.x * kNormWaves + threadIdx.x / kWave : blockIdx.x;
  if (WAVE && row >= A.rows) return;
  const int units = A.H / 8;
  const int64_t at = row * A.H;
  float r[U][8];
  float ss = 0.0f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = tid + u * threads;
    v4u a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
    if (c < units) {
      a = ld16(reinterpret_cast<const v4u*>(A.x + at) + c);
      if (A.residual) b = ld16(reinterpret_cast<const v4u*>(A.residual + at) + c);
    }
    unpack8(a, r[u]);
    if (A.residual) {
      float v[8];
      unpack8(b, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) r[u][i] += v[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(r[u][i], r[u][i], ss);
  }
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) ss += __shfl_xor(ss, d);
  if constexpr (!WAVE) {
    if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = ss;
    __syncthreads();
    ss = 0.0f;
    for (int w = 0; w < (int)blockDim.x / kWave; ++w) ss += part[w];
  }
  const float inv = 1.0f / sqrtf(ss / (float)A.H + A.eps);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = tid + u * threads;
    const bool act = c < units;
    if (A.res_out && act) {
      v4u o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = pack_bf16(r[u][2 * i], r[u][2 * i + 1]);
      st16(reinterpret_cast<v4u*>(A.res_out + at) + c, o);
    }
    float g[8];
    unpack8(act ? *(reinterpret_cast<const v4u*>(A.gamma) + c) : v4u{0, 0, 0, 0}, g);
    int am = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      r[u][i] = r[u][i] * inv * g[i];
      am = max(am, abs_bits(r[u][i]));
    }
    if (A.y && act) {
      v4u o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = pack_bf16(r[u][2 * i], r[u][2 * i + 1]);
      st16(reinterpret_cast<v4u*>(A.y + at) + c, o);
    }
    if (A.q) {
      const float scale = block_scale(max16_lanes(am));
      if (act) {
        typedef unsigned int v2u __attribute__((ext_vector_type(2)));
        const v2u o = {quant4_scaled(r[u], scale), quant4_scaled(r[u] + 4, scale)};
        __builtin_nontemporal_store(o, reinterpret_cast<v2u*>(A.q + at) + c);
        if ((c & 15) == 0) A.s[at / kScaleBlock + c / 16] = scale;
      }
    }
  }
}

}  // namespace

int launch_rmsnorm_quant(const Dims& D, const uint16_t* x, const uint16_t* residual, const uint16_t* gamma, float eps,
                         uint16_t* res_out, uint16_t* y, uint8_t* y_q, float* y_s, hipStream_t st) {
  const int64_t rows = (int64_t)D.N * D.T;
  const int units = D.H / 8;
  const char* name = "k_rmsnorm_quant";
  auto threads = [&](int u) { return dim3((units + u * kWave - 1) / (u * kWave) * kWave); };
  for (int64_t r0 = 0; r0 < rows; r0 += kNormLaunchRows) {
    const int64_t n = rows - r0 < kNormLaunchRows ? rows - r0 : kNormLaunchRows, at = r0 * D.H;
    auto from = [](auto* p, int64_t i) { return p ? p + i : p; };
    const NormArgs A = {x + at, from(residual, at), gamma, from(res_out, at), from(y, at), from(y_q, at),
                        from(y_s, at / kScaleBlock), eps, n, D.H};
    const dim3 some((uint32_t)((n + kNormWaves - 1) / kNormWaves)), all((uint32_t)n);
    int rc;
    if (units <= kWave) rc = launch(name, k_rmsnorm_quant<1, true>, some, dim3(kNormWaves * kWave), 0, st, A);
    else if (units <= 2 * kWave) rc = launch(name, k_rmsnorm_quant<2, true>, some, dim3(kNormWaves * kWave), 0, st, A);
    else if (units <= 2 * kNormMaxThreads) rc = launch(name, k_rmsnorm_quant<2, false>, all, threads(2), 0, st, A);
    else rc = launch(name, k_rmsnorm_quant<4, false>, all, threads(4), 0, st, A);
    if (rc != MOE_OK) return rc;
  }
  return MOE_OK;
}

}  // namespace moe
