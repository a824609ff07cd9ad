// What the grouped products share (8-bit in gemm.hip, bfloat16 in ffn.hip):
// an expert's rows, the numbering of tiles, loads straight into LDS.
//
// Args has exp_off, N, L, E, R (ranks, experts per rank, experts, fixed region
// rows or 0), rows (of the arrays) and bn (rows of a tile at most, a multiple
// of 16).
#pragma once

#include "moe_internal.h"

namespace moe {

// Rows of expert e (rank d, l-th of the rank), and in *off its offset inside
// the rank's region.
template <class Args>
__device__ __forceinline__ int expert_rows(const Args& A, int e, int* off) {
  const int d = e / A.L, l = e - d * A.L;
  const int* eo = A.exp_off + d * (A.L + 1) + l;
  const int cap = A.R ? A.R : A.rows;
  const int a = min(max(eo[0], 0), cap), b = min(max(eo[1], a), cap);
  *off = a;
  return b - a;
}

// A workgroup's tile: up to A.bn rows of one expert and one block of features.
struct Tile {
  int e;      // expert, -1 for none
  int row;    // first row
  int n;      // rows, at most A.bn
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
template <int EPL, class Args>
__device__ __forceinline__ Tile find_tile(const Args& A, int nf) {
  const int lane = threadIdx.x & (kWave - 1);
  int n[EPL], off[EPL];
  int rows = 0, tiles = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * EPL + i;
    n[i] = expert_rows(A, min(e, A.E - 1), &off[i]);
    if (e >= A.E) n[i] = 0;
    rows += n[i];
    tiles += (n[i] + A.bn - 1) / A.bn;
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
    const int ci = (n[i] + A.bn - 1) / A.bn;
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
  const int tile = g0 + x % gs, share = min(((m + c - 1) / c + 15) & ~15, A.bn);
  const int cap = A.R ? A.R * (e / A.L + 1) : A.rows;
  T.e = e;
  T.f = x / gs;
  T.row = min(max(row + tile * share, 0), cap);
  T.n = min(min(m - tile * share, share), cap - T.row);
  return T;
}

// 16 bytes per lane straight from global memory (base + the lane's offset)
// into LDS: lane i's bytes land at dst + 16*i (dst wave-uniform).  There is no
// register result, and the wait is wait_and_barrier's: with the builtin the
// compiler waits for all of these loads before the next LDS read that follows
// one, however far apart their buffers are.  The bytes arrive after the
// statement: no wave reads them before the wait_and_barrier that follows it,
// and none overwrites what another still reads, since every stage's and scale
// buffer's last reader passed a barrier before its next load is issued.
__device__ __forceinline__ uint32_t lds_address(const void* dst) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)dst);
}
__device__ __forceinline__ void load_lds16(const void* base, uint32_t off, void* dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds_address(dst)), "v"(off),
               "s"(base)
               : "m0", "memory");
}
// The same with 4 bytes a lane.
__device__ __forceinline__ void load_lds4(const void* base, uint32_t off, void* dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(lds_address(dst)), "v"(off),
               "s"(base)
               : "m0", "memory");
}

// Wait until at most `Left` of this wave's LDS loads are on their way and all
// its LDS reads are done, then for the other waves.
template <int Left>
__device__ __forceinline__ void wait_and_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(Left) : "memory");
}

// Rows of a tile: BN, or where the tiles do not fill the compute units twice,
// the number of rows whose rounds over them cost least, a step's time being
// about as bn + 48 (1337 rows of one expert, K = 7168 -> 4096: 96 rows, 61 us;
// 67 us with 128).
inline int tile_rows(int64_t avg, int64_t active, int nf, int BN, int cus) {
  auto tiles = [&](int bn) { return active * ((avg + bn - 1) / bn) * nf; };
  if (tiles(BN) >= 2 * cus) return BN;
  int best = BN;
  int64_t least = INT64_MAX;
  for (int bn = BN; bn >= 32; bn -= 16) {
    const int64_t cost = (tiles(bn) + cus - 1) / cus * (bn + 48);
    if (cost < least) {
      least = cost;
      best = bn;
    }
  }
  return best;
}

}  // namespace moe
