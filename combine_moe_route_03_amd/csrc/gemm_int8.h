// gemm_int8.h -- pieces shared by the grouped products of 8-bit integer operands.
#pragma once

#include "device.h"
#include "gemm_fp8.h"

namespace moe {

// One 16 x 16 x 64 product of 8-bit integers added to 32-bit sums, exact: lane l holds 16
// columns from 16 (l / 16) on of row l % 16 of each operand, and of the result rows
// 4 (l / 16) + 0..3 of the first operand, column l % 16 (the second's row).
__device__ __forceinline__ i32x4 mfma_int8(i32x4 a, i32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// find_tile (gemm_fp8.h) by every wave for itself: C experts a lane, all of them loaded at once,
// and no trip through LDS. E <= 64 C. A block of few rows lives for about 5 us, of which
// find_tile's dependent loads and barrier took one.
struct WaveTile {
  int e, row0, rows, ntile;  // e < 0: no tile for this block
  int len;                   // rows of the expert
};
template <int BM, int C>
__device__ __forceinline__ WaveTile find_tile_wave(const int32_t* __restrict__ offs,
                                               const int32_t* __restrict__ cnts, int E,
                                               int64_t rows_total, int ntiles) {
  const int lane = threadIdx.x & (kWave - 1);
  int o[C], n[C], t[C], mine = 0;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int e = lane * C + i;
    o[i] = e < E ? offs[e] : 0;
    n[i] = e < E ? cnts[e] : 0;
  }
  const int most = most_tiles<BM>(E, rows_total);
#pragma unroll
  for (int i = 0; i < C; ++i) {
    t[i] = bucket_tiles<BM>(o[i], n[i], rows_total);
    mine += t[i];
  }
  mine = mine < most ? mine : most;
  int incl = mine;
  for (int d = 1; d < kWave; d <<= 1) {
    const int y = __shfl_up(incl, d);
    if (lane >= d) incl += y;
  }
  const int all = lane_value(incl, kWave - 1), MT = all < most ? all : most;
  const int slot = blockIdx.x / kXCD;
  const int lin = ((slot / kGroupM) * kXCD + blockIdx.x % kXCD) * kGroupM + slot % kGroupM;
  if (lin >= MT * ntiles) return {-1, 0, 0, 0, 0};
  const int grp = lin / (kGroupM * ntiles), r = lin - grp * kGroupM * ntiles;
  const int gh = MT - grp * kGroupM < kGroupM ? MT - grp * kGroupM : kGroupM;
  const int ntile = r / gh, mt = grp * kGroupM + (r - ntile * gh);
  // the lane of the tile's expert: it knows the rest
  int base = incl - mine, e = -1, row0 = 0, rows = 0, len = 0;
  const uint64_t has = __ballot(mt >= base && mt < incl);
  if (has == 0) return {-1, 0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < C; ++i) {
    if (mt >= base && mt < base + t[i]) {
      const int m0 = (mt - base) * BM, left = n[i] - m0;
      e = lane * C + i;
      row0 = o[i] + m0;
      rows = left < BM ? left : BM;
      len = n[i];
    }
    base += t[i];
  }
  const int at = __builtin_ctzll(has);
  return {lane_value(e, at), lane_value(row0, at), lane_value(rows, at), ntile, lane_value(len, at)};
}

// A sum with the scales of its row and its column, each product rounded to fp32.
__device__ __forceinline__ float scaled(int sum, float row_scale, float col_scale) {
  return (float)sum * row_scale * col_scale;
}

}  // namespace moe
