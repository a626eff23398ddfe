// gemm_fp8.h -- pieces shared by the grouped products of 8-bit operands: the matrix
// instruction and the map from blocks to (expert, row tile, column tile).
#pragma once

#include "device.h"
#include "ffn_device.h"
#include "stream.h"

namespace moe {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kGroupM = 4;  // m-tiles per rasterisation patch
constexpr int kMaxExperts = 1024;
constexpr int kUnitsPerXcd = 32;  // compute units
constexpr int kBK = 128;          // K step of the tiled products: one 128-byte tile row

// One 16 x 16 x 128 product of e4m3 operands, started from zero. Inside, the
// instruction aligns each run of 8 products to the largest and drops what lies
// below 2^-13 of it, then adds the runs in fp32 (observed; the 16x16x32 form does
// the same): a run is off by at most 2^-10 of its magnitudes, of either sign,
// which is far below the 2^-4 the operands were rounded by and, over K, below
// the rounding to bf16 that follows. Widening to bf16 would keep those bits at
// half the matrix rate.
__device__ __forceinline__ f32x4 mfma_fp8(i32x8 a, i32x8 b) {
  // format 0 = e4m3 for both; zero scale operands select the unscaled form
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
}

// A block barrier behind this wave's LDS operations, not its loads.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

struct Tile {
  int e, row0, rows, ntile;  // e < 0: no tile for this block
};

// Row tiles of a bucket: none for one that does not lie in [0, rows_total), so that what
// it claims takes no place in a list that is sized for buckets that do.
template <int BM>
__device__ __forceinline__ int bucket_tiles(int off, int n, int64_t rows_total) {
  return n > 0 && off >= 0 && (int64_t)off + n <= rows_total ? (n - 1) / BM + 1 : 0;
}
// Most row tiles of buckets that do not overlap. Lists end there, so that any offsets and
// counts make a bounded list. (The entry's limits keep it below 2^23 + 2^10, so 64 lanes'
// shares, each cut to it, add up in an int.)
template <int BM>
__device__ __forceinline__ int most_tiles(int E, int64_t rows_total) {
  return (int)(rows_total / BM + (rows_total < E ? rows_total : E));
}

// Block -> tile, for tiles that share weights with their neighbours at most. The
// tiles of all experts, in patches of kGroupM m-tiles by all n-tiles, form one list;
// workgroups are dealt to the 8 XCDs round-robin and each XCD takes every eighth
// run of kGroupM tiles: the m-tiles of a long expert read the same weights through
// one L2, and the long experts' tiles, which take longer, spread over the XCDs
// (contiguous shares: decode product with hot experts 243 us). Called by the whole
// block; info: 4 ints of LDS.
template <int BM>
__device__ __forceinline__ Tile find_tile(const int32_t* __restrict__ offs,
                                          const int32_t* __restrict__ cnts, int E,
                                          int64_t rows_total, int ntiles, int* info) {
  const int lane = threadIdx.x & (kWave - 1);
  if (threadIdx.x < kWave) {
    if (lane == 0) info[0] = -1;
    const int c = (E + kWave - 1) / kWave;  // lane l scans experts [l*c, l*c + c)
    const int e0 = lane * c, e1 = (e0 + c < E) ? e0 + c : E;
    const int most = most_tiles<BM>(E, rows_total);
    const auto mtiles = [&](int e) { return bucket_tiles<BM>(offs[e], cnts[e], rows_total); };
    int mine = 0;
    for (int e = e0; e < e1; ++e) mine += mtiles(e);
    mine = mine < most ? mine : most;
    int incl = mine;
    for (int o = 1; o < kWave; o <<= 1) {
      const int y = __shfl_up(incl, o);
      if (lane >= o) incl += y;
    }
    const int all = __shfl(incl, kWave - 1), MT = all < most ? all : most;
    const int total = MT * ntiles;
    const int slot = blockIdx.x / kXCD;
    const int lin = ((slot / kGroupM) * kXCD + blockIdx.x % kXCD) * kGroupM + slot % kGroupM;
    if (lin < total) {
      const int grp = lin / (kGroupM * ntiles), r = lin - grp * kGroupM * ntiles;
      const int gh = MT - grp * kGroupM < kGroupM ? MT - grp * kGroupM : kGroupM;
      const int ntile = r / gh, mt = grp * kGroupM + (r - ntile * gh);
      int base = incl - mine;
      if (mt >= base && mt < incl) {
        for (int e = e0; e < e1; ++e) {
          const int n = mtiles(e);
          if (mt < base + n) {
            const int m0 = (mt - base) * BM;
            const int rows = cnts[e] - m0;
            info[0] = e;
            info[1] = offs[e] + m0;
            info[2] = rows < BM ? rows : BM;
            info[3] = ntile;
            break;
          }
          base += n;
        }
      }
    }
  }
  __syncthreads();
  return {__builtin_amdgcn_readfirstlane(info[0]), __builtin_amdgcn_readfirstlane(info[1]),
          __builtin_amdgcn_readfirstlane(info[2]), __builtin_amdgcn_readfirstlane(info[3])};
}

// LDS tile: rows of 128 bytes = eight 16-byte chunks; chunk c of row r sits at
// chunk c ^ key(r), so that the 16 lanes that read one chunk column of a
// fragment in the same cycle hit distinct banks (two rows span the 64 banks).
// A fragment's rows are 16 consecutive ones. B fragments come in pairs over 32
// rows, fragment h of a pair taking rows 8 (i / 4) + 4 h + i % 4, i = 0..15:
// a lane's four outputs of both are then eight consecutive columns.
__device__ __forceinline__ int a_key(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int b_key(int r) { return ((r >> 1) & 1) | (((r >> 3) & 3) << 1); }

__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t voff,
                                         int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lptr_t)lds, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void load_lds4(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t voff,
                                          int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lptr_t)lds, 4, voff, soff, 0, 0);
}

// m-tile prefix sums of the experts in LDS: pre[e] m-tiles before expert e, pre[E] in
// all (bucket_tiles says which buckets count). Called by the whole block.
template <int BM>
__device__ __forceinline__ void tile_prefix(const int32_t* __restrict__ offs,
                                            const int32_t* __restrict__ cnts, int E,
                                            int64_t rows_total, int* pre) {
  if (threadIdx.x < kWave) {
    const int lane = threadIdx.x;
    const int c = (E + kWave - 1) / kWave;  // lane l scans experts [l*c, l*c + c)
    const int e0 = lane * c, e1 = (e0 + c < E) ? e0 + c : E;
    const int most = most_tiles<BM>(E, rows_total);
    int mine = 0;
    for (int e = e0; e < e1; ++e) {
      mine += bucket_tiles<BM>(offs[e], cnts[e], rows_total);
      pre[e + 1] = mine;
    }
    mine = mine < most ? mine : most;
    int incl = mine;
    for (int o = 1; o < kWave; o <<= 1) {
      const int y = __shfl_up(incl, o);
      if (lane >= o) incl += y;
    }
    for (int e = e0; e < e1; ++e) {
      const int p = pre[e + 1] + incl - mine;
      pre[e + 1] = p < most ? p : most;
    }
    if (lane == 0) pre[0] = 0;
  }
  __syncthreads();
}

// Tile number lin of the list (patches of kGroupM m-tiles by all n-tiles). Uniform, no
// barrier.
template <int BM>
__device__ __forceinline__ Tile tile_at_place(const int* pre, const int32_t* __restrict__ offs,
                                              const int32_t* __restrict__ cnts, int E,
                                              int ntiles, int lin) {
  const int lane = threadIdx.x & (kWave - 1);
  const int MT = __builtin_amdgcn_readfirstlane(pre[E]);
  const int grp = lin / (kGroupM * ntiles), r = lin - grp * kGroupM * ntiles;
  const int gh = MT - grp * kGroupM < kGroupM ? MT - grp * kGroupM : kGroupM;
  const int ntile = r / gh, mt = grp * kGroupM + (r - ntile * gh);
  // the expert with pre[e] <= mt < pre[e + 1]: the 64th of the experts, then in it
  const int c = (E + kWave - 1) / kWave;
  const int hi = (lane + 1) * c < E ? (lane + 1) * c : E;
  const int part = __popcll(__ballot(pre[hi] <= mt));
  const int at = part * c + 1 + lane;
  const int e = part * c + __popcll(__ballot(lane < c && at <= E && pre[at < E ? at : E] <= mt));
  const int m0 = (mt - __builtin_amdgcn_readfirstlane(pre[e])) * BM;
  const int left = cnts[e] - m0;
  return {e, offs[e] + m0, left < BM ? left : BM, ntile};
}

}  // namespace moe
