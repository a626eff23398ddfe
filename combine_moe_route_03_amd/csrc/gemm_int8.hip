// gemm_int8.hip -- grouped products of 8-bit integer rows with 8-bit integer expert
// weights, a scale for each row and each column of the result, and the SwiGLU expert FFN
// made of two of them (expert compute on each expert's contiguous rows: MoE systems
// survey section 1.1, EP flow step 3; variable-size batched GEMMs driven by the counts,
// survey section 4.1).
//
//   product   out[m][n] = sa[m] sw[n] sum_j a[m][j] w[n][j],  the sum exact in 32 bits
//   gate/up   h = SiLU(g) u in fp32, g and u as above; its rows are quantised by a launch
//             of their own, since a row's scale needs all of its columns
//
// With one scale a row and a column the matrix instruction adds up all of K, and both
// scales are taken in the epilogue. The weights are the first operand: a lane then holds
// four outputs of ONE row m (n = 4 (lane / 16) + 0..3, m = lane % 16). The rows are those of
// the send buffer, or tokens picked by index on their way into LDS, so that a layer needs no
// dispatch copy.
#include <type_traits>

#include "device.h"
#include "ffn_device.h"
#include "gemm_int8.h"
#include "launch.h"

namespace moe {
namespace {

enum class Out { kBF16, kF32, kGateUp };

// Block tiles of BM x BN by WM x WN waves, each wave BM/WM x BN/WN as MI x NI
// fragments of 16 x 16; the wave's row fragments are 16 WM rows apart, so the waves
// share the rows of a partial tile evenly, and tiles of up to a quarter or a half of
// the rows run with one or two fragments a wave. N: rows of one expert's B (2 I
// for gate/up). One block a compute unit; it takes every gridDim.x / 8-th tile of
// its XCD's share of the list (contiguous, so the XCD's L2 serves its rows and
// weights), and the K steps of its tiles are one stream: the loads run NS steps
// ahead, into the next tile's first steps while this one's last run and its results are
// stored. The tiles of an XCD's last, partial round are cut into two or four by
// rows where that still gives each unit one.
//
// Two shapes. 256 x 256, two stages: the fewest loads a product, for many rows. 8192 x 4096 x
// 7168 take 175-180 us, 2.7 POP/s; in the K loop the matrix pipes are 71% busy, and the clock
// falls from 2.4 to 1.9 GHz under it: power bounds it, so what saves energy counts (the
// 32 x 32 x 32 instruction, with twice the sums' traffic a product, ran at 1.7 GHz: 213 us;
// 4 waves of 128 x 128 spill: 222). 128 x 256, three stages: twice the time for a load to land,
// for few tiles, whose steps are as long as a load takes (0.95 us with two stages, 0.5 with
// three: 1024 x 4096 x 4096 32 against 23 us), and for short experts; with many rows its 1.5
// times the loads cost more than it gains (the 8192 rows 212 us).
template <Out kOut, bool kGather, int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__(kWave * WM * WN, 1) void gemm_int8_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ Asc, const int32_t* __restrict__ idx,
    uint32_t tokens, const int32_t* __restrict__ offs, const int32_t* __restrict__ cnts, int E,
    int64_t rows_total, const uint8_t* __restrict__ B, const float* __restrict__ Bsc, int N, int K,
    void* __restrict__ C, int ntiles) {
  constexpr bool kGateUp = kOut == Out::kGateUp;
  constexpr int NW = WM * WN;
  constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
  constexpr int AI = BM / NW / 8, BI = BN / NW / 8;  // 1 KiB loads per wave per K step
  constexpr int kStage = (BM + BN) * kBK;
  constexpr int NO = kGateUp ? BN / 2 : BN;          // output columns of a tile
  static_assert(AI >= 1 && BI >= 1 && BM % 64 == 0 && NW >= (BM + BN) / 64, "tile shape");
  // separate arrays: the loads into one stage and the reads of the other do not alias
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t lds1[kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t lds2[NS == 3 ? kStage : 16];
  // scales of three tiles (one wave may still store the last while another loads the
  // next): BM rows, then BN rows of B
  __shared__ __attribute__((aligned(1024))) float scale[3][BM + BN];
  __shared__ int pre[kMaxExperts + 1];
  const auto stage = [&](auto S) -> uint8_t* {
    constexpr int V = decltype(S)::value % NS;
    if constexpr (V == 0) return lds0;
    else if constexpr (V == 1) return lds1;
    else return lds2;
  };
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wid = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wid / WN, wn = wid % WN;
  const int KB = (K + kBK - 1) / kBK, I = N / 2;

  // ---- the block's tiles: places place, place + hop, ... below limit
  tile_prefix<BM>(offs, cnts, E, rows_total, pre);
  const int total = __builtin_amdgcn_readfirstlane(pre[E]) * ntiles;
  const int per = (total + kXCD - 1) / kXCD;
  const int hop = gridDim.x / kXCD;
  const int first = blockIdx.x % kXCD * per;
  const int mine = total - first < per ? total - first : per;  // the XCD's tiles
  const int whole = mine > 0 ? mine / hop * hop : 0, rest = mine - whole;
  const int cut = rest * 4 <= hop ? 4 : (rest * 2 <= hop ? 2 : 1);
  int place = blockIdx.x / kXCD;
  // Parts first: blocks then end their tiles, and store, at different times. Not long parts
  // ahead of two rounds or more: the first loads of all blocks come from HBM at one time, and
  // a part waits for them step by step (16384 rows of 16 experts, N 2816, K 4096: 207 us,
  // 198 with them last; 24558 rows of 64, N 2048, K 1408: 105 and 108; 4096 rows of 4, N and
  // K 4096: 77 and 80).
  const bool early = KB < 16 || whole < 2 * hop;
  const bool parts = place < rest * cut;
  const int limit = parts ? whole + hop : whole;
  if (mine <= 0 || place >= limit) return;  // uniform over the block
  const auto tile_of = [&](int p) {
    if (p >= limit) return Tile{-1, 0, 0, 0};
    const bool part = parts && (early ? p < hop : p >= whole);
    const int q = part && !early ? p - whole : p;  // of the parts
    Tile t = tile_at_place<BM>(pre, offs, cnts, E, ntiles,
                               first + (part ? whole + q / cut : parts && early ? p - hop : p));
    if (part && cut > 1) {
      const int r0 = q % cut * (BM / cut), left = t.rows - r0;
      t.rows = left < BM / cut ? left : BM / cut;
      t.row0 += r0;
      if (left <= 0) t = {-1, 0, 0, 0};
    }
    return t;
  };

  // ---- loads: one wave instruction fills eight 128-byte tile rows, lane l the
  // slot l % 8 of row l / 8. The descriptors begin at the tile (of B: at its
  // first weight row), so the lanes' offsets are the same for every tile, but for rows
  // picked by index; rows past the last one are out of range and read as zeros, and so is
  // what lies past the end of a row of A in the last K step (whatever B has there then
  // adds nothing).
  struct Source {
    const uint8_t *a, *b;
    const float *as, *bs;
    uint32_t abytes, bbytes, asbytes, bsbytes;
  };
  // (No tile: the first rows and weights, which nothing uses. A descriptor is never
  // shorter than the K step's offset that is added to it, also where there are no tokens
  // and every lane's offset is outside.)
  const auto source_of = [&](const Tile& t) -> Source {
    const int n0 = t.e < 0 ? 0 : t.ntile * NO, e = t.e < 0 ? 0 : t.e;
    const int rows = t.e < 0 ? (rows_total < BM ? (int)rows_total : BM) : t.rows;
    return {kGather ? A : A + (int64_t)t.row0 * K,
            B + ((int64_t)e * N + n0) * K,
            kGather ? Asc : Asc + t.row0,
            Bsc + (int64_t)e * N + n0,
            (kGather ? (tokens ? tokens : 1) : (uint32_t)rows) * (uint32_t)K,
            (uint32_t)(N - n0) * (uint32_t)K,
            (kGather ? tokens : (uint32_t)rows) * 4,
            (uint32_t)(N - n0) * 4};
  };
  // byte offsets of the lane's rows: of its AI rows of A, of its row scale
  struct Rows {
    uint32_t a[AI], s;
  };
  const int srow = wid % (BM / 64) * 64 + lane;  // the row whose scale this lane loads
  const auto rows_of = [&](const Tile& t) -> Rows {
    Rows out;
    const auto token = [&](int r) -> uint32_t {
      if constexpr (!kGather) return (uint32_t)r;
      else return t.e >= 0 && r < t.rows ? (uint32_t)idx[t.row0 + r] : tokens;
    };
#pragma unroll
    for (int i = 0; i < AI; ++i) {
      const int r = wid * (BM / NW) + 8 * i + (lane >> 3);
      const uint32_t k = token(r);
      out.a[i] = kGather && k >= tokens ? kOutside
                                        : k * (uint32_t)K + (((lane & 7) ^ a_key(r)) << 4);
    }
    const uint32_t k = token(srow);
    out.s = kGather && k >= tokens ? kOutside : k * 4;
    return out;
  };
  uint32_t boff[BI];
#pragma unroll
  for (int i = 0; i < BI; ++i) {
    const int r = wid * (BN / NW) + 8 * i + (lane >> 3);
    const int n = kGateUp && r >= NO ? I + r - NO : r;
    boff[i] = (uint32_t)n * (uint32_t)K + (((lane & 7) ^ b_key(r)) << 4);
  }
  bool keep[AI];  // the lane's chunk of the last K step is in the row
#pragma unroll
  for (int i = 0; i < AI; ++i) {
    const int r = wid * (BM / NW) + 8 * i + (lane >> 3);
    keep[i] = (((lane & 7) ^ a_key(r)) << 4) < K - (KB - 1) * kBK;
  }
  constexpr int kLoads = AI + BI;
  Source src, after;  // of what is loaded now, and of the tile after the one computed
  Rows at, then;
  int lk = 0;         // K step that is loaded
  // load number q of the step's kLoads
  auto issue = [&](uint8_t* st, int q) __attribute__((always_inline)) {
    if (q < BI)
      load_lds(make_rsrc(src.b, src.bbytes), st + (BM + wid * (BN / NW) + 8 * q) * kBK,
               boff[q % BI], lk * kBK);
    else
      load_lds(make_rsrc(src.a, src.abytes), st + (wid * (BM / NW) + 8 * (q - BI)) * kBK,
               lk == KB - 1 && !keep[(q - BI) % AI] ? kOutside : at.a[(q - BI) % AI], lk * kBK);
  };
  // the scales of a tile, 64 a wave: the rows', then those of B's rows
  auto issue_scales = [&](const Source& src, const Rows& at, float* to) __attribute__((always_inline)) {
    if (wid < BM / 64) {
      load_lds4(make_rsrc(src.as, src.asbytes), reinterpret_cast<uint8_t*>(to + wid * 64), at.s, 0);
    } else if (wid < (BM + BN) / 64) {
      const int r = wid * 64 - BM + lane;
      load_lds4(make_rsrc(src.bs, src.bsbytes), reinterpret_cast<uint8_t*>(to + wid * 64),
                (uint32_t)(kGateUp && r >= NO ? I + r - NO : r) * 4, 0);
    }
  };
  // K >= NS steps, so the loads enter the next tile once while a tile is computed
  auto next_load = [&]() __attribute__((always_inline)) {
    const bool wrap = ++lk == KB;
    lk = wrap ? 0 : lk;
    src.a = wrap ? after.a : src.a;
    src.b = wrap ? after.b : src.b;
    src.abytes = wrap ? after.abytes : src.abytes;
    src.bbytes = wrap ? after.bbytes : src.bbytes;
    if constexpr (kGather) {
#pragma unroll
      for (int i = 0; i < AI; ++i) at.a[i] = wrap ? then.a[i] : at.a[i];
    }
  };

  // ---- fragments: lane l holds row (l % 16), chunks l / 16 and l / 16 + 4 of its
  // 128 bytes (both operands alike, so the order of k does not matter): two
  // instructions' worth. A 16-byte LDS read is served to 16 lanes at a time, eight of one
  // l / 16 and eight of the next (lanes 0-3, 12-15, 20-27 and so on): chunks of
  // neighbours that differ in bit 0 keep those apart.
  const int fi = lane & 15, fc = lane >> 4;
  const int arow = wm * 16 + fi;  // of fragment 0; the others 16 WM rows apart
  const int a0 = arow * kBK + ((fc ^ a_key(arow)) << 4);
  const int a1 = arow * kBK + (((fc + 4) ^ a_key(arow)) << 4);
  const int brow = (kGateUp ? wn * (NO / WN) : wn * (BN / WN)) + 8 * (fi >> 2) + (fi & 3);
  const int b0 = (BM + brow) * kBK + ((fc ^ b_key(brow)) << 4);
  const int b1 = (BM + brow) * kBK + (((fc + 4) ^ b_key(brow)) << 4);
  struct Frag {
    i32x4 h[2];
  };
  auto frag = [&](const uint8_t* st, int o0, int o1, int off) __attribute__((always_inline)) -> Frag {
    return {*reinterpret_cast<const i32x4*>(st + o0 + off),
            *reinterpret_cast<const i32x4*>(st + o1 + off)};
  };
  constexpr int kFragRows = 16 * WM;
  auto read_a = [&](const uint8_t* st, int mi) { return frag(st, a0, a1, mi * kFragRows * kBK); };
  // rows of B fragment ni past the wave's first: pairs of 32, four apart inside
  auto b_row = [](int ni) {
    const int q = kGateUp ? ni % (NI / 2) : ni;
    return 32 * (q >> 1) + 4 * (q & 1) + (kGateUp && ni >= NI / 2 ? NO : 0);
  };
  auto read_b = [&](const uint8_t* st, int ni) { return frag(st, b0, b1, b_row(ni) * kBK); };

  Tile tile = tile_of(place);
  i32x4 acc[NI][MI];
  Frag fa[MI], fb[4];
  // The first fragments of a step: all of A's, whichever tile comes next.
  auto first_frags = [&](const uint8_t* st) __attribute__((always_inline)) {
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) fa[mi] = read_a(st, mi);
    fb[0] = read_b(st, 0);
    fb[1] = read_b(st, 1);
  };

  // A step reads stage S. Its fragments of A and the first two fragments of B are in
  // registers already. Once a wave has read the last fragments of the stage and its
  // loads of the next step have landed, there is one barrier; the MFMAs of the last two
  // columns run behind it, so that the first fragments of the next step are read while
  // they do. The loads of the step NS on into this stage are spread: kAfter of them
  // among those MFMAs, the rest every kEvery-th MFMA of the next step. With three stages
  // those of one more step may be pending at the barrier, and, in a tile's first step
  // (behind), the last tile's stores, which were issued among them. The order is held by
  // fences: left to itself the scheduler moves half the loads to the end of the step, next
  // to their wait, and fragments next to their use (8192 x 4096 x 7168: 203 us; so 187;
  // all loads behind the barrier 192).
  constexpr int kAfter = kLoads / 2, kEvery = 4;
  constexpr int kLeast = (kOut == Out::kF32 ? NI : NI / 2) * (MI / 4);  // stores of a tile
  auto step = [&](auto ml, auto S, bool behind) __attribute__((always_inline)) {
    constexpr int ML = decltype(ml)::value, V = decltype(S)::value;
    uint8_t* cur = stage(S);
    uint8_t* nxt = stage(std::integral_constant<int, V + 1>{});
    uint8_t* end = stage(std::integral_constant<int, V + NS - 1>{});
    constexpr int kBefore = (NI - 2) * ML * 2;  // MFMAs before the barrier
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int ni = 0; ni < NI - 2; ++ni) {
      fb[(ni + 2) % 4] = read_b(cur, ni + 2);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int mi = 0; mi < ML; ++mi) {
          const int j = (ni * 2 + h) * ML + mi, q = kAfter + j / kEvery;
          acc[ni][mi] = mfma_int8(fb[ni % 4].h[h], fa[mi].h[h], acc[ni][mi]);
          if (j % kEvery == 0 && q < kLoads) issue(end, q);
        }
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_setprio(0);
#pragma unroll
    for (int q = kAfter + (kBefore + kEvery - 1) / kEvery; q < kLoads; ++q) issue(end, q);  // with few MFMAs
    next_load();
    if constexpr (NS == 2) {
      __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
    } else {
      if (behind) __builtin_amdgcn_s_waitcnt(wait_vmcnt(kLoads + kLeast));
      else __builtin_amdgcn_s_waitcnt(wait_vmcnt(kLoads));
    }
    lds_barrier();
#pragma unroll
    for (int mi = 0; mi < ML; ++mi) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int ni = NI - 2; ni < NI; ++ni)
          acc[ni][mi] = mfma_int8(fb[ni % 4].h[h], fa[mi].h[h], acc[ni][mi]);
#pragma unroll
      for (int q = 0; q < kAfter; ++q)
        if (q * ML / kAfter == mi) issue(cur, q);
      fa[mi] = read_a(nxt, mi);
      if (mi < 2) fb[mi] = read_b(nxt, mi);
      if (ML == 1) fb[1] = read_b(nxt, 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (NS == 3) {
#pragma unroll
      for (int mi = ML; mi < MI; ++mi) fa[mi] = read_a(nxt, mi);
    }
  };

  // ---- results: the stores go through descriptors over the tile's rows, whose
  // range check drops the rows past the last one. sc: the tile's scales.
  auto finish = [&](auto ml, const float* sc) __attribute__((always_inline)) {
    constexpr int ML = decltype(ml)::value;
    const int g = lane >> 4;
    const int ncol = tile.ntile * NO + wn * (NO / WN);  // the wave's first output column
    float sa[ML];
#pragma unroll
    for (int mi = 0; mi < ML; ++mi) sa[mi] = sc[arow + mi * kFragRows];
    // scales of the lane's columns in fragment ni
    const auto cols = [&](int ni) {
      const int r = (kGateUp ? wn * (NO / WN) : wn * (BN / WN)) + b_row(ni) + 8 * g;
      return *reinterpret_cast<const f32x4*>(sc + BM + r);
    };
    if constexpr (kOut == Out::kBF16) {
      const __amdgpu_buffer_rsrc_t crsrc = make_rsrc(
          static_cast<uint16_t*>(C) + (int64_t)tile.row0 * N, (int64_t)tile.rows * N * 2);
      // Lanes 8 apart swap halves, so that one store is 8 rows of whole 128-byte lines
      // instead of 16 rows of half ones, and the lines go past the caches, which keep
      // operands.
      const bool low = (lane & 8) == 0;
      const int row = wm * 16 + (fi & 7);
#pragma unroll
      for (int p = 0; p < NI / 2; p += 2) {
        const int n = ncol + 32 * p + 8 * g + (low ? 0 : 32);
        f32x4 sw[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) sw[q] = cols(2 * p + q);
#pragma unroll
        for (int mi = 0; mi < ML; ++mi) {
          v4u v[2];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const i32x4 lo = acc[2 * (p + q)][mi], hi = acc[2 * (p + q) + 1][mi];
            const f32x4 wl = sw[2 * q], wh = sw[2 * q + 1];
            const auto two = [&](const i32x4& s, const f32x4& w, int r) {
              return bf16x2_rne(scaled(s[r], sa[mi], w[r]), scaled(s[r + 1], sa[mi], w[r + 1]));
            };
            v[q] = v4u{two(lo, wl, 0), two(lo, wl, 2), two(hi, wh, 0), two(hi, wh, 2)};
          }
          v4u top, bottom;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t give = low ? v[1][j] : v[0][j];
            const uint32_t got = (uint32_t)__builtin_amdgcn_mov_dpp((int)give, 0x128, 0xF, 0xF, true);
            top[j] = low ? v[0][j] : got;
            bottom[j] = low ? got : v[1][j];
          }
          // columns past N would wrap into the next row: offset out of range instead
          const uint32_t to = ((uint32_t)(row + mi * kFragRows) * (uint32_t)N + n) * 2;
          __builtin_amdgcn_raw_buffer_store_b128(top, crsrc, n < N ? to : kOutside, 0, kStream);
          __builtin_amdgcn_raw_buffer_store_b128(bottom, crsrc, n < N ? to + 16 * (uint32_t)N : kOutside,
                                                 0, kStream);
        }
      }
    } else {
      const int width = kGateUp ? I : N;
      const __amdgpu_buffer_rsrc_t crsrc = make_rsrc(
          static_cast<float*>(C) + (int64_t)tile.row0 * width, (int64_t)tile.rows * width * 4);
      constexpr int NF = kGateUp ? NI / 2 : NI;  // fragments of output columns
#pragma unroll
      for (int ni = 0; ni < NF; ++ni) {
        const int n = ncol + 32 * (ni >> 1) + 4 * (ni & 1) + 8 * g;
        const f32x4 sw = cols(ni), su = cols(kGateUp ? ni + NI / 2 : ni);
#pragma unroll
        for (int mi = 0; mi < ML; ++mi) {
          f32x4 o;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            o[r] = scaled(acc[ni][mi][r], sa[mi], sw[r]);
            if constexpr (kGateUp)
              o[r] = silu(o[r]) * scaled(acc[ni + NI / 2][mi][r], sa[mi], su[r]);
          }
          const uint32_t to = ((uint32_t)(arow + mi * kFragRows) * (uint32_t)width + n) * 4;
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, o), crsrc,
                                                 n < width ? to : kOutside, 0, 0);
        }
      }
    }
  };
  // The first NS - 1 steps and the first kAfter loads of one more, then tile by tile; par: the
  // stage of the tile's first step.
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  src = after = source_of(tile);
  at = then = rows_of(tile);
  issue_scales(src, at, scale[0]);
#pragma unroll
  for (int q = 0; q < kLoads; ++q) issue(lds0, q);
  next_load();
  if constexpr (NS == 3) {
#pragma unroll
    for (int q = 0; q < kLoads; ++q) issue(lds1, q);
    next_load();
  }
#pragma unroll
  for (int q = 0; q < kAfter; ++q) issue(NS == 3 ? lds2 : lds1, q);
  __builtin_amdgcn_s_waitcnt(wait_vmcnt(kLoads * (NS - 2) + kAfter));
  __syncthreads();
  if constexpr (NS == 3) first_frags(lds0);
  bool behind = false;  // a tile's stores are behind the loads of the next step
  for (int par = 0, spar = 0;; spar = spar == 2 ? 0 : spar + 1) {
    const Tile ahead = tile_of(place + hop);
    after = source_of(ahead);
    if constexpr (kGather) then = rows_of(ahead);
    auto compute = [&](auto ml) __attribute__((always_inline)) {
      constexpr int ML = decltype(ml)::value;
      if constexpr (NS == 2) first_frags(par ? lds1 : lds0);
#pragma unroll
      for (int ni = 0; ni < NI; ++ni)
#pragma unroll
        for (int mi = 0; mi < ML; ++mi) acc[ni][mi] = i32x4{0, 0, 0, 0};
      issue_scales(after, then, scale[spar == 2 ? 0 : spar + 1]);
      int kt = 0;
      if constexpr (NS == 2) {
        if (par) {
          step(ml, I1{}, false);
          ++kt;
        }
        for (; kt + 2 <= KB; kt += 2) {
          step(ml, I0{}, false);
          step(ml, I1{}, false);
        }
        if (kt < KB) step(ml, I0{}, false);
        // The loads that run ahead land here, where it costs the least: past this point
        // nothing is pending in either stage, whichever the next tile begins with.
        __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
      } else {
        if (par == 1) {
          step(ml, I1{}, behind);
          step(ml, I2{}, false);
          kt = 2;
        } else if (par == 2) {
          step(ml, I2{}, behind);
          kt = 1;
        }
        for (; kt + 3 <= KB; kt += 3) {
          step(ml, I0{}, behind && kt == 0);
          step(ml, I1{}, false);
          step(ml, I2{}, false);
        }
        if (kt < KB) {
          step(ml, I0{}, false);
          if (kt + 1 < KB) step(ml, I1{}, false);
        }
      }
      finish(ml, scale[spar]);
    };
    if (tile.rows > BM / 2) compute(std::integral_constant<int, MI>{});
    else if (tile.rows > BM / 4) compute(std::integral_constant<int, MI / 2>{});
    else compute(std::integral_constant<int, MI / 4>{});
    par = (par + KB) % NS;
    behind = true;
    place += hop;
    if (place >= limit) break;
    tile = ahead;
  }
  // the trailing loads must land before the block's LDS is released
  __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
}

template <Out kOut, bool kGather, int BM, int WM, int WN, int NS>
hipError_t run_gemm(const Int8Rows& a, int64_t rows, int E, const int32_t* offs,
                    const int32_t* cnts, const void* w, const float* wsc, int N, int K, void* c,
                    hipStream_t s) {
  constexpr int BN = 256;
  constexpr int NO = kOut == Out::kGateUp ? BN / 2 : BN;
  const int cols = kOut == Out::kGateUp ? N / 2 : N;
  const int ntiles = (cols + NO - 1) / NO;
  // every expert with rows adds at most one partial m-tile
  const int64_t mt = rows / BM + (rows < E ? rows : E);
  // one block a compute unit (a tile alone on its XCD is cut into four)
  int64_t per = 4 * ((mt * ntiles + kXCD - 1) / kXCD);
  if (per > kUnitsPerXcd) per = kUnitsPerXcd;
  return launch(gemm_int8_kernel<kOut, kGather, BM, BN, WM, WN, NS>, dim3((unsigned)(per * kXCD)),
                dim3(kWave * 8), 0, s, static_cast<const uint8_t*>(a.q), a.scale, a.index,
                (uint32_t)a.rows, offs, cnts, E, rows, static_cast<const uint8_t*>(w), wsc, N, K, c,
                ntiles);
}

hipError_t gemm(Out out, const Int8Rows& a, int64_t rows, int E, const int32_t* offs,
                const int32_t* cnts, const void* w, const float* wsc, int N, int K, void* c,
                hipStream_t s) {
  if (gemm_int8_streams(rows, E, N, K))
    return launch_gemm_int8_stream(out == Out::kGateUp, out != Out::kBF16, a, rows, E, offs, cnts, w,
                                   wsc, N, K, c, s);
  // Tiles of 128 rows where they are one round of the units at most (half a tile more an expert
  // on average), or the experts have no more rows than that; the stream of loads is at least as
  // many steps long as there are stages. 128 against 256 rows a tile (us), even routing:
  //   N, K 4096, one expert: 1992 rows, 256 tiles 31.8, 36.1; 2504 rows, 320 tiles 47.0, 42.3
  //   N 4096, K 1024: 13.4, 14.6; 18.1, 17.3        K 7168: 53.8, 68.7; 78.4, 69.2
  //   N 4096, K 7168, 8 experts of 160 rows, 256 tiles 49.4, 60.7; of 288 rows 84.6, 81.2
  //   N 2816, K 4096, 64 experts of 128 rows 168, 183; of 160 196, 200; of 224 217, 210
  //   N 2048, K 1408, 64 experts of 128 rows 36.6, 41.4; of 160 45.4, 43.9; of 224 50.3, 48.2
  const int64_t tiles = (rows + 64 * (rows < E ? rows : E)) / 128 * ((N + 255) / 256);
  const bool small = K > 256 && (rows <= (int64_t)128 * E || tiles <= kUnitsPerXcd * kXCD);
  const auto of = [&](auto o) {
    constexpr Out O = decltype(o)::value;
    if (small)
      return a.index ? run_gemm<O, true, 128, 2, 4, 3>(a, rows, E, offs, cnts, w, wsc, N, K, c, s)
                     : run_gemm<O, false, 128, 2, 4, 3>(a, rows, E, offs, cnts, w, wsc, N, K, c, s);
    return a.index ? run_gemm<O, true, 256, 4, 2, 2>(a, rows, E, offs, cnts, w, wsc, N, K, c, s)
                   : run_gemm<O, false, 256, 4, 2, 2>(a, rows, E, offs, cnts, w, wsc, N, K, c, s);
  };
  if (out == Out::kGateUp) return of(std::integral_constant<Out, Out::kGateUp>{});
  return out == Out::kF32 ? of(std::integral_constant<Out, Out::kF32>{})
                          : of(std::integral_constant<Out, Out::kBF16>{});
}

}  // namespace

hipError_t launch_gemm_int8(const Int8Rows& a, int64_t rows, int E, const int32_t* offs,
                            const int32_t* cnts, const void* w, const float* wsc, int N, int K,
                            int out_dtype, void* out, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  return gemm(out_dtype == MOE_F32 ? Out::kF32 : Out::kBF16, a, rows, E, offs, cnts, w, wsc, N, K,
              out, s);
}

hipError_t launch_expert_swiglu_int8(const Int8Rows& a, int64_t rows, int H, int I, int E,
                                     const int32_t* offs, const int32_t* cnts,
                                     const void* w_gate_up, const float* gsc, const void* w_down,
                                     const float* dsc, float* h, void* hq, float* hs, void* out,
                                     hipStream_t s) {
  if (rows == 0) return hipSuccess;
  hipError_t err = gemm(Out::kGateUp, a, rows, E, offs, cnts, w_gate_up, gsc, 2 * I, H, h, s);
  if (err != hipSuccess) return err;
  if (rows <= kInnerRows && I <= kInnerCols)  // the second product makes them integers
    return launch_gemm_int8_inner(h, rows, E, offs, cnts, w_down, dsc, H, I, out, s);
  err = launch_quantize_int8(h, MOE_F32, rows, I, hq, hs, s);
  if (err != hipSuccess) return err;
  return gemm(Out::kBF16, {hq, hs, nullptr, rows}, rows, E, offs, cnts, w_down, dsc, H, I, out, s);
}

}  // namespace moe
