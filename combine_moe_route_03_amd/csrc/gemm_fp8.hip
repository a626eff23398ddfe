// gemm_fp8.hip -- grouped products of 8-bit rows with 8-bit expert weights, each
// operand e4m3 with an fp32 scale per block of 128 (rows: 1 x 128, weights:
// 128 x 128), and the SwiGLU expert FFN made of two of them (expert compute on
// each expert's contiguous rows: MoE systems survey section 1.1, EP flow step
// 3; variable-size batched GEMMs driven by the counts, survey section 4.1).
//
//   product    out[m][n] = bf16( sum_b sa[m][b] sw[n/128][b] P_b[m][n] ),
//              P_b[m][n] = sum over the 128 columns j of block b of a[m][j] w[n][j]
//   gate/up    g, u as above; h = SiLU(g) u; hq, hs = the row quantisation of h
//              (quant.h), written instead of a bf16 intermediate
//
// v_mfma_f32_16x16x128_f8f6f4 makes one P_b for 16 x 16 outputs in one
// instruction, started from zero, and the vector unit folds it into the fp32
// accumulators with one fused multiply-add an output while the next product
// runs, so scales need not be powers of two (gemm_fp8.h says how exact the product is).
// The factor of the fold is sa sw rounded to fp32, hence the range that the header asks
// of it. The weights are the first operand: a lane then holds four outputs of ONE row m
// (n = 4 (lane / 16) + 0..3, m = lane % 16), so the row scale is one register
// a lane, the weight scale is uniform, and stores are 16 bytes a lane.
//
// Bound by the K loop: 8192 x 4096 x 7168 takes 196-213 us, 2.3-2.4 PFLOP/s, the
// matrix pipes 54% busy. Of 229 us, before the results were stored past the caches,
// timing-only copies took 178 without the loads into LDS, 153 without loads and folds;
// the matrix instructions alone would take 109.
// The FFN of 16384 rows, 16 experts, H 4096, I 1408: 353-367 us (gate/up 244, down
// 120), 1.55-1.6 PFLOP/s.
#include <type_traits>

#include "device.h"
#include "ffn_device.h"
#include "gemm_fp8.h"
#include "launch.h"
#include "quant.h"

namespace moe {
namespace {

static_assert(kBK == kQuantBlock, "a K step is one scale block");

// Block tiles of BM x BN by WM x WN waves, each wave BM/WM x BN/WN as MI x NI
// fragments of 16 x 16; the wave's row fragments are 16 WM rows apart, so the waves
// share the rows of a partial tile evenly, and tiles of up to a quarter or a half of
// the rows run with one or two fragments a wave. N: rows of one expert's B (2 I
// for gate/up). One block a compute unit; it takes every gridDim.x / 8-th tile of
// its XCD's share of the list (contiguous, so the XCD's L2 serves its rows and
// weights), and the K steps of its tiles are one stream: the loads run two steps
// ahead, into the next tile's first steps while this one's last run and its results are
// stored. The tiles of an XCD's last, partial round are cut into two or four by
// rows where that still gives each unit one, and come first: blocks then end their
// tiles, and store, at different times (24558 rows of 64 experts, N 2048, K 1408:
// 118 us with them last, 114 so).
template <bool kGateUp, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(kWave * WM * WN, 1) void gemm_fp8_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ Asc,
    const int32_t* __restrict__ offs, const int32_t* __restrict__ cnts, int E,
    int64_t rows_total, const uint8_t* __restrict__ B, const float* __restrict__ Bsc, int N, int K,
    void* __restrict__ C, float* __restrict__ Csc, int ntiles) {
  constexpr int NW = WM * WN;
  constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
  constexpr int AI = BM / NW / 8, BI = BN / NW / 8;  // 1 KiB loads per wave per K step
  constexpr int kStage = (BM + BN) * kBK + BM * 4;   // A, B, A scales
  constexpr int NO = kGateUp ? BN / 2 : BN;          // output columns of a tile
  static_assert(AI >= 1 && BI >= 1 && BM % 64 == 0 && BN / WN <= 128, "tile shape");
  static_assert(!kGateUp || (NO == kQuantBlock && NI % 4 == 0), "one scale block of h per tile");
  // separate arrays: the loads into one stage and the reads of the other do not alias
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t lds1[kStage];
  __shared__ uint32_t ex[kGateUp ? WN * BM : 1];  // row maxima of h, a wave column each
  __shared__ int pre[kMaxExperts + 1];
  const auto stage = [&](auto S) -> uint8_t* {
    if constexpr (decltype(S)::value % 2 == 0) return lds0;
    else return lds1;
  };
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wid = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wid / WN, wn = wid % WN;
  const int KB = K / kBK, I = N / 2, NB = (N + kQuantBlock - 1) / kQuantBlock;

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
  const bool begins = place < rest * cut;  // with a part of a tile; then the whole rounds
  const int limit = begins ? whole + hop : whole;
  if (mine <= 0 || place >= limit) return;  // uniform over the block
  const auto tile_of = [&](int p) {
    if (p >= limit) return Tile{-1, 0, 0, 0};
    const bool part = begins && p < hop;
    Tile t = tile_at_place<BM>(pre, offs, cnts, E, ntiles,
                               first + (part ? whole + p / cut : begins ? p - hop : p));
    if (part && cut > 1) {
      const int r0 = p % cut * (BM / cut), left = t.rows - r0;
      t.rows = left < BM / cut ? left : BM / cut;
      t.row0 += r0;
      if (left <= 0) t = {-1, 0, 0, 0};
    }
    return t;
  };

  // ---- loads: one wave instruction fills eight 128-byte tile rows, lane l the
  // slot l % 8 of row l / 8. The descriptors begin at the tile (of B: at its
  // first weight row), so the lanes' offsets are the same for every tile; rows past the last
  // one are out of range and read as zeros.
  struct Source {
    const uint8_t *a, *b;
    const float* sc;
    uint32_t abytes, bbytes, sbytes;
  };
  // (No tile: the first rows and weights, which nothing uses. A descriptor is never
  // shorter than the K step's offset that is added to it.)
  const auto source_of = [&](const Tile& t) -> Source {
    const int n0 = t.e < 0 ? 0 : t.ntile * NO;
    const int rows = t.e < 0 ? (rows_total < BM ? (int)rows_total : BM) : t.rows;
    return {A + (int64_t)t.row0 * K,
            B + ((int64_t)(t.e < 0 ? 0 : t.e) * N + n0) * K,
            Asc + (int64_t)t.row0 * KB,
            (uint32_t)rows * (uint32_t)K,
            (uint32_t)(N - n0) * (uint32_t)K,
            (uint32_t)rows * (uint32_t)KB * 4};
  };
  uint32_t aoff[AI], boff[BI];
#pragma unroll
  for (int i = 0; i < AI; ++i) {
    const int r = wid * (BM / NW) + 8 * i + (lane >> 3);
    aoff[i] = (uint32_t)r * (uint32_t)K + (((lane & 7) ^ a_key(r)) << 4);
  }
#pragma unroll
  for (int i = 0; i < BI; ++i) {
    const int r = wid * (BN / NW) + 8 * i + (lane >> 3);
    const int n = kGateUp && r >= NO ? I + r - NO : r;
    boff[i] = (uint32_t)n * (uint32_t)K + (((lane & 7) ^ b_key(r)) << 4);
  }
  const int srow = wid % (BM / 64) * 64;  // the 64 row scales this wave loads
  const uint32_t soff = (uint32_t)(srow + lane) * (uint32_t)KB * 4;
  constexpr int kLoads = AI + BI + 1;
  Source src, after;  // of what is loaded now, and of the tile after the one computed
  int lk = 0;         // K step that is loaded
  // load number q of the step's kLoads
  auto issue = [&](uint8_t* st, int q) __attribute__((always_inline)) {
    if (q < BI)
      load_lds(make_rsrc(src.b, src.bbytes), st + (BM + wid * (BN / NW) + 8 * q) * kBK,
               boff[q % BI], lk * kBK);
    else if (q < BI + AI)
      load_lds(make_rsrc(src.a, src.abytes), st + (wid * (BM / NW) + 8 * (q - BI)) * kBK,
               aoff[(q - BI) % AI], lk * kBK);
    else
      load_lds4(make_rsrc(src.sc, src.sbytes), st + (BM + BN) * kBK + srow * 4, soff, lk * 4);
  };
  // K >= 2 steps, so the loads enter the next tile once while a tile is computed
  auto next_load = [&]() __attribute__((always_inline)) {
    const bool wrap = ++lk == KB;
    lk = wrap ? 0 : lk;
    src.a = wrap ? after.a : src.a;
    src.b = wrap ? after.b : src.b;
    src.sc = wrap ? after.sc : src.sc;
    src.abytes = wrap ? after.abytes : src.abytes;
    src.bbytes = wrap ? after.bbytes : src.bbytes;
    src.sbytes = wrap ? after.sbytes : src.sbytes;
  };

  // ---- fragments: lane l holds row (l % 16), chunks l / 16 and l / 16 + 4 of its
  // 128 bytes (both operands alike, so the order of k does not matter). A 16-byte
  // LDS read is served to 16 lanes at a time, eight of one l / 16 and eight of
  // the next (lanes 0-3, 12-15, 20-27 and so on): chunks of neighbours that differ in
  // bit 0 keep those apart; in bit 1 (2 (l / 16) and the next) half the LDS
  // cycles were bank conflicts.
  const int fi = lane & 15, fc = lane >> 4;
  const int arow = wm * 16 + fi;  // of fragment 0; the others 16 WM rows apart
  const int a0 = arow * kBK + ((fc ^ a_key(arow)) << 4);
  const int a1 = arow * kBK + (((fc + 4) ^ a_key(arow)) << 4);
  const int brow = (kGateUp ? wn * (NO / WN) : wn * (BN / WN)) + 8 * (fi >> 2) + (fi & 3);
  const int b0 = (BM + brow) * kBK + ((fc ^ b_key(brow)) << 4);
  const int b1 = (BM + brow) * kBK + (((fc + 4) ^ b_key(brow)) << 4);
  auto frag = [&](const uint8_t* st, int o0, int o1, int off) __attribute__((always_inline)) -> i32x8 {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(st + o0 + off);
    const i32x4 hi = *reinterpret_cast<const i32x4*>(st + o1 + off);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  constexpr int kFragRows = 16 * WM;
  auto read_a = [&](const uint8_t* st, int mi) { return frag(st, a0, a1, mi * kFragRows * kBK); };
  auto read_b = [&](const uint8_t* st, int ni) {
    // rows of fragment ni past this wave's first: pairs of 32, four apart inside
    const int q = kGateUp ? ni % (NI / 2) : ni;
    const int r = 32 * (q >> 1) + 4 * (q & 1) + (kGateUp && ni >= NI / 2 ? NO : 0);
    return frag(st, b0, b1, r * kBK);
  };
  auto read_s = [&](const uint8_t* st, int mi) -> float {
    return *reinterpret_cast<const float*>(st + (BM + BN) * kBK + (arow + mi * kFragRows) * 4);
  };

  // ---- the tile being computed
  Tile tile = tile_of(place);
  int ncol;             // first output column of the wave
  const float *bs0, *bs1;  // weight scales of its column block(s), one a K step
  auto enter = [&](const Tile& t) __attribute__((always_inline)) {
    tile = t;
    ncol = t.ntile * NO + wn * (NO / WN);
    const int nb = ncol / kQuantBlock < NB ? ncol / kQuantBlock : NB - 1;
    bs0 = Bsc + ((int64_t)(t.e < 0 ? 0 : t.e) * NB + nb) * KB;
    bs1 = kGateUp ? bs0 + (int64_t)(I / kQuantBlock) * KB : bs0;
  };
  enter(tile);

  f32x4 acc[NI][MI];
  i32x8 fa[MI], fb[4];
  float sa[MI];
  // ML: the wave's row fragments in use
  auto first_frags = [&](auto ml, const uint8_t* st) __attribute__((always_inline)) {
    constexpr int ML = decltype(ml)::value;
#pragma unroll
    for (int mi = 0; mi < ML; ++mi) {
      fa[mi] = read_a(st, mi);
      sa[mi] = read_s(st, mi);
    }
    fb[0] = read_b(st, 0);
    fb[1] = read_b(st, 1);
#pragma unroll
    for (int ni = 0; ni < NI; ++ni)
#pragma unroll
      for (int mi = 0; mi < ML; ++mi) acc[ni][mi] = f32x4{0, 0, 0, 0};
  };

  // A step reads stage S. Its fragments of A, the row scales and the first two
  // fragments of B are in registers already. Once a wave has read the last
  // fragments of the stage and its loads of the next step have landed, there is
  // one barrier; the MFMAs of the last two columns run behind it, so that the first
  // fragments of the next step are read while they do. The loads of the step after
  // next into this stage are spread: kAfter of them among those MFMAs, the rest one every
  // second MFMA of the next step. All at once after the barrier, the eight waves'
  // 72 loads (16 cycles each in the address unit) held up the MFMAs behind them
  // (8192 x 4096 x 7168: 221 against 213 us; spread over the next step alone 245,
  // too late). Each MFMA's result is folded two MFMAs later; the issue priority is
  // raised for the columns before the barrier (gate/up 455 against 415 us, also because the
  // scheduling fence keeps the registers from spilling).
  constexpr int kAfter = 5;
  auto step = [&](auto ml, auto S, int kt) __attribute__((always_inline)) {
    constexpr int ML = decltype(ml)::value;
    uint8_t* cur = stage(S);
    uint8_t* nxt = stage(std::integral_constant<int, decltype(S)::value + 1>{});
    const float w0 = bs0[kt], w1 = bs1[kt];
    float s0[ML], s1[ML];
#pragma unroll
    for (int mi = 0; mi < ML; ++mi) {
      s0[mi] = sa[mi] * w0;
      s1[mi] = kGateUp ? sa[mi] * w1 : s0[mi];
    }
    constexpr int kRing = 4, kLag = 2;                      // results in flight
    constexpr int kBefore = (NI - 2) * ML, kAll = NI * ML;  // MFMAs before the barrier, in all
    auto ni_of = [](int j) { return j < kBefore ? j / ML : NI - 2 + (j - kBefore) % 2; };
    auto mi_of = [](int j) { return j < kBefore ? j % ML : (j - kBefore) / 2; };
    f32x4 t[kRing];
    auto fold = [&](int j) __attribute__((always_inline)) {
      const int ni = ni_of(j), mi = mi_of(j);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        acc[ni][mi][r] = __builtin_fmaf(
            t[j % kRing][r], kGateUp && ni >= NI / 2 ? s1[mi] : s0[mi], acc[ni][mi][r]);
    };
    auto mma = [&](int j) __attribute__((always_inline)) {
      t[j % kRing] = mfma_fp8(fb[ni_of(j) % 4], fa[mi_of(j)]);
      if (j >= kLag) fold(j - kLag);
    };
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int ni = 0; ni < NI - 2; ++ni) {
      fb[(ni + 2) % 4] = read_b(cur, ni + 2);
#pragma unroll
      for (int mi = 0; mi < ML; ++mi) {
        const int j = ni * ML + mi, q = kAfter + j / 2;
        mma(j);
        if (j % 2 == 0 && q < kLoads) issue(nxt, q);
      }
    }
    __builtin_amdgcn_s_setprio(0);
#pragma unroll
    for (int q = kAfter + (kBefore + 1) / 2; q < kLoads; ++q) issue(nxt, q);  // with few MFMAs
    next_load();
    __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
    __syncthreads();
#pragma unroll
    for (int mi = 0; mi < ML; ++mi) {
      mma(kBefore + 2 * mi);
      mma(kBefore + 2 * mi + 1);
#pragma unroll
      for (int q = 0; q < kAfter; ++q)
        if (q * ML / kAfter == mi) issue(cur, q);
      fa[mi] = read_a(nxt, mi);
      sa[mi] = read_s(nxt, mi);
      if (mi < 2) fb[mi] = read_b(nxt, mi);
      if (ML == 1) fb[1] = read_b(nxt, 1);
    }
#pragma unroll
    for (int j = kAll - kLag; j < kAll; ++j) fold(j);
  };

  // ---- results: the stores go through descriptors over the tile's rows, whose
  // range check drops the rows past the last one.
  auto finish = [&](auto ml) __attribute__((always_inline)) {
    constexpr int ML = decltype(ml)::value;
    const int g = lane >> 4;
    if constexpr (!kGateUp) {
      const __amdgpu_buffer_rsrc_t crsrc = make_rsrc(
          static_cast<uint16_t*>(C) + (int64_t)tile.row0 * N, (int64_t)tile.rows * N * 2);
      // Lanes 8 apart swap halves, so that one store is 8 rows of whole 128-byte lines
      // instead of 16 rows of half ones, and the lines go past the caches, which keep
      // operands (8192 x 4096 x 7168: 215 us, cached whole lines 212, so 198; 24558
      // rows, N 2048, K 1408: 113, 110 and 108; without any stores 195 and 89).
      const bool low = (lane & 8) == 0;
      const int row = wm * 16 + (fi & 7);
#pragma unroll
      for (int p = 0; p < NI / 2; p += 2) {
        const int n = ncol + 32 * p + 8 * g + (low ? 0 : 32);
#pragma unroll
        for (int mi = 0; mi < ML; ++mi) {
          v4u v[2];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const f32x4 lo = acc[2 * (p + q)][mi], hi = acc[2 * (p + q) + 1][mi];
            v[q] = v4u{bf16x2_rne(lo[0], lo[1]), bf16x2_rne(lo[2], lo[3]),
                       bf16x2_rne(hi[0], hi[1]), bf16x2_rne(hi[2], hi[3])};
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
          const uint32_t at = ((uint32_t)(row + mi * kFragRows) * (uint32_t)N + n) * 2;
          __builtin_amdgcn_raw_buffer_store_b128(top, crsrc, n < N ? at : kOutside, 0, kStream);
          __builtin_amdgcn_raw_buffer_store_b128(bottom, crsrc, n < N ? at + 16 * (uint32_t)N : kOutside,
                                                 0, kStream);
        }
      }
    } else {
      // h = SiLU(g) u in place of g; the row maximum over the tile's 128 columns:
      // this lane's, the other lanes' of the row (16 and 32 apart), the other
      // waves' through LDS. Rows are whole scale blocks of h.
      {
#pragma unroll
        for (int mi = 0; mi < ML; ++mi) {
          uint32_t m = 0;
#pragma unroll
          for (int ni = 0; ni < NI / 2; ++ni)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float h = silu(acc[ni][mi][r]) * acc[ni + NI / 2][mi][r];
              acc[ni][mi][r] = h;
              const uint32_t u = finite_bits(h);
              m = u > m ? u : m;
            }
          uint32_t o = (uint32_t)__shfl_xor((int)m, 16);
          m = o > m ? o : m;
          o = (uint32_t)__shfl_xor((int)m, 32);
          m = o > m ? o : m;
          if (g == 0) ex[wn * BM + arow + mi * kFragRows] = m;
        }
      }
      lds_barrier();  // the maxima are read before the next step's barrier, so before they change
      const __amdgpu_buffer_rsrc_t crsrc =
          make_rsrc(static_cast<uint8_t*>(C) + (int64_t)tile.row0 * I, (int64_t)tile.rows * I);
      const int IB = I / kQuantBlock;
#pragma unroll
      for (int mi = 0; mi < ML; ++mi) {
        const int m = arow + mi * kFragRows;
        uint32_t a = 0;
#pragma unroll
        for (int w = 0; w < WN; ++w) a = ex[w * BM + m] > a ? ex[w * BM + m] : a;
        const int p2 = scale_exponent(a);
        const float inv = power_of_two(-p2);
        if (g == 0 && wn == 0 && m < tile.rows)
          Csc[(int64_t)(tile.row0 + m) * IB + tile.ntile] = power_of_two(p2);
#pragma unroll
        for (int p = 0; p < NI / 4; ++p) {
          const f32x4 lo = acc[2 * p][mi], hi = acc[2 * p + 1][mi];
          const uint32_t q0 = e4m3x4(e4m3_clamp(lo[0] * inv), e4m3_clamp(lo[1] * inv),
                                     e4m3_clamp(lo[2] * inv), e4m3_clamp(lo[3] * inv));
          const uint32_t q1 = e4m3x4(e4m3_clamp(hi[0] * inv), e4m3_clamp(hi[1] * inv),
                                     e4m3_clamp(hi[2] * inv), e4m3_clamp(hi[3] * inv));
          typedef uint32_t v2u __attribute__((ext_vector_type(2)));
          __builtin_amdgcn_raw_buffer_store_b64(v2u{q0, q1}, crsrc,
                                                (uint32_t)m * (uint32_t)I + ncol + 32 * p + 8 * g, 0, 0);
        }
      }
    }
  };
  // Steps 0 and (the first kAfter loads) 1 of the stream, then tile by tile; par: the
  // stage of the tile's first step.
  src = after = source_of(tile);
#pragma unroll
  for (int q = 0; q < kLoads; ++q) issue(lds0, q);
  next_load();
#pragma unroll
  for (int q = 0; q < kAfter; ++q) issue(lds1, q);
  __builtin_amdgcn_s_waitcnt(wait_vmcnt(kAfter));
  __syncthreads();
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  for (int par = 0;;) {
    const Tile ahead = tile_of(place + hop);
    after = source_of(ahead);
    auto compute = [&](auto ml) __attribute__((always_inline)) {
      first_frags(ml, par ? lds1 : lds0);
      int kt = 0;
      if (par) step(ml, I1{}, kt++);
      for (; kt + 2 <= KB; kt += 2) {
        step(ml, I0{}, kt);
        step(ml, I1{}, kt + 1);
      }
      if (kt < KB) step(ml, I0{}, kt);
      // The loads that run ahead land here, where it costs the least: past this point
      // nothing is pending in either stage, whichever the next tile begins with.
      __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
      finish(ml);
    };
    if (tile.rows > BM / 2) compute(std::integral_constant<int, MI>{});
    else if (tile.rows > BM / 4) compute(std::integral_constant<int, MI / 2>{});
    else compute(std::integral_constant<int, MI / 4>{});
    par = (par + KB) & 1;
    place += hop;
    if (place >= limit) break;
    enter(ahead);
  }
  // the trailing loads must land before the block's LDS is released
  __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
}

template <bool kGateUp, int BM, int BN, int WM, int WN>
hipError_t run_gemm(const void* a, const float* asc, int64_t rows, int E, const int32_t* offs,
                    const int32_t* cnts, const void* w, const float* wsc, int N, int K, void* c,
                    float* csc, hipStream_t s) {
  constexpr int NO = kGateUp ? BN / 2 : BN;
  const int cols = kGateUp ? N / 2 : N;
  const int ntiles = (cols + NO - 1) / NO;
  // every expert with rows adds at most one partial m-tile
  const int64_t mt = rows / BM + (rows < E ? rows : E);
  // one block a compute unit (a tile alone on its XCD is cut into four)
  int64_t per = 4 * ((mt * ntiles + kXCD - 1) / kXCD);
  if (per > kUnitsPerXcd) per = kUnitsPerXcd;
  return launch(gemm_fp8_kernel<kGateUp, BM, BN, WM, WN>, dim3((unsigned)(per * kXCD)),
                dim3(kWave * WM * WN), 0, s, static_cast<const uint8_t*>(a), asc, offs, cnts, E,
                rows, static_cast<const uint8_t*>(w), wsc, N, K, c, csc, ntiles);
}

}  // namespace

hipError_t launch_gemm_fp8(const void* a, const float* asc, int64_t rows, int E,
                           const int32_t* offs, const int32_t* cnts, const void* w,
                           const float* wsc, int N, int K, void* out, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  if (gemm_fp8_streams(rows, E, K))
    return launch_gemm_fp8_stream(false, a, asc, rows, E, offs, cnts, w, wsc, N, K, out, nullptr, s);
  return run_gemm<false, 256, 256, 4, 2>(a, asc, rows, E, offs, cnts, w, wsc, N, K, out, nullptr,
                                            s);
}

hipError_t launch_expert_swiglu_fp8(const void* send, const float* ssc, int64_t rows, int H, int I,
                                    int E, const int32_t* offs, const int32_t* cnts,
                                    const void* w_gate_up, const float* gsc, const void* w_down,
                                    const float* dsc, void* hq, float* hs, void* out,
                                    hipStream_t s) {
  if (rows == 0) return hipSuccess;
  const hipError_t err =
      gemm_fp8_streams(rows, E, H)
          ? launch_gemm_fp8_stream(true, send, ssc, rows, E, offs, cnts, w_gate_up, gsc, 2 * I, H, hq,
                                   hs, s)
          : run_gemm<true, 256, 256, 4, 2>(send, ssc, rows, E, offs, cnts, w_gate_up, gsc, 2 * I,
                                              H, hq, hs, s);
  if (err != hipSuccess) return err;
  return launch_gemm_fp8(hq, hs, rows, E, offs, cnts, w_down, dsc, H, I, out, s);
}

}  // namespace moe
