// gemm_int8_stream.hip -- grouped products of 8-bit integer rows with 8-bit integer
// expert weights for few rows an expert, where the weights' HBM bytes bound them:
// each live expert's weights are streamed once from memory through registers
// (stream.h), a block taking up to 32 rows of an expert.
//
//   out[m][n] = sa[m] sw[n] sum_j a[m][j] w[n][j],  the sum exact in 32 bits
//   gate/up:  h = SiLU(g) u in fp32, g and u as above
//
// A wave computes 32 weight rows by up to 32 tokens, K steps of 128 bytes. With one
// scale a row and a column the sums need no step of their own: the matrix instruction
// adds them up through the whole of K. 1024 rows of 128 experts, N 2816, K 4096: 194 us, 6.4
// TB/s; 5 rows of one, N 4096, K 7168: 8.9 us, of which a product of next to nothing takes
// 5.4 (launch, tile, first loads, the join).
#include <type_traits>

#include "device.h"
#include "ffn_device.h"
#include "gemm_int8.h"
#include "launch.h"
#include "quant_int8.h"
#include "stream.h"

namespace moe {
namespace {

constexpr int kRows = kStreamRows;  // rows of a tile
constexpr int kWaves = kStreamThreads / kWave;
constexpr int kStageBytes = 4096 + kRows * 128;  // a wave's LDS: a step's weights and tokens

// Whether rows of K bytes from w on are whole 128-byte lines.
bool whole_lines(const void* w, int K) {
  return ((reinterpret_cast<uintptr_t>(w) | (uintptr_t)K) & 127) == 0;
}

// Steps in flight of F fragments of 16 weight rows: what fits 128 registers (four waves a
// SIMD).
template <int NB, int F>
constexpr int kRing = F == 1 ? (NB == 4 ? 3 : 5) : (NB == 4 ? 2 : 3);

// acc[f][t] += products of weight fragment f (16 rows) with tokens 16 t .. 16 t + 15
// over the K steps s0 .. s0 + n - 1, beginning with step s0 + rot. woff: byte offsets in
// wb of the lane's four weight rows (two a fragment) at its chunk, wrow their LDS rows in
// the fragment; xoff[b]: in xb of its token of group b at its chunk (kOutside: none).
// last, keep: the step that holds the end of a row, and whether the lane's chunk of it is
// in the row; past it the tokens are zeros, so it does not matter what the weights are.
// kShared: other blocks read these weights.
template <int NB, int F, bool kShared>
__device__ __forceinline__ void dot_steps(uint8_t* stage, const Buffer& wb,
                                          const uint32_t (&woff)[2 * F], const int (&wrow)[2],
                                          const Buffer& xb, const uint32_t (&xoff)[NB], int s0,
                                          int n, int rot, int last, bool keep,
                                          i32x4 (&acc)[F][(NB + 1) / 2]) {
  constexpr int NTL = (NB + 1) / 2, D = kRing<NB, F>;
  const int lane = threadIdx.x & (kWave - 1);
  const int lr = lane >> 3, lc = lane & 7, i = lane & 15, g = lane >> 4;
  v4u w[D][2 * F], x[D][NB];
  auto load = [&](int u, int q) __attribute__((always_inline)) {
    const bool in = q < n;
    const uint32_t s = in ? (uint32_t)(s0 + (q + rot >= n ? q + rot - n : q + rot)) : 0;
    const bool cut = (int)s == last && !keep;
#pragma unroll
    for (int r = 0; r < 2 * F; ++r)
      w[u][r] = kShared ? load16(wb.at(in), woff[r], s * 128)
                        : load16_stream(wb.at(in), woff[r], s * 128);
#pragma unroll
    for (int b = 0; b < NB; ++b) x[u][b] = load16(xb.at(in), cut ? kOutside : xoff[b], s * 128);
  };
  uint8_t* xs = stage + 4096;
  auto frag = [&](const uint8_t* base, int r, int c) __attribute__((always_inline)) -> i32x4 {
    return *reinterpret_cast<const i32x4*>(base + tile_at(r, c));
  };
  auto compute = [&](int u) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < 2 * F; ++r)
      *reinterpret_cast<v4u*>(stage + 2048 * (r >> 1) + tile_at(wrow[r & 1], lc)) = w[u][r];
#pragma unroll
    for (int b = 0; b < NB; ++b) *reinterpret_cast<v4u*>(xs + tile_at(8 * b + lr, lc)) = x[u][b];
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // halves of the 128 bytes
      i32x4 a[F];
#pragma unroll
      for (int f = 0; f < F; ++f) a[f] = frag(stage + 2048 * f, i, g + 4 * h);
#pragma unroll
      for (int t = 0; t < NTL; ++t) {
        // with one group of 8 tokens its rows twice (columns 8-15 unused)
        const i32x4 tok = frag(xs, NB == 1 ? i & 7 : 16 * t + i, g + 4 * h);
#pragma unroll
        for (int f = 0; f < F; ++f) acc[f][t] = mfma_int8(a[f], tok, acc[f][t]);
      }
    }
    __builtin_amdgcn_wave_barrier();
  };
#pragma unroll
  for (int u = 0; u < D; ++u) load(u, u);
  for (int q = 0; q < n; q += D) {
#pragma unroll
    for (int u = 0; u < D; ++u) {
      compute(u);  // past the last step: zeros
      load(u, q + u + D);
    }
  }
}

// A block: one tile of up to kRows rows; its 8 waves are 8 / WK groups of 32 weight rows,
// each group's WK waves taking a share of K whose sums meet in LDS. Plain: 32 output
// columns a group. Gate/up: 16 columns a group (their gate and up rows interleaved in a
// fragment so that a lane's four results are g, g, u, u of two neighbouring columns), C
// = h in fp32. N: rows of one expert's B (2 I for gate/up). tokens: rows of A that idx
// may name, or null and A's rows lie in expert order.
// kLines: rows of B are whole lines (16 tokens, 8 of 128 experts, H 4080, I 1392: the FFN 328
// -> 275 us with lines that are not whole kept for the next step).
// F: fragments of 16 weight rows a wave, 2, or 1 where the columns are few (groups of 16).
template <bool kGateUp, int WK, bool kF32Out, bool kLines, int F>
__global__ __launch_bounds__(kWave * kWaves, 4) void gemm_int8_stream_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ Asc, const int32_t* __restrict__ idx,
    uint32_t tokens, const int32_t* __restrict__ offs, const int32_t* __restrict__ cnts, int E,
    int64_t rows_total, const uint8_t* __restrict__ B, const float* __restrict__ Bsc, int N, int K,
    void* __restrict__ C, int ntiles) {
  constexpr int kGroups = kWaves / WK;
  constexpr int kGroupCols = kGateUp ? 16 : 16 * F;
  static_assert(F == 2 || !kGateUp, "gate and up rows");
  constexpr int kNO = kGroups * kGroupCols;  // output columns of a tile
  __shared__ __attribute__((aligned(16))) uint8_t stage[kWaves][kStageBytes];
  __shared__ __attribute__((aligned(16))) float row_scale[kWave], col_scale[kStreamCols];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wid = __builtin_amdgcn_readfirstlane(tid / kWave);
  const WaveTile tile =
      E <= kWave       ? find_tile_wave<kRows, 1>(offs, cnts, E, rows_total, ntiles)
      : E <= 2 * kWave ? find_tile_wave<kRows, 2>(offs, cnts, E, rows_total, ntiles)
      : E <= 4 * kWave ? find_tile_wave<kRows, 4>(offs, cnts, E, rows_total, ntiles)
                       : find_tile_wave<kRows, kMaxExperts / kWave>(offs, cnts, E, rows_total, ntiles);
  if (tile.e < 0) return;  // uniform over the block
  const int e = tile.e, row0 = tile.row0, rows = tile.rows;
  const int i = lane & 15, g = lane >> 4, lr = lane >> 3, lc = lane & 7;
  const int KB = (K + 127) / 128, I = N / 2;
  const int group = wid / WK, part = wid % WK;
  const Buffer wb = {B + (int64_t)e * N * K, (uint32_t)N * (uint32_t)K};
  // (never shorter than a step's offset: without tokens every lane's row is outside)
  const Buffer xb = {idx ? A : A + (int64_t)row0 * K,
                     (idx ? (tokens ? tokens : 1) : (uint32_t)rows) * (uint32_t)K};
  const int n0 = tile.ntile * kNO + group * kGroupCols;  // the group's first column
  uint32_t woff[2 * F];
#pragma unroll
  for (int r = 0; r < 2 * F; ++r) {
    // gate/up: gate and up rows of 8 columns a fragment; plain: 8 rows each (those
    // past the last one, in the last tile, do not exist)
    const int c = kGateUp ? n0 + 8 * (r >> 1) + lr : n0 + 8 * r + lr;
    const int n = kGateUp ? (r & 1 ? I : 0) + c : c;
    woff[r] = c < (kGateUp ? I : N) ? (uint32_t)n * (uint32_t)K + 16 * lc : kOutside;
  }
  const int wrow[2] = {kGateUp ? 4 * (lr >> 1) + (lr & 1) : lr,
                       kGateUp ? 4 * (lr >> 1) + (lr & 1) + 2 : 8 + lr};
  // the row of A behind row m of the tile (past the last one where there is none)
  const auto source = [&](int m) -> uint32_t {
    if (m >= rows) return tokens;
    return idx ? (uint32_t)idx[row0 + m] : (uint32_t)(row0 + m);
  };
  // The tile's scales go straight into LDS, where they are when the products are: rows of
  // w by waves 0 and up (gate/up: the gate rows, then the up rows), rows of A by the last.
  constexpr int kWRows = kGroups * 16 * F;
  if (wid * kWave < kWRows) {
    const int r = wid * kWave + lane, c = kGateUp && r >= kNO ? r - kNO : r;
    const int n = tile.ntile * kNO + c + (kGateUp && r >= kNO ? I : 0);
    load_lds4(make_rsrc(Bsc + (int64_t)e * N, (int64_t)N * 4),
              reinterpret_cast<uint8_t*>(col_scale + wid * kWave), r < kWRows ? n * 4 : kOutside, 0);
  }
  if (wid == kWaves - 1) {
    const uint32_t r = source(lane);
    load_lds4(make_rsrc(Asc, (int64_t)tokens * 4), reinterpret_cast<uint8_t*>(row_scale),
              r < tokens ? r * 4 : kOutside, 0);
  }

  auto pass = [&](auto nb_, auto shared) __attribute__((always_inline)) {
    constexpr int NB = decltype(nb_)::value, NTL = (NB + 1) / 2;
    uint32_t xoff[NB];
    i32x4 acc[F][NTL];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint32_t m = 8 * b + lr, r = idx ? source(m) : m;
      xoff[b] = (int)m < rows && (!idx || r < tokens) ? r * (uint32_t)K + 16 * lc : kOutside;
    }
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int t = 0; t < NTL; ++t) acc[f][t] = i32x4{0, 0, 0, 0};
    const int s0 = KB * part / WK, n = KB * (part + 1) / WK - s0;
    if (n > 0)  // uniform over the wave
      dot_steps<NB, F, decltype(shared)::value>(stage[wid], wb, woff, wrow, xb, xoff, s0, n,
                                             (int)((uint32_t)(tile.ntile + row0) * 5 % (uint32_t)n), KB - 1,
                                             16 * lc < K - 128 * (KB - 1), acc);
    // lane l's results of fragments f and t: columns n0 + 16 f (8 f) + ..., token 16 t + i
    const auto emit = [&](int f, int t, i32x4 v) __attribute__((always_inline)) {
      const int m = 16 * t + i;
      if (m >= rows || (NB == 1 && i >= 8)) return;
      const float sa = row_scale[m];
      if constexpr (kGateUp) {
        const int c = group * kGroupCols + 8 * f + 2 * g, n = tile.ntile * kNO + c;
        if (n >= I) return;
        const float2 sg = *reinterpret_cast<const float2*>(col_scale + c);
        const float2 su = *reinterpret_cast<const float2*>(col_scale + kNO + c);
        float2 h;
        h.x = silu(scaled(v[0], sa, sg.x)) * scaled(v[2], sa, su.x);
        h.y = silu(scaled(v[1], sa, sg.y)) * scaled(v[3], sa, su.y);
        *reinterpret_cast<float2*>(static_cast<float*>(C) + (int64_t)(row0 + m) * I + n) = h;
      } else {
        const int c = group * kGroupCols + 16 * f + 4 * g, n = tile.ntile * kNO + c;
        if (n >= N) return;
        const float4 sw = *reinterpret_cast<const float4*>(col_scale + c);
        const float o[4] = {scaled(v[0], sa, sw.x), scaled(v[1], sa, sw.y), scaled(v[2], sa, sw.z),
                            scaled(v[3], sa, sw.w)};
        const int64_t at = (int64_t)(row0 + m) * N + n;
        if constexpr (kF32Out)
          *reinterpret_cast<float4*>(static_cast<float*>(C) + at) = make_float4(o[0], o[1], o[2], o[3]);
        else
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(C) + at) =
              make_uint2(bf16x2_rne(o[0], o[1]), bf16x2_rne(o[2], o[3]));
      }
    };
    // Every wave's sums in its stage, of which the group's waves then take the fragments
    // in turn (also a wave alone: results straight from the registers made it spill).
    constexpr int kFrags = F * NTL;
    i32x4* own = reinterpret_cast<i32x4*>(stage[wid]);
    static_assert(kFrags * kWave * 16 <= kStageBytes, "sums fit the stage");
#pragma unroll
    for (int j = 0; j < kFrags; ++j) own[j * kWave + lane] = acc[j / NTL][j % NTL];
    __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);  // the scales
    __syncthreads();
#pragma unroll 1
    for (int j = part; j < kFrags; j += WK) {
      i32x4 v = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < WK; ++w)
        v += reinterpret_cast<const i32x4*>(stage[group * WK + w])[j * kWave + lane];
      emit(j / NTL, j % NTL, v);
    }
  };
  // Weights stay in the caches where the expert's other tiles read them too, or the next K
  // step takes the rest of a line; else they go past them (gate/up of 128 tokens, 128 experts,
  // N 2816, K 4096: 222 -> 195 us).
  const std::bool_constant<!kLines> shared;
  if (tile.len > kRows) pass(std::integral_constant<int, 4>{}, std::true_type{});
  else if (rows <= 8) pass(std::integral_constant<int, 1>{}, shared);
  else if (rows <= 16) pass(std::integral_constant<int, 2>{}, shared);
  else pass(std::integral_constant<int, 4>{}, shared);
}

// The FFN's second product for a few rows, from the inner rows in fp32: up to kInnerRows
// rows of kInnerCols columns, a vector of four a thread. Every block makes integers of its
// tile's rows itself (the steps of quantize_int8_kernel, the same bits) while its first
// weights are on their way, and keeps them in LDS: a launch less. The FFN of one token, 8 of
// 128 experts, H 4096, I 1408: 33.9 -> 31.4 us; 6 of 64, H 2048: 24.8 -> 22.3; 8 rows of one
// expert, all of which every block then makes: 18.5 -> 17.5 us, and 21.4 -> 21.6 at H 7168,
// I 2048. Blocks, groups and parts of K as in the kernel above.
//
// A row in LDS: 32 bytes past a multiple of 256, so that the 16-byte reads of 8 rows in two
// neighbouring chunks miss each other.
constexpr int kInnerStride = kInnerCols + 32;
static_assert(kInnerCols == 4 * kWave * kWaves && kInnerRows == 8, "a vector a thread; one group of rows");

// kLines: rows of B are whole lines, which then go past the caches.
template <int WK, bool kLines>
__global__ __launch_bounds__(kWave * kWaves, 4) void gemm_int8_inner_kernel(
    const float* __restrict__ h, const int32_t* __restrict__ offs, const int32_t* __restrict__ cnts,
    int E, int64_t rows_total, const uint8_t* __restrict__ B, const float* __restrict__ Bsc, int N,
    int K, uint16_t* __restrict__ C, int ntiles) {
  constexpr int kNO = kWaves / WK * 32;  // output columns of a tile
  constexpr int D = 3;                   // steps in flight
  __shared__ __attribute__((aligned(16))) uint8_t stage[kWaves][4096];
  __shared__ __attribute__((aligned(16))) uint8_t x[kInnerRows * kInnerStride];
  __shared__ uint2 tops[kInnerRows][kWaves];
  __shared__ __attribute__((aligned(16))) float row_scale[kInnerRows], col_scale[kStreamCols];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wid = __builtin_amdgcn_readfirstlane(tid / kWave);
  const WaveTile tile =
      E <= kWave       ? find_tile_wave<kRows, 1>(offs, cnts, E, rows_total, ntiles)
      : E <= 2 * kWave ? find_tile_wave<kRows, 2>(offs, cnts, E, rows_total, ntiles)
      : E <= 4 * kWave ? find_tile_wave<kRows, 4>(offs, cnts, E, rows_total, ntiles)
                       : find_tile_wave<kRows, kMaxExperts / kWave>(offs, cnts, E, rows_total, ntiles);
  if (tile.e < 0) return;  // uniform over the block
  const int rows = tile.rows, i = lane & 15, g = lane >> 4, lr = lane >> 3, lc = lane & 7;
  const int group = wid / WK, part = wid % WK;
  // What lies past a row's end, or past the last row, comes as zeros.
  v4u f[kInnerRows];
  const __amdgpu_buffer_rsrc_t hr = make_rsrc(h + (int64_t)tile.row0 * K, (int64_t)rows * K * 4);
#pragma unroll
  for (int r = 0; r < kInnerRows; ++r)
    f[r] = load16(hr, 4 * tid < K ? (uint32_t)(r * K + 4 * tid) * 4 : kOutside, 0);
  const int n0 = tile.ntile * kNO;
  if (wid * kWave < kNO) {  // the tile's column scales, straight into LDS
    const int c = wid * kWave + lane;
    load_lds4(make_rsrc(Bsc + (int64_t)tile.e * N, (int64_t)N * 4),
              reinterpret_cast<uint8_t*>(col_scale + wid * kWave), c < kNO ? (n0 + c) * 4 : kOutside, 0);
  }
  const Buffer wb = {B + (int64_t)tile.e * N * K, (uint32_t)N * (uint32_t)K};
  uint32_t woff[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int n = n0 + group * 32 + 8 * r + lr;
    woff[r] = n < N ? (uint32_t)n * (uint32_t)K + 16 * lc : kOutside;
  }
  // the wave's K steps, beginning with the one at rot; past the last step: weights of zeros
  const int KB = (K + 127) / 128, s0 = KB * part / WK, n = KB * (part + 1) / WK - s0;
  const int rot = n > 0 ? (int)((uint32_t)(tile.ntile + tile.row0) * 5 % (uint32_t)n) : 0;
  const auto step_of = [&](int q) { return q < n ? s0 + (q + rot >= n ? q + rot - n : q + rot) : 0; };
  v4u w[D][4];
  const auto load = [&](int u, int q) __attribute__((always_inline)) {
    const uint32_t at = (uint32_t)step_of(q) * 128;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      w[u][r] = kLines ? load16_stream(wb.at(q < n), woff[r], at) : load16(wb.at(q < n), woff[r], at);
  };
  __builtin_amdgcn_sched_barrier(0);  // the rows, which are waited for first, come first
#pragma unroll
  for (int u = 0; u < D; ++u) load(u, u);
  __builtin_amdgcn_sched_barrier(0);

  const auto max = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
#pragma unroll
  for (int r = 0; r < kInnerRows; ++r) {
    if (r >= rows) break;
    uint32_t top = 0, all = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t u = f[r][j] & 0x7FFFFFFFu;
      top = max(top, u < kInfBits ? u : 0u);
      all = max(all, u);
    }
    all = group_reduce(all, kWave, max);
    top = group_reduce(top, kWave, max);
    if (lane == 0) tops[r][wid] = make_uint2(all, top);
  }
  lds_barrier();
#pragma unroll
  for (int r = 0; r < kInnerRows; ++r) {
    if (r >= rows) break;
    uint2 m = tops[r][lane & (kWaves - 1)];
    m.x = group_reduce(m.x, kWaves, max);
    m.y = group_reduce(m.y, kWaves, max);
    const Int8Row how = int8_row(m.x, m.y);
    const auto q = [&](int j) { return how.round(__uint_as_float(f[r][j])); };
    *reinterpret_cast<uint32_t*>(x + r * kInnerStride + 4 * tid) = pack_int8(q(0), q(1), q(2), q(3));
    if (tid == 0) row_scale[r] = how.scale;
  }
  lds_barrier();

  i32x4 acc[2] = {i32x4{0, 0, 0, 0}, i32x4{0, 0, 0, 0}};
  uint8_t* own = stage[wid];
  const auto frag = [&](const uint8_t* base, int c) __attribute__((always_inline)) -> i32x4 {
    return *reinterpret_cast<const i32x4*>(base + tile_at(i, c));
  };
  for (int q0 = 0; q0 < n; q0 += D) {
#pragma unroll
    for (int u = 0; u < D; ++u) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *reinterpret_cast<v4u*>(own + 2048 * (r >> 1) + tile_at(8 * (r & 1) + lr, lc)) = w[u][r];
      // rows past the last one: whatever is there, in columns of the result that nobody stores
      const uint8_t* rows8 = x + (i & 7) * kInnerStride + step_of(q0 + u) * 128 + 16 * g;
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const i32x4 tok = *reinterpret_cast<const i32x4*>(rows8 + 64 * half);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          acc[k] = mfma_int8(frag(own + 2048 * k, g + 4 * half), tok, acc[k]);
      }
      __builtin_amdgcn_wave_barrier();
      load(u, q0 + u + D);
    }
  }
  // Sums of the group's waves, of which the first two emit a fragment of 16 columns each
  // (a wave alone: both).
  i32x4* sums = reinterpret_cast<i32x4*>(own);
#pragma unroll
  for (int k = 0; k < 2; ++k) sums[k * kWave + lane] = acc[k];
  __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);  // the scales
  __syncthreads();
#pragma unroll 1
  for (int k = part; k < 2; k += WK) {
    i32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int p = 0; p < WK; ++p)
      v += reinterpret_cast<const i32x4*>(stage[group * WK + p])[k * kWave + lane];
    const int c = group * 32 + 16 * k + 4 * g;
    if (i >= rows || n0 + c >= N) continue;
    const float sa = row_scale[i];
    const float4 sw = *reinterpret_cast<const float4*>(col_scale + c);
    *reinterpret_cast<uint2*>(C + (int64_t)(tile.row0 + i) * N + n0 + c) =
        make_uint2(bf16x2_rne(scaled(v[0], sa, sw.x), scaled(v[1], sa, sw.y)),
                   bf16x2_rne(scaled(v[2], sa, sw.z), scaled(v[3], sa, sw.w)));
  }
}

// The blocks of a product of so many rows and column tiles, in runs of an XCD's.
unsigned blocks(int64_t rows, int E, int ntiles) {
  const int64_t mt = rows / kRows + (rows < E ? rows : E);
  const int64_t runs = (mt * ntiles + kGroupM * kXCD - 1) / (kGroupM * kXCD);
  return (unsigned)(runs * kGroupM * kXCD);
}

template <bool kGateUp, int WK, bool kF32Out, int F = 2>
hipError_t run(const Int8Rows& a, int64_t rows, int E, const int32_t* offs, const int32_t* cnts,
               const void* w, const float* wsc, int N, int K, void* c, hipStream_t s) {
  const int cols = kGateUp ? N / 2 : N;
  constexpr int kNO = kWaves / WK * (kGateUp ? 16 : 16 * F);
  const int ntiles = (cols + kNO - 1) / kNO;
  return launch(whole_lines(w, K) ? gemm_int8_stream_kernel<kGateUp, WK, kF32Out, true, F>
                                  : gemm_int8_stream_kernel<kGateUp, WK, kF32Out, false, F>,
                dim3(blocks(rows, E, ntiles)), dim3(kWave * kWaves), 0, s,
                static_cast<const uint8_t*>(a.q), a.scale, a.index, (uint32_t)a.rows, offs, cnts, E,
                rows, static_cast<const uint8_t*>(w), wsc, N, K, c, ntiles);
}

template <typename F>
hipError_t by_splits(int64_t rows, int E, int N, int K, const F& f) {
  switch (gemm_int8_splits(rows, E, N, K)) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 4: return f(std::integral_constant<int, 4>{});
    default: return f(std::integral_constant<int, 8>{});
  }
}

}  // namespace

hipError_t launch_gemm_int8_stream(bool gate_up, bool f32_out, const Int8Rows& a, int64_t rows,
                                   int E, const int32_t* offs, const int32_t* cnts, const void* w,
                                   const float* wsc, int N, int K, void* c, hipStream_t s) {
  return by_splits(rows, E, N, K, [&](auto wk) {
    constexpr int WK = decltype(wk)::value;
    if (gate_up) return run<true, WK, true>(a, rows, E, offs, cnts, w, wsc, N, K, c, s);
    // Half the units and more without a block: groups of 16 columns, the same bytes of
    // weights in flight a wave (5 rows, N 4096, K 7168: 10.2 -> 8.9 us; 30 rows, N 2048: 12.6 ->
    // 10.8; 1 row, K 14336: 15.1 -> 12.0; 64 rows, N 2048, K 7168: 10.4 and 10.5).
    if constexpr (WK == kWaves) {
      if ((rows / kRows + (rows < E ? rows : E)) * ((N + 31) / 32) <= 128)
        return f32_out ? run<false, WK, true, 1>(a, rows, E, offs, cnts, w, wsc, N, K, c, s)
                       : run<false, WK, false, 1>(a, rows, E, offs, cnts, w, wsc, N, K, c, s);
    }
    return f32_out ? run<false, WK, true>(a, rows, E, offs, cnts, w, wsc, N, K, c, s)
                   : run<false, WK, false>(a, rows, E, offs, cnts, w, wsc, N, K, c, s);
  });
}

hipError_t launch_gemm_int8_inner(const float* h, int64_t rows, int E, const int32_t* offs,
                                  const int32_t* cnts, const void* w, const float* wsc, int N, int K,
                                  void* c, hipStream_t s) {
  return by_splits(rows, E, N, K, [&](auto wk) {
    constexpr int WK = decltype(wk)::value, kNO = kWaves / WK * 32;
    const int ntiles = (N + kNO - 1) / kNO;
    return launch(whole_lines(w, K) ? gemm_int8_inner_kernel<WK, true> : gemm_int8_inner_kernel<WK, false>,
                  dim3(blocks(rows, E, ntiles)), dim3(kWave * kWaves), 0, s, h, offs, cnts, E, rows,
                  static_cast<const uint8_t*>(w), wsc, N, K, static_cast<uint16_t*>(c), ntiles);
  });
}

}  // namespace moe
