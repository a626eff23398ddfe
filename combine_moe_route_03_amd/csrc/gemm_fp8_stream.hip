// gemm_fp8_stream.hip -- the grouped products of gemm_fp8.hip for few rows an
// expert (the decode regime), where they are bound by the HBM bytes of the live
// experts' weights: the weights are streamed once from memory through registers
// (stream.h) instead of through tiles shared by a block, and a block takes up to
// 32 rows of an expert. An expert with more rows is several row tiles, adjacent
// in the tile list, so they run at one time on one XCD and the weights come from
// its L2: those tiles load them cached, all others past the caches (128 experts, N
// 2816, K 4096, 128 tokens most of whose picks go to 8 experts: 243 us with every
// load past the caches, 211 with the cached ones for 17 to 32 rows of any expert,
// 198 = 6.2 TB/s as it is, 6.4 TB/s with even routing; memory reads 1.48, 1.37 and
// 1.33 GB for 1.23 GB of weights).
//
// A wave computes 32 weight rows by up to 32 tokens (two fragments of 16 rows, so
// that a token fragment is loaded once for both), one
// v_mfma_f32_16x16x128_f8f6f4 a K step of 128, 16 rows and 16 tokens, folded with
// the two scales into fp32 as in gemm_fp8.hip. The tile's row scales are kept in
// LDS: read from memory a step at a time they cost 7-18% (16 lines a load). They are
// requested before the first steps' weights and put there behind them (the weights
// only after that: 2-4% more, N 4096, K 1408, even routing 125 against 122 us).
#include <type_traits>

#include "device.h"
#include "ffn_device.h"
#include "gemm_fp8.h"
#include "launch.h"
#include "quant.h"
#include "stream.h"

namespace moe {
namespace {

constexpr int kRows = kStreamRows;  // rows of a tile
constexpr int kWaves = kStreamThreads / kWave;
constexpr int kChunk = 64;   // K steps whose scales are held at a time
constexpr int kSPitch = kChunk + 1;

constexpr int kStageBytes = 4096 + kRows * 128;  // a wave's LDS: a step's weights and tokens

// Steps in flight: what fits 128 registers (four waves a SIMD).
template <int NB>
constexpr int kRing = NB == 4 ? 2 : 3;

// acc[f][t] += the scaled products of weight fragment f (16 rows) with tokens 16 t ..
// 16 t + 15 over the n <= kChunk K steps from s0, beginning with step s0 + rot. woff:
// byte offsets in wb of the lane's four weight rows (two a fragment) at its
// chunk, wrow their LDS rows in the fragment; xoff[b]: in xb of its token of
// group b at its chunk (kOutside: none); ss: row scales [kRows][kSPitch] of these
// steps; c0, c1: weight scales of D registers 0-1 and 2-3, lane l's of step s0 + l.
// kShared: other blocks read these weights. settle: called when the first loads are
// on their way; ss, c0 and c1 are there when it returns.
template <bool kTwoScales, int NB, bool kShared, typename Settle>
__device__ __forceinline__ void dot_steps8(uint8_t* stage, const Buffer& wb,
                                           const uint32_t (&woff)[4], const int (&wrow)[2],
                                           const Buffer& xb, const uint32_t (&xoff)[NB],
                                           const float* ss, const float& c0, const float& c1,
                                           int s0, int n, int rot, f32x4 (&acc)[2][(NB + 1) / 2],
                                           const Settle& settle) {
  constexpr int NTL = (NB + 1) / 2, D = kRing<NB>;
  const int lane = threadIdx.x & (kWave - 1);
  const int lr = lane >> 3, lc = lane & 7, i = lane & 15, g = lane >> 4;
  v4u w[D][4], x[D][NB];
  const auto step_of = [&](int q) { return q + rot >= n ? q + rot - n : q + rot; };
  auto load = [&](int u, int q) __attribute__((always_inline)) {
    const bool in = q < n;
    const uint32_t s = in ? (uint32_t)(s0 + step_of(q)) : 0;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      w[u][r] = kShared ? load16(wb.at(in), woff[r], s * 128)
                        : load16_stream(wb.at(in), woff[r], s * 128);
#pragma unroll
    for (int b = 0; b < NB; ++b) x[u][b] = load16(xb.at(in), xoff[b], s * 128);
  };
  uint8_t* xs = stage + 4096;
  auto frag = [&](const uint8_t* base, int r) __attribute__((always_inline)) -> i32x8 {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(base + tile_at(r, g));
    const i32x4 hi = *reinterpret_cast<const i32x4*>(base + tile_at(r, g + 4));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto compute = [&](int u, int q) __attribute__((always_inline)) {
    // past the last step: any (the products are zero)
    const int l = q < n ? step_of(q) : 0;
    const float w0 = __uint_as_float(lane_value(__float_as_uint(c0), l));
    const float w1 = kTwoScales ? __uint_as_float(lane_value(__float_as_uint(c1), l)) : w0;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      *reinterpret_cast<v4u*>(stage + 2048 * (r >> 1) + tile_at(wrow[r & 1], lc)) = w[u][r];
#pragma unroll
    for (int b = 0; b < NB; ++b) *reinterpret_cast<v4u*>(xs + tile_at(8 * b + lr, lc)) = x[u][b];
    __builtin_amdgcn_wave_barrier();
    const i32x8 a[2] = {frag(stage, i), frag(stage + 2048, i)};
#pragma unroll
    for (int t = 0; t < NTL; ++t) {
      // with one group of 8 tokens its rows twice (columns 8-15 unused)
      const int tr = NB == 1 ? i & 7 : 16 * t + i;
      const i32x8 tok = frag(xs, tr);
      const float sa = ss[tr * kSPitch + l];
      const float f0 = sa * w0, f1 = kTwoScales ? sa * w1 : f0;
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const f32x4 d = mfma_fp8(a[f], tok);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[f][t][r] = __builtin_fmaf(d[r], r < 2 ? f0 : f1, acc[f][t][r]);
      }
    }
    __builtin_amdgcn_wave_barrier();
  };
#pragma unroll
  for (int u = 0; u < D; ++u) load(u, u);
  settle();
  for (int q = 0; q < n; q += D) {
#pragma unroll
    for (int u = 0; u < D; ++u) {
      compute(u, q + u);
      load(u, q + u + D);
    }
  }
}

// A block: one tile of up to kRows rows, kWaves waves of 32 weight rows. Plain: 32
// output columns a wave. Gate/up: 16 columns a wave (their gate and up rows
// interleaved in a fragment so that a lane's four results are g, g, u, u of two
// neighbouring columns); h is collected in LDS, where the tile's rows are whole
// scale blocks, and quantised. N: rows of one expert's B (2 I for gate/up).
template <bool kGateUp>
__global__ __launch_bounds__(kWave * kWaves, 4) void gemm_fp8_stream_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ Asc,
    const int32_t* __restrict__ offs, const int32_t* __restrict__ cnts, int E,
    int64_t rows_total, const uint8_t* __restrict__ B, const float* __restrict__ Bsc, int N, int K,
    void* __restrict__ C, float* __restrict__ Csc, int ntiles) {
  constexpr int kWaveCols = kGateUp ? 16 : 32;
  constexpr int kNO = kWaves * kWaveCols;  // output columns of a tile
  constexpr int kPitch = kNO + 4;          // floats of an h row in LDS
  static_assert(!kGateUp || kNO == kQuantBlock, "one scale block of h per tile");
  static_assert(kNO * (kGateUp ? 2 : 1) == kStreamCols, "rows of w a tile");
  __shared__ __attribute__((aligned(16))) uint8_t stage[kWaves][kStageBytes];
  __shared__ __attribute__((aligned(16))) float ss[kRows * kSPitch];
  __shared__ int info[4];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wid = __builtin_amdgcn_readfirstlane(tid / kWave);
  const Tile tile = find_tile<kRows>(offs, cnts, E, rows_total, ntiles, info);
  if (tile.e < 0) return;  // uniform over the block
  const int e = tile.e, row0 = tile.row0, rows = tile.rows;
  const int i = lane & 15, g = lane >> 4, lr = lane >> 3, lc = lane & 7;
  const int KB = K / 128, I = N / 2, NB128 = (N + kQuantBlock - 1) / kQuantBlock;
  const Buffer wb = {B + (int64_t)e * N * K, (uint32_t)N * (uint32_t)K};
  const Buffer xb = {A + (int64_t)row0 * K, (uint32_t)rows * (uint32_t)K};
  const int c = wid * kWaveCols;           // the wave's first column in the tile
  const int n0 = tile.ntile * kNO + c;
  // weight scales of the wave's columns (gate/up: of its gate and its up rows)
  const int nb = n0 / kQuantBlock < NB128 ? n0 / kQuantBlock : NB128 - 1;
  const float* bs0 = Bsc + ((int64_t)e * NB128 + nb) * KB;
  const float* bs1 = kGateUp ? bs0 + (int64_t)(I / kQuantBlock) * KB : bs0;
  uint32_t woff[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    // gate/up: gate and up rows of 8 columns a fragment; plain: 8 rows each (those
    // past N, in the last tile, do not exist)
    const int n = kGateUp ? (r & 1 ? I : 0) + n0 + 8 * (r >> 1) + lr : n0 + 8 * r + lr;
    woff[r] = n < N ? (uint32_t)n * (uint32_t)K + 16 * lc : kOutside;
  }
  const int wrow[2] = {kGateUp ? 4 * (lr >> 1) + (lr & 1) : lr,
                       kGateUp ? 4 * (lr >> 1) + (lr & 1) + 2 : 8 + lr};
  float* hs = reinterpret_cast<float*>(&stage[0][0]);  // [kRows][kPitch], after the products
  static_assert(kRows * kPitch * 4 <= kWaves * kStageBytes || !kGateUp, "h fits the stage");

  auto pass = [&](auto nb_, auto shared) __attribute__((always_inline)) {
    constexpr int NB = decltype(nb_)::value, NTL = (NB + 1) / 2;
    uint32_t xoff[NB];
    f32x4 acc[2][NTL];
#pragma unroll
    for (int b = 0; b < NB; ++b)
      xoff[b] = 8 * b + lr < rows ? (uint32_t)(8 * b + lr) * (uint32_t)K + 16 * lc : kOutside;
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int t = 0; t < NTL; ++t) acc[f][t] = f32x4{0, 0, 0, 0};
    constexpr int kThreads = kWave * kWaves, kPer = kRows * kChunk / kThreads;
    for (int s0 = 0; s0 < KB; s0 += kChunk) {
      const int n = KB - s0 < kChunk ? KB - s0 : kChunk;
      // the scales first, then the first steps' loads, which do not wait for them
      const int l = s0 + (lane < n ? lane : 0);
      float c0 = bs0[l], c1 = bs1[l];
      float sc[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int r = tid / kChunk + j * (kThreads / kChunk), k = tid % kChunk;
        sc[j] = r < rows && k < n ? Asc[(int64_t)(row0 + r) * KB + s0 + k] : 0.f;
      }
      const auto settle = [&]() __attribute__((always_inline)) {
        // landed here: a use inside the step loop would wait for the ring's loads too
        asm volatile("" : "+v"(c0), "+v"(c1));
        if (s0 > 0) lds_barrier();
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          ss[(tid / kChunk + j * (kThreads / kChunk)) * kSPitch + tid % kChunk] = sc[j];
        lds_barrier();
      };
      dot_steps8<kGateUp, NB, decltype(shared)::value>(stage[wid], wb, woff, wrow, xb, xoff, ss, c0,
                                                       c1, s0, n, (tile.ntile + row0) * 5 % n, acc,
                                                       settle);
    }
    if constexpr (kGateUp) {
      __syncthreads();  // every wave is done with its stage
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int t = 0; t < NTL; ++t)
          if (NB > 1 || i < 8) {
            float2 v;
            v.x = silu(acc[f][t][0]) * acc[f][t][2];
            v.y = silu(acc[f][t][1]) * acc[f][t][3];
            *reinterpret_cast<float2*>(&hs[(16 * t + i) * kPitch + c + 8 * f + 2 * g]) = v;
          }
    } else {
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int t = 0; t < NTL; ++t) {
          const int m = 16 * t + i;
          if (m < rows && (NB > 1 || i < 8) && n0 + 16 * f < N) {
            uint2 v;
            v.x = bf16x2_rne(acc[f][t][0], acc[f][t][1]);
            v.y = bf16x2_rne(acc[f][t][2], acc[f][t][3]);
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(C) + (int64_t)(row0 + m) * N + n0 +
                                      16 * f + 4 * g) = v;
          }
        }
    }
  };
  // the expert's other tiles read the same weights
  if (cnts[e] > kRows) pass(std::integral_constant<int, 4>{}, std::true_type{});
  else if (rows <= 8) pass(std::integral_constant<int, 1>{}, std::false_type{});
  else if (rows <= 16) pass(std::integral_constant<int, 2>{}, std::false_type{});
  else pass(std::integral_constant<int, 4>{}, std::false_type{});

  if constexpr (kGateUp) {
    __syncthreads();
    // 16 lanes a row, 8 columns a lane
    const int m = tid >> 4, j0 = (tid & 15) * 8;
    static_assert(kWave * kWaves == 16 * kRows, "a thread for every 8 values of h");
    const float4 v0 = *reinterpret_cast<const float4*>(&hs[m * kPitch + j0]);
    const float4 v1 = *reinterpret_cast<const float4*>(&hs[m * kPitch + j0 + 4]);
    const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    uint32_t a = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t u = finite_bits(v[j]);
      a = u > a ? u : a;
    }
    a = group_reduce(a, 16, [](uint32_t p, uint32_t q) { return p > q ? p : q; });
    const int p = scale_exponent(a);
    const float inv = power_of_two(-p);
    if (m < rows) {
      uint2 o;
      o.x = e4m3x4(e4m3_clamp(v[0] * inv), e4m3_clamp(v[1] * inv), e4m3_clamp(v[2] * inv),
                   e4m3_clamp(v[3] * inv));
      o.y = e4m3x4(e4m3_clamp(v[4] * inv), e4m3_clamp(v[5] * inv), e4m3_clamp(v[6] * inv),
                   e4m3_clamp(v[7] * inv));
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(C) + (int64_t)(row0 + m) * I +
                                tile.ntile * kNO + j0) = o;
      if ((tid & 15) == 0)
        Csc[(int64_t)(row0 + m) * (I / kQuantBlock) + tile.ntile] = power_of_two(p);
    }
  }
}

template <bool kGateUp>
hipError_t run(const void* a, const float* asc, int64_t rows, int E, const int32_t* offs,
               const int32_t* cnts, const void* w, const float* wsc, int N, int K, void* c,
               float* csc, hipStream_t s) {
  const int cols = kGateUp ? N / 2 : N;
  constexpr int kNO = kWaves * (kGateUp ? 16 : 32);
  const int ntiles = (cols + kNO - 1) / kNO;
  const int64_t mt = rows / kRows + (rows < E ? rows : E);
  const int64_t runs = (mt * ntiles + kGroupM * kXCD - 1) / (kGroupM * kXCD);
  return launch(gemm_fp8_stream_kernel<kGateUp>, dim3((unsigned)(runs * kGroupM * kXCD)),
                dim3(kWave * kWaves), 0, s, static_cast<const uint8_t*>(a), asc, offs, cnts, E, rows,
                static_cast<const uint8_t*>(w), wsc, N, K, c, csc, ntiles);
}

}  // namespace

hipError_t launch_gemm_fp8_stream(bool gate_up, const void* a, const float* asc, int64_t rows,
                                  int E, const int32_t* offs, const int32_t* cnts, const void* w,
                                  const float* wsc, int N, int K, void* c, float* csc,
                                  hipStream_t s) {
  return gate_up ? run<true>(a, asc, rows, E, offs, cnts, w, wsc, N, K, c, csc, s)
                 : run<false>(a, asc, rows, E, offs, cnts, w, wsc, N, K, c, csc, s);
}

}  // namespace moe
