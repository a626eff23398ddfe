// layer.hip -- a whole MoE layer for a few tokens (the decode regime: T <= 128
// tokens and T * k <= 1024 picks): top-k gating (MoE systems survey section
// 1.1, eq. (2)), the SwiGLU experts (EP flow step 3) and the gate-weighted sum
// (eq. (1)) in two launches for up to 8 tokens (one more to route, and one
// more again where a block cannot route all of them at a time, for more),
// without a permuted copy of the rows:
//
//   gate/up   h[p][j] = bf16( SiLU(x_t . Wg[e][j]) (x_t . Wu[e][j]) ) for every
//             pick p = t k + i of expert e
//   down      y[t][c] = bf16( sum_i w[t][i] (h[t k + i] . Wd[e_i][c]) )
//
// Bound by the HBM bytes of the live experts' weights, each read once: a
// token's rows are small and come from the caches, and the matrix pipes idle
// mostly. The weights go from memory into registers past the caches, whole
// 128-byte lines of 8 rows a load, are turned into fragments in the wave's own
// LDS, and are the first operand of v_mfma_f32_16x16x32_bf16; the second holds
// up to 16 tokens of one expert, so an expert with one token costs the same
// bytes as one with sixteen. A wave takes all tokens of its expert, up to 128,
// through one pass over its weights. 8-bit weights are widened in registers
// (e4m3 to bf16 is exact) and each 128-column block's product is folded with
// its scale: half the bytes, the same arithmetic on the tokens.
//
// Measured (H 4096, I 1408, 128 experts, k 8): one token 277 MB in 54 us (gate/up
// 36, down 18); 128 tokens on 107 experts, most on 8 of them, 3.69 GB in 580-600 us,
// 6.1-6.3 TB/s (gate/up 385-396, down 193-201); on all 128 experts 4.43 GB in 683
// us, 6.5 TB/s.
#include <type_traits>

#include "device.h"
#include "ffn_device.h"
#include "launch.h"
#include "quant.h"
#include "route_token.h"
#include "stream.h"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kMaxPicks = 1024;
constexpr int kMaxE = 1024;
constexpr int kRouteT = 8;     // most tokens that every gate/up block routes itself
constexpr uint32_t kLdsBytes = 160 * 1024;  // of a compute unit
constexpr int kUpWaves = 4;    // waves of a gate/up block
constexpr int kUpCols = 8;     // intermediate columns of a unit (8 gate + 8 up rows)

// The live experts in id order and their picks: what both launches need of the
// routing. An expert with more than kGroup picks is listed 2 or 4 times (its
// "parts": its share of the down kernel's work), those experts first: their waves
// take the longest, and at the list's end the chip idled behind them (128 tokens,
// most on 8 experts, gate/up: 454 us in id order, 398 so). Each list entry ("slot")
// is one word: expert, first entry in pick, part, picks of the expert (0: no slot).
constexpr int kGroup = 32;
__host__ __device__ __forceinline__ int parts_of(int cnt) { return cnt <= 32 ? 1 : (cnt <= 64 ? 2 : 4); }
__device__ __forceinline__ uint32_t slot_word(int e, int first, int part, int cnt) {
  return (uint32_t)e | (uint32_t)first << 10 | (uint32_t)part << 20 | (uint32_t)cnt << 22;
}
__device__ __forceinline__ int slot_expert(uint32_t s) { return s & 1023; }
__device__ __forceinline__ int slot_first(uint32_t s) { return (s >> 10) & 1023; }
__device__ __forceinline__ int slot_part(uint32_t s) { return (s >> 20) & 3; }
__device__ __forceinline__ int slot_count(uint32_t s) { return s >> 22; }
static_assert(kMaxE <= 1024 && kMaxPicks <= 1024 && kLayerMaxT <= 4 * kGroup, "fields of a slot word");
// Most slots: one an expert, and up to three more for 65 picks (one for 33).
__host__ __device__ constexpr int max_slots(int E, int np) { return (np < E ? np : E) + np / 21; }

struct Plan {
  int32_t* n;      // slots in use
  uint32_t* slot;  // [slots], zero past those in use
  int32_t* pick;   // [T*k] picks (t * k + i) grouped by slot
};

__host__ __device__ __forceinline__ Plan plan_at(int32_t* ws, int slots) {
  return {ws, reinterpret_cast<uint32_t*>(ws + 4), ws + 4 + slots};
}

template <int NP>  // most picks
struct PlanLds {
  int32_t idx[NP];     // expert of each pick
  int32_t pick[NP];    // picks grouped by slot
  int32_t cur[kMaxE];  // counts, then the next free entry of each expert
  uint32_t slot[max_slots(NP, NP)];
  int32_t part[16];
  int32_t n;
};

// Routes all T tokens (G lanes a token, V >= E / G logits a lane; V = 0: reads
// the picks of an earlier launch) and groups the picks, all in one block of NT
// threads. The order of the picks inside an
// expert is not fixed (LDS atomics), and nothing depends on it: a pick is a
// column of a matrix product and goes to a token of its own. publish: this
// block also writes the plan, the picks and weights.
template <int NT, int V, int NP>
__device__ __forceinline__ void route_and_plan(PlanLds<NP>& P, const float* __restrict__ logits, int T,
                                               int E, int k, int G, bool publish,
                                               int32_t* __restrict__ topk_idx,
                                               float* __restrict__ topk_w, const Plan& out,
                                               int slots) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wid = tid / kWave;
  constexpr int NW = NT / kWave;
  for (int e = tid; e < E; e += NT) P.cur[e] = 0;
  const int np = T * k;
  if constexpr (V > 0) {
    const int g = lane & (G - 1), per_pass = NT / G;
    for (int t0 = 0; t0 < T; t0 += per_pass) {
      const int t = t0 + tid / G;
      int id;
      float w;
      route_token<V, false>(logits, t, t < T, E, k, G, g, id, w);
      if (id >= 0) {
        P.idx[t * k + g] = id;
        if (publish) {
          topk_idx[t * k + g] = id;
          topk_w[t * k + g] = w;
        }
      }
    }
  } else {
    for (int p = tid; p < np; p += NT) P.idx[p] = topk_idx[p];
  }
  __syncthreads();
  for (int p = tid; p < np; p += NT) atomicAdd(&P.cur[P.idx[p]], 1);
  __syncthreads();
  // exclusive scan over the experts of three sums in one word: picks, slots of
  // experts with parts (which are listed first: they take the longest), other slots
  constexpr int kHot = 11, kCold = 19;
  static_assert(kMaxPicks < 1 << kHot && 4 * kMaxPicks / 33 < 1 << (kCold - kHot), "fields");
  const auto word_of = [](int c) {
    return c == 0 ? 0 : c > kGroup ? (parts_of(c) << kHot) + c : (1 << kCold) + c;
  };
  const int per = (E + NT - 1) / NT;
  int mine = 0;
  for (int j = 0; j < per; ++j) {
    const int e = tid * per + j;
    const int c = e < E ? P.cur[e] : 0;
    mine += word_of(c);
  }
  int incl = mine;
  for (int o = 1; o < kWave; o <<= 1) {
    const int y = __shfl_up(incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == kWave - 1) P.part[wid] = incl;
  __syncthreads();
  int at = incl - mine, total = 0;
  for (int w = 0; w < NW; ++w) {
    at += w < wid ? P.part[w] : 0;
    total += P.part[w];
  }
  const auto hot_of = [](int w) { return w >> kHot & ((1 << (kCold - kHot)) - 1); };
  const int hot = hot_of(total), n = hot + (total >> kCold);
  for (int j = 0; j < per; ++j) {
    const int e = tid * per + j;
    const int c = e < E ? P.cur[e] : 0;
    if (c > 0) {
      const int first = at & ((1 << kHot) - 1), to = c > kGroup ? hot_of(at) : hot + (at >> kCold);
      const int parts = parts_of(c);
      for (int q = 0; q < parts; ++q) P.slot[to + q] = slot_word(e, first, q, c);
      P.cur[e] = first;
      at += word_of(c);
    }
  }
  if (tid == 0) P.n = n;
  __syncthreads();
  for (int p = tid; p < np; p += NT) P.pick[atomicAdd(&P.cur[P.idx[p]], 1)] = p;
  __syncthreads();
  if (publish) {
    if (tid == 0) *out.n = n;
    for (int s = tid; s < slots; s += NT) out.slot[s] = s < n ? P.slot[s] : 0;
    for (int p = tid; p < np; p += NT) out.pick[p] = P.pick[p];
  }
}

// Two bf16 from two e4m3 (exact).
template <bool kHi>
__device__ __forceinline__ bf16x2 widen2(uint32_t u) {
  return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u, 1.0f, kHi);
}
__device__ __forceinline__ bf16x8 widen8(uint32_t a, uint32_t b) {
  const bf16x2 w0 = widen2<false>(a), w1 = widen2<true>(a), w2 = widen2<false>(b),
               w3 = widen2<true>(b);
  return bf16x8{w0[0], w0[1], w1[0], w1[1], w2[0], w2[1], w3[0], w3[1]};
}

// K steps of the weight stream (stream.h): 64 bf16 or 128 e4m3 columns.
template <bool kFp8>
struct Step {
  static constexpr int kCols = kFp8 ? 128 : 64;
  // 128-byte pieces of a token row a step; their offset is scalar (on the lane's side: 17
  // tokens, H 2048, 64 experts of 8 bits 90 against 88 us).
  static constexpr int kB = kFp8 ? 2 : 1;
};

// Bytes of LDS a wave needs for NB groups of 8 tokens, and the steps in flight: what
// fits 168 registers (three waves a SIMD), or 128 with 8 rows (four).
constexpr int stage_bytes(int NB) { return 2048 + NB * 1024; }
template <bool kFp8, int RW, int NB>
constexpr int kRing = kFp8 ? (NB == 1 ? (RW == 8 ? 6 : 4) : (NB == 2 ? 3 : 2))
                           : (NB == 1 ? (RW == 8 ? 8 : 6) : (NB == 2 ? 4 : (RW == 8 ? 2 : 3)));

// acc[t] += the product of one K step: w, the lane's 16 bytes of two rows (RW = 8: of
// one) and x, of its token of each group of 8; wrow: LDS rows of the weight rows;
// f0, f1 (e4m3): scales of D registers 0-1 and 2-3.
template <bool kFp8, int RW, int NB>
__device__ __forceinline__ void step_product(uint8_t* stage, const int (&wrow)[2],
                                             const v4u (&w)[RW / 8],
                                             const v4u (&x)[NB][Step<kFp8>::kB], float f0, float f1,
                                             f32x4 (&acc)[(NB + 1) / 2]) {
  constexpr int NTL = (NB + 1) / 2;
  const int lane = threadIdx.x & (kWave - 1);
  const int lr = lane >> 3, lc = lane & 7, i = lane & 15, g = lane >> 4;
  uint8_t* xs = stage + 2048;
  const int arow = RW == 8 ? i & 7 : i;  // rows 8-15 of an 8-row unit repeat: not used
#pragma unroll
  for (int r = 0; r < RW / 8; ++r) *reinterpret_cast<v4u*>(stage + tile_at(wrow[r], lc)) = w[r];
  auto put_x = [&](int p) __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < NB; ++b) *reinterpret_cast<v4u*>(xs + tile_at(8 * b + lr, lc)) = x[b][p];
    __builtin_amdgcn_wave_barrier();
  };
  put_x(0);
  // a token tile's rows; with one group of 8 its rows twice (columns 8-15 unused)
  auto trow = [&](int t) { return NB == 1 ? i & 7 : 16 * t + i; };
  if constexpr (kFp8) {
    f32x4 d[NTL];
#pragma unroll
    for (int t = 0; t < NTL; ++t) d[t] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      if (m > 0) put_x(m);
      const v4u q = *reinterpret_cast<const v4u*>(stage + tile_at(arow, 4 * m + g));
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const bf16x8 a = widen8(q[2 * hh], q[2 * hh + 1]);
#pragma unroll
        for (int t = 0; t < NTL; ++t)
          d[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              a, *reinterpret_cast<const bf16x8*>(xs + tile_at(trow(t), 2 * g + hh)), d[t], 0, 0, 0);
      }
      __builtin_amdgcn_wave_barrier();
    }
#pragma unroll
    for (int t = 0; t < NTL; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        acc[t][r] = __builtin_fmaf(d[t][r], r < 2 ? f0 : f1, acc[t][r]);
  } else {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const bf16x8 a = *reinterpret_cast<const bf16x8*>(stage + tile_at(arow, 4 * m + g));
#pragma unroll
      for (int t = 0; t < NTL; ++t)
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            a, *reinterpret_cast<const bf16x8*>(xs + tile_at(trow(t), 4 * m + g)), acc[t], 0, 0, 0);
    }
  }
  __builtin_amdgcn_wave_barrier();
}

// acc[t] += the products of the unit's rows with NB x 8 tokens over n K steps
// from s0, beginning with step s0 + rot. woff: byte offsets in wb of the lane's two
// rows at its chunk (RW = 8: the first only), wrow their LDS rows; xoff[b]: in xb
// of its token of group b at its chunk (kOutside without a token); c0, c1 (e4m3):
// scales of D registers 0-1 and 2-3, one a step (uniform: scalar loads; through the
// vector path they were two of six load instructions a step).
template <bool kFp8, int RW, int NB, int D>
__device__ __forceinline__ void dot_steps(uint8_t* stage, const Buffer& wb,
                                          const uint32_t (&woff)[2], const int (&wrow)[2],
                                          const Buffer& xb, const uint32_t (&xoff)[NB],
                                          const float* __restrict__ c0,
                                          const float* __restrict__ c1,
                                          int s0, int n, int rot, f32x4 (&acc)[(NB + 1) / 2]) {
  constexpr int kB = Step<kFp8>::kB, RI = RW / 8;
  v4u w[D][RI], x[D][NB][kB];
  float a0[D], a1[D];
  auto load = [&](int u, int q) __attribute__((always_inline)) {
    const bool in = q < n;
    int o = q + rot;
    o = o >= n ? o - n : o;
    const uint32_t s = in ? (uint32_t)(s0 + o) : 0;
#pragma unroll
    for (int r = 0; r < RI; ++r) w[u][r] = load16_stream(wb.at(in), woff[r], s * 128);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int p = 0; p < kB; ++p)
        x[u][b][p] = load16(xb.at(in), xoff[b], in ? s * (Step<kFp8>::kCols * 2) + 128 * p : 0);
    if constexpr (kFp8) {
      a0[u] = c0[in ? s : (uint32_t)s0];
      a1[u] = c1[in ? s : (uint32_t)s0];
    }
  };
#pragma unroll
  for (int u = 0; u < D; ++u) load(u, u);
  for (int q = 0; q < n; q += D) {
#pragma unroll
    for (int u = 0; u < D; ++u) {
      step_product<kFp8, RW, NB>(stage, wrow, w[u], x[u], kFp8 ? a0[u] : 0.f, kFp8 ? a1[u] : 0.f, acc);
      load(u, q + u + D);
    }
  }
}

// The same for NG groups of kGroup tokens, each step's weights loaded once for all of
// them: xoff[q], acc[q] are group q's; XD: groups of tokens in flight. (A pass over
// the weights for each group, 128 tokens, most on 8 experts: gate/up 478 against
// 454 us, down 249 against 212; memory reads 2.84 and 1.51 GB for 2.47 and 1.23 GB.)
template <bool kFp8, int RW, int NG, int XD>
__device__ __forceinline__ void dot_steps_groups(uint8_t* stage, const Buffer& wb,
                                                 const uint32_t (&woff)[2], const int (&wrow)[2],
                                                 const Buffer& xb, const uint32_t (&xoff)[NG][4],
                                                 const float* __restrict__ c0,
                                                 const float* __restrict__ c1, int s0, int n,
                                                 int rot, f32x4 (&acc)[NG][2]) {
  constexpr int kB = Step<kFp8>::kB, RI = RW / 8, kM = kFp8 ? 2 : 1;
  static_assert(2 * NG % XD == 0, "two steps' groups are whole turns of the ring");
  const int lane = threadIdx.x & (kWave - 1);
  const int lr = lane >> 3, lc = lane & 7, i = lane & 15, g = lane >> 4;
  v4u w[2][RI], x[XD][4][kB];
  float a0[2], a1[2];
  const auto step_at = [&](int q) -> uint32_t {
    const int o = q + rot;
    return q < n ? (uint32_t)(s0 + (o >= n ? o - n : o)) : 0;
  };
  auto load_w = [&](int u, int q) __attribute__((always_inline)) {
    const uint32_t s = step_at(q);
#pragma unroll
    for (int r = 0; r < RI; ++r) w[u][r] = load16_stream(wb.at(q < n), woff[r], s * 128);
    if constexpr (kFp8) {
      a0[u] = c0[q < n ? s : (uint32_t)s0];
      a1[u] = c1[q < n ? s : (uint32_t)s0];
    }
  };
  auto load_x = [&](int u, int q, int grp) __attribute__((always_inline)) {
    const uint32_t s = step_at(q);
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int p = 0; p < kB; ++p)
        x[u][b][p] = load16(xb.at(q < n), xoff[grp][b],
                            q < n ? s * (Step<kFp8>::kCols * 2) + 128 * p : 0);
  };
  uint8_t* xs = stage + 2048;
  const int arow = RW == 8 ? i & 7 : i;
  load_w(0, 0);
  load_w(1, 1);
#pragma unroll
  for (int e = 0; e < XD; ++e) load_x(e, e / NG, e % NG);
  for (int q = 0; q < n; q += 2) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int r = 0; r < RI; ++r) *reinterpret_cast<v4u*>(stage + tile_at(wrow[r], lc)) = w[u][r];
      __builtin_amdgcn_wave_barrier();
      bf16x8 a[2][kM];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        if constexpr (kFp8) {
          const v4u v = *reinterpret_cast<const v4u*>(stage + tile_at(arow, 4 * m + g));
          a[m][0] = widen8(v[0], v[1]);
          a[m][1] = widen8(v[2], v[3]);
        } else {
          a[m][0] = *reinterpret_cast<const bf16x8*>(stage + tile_at(arow, 4 * m + g));
        }
      }
      const float f0 = kFp8 ? a0[u] : 0.f, f1 = kFp8 ? a1[u] : 0.f;
      load_w(u, q + u + 2);
#pragma unroll
      for (int grp = 0; grp < NG; ++grp) {
        const int v = (u * NG + grp) % XD;
        f32x4 d[2] = {acc[grp][0], acc[grp][1]};
        if constexpr (kFp8) d[0] = d[1] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int p = 0; p < kB; ++p) {
#pragma unroll
          for (int b = 0; b < 4; ++b)
            *reinterpret_cast<v4u*>(xs + tile_at(8 * b + lr, lc)) = x[v][b][p];
          __builtin_amdgcn_wave_barrier();
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int t = 0; t < 2; ++t)
              d[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  kFp8 ? a[p][m] : a[m][0],
                  *reinterpret_cast<const bf16x8*>(
                      xs + tile_at(16 * t + i, kFp8 ? 2 * g + m : 4 * m + g)),
                  d[t], 0, 0, 0);
          __builtin_amdgcn_wave_barrier();
        }
        load_x(v, q + u + (grp + XD) / NG, (grp + XD) % NG);
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if constexpr (kFp8) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[grp][t][r] = __builtin_fmaf(d[t][r], r < 2 ? f0 : f1, acc[grp][t][r]);
          } else {
            acc[grp][t] = d[t];
          }
      }
    }
  }
}

// Gate/up: a unit is kUpCols intermediate columns of one live expert (8 gate and
// 8 up rows) for all its picks, computed by KS waves, each a part of the K
// steps (their sums are added in LDS in a fixed order); a block has kUpWaves /
// KS units. MFMA row i is gate row 2 (i / 4) + i % 4 for i % 4 < 2, else the up
// row of the same column, so a lane's four results are g, g, u, u of two
// neighbouring columns. kV > 0: the block routes all tokens itself (kV logits a
// lane), block (0, 0) publishes; kV = 0: the plan is in the workspace. kMaxNB:
// most eights of picks in a pass (1 with up to kRouteT tokens).
template <int kV, int KS, bool kFp8, int kMaxNB>
__global__ __launch_bounds__(kWave * kUpWaves, kFp8 || kMaxNB > 1 ? 3 : 4) void layer_gate_up_kernel(
    const float* __restrict__ logits, const uint16_t* __restrict__ x, int T, int H, int E, int k,
    int I, int G, const uint8_t* __restrict__ w, const float* __restrict__ wsc,
    int32_t* __restrict__ topk_idx, float* __restrict__ topk_w, Plan plan,
    uint16_t* __restrict__ h) {
  static_assert(kV == 0 || kRouteT <= 8 * kMaxNB, "a routing block's picks fit one pass");
  __shared__ typename std::conditional<(kV > 0), PlanLds<32 * kRouteT>, int>::type P;
  __shared__ __attribute__((aligned(16))) uint8_t stage[kUpWaves][stage_bytes(kMaxNB)];
  __shared__ f32x4 red[KS > 1 ? kUpWaves : 1][(kMaxNB + 1) / 2][kWave];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wid = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int slot = blockIdx.y;
  const int32_t* pick;
  uint32_t word;
  if constexpr (kV > 0) {
    route_and_plan<kWave * kUpWaves, kV>(P, logits, T, E, k, G, blockIdx.x == 0 && slot == 0,
                                         topk_idx, topk_w, plan, gridDim.y);
    word = slot < P.n ? P.slot[slot] : 0;
    pick = P.pick;
  } else {
    word = plan.slot[slot];
    pick = plan.pick;
  }
  word = __builtin_amdgcn_readfirstlane(word);
  const int e = slot_expert(word);
  const int cnt = slot_count(word);
  if (cnt == 0 || slot_part(word) > 0) return;  // uniform over the block
  const int ks = wid % KS, unit = (int)blockIdx.x * (kUpWaves / KS) + wid / KS;
  pick += slot_first(word);
  const int j0 = unit * kUpCols;
  const int i = lane & 15, g = lane >> 4, lr = lane >> 3, lc = lane & 7;
  constexpr int kWB = kFp8 ? 1 : 2;  // bytes of a weight
  const Buffer wb = {w + (int64_t)e * 2 * I * H * kWB, (uint32_t)(2 * I) * (uint32_t)(H * kWB)};
  const Buffer xb = {x, (uint32_t)T * (uint32_t)(2 * H)};
  const uint32_t woff[2] = {(uint32_t)(j0 + lr) * (uint32_t)(H * kWB) + 16 * lc,
                            (uint32_t)(I + j0 + lr) * (uint32_t)(H * kWB) + 16 * lc};
  const int wrow[2] = {4 * (lr >> 1) + (lr & 1), 4 * (lr >> 1) + (lr & 1) + 2};
  const int steps = H / Step<kFp8>::kCols;
  const int s0 = steps * ks / KS, n = steps * (ks + 1) / KS - s0;
  const int rot = n > 0 ? (int)(blockIdx.x + slot) * 5 % n : 0;  // alike in a block: x from L1
  const float *c0 = nullptr, *c1 = nullptr;
  if constexpr (kFp8) {
    c0 = wsc + ((int64_t)e * (2 * I / kQuantBlock) + j0 / kQuantBlock) * steps;
    c1 = c0 + (int64_t)(I / kQuantBlock) * steps;
  }
  const auto offset_of = [&](int c) {
    return c < cnt ? (uint32_t)(pick[c] / k) * (uint32_t)(2 * H) + 16 * lc : kOutside;
  };
  const auto store = [&](int c, const f32x4& v, bool on) __attribute__((always_inline)) {
    if (c < cnt && on) {
      const uint32_t hv = bf16x2_rne(silu(v[0]) * v[2], silu(v[1]) * v[3]);
      *reinterpret_cast<uint32_t*>(h + (int64_t)pick[c] * I + j0 + 2 * g) = hv;
    }
  };
  auto pass = [&](auto nb_) __attribute__((always_inline)) {
    constexpr int NB = decltype(nb_)::value, NTL = (NB + 1) / 2;
    uint32_t xoff[NB];
    f32x4 acc[NTL];
#pragma unroll
    for (int b = 0; b < NB; ++b) xoff[b] = offset_of(8 * b + lr);
#pragma unroll
    for (int t = 0; t < NTL; ++t) acc[t] = f32x4{0, 0, 0, 0};
    dot_steps<kFp8, 16, NB, kRing<kFp8, 16, NB>>(stage[wid], wb, woff, wrow, xb, xoff, c0, c1, s0,
                                             n, rot, acc);
    if constexpr (KS > 1) {
#pragma unroll
      for (int t = 0; t < NTL; ++t) red[wid][t][lane] = acc[t];
      __syncthreads();
    }
#pragma unroll
    for (int t = 0; t < NTL; ++t) {
      if (KS > 1 && t % KS != ks) continue;  // uniform over the wave
      f32x4 v = acc[t];
      if constexpr (KS > 1) {
        v = red[wid - ks][t][lane];
#pragma unroll
        for (int q = 1; q < KS; ++q) v += red[wid - ks + q][t][lane];
      }
      store(16 * t + i, v, NB > 1 || i < 8);
    }
  };
  auto groups = [&](auto ng_) __attribute__((always_inline)) {
    constexpr int NG = decltype(ng_)::value;
    uint32_t xoff[NG][4];
    f32x4 acc[NG][2];
#pragma unroll
    for (int q = 0; q < NG; ++q)
#pragma unroll
      for (int b = 0; b < 4; ++b) xoff[q][b] = offset_of(q * kGroup + 8 * b + lr);
#pragma unroll
    for (int q = 0; q < NG; ++q) acc[q][0] = acc[q][1] = f32x4{0, 0, 0, 0};
    dot_steps_groups<kFp8, 16, NG, kFp8 ? 1 : 2>(stage[wid], wb, woff, wrow, xb, xoff, c0, c1, s0,
                                                 n, rot, acc);
#pragma unroll
    for (int q = 0; q < NG; ++q)
#pragma unroll
      for (int t = 0; t < 2; ++t) store(q * kGroup + 16 * t + i, acc[q][t], true);
  };
  if (kMaxNB == 1 || cnt <= 8) {
    pass(std::integral_constant<int, 1>{});
  } else if constexpr (kMaxNB > 1) {
    static_assert(KS == 1, "the groups' sums are not joined");
    if (cnt <= 16) pass(std::integral_constant<int, 2>{});
    else if (cnt <= kGroup) pass(std::integral_constant<int, 4>{});
    else if (cnt <= 2 * kGroup) groups(std::integral_constant<int, 2>{});
    else groups(std::integral_constant<int, 4>{});
  }
}

// Routing and plan alone (one block), where routing in every gate/up block
// would cost more; V = 0: the plan of picks already made.
template <int V>
__global__ __launch_bounds__(1024) void layer_plan_kernel(const float* __restrict__ logits, int T,
                                                          int E, int k, int G, int slots,
                                                          int32_t* __restrict__ topk_idx,
                                                          float* __restrict__ topk_w, Plan plan) {
  __shared__ PlanLds<kMaxPicks> P;
  route_and_plan<1024, V>(P, logits, T, E, k, G, true, topk_idx, topk_w, plan, slots);
}

// Down and combine: a block computes RW columns of y for all tokens. The K steps
// of all slots in a row are cut into one range a wave (an expert's parts are one
// run of them, in which a step of its weights counts once a part); at the end of
// an expert's share of its range a wave adds gate weight x result to its own fp32
// rows of y in LDS (an expert's picks are different tokens), and the waves' rows
// are added in a fixed order at the end. Sixteen waves have registers for two
// groups of tokens at a time, so four take two passes.
template <bool kFp8, int RW, int kMaxNB, int DW>
__global__ __launch_bounds__(kWave * DW) void layer_down_kernel(
    const uint16_t* __restrict__ h, int T, int H, int k, int I, int slots,
    const uint8_t* __restrict__ w, const float* __restrict__ wsc,
    const float* __restrict__ topk_w, Plan plan, uint16_t* __restrict__ y) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int np = T * k;
  uint8_t* stage = lds;                                       // [DW][stage_bytes]
  float* ya = reinterpret_cast<float*>(lds + DW * stage_bytes(kMaxNB));
  float* gw = ya + (size_t)DW * T * RW;               // [np], ya: [DW][T][RW]
  uint32_t* sl = reinterpret_cast<uint32_t*>(gw + np);        // [slots]
  uint16_t* pk = reinterpret_cast<uint16_t*>(sl + slots);     // [np]
  constexpr int NT = kWave * DW;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wid = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c0 = blockIdx.x * RW;
  const int n = *plan.n;
  for (int p = tid; p < np; p += NT) {
    gw[p] = topk_w[p];
    pk[p] = (uint16_t)plan.pick[p];
  }
  for (int s = tid; s < slots; s += NT) sl[s] = plan.slot[s];
  for (int q = tid; q < DW * T * RW; q += NT) ya[q] = 0.f;
  __syncthreads();
  const int steps = I / Step<kFp8>::kCols;
  const int64_t total = (int64_t)n * steps;
  int at = (int)(total * wid / DW);
  const int end = (int)(total * (wid + 1) / DW);
  const int i = lane & 15, g = lane >> 4, lr = lane >> 3, lc = lane & 7;
  float* mine = ya + (size_t)wid * T * RW;
  constexpr int kWB = kFp8 ? 1 : 2;
  const Buffer hb = {h, (uint32_t)np * (uint32_t)(2 * I)};
  const uint32_t woff[2] = {(uint32_t)(c0 + lr) * (uint32_t)(I * kWB) + 16 * lc,
                            (uint32_t)(c0 + 8 + lr) * (uint32_t)(I * kWB) + 16 * lc};
  const int wrow[2] = {lr, 8 + lr};
  uint8_t* const my_stage = stage + wid * stage_bytes(kMaxNB);
  const auto weights_of = [&](uint32_t word) -> Buffer {
    return {w + (int64_t)slot_expert(word) * H * I * kWB, (uint32_t)H * (uint32_t)(I * kWB)};
  };
  const auto scales_of = [&](uint32_t word) -> const float* {
    return kFp8 ? wsc + ((int64_t)slot_expert(word) * (H / kQuantBlock) + c0 / kQuantBlock) * steps
                : nullptr;
  };
  const auto offset_of = [&](uint32_t word, int c) {
    return c < slot_count(word)
               ? (uint32_t)pk[slot_first(word) + c] * (uint32_t)(2 * I) + 16 * lc
               : kOutside;
  };
  // gate weight x result of the 16 picks from p0, to the wave's own rows of y
  auto add = [&](uint32_t word, int p0, const f32x4& d, bool on) __attribute__((always_inline)) {
    const int c = p0 + i;
    if (c < slot_count(word) && on && (RW == 16 || g < 2)) {
      const int p = pk[slot_first(word) + c];
      const float gp = gw[p];
      f32x4* dst = reinterpret_cast<f32x4*>(mine + (p / k) * RW + 4 * g);
      f32x4 v = *dst;
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = __builtin_fmaf(gp, d[r], v[r]);
      *dst = v;
    }
  };
  // The run of experts of up to 8 picks (the most of them) that begins here: their
  // K steps are one stream, the loads run into the next expert while this one's last
  // steps are computed (each expert a stream of its own: 17 tokens, H 2048, 64 experts
  // of 8 bits 43 against 34 us; 128 tokens, H 4096, 128 experts 211 against 201).
  auto run_of_few = [&]() __attribute__((always_inline)) {
    constexpr int D = kRing<kFp8, RW, 1>, kB = Step<kFp8>::kB, RI = RW / 8;
    v4u wv[D][RI], x[D][1][kB];
    float a0[D];
    // loads: the slot they are in, its steps [s0, s0 + n) beginning with s0 + o, left of them
    int lslot = at / steps, s0 = at - lslot * steps, next = s0, n = 0, o = 0, left = 0, total = 0;
    bool on = true;
    Buffer wb = {w, 0};
    uint32_t hoff = kOutside;
    const float* sc = wsc;
    auto enter = [&]() __attribute__((always_inline)) {
      const uint32_t word =
          at + total < end ? (uint32_t)__builtin_amdgcn_readfirstlane(sl[lslot]) : 0;
      on = slot_count(word) > 0 && slot_count(word) <= 8;
      if (on) {
        s0 = next;
        n = steps - s0 < end - at - total ? steps - s0 : end - at - total;
        wb = weights_of(word);
        sc = scales_of(word);
        hoff = offset_of(word, lr);
        o = blockIdx.x * 5 % n;
        left = n;
        total += n;
        next = 0;
        ++lslot;
      }
    };
    auto load = [&](int u) __attribute__((always_inline)) {
      const uint32_t s = on ? (uint32_t)(s0 + o) : 0;
#pragma unroll
      for (int r = 0; r < RI; ++r) wv[u][r] = load16_stream(wb.at(on), woff[r], s * 128);
#pragma unroll
      for (int p = 0; p < kB; ++p)
        x[u][0][p] = load16(hb.at(on), hoff, on ? s * (Step<kFp8>::kCols * 2) + 128 * p : 0);
      if constexpr (kFp8) a0[u] = sc[on ? s : (uint32_t)s0];
      o = o + 1 == n ? 0 : o + 1;
      if (on && --left == 0) enter();
    };
    enter();
    int cslot = at / steps, cleft = n, done = 0;  // the slot computed, what is left of it
    f32x4 acc[1] = {f32x4{0, 0, 0, 0}};
#pragma unroll
    for (int u = 0; u < D; ++u) load(u);
    for (int q = 0; q < total; q += D) {
#pragma unroll
      for (int u = 0; u < D; ++u) {
        step_product<kFp8, RW, 1>(my_stage, wrow, wv[u], x[u], kFp8 ? a0[u] : 0.f,
                                  kFp8 ? a0[u] : 0.f, acc);
        ++done;
        if (--cleft == 0) {
          add(__builtin_amdgcn_readfirstlane(sl[cslot++]), 0, acc[0], i < 8);
          acc[0] = f32x4{0, 0, 0, 0};
          // the loads are in the next slot of the run already, if there is one
          cleft = total - done < steps ? total - done : steps;
        }
        load(u);
      }
    }
    at += total;
  };
  while (at < end) {
    const int slot = at / steps;
    const uint32_t word = __builtin_amdgcn_readfirstlane(sl[slot]);
    const int cnt = slot_count(word), parts = parts_of(cnt);
    if (kMaxNB == 1 || cnt <= 8) {
      run_of_few();
      continue;
    }
    // the parts of an expert are one run of parts * steps entries, parts of them a step
    const int from = at - (slot - slot_part(word)) * steps;
    const int to = end - at < parts * steps - from ? from + (end - at) : parts * steps;
    at += to - from;
    const int s0 = (from + parts - 1) / parts, s1 = (to + parts - 1) / parts;
    if (s0 == s1) continue;
    const int rot = blockIdx.x * 5 % (s1 - s0);
    const Buffer wb = weights_of(word);
    const float* sc = scales_of(word);
    auto pass = [&](auto nb_) __attribute__((always_inline)) {
      constexpr int NB = decltype(nb_)::value, NTL = (NB + 1) / 2;
      uint32_t hoff[NB];
      f32x4 acc[NTL];
#pragma unroll
      for (int b = 0; b < NB; ++b) hoff[b] = offset_of(word, 8 * b + lr);
#pragma unroll
      for (int t = 0; t < NTL; ++t) acc[t] = f32x4{0, 0, 0, 0};
      dot_steps<kFp8, RW, NB, kRing<kFp8, RW, NB>>(my_stage, wb, woff, wrow, hb, hoff, sc, sc, s0,
                                                   s1 - s0, rot, acc);
#pragma unroll
      for (int t = 0; t < NTL; ++t) add(word, 16 * t, acc[t], true);
    };
    auto groups = [&](auto ng_, int first) __attribute__((always_inline)) {
      constexpr int NG = decltype(ng_)::value;
      uint32_t hoff[NG][4];
      f32x4 acc[NG][2];
#pragma unroll
      for (int q = 0; q < NG; ++q)
#pragma unroll
        for (int b = 0; b < 4; ++b) hoff[q][b] = offset_of(word, first + q * kGroup + 8 * b + lr);
#pragma unroll
      for (int q = 0; q < NG; ++q) acc[q][0] = acc[q][1] = f32x4{0, 0, 0, 0};
      dot_steps_groups<kFp8, RW, NG, DW == 16 ? 1 : (kFp8 ? 2 : 4)>(
          my_stage, wb, woff, wrow, hb, hoff, sc, sc, s0, s1 - s0, rot, acc);
#pragma unroll
      for (int q = 0; q < NG; ++q)
#pragma unroll
        for (int t = 0; t < 2; ++t) add(word, first + q * kGroup + 16 * t, acc[q][t], true);
    };
    if constexpr (kMaxNB > 1) {
      if (cnt <= 16) pass(std::integral_constant<int, 2>{});
      else if (cnt <= kGroup) pass(std::integral_constant<int, 4>{});
      else if (DW == 8 && parts == 4) groups(std::integral_constant<int, DW == 8 ? 4 : 2>{}, 0);
      else
        for (int q = 0; q < parts; q += 2) groups(std::integral_constant<int, 2>{}, q * kGroup);
    }
  }
  __syncthreads();
  for (int q = tid; q < T * RW / 2; q += NT) {
    const int t = q / (RW / 2), c = (q - t * (RW / 2)) * 2;
    float2 a = {0.f, 0.f};
#pragma unroll
    for (int v = 0; v < DW; ++v) {
      const float2 u = *reinterpret_cast<const float2*>(ya + ((size_t)v * T + t) * RW + c);
      a.x += u.x;
      a.y += u.y;
    }
    *reinterpret_cast<uint32_t*>(y + (int64_t)t * H + c0 + c) = bf16x2_rne(a.x, a.y);
  }
}

// Lanes a token (a power of two >= k): as few as leave at most V logits a lane.
int route_lanes(int E, int k, int V) {
  int G = 1;
  while (G < kWave && (G < k || G * V < E)) G <<= 1;
  return G;
}

}  // namespace

int64_t layer_plan_ints(int T, int E, int k) {
  return 4 + (int64_t)max_slots(E, T * k) + T * k;
}

namespace {

template <bool kFp8>
hipError_t run_layer(const float* logits, const void* x, int T, int H, int E, int k, int I,
                     const void* w_gate_up, const float* s_gate_up, const void* w_down,
                     const float* s_down, int32_t* topk_idx, float* topk_w, void* h,
                     int32_t* plan_ws, void* y, hipStream_t s) {
  const int np = T * k;
  const int slots = T > kGroup ? max_slots(E, np) : (np < E ? np : E);  // no parts with few tokens
  const Plan plan = plan_at(plan_ws, slots);
  auto up = [&](auto kernel, int KS, int G) {
    return launch(kernel, dim3((unsigned)(I / kUpCols * KS / kUpWaves), (unsigned)slots),
                  dim3(kWave * kUpWaves), 0, s, logits, static_cast<const uint16_t*>(x), T, H, E, k,
                  I, G, static_cast<const uint8_t*>(w_gate_up), s_gate_up, topk_idx, topk_w, plan,
                  static_cast<uint16_t*>(h));
  };
  hipError_t err;
  if (T <= kRouteT) {
    // two waves a unit while that is what fills the chip (16 waves a compute
    // unit): T = 1 up launch 36 us against 41 with four; T = 8 with 8-bit weights
    // 101 us with one against 119 with two
    const int G4 = route_lanes(E, k, 4), G16 = route_lanes(E, k, 16);
    if (slots * (I / kUpCols) >= 4096)
      err = E <= 256 ? up(layer_gate_up_kernel<4, 1, kFp8, 1>, 1, G4)
                     : up(layer_gate_up_kernel<16, 1, kFp8, 1>, 1, G16);
    else
      err = E <= 256 ? up(layer_gate_up_kernel<4, 2, kFp8, 1>, 2, G4)
                     : up(layer_gate_up_kernel<16, 2, kFp8, 1>, 2, G16);
  } else {
    auto go = [&](auto kernel, int V) {
      return launch(kernel, dim3(1), dim3(1024), 0, s, logits, T, E, k, route_lanes(E, k, V), slots,
                    topk_idx, topk_w, plan);
    };
    // one block routes as many tokens as it can take at a time; more of them
    // are routed by a launch of their own (T = 128, E = 128, k = 8: 19 us for both
    // in one block)
    if (T * route_lanes(E, k, 4) <= 1024 && E <= 256) {
      err = go(layer_plan_kernel<4>, 4);
    } else {
      err = launch_route(logits, T, E, k, topk_idx, topk_w, s);
      if (err != hipSuccess) return err;
      err = go(layer_plan_kernel<0>, 4);
    }
    if (err != hipSuccess) return err;
    err = up(layer_gate_up_kernel<0, 1, kFp8, 4>, 1, 0);
  }
  if (err != hipSuccess) return err;
  auto lds = [&](int RW, int NB, int DW) {
    return (uint32_t)(DW * (stage_bytes(NB) + T * RW * 4) + np * 4 + slots * 4 + np * 2);
  };
  auto down = [&](auto rw, auto nb, auto dw) {
    constexpr int RW = decltype(rw)::value, NB = decltype(nb)::value, DW = decltype(dw)::value;
    return launch(layer_down_kernel<kFp8, RW, NB, DW>, dim3((unsigned)(H / RW)), dim3(kWave * DW),
                  lds(RW, NB, DW), s, static_cast<const uint16_t*>(h), T, H, k, I, slots,
                  static_cast<const uint8_t*>(w_down), s_down, topk_w, plan,
                  static_cast<uint16_t*>(y));
  };
  auto columns = [&](auto rw) {
    using I1 = std::integral_constant<int, 1>;
    using I4 = std::integral_constant<int, 4>;
    using I8 = std::integral_constant<int, 8>;
    using I16 = std::integral_constant<int, 16>;
    if (T <= 8) return down(rw, I1{}, I16{});
    if constexpr (decltype(rw)::value == 8)
      if (lds(8, 4, 16) <= kLdsBytes) return down(rw, I4{}, I16{});
    return down(rw, I4{}, I8{});
  };
  // 16 columns a block where that makes a block for every compute unit
  return H / 16 >= 256 ? columns(std::integral_constant<int, 16>{})
                       : columns(std::integral_constant<int, 8>{});
}

}  // namespace

hipError_t launch_layer(const float* logits, const void* x, int T, int H, int E, int k, int I,
                        bool fp8, const void* w_gate_up, const float* s_gate_up,
                        const void* w_down, const float* s_down, int32_t* topk_idx, float* topk_w,
                        void* h, int32_t* plan_ws, void* y, hipStream_t s) {
  if (T == 0) return hipSuccess;
  return fp8 ? run_layer<true>(logits, x, T, H, E, k, I, w_gate_up, s_gate_up, w_down, s_down,
                               topk_idx, topk_w, h, plan_ws, y, s)
             : run_layer<false>(logits, x, T, H, E, k, I, w_gate_up, s_gate_up, w_down, s_down,
                                topk_idx, topk_w, h, plan_ws, y, s);
}

}  // namespace moe
