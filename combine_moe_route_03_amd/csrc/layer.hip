// layer.hip -- a whole MoE layer for a few tokens (the decode regime: T <= 128
// tokens and T * k <= 1024 picks): top-k gating (MoE systems survey section
// 1.1, eq. (2)), the SwiGLU experts (EP flow step 3) and the gate-weighted sum
// (eq. (1)) in two launches, without a permuted copy of the rows:
//
//   gate/up   h[p][j] = bf16( SiLU(x_t . Wg[e][j]) (x_t . Wu[e][j]) ) for every
//             pick p = t k + i of expert e
//   down      y[t][c] = bf16( sum_i w[t][i] (h[t k + i] . Wd[e_i][c]) )
//
// Bound by the HBM bytes of the live experts' weights, each read once: a
// token's rows are small and come from the caches, and the matrix pipes idle
// mostly. The weights go from memory into registers (nothing re-uses a weight
// inside a block, so LDS would only add a stop), as the first operand of
// v_mfma_f32_16x16x32_bf16; the second holds up to 16 tokens of one expert, so
// an expert with one token costs the same bytes as one with sixteen. 8-bit
// weights are widened in registers (e4m3 to bf16 is exact) and each 128-column
// block's product is folded with its scale: half the bytes, the same
// arithmetic on the tokens.
#include <type_traits>

#include "device.h"
#include "ffn_device.h"
#include "launch.h"
#include "quant.h"
#include "route_token.h"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxPicks = 1024;
constexpr int kRouteT = 4;  // most tokens that every gate/up block routes itself
constexpr int kMaxE = 1024;
constexpr int kUpWaves = 4;    // waves of a gate/up block: each takes every fourth K step
constexpr int kUpCols = 8;     // intermediate columns of a gate/up block (8 gate + 8 up rows)
constexpr int kDownWaves = 8;  // waves of a down block: each takes one range of K steps
constexpr int kDownCols = 16;  // output columns of a down block

// The live experts in id order and their picks: what both launches need of the
// routing. In the workspace and, while it is built, in LDS.
struct Plan {
  int32_t* n;       // live experts ("slots")
  int32_t* expert;  // [slots]
  int32_t* first;   // [slots + 1] first entry of each slot in pick
  int32_t* pick;    // [T*k] picks (t * k + i) grouped by slot
};

__host__ __device__ __forceinline__ Plan plan_at(int32_t* ws, int slots) {
  return {ws, ws + 4, ws + 4 + slots, ws + 4 + 2 * slots + 1};
}

template <int NP>  // most picks
struct PlanLds {
  int32_t idx[NP];     // expert of each pick
  int32_t pick[NP];    // picks grouped by slot
  int32_t cur[kMaxE];  // counts, then the next free entry of each expert
  int32_t expert[NP];
  int32_t first[NP + 1];
  int32_t part[16];
  int32_t n;
};

// Routes all T tokens (one wave a token at a time, V >= E / 64 logits a lane)
// and groups the picks, all in one block of NT threads. The order of the picks
// inside a slot is not fixed (LDS atomics), and nothing depends on it: a pick
// is a column of a matrix product and goes to a token of its own.
template <int NT, int V, int NP>
__device__ __forceinline__ void route_and_plan(PlanLds<NP>& P, const float* __restrict__ logits, int T,
                                               int E, int k, bool publish,
                                               int32_t* __restrict__ topk_idx,
                                               float* __restrict__ topk_w, const Plan& out) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wid = tid / kWave;
  constexpr int NW = NT / kWave;
  for (int e = tid; e < E; e += NT) P.cur[e] = 0;
  for (int t = wid; t < T; t += NW) {
    int id;
    float w;
    route_token<V, false>(logits, t, true, E, k, kWave, lane, id, w);
    if (id >= 0) {
      P.idx[t * k + lane] = id;
      if (publish) {
        topk_idx[t * k + lane] = id;
        topk_w[t * k + lane] = w;
      }
    }
  }
  __syncthreads();
  const int np = T * k;
  for (int p = tid; p < np; p += NT) atomicAdd(&P.cur[P.idx[p]], 1);
  __syncthreads();
  // exclusive scan over the experts of (live << 16) + count
  const int per = (E + NT - 1) / NT;
  int mine = 0;
  for (int j = 0; j < per; ++j) {
    const int e = tid * per + j;
    const int c = e < E ? P.cur[e] : 0;
    mine += c > 0 ? (1 << 16) + c : 0;
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
  for (int j = 0; j < per; ++j) {
    const int e = tid * per + j;
    const int c = e < E ? P.cur[e] : 0;
    if (c > 0) {
      P.expert[at >> 16] = e;
      P.first[at >> 16] = at & 0xFFFF;
      P.cur[e] = at & 0xFFFF;
      at += (1 << 16) + c;
    }
  }
  const int n = total >> 16;
  if (tid == 0) {
    P.n = n;
    P.first[n] = np;
  }
  __syncthreads();
  for (int p = tid; p < np; p += NT) P.pick[atomicAdd(&P.cur[P.idx[p]], 1)] = p;
  __syncthreads();
  if (publish) {
    if (tid == 0) *out.n = n;
    for (int s = tid; s < n; s += NT) out.expert[s] = P.expert[s];
    for (int s = tid; s <= n; s += NT) out.first[s] = P.first[s];
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

// One K step is 128 bytes of a weight row: 64 bf16 or 128 e4m3 columns. Lane
// l takes bytes [32 g, 32 g + 32) of row l % 16, g = l / 16, and the same
// columns of token l % 16 (the order of k is the same in both operands, so it
// does not matter which of an instruction's k they are).
template <bool kFp8>
struct Step {
  static constexpr int kCols = kFp8 ? 128 : 64;
  static constexpr int kB = kFp8 ? 4 : 2;  // 16-byte token vectors and MFMAs a step
};

// acc[nt] += the products of this lane's weight row with NT x 16 tokens over
// the K steps s0, s0 + stride, ... < s1. wp: the lane's weight row at its g
// offset; xp[nt]: the lane's token rows at theirs. scale0 / scale1 (e4m3):
// scales of the row blocks of D registers 0-1 and 2-3, one a step.
template <bool kFp8, int NT, int U>
__device__ __forceinline__ void dot_steps(const uint8_t* __restrict__ wp,
                                          const uint16_t* const (&xp)[NT],
                                          const float* __restrict__ scale0,
                                          const float* __restrict__ scale1, int s0, int s1,
                                          int stride, f32x4 (&acc)[NT]) {
  constexpr int kB = Step<kFp8>::kB;
  auto group = [&](auto un, int s) __attribute__((always_inline)) {
    constexpr int N = decltype(un)::value;
    v4u w[N][2], x[N][NT][kB];
    float c0[N], c1[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const v4u* p = reinterpret_cast<const v4u*>(wp + (int64_t)(s + u * stride) * 128);
      w[u][0] = load_stream(p);
      w[u][1] = load_stream(p + 1);
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const v4u* p =
            reinterpret_cast<const v4u*>(xp[nt] + (int64_t)(s + u * stride) * Step<kFp8>::kCols);
#pragma unroll
        for (int b = 0; b < kB; ++b) x[u][nt][b] = p[b];
      }
      if constexpr (kFp8) {
        c0[u] = scale0[s + u * stride];
        c1[u] = scale1[s + u * stride];
      }
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
      if constexpr (kFp8) {
        bf16x8 a[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) a[b] = widen8(w[u][b >> 1][2 * (b & 1)], w[u][b >> 1][2 * (b & 1) + 1]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          f32x4 t = {0, 0, 0, 0};
#pragma unroll
          for (int b = 0; b < 4; ++b)
            t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                a[b], __builtin_bit_cast(bf16x8, x[u][nt][b]), t, 0, 0, 0);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[nt][r] = __builtin_fmaf(t[r], r < 2 ? c0[u] : c1[u], acc[nt][r]);
        }
      } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int b = 0; b < 2; ++b)
            acc[nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8, w[u][b]), __builtin_bit_cast(bf16x8, x[u][nt][b]),
                acc[nt], 0, 0, 0);
      }
    }
  };
  int s = s0;
  for (; s + (U - 1) * stride < s1; s += U * stride) group(std::integral_constant<int, U>{}, s);
  for (; s < s1; s += stride) group(std::integral_constant<int, 1>{}, s);
}

// Gate/up: block (unit, slot) computes kUpCols intermediate columns of one live
// expert for all its picks. MFMA row i is gate row 2 (i / 4) + i % 4 for i % 4
// < 2, else the up row of the same column, so a lane's four results are g, g,
// u, u of two neighbouring columns. kV > 0: the block routes all tokens itself
// (kV logits a lane), block (0, 0) publishes; kV = 0: the plan is in the
// workspace.
template <int kV, bool kFp8>
__global__ __launch_bounds__(kWave * kUpWaves) void layer_gate_up_kernel(
    const float* __restrict__ logits, const uint16_t* __restrict__ x, int T, int H, int E, int k,
    int I, const uint8_t* __restrict__ w, const float* __restrict__ wsc,
    int32_t* __restrict__ topk_idx, float* __restrict__ topk_w, Plan plan,
    uint16_t* __restrict__ h) {
  // a block that routes holds at most kRouteT tokens: one MFMA column group
  constexpr int kMaxNT = kV > 0 ? 1 : 4;
  __shared__ typename std::conditional<(kV > 0), PlanLds<32 * kRouteT>, int>::type P;
  __shared__ f32x4 red[kUpWaves][kMaxNT][kWave];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wid = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int slot = blockIdx.y;
  const int32_t* pick;
  int e, first, cnt;
  if constexpr (kV > 0) {
    route_and_plan<kWave * kUpWaves, kV>(P, logits, T, E, k, blockIdx.x == 0 && slot == 0,
                                         topk_idx, topk_w, plan);
    if (slot >= P.n) return;
    e = P.expert[slot];
    first = P.first[slot];
    cnt = P.first[slot + 1] - first;
    pick = P.pick + first;
  } else {
    if (slot >= *plan.n) return;
    e = plan.expert[slot];
    first = plan.first[slot];
    cnt = plan.first[slot + 1] - first;
    pick = plan.pick + first;
  }
  e = __builtin_amdgcn_readfirstlane(e);
  cnt = __builtin_amdgcn_readfirstlane(cnt);
  const int j0 = blockIdx.x * kUpCols;
  const int i = lane & 15, g = lane >> 4;
  const int row = (i & 3) < 2 ? j0 + 2 * (i >> 2) + (i & 3) : I + j0 + 2 * (i >> 2) + (i & 3) - 2;
  const uint8_t* wp = w + ((int64_t)e * 2 * I + row) * H * (kFp8 ? 1 : 2) + 32 * g;
  const int steps = H / Step<kFp8>::kCols;
  const float *sc0 = nullptr, *sc1 = nullptr;
  if constexpr (kFp8) {
    sc0 = wsc + ((int64_t)e * (2 * I / kQuantBlock) + j0 / kQuantBlock) * steps;
    sc1 = sc0 + (int64_t)(I / kQuantBlock) * steps;
  }
  // up to 64 picks a pass over the weights
  for (int c0 = 0; c0 < cnt; c0 += 64) {
    auto pass = [&](auto nt_) __attribute__((always_inline)) {
      constexpr int NT = decltype(nt_)::value;
      const uint16_t* xp[NT];
      f32x4 acc[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        // columns past the last pick repeat the first: never stored
        const int c = c0 + 16 * nt + i;
        xp[nt] = x + (int64_t)(pick[c < cnt ? c : 0] / k) * H + (Step<kFp8>::kCols / 4) * g;
        acc[nt] = f32x4{0, 0, 0, 0};
      }
      dot_steps<kFp8, NT, NT == 1 ? 4 : (NT == 2 ? 2 : 1)>(wp, xp, sc0, sc1, wid, steps, kUpWaves,
                                                          acc);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) red[wid][nt][lane] = acc[nt];
      __syncthreads();
      for (int nt = wid; nt < NT; nt += kUpWaves) {
        f32x4 v = red[0][nt][lane];
#pragma unroll
        for (int q = 1; q < kUpWaves; ++q) v += red[q][nt][lane];
        const int c = c0 + 16 * nt + i;
        if (c < cnt) {
          const uint32_t hv = bf16x2_rne(silu(v[0]) * v[2], silu(v[1]) * v[3]);
          *reinterpret_cast<uint32_t*>(h + (int64_t)pick[c] * I + j0 + 2 * g) = hv;
        }
      }
      __syncthreads();
    };
    const int left = cnt - c0;
    if (kMaxNT == 1 || left <= 16) {
      pass(std::integral_constant<int, 1>{});
    } else if constexpr (kMaxNT > 1) {
      if (left <= 32) pass(std::integral_constant<int, 2>{});
      else pass(std::integral_constant<int, 4>{});
    }
  }
}

// Routing and plan alone (one block), where routing in every gate/up block
// would cost more.
template <int V>
__global__ __launch_bounds__(1024) void layer_plan_kernel(const float* __restrict__ logits, int T,
                                                          int E, int k,
                                                          int32_t* __restrict__ topk_idx,
                                                          float* __restrict__ topk_w, Plan plan) {
  __shared__ PlanLds<kMaxPicks> P;
  route_and_plan<1024, V>(P, logits, T, E, k, true, topk_idx, topk_w, plan);
}

// Down and combine: a block computes kDownCols columns of y for all tokens. The
// K steps of all live experts in a row are cut into one range a wave; at the
// end of an expert's part of its range a wave adds gate weight x result to its
// own fp32 rows of y in LDS (an expert's picks are different tokens), and the
// waves' rows are added in a fixed order at the end.
template <bool kFp8>
__global__ __launch_bounds__(kWave * kDownWaves) void layer_down_kernel(
    const uint16_t* __restrict__ h, int T, int H, int k, int I, const uint8_t* __restrict__ w,
    const float* __restrict__ wsc, const float* __restrict__ topk_w, Plan plan,
    uint16_t* __restrict__ y) {
  extern __shared__ __attribute__((aligned(16))) float ya[];  // [kDownWaves][T][kDownCols]
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wid = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c0 = blockIdx.x * kDownCols;
  for (int q = tid; q < kDownWaves * T * kDownCols; q += kWave * kDownWaves) ya[q] = 0.f;
  __syncthreads();
  const int n = *plan.n;
  const int steps = I / Step<kFp8>::kCols;
  const int total = n * steps;
  int at = (int)((int64_t)total * wid / kDownWaves);
  const int end = (int)((int64_t)total * (wid + 1) / kDownWaves);
  const int i = lane & 15, g = lane >> 4;
  float* mine = ya + (size_t)wid * T * kDownCols;
  while (at < end) {
    const int slot = at / steps;
    const int s0 = at - slot * steps;
    const int s1 = end - at < steps - s0 ? s0 + (end - at) : steps;
    at += s1 - s0;
    const int e = __builtin_amdgcn_readfirstlane(plan.expert[slot]);
    const int first = __builtin_amdgcn_readfirstlane(plan.first[slot]);
    const int cnt = __builtin_amdgcn_readfirstlane(plan.first[slot + 1]) - first;
    const int32_t* pick = plan.pick + first;
    const uint8_t* wp = w + ((int64_t)e * H + c0 + i) * I * (kFp8 ? 1 : 2) + 32 * g;
    const float* sc = nullptr;
    if constexpr (kFp8)
      sc = wsc + ((int64_t)e * (H / kQuantBlock) + c0 / kQuantBlock) * steps;
    for (int b0 = 0; b0 < cnt; b0 += 64) {
      auto pass = [&](auto nt_) __attribute__((always_inline)) {
        constexpr int NT = decltype(nt_)::value;
        const uint16_t* hp[NT];
        f32x4 acc[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int c = b0 + 16 * nt + i;
          hp[nt] = h + (int64_t)pick[c < cnt ? c : 0] * I + (Step<kFp8>::kCols / 4) * g;
          acc[nt] = f32x4{0, 0, 0, 0};
        }
        dot_steps<kFp8, NT, NT == 1 ? 4 : (NT == 2 ? 2 : 1)>(wp, hp, sc, sc, s0, s1, 1, acc);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int c = b0 + 16 * nt + i;
          if (c < cnt) {
            const int p = pick[c];
            const float gw = topk_w[p];
            f32x4* dst = reinterpret_cast<f32x4*>(mine + (p / k) * kDownCols + 4 * g);
            f32x4 v = *dst;
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = __builtin_fmaf(gw, acc[nt][r], v[r]);
            *dst = v;
          }
        }
      };
      const int left = cnt - b0;
      if (left <= 16) pass(std::integral_constant<int, 1>{});
      else if (left <= 32) pass(std::integral_constant<int, 2>{});
      else pass(std::integral_constant<int, 4>{});
    }
  }
  __syncthreads();
  for (int q = tid; q < T * kDownCols / 2; q += kWave * kDownWaves) {
    const int t = q / (kDownCols / 2), c = (q - t * (kDownCols / 2)) * 2;
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int v = 0; v < kDownWaves; ++v) {
      const float2 u = *reinterpret_cast<const float2*>(ya + ((size_t)v * T + t) * kDownCols + c);
      a += u.x;
      b += u.y;
    }
    *reinterpret_cast<uint32_t*>(y + (int64_t)t * H + c0 + c) = bf16x2_rne(a, b);
  }
}

}  // namespace

int64_t layer_plan_ints(int T, int E, int k) {
  const int np = T * k, slots = np < E ? np : E;
  return 4 + 2 * (int64_t)slots + 1 + np;
}

hipError_t launch_layer(const float* logits, const void* x, int T, int H, int E, int k, int I,
                        bool fp8, const void* w_gate_up, const float* s_gate_up,
                        const void* w_down, const float* s_down, int32_t* topk_idx, float* topk_w,
                        void* h, int32_t* plan_ws, void* y, hipStream_t s) {
  if (T == 0) return hipSuccess;
  const int np = T * k, slots = np < E ? np : E;
  const Plan plan = plan_at(plan_ws, slots);
  const dim3 grid((unsigned)(I / kUpCols), (unsigned)slots), block(kWave * kUpWaves);
  auto up = [&](auto kernel) {
    return launch(kernel, grid, block, 0, s, logits, static_cast<const uint16_t*>(x), T, H, E, k, I,
                  static_cast<const uint8_t*>(w_gate_up), s_gate_up, topk_idx, topk_w, plan,
                  static_cast<uint16_t*>(h));
  };
  hipError_t err;
  if (T <= kRouteT) {
    err = E <= 256 ? (fp8 ? up(layer_gate_up_kernel<4, true>) : up(layer_gate_up_kernel<4, false>))
                   : (fp8 ? up(layer_gate_up_kernel<16, true>) : up(layer_gate_up_kernel<16, false>));
  } else {
    auto go = [&](auto kernel) {
      return launch(kernel, dim3(1), dim3(1024), 0, s, logits, T, E, k, topk_idx, topk_w, plan);
    };
    err = E <= 256 ? go(layer_plan_kernel<4>) : go(layer_plan_kernel<16>);
    if (err != hipSuccess) return err;
    err = fp8 ? up(layer_gate_up_kernel<0, true>) : up(layer_gate_up_kernel<0, false>);
  }
  if (err != hipSuccess) return err;
  const dim3 dgrid((unsigned)(H / kDownCols)), dblock(kWave * kDownWaves);
  const uint32_t lds = (uint32_t)(kDownWaves * T * kDownCols * 4);
  auto down = [&](auto kernel) {
    return launch(kernel, dgrid, dblock, lds, s, static_cast<const uint16_t*>(h), T, H, k, I,
                  static_cast<const uint8_t*>(w_down), s_down, topk_w, plan,
                  static_cast<uint16_t*>(y));
  };
  return fp8 ? down(layer_down_kernel<true>) : down(layer_down_kernel<false>);
}

}  // namespace moe
