// quant.h -- 8-bit block quantisation: e4m3 values (4 exponent bits, 3 mantissa
// bits, largest finite value 448, no infinity) with one fp32 scale for each
// block of 128 columns (of one row, or of 128 rows).
//
// The scale of a block is a power of two, 2^p with p the smallest integer
// >= -126 for which amax <= 448 * 2^p (amax: largest finite magnitude of the
// block; scale 1 for a block without a finite nonzero element). x * 2^-p is then
// exact (or so far below the smallest e4m3 step that it rounds to zero either
// way), so the one rounding of a value is the one to e4m3 (nearest, ties to
// even), and the result does not depend on how a division rounds. Against
// amax / 448 it costs at most one binade at the subnormal end: the relative
// precision of a floating type does not change with a power-of-two scale.
// Infinities saturate to +-448, NaN stays NaN; neither enters amax.
#pragma once

#include <type_traits>

#include "device.h"

namespace moe {

constexpr int kQuantBlock = 128;    // columns a scale covers
constexpr float kE4M3Max = 448.0f;  // 1.75 * 2^8
constexpr uint32_t kInfBits = 0x7F800000u;

// Exponent p of the block scale from the bit pattern of amax (finite, >= 0).
__device__ __forceinline__ int scale_exponent(uint32_t amax_bits) {
  // amax = (1 + m / 2^23) 2^(e - 127) <= 1.75 * 2^8 * 2^p  <=>  p >= e - 135 + (m > 0.75 2^23)
  const int p = (int)(amax_bits >> 23) - 135 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return amax_bits == 0 ? 0 : (p < -126 ? -126 : p);
}

// 2^p for p in [-126, 127].
__device__ __forceinline__ float power_of_two(int p) { return __uint_as_float((uint32_t)(127 + p) << 23); }

// Magnitude bits of v for the block maximum: 0 for an infinity or a NaN.
__device__ __forceinline__ uint32_t finite_bits(float v) {
  const uint32_t u = __float_as_uint(v) & 0x7FFFFFFFu;
  return u < kInfBits ? u : 0u;
}

__device__ __forceinline__ float e4m3_clamp(float v) {
  return v > kE4M3Max ? kE4M3Max : (v < -kE4M3Max ? -kE4M3Max : v);  // NaN passes
}

// Four floats (already scaled, |v| <= 448 or NaN) to four e4m3 bytes, nearest
// even: two v_cvt_pk_fp8_f32.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return (uint32_t)w;
}

// One 16-byte load of a row: 8 bf16 or 4 fp32 elements. (Consecutive lanes take
// consecutive 16 bytes; with 32 bytes a lane in two loads every instruction
// touched half of each line: 128 x 128 blocks of 16 x 2816 x 4096 bf16 105 us
// instead of 92.)
template <bool kBF16>
struct QuantVec {
  static constexpr int N = kBF16 ? 8 : 4;                 // elements
  static constexpr int kLanes = kQuantBlock / N;          // lanes of a scale's 128 columns
  typedef typename std::conditional<kBF16, uint2, uint32_t>::type Out;  // N e4m3 bytes
  v4u v;
  __device__ __forceinline__ float get(int i) const {
    if constexpr (kBF16) return (i & 1) ? bf16_hi(v[i >> 1]) : bf16_lo(v[i >> 1]);
    else return __uint_as_float(v[i]);
  }
  // Largest finite magnitude, as bits.
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t u = finite_bits(get(i));
      m = u > m ? u : m;
    }
    return m;
  }
  // The values times inv as e4m3.
  __device__ __forceinline__ Out quantize(float inv) const {
    uint32_t w[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      w[i] = e4m3x4(e4m3_clamp(get(4 * i) * inv), e4m3_clamp(get(4 * i + 1) * inv),
                    e4m3_clamp(get(4 * i + 2) * inv), e4m3_clamp(get(4 * i + 3) * inv));
    if constexpr (kBF16) return make_uint2(w[0], w[1]);
    else return w[0];
  }
};

// Maximum over aligned groups of G lanes (all lanes of the wave active).
template <int G>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  return group_reduce(v, G, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

}  // namespace moe
