// quant_int8.h -- rows as 8-bit integers with one fp32 scale a row:
// scale = amax / 127 (amax: largest finite magnitude of the row; rounded once to fp32,
// at least 2^-126, 1 for a row without a finite nonzero element), q = x / scale to the
// nearest integer, ties to even. Infinities saturate to +-127 and do not enter amax; a
// row with a NaN has scale NaN and q 0, so that what is computed from it is NaN.
#pragma once

#include "device.h"
#include "quant.h"

namespace moe {

__device__ __forceinline__ float int8_scale(double amax) {
  if (amax == 0.0) return 1.0f;
  const double s = amax / 127.0;
  return s < 0x1p-126 ? 0x1p-126f : (s > 3.4028234663852886e38 ? 3.4028234663852886e38f : (float)s);
}

// v / scale to the nearest integer, |v| <= 127 scale; inv = 1 / scale, rounded to 64 bits. The
// sum leaves an integer, rounded to nearest even, in the low word.
//
// Any v: off by inv's rounding, 2^-46 of a step at most.
__device__ __forceinline__ int int8_round(double v, double inv) {
  return (int)(uint32_t)__double_as_longlong(__builtin_fma(v, inv, 0x1.8p52));
}
// Fp32 v and scale: the result of the exact quotient. One that is not half way between two
// integers is at least 2^-25 from there; the first sum leaves multiples of 2^-32, so one
// that is comes out so although inv is rounded.
__device__ __forceinline__ int int8_round_exact(float v, double inv) {
  constexpr double kFine = 0x1.8p20, kWhole = 0x1.8p52;
  const double fine = __builtin_fma((double)v, inv, kFine);
  return (int)(uint32_t)__double_as_longlong(fine + (kWhole - kFine));
}

// How an fp32 row is rounded. all, top: the largest magnitude (as bits) of its values and of
// its finite ones.
struct Int8Row {
  float scale;  // NaN: of a row with one
  float most;   // of a value's magnitude
  double inv;
  __device__ __forceinline__ int round(float v) const {
    return int8_round_exact(__builtin_amdgcn_fmed3f(v, -most, most), inv);
  }
};
__device__ __forceinline__ Int8Row int8_row(uint32_t all, uint32_t top) {
  const bool nan = all > kInfBits;
  const float s = int8_scale((double)__uint_as_float(top));
  return {nan ? __builtin_nanf("") : s, fminf(127.0f * s, 3.4028234663852886e38f),
          nan ? 0.0 : 1.0 / (double)s};
}

// Four integers in [-127, 127] as bytes.
__device__ __forceinline__ uint32_t pack_int8(int a, int b, int c, int d) {
  const uint32_t lo = __builtin_amdgcn_perm((uint32_t)b, (uint32_t)a, 0x0C0C0400u);
  const uint32_t hi = __builtin_amdgcn_perm((uint32_t)d, (uint32_t)c, 0x04000C0Cu);
  return lo | hi;
}

// Exponent p of the e4m3 block scale (quant.h) from an amax held in 64 bits; p <= 127.
__device__ __forceinline__ int scale_exponent(double amax) {
  if (amax == 0.0) return 0;
  const uint64_t u = (uint64_t)__double_as_longlong(amax);
  const int p = (int)(u >> 52) - 1023 - 8 + ((u & 0xFFFFFFFFFFFFFull) > 0xC000000000000ull ? 1 : 0);
  return p < -126 ? -126 : (p > 127 ? 127 : p);
}

}  // namespace moe
