// ffn_device.h -- pieces shared by the expert GEMM kernels: the bf16 rounding and
// SiLU of their epilogues, raw buffer descriptors with loads straight into LDS.
#pragma once

#include "device.h"

namespace moe {

constexpr int kXCD = 8;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Two floats to a pair of bf16 (low half = a), round to nearest even: on
// gfx950 one v_cvt_pk_bf16_f32, which rounds every non-NaN float exactly as
// the bit-twiddling f32_to_bf16_rne does (checked on the device over 16M bit
// patterns: denormals, ties of both parities, overflow to infinity); a NaN
// keeps its payload instead of becoming the canonical one.
__device__ __forceinline__ uint32_t bf16x2_rne(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// SiLU(g) = g / (1 + e^-g), evaluated as num / (1 + e^-|g|) with num = g for
// g >= 0 and g e^-|g| below, so the denominator stays in (1, 2]: e^-|g| is
// the hardware base-2 exponential of -|g| log2(e), the product split into a
// rounded part and its error (log2(e) as a float plus its remainder, the
// error carried to first order after the exponential), and the reciprocal is
// the hardware one refined by one Newton step. |g| is cut to 128 for it (e^-128 is
// zero in fp32 already): the product with log2(e) would overflow from 2.36e38 on, and
// its error then be NaN. For finite g (minus infinity gives NaN) the relative
// error is at most 4.6 x 2^-24 against the exact SiLU over 16M arguments in
// [-100, 100] (3.1 x 2^-24 for expf and an IEEE division), in ~14 instructions
// instead of ~25: the gate/up epilogue is bound by its instruction count.
__device__ __forceinline__ float silu(float g) {
  constexpr float kL1 = 1.44269504f;            // log2(e) rounded to float
  constexpr float kL2 = 1.925963033500011e-08f;  // log2(e) - kL1
  constexpr float kLn2 = 0.693147181f;
  const float a = __builtin_amdgcn_fmed3f(-__builtin_fabsf(g), -128.0f, 0.0f);
  const float t = a * kL1;
  const float tl = __builtin_fmaf(a, kL1, -t) + a * kL2;  // a log2(e) - t
  const float e0 = __builtin_amdgcn_exp2f(t);
  const float e = __builtin_fmaf(e0, tl * kLn2, e0);      // e^-|g|
  const float d = 1.0f + e;
  float r = __builtin_amdgcn_rcpf(d);
  r = __builtin_fmaf(r, __builtin_fmaf(-d, r, 1.0f), r);
  return (g >= 0.0f ? g : g * e) * r;
}

typedef __attribute__((address_space(3))) void* lptr_t;

// Word 3 of a raw buffer descriptor on gfx9-family parts (32-bit data format,
// no swizzle, no index stride).
constexpr int kRsrcWord3 = 0x00020000;

// s_waitcnt immediate for vmcnt <= n with the other counters left free (gfx9
// encoding: vmcnt [3:0] and [15:14], expcnt [6:4], lgkmcnt [11:8]).
constexpr int wait_vmcnt(int n) { return (n & 0xF) | ((n >> 4) << 14) | 0x0F70; }
constexpr int kWaitVmcnt0 = wait_vmcnt(0);

// Buffer-instruction helpers (plain device functions, so that the kernel's
// lambdas stay valid in the host compilation pass).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, kRsrcWord3);
}
// 16 bytes a lane from base + voff + soff into LDS at lds + 16 * lane.
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, uint16_t* lds, uint32_t voff,
                                           int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lptr_t)lds, 16, voff, soff, 0, 0);
}

}  // namespace moe
