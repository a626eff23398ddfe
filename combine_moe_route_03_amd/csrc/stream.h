// stream.h -- streaming weights that are read once through registers, shared by
// the few-token layer and the 8-bit products of few rows an expert.
//
// A unit is 16 (or 8) weight rows; a K step is 128 bytes
// of each. Every load instruction takes whole
// 128-byte lines, lane l chunk l % 8 of row l / 8 (16 bytes a lane): lanes in
// the order of an MFMA operand, 16 rows by 64 bytes, reached 5.6-6.2 TB/s on the
// same stream, this order 6.9-7.0. The loads of D steps are in flight in
// a register ring; a step's registers then go through the wave's own piece of
// LDS into operand order (no barrier: a wave's LDS operations are in order).
// Units start at different steps, since weight rows a power of two apart would
// otherwise have all waves on the same memory channels at one time (5.9 against
// 6.2-7.0 TB/s).
#pragma once

#include "device.h"
#include "ffn_device.h"

namespace moe {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// Byte offset of what is not there: every descriptor is shorter than 2^31 bytes,
// so a load from there, at any step, is out of range and reads zeros without a
// memory access.
constexpr uint32_t kOutside = 0x80000000u;
constexpr int kStream = 2;  // cache policy: weights are read once

// A buffer whose loads can be switched off: past the last step of a stream its
// descriptor is empty, so the loop needs neither branches nor address selects. The
// scalar offset (step) has to be 0 then: the range check takes it from the
// descriptor's size, and with more the difference could wrap and let every lane in.
struct Buffer {
  const void* base;
  uint32_t bytes;
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t at(bool on) const {
    return make_rsrc(base, on ? bytes : 0);
  }
};

// 16 bytes at off + step (step uniform).
__device__ __forceinline__ v4u load16(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t step) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, off, step, 0);
}
__device__ __forceinline__ v4u load16_stream(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t step) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, off, step, kStream);
}

// Byte offset of 16-byte chunk c of LDS tile row r (rows of 128 bytes): the 16
// lanes that read one chunk column at a time hit distinct banks.
__device__ __forceinline__ int tile_at(int r, int c) { return r * 128 + ((c ^ ((r >> 1) & 7)) << 4); }

}  // namespace moe
