// Shared by the kernels of libmoe_block.so: argument checks and bf16 values.
#pragma once

#include "moe_block.h"
#include "moe_common.h"

namespace moe_block {

// Most tokens of a call: row counters are 32-bit and step past the last row.
constexpr int kMaxRows = 1 << 30;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool real_dtype(int d) { return d == MOE_F32 || d == MOE_BF16; }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return static_cast<uint32_t>(moe::f32_to_bf16(a)) | (static_cast<uint32_t>(moe::f32_to_bf16(b)) << 16);
}
// the value as its storage type holds it
template <typename T> __device__ __forceinline__ float as_stored(float v);
template <> __device__ __forceinline__ float as_stored<float>(float v) { return v; }
template <> __device__ __forceinline__ float as_stored<uint16_t>(float v) {
  return moe::bf16_to_f32(moe::f32_to_bf16(v));
}

}  // namespace moe_block
