// Shared by the kernels of libmoe_block.so: argument checks and bf16 values.
#pragma once

#include "moe_block.h"
#include "moe_common.h"

namespace moe_block {

// Most tokens of a call: row counters are 32-bit and step past the last row.
constexpr int kMaxRows = 1 << 30;

// Lanes of one launch: a dispatch counts them in 32 bits, so calls of more rows
// than that are launched in slices.
constexpr int64_t kMaxLanes = 1ll << 31;

// launch(first, rows) over T rows that take `lanes` lanes each; the slices are
// multiples of 64 rows.
template <typename F> moe_status in_slices(int64_t T, int64_t lanes, F launch) {
  const int64_t most = kMaxLanes / lanes / 64 * 64;
  for (int64_t t = 0; t < T; t += most) {
    launch(t, static_cast<int>(T - t < most ? T - t : most));
    MOE_LAUNCH_CHECK();
  }
  return MOE_OK;
}

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
