// ckpt.cuh -- the 8-bit checkpoint row shared by layer_norm.cu, act_ckpt.cu
// and grouped_wgrad.cu, and the element types of the training operators.
//
// A row of C columns: C signed bytes q, from byte align16(C) on one scale
// byte s per block of 128 columns, padding to a multiple of 32 bytes. A value
// is q * 2^(s - 127). Per block, with a = max |x|: k = max(floor(log2 a) - 6,
// -126), s = k + 127, q = rint(x * 2^-k) (ties to even) kept within +-127.
// a * 2^-k lies in [64, 128), so a bf16 x (8 significant bits: at most 127.5)
// is off by at most half a step, 2^(k-1). Every factor is a power of two:
// the rounding to q is the only one, and q * 2^k is exact in bf16, which is
// what lets a tensor-core product run on exactly the kept values. Fixed
// point rather than an 8-bit float: the step is a / 64 at most over the whole
// block, where a 3-bit mantissa is off by up to 1/16 of every large value.
// A block that holds an infinity or a NaN gets s = 255: its values come back
// as NaN, so that an overflow stays visible in the gradients.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "mep_common.cuh"
#include "vec.cuh"

namespace mep {
namespace {

constexpr int kCkptBlock = 128;   // columns that share one scale byte
constexpr int kCkptNan = 255;     // scale byte of a block with a non-finite value

__host__ __device__ __forceinline__ int ckpt_scale_at(int C) { return (C + 15) & ~15; }
__host__ __device__ __forceinline__ long long ckpt_row_bytes(long long C) {
  return (((C + 15) & ~15LL) + (C + kCkptBlock - 1) / kCkptBlock + 31) & ~31LL;
}

// Scale byte of a block whose largest magnitude is `amax` (a NaN or an
// infinity anywhere in the block must arrive here as one).
__device__ __forceinline__ int ckpt_scale(float amax) {
  const int e = int(__float_as_uint(amax) >> 23);  // biased exponent; 0 also for zero and subnormals
  return e == 255 ? kCkptNan : max(e - 6, 1);
}
// 2^-k and 2^k of a scale byte s = k + 127, 1 <= s <= 248; 0 and NaN for 255.
__device__ __forceinline__ float ckpt_inv_step(int s) {
  return s == kCkptNan ? 0.f : __uint_as_float(uint32_t(254 - s) << 23);
}
__device__ __forceinline__ float ckpt_step(int s) {
  return __uint_as_float(s == kCkptNan ? 0x7fc00000u : uint32_t(s) << 23);
}
// One value as a byte. In a block with s = 255 every finite value becomes 0
// (times 0) and the non-finite ones convert to some byte that is never read
// as a value.
__device__ __forceinline__ int ckpt_q(float x, float inv_step) {
  return max(-127, min(127, __float2int_rn(x * inv_step)));
}
// max that keeps a NaN (fmaxf drops it)
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

}  // namespace
}  // namespace mep
