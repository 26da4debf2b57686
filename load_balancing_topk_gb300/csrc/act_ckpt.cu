// act_ckpt.cu -- 8-bit activation checkpoints (mep_ckpt_save, mep_ckpt_load)
// and the experts' gated activation that writes and reads them (mep_swiglu,
// mep_swiglu_backward).

#include "ckpt.cuh"

namespace mep {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v = max_nan(v, __shfl_xor_sync(MEP_FULL_MASK, v, d));
  return v;
}

// One warp per (row, block of 128 columns).
template <typename T>
__global__ void __launch_bounds__(32 * kWarps)
    k_ckpt_save(const T* __restrict__ x, long long N, int C, uint8_t* __restrict__ ckpt) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int nb = (C + kCkptBlock - 1) / kCkptBlock;
  const long long rb = ckpt_row_bytes(C), items = N * nb;
  for (long long i = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); i < items;
       i += (long long)gridDim.x * kWarps) {
    const long long r = i / nb;
    const int b = int(i % nb), c0 = b * kCkptBlock;
    float v[4], top = 0.f;
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + 32 * j + lane;
      v[j] = c < C ? to_f32(x[r * C + c]) : 0.f;
      top = max_nan(top, fabsf(v[j]));
    }
    const int s = ckpt_scale(warp_max_nan(top));
    const float inv = ckpt_inv_step(s);
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + 32 * j + lane;
      if (c < C) ckpt[r * rb + c] = uint8_t(ckpt_q(v[j], inv));
    }
    if (lane == 0) ckpt[r * rb + ckpt_scale_at(C) + b] = uint8_t(s);
    if (b == nb - 1)
      for (int p = ckpt_scale_at(C) + nb + lane; p < rb; p += 32) ckpt[r * rb + p] = 0;
    if (b == nb - 1 && C + lane < ckpt_scale_at(C)) ckpt[r * rb + C + lane] = 0;
  }
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps)
    k_ckpt_load(const uint8_t* __restrict__ ckpt, long long N, int C, T* __restrict__ x) {
  pdl_wait();
  pdl_launch_dependents();
  const long long rb = ckpt_row_bytes(C), n = N * C;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (long long)gridDim.x * blockDim.x) {
    const long long r = i / C;
    const int c = int(i % C);
    const uint8_t* row = ckpt + r * rb;
    x[i] = from_f32<T>(float(int8_t(row[c])) * ckpt_step(row[ckpt_scale_at(C) + c / kCkptBlock]));
  }
}

__device__ __forceinline__ float sigmoid(float g) { return 1.f / (1.f + __expf(-g)); }

template <bool CKPT>
__global__ void __launch_bounds__(32 * kWarps)
    k_swiglu(const __nv_bfloat16* __restrict__ gu, long long rows, int F,
             __nv_bfloat16* __restrict__ a, uint8_t* __restrict__ ckpt) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int nb = (F + kCkptBlock - 1) / kCkptBlock;
  const long long rb = ckpt_row_bytes(F), items = rows * nb;
  for (long long i = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); i < items;
       i += (long long)gridDim.x * kWarps) {
    const long long r = i / nb;
    const int b = int(i % nb), c0 = b * kCkptBlock;
    float v[2][4], top[2] = {0.f, 0.f};
    for (int h = 0; h < 2; ++h)
      for (int j = 0; j < 4; ++j) {
        const int c = c0 + 32 * j + lane;
        v[h][j] = c < F ? to_f32(gu[(2 * r + h) * F + c]) : 0.f;
        top[h] = max_nan(top[h], fabsf(v[h][j]));
      }
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + 32 * j + lane;
      if (c < F) a[r * F + c] = from_f32<__nv_bfloat16>(v[0][j] * sigmoid(v[0][j]) * v[1][j]);
    }
    if (CKPT)
      for (int h = 0; h < 2; ++h) {
        uint8_t* row = ckpt + (2 * r + h) * rb;
        const int s = ckpt_scale(warp_max_nan(top[h]));
        const float inv = ckpt_inv_step(s);
        for (int j = 0; j < 4; ++j) {
          const int c = c0 + 32 * j + lane;
          if (c < F) row[c] = uint8_t(ckpt_q(v[h][j], inv));
        }
        if (lane == 0) row[ckpt_scale_at(F) + b] = uint8_t(s);
        if (b == nb - 1) {
          for (int p = ckpt_scale_at(F) + nb + lane; p < rb; p += 32) row[p] = 0;
          if (F + lane < ckpt_scale_at(F)) row[F + lane] = 0;
        }
      }
  }
}

template <bool CKPT>
__global__ void __launch_bounds__(32 * kWarps)
    k_swiglu_backward(const __nv_bfloat16* __restrict__ da, const void* __restrict__ gu_,
                      long long rows, int F, __nv_bfloat16* __restrict__ dgu,
                      __nv_bfloat16* __restrict__ a) {
  pdl_wait();
  pdl_launch_dependents();
  const long long rb = ckpt_row_bytes(F), n = rows * F;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (long long)gridDim.x * blockDim.x) {
    const long long r = i / F;
    const int c = int(i % F);
    float v[2];
    for (int h = 0; h < 2; ++h) {
      if (CKPT) {
        const uint8_t* row = static_cast<const uint8_t*>(gu_) + (2 * r + h) * rb;
        v[h] = float(int8_t(row[c])) * ckpt_step(row[ckpt_scale_at(F) + c / kCkptBlock]);
      } else {
        v[h] = to_f32(static_cast<const __nv_bfloat16*>(gu_)[(2 * r + h) * F + c]);
      }
    }
    const float d = to_f32(da[i]), s = sigmoid(v[0]);
    dgu[2 * r * F + c] = from_f32<__nv_bfloat16>(d * v[1] * s * (1.f + v[0] * (1.f - s)));
    dgu[(2 * r + 1) * F + c] = from_f32<__nv_bfloat16>(d * v[0] * s);
    if (a != nullptr) a[i] = from_f32<__nv_bfloat16>(v[0] * s * v[1]);
  }
}

int grid_for(long long items, int per) {
  const long long want = (items + per - 1) / per, cap = (long long)sm_count() * 64;
  return int(want < cap ? want : cap);
}

}  // namespace
}  // namespace mep

using namespace mep;

extern "C" int mep_ckpt_row_bytes(int64_t C, size_t* bytes) {
  if (bytes == nullptr || C < 1 || C > MEP_MAX_CKPT_C) return MEP_ERR_INVALID_ARG;
  *bytes = size_t(ckpt_row_bytes(C));
  return MEP_OK;
}

static int ckpt_check(const void* x, int type, int64_t N, int64_t C, const void* ckpt) {
  if (N < 0 || N > 0x7fffffffLL || C < 1 || C > MEP_MAX_CKPT_C) return MEP_ERR_INVALID_ARG;
  if (type != MEP_BF16 && type != MEP_F32) return MEP_ERR_INVALID_ARG;
  if (N == 0) return MEP_OK;
  if (x == nullptr || ckpt == nullptr || !aligned16(x) || !aligned16(ckpt)) return MEP_ERR_INVALID_ARG;
  return MEP_OK;
}

extern "C" int mep_ckpt_save(const void* x, int x_type, int64_t N, int64_t C, uint8_t* ckpt,
                             void* stream) {
  const int rc = ckpt_check(x, x_type, N, C, ckpt);
  if (rc != MEP_OK || N == 0) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int grid = grid_for(N * ((C + kCkptBlock - 1) / kCkptBlock), kWarps);
  const cudaError_t err =
      x_type == MEP_BF16
          ? launch_pdl(k_ckpt_save<__nv_bfloat16>, dim3(grid), dim3(32 * kWarps), 0, st,
                       static_cast<const __nv_bfloat16*>(x), (long long)N, int(C), ckpt)
          : launch_pdl(k_ckpt_save<float>, dim3(grid), dim3(32 * kWarps), 0, st,
                       static_cast<const float*>(x), (long long)N, int(C), ckpt);
  return err == cudaSuccess ? MEP_OK : MEP_ERR_CUDA;
}

extern "C" int mep_ckpt_load(const uint8_t* ckpt, int64_t N, int64_t C, int x_type, void* x,
                             void* stream) {
  const int rc = ckpt_check(x, x_type, N, C, ckpt);
  if (rc != MEP_OK || N == 0) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int grid = grid_for(N * C, 32 * kWarps);
  const cudaError_t err =
      x_type == MEP_BF16 ? launch_pdl(k_ckpt_load<__nv_bfloat16>, dim3(grid), dim3(32 * kWarps), 0,
                                      st, ckpt, (long long)N, int(C), static_cast<__nv_bfloat16*>(x))
                         : launch_pdl(k_ckpt_load<float>, dim3(grid), dim3(32 * kWarps), 0, st, ckpt,
                                      (long long)N, int(C), static_cast<float*>(x));
  return err == cudaSuccess ? MEP_OK : MEP_ERR_CUDA;
}

extern "C" int mep_swiglu(const mep_bf16* gu, int64_t rows, int64_t F, mep_bf16* a, uint8_t* ckpt,
                          void* stream) {
  if (rows < 0 || rows > 0x3fffffffLL || F < 1 || F > MEP_MAX_CKPT_C) return MEP_ERR_INVALID_ARG;
  if (rows == 0) return MEP_OK;
  if (gu == nullptr || a == nullptr || !aligned16(gu) || !aligned16(a) || !aligned16(ckpt))
    return MEP_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int grid = grid_for(rows * ((F + kCkptBlock - 1) / kCkptBlock), kWarps);
  const __nv_bfloat16* in = reinterpret_cast<const __nv_bfloat16*>(gu);
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a);
  const cudaError_t err =
      ckpt != nullptr ? launch_pdl(k_swiglu<true>, dim3(grid), dim3(32 * kWarps), 0, st, in,
                                   (long long)rows, int(F), out, ckpt)
                      : launch_pdl(k_swiglu<false>, dim3(grid), dim3(32 * kWarps), 0, st, in,
                                   (long long)rows, int(F), out, ckpt);
  return err == cudaSuccess ? MEP_OK : MEP_ERR_CUDA;
}

extern "C" int mep_swiglu_backward(const mep_bf16* da, const void* gu, int gu_type, int64_t rows,
                                   int64_t F, mep_bf16* dgu, mep_bf16* a, void* stream) {
  if (rows < 0 || rows > 0x3fffffffLL || F < 1 || F > MEP_MAX_CKPT_C) return MEP_ERR_INVALID_ARG;
  if (gu_type != MEP_BF16 && gu_type != MEP_CKPT8) return MEP_ERR_INVALID_ARG;
  if (rows == 0) return MEP_OK;
  if (da == nullptr || gu == nullptr || dgu == nullptr || !aligned16(da) || !aligned16(gu) ||
      !aligned16(dgu) || !aligned16(a))
    return MEP_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int grid = grid_for(rows * F, 32 * kWarps);
  const __nv_bfloat16* in = reinterpret_cast<const __nv_bfloat16*>(da);
  __nv_bfloat16 *o = reinterpret_cast<__nv_bfloat16*>(dgu), *oa = reinterpret_cast<__nv_bfloat16*>(a);
  const cudaError_t err =
      gu_type == MEP_CKPT8 ? launch_pdl(k_swiglu_backward<true>, dim3(grid), dim3(32 * kWarps), 0, st,
                                        in, gu, (long long)rows, int(F), o, oa)
                           : launch_pdl(k_swiglu_backward<false>, dim3(grid), dim3(32 * kWarps), 0,
                                        st, in, gu, (long long)rows, int(F), o, oa);
  return err == cudaSuccess ? MEP_OK : MEP_ERR_CUDA;
}
