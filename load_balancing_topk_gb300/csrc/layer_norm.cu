// layer_norm.cu -- layer norm over the hidden width (mep_layer_norm) and its
// backward pass (mep_layer_norm_backward), with 8-bit checkpoint rows as a
// by-product of the first and as input of the second.

#include "ckpt.cuh"

namespace mep {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxH = MEP_MAX_NORM_H;
constexpr int kParts = 304;

__device__ __forceinline__ float block_sum(float v, float* s) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(MEP_FULL_MASK, v, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int w = 0; w < kThreads / 32; ++w) v += s[w];
  return v;
}

__device__ __forceinline__ float param(const void* p, int type, int h, float none) {
  if (p == nullptr) return none;
  return type == MEP_F32 ? static_cast<const float*>(p)[h]
                         : to_f32(static_cast<const __nv_bfloat16*>(p)[h]);
}

// One warp per block of 128 columns of a row held in shared memory.
__device__ void save_row(const float* v, int H, uint8_t* row) {
  const int lane = threadIdx.x & 31, nb = (H + kCkptBlock - 1) / kCkptBlock;
  for (int b = threadIdx.x >> 5; b < nb; b += kThreads / 32) {
    float top = 0.f;
    for (int j = 0; j < 4; ++j) {
      const int c = b * kCkptBlock + 32 * j + lane;
      if (c < H) top = max_nan(top, fabsf(v[c]));
    }
    for (int d = 16; d >= 1; d >>= 1) top = max_nan(top, __shfl_xor_sync(MEP_FULL_MASK, top, d));
    const int s = ckpt_scale(top);
    const float inv = ckpt_inv_step(s);
    for (int j = 0; j < 4; ++j) {
      const int c = b * kCkptBlock + 32 * j + lane;
      if (c < H) row[c] = uint8_t(ckpt_q(v[c], inv));
    }
    if (lane == 0) row[ckpt_scale_at(H) + b] = uint8_t(s);
  }
  for (int p = H + threadIdx.x; p < ckpt_scale_at(H); p += kThreads) row[p] = 0;
  for (int p = ckpt_scale_at(H) + nb + threadIdx.x; p < ckpt_row_bytes(H); p += kThreads) row[p] = 0;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_norm(const T* __restrict__ x, const void* w, const void* b, int p_type, float eps, long long N,
           int H, T* __restrict__ y, float* mean, float* rstd, uint8_t* x_ckpt, uint8_t* y_ckpt) {
  pdl_wait();
  pdl_launch_dependents();
  extern __shared__ float row[];
  __shared__ float s[32];
  for (long long r = blockIdx.x; r < N; r += gridDim.x) {
    float sum = 0.f, sq = 0.f;
    for (int h = threadIdx.x; h < H; h += kThreads) sum += row[h] = to_f32(x[r * H + h]);
    const float m = block_sum(sum, s) / H;
    for (int h = threadIdx.x; h < H; h += kThreads) sq += (row[h] - m) * (row[h] - m);
    const float rs = 1.f / sqrtf(block_sum(sq, s) / H + eps);
    if (threadIdx.x == 0) {
      mean[r] = m;
      rstd[r] = rs;
    }
    if (x_ckpt != nullptr) save_row(row, H, x_ckpt + r * ckpt_row_bytes(H));
    __syncthreads();
    for (int h = threadIdx.x; h < H; h += kThreads) {
      const T o = from_f32<T>((row[h] - m) * rs * param(w, p_type, h, 1.f) + param(b, p_type, h, 0.f));
      y[r * H + h] = o;
      row[h] = to_f32(o);
    }
    __syncthreads();
    if (y_ckpt != nullptr) save_row(row, H, y_ckpt + r * ckpt_row_bytes(H));
    __syncthreads();
  }
}

template <typename T, bool CKPT>
__device__ __forceinline__ float load_x(const void* x, long long r, int h, int H) {
  if (!CKPT) return to_f32(static_cast<const T*>(x)[r * H + h]);
  const uint8_t* row = static_cast<const uint8_t*>(x) + r * ckpt_row_bytes(H);
  return float(int8_t(row[h])) * ckpt_step(row[ckpt_scale_at(H) + h / kCkptBlock]);
}

template <typename T, bool CKPT>
__global__ void __launch_bounds__(kThreads)
    k_norm_dx(const T* __restrict__ dy, const void* x, const void* w, int p_type,
              const float* __restrict__ mean, const float* __restrict__ rstd, long long N, int H,
              T* __restrict__ dx) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float s[32];
  for (long long r = blockIdx.x; r < N; r += gridDim.x) {
    const float m = mean[r], rs = rstd[r];
    float s1 = 0.f, s2 = 0.f;
    for (int h = threadIdx.x; h < H; h += kThreads) {
      const float t = to_f32(dy[r * H + h]) * param(w, p_type, h, 1.f);
      s1 += t;
      s2 += t * (load_x<T, CKPT>(x, r, h, H) - m) * rs;
    }
    s1 = block_sum(s1, s) / H;
    s2 = block_sum(s2, s) / H;
    for (int h = threadIdx.x; h < H; h += kThreads) {
      const float t = to_f32(dy[r * H + h]) * param(w, p_type, h, 1.f);
      const float xhat = (load_x<T, CKPT>(x, r, h, H) - m) * rs;
      dx[r * H + h] = from_f32<T>(rs * (t - s1 - xhat * s2));
    }
  }
}

// Column sums: part p adds its rows p, p + parts, ... in order.
template <typename T, bool CKPT>
__global__ void __launch_bounds__(kThreads)
    k_norm_dw_parts(const T* __restrict__ dy, const void* x, const float* __restrict__ mean,
                    const float* __restrict__ rstd, long long N, int H, int parts,
                    float* __restrict__ ws) {
  pdl_wait();
  pdl_launch_dependents();
  const int h = blockIdx.x * kThreads + threadIdx.x, p = blockIdx.y;
  if (h >= H) return;
  float dw = 0.f, db = 0.f;
  for (long long r = p; r < N; r += parts) {
    const float d = to_f32(dy[r * H + h]);
    dw += d * ((load_x<T, CKPT>(x, r, h, H) - mean[r]) * rstd[r]);
    db += d;
  }
  ws[(long long)(2 * p) * H + h] = dw;
  ws[(long long)(2 * p + 1) * H + h] = db;
}

__global__ void __launch_bounds__(kThreads)
    k_norm_dw_sum(const float* __restrict__ ws, int H, int parts, int accumulate, float* dweight,
                  float* dbias) {
  pdl_wait();
  pdl_launch_dependents();
  const int h = blockIdx.x * kThreads + threadIdx.x;
  if (h >= H) return;
  for (int k = 0; k < 2; ++k) {
    float* out = k == 0 ? dweight : dbias;
    if (out == nullptr) continue;
    float v = 0.f;
    for (int p = 0; p < parts; ++p) v += ws[(long long)(2 * p + k) * H + h];
    out[h] = accumulate ? out[h] + v : v;
  }
}

int norm_parts(long long N) { return int(N < 1 ? 1 : N < kParts ? N : kParts); }

int norm_check(int type, int64_t N, int64_t H, int p_type) {
  if (type != MEP_BF16 && type != MEP_F32) return MEP_ERR_INVALID_ARG;
  if (p_type != MEP_BF16 && p_type != MEP_F32) return MEP_ERR_INVALID_ARG;
  if (N < 0 || N > 0x7fffffffLL || H < 1 || H > kMaxH) return MEP_ERR_INVALID_ARG;
  return MEP_OK;
}

int grid_rows(long long N) {
  const long long cap = (long long)sm_count() * 32;
  return int(N < cap ? N : cap);
}

template <typename T>
cudaError_t run_norm(const void* x, const void* w, const void* b, int p_type, float eps, long long N,
                     int H, void* y, float* mean, float* rstd, uint8_t* xc, uint8_t* yc,
                     cudaStream_t st) {
  const int smem = H * 4;
  if (set_max_dynamic_smem(reinterpret_cast<const void*>(k_norm<T>), smem)) return cudaErrorInvalidValue;
  return launch_pdl(k_norm<T>, dim3(grid_rows(N)), dim3(kThreads), smem, st, static_cast<const T*>(x),
                    w, b, p_type, eps, N, H, static_cast<T*>(y), mean, rstd, xc, yc);
}

template <typename T, bool CKPT>
cudaError_t run_norm_backward(const void* dy, const void* x, const void* w, int p_type,
                              const float* mean, const float* rstd, long long N, int H, float* ws,
                              void* dx, float* dweight, float* dbias, int accumulate,
                              cudaStream_t st) {
  const int parts = norm_parts(N);
  cudaError_t err = cudaSuccess;
  if (N > 0) {
    err = launch_pdl(k_norm_dx<T, CKPT>, dim3(grid_rows(N)), dim3(kThreads), 0, st,
                     static_cast<const T*>(dy), x, w, p_type, mean, rstd, N, H, static_cast<T*>(dx));
    if (err != cudaSuccess) return err;
  }
  if (dweight == nullptr && dbias == nullptr) return err;
  const int cols = (H + kThreads - 1) / kThreads;
  err = launch_pdl(k_norm_dw_parts<T, CKPT>, dim3(cols, parts), dim3(kThreads), 0, st,
                   static_cast<const T*>(dy), x, mean, rstd, N, H, parts, ws);
  if (err != cudaSuccess) return err;
  return launch_pdl(k_norm_dw_sum, dim3(cols), dim3(kThreads), 0, st, ws, H, parts, accumulate,
                    dweight, dbias);
}

}  // namespace
}  // namespace mep

using namespace mep;

extern "C" int mep_layer_norm(const void* x, int x_type, const void* weight, const void* bias,
                              int p_type, float eps, int64_t N, int64_t H, void* y, float* mean,
                              float* rstd, uint8_t* x_ckpt, uint8_t* y_ckpt, void* stream) {
  if (norm_check(x_type, N, H, p_type) != MEP_OK || !(eps >= 0.f)) return MEP_ERR_INVALID_ARG;
  if (N == 0) return MEP_OK;
  if (x == nullptr || y == nullptr || mean == nullptr || rstd == nullptr) return MEP_ERR_INVALID_ARG;
  for (const void* p : {x, weight, bias, static_cast<const void*>(y), static_cast<const void*>(mean),
                        static_cast<const void*>(rstd), static_cast<const void*>(x_ckpt),
                        static_cast<const void*>(y_ckpt)})
    if (!aligned16(p)) return MEP_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t err =
      x_type == MEP_BF16
          ? run_norm<__nv_bfloat16>(x, weight, bias, p_type, eps, N, int(H), y, mean, rstd, x_ckpt, y_ckpt, st)
          : run_norm<float>(x, weight, bias, p_type, eps, N, int(H), y, mean, rstd, x_ckpt, y_ckpt, st);
  return err == cudaSuccess ? MEP_OK : MEP_ERR_CUDA;
}

extern "C" int mep_layer_norm_backward_workspace_bytes(int64_t N, int64_t H, size_t* bytes) {
  if (bytes == nullptr || norm_check(MEP_F32, N, H, MEP_F32) != MEP_OK) return MEP_ERR_INVALID_ARG;
  *bytes = size_t(norm_parts(N)) * 2 * H * sizeof(float);
  return MEP_OK;
}

extern "C" int mep_layer_norm_backward(const void* dy, int dy_type, const void* x, int x_type,
                                       const void* weight, int p_type, const float* mean,
                                       const float* rstd, int64_t N, int64_t H, void* ws,
                                       size_t ws_bytes, void* dx, float* dweight, float* dbias,
                                       int accumulate, void* stream) {
  size_t need = 0;
  if (norm_check(dy_type, N, H, p_type) != MEP_OK || (x_type != dy_type && x_type != MEP_CKPT8))
    return MEP_ERR_INVALID_ARG;
  mep_layer_norm_backward_workspace_bytes(N, H, &need);
  if (N > 0 && (dy == nullptr || x == nullptr || mean == nullptr || rstd == nullptr || dx == nullptr))
    return MEP_ERR_INVALID_ARG;
  if ((dweight != nullptr || dbias != nullptr) && (ws == nullptr || ws_bytes < need))
    return MEP_ERR_INVALID_ARG;
  for (const void* p : {dy, x, weight, static_cast<const void*>(mean), static_cast<const void*>(rstd),
                        static_cast<const void*>(ws), static_cast<const void*>(dx),
                        static_cast<const void*>(dweight), static_cast<const void*>(dbias)})
    if (!aligned16(p)) return MEP_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  float* w = static_cast<float*>(ws);
  cudaError_t err;
  if (dy_type == MEP_BF16)
    err = x_type == MEP_CKPT8
              ? run_norm_backward<__nv_bfloat16, true>(dy, x, weight, p_type, mean, rstd, N, int(H), w, dx, dweight, dbias, accumulate, st)
              : run_norm_backward<__nv_bfloat16, false>(dy, x, weight, p_type, mean, rstd, N, int(H), w, dx, dweight, dbias, accumulate, st);
  else
    err = x_type == MEP_CKPT8
              ? run_norm_backward<float, true>(dy, x, weight, p_type, mean, rstd, N, int(H), w, dx, dweight, dbias, accumulate, st)
              : run_norm_backward<float, false>(dy, x, weight, p_type, mean, rstd, N, int(H), w, dx, dweight, dbias, accumulate, st);
  return err == cudaSuccess ? MEP_OK : MEP_ERR_CUDA;
}
