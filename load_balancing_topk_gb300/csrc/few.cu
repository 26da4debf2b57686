// few.cu -- the whole layer for a few tokens (mep_expert_layer) and the product
// of a few rows with a matrix in 4 bits (mep_w4_product).
//
// A block of 256 threads takes 32 columns, eight threads a column; every thread
// adds up its share of the sum in fp32, and the shares are joined in order.

#include "ckpt.cuh"
#include "w4.cuh"

namespace mep {
namespace {

constexpr int kThreads = 256, kColumns = 32, kShares = kThreads / kColumns;

// Weight (k, n) of a matrix, as it lies or in 4 bits.
struct Plain {
  const __nv_bfloat16* w;
  long long ld;
  __device__ __forceinline__ float get(long long k, long long n) const { return __bfloat162float(w[k * ld + n]); }
};
struct Quarter {
  const uint8_t* w;
  long long panel;
  int group;
  __device__ __forceinline__ float get(long long k, long long n) const {
    const uint8_t* b = w + n / kW4Cols * panel + k / kW4Rows * w4_block_bytes(group);
    const int r = int(k % kW4Rows), m = int(n % kW4Cols);
    const int h = r / 64, j = r / 16 % 4, i = r / 8 % 2, t = r / 2 % 4, e = r % 2, c = m / 16, l = m / 8 % 2, g = m % 8;
    const int q = (b[((((4 * h + c) * 8 + g) * 4 + t) * 4 + j) * 4 + 2 * e + i] >> (4 * l) & 15) - 8;
    return q * __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(b + kW4Pairs)[r / group * 64 + 16 * c + 2 * g + l]);
  }
};
__device__ __forceinline__ Plain matrix(const __nv_bfloat16* w, long long m, long long K, long long N, int) {
  return {w + m * K * N, N};
}
__device__ __forceinline__ Quarter matrix(const uint8_t* w, long long m, long long K, long long N, int group) {
  return {w + m * w4_matrix_bytes(K, N, group), w4_panel_bytes(K, group), group};
}

// Sum over k of x[k] * W[k, n] for this block's columns; the same in all of a column's threads.
template <typename M>
__device__ __forceinline__ float column_sum(const __nv_bfloat16* x, const M& w, long long K, long long n, bool in,
                                            float* s_part) {
  const int share = threadIdx.x / kColumns, c = threadIdx.x % kColumns;
  float sum = 0.f;
  if (in)
    for (long long k = share; k < K; k += kShares) sum = fmaf(__bfloat162float(x[k]), w.get(k, n), sum);
  __syncthreads();
  s_part[threadIdx.x] = sum;
  __syncthreads();
  sum = 0.f;
  for (int i = 0; i < kShares; ++i) sum += s_part[i * kColumns + c];
  return sum;
}

__global__ void __launch_bounds__(kThreads) k_few_check(const int32_t* idx, int T, int K, int E, int32_t* status,
                                                        int* go) {
  __shared__ int s_bad;
  pdl_launch_dependents();
  pdl_wait();
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  for (int a = threadIdx.x; a < T * K; a += kThreads) {
    const int e = idx[a];
    bool bad = e < -1 || e >= E;
    for (int b = a / K * K; b < a; ++b) bad |= e >= 0 && idx[b] == e;
    if (bad) s_bad = 1;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    const bool run = read_status(status) == 0;
    if (run && s_bad) set_status(status, MEP_ERR_BAD_ROUTING);
    *go = run && !s_bad;
  }
}

template <typename W>
__global__ void __launch_bounds__(kThreads) k_few_up(const __nv_bfloat16* x, const int32_t* idx, const W* w1, int group,
                                                     const int* go, int K, long long H, long long F,
                                                     __nv_bfloat16* act) {
  __shared__ float s_part[kThreads];
  pdl_launch_dependents();
  pdl_wait();
  const int a = blockIdx.y, e = *go ? idx[a] : -1;
  if (e < 0) return;
  const long long f = (long long)blockIdx.x * kColumns + threadIdx.x % kColumns;
  float g, u;
  if (sizeof(W) == 1) {
    const auto wg = matrix(w1, 2LL * e, H, F, group), wu = matrix(w1, 2LL * e + 1, H, F, group);
    g = column_sum(x + a / K * H, wg, H, f, f < F, s_part);
    u = column_sum(x + a / K * H, wu, H, f, f < F, s_part);
  } else {
    const auto w = matrix(w1, e, H, 2 * F, group);
    g = column_sum(x + a / K * H, w, H, f, f < F, s_part);
    u = column_sum(x + a / K * H, w, H, F + f, f < F, s_part);
  }
  if (threadIdx.x < kColumns && f < F) act[(long long)a * F + f] = __float2bfloat16_rn(g / (1.f + expf(-g)) * u);
}

template <typename W>
__global__ void __launch_bounds__(kThreads) k_few_down(const __nv_bfloat16* act, const int32_t* idx, const float* topk_w,
                                                       const W* w2, int group, const int* go, int K, long long H,
                                                       long long F, __nv_bfloat16* out) {
  __shared__ float s_part[kThreads];
  pdl_launch_dependents();
  pdl_wait();
  if (!*go) return;
  const long long n = (long long)blockIdx.x * kColumns + threadIdx.x % kColumns;
  float sum = 0.f;
  for (int k = 0; k < K; ++k) {
    const int a = blockIdx.y * K + k, e = idx[a];
    if (e < 0) continue;
    const float y = column_sum(act + (long long)a * F, matrix(w2, e, F, H, group), F, n, n < H, s_part);
    sum = fmaf(topk_w[a], y, sum);
  }
  if (threadIdx.x < kColumns && n < H) out[blockIdx.y * H + n] = __float2bfloat16_rn(sum);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_w4_product(const __nv_bfloat16* x, const uint8_t* w4, int32_t* status,
                                                         long long K, long long N, int group, T* y) {
  __shared__ float s_part[kThreads];
  pdl_launch_dependents();
  pdl_wait();
  if (read_status(status) != 0) return;
  const long long n = (long long)blockIdx.x * kColumns + threadIdx.x % kColumns;
  const float sum = column_sum(x + blockIdx.y * K, matrix(w4, 0, K, N, group), K, n, n < N, s_part);
  if (threadIdx.x < kColumns && n < N) y[blockIdx.y * N + n] = from_f32<T>(sum);
}

template <typename W>
int layer(const __nv_bfloat16* x, const int32_t* idx, const float* topk_w, const W* w1, const W* w2, int group,
          int32_t* status, int T, int K, int E, long long H, long long F, void* ws, __nv_bfloat16* out, cudaStream_t st) {
  int* go = static_cast<int*>(ws);
  __nv_bfloat16* act = reinterpret_cast<__nv_bfloat16*>(static_cast<char*>(ws) + 256);
  const auto blocks = [](long long n) { return unsigned((n + kColumns - 1) / kColumns); };
  if (launch_pdl(k_few_check, dim3(1), dim3(kThreads), 0, st, idx, T, K, E, status, go) != cudaSuccess ||
      launch_pdl(k_few_up<W>, dim3(blocks(F), T * K), dim3(kThreads), 0, st, x, idx, w1, group, go, K, H, F, act) !=
          cudaSuccess ||
      launch_pdl(k_few_down<W>, dim3(blocks(H), T), dim3(kThreads), 0, st, act, idx, topk_w, w2, group, go, K, H, F,
                 out) != cudaSuccess)
    return MEP_ERR_CUDA;
  return MEP_OK;
}

}  // namespace
}  // namespace mep

using namespace mep;

extern "C" int mep_w4_product_workspace_bytes(int T, int64_t K, int64_t N, int group, size_t* bytes) {
  if (bytes == nullptr || T < 0 || T > MEP_MAX_FEW || !w4_sizes_ok(K, N, group)) return MEP_ERR_INVALID_ARG;
  *bytes = 256;
  return MEP_OK;
}

extern "C" int mep_w4_product(const mep_bf16* x, const uint8_t* w4, int32_t* status, int T, int64_t K, int64_t N,
                              int group, void* ws, size_t ws_bytes, int y_type, void* y, void* stream) {
  size_t need = 0;
  if (mep_w4_product_workspace_bytes(T, K, N, group, &need) != MEP_OK || (y_type != MEP_BF16 && y_type != MEP_F32))
    return MEP_ERR_INVALID_ARG;
  if (T == 0) return MEP_OK;
  if (x == nullptr || w4 == nullptr || y == nullptr || ws == nullptr || ws_bytes < need) return MEP_ERR_INVALID_ARG;
  if (!aligned16(w4) || !aligned16(ws) || reinterpret_cast<uintptr_t>(x) % (K % 8 == 0 ? 16 : 2) != 0 ||
      reinterpret_cast<uintptr_t>(y) % (y_type == MEP_BF16 ? 2 : 4) != 0)
    return MEP_ERR_INVALID_ARG;
  const dim3 grid(unsigned((N + kColumns - 1) / kColumns), T);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const __nv_bfloat16* in = reinterpret_cast<const __nv_bfloat16*>(x);
  const cudaError_t e = y_type == MEP_BF16
                            ? launch_pdl(k_w4_product<__nv_bfloat16>, grid, dim3(kThreads), 0, st, in, w4, status, K, N,
                                         group, static_cast<__nv_bfloat16*>(y))
                            : launch_pdl(k_w4_product<float>, grid, dim3(kThreads), 0, st, in, w4, status, K, N, group,
                                         static_cast<float*>(y));
  return e == cudaSuccess ? MEP_OK : MEP_ERR_CUDA;
}

extern "C" int mep_expert_layer_workspace_bytes(int T, int K, int E, int64_t H, int64_t F, int w_type, int group,
                                                size_t* bytes) {
  if (bytes == nullptr || T < 0 || T > MEP_MAX_FEW || K < 1 || K > MEP_MAX_K || E < 1 || E > MEP_MAX_E || H < 8 ||
      F < 8 || H % 8 != 0 || F % 8 != 0 || H > MEP_MAX_W4 || F > MEP_MAX_W4 / 2)
    return MEP_ERR_INVALID_ARG;
  if (w_type != MEP_BF16 && (w_type != MEP_W4 || !w4_sizes_ok(H, F, group))) return MEP_ERR_INVALID_ARG;
  *bytes = 256 + (size_t)T * K * F * 2;
  return MEP_OK;
}

extern "C" int mep_expert_layer(const mep_bf16* x, const int32_t* topk_idx, const float* topk_w, const void* w1,
                                const void* w2, int w_type, int group, int32_t* status, int T, int K, int E, int64_t H,
                                int64_t F, void* ws, size_t ws_bytes, mep_bf16* out, void* stream) {
  size_t need = 0;
  if (mep_expert_layer_workspace_bytes(T, K, E, H, F, w_type, group, &need) != MEP_OK) return MEP_ERR_INVALID_ARG;
  if (T == 0) return MEP_OK;
  if (x == nullptr || topk_idx == nullptr || topk_w == nullptr || w1 == nullptr || w2 == nullptr || ws == nullptr ||
      out == nullptr || ws_bytes < need)
    return MEP_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w1) || !aligned16(w2) || !aligned16(ws) || !aligned16(out) ||
      reinterpret_cast<uintptr_t>(topk_idx) % 4 != 0 || reinterpret_cast<uintptr_t>(topk_w) % 4 != 0)
    return MEP_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const __nv_bfloat16* in = reinterpret_cast<const __nv_bfloat16*>(x);
  __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(out);
  return w_type == MEP_BF16
             ? layer(in, topk_idx, topk_w, static_cast<const __nv_bfloat16*>(w1), static_cast<const __nv_bfloat16*>(w2),
                     group, status, T, K, E, H, F, ws, o, st)
             : layer(in, topk_idx, topk_w, static_cast<const uint8_t*>(w1), static_cast<const uint8_t*>(w2), group,
                     status, T, K, E, H, F, ws, o, st);
}
