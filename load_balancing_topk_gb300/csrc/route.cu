// route.cu -- the router's choice from its logits (mep_route) and the logits'
// gradient (mep_route_backward).
//
// A warp takes a token's row. Forward, the logits become whole numbers of the
// same order; K times the warp takes the largest one that is left (a maximum
// over the lanes, then the lowest index that has it). Backward, the row is
// zeros but for K places.

#include <math.h>

#include "ckpt.cuh"

namespace mep {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;

// A number whose order is that of the values, equal for both zeros, NaN on top.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  if ((b & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_route(const T* __restrict__ logits, const float* __restrict__ bias,
                                                    long long N, int E, int K, int skip_masked,
                                                    int32_t* __restrict__ idx, float* __restrict__ w) {
  extern __shared__ uint32_t s_keys[];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* key = s_keys + warp * E;
  for (long long row = (long long)blockIdx.x * kWarps + warp; row < N; row += (long long)gridDim.x * kWarps) {
    const T* in = logits + row * E;
    for (int e = lane; e < E; e += 32) {
      const float l = to_f32(in[e]);
      key[e] = order_of(bias == nullptr ? l : l + bias[e]);
    }
    __syncwarp();
    int mine[2] = {0, 0};  // chosen number lane, and lane + 32
    for (int k = 0; k < K; ++k) {
      uint32_t best = 0;
      int at = 0x7fffffff;
      for (int e = lane; e < E; e += 32)  // 0 is no value's order: it marks what is taken
        if (key[e] > best) best = key[e], at = e;
      const uint32_t top = __reduce_max_sync(MEP_FULL_MASK, best);
      at = __reduce_min_sync(MEP_FULL_MASK, best == top ? at : 0x7fffffff);
      if (lane == 0) key[at] = 0;
      if ((k & 31) == lane) mine[k >> 5] = at;
      __syncwarp();
    }
    float l[2], m = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] = 32 * i + lane < K ? to_f32(in[mine[i]]) : -INFINITY;
      nan |= isnan(l[i]);
      m = fmaxf(m, l[i]);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(MEP_FULL_MASK, m, d));
    nan = __any_sync(MEP_FULL_MASK, nan);
    float ex[2], sum = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ex[i] = l[i] == -INFINITY ? 0.f : expf(l[i] - m);
      sum += ex[i];
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(MEP_FULL_MASK, sum, d);
    if (nan) sum = __uint_as_float(0x7fc00000u);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = 32 * i + lane;
      if (k < K) {
        idx[row * K + k] = skip_masked && l[i] == -INFINITY ? -1 : mine[i];
        w[row * K + k] = sum == 0.f ? 0.f : ex[i] / sum;
      }
    }
    __syncwarp();
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_route_backward(const float* __restrict__ dw, const float* __restrict__ w,
                                                             const int32_t* __restrict__ idx, int32_t* status,
                                                             long long N, int E, int K, T* __restrict__ dlogits) {
  extern __shared__ float s_rows[];
  pdl_launch_dependents();
  pdl_wait();
  if (read_status(status) != 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* d = s_rows + warp * E;
  bool bad = false;
  for (long long row = (long long)blockIdx.x * kWarps + warp; row < N; row += (long long)gridDim.x * kWarps) {
    for (int e = lane; e < E; e += 32) d[e] = 0.f;
    float wk[2], dk[2], sum = 0.f;
    int at[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = 32 * i + lane;
      wk[i] = k < K ? w[row * K + k] : 0.f;
      dk[i] = k < K ? dw[row * K + k] : 0.f;
      at[i] = k < K ? idx[row * K + k] : -1;
      bad |= at[i] < -1 || at[i] >= E;
      sum += k < K ? wk[i] * dk[i] : 0.f;
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(MEP_FULL_MASK, sum, s);
    __syncwarp();
    for (int k = 0; k < K; ++k) {  // one after another: an expert that stands twice gets both, in order
      const float v = wk[k >> 5] * (dk[k >> 5] - sum);
      if ((k & 31) == lane && at[k >> 5] >= 0 && at[k >> 5] < E) d[at[k >> 5]] += v;
      __syncwarp();
    }
    for (int e = lane; e < E; e += 32) dlogits[row * E + e] = from_f32<T>(d[e]);
    __syncwarp();
  }
  if (bad) set_status(status, MEP_ERR_BAD_ROUTING);
}

bool sizes_ok(int64_t N, int E, int K, int type) {
  return N >= 0 && N <= 0x7fffffffLL && E >= 1 && E <= MEP_MAX_E && K >= 1 && K <= E && K <= MEP_MAX_K &&
         (type == MEP_BF16 || type == MEP_F32);
}
bool on(const void* p, unsigned size) { return p != nullptr && reinterpret_cast<uintptr_t>(p) % size == 0; }

template <typename Kernel, typename... Args>
int launch_rows(Kernel kernel, int64_t N, int E, cudaStream_t st, Args... args) {
  const int smem = kWarps * E * 4;
  if (set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), smem)) return MEP_ERR_CUDA;
  const long long blocks = (N + kWarps - 1) / kWarps, most = 16LL * sm_count();
  return launch_pdl(kernel, dim3(unsigned(blocks < most ? blocks : most)), dim3(kThreads), smem, st, args...) ==
                 cudaSuccess
             ? MEP_OK
             : MEP_ERR_CUDA;
}

}  // namespace
}  // namespace mep

using namespace mep;

extern "C" int mep_route(const void* logits, int type, const float* bias, int64_t N, int E, int K, int skip_masked,
                         int32_t* topk_idx, float* topk_w, void* stream) {
  if (!sizes_ok(N, E, K, type)) return MEP_ERR_INVALID_ARG;
  if (N == 0) return MEP_OK;
  if (!on(logits, type == MEP_BF16 ? 2 : 4) || (bias != nullptr && !on(bias, 4)) || !on(topk_idx, 4) || !on(topk_w, 4))
    return MEP_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return type == MEP_BF16 ? launch_rows(k_route<__nv_bfloat16>, N, E, st, static_cast<const __nv_bfloat16*>(logits),
                                        bias, N, E, K, skip_masked, topk_idx, topk_w)
                          : launch_rows(k_route<float>, N, E, st, static_cast<const float*>(logits), bias, N, E, K,
                                        skip_masked, topk_idx, topk_w);
}

extern "C" int mep_route_backward(const float* dtopk_w, const float* topk_w, const int32_t* topk_idx, int32_t* status,
                                  int64_t N, int E, int K, int type, void* dlogits, void* stream) {
  if (!sizes_ok(N, E, K, type)) return MEP_ERR_INVALID_ARG;
  if (N == 0) return MEP_OK;
  if (!on(dtopk_w, 4) || !on(topk_w, 4) || !on(topk_idx, 4) || !on(dlogits, type == MEP_BF16 ? 2 : 4))
    return MEP_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return type == MEP_BF16 ? launch_rows(k_route_backward<__nv_bfloat16>, N, E, st, dtopk_w, topk_w, topk_idx, status, N,
                                        E, K, static_cast<__nv_bfloat16*>(dlogits))
                          : launch_rows(k_route_backward<float>, N, E, st, dtopk_w, topk_w, topk_idx, status, N, E, K,
                                        static_cast<float*>(dlogits));
}
