// route.cu -- the router's choice from its logits (mep_route) and the logits'
// gradient (mep_route_backward).
//
// A warp takes a token's row. Forward, the logits become whole numbers of the
// same order. Up to 512 experts a lane has its values in registers: the K-th
// largest of the lanes' maxima (K times a maximum over the warp, without whose it
// is) is a bound that the K largest values and few others reach, a dozen of 256
// normal logits with K = 8; those are put together, one a lane, and each finds
// its place by comparing itself with the others. Only where more than 32 values
// reach the bound (many equal ones) the warp takes the largest that is left K
// times. What bounds it is what a warp has to issue. More experts: the orders lie
// in shared memory, and the largest is taken K times.
// Backward, the row is zeros but for K places: built in shared memory, which
// stays zero otherwise, and written out in vectors. What bounds it is again a
// warp's row: half the issue slots are taken, and its bytes alone would take half
// the time.
//
// Measured, fp32 logits, L2 flushed before: [65536, 256], K 8: 36.4 us forward,
// 21.6 backward, where 71 MB each way take 10.7 at the copy rate (bf16 40 and 19.6,
// 5.6); [65536, 384], K 8: 46 and 26 (16); [32768, 64], K 6: 17.5 and 13.4 (1.5);
// [65536, 640], K 8: 100 and 34 (26); [65536, 256], K 40: 194 and 138 (13). Steps of the first: the largest taken
// K times out of shared memory 78 (384 experts, as every larger number still is),
// out of registers with the lanes' best two kept 56, the bound and the ranking of
// what reaches it 42, the next row's values on their way 39.6, orders in two
// operations and the softmax's maximum by one reduction 37.5, four maxima of the
// bound to a turn of its loop 36.1. In bf16 40.1: equal values send some rows the
// long way.

#include <math.h>

#include "ckpt.cuh"

namespace mep {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kCheckThreads = 256, kCheckEach = 8;  // indices that a thread has on their way at once

// A number whose order is that of the values, equal for both zeros and for all
// NaN (a sum that is a NaN is the canonical one), NaN on top.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}

// The value of an order (+0 for either zero).
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

// Weights of the chosen: lane and lane + 32 have number lane and lane + 32, their
// logits l.
__device__ __forceinline__ void put_row(const float (&l)[2], const int (&at)[2], int K, int skip_masked, int32_t* idx,
                                        float* w) {
  const int lane = threadIdx.x & 31;
  float m = fmaxf(l[0], l[1]);
  bool nan = isnan(l[0]) || isnan(l[1]);
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
      idx[k] = skip_masked && l[i] == -INFINITY ? -1 : at[i];
      w[k] = sum == 0.f ? 0.f : ex[i] / sum;
    }
  }
}

// Up to 32 NV experts, K <= 32: expert lane + 32 i is value i of the lane, or with
// rows of whole vectors four experts next to one another are four of its values:
// in bf16, where loads of two bytes cost more than widening eight at once (E 384, K
// 8: 66 us without, 50 with; 512, K 16: 112 and 103; 256, K 8: 42 both). In fp32 the
// vectors' arrival together costs more than they save (256, K 8: 38 without, 40
// with; 384: 46 and 54).
template <typename T, int NV, bool VEC>
__global__ void __launch_bounds__(kThreads) k_route_few(const T* __restrict__ logits, const float* __restrict__ bias,
                                                        long long N, int E, int K, int skip_masked,
                                                        int32_t* __restrict__ idx, float* __restrict__ w) {
  __shared__ uint2 s_found[kWarps][32];  // order, expert
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint2* found = s_found[warp];
  const long long step = (long long)gridDim.x * kWarps;
  long long row = (long long)blockIdx.x * kWarps + warp;
  const auto expert = [&](int i) { return VEC ? 128 * (i / 4) + 4 * lane + i % 4 : lane + 32 * i; };
  float v[NV];  // of the next row, on its way while this one is worked on
  const auto load = [&](long long r) {
    if (VEC) {
#pragma unroll
      for (int i = 0; i < NV; i += 4) {
        const uint2 f = r < N && expert(i) < E ? *reinterpret_cast<const uint2*>(logits + r * E + expert(i)) : make_uint2(0u, 0u);
        v[i] = __uint_as_float(f.x << 16), v[i + 1] = __uint_as_float(f.x & 0xffff0000u);
        v[i + 2] = __uint_as_float(f.y << 16), v[i + 3] = __uint_as_float(f.y & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = r < N && expert(i) < E ? to_f32(logits[r * E + expert(i)]) : 0.f;
    }
  };
  load(row);
  for (; row < N; row += step) {
    uint32_t key[NV], most = 0;  // 0: no expert
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = expert(i);
      key[i] = e < E ? order_of(bias == nullptr ? v[i] : v[i] + bias[e]) : 0u;
      most = max(most, key[i]);
    }
    load(row + step);
    uint32_t bound = 0;
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
      bound = __reduce_max_sync(MEP_FULL_MASK, most);
      if (most == bound) most = 0;
    }
    bound = max(bound, 1u);
    int count = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) count += key[i] >= bound;
    int at = warp_incl_scan(count);
    const int all = __shfl_sync(MEP_FULL_MASK, at, 31);
    int mine = 0, rank = 32;  // expert, and its place among the chosen
    uint32_t order = 0;
    if (all <= 32) {
      at -= count;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (key[i] >= bound) found[at++] = make_uint2(key[i], expert(i));
      __syncwarp();
      const uint2 f = lane < all ? found[lane] : make_uint2(0u, 0u);
      mine = int(f.y), order = f.x, rank = lane < all ? 0 : 32;
#pragma unroll 4
      for (int o = 0; o < all; ++o) {
        const uint2 other = found[o];
        rank += other.x > f.x || (other.x == f.x && other.y < f.y);
      }
      __syncwarp();
    } else {
      uint32_t last = 0xffffffffu;  // order and place of the last one taken
      int last_at = -1;
#pragma unroll 1
      for (int k = 0; k < K; ++k) {
        uint32_t best = 0;
        int e = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int here = expert(i);
          if ((key[i] < last || (key[i] == last && here > last_at)) && key[i] > best) best = key[i], e = here;
        }
        last = __reduce_max_sync(MEP_FULL_MASK, best);
        last_at = __reduce_min_sync(MEP_FULL_MASK, best == last ? e : 0x7fffffff);
        if (k == lane) mine = last_at, order = last, rank = k;
      }
    }
    // the chosen, in any order of lanes: each one's weight goes to its place
    const bool chosen = rank < K;
    const float l = !chosen ? -INFINITY : bias == nullptr ? value_of(order) : to_f32(logits[row * E + mine]);
    float m = l;
    if (bias == nullptr) {
      m = value_of(__reduce_max_sync(MEP_FULL_MASK, chosen ? order : 0u));
    } else {
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(MEP_FULL_MASK, m, d));
    }
    float ex = l == -INFINITY ? 0.f : expf(l - m), sum = ex;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(MEP_FULL_MASK, sum, d);
    if (chosen) {
      idx[row * K + rank] = skip_masked && l == -INFINITY ? -1 : mine;
      w[row * K + rank] = sum == 0.f ? 0.f : ex / sum;
    }
  }
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
    float l[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) l[i] = 32 * i + lane < K ? to_f32(in[mine[i]]) : -INFINITY;
    put_row(l, mine, K, skip_masked, idx + row * K, w + row * K);
    __syncwarp();
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) k_route_backward(const float* __restrict__ dw, const float* __restrict__ w,
                                                             const int32_t* __restrict__ idx, const int32_t* status,
                                                             long long N, int E, int K, T* __restrict__ dlogits) {
  extern __shared__ __align__(16) float s_rows[];
  pdl_launch_dependents();
  pdl_wait();
  if (read_status(status) != 0) return;  // set before the launch: k_route_check, which sets it, runs after the last block
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, pitch = (E + 7) & ~7;
  float* d = s_rows + warp * pitch;
  for (int e = lane; e < pitch; e += 32) d[e] = 0.f;
  const long long step = (long long)gridDim.x * kWarps;
  long long row = (long long)blockIdx.x * kWarps + warp;
  float wn[2], dn[2];  // of the next row
  int an[2];
  const auto load = [&](long long r) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool there = r < N && 32 * i + lane < K;
      const long long k = r * K + 32 * i + lane;
      wn[i] = there ? w[k] : 0.f, dn[i] = there ? dw[k] : 0.f, an[i] = there ? idx[k] : -1;
    }
  };
  load(row);
  for (; row < N; row += step) {
    float wk[2], dk[2], sum = 0.f;
    int at[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      wk[i] = wn[i], dk[i] = dn[i], at[i] = an[i];
      if (at[i] >= E) at[i] = -1;  // below -1 it counts as -1 as it is
      sum += at[i] >= 0 ? wk[i] * dk[i] : 0.f;
    }
    load(row + step);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(MEP_FULL_MASK, sum, s);
    // an expert that stands twice gets both, one after another
    const unsigned same = __match_any_sync(MEP_FULL_MASK, at[0]);
    const bool once = at[0] < 0 || (same & (same - 1)) == 0;
    __syncwarp();
    if (K <= 32 && __all_sync(MEP_FULL_MASK, once)) {
      if (at[0] >= 0) d[at[0]] = wk[0] * (dk[0] - sum);
      __syncwarp();
    } else {
      for (int k = 0; k < K; ++k) {
        const int i = k >> 5;
        if ((k & 31) == lane && at[i] >= 0) d[at[i]] += wk[i] * (dk[i] - sum);
        __syncwarp();
      }
    }
    T* out = dlogits + row * E;
    if (VEC) {
      for (int e = 4 * lane; e < E; e += 128) {
        const float4 v = *reinterpret_cast<const float4*>(d + e);
        if (sizeof(T) == 4) {
          __stcs(reinterpret_cast<float4*>(out + e), v);
        } else {
          __nv_bfloat162 p[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
          __stcs(reinterpret_cast<uint2*>(out + e), *reinterpret_cast<const uint2*>(p));
        }
      }
    } else {
      for (int e = lane; e < E; e += 32) out[e] = from_f32<T>(d[e]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (at[i] >= 0) d[at[i]] = 0.f;
    __syncwarp();
  }
}

// The status word of a backward pass, in a launch of its own behind it: a block of
// the pass that set the word itself would turn away those that start later, whose
// rows then stayed unwritten (up to a third of 300007 rows). It adds 3.8 us to
// the 11.4 of [65536, 256], K 8, back to back, 1.5 to the smallest calls, and
// nothing where there is no status word.
__global__ void __launch_bounds__(kCheckThreads) k_route_check(const int32_t* __restrict__ idx, int32_t* status, long long n, int E) {
  pdl_launch_dependents();
  pdl_wait();
  if (read_status(status) != 0) return;
  const long long step = (long long)gridDim.x * kCheckThreads * kCheckEach;
  bool bad = false;
  for (long long i = (long long)blockIdx.x * kCheckThreads * kCheckEach + threadIdx.x; i < n; i += step) {
#pragma unroll
    for (int q = 0; q < kCheckEach; ++q) {
      const long long at = i + q * kCheckThreads;
      const int e = at < n ? idx[at] : -1;
      bad |= e < -1 || e >= E;
    }
  }
  if (__any_sync(MEP_FULL_MASK, bad) && (threadIdx.x & 31) == 0) set_status(status, MEP_ERR_BAD_ROUTING);
}

bool sizes_ok(int64_t N, int E, int K, int type) {
  return N >= 0 && N <= 0x7fffffffLL && E >= 1 && E <= MEP_MAX_E && K >= 1 && K <= E && K <= MEP_MAX_K &&
         (type == MEP_BF16 || type == MEP_F32);
}
bool on(const void* p, unsigned size) { return p != nullptr && reinterpret_cast<uintptr_t>(p) % size == 0; }

template <typename Kernel, typename... Args>
int launch_rows(Kernel kernel, int64_t N, int smem, cudaStream_t st, Args... args) {
  if (set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), smem)) return MEP_ERR_CUDA;
  const long long blocks = (N + kWarps - 1) / kWarps, most = 16LL * sm_count();
  return launch_pdl(kernel, dim3(unsigned(blocks < most ? blocks : most)), dim3(kThreads), smem, st, args...) ==
                 cudaSuccess
             ? MEP_OK
             : MEP_ERR_CUDA;
}
template <typename T>
int route(const T* logits, const float* bias, int64_t N, int E, int K, int skip_masked, int32_t* idx, float* w,
          cudaStream_t st) {
  const auto few = [&](auto kernel) { return launch_rows(kernel, N, 0, st, logits, bias, N, E, K, skip_masked, idx, w); };
  if (K > 32) return launch_rows(k_route<T>, N, kWarps * E * 4, st, logits, bias, N, E, K, skip_masked, idx, w);
  if (E <= 32) return few(k_route_few<T, 1, false>);
  if (E <= 64) return few(k_route_few<T, 2, false>);
  constexpr bool V = sizeof(T) == 2;  // fp32 has no such form
  const bool vec = V && E % 4 == 0 && reinterpret_cast<uintptr_t>(logits) % 8 == 0;
  if (E <= 128) return few(vec ? k_route_few<T, 4, V> : k_route_few<T, 4, false>);
  if (E <= 256) return few(vec ? k_route_few<T, 8, V> : k_route_few<T, 8, false>);
  if (E <= 512) return few(vec ? k_route_few<T, 16, V> : k_route_few<T, 16, false>);
  return launch_rows(k_route<T>, N, kWarps * E * 4, st, logits, bias, N, E, K, skip_masked, idx, w);
}
template <typename T>
int route_backward(const float* dw, const float* w, const int32_t* idx, int32_t* status, int64_t N, int E, int K, T* d,
                   cudaStream_t st) {
  const int smem = kWarps * ((E + 7) & ~7) * 4;
  const bool vec = E % 4 == 0 && reinterpret_cast<uintptr_t>(d) % (4 * sizeof(T)) == 0;
  const int rc = vec ? launch_rows(k_route_backward<T, true>, N, smem, st, dw, w, idx, status, N, E, K, d)
                     : launch_rows(k_route_backward<T, false>, N, smem, st, dw, w, idx, status, N, E, K, d);
  if (rc != MEP_OK || status == nullptr) return rc;
  const long long n = N * K, blocks = (n + kCheckThreads * kCheckEach - 1) / (kCheckThreads * kCheckEach), most = 8LL * sm_count();
  return launch_pdl(k_route_check, dim3(unsigned(blocks < most ? blocks : most)), dim3(kCheckThreads), 0, st, idx, status, n, E) ==
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
  return type == MEP_BF16
             ? route(static_cast<const __nv_bfloat16*>(logits), bias, N, E, K, skip_masked, topk_idx, topk_w, st)
             : route(static_cast<const float*>(logits), bias, N, E, K, skip_masked, topk_idx, topk_w, st);
}

extern "C" int mep_route_backward(const float* dtopk_w, const float* topk_w, const int32_t* topk_idx, int32_t* status,
                                  int64_t N, int E, int K, int type, void* dlogits, void* stream) {
  if (!sizes_ok(N, E, K, type)) return MEP_ERR_INVALID_ARG;
  if (N == 0) return MEP_OK;
  if (!on(dtopk_w, 4) || !on(topk_w, 4) || !on(topk_idx, 4) || !on(dlogits, type == MEP_BF16 ? 2 : 4))
    return MEP_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return type == MEP_BF16 ? route_backward(dtopk_w, topk_w, topk_idx, status, N, E, K, static_cast<__nv_bfloat16*>(dlogits), st)
                          : route_backward(dtopk_w, topk_w, topk_idx, status, N, E, K, static_cast<float*>(dlogits), st);
}
