// act_ckpt.cu -- 8-bit activation checkpoints (mep_ckpt_save, mep_ckpt_load)
// and the experts' gated activation that writes and reads them (mep_swiglu,
// mep_swiglu_backward).
//
// All four are one pass over memory: each byte is read once and written once
// (save 2 + 1.01 bytes a bf16 value, load the reverse; per value of the
// activation 4 in, 2 + 2.02 out forward, 2 + 2.02 in, 4 + 2 out backward).
// A half warp takes a block of 128 columns, eight values a lane, and gets the
// block's largest magnitude in four shuffles; a thread holds a few blocks at a
// time, all loaded before the first is used. Where a row is a multiple of 8
// columns a lane's values are one 16-byte vector; otherwise they are fetched
// one by one, coalesced over the half warp.
// What bounds them is DRAM, and in small calls the launch. The activation
// forward and backward on [196608, 2, 1408] takes 737 us, 6.8 TB/s (a copy
// runs at 6.8); saving and loading [32768, 2048] 70 us, 5.8 TB/s, of which some
// 4 us a launch are its start and end. Rows one by one issue two to three times
// as much: [32768, 2047] 108 us, the activation on [65536, 2, 1407] 398
// where 1408 columns take 255.

#include "ckpt.cuh"

namespace mep {
namespace {

constexpr int kThreads = 256;
// Blocks a thread holds. Saving and loading [32768, 2048] in bf16 with 2, 4, 6
// and 8: 76, 76, 85 and 101 us, more registers and so fewer warps; the
// activation on [196608, 2, 1408] with 1, 2, 3 and 4: 781, 740, 750 and 876. fp32
// has half as many (1, 2, 4: 128, 126, 126 us). Without vectors one, as eight
// loads are under way then: the activation on [65536, 2, 1407] with 1, 2 and 4:
// 399, 398 and 573 us.
constexpr int kCkptUnroll = 4, kSwigluUnroll = 2;

// Where the U blocks of this half warp are. Blocks are numbered over the whole
// tensor; a thread's are kThreads / 16 apart.
struct Where {
  long long row;
  int block;
  bool in;
};
// Blocks: how many there are, how many a row has, and the quotient i / per_row
// of i < 2^31 by a product: with 2^l >= per_row and m = floor(2^(31+l) /
// per_row) + 1, m * per_row is off 2^(31+l) by at most 2^l, too little to
// reach the next quotient. (Divisions were a tenth of what the kernels issue.)
struct Blocks {
  uint32_t all, per_row, m;
  int shift;
};
Blocks blocks_of(uint32_t all, int C) {
  const uint32_t d = (C + kCkptBlock - 1) / kCkptBlock;
  int l = 0;
  while ((1u << l) < d) ++l;
  return {all, d, d == 1 ? 0u : uint32_t((1ull << (31 + l)) / d + 1), l - 1};
}
template <int U> __device__ __forceinline__ void where(Where (&w)[U], const Blocks& b) {
  const uint32_t first = blockIdx.x * uint32_t(U * kThreads / kHalf) + threadIdx.x / kHalf;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = first + u * (kThreads / kHalf), row = b.per_row == 1 ? i : __umulhi(i, b.m) >> b.shift;
    w[u].in = i < b.all;
    w[u].row = row;
    w[u].block = int(i - row * b.per_row);
  }
}

// (six CTAs an SM: 40 registers; left to itself it takes 44, five CTAs, 2.5%
// longer, and with 32 spills)
template <int KIND, bool VEC, int U>
__global__ void __launch_bounds__(kThreads, 6)
    k_ckpt_save(const void* __restrict__ x, Blocks blocks, int C, uint8_t* __restrict__ ckpt) {
  pdl_wait();
  pdl_launch_dependents();
  const int l = threadIdx.x % kHalf;
  Where w[U];
  where<U>(w, blocks);
  Pack<KIND> p[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (w[u].in)
      p[u].template load<VEC>(x, w[u].row, C, w[u].block, l);
    else
      p[u].clear();
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    Kept<1> k{{ckpt + w[u].row * ckpt_row_bytes(C)}, {w[u].block}, {w[u].in}, {p[u].top()}};
#pragma unroll
    for (int j = 0; j < 4; ++j) k.v[0][j] = p[u].at(j);
    save8<VEC>(k, C, l);
  }
}

template <typename T, bool VEC, int U>
__global__ void __launch_bounds__(kThreads)
    k_ckpt_load(const uint8_t* __restrict__ ckpt, Blocks blocks, int C, T* __restrict__ x) {
  pdl_wait();
  pdl_launch_dependents();
  const int l = threadIdx.x % kHalf;
  Where w[U];
  where<U>(w, blocks);
  Pack<MEP_CKPT8> p[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (w[u].in) p[u].template load<VEC>(ckpt, w[u].row, C, w[u].block, l);
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (w[u].in) {
      F2 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = p[u].at(j);
      store8<T, VEC>(x + w[u].row * C, C, w[u].block, l, v);
    }
}

// sigmoid(g) = k / (k + k e^-g) with k = 2^-24: e^-g stays below 2^126, where
// the reciprocal instruction still has a result, down to g = -104, where
// sigmoid itself leaves fp32's range. Without k it was flushed to 0 below g =
// -87.3 already, which u = 1e38 makes an activation of -87; to scale costs
// nothing, as k e^-g = 2^(-g log2 e - 24) is one fma where e^-g is a product.
// (e^-|g| and its numerator by the sign of g: 780 us for the activation forward
// and backward on [196608, 2, 1408], this 740.) Relative error, in units of
// 2^-24: 17 + 2 |g| of the exponent, 3 of ex2, 1 of the sum, 2 of the reciprocal.
__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ F2 sigmoid2(F2 g) {
  constexpr float kLog2e = 1.44269504f, k = 1.f / (1 << 24);
  const F2 v = fma2(g, both(-kLog2e), both(-24.f));
  const F2 y = add2(pair(ex2(v.x()), ex2(v.y())), both(k));
  return mul2(pair(rcp(y.x()), rcp(y.y())), both(k));
}

// (five CTAs an SM for both: 48 registers, left to themselves 50, four CTAs:
// forward with a checkpoint on [196608, 2, 1408] 338 us and 352, backward from
// it 409 and 432; without vectors the forward pass has 40, six CTAs, and given
// more ran slower, on [65536, 2, 1407] 190 us for 176)
template <bool VEC, bool CKPT, int U>
__global__ void __launch_bounds__(kThreads, VEC ? 5 : 6)
    k_swiglu(const __nv_bfloat16* __restrict__ gu, Blocks blocks, int F,
             __nv_bfloat16* __restrict__ a, uint8_t* __restrict__ ckpt) {
  pdl_wait();
  pdl_launch_dependents();
  const int l = threadIdx.x % kHalf;
  Where w[U];
  where<U>(w, blocks);
  Pack<MEP_BF16> p[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (w[u].in)
        p[u][h].template load<VEC>(gu, 2 * w[u].row + h, F, w[u].block, l);
      else
        p[u][h].clear();
    }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    F2 o[4];
    Kept<2> k;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      k.v[0][j] = p[u][0].at(j);
      k.v[1][j] = p[u][1].at(j);
      o[j] = mul2(mul2(k.v[0][j], sigmoid2(k.v[0][j])), k.v[1][j]);
    }
    if (w[u].in) store8<__nv_bfloat16, VEC>(a + w[u].row * F, F, w[u].block, l, o);
    if (CKPT) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        k.row[h] = ckpt + (2 * w[u].row + h) * ckpt_row_bytes(F);
        k.block[h] = w[u].block;
        k.in[h] = w[u].in;
        k.top[h] = p[u][h].top();
      }
      save8<VEC>(k, F, l);
    }
  }
}

template <int KIND, bool VEC, int U>
__global__ void __launch_bounds__(kThreads, KIND == MEP_CKPT8 ? 5 : 1)
    k_swiglu_backward(const __nv_bfloat16* __restrict__ da, const void* __restrict__ gu,
                      Blocks blocks, int F, __nv_bfloat16* __restrict__ dgu,
                      __nv_bfloat16* __restrict__ a) {
  pdl_wait();
  pdl_launch_dependents();
  const int l = threadIdx.x % kHalf;
  Where w[U];
  where<U>(w, blocks);
  Pack<KIND> p[U][2];
  Pack<MEP_BF16> d[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (w[u].in) {
      p[u][0].template load<VEC>(gu, 2 * w[u].row, F, w[u].block, l);
      p[u][1].template load<VEC>(gu, 2 * w[u].row + 1, F, w[u].block, l);
      d[u].template load<VEC>(da, w[u].row, F, w[u].block, l);
    }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (w[u].in) {
      F2 dg[4], du[4], o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const F2 g = p[u][0].at(j), up = p[u][1].at(j), dv = d[u].at(j), s = sigmoid2(g);
        const F2 one = both(1.f), gs = mul2(g, s), rest = fma2(both(-1.f), s, one);  // 1 - s
        dg[j] = mul2(mul2(mul2(dv, up), s), fma2(g, rest, one));
        du[j] = mul2(dv, gs);
        o[j] = mul2(gs, up);
      }
      store8<__nv_bfloat16, VEC>(dgu + 2 * w[u].row * F, F, w[u].block, l, dg);
      store8<__nv_bfloat16, VEC>(dgu + (2 * w[u].row + 1) * F, F, w[u].block, l, du);
      if (a != nullptr) store8<__nv_bfloat16, VEC>(a + w[u].row * F, F, w[u].block, l, o);
    }
}

// Runs f(first row, blocks, grid) over slices of rows whose blocks fit 32 bits.
template <int U, typename F> int sliced(long long rows, long long C, F f) {
  const long long nb = (C + kCkptBlock - 1) / kCkptBlock, most = 0x40000000LL / nb;
  constexpr int per = U * kThreads / kHalf;
  for (long long r = 0; r < rows; r += most) {
    const long long n = (rows - r < most ? rows - r : most) * nb;
    if (f(r, blocks_of(uint32_t(n), int(C)), dim3(unsigned((n + per - 1) / per))) != cudaSuccess) return MEP_ERR_CUDA;
  }
  return MEP_OK;
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
  if (x == nullptr || ckpt == nullptr || !may_start(x, type, C) || !aligned16(ckpt)) return MEP_ERR_INVALID_ARG;
  return MEP_OK;
}

extern "C" int mep_ckpt_save(const void* x, int x_type, int64_t N, int64_t C, uint8_t* ckpt,
                             void* stream) {
  const int rc = ckpt_check(x, x_type, N, C, ckpt);
  if (rc != MEP_OK || N == 0) return rc;
  constexpr int U = kCkptUnroll;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf16 = x_type == MEP_BF16, vec = C % 8 == 0;
  const auto kernel = bf16 ? (vec ? k_ckpt_save<MEP_BF16, true, U> : k_ckpt_save<MEP_BF16, false, 1>)
                           : (vec ? k_ckpt_save<MEP_F32, true, U / 2> : k_ckpt_save<MEP_F32, false, 1>);
  const auto f = [&](long long r, Blocks blocks, dim3 grid) {
    const void* p = static_cast<const char*>(x) + r * C * (bf16 ? 2 : 4);
    return launch_pdl(kernel, grid, dim3(kThreads), 0, st, p, blocks, int(C), ckpt + r * ckpt_row_bytes(C));
  };
  return !vec ? sliced<1>(N, C, f) : bf16 ? sliced<U>(N, C, f) : sliced<U / 2>(N, C, f);
}

extern "C" int mep_ckpt_load(const uint8_t* ckpt, int64_t N, int64_t C, int x_type, void* x,
                             void* stream) {
  const int rc = ckpt_check(x, x_type, N, C, ckpt);
  if (rc != MEP_OK || N == 0) return rc;
  constexpr int U = kCkptUnroll;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool vec = C % 8 == 0;
  const auto run = [&](auto* out, auto kernel) {
    return [=](long long r, Blocks blocks, dim3 grid) {
      return launch_pdl(kernel, grid, dim3(kThreads), 0, st, ckpt + r * ckpt_row_bytes(C), blocks, int(C),
                        out + r * C);
    };
  };
  if (x_type == MEP_BF16) {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(x);
    return vec ? sliced<U>(N, C, run(o, k_ckpt_load<__nv_bfloat16, true, U>))
               : sliced<1>(N, C, run(o, k_ckpt_load<__nv_bfloat16, false, 1>));
  }
  float* o = static_cast<float*>(x);
  return vec ? sliced<U>(N, C, run(o, k_ckpt_load<float, true, U>))
             : sliced<1>(N, C, run(o, k_ckpt_load<float, false, 1>));
}

extern "C" int mep_swiglu(const mep_bf16* gu, int64_t rows, int64_t F, mep_bf16* a, uint8_t* ckpt,
                          void* stream) {
  if (rows < 0 || rows > 0x3fffffffLL || F < 1 || F > MEP_MAX_CKPT_C) return MEP_ERR_INVALID_ARG;
  if (rows == 0) return MEP_OK;
  if (gu == nullptr || a == nullptr || !may_start(gu, MEP_BF16, F) || !may_start(a, MEP_BF16, F) || !aligned16(ckpt))
    return MEP_ERR_INVALID_ARG;
  constexpr int U = kSwigluUnroll;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const __nv_bfloat16* in = reinterpret_cast<const __nv_bfloat16*>(gu);
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a);
  const bool vec = F % 8 == 0;
  const auto kernel = vec ? (ckpt != nullptr ? k_swiglu<true, true, U> : k_swiglu<true, false, U>)
                          : (ckpt != nullptr ? k_swiglu<false, true, 1> : k_swiglu<false, false, 1>);
  const auto f = [&](long long r, Blocks blocks, dim3 grid) {
    return launch_pdl(kernel, grid, dim3(kThreads), 0, st, in + 2 * r * F, blocks, int(F), out + r * F,
                      ckpt == nullptr ? nullptr : ckpt + 2 * r * ckpt_row_bytes(F));
  };
  return vec ? sliced<U>(rows, F, f) : sliced<1>(rows, F, f);
}

extern "C" int mep_swiglu_backward(const mep_bf16* da, const void* gu, int gu_type, int64_t rows,
                                   int64_t F, mep_bf16* dgu, mep_bf16* a, void* stream) {
  if (rows < 0 || rows > 0x3fffffffLL || F < 1 || F > MEP_MAX_CKPT_C) return MEP_ERR_INVALID_ARG;
  if (gu_type != MEP_BF16 && gu_type != MEP_CKPT8) return MEP_ERR_INVALID_ARG;
  if (rows == 0) return MEP_OK;
  if (da == nullptr || gu == nullptr || dgu == nullptr || !may_start(da, MEP_BF16, F) ||
      !may_start(gu, gu_type, F) || !may_start(dgu, MEP_BF16, F) || !may_start(a, MEP_BF16, F))
    return MEP_ERR_INVALID_ARG;
  constexpr int U = kSwigluUnroll;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const __nv_bfloat16* in = reinterpret_cast<const __nv_bfloat16*>(da);
  __nv_bfloat16 *o = reinterpret_cast<__nv_bfloat16*>(dgu), *oa = reinterpret_cast<__nv_bfloat16*>(a);
  const bool vec = F % 8 == 0, kept = gu_type == MEP_CKPT8;
  const auto kernel = kept ? (vec ? k_swiglu_backward<MEP_CKPT8, true, U> : k_swiglu_backward<MEP_CKPT8, false, 1>)
                           : (vec ? k_swiglu_backward<MEP_BF16, true, U> : k_swiglu_backward<MEP_BF16, false, 1>);
  const auto f = [&](long long r, Blocks blocks, dim3 grid) {
    const void* p = static_cast<const char*>(gu) + r * (kept ? 2 * ckpt_row_bytes(F) : 4 * F);
    return launch_pdl(kernel, grid, dim3(kThreads), 0, st, in + r * F, p, blocks, int(F), o + 2 * r * F,
                      oa == nullptr ? nullptr : oa + r * F);
  };
  return vec ? sliced<U>(rows, F, f) : sliced<1>(rows, F, f);
}
