// layer_norm.cu -- layer norm over the hidden width (mep_layer_norm) and its
// backward pass (mep_layer_norm_backward), with 8-bit checkpoint rows as a
// by-product of the first and as input of the second.
//
// Both are one pass over memory with the row in registers: a row belongs to W
// warps, whose half warps hold blocks of 128 columns, eight values a lane
// (the checkpoint's blocks, so that a block's largest magnitude is four
// shuffles away). Sums over a row go through shuffles and, for W > 1, a few
// words of shared memory.
//   k_norm       the mean first, then the sum of the centred squares: with
//                the row in registers the second pass costs no memory, and a
//                row far from zero loses nothing to cancellation.
//   k_norm_dx    dx of U rows at a time; every thread also keeps the sums
//                over its rows for its own columns of dweight and dbias, which
//                the CTA's row groups join at the end and write to the
//                workspace, one pair of rows of H per CTA.
//   k_norm_dw    adds those up, in order of the CTA.

#include "ckpt.cuh"

namespace mep {
namespace {

constexpr int kMaxH = MEP_MAX_NORM_H;
constexpr int kMaxWarps = 32;

// ---------------------------------------------------------------------------
// Barrier of one row group: W warps (of a CTA that may hold several groups).
__device__ __forceinline__ void group_sync(int group, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
}

__device__ __forceinline__ float param(const void* p, int type, int h) {
  return type == MEP_F32 ? __ldg(static_cast<const float*>(p) + h)
                         : to_f32(static_cast<const __nv_bfloat16*>(p)[h]);
}
// Eight parameters of a block; `none` without the tensor, 0 beyond H.
template <bool VEC>
__device__ __forceinline__ void load_params(const void* p, int type, int H, int block, int l,
                                            float none, float (&v)[8]) {
  if (p == nullptr) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = none;
  } else if (VEC && type == MEP_F32) {
    Pack<MEP_F32> q;
    q.load<true>(p, 0, H, block, l);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = q.get(j);
  } else if (VEC) {
    Pack<MEP_BF16> q;
    q.load<true>(p, 0, H, block, l);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = q.get(j);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int h = half_col<false>(block, l, j);
      v[j] = h < H ? param(p, type, h) : 0.f;
    }
  }
}

// Sum of v over the W warps of a group; s holds W words, not in use elsewhere
// before the next barrier of the group.
__device__ __forceinline__ float group_sum(float v, float* s, int W, int warp, int group) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(MEP_FULL_MASK, v, d);
  if (W == 1) return v;
  if (lane == 0) s[warp] = v;
  group_sync(group, 32 * W);
  v = lane < W ? s[lane] : 0.f;
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(MEP_FULL_MASK, v, d);
  return v;
}

// J blocks a half warp, W warps a row: 2 J W >= blocks of a row.
template <typename T, int KIND, bool VEC, int J>
__global__ void __launch_bounds__(32 * kMaxWarps / (J > 2 ? 2 : 1))
    k_norm(const T* __restrict__ x, const void* __restrict__ w, const void* __restrict__ b, int p_type,
           float eps, long long N, int H, int W, T* __restrict__ y, float* __restrict__ mean,
           float* __restrict__ rstd, uint8_t* __restrict__ x_ckpt, uint8_t* __restrict__ y_ckpt) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float s_sum[4][kMaxWarps];  // [mean and square, twice][warps of all groups]
  const int l = threadIdx.x % kHalf;
  const int group = (threadIdx.x >> 5) / W, groups = blockDim.x / (32 * W);
  const int warp = (threadIdx.x >> 5) - group * W, half = 2 * warp + ((threadIdx.x >> 4) & 1);
  const int nb = (H + kCkptBlock - 1) / kCkptBlock;
  const float inv_h = 1.f / H;
  int turn = 0;
  for (long long r = (long long)blockIdx.x * groups + group; r < N;
       r += (long long)gridDim.x * groups, turn ^= 2) {
    Pack<KIND> p[J];
#pragma unroll
    for (int i = 0; i < J; ++i) p[i].template load<VEC>(x, r, H, half + 2 * W * i, l);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < J; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += p[i].get(j);
    const float m = group_sum(sum, &s_sum[turn][group * W], W, warp, group) * inv_h;
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < J; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float c = half_col<VEC>(half + 2 * W * i, l, j) < H ? p[i].get(j) - m : 0.f;
        sq = fmaf(c, c, sq);
      }
    const float rs = 1.f / sqrtf(group_sum(sq, &s_sum[turn + 1][group * W], W, warp, group) * inv_h + eps);
    if (warp == 0 && (threadIdx.x & 31) == 0) {
      mean[r] = m;
      rstd[r] = rs;
    }
#pragma unroll
    for (int i = 0; i < J; ++i) {
      const int block = half + 2 * W * i;
      const bool in = block < nb;
      float v[8], wv[8], bv[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = p[i].get(j);
      if (x_ckpt != nullptr) save8<VEC>(x_ckpt, r, H, block, l, in, v);
      load_params<VEC>(w, p_type, H, block, l, 1.f, wv);
      load_params<VEC>(b, p_type, H, block, l, 0.f, bv);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = half_col<VEC>(block, l, j) < H ? fmaf((v[j] - m) * rs, wv[j], bv[j]) : 0.f;
      store8<T, VEC>(y, r, H, block, l, v);
      if (y_ckpt != nullptr) save8<VEC>(y_ckpt, r, H, block, l, in, v);
    }
  }
}

// Sums over a group of 2U values a thread, two for each of U rows: the lanes
// first share the values out among themselves (each step halves the values a
// lane still carries), so that a warp needs 2U + 5 - log2(2U) - 1 shuffles
// and not 10U.
template <int U>
__device__ __forceinline__ void group_sums(float (&v)[2 * U], float* s, int W, int warp, int group) {
  constexpr int n = 2 * U;
  const int lane = threadIdx.x & 31;
  int d = 16;
#pragma unroll
  for (int k = n / 2; k >= 1; k >>= 1, d >>= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int i = 0; i < k; ++i) {
      const float give = up ? v[i] : v[i + k], keep = up ? v[i + k] : v[i];
      v[i] = keep + __shfl_xor_sync(MEP_FULL_MASK, give, d);
    }
  }
  float t = v[0];  // of value `mine`, over the lanes that share d's remaining bits
  for (; d >= 1; d >>= 1) t += __shfl_xor_sync(MEP_FULL_MASK, t, d);
  // lane bits 4, 3, ... choose the value, high bit first
  const int mine = lane / (32 / n);
  if (W > 1) {
    if (lane % (32 / n) == 0) s[warp * n + mine] = t;
    group_sync(group, 32 * W);
    t = 0.f;
    for (int k = lane % (32 / n); k < W; k += 32 / n) t += s[k * n + mine];
#pragma unroll
    for (int e = 16 / n; e >= 1; e >>= 1) t += __shfl_xor_sync(MEP_FULL_MASK, t, e);
  }
#pragma unroll
  for (int i = 0; i < n; ++i) v[i] = __shfl_sync(MEP_FULL_MASK, t, i * (32 / n));
}

template <typename T, int KIND, int XKIND, bool VEC, int J, int U>
__global__ void __launch_bounds__(U == 4 ? 512 : 1024)
    k_norm_dx(const T* __restrict__ dy, const void* __restrict__ x, const void* __restrict__ w,
              int p_type, const float* __restrict__ mean, const float* __restrict__ rstd, long long N,
              int H, int W, T* __restrict__ dx, float* __restrict__ ws) {
  pdl_wait();
  pdl_launch_dependents();
  extern __shared__ float s_part[];                   // [groups][2][columns of a group]
  __shared__ float s_sum[2][kMaxWarps * 2 * U];
  const int l = threadIdx.x % kHalf;
  const int group = (threadIdx.x >> 5) / W, groups = blockDim.x / (32 * W);
  const int warp = (threadIdx.x >> 5) - group * W, half = 2 * warp + ((threadIdx.x >> 4) & 1);
  const float inv_h = 1.f / H;
  float dw[J][8], db[J][8], wv[J][8];
#pragma unroll
  for (int i = 0; i < J; ++i) {
    load_params<VEC>(w, p_type, H, half + 2 * W * i, l, 1.f, wv[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = db[i][j] = 0.f;
  }
  int turn = 0;
  for (long long r0 = ((long long)blockIdx.x * groups + group) * U; r0 < N;
       r0 += (long long)gridDim.x * groups * U, turn ^= 1) {
    Pack<KIND> d[U][J];
    Pack<XKIND> p[U][J];
    float m[U], rs[U], sums[2 * U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = r0 + u < N;
#pragma unroll
      for (int i = 0; i < J; ++i) {
        if (in) {
          d[u][i].template load<VEC>(dy, r0 + u, H, half + 2 * W * i, l);
          p[u][i].template load<VEC>(x, r0 + u, H, half + 2 * W * i, l);
        } else {
          d[u][i].clear();
          p[u][i].clear();
        }
      }
      m[u] = in ? __ldg(mean + r0 + u) : 0.f;
      rs[u] = in ? __ldg(rstd + r0 + u) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int i = 0; i < J; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float g = d[u][i].get(j);
          const float xhat = (p[u][i].get(j) - m[u]) * rs[u], t = g * wv[i][j];
          s1 += t;
          s2 = fmaf(t, xhat, s2);
          dw[i][j] = fmaf(g, xhat, dw[i][j]);
          db[i][j] += g;
        }
      sums[u] = s1;
      sums[U + u] = s2;
    }
    group_sums<U>(sums, &s_sum[turn][group * W * 2 * U], W, warp, group);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float c1 = sums[u] * inv_h, c2 = sums[U + u] * inv_h;
      if (r0 + u < N) {
#pragma unroll
        for (int i = 0; i < J; ++i) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float xhat = (p[u][i].get(j) - m[u]) * rs[u];
            v[j] = rs[u] * (fmaf(d[u][i].get(j), wv[i][j], -c1) - xhat * c2);
          }
          store8<T, VEC>(dx, r0 + u, H, half + 2 * W * i, l, v);
        }
      }
    }
  }
  if (ws == nullptr) return;
  // join the groups' column sums: laid out by thread, then by value
  const int tid = threadIdx.x - group * 32 * W, threads = 32 * W, cols = threads * 8 * J;
  if (groups > 1) {
#pragma unroll
    for (int i = 0; i < J; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s_part[(2 * group) * cols + (8 * i + j) * threads + tid] = dw[i][j];
        s_part[(2 * group + 1) * cols + (8 * i + j) * threads + tid] = db[i][j];
      }
    __syncthreads();
    if (group != 0) return;
    for (int g = 1; g < groups; ++g)
#pragma unroll
      for (int i = 0; i < J; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dw[i][j] += s_part[(2 * g) * cols + (8 * i + j) * threads + tid];
          db[i][j] += s_part[(2 * g + 1) * cols + (8 * i + j) * threads + tid];
        }
  }
  float* out = ws + (long long)blockIdx.x * 2 * H;
#pragma unroll
  for (int i = 0; i < J; ++i) {
    store8<float, VEC>(out, 0, H, half + 2 * W * i, l, dw[i]);
    store8<float, VEC>(out + H, 0, H, half + 2 * W * i, l, db[i]);
  }
}

// 32 columns of one of the two sums per CTA; warp k adds parts k, k + 32, ...
__global__ void __launch_bounds__(1024)
    k_norm_dw(const float* __restrict__ ws, int H, int parts, int accumulate,
              float* __restrict__ dweight, float* __restrict__ dbias) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float s[32][33];
  float* out = blockIdx.y == 0 ? dweight : dbias;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5, h = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (h < H)
#pragma unroll 4
    for (int p = k; p < parts; p += 32) v += ws[((long long)2 * p + blockIdx.y) * H + h];
  s[k][lane] = v;
  __syncthreads();
  v = s[lane][k];
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(MEP_FULL_MASK, v, d);
  const int c = blockIdx.x * 32 + k;
  if (lane == 0 && c < H) out[c] = accumulate ? out[c] + v : v;
}

// ---------------------------------------------------------------------------
int norm_check(int type, int64_t N, int64_t H, int p_type) {
  if (type != MEP_BF16 && type != MEP_F32) return MEP_ERR_INVALID_ARG;
  if (p_type != MEP_BF16 && p_type != MEP_F32) return MEP_ERR_INVALID_ARG;
  if (N < 0 || N > 0x7fffffffLL || H < 1 || H > kMaxH) return MEP_ERR_INVALID_ARG;
  return MEP_OK;
}

int ceil_div(long long a, long long b) { return int((a + b - 1) / b); }

// How the backward pass lays a row out: J blocks a half warp, W warps a row,
// U rows at a time, `groups` rows' worth of warps in a CTA.
struct Shape {
  int J, U, W, groups, parts;
};
Shape backward_shape(long long N, int H, int type) {
  Shape s;
  const int nb = ceil_div(H, kCkptBlock);
  s.J = nb > 64 ? 2 : 1;
  s.U = s.J == 2 ? 1 : (type == MEP_F32 ? 2 : 4);
  if (nb > 32 && s.U > 2) s.U = 2;
  s.W = ceil_div(nb, 2 * s.J);
  s.groups = s.W >= 4 ? 1 : 8 / s.W;
  const int want = ceil_div(N < 1 ? 1 : N, s.U * s.groups);
  const int warps = s.W * s.groups, cap = 152 * (warps > 16 ? 1 : warps > 8 ? 2 : 4);
  s.parts = want < cap ? want : cap;
  return s;
}

template <typename T, int KIND, bool VEC, int J>
cudaError_t run_norm(const void* x, const void* w, const void* b, int p_type, float eps, long long N,
                     int H, void* y, float* mean, float* rstd, uint8_t* xc, uint8_t* yc,
                     cudaStream_t st) {
  const int W = ceil_div(ceil_div(H, kCkptBlock), 2 * J), groups = W >= 4 ? 1 : 4 / W;
  const int want = ceil_div(N, groups), cap = sm_count() * (64 / (W * groups));
  return launch_pdl(k_norm<T, KIND, VEC, J>, dim3(want < cap ? want : cap), dim3(32 * W * groups), 0, st,
                    static_cast<const T*>(x), w, b, p_type, eps, N, H, W, static_cast<T*>(y), mean, rstd,
                    xc, yc);
}

template <typename T, int KIND, bool VEC>
cudaError_t pick_norm(const void* x, const void* w, const void* b, int p_type, float eps, long long N,
                      int H, void* y, float* mean, float* rstd, uint8_t* xc, uint8_t* yc,
                      cudaStream_t st) {
  const auto run = H <= 2 * kCkptBlock   ? run_norm<T, KIND, VEC, 1>
                   : H <= 4 * kCkptBlock ? run_norm<T, KIND, VEC, 2>
                                         : run_norm<T, KIND, VEC, 4>;
  return run(x, w, b, p_type, eps, N, H, y, mean, rstd, xc, yc, st);
}

template <typename T, int KIND, int XKIND, bool VEC, int J, int U>
cudaError_t run_dx(const Shape& s, const void* dy, const void* x, const void* w, int p_type,
                   const float* mean, const float* rstd, long long N, int H, void* dx, float* ws,
                   cudaStream_t st) {
  const int threads = 32 * s.W * s.groups;
  const int smem = s.groups > 1 ? s.groups * 2 * 32 * s.W * 8 * J * 4 : 0;
  const auto kernel = k_norm_dx<T, KIND, XKIND, VEC, J, U>;
  if (set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), smem)) return cudaErrorInvalidValue;
  return launch_pdl(kernel, dim3(s.parts), dim3(threads), smem, st, static_cast<const T*>(dy), x, w,
                    p_type, mean, rstd, N, H, s.W, static_cast<T*>(dx), ws);
}

template <typename T, int KIND, int XKIND, bool VEC>
cudaError_t pick_dx(const Shape& s, const void* dy, const void* x, const void* w, int p_type,
                    const float* mean, const float* rstd, long long N, int H, void* dx, float* ws,
                    cudaStream_t st) {
  const auto run = s.J == 2   ? run_dx<T, KIND, XKIND, VEC, 2, 1>
                   : s.U == 2 ? run_dx<T, KIND, XKIND, VEC, 1, 2>
                              : run_dx<T, KIND, XKIND, VEC, 1, 4>;
  return run(s, dy, x, w, p_type, mean, rstd, N, H, dx, ws, st);
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
  const bool vec = H % 8 == 0;
  const auto run = x_type == MEP_BF16
                       ? (vec ? pick_norm<__nv_bfloat16, MEP_BF16, true> : pick_norm<__nv_bfloat16, MEP_BF16, false>)
                       : (vec ? pick_norm<float, MEP_F32, true> : pick_norm<float, MEP_F32, false>);
  const cudaError_t err = run(x, weight, bias, p_type, eps, N, int(H), y, mean, rstd, x_ckpt, y_ckpt,
                              static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? MEP_OK : MEP_ERR_CUDA;
}

extern "C" int mep_layer_norm_backward_workspace_bytes(int64_t N, int64_t H, size_t* bytes) {
  if (bytes == nullptr || norm_check(MEP_F32, N, H, MEP_F32) != MEP_OK) return MEP_ERR_INVALID_ARG;
  const int a = backward_shape(N, int(H), MEP_BF16).parts, b = backward_shape(N, int(H), MEP_F32).parts;
  *bytes = size_t(a > b ? a : b) * 2 * H * sizeof(float);
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
  const bool params = dweight != nullptr || dbias != nullptr;
  if (params && (ws == nullptr || ws_bytes < need)) return MEP_ERR_INVALID_ARG;
  for (const void* p : {dy, x, weight, static_cast<const void*>(mean), static_cast<const void*>(rstd),
                        static_cast<const void*>(ws), static_cast<const void*>(dx),
                        static_cast<const void*>(dweight), static_cast<const void*>(dbias)})
    if (!aligned16(p)) return MEP_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Shape s = backward_shape(N, int(H), dy_type);
  float* part = params ? static_cast<float*>(ws) : nullptr;
  const bool vec = H % 8 == 0, kept = x_type == MEP_CKPT8;
  if (N > 0) {
    const auto run =
        dy_type == MEP_BF16
            ? (kept ? (vec ? pick_dx<__nv_bfloat16, MEP_BF16, MEP_CKPT8, true>
                           : pick_dx<__nv_bfloat16, MEP_BF16, MEP_CKPT8, false>)
                    : (vec ? pick_dx<__nv_bfloat16, MEP_BF16, MEP_BF16, true>
                           : pick_dx<__nv_bfloat16, MEP_BF16, MEP_BF16, false>))
            : (kept ? (vec ? pick_dx<float, MEP_F32, MEP_CKPT8, true> : pick_dx<float, MEP_F32, MEP_CKPT8, false>)
                    : (vec ? pick_dx<float, MEP_F32, MEP_F32, true> : pick_dx<float, MEP_F32, MEP_F32, false>));
    if (run(s, dy, x, weight, p_type, mean, rstd, N, int(H), dx, part, st) != cudaSuccess) return MEP_ERR_CUDA;
  }
  if (!params) return MEP_OK;
  const cudaError_t err = launch_pdl(k_norm_dw, dim3(ceil_div(H, 32), 2), dim3(1024), 0, st,
                                     static_cast<const float*>(ws), int(H), N > 0 ? s.parts : 0, accumulate,
                                     dweight, dbias);
  return err == cudaSuccess ? MEP_OK : MEP_ERR_CUDA;
}
