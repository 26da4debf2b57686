// grouped_wgrad.cu -- the experts' weight gradients over the static buffer
// (mep_grouped_wgrad).
//
// Source: "月之暗面开源MoonEP：面向MoE训练的专家并行通信库", section
// 内存契约与权重布局: the weights of one projection are one [E+B, H, H']
// tensor, gradients are fp32, those of the prefetch slots lie in a buffer of
// their own seen as [R, B, H, H'], which mep_reduce_grad folds into the home
// experts' gradients.

#include "ckpt.cuh"

namespace mep {
namespace {

constexpr int kT = 64;   // tile edge
constexpr int kRows = 16;

__global__ void __launch_bounds__(1024)
    k_wgrad_check(const int32_t* __restrict__ cu, int R, int G, int SK, int32_t* status, int* ok) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ int s_bad;
  if (threadIdx.x == 0) s_bad = read_status(status) != 0 ? 2 : 0;
  __syncthreads();
  for (long long p = threadIdx.x; p < (long long)R * G; p += blockDim.x) {
    const int j = int(p % G), v = cu[p], prev = j == 0 ? 0 : cu[p - 1];
    if (v < prev || (j == G - 1 && v != SK)) s_bad = s_bad | 1;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    *ok = s_bad == 0;
    if (s_bad == 1) set_status(status, MEP_ERR_BAD_SEQLENS);
  }
}

template <bool CKPT>
__device__ __forceinline__ float load_x(const void* x, long long r, int h, int H) {
  if (!CKPT) return to_f32(static_cast<const __nv_bfloat16*>(x)[r * H + h]);
  const uint8_t* row = static_cast<const uint8_t*>(x) + r * ckpt_row_bytes(H);
  return float(int8_t(row[h])) * ckpt_step(row[ckpt_scale_at(H) + h / kCkptBlock]);
}

// One CTA per (weight row, 64 x 64 tile): 16 x 16 threads with 4 x 4 sums
// each, 16 rows of x and dy at a time in shared memory.
template <bool CKPT>
__global__ void __launch_bounds__(256)
    k_wgrad(const void* __restrict__ x, const __nv_bfloat16* __restrict__ dy,
            const int32_t* __restrict__ cu, const int* __restrict__ ok, int R, int SK, int E, int B,
            int H, int Hp, int accumulate, float* __restrict__ home, float* __restrict__ slot) {
  pdl_wait();
  pdl_launch_dependents();
  if (*ok == 0) return;
  __shared__ float sx[kRows][kT], sd[kRows][kT];
  const int G = E + B, wrow = blockIdx.z, h0 = blockIdx.y * kT, n0 = blockIdx.x * kT;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const bool is_home = wrow < E;
  const int r0 = is_home ? 0 : (wrow - E) / B, r1 = is_home ? R : r0 + 1;
  const int j = is_home ? wrow : E + (wrow - E) % B;
  float acc[4][4] = {};
  bool any = false;
  for (int r = r0; r < r1; ++r) {
    const int lo = j == 0 ? 0 : cu[r * G + j - 1], hi = cu[r * G + j];
    for (int k0 = lo; k0 < hi; k0 += kRows) {
      any = true;
      for (int i = threadIdx.x; i < kRows * kT; i += 256) {
        const int k = i / kT, c = i % kT;
        const bool in = k0 + k < hi;
        const long long row = (long long)r * SK + k0 + k;
        sx[k][c] = in && h0 + c < H ? load_x<CKPT>(x, row, h0 + c, H) : 0.f;
        sd[k][c] = in && n0 + c < Hp ? to_f32(dy[row * Hp + n0 + c]) : 0.f;
      }
      __syncthreads();
      for (int k = 0; k < kRows; ++k)
        for (int a = 0; a < 4; ++a)
          for (int b = 0; b < 4; ++b) acc[a][b] += sx[k][ty + 16 * a] * sd[k][tx + 16 * b];
      __syncthreads();
    }
  }
  if (!any && (accumulate || !is_home)) return;
  float* out = is_home ? home + (long long)wrow * H * Hp : slot + (long long)(wrow - E) * H * Hp;
  for (int a = 0; a < 4; ++a)
    for (int b = 0; b < 4; ++b) {
      const int h = h0 + ty + 16 * a, n = n0 + tx + 16 * b;
      if (h < H && n < Hp) {
        float* o = out + (long long)h * Hp + n;
        *o = accumulate ? *o + acc[a][b] : acc[a][b];
      }
    }
}

}  // namespace
}  // namespace mep

using namespace mep;

extern "C" int mep_grouped_wgrad_workspace_bytes(int R, int S, int K, int E, int B, size_t* bytes) {
  if (bytes == nullptr || R < 1 || S < 0 || K < 1 || E < 1 || B < 0) return MEP_ERR_INVALID_ARG;
  if (R > MEP_MAX_R || E > MEP_MAX_E || K > MEP_MAX_K || (long long)R * B > MEP_MAX_SLOTS)
    return MEP_ERR_INVALID_ARG;
  *bytes = 16;
  return MEP_OK;
}

extern "C" int mep_grouped_wgrad(const void* x, int x_type, const mep_bf16* dy,
                                 const int32_t* cu_seqlens, int32_t* status, int R, int S, int K,
                                 int E, int B, int H, int Hp, int accumulate, void* ws,
                                 size_t ws_bytes, float* home_grad, float* slot_grad, void* stream) {
  size_t need = 0;
  if (mep_grouped_wgrad_workspace_bytes(R, S, K, E, B, &need) != MEP_OK) return MEP_ERR_INVALID_ARG;
  if (x_type != MEP_BF16 && x_type != MEP_CKPT8) return MEP_ERR_INVALID_ARG;
  if (H < 8 || H % 8 != 0 || Hp < 8 || Hp % 8 != 0) return MEP_ERR_INVALID_ARG;
  const long long SK = (long long)S * K, rows = (long long)R * SK;
  if (rows > 0x7fffff00LL) return MEP_ERR_INVALID_ARG;
  if (cu_seqlens == nullptr || home_grad == nullptr || ws == nullptr || ws_bytes < need ||
      (B > 0 && slot_grad == nullptr) || (rows > 0 && (x == nullptr || dy == nullptr)))
    return MEP_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(dy) || !aligned16(home_grad) || !aligned16(slot_grad) || !aligned16(ws))
    return MEP_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int* ok = static_cast<int*>(ws);
  cudaError_t err = launch_pdl(k_wgrad_check, dim3(1), dim3(1024), 0, st, cu_seqlens, R, E + B,
                               int(SK), status, ok);
  if (err != cudaSuccess) return MEP_ERR_CUDA;
  const dim3 grid((Hp + kT - 1) / kT, (H + kT - 1) / kT, E + R * B);
  const __nv_bfloat16* d = reinterpret_cast<const __nv_bfloat16*>(dy);
  err = x_type == MEP_CKPT8 ? launch_pdl(k_wgrad<true>, grid, dim3(256), 0, st, x, d, cu_seqlens, ok, R,
                                         int(SK), E, B, H, Hp, accumulate, home_grad, slot_grad)
                            : launch_pdl(k_wgrad<false>, grid, dim3(256), 0, st, x, d, cu_seqlens, ok, R,
                                         int(SK), E, B, H, Hp, accumulate, home_grad, slot_grad);
  return err == cudaSuccess ? MEP_OK : MEP_ERR_CUDA;
}
