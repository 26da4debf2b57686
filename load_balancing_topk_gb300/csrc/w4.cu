// w4.cu -- weight matrices to 4 bits and back (mep_w4_save, mep_w4_load).
//
// A warp holds 16 columns of a block, a lane columns g and g + 8 at the rows
// whose pairs it writes (w4.cuh): 32 rows, of which every group has its share
// in each of the four lanes t, so that a group's largest magnitude is two
// shuffles away. q = w / s is a division, as the format is defined by it; the
// scale itself is a product by fp32's 1/7.

#include "ckpt.cuh"
#include "w4.cuh"

namespace mep {
namespace {

constexpr int kThreads = 128;  // a warp for each 16 columns of a block

struct Matrices {
  long long K, N;   // of a part
  int parts, kb;    // parts of a matrix; blocks of a panel
  long long panels; // of a part
};

// Block number -> where its values lie: part p of matrix m, first row and column.
struct At {
  long long base, k0, n0, ld;  // element of (row 0, column 0) of the part; row pitch
};
__device__ __forceinline__ At at_block(const Matrices& s, long long b) {
  const long long kb = b % s.kb, panel = b / s.kb % s.panels, mp = b / s.kb / s.panels;
  const long long m = mp / s.parts, p = mp % s.parts;
  At a;
  a.ld = s.N * s.parts;
  a.base = m * s.K * a.ld + p * s.N;
  a.k0 = kb * kW4Rows;
  a.n0 = panel * kW4Cols;
  return a;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_w4_save(const T* __restrict__ w, Matrices s, int group,
                                                      uint8_t* __restrict__ w4) {
  pdl_launch_dependents();
  pdl_wait();
  const At a = at_block(s, blockIdx.x);
  const int c = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint8_t* out = w4 + (long long)blockIdx.x * w4_block_bytes(group);
  float v[2][4][4][2];  // h, j, (i, e), l
  float top[4][2];      // of 32 rows: h, j / 2
#pragma unroll
  for (int q = 0; q < 4; ++q) top[q][0] = top[q][1] = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int l = 0; l < 2; ++l) {
          const long long k = a.k0 + 64 * h + 16 * j + 8 * (r & 1) + 2 * t + (r >> 1);
          const long long n = a.n0 + 16 * c + 8 * l + g;
          const float x = k < s.K && n < s.N ? to_f32(w[a.base + k * a.ld + n]) : 0.f;
          v[h][j][r][l] = x;
          float& m = top[2 * h + j / 2][l];
          // the larger magnitude, as bits: an infinity and then a NaN above all numbers
          m = __uint_as_float(max(__float_as_uint(m), __float_as_uint(x) & 0x7fffffffu));
        }
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int l = 0; l < 2; ++l) {
      uint32_t m = __float_as_uint(top[q][l]);
      m = max(m, __shfl_xor_sync(MEP_FULL_MASK, m, 1));
      m = max(m, __shfl_xor_sync(MEP_FULL_MASK, m, 2));
      top[q][l] = __uint_as_float(m);
    }
  float scale[4][2];
#pragma unroll
  for (int l = 0; l < 2; ++l) {
    uint32_t m[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) m[q] = __float_as_uint(top[q][l]);
    if (group >= 64) m[0] = m[1] = max(m[0], m[1]), m[2] = m[3] = max(m[2], m[3]);
    if (group >= 128) m[0] = m[1] = m[2] = m[3] = max(m[0], m[2]);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      scale[q][l] = m[q] >= 0x7f800000u ? __uint_as_float(0x7fc00000u)
                                        : __bfloat162float(__float2bfloat16_rn(__uint_as_float(m[q]) * (1.f / kW4Top)));
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t word[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      word[j] = 0;
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int l = 0; l < 2; ++l) {
          const float sc = scale[2 * h + j / 2][l];
          const float q = sc > 0.f ? rintf(v[h][j][r][l] / sc) : 0.f;
          word[j] |= (uint32_t)(int(fminf(fmaxf(q, -kW4Top), kW4Top)) + 8) << (8 * r + 4 * l);
        }
    }
    reinterpret_cast<uint4*>(out)[((h * 4 + c) * 8 + g) * 4 + t] = make_uint4(word[0], word[1], word[2], word[3]);
  }
  if (t < kW4Rows / group) {
    __nv_bfloat162 pair;
    const int q = t * (group / 32);
    pair.x = __float2bfloat16_rn(q == 0 ? scale[0][0] : q == 1 ? scale[1][0] : q == 2 ? scale[2][0] : scale[3][0]);
    pair.y = __float2bfloat16_rn(q == 0 ? scale[0][1] : q == 1 ? scale[1][1] : q == 2 ? scale[2][1] : scale[3][1]);
    reinterpret_cast<__nv_bfloat162*>(out + kW4Pairs)[t * 32 + c * 8 + g] = pair;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_w4_load(const uint8_t* __restrict__ w4, Matrices s, int group,
                                                      T* __restrict__ w) {
  pdl_launch_dependents();
  pdl_wait();
  const At a = at_block(s, blockIdx.x);
  const int c = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint8_t* in = w4 + (long long)blockIdx.x * w4_block_bytes(group);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 q4 = reinterpret_cast<const uint4*>(in)[((h * 4 + c) * 8 + g) * 4 + t];
    const uint32_t word[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 sc =
          reinterpret_cast<const __nv_bfloat162*>(in + kW4Pairs)[(64 * h + 16 * j) / group * 32 + c * 8 + g];
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int l = 0; l < 2; ++l) {
          const long long k = a.k0 + 64 * h + 16 * j + 8 * (r & 1) + 2 * t + (r >> 1);
          const long long n = a.n0 + 16 * c + 8 * l + g;
          const float q = float(int(word[j] >> (8 * r + 4 * l) & 15u) - 8);
          if (k < s.K && n < s.N) w[a.base + k * a.ld + n] = from_f32<T>(q * __bfloat162float(l ? sc.y : sc.x));
        }
    }
  }
}

int w4_check(const void* w, int type, int64_t M, int64_t K, int64_t N, int parts, int group, const void* w4,
             Matrices* s, long long* blocks) {
  if ((type != MEP_BF16 && type != MEP_F32) || M < 0 || parts < 1 || N < 1 || N % parts != 0 ||
      !w4_sizes_ok(K, N / parts, group))
    return MEP_ERR_INVALID_ARG;
  if (M > 0x7fffffffLL || M * parts > 0x7fffffffLL) return MEP_ERR_INVALID_ARG;
  s->K = K, s->N = N / parts, s->parts = parts;
  s->kb = int((K + kW4Rows - 1) / kW4Rows), s->panels = (s->N + kW4Cols - 1) / kW4Cols;
  if (M * parts > (1LL << 46) / ((long long)s->kb * s->panels)) return MEP_ERR_INVALID_ARG;
  *blocks = M * parts * s->kb * s->panels;
  if (M == 0) return MEP_OK;
  if (w == nullptr || w4 == nullptr || !aligned16(w4) ||
      reinterpret_cast<uintptr_t>(w) % (type == MEP_BF16 ? 2 : 4) != 0)
    return MEP_ERR_INVALID_ARG;
  return MEP_OK;
}

}  // namespace
}  // namespace mep

using namespace mep;

extern "C" int mep_w4_bytes(int64_t K, int64_t N, int group, size_t* bytes) {
  if (bytes == nullptr || !w4_sizes_ok(K, N, group)) return MEP_ERR_INVALID_ARG;
  *bytes = (size_t)w4_matrix_bytes(K, N, group);
  return MEP_OK;
}

extern "C" int mep_w4_save(const void* w, int w_type, int64_t M, int64_t K, int64_t N, int parts, int group,
                           uint8_t* w4, void* stream) {
  Matrices s;
  long long blocks = 0;
  const int rc = w4_check(w, w_type, M, K, N, parts, group, w4, &s, &blocks);
  if (rc != MEP_OK || blocks == 0) return rc;
  if (blocks > 0x7fffffffLL) return MEP_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      w_type == MEP_BF16
          ? launch_pdl(k_w4_save<__nv_bfloat16>, dim3(unsigned(blocks)), dim3(kThreads), 0, st,
                       static_cast<const __nv_bfloat16*>(w), s, group, w4)
          : launch_pdl(k_w4_save<float>, dim3(unsigned(blocks)), dim3(kThreads), 0, st, static_cast<const float*>(w), s,
                       group, w4);
  return e == cudaSuccess ? MEP_OK : MEP_ERR_CUDA;
}

extern "C" int mep_w4_load(const uint8_t* w4, int64_t M, int64_t K, int64_t N, int parts, int group, int w_type,
                           void* w, void* stream) {
  Matrices s;
  long long blocks = 0;
  const int rc = w4_check(w, w_type, M, K, N, parts, group, w4, &s, &blocks);
  if (rc != MEP_OK || blocks == 0) return rc;
  if (blocks > 0x7fffffffLL) return MEP_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      w_type == MEP_BF16
          ? launch_pdl(k_w4_load<__nv_bfloat16>, dim3(unsigned(blocks)), dim3(kThreads), 0, st, w4, s, group,
                       static_cast<__nv_bfloat16*>(w))
          : launch_pdl(k_w4_load<float>, dim3(unsigned(blocks)), dim3(kThreads), 0, st, w4, s, group,
                       static_cast<float*>(w));
  return e == cudaSuccess ? MEP_OK : MEP_ERR_CUDA;
}
