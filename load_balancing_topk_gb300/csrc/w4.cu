// w4.cu -- weight matrices to 4 bits and back (mep_w4_save, mep_w4_load).
//
// One pass over memory, a CTA a block of 128 rows and 64 columns, which goes
// through shared memory: rows outside in 16-byte vectors, inside the 32 rows of
// two columns that a lane's pairs are of (w4.cuh). A warp holds 16 columns; a
// group has its share in each of the four lanes t, so that its largest magnitude
// is two shuffles away. Rows that do not start on 16-byte boundaries are read and
// written element by element, coalesced over a row's 64 columns.
// q = w / s is a division, as the format is defined by it. From bf16 it is a
// product by 1 / s and a correction by the remainder, which two fused
// multiply-adds give: the quotient of two numbers of eight bits is 2^-9 or more
// from every half step unless it is one, and one it meets exactly. (Scales below
// 2^-100, whose reciprocal leaves fp32, divide.) Adding 1.5 * 2^23 + 8 rounds to
// a whole number, ties to even, and leaves q + 8 in the low bits.

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
  long long base;  // element of the block's first row and column
  long long ld;    // row pitch
  int rows, cols;  // that there are
};
__device__ __forceinline__ At at_block(const Matrices& s, uint32_t b) {
  const uint32_t panel_all = b / uint32_t(s.kb), kb = b - panel_all * s.kb;
  const uint32_t mp = panel_all / uint32_t(s.panels), panel = panel_all - mp * uint32_t(s.panels);
  const uint32_t m = mp / uint32_t(s.parts), p = mp - m * s.parts;
  At a;
  a.ld = s.N * s.parts;
  const long long k0 = (long long)kb * kW4Rows, n0 = (long long)panel * kW4Cols;
  a.base = (m * s.K + k0) * a.ld + p * s.N + n0;
  a.rows = int(min((long long)kW4Rows, s.K - k0)), a.cols = int(min((long long)kW4Cols, s.N - n0));
  return a;
}
// A block's values in shared memory: a row's pitch in elements, which puts the
// four rows and eight columns of a warp's access into different banks.
template <typename T> constexpr int kPitch = sizeof(T) == 2 ? 72 : 68;

// A block's rows into shared memory, zeros where there are none.
template <typename T, bool VEC> __device__ __forceinline__ void rows_in(const T* __restrict__ w, const At& a, T* tile) {
  constexpr int V = VEC ? 16 / sizeof(T) : 1, per_row = kW4Cols / V;
  if (VEC) {
    uint4 v[kW4Rows * per_row / kThreads];
#pragma unroll
    for (int i = 0; i < kW4Rows * per_row / kThreads; ++i) {
      const int q = i * kThreads + threadIdx.x, r = q / per_row, c = q % per_row * V;
      v[i] = r < a.rows && c < a.cols ? __ldg(reinterpret_cast<const uint4*>(w + a.base + r * a.ld + c)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kW4Rows * per_row / kThreads; ++i) {
      const int q = i * kThreads + threadIdx.x;
      *reinterpret_cast<uint4*>(tile + q / per_row * kPitch<T> + q % per_row * V) = v[i];
    }
  } else {
#pragma unroll 16
    for (int q = threadIdx.x; q < kW4Rows * kW4Cols; q += kThreads) {
      const int r = q / kW4Cols, c = q % kW4Cols;
      tile[r * kPitch<T> + c] = r < a.rows && c < a.cols ? w[a.base + r * a.ld + c] : from_f32<T>(0.f);
    }
  }
}
template <typename T, bool VEC> __device__ __forceinline__ void rows_out(const T* tile, const At& a, T* __restrict__ w) {
  constexpr int V = VEC ? 16 / sizeof(T) : 1, per_row = kW4Cols / V;
#pragma unroll 8
  for (int q = threadIdx.x; q < kW4Rows * per_row; q += kThreads) {
    const int r = q / per_row, c = q % per_row * V;
    if (r < a.rows && c < a.cols) {
      if (VEC)
        __stcs(reinterpret_cast<uint4*>(w + a.base + r * a.ld + c), *reinterpret_cast<const uint4*>(tile + r * kPitch<T> + c));
      else
        w[a.base + r * a.ld + c] = tile[r * kPitch<T> + c];
    }
  }
}
// Row of the block that pair (i, e) of word j of half h has in lane t.
__device__ __forceinline__ constexpr int row_of(int h, int j, int r, int t) { return 64 * h + 16 * j + 8 * (r & 1) + 2 * t + (r >> 1); }

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) k_w4_save(const T* __restrict__ w, Matrices s, int group,
                                                      uint8_t* __restrict__ w4) {
  __shared__ __align__(16) T tile[kW4Rows * kPitch<T>];
  pdl_launch_dependents();
  pdl_wait();
  const At a = at_block(s, blockIdx.x);
  rows_in<T, VEC>(w, a, tile);
  __syncthreads();
  const int c = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint8_t* out = w4 + (long long)blockIdx.x * w4_block_bytes(group);
  const T* mine = tile + 16 * c + g;
  // the larger magnitude, as bits: an infinity and then a NaN above all numbers
  uint32_t top[4][2] = {};  // of 32 rows
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int l = 0; l < 2; ++l) {
          const float x = to_f32(mine[row_of(h, j, r, t) * kPitch<T> + 8 * l]);
          top[2 * h + j / 2][l] = max(top[2 * h + j / 2][l], __float_as_uint(x) & 0x7fffffffu);
        }
  float scale[4][2];
#pragma unroll
  for (int l = 0; l < 2; ++l) {
    uint32_t m[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      m[q] = max(top[q][l], __shfl_xor_sync(MEP_FULL_MASK, top[q][l], 1));
      m[q] = max(m[q], __shfl_xor_sync(MEP_FULL_MASK, m[q], 2));
    }
    if (group >= 64) m[0] = m[1] = max(m[0], m[1]), m[2] = m[3] = max(m[2], m[3]);
    if (group >= 128) m[0] = m[1] = m[2] = m[3] = max(m[0], m[2]);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      scale[q][l] = m[q] >= 0x7f800000u ? __uint_as_float(0x7fc00000u)
                                        : __bfloat162float(__float2bfloat16_rn(__uint_as_float(m[q]) * (1.f / kW4Top)));
  }
  constexpr float kShift = 12582912.f + 8.f;
  float inv[4][2];
  bool divide = sizeof(T) == 4;
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int l = 0; l < 2; ++l) {
      // a scale of zero or NaN: every q is 0
      inv[q][l] = scale[q][l] > 0.f ? 1.f / scale[q][l] : 0.f;
      divide |= scale[q][l] > 0.f && scale[q][l] < 0x1p-100f;
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
          const float sc = scale[2 * h + j / 2][l], in = inv[2 * h + j / 2][l];
          const float x = to_f32(mine[row_of(h, j, r, t) * kPitch<T> + 8 * l]);
          float q;
          if (divide) {
            q = in > 0.f ? x / sc : 0.f;
          } else {
            q = in > 0.f ? x * in : 0.f;
            q = in > 0.f ? fmaf(fmaf(-q, sc, x), in, q) : 0.f;
          }
          const uint32_t bits = __float_as_uint(fminf(fmaxf(q, -kW4Top), kW4Top) + kShift) & 15u;
          word[j] |= bits << (8 * r + 4 * l);
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

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) k_w4_load(const uint8_t* __restrict__ w4, Matrices s, int group,
                                                      T* __restrict__ w) {
  __shared__ __align__(16) T tile[kW4Rows * kPitch<T>];
  pdl_launch_dependents();
  pdl_wait();
  const At a = at_block(s, blockIdx.x);
  const int c = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint8_t* in = w4 + (long long)blockIdx.x * w4_block_bytes(group);
  const __nv_bfloat162* scales = reinterpret_cast<const __nv_bfloat162*>(in + kW4Pairs) + c * 8 + g;
  T* mine = tile + 16 * c + g;
  uint4 pairs[2];
  __nv_bfloat162 sc[4];  // of 32 rows
#pragma unroll
  for (int h = 0; h < 2; ++h) pairs[h] = __ldcs(reinterpret_cast<const uint4*>(in) + ((h * 4 + c) * 8 + g) * 4 + t);
#pragma unroll
  for (int q = 0; q < 4; ++q) sc[q] = scales[(group == 32 ? q : group == 64 ? q / 2 : 0) * 32];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t word[4] = {pairs[h].x, pairs[h].y, pairs[h].z, pairs[h].w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int l = 0; l < 2; ++l) {
          // q + 8 under 2^23, less 2^23 + 8
          const float q = __uint_as_float(((word[j] >> (8 * r + 4 * l)) & 15u) | 0x4b000000u) - 8388616.f;
          const __nv_bfloat162 p = sc[2 * h + j / 2];
          mine[row_of(h, j, r, t) * kPitch<T> + 8 * l] = from_f32<T>(q * __bfloat162float(l ? p.y : p.x));
        }
  }
  __syncthreads();
  rows_out<T, VEC>(tile, a, w);
}

int w4_check(const void* w, int type, int64_t M, int64_t K, int64_t N, int parts, int group, const void* w4,
             Matrices* s, long long* blocks) {
  if ((type != MEP_BF16 && type != MEP_F32) || M < 0 || parts < 1 || N < 1 || N % parts != 0 ||
      !w4_sizes_ok(K, N / parts, group))
    return MEP_ERR_INVALID_ARG;
  if (M > 0x7fffffffLL || M * parts > 0x7fffffffLL) return MEP_ERR_INVALID_ARG;
  s->K = K, s->N = N / parts, s->parts = parts;
  s->kb = int((K + kW4Rows - 1) / kW4Rows), s->panels = (s->N + kW4Cols - 1) / kW4Cols;
  if (M * parts > 0x7fffffffLL / ((long long)s->kb * s->panels)) return MEP_ERR_INVALID_ARG;
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

namespace {
// Whole vectors: every row of every part starts on a 16-byte boundary.
bool vectors(const void* w, int type, const Matrices& s) {
  const int v = type == MEP_BF16 ? 8 : 4;
  return aligned16(w) && s.N % v == 0;
}
template <typename... KArgs, typename... Args>
int launch_blocks(void (*kernel)(KArgs...), long long blocks, void* stream, Args... args) {
  return launch_pdl(kernel, dim3(unsigned(blocks)), dim3(kThreads), 0, static_cast<cudaStream_t>(stream), args...) == cudaSuccess
             ? MEP_OK
             : MEP_ERR_CUDA;
}
}  // namespace

extern "C" int mep_w4_save(const void* w, int w_type, int64_t M, int64_t K, int64_t N, int parts, int group,
                           uint8_t* w4, void* stream) {
  Matrices s;
  long long blocks = 0;
  const int rc = w4_check(w, w_type, M, K, N, parts, group, w4, &s, &blocks);
  if (rc != MEP_OK || blocks == 0) return rc;
  const bool vec = vectors(w, w_type, s);
  if (w_type == MEP_BF16)
    return launch_blocks(vec ? k_w4_save<__nv_bfloat16, true> : k_w4_save<__nv_bfloat16, false>, blocks, stream,
                         static_cast<const __nv_bfloat16*>(w), s, group, w4);
  return launch_blocks(vec ? k_w4_save<float, true> : k_w4_save<float, false>, blocks, stream, static_cast<const float*>(w), s,
                       group, w4);
}

extern "C" int mep_w4_load(const uint8_t* w4, int64_t M, int64_t K, int64_t N, int parts, int group, int w_type,
                           void* w, void* stream) {
  Matrices s;
  long long blocks = 0;
  const int rc = w4_check(w, w_type, M, K, N, parts, group, w4, &s, &blocks);
  if (rc != MEP_OK || blocks == 0) return rc;
  const bool vec = vectors(w, w_type, s);
  if (w_type == MEP_BF16)
    return launch_blocks(vec ? k_w4_load<__nv_bfloat16, true> : k_w4_load<__nv_bfloat16, false>, blocks, stream, w4, s, group,
                         static_cast<__nv_bfloat16*>(w));
  return launch_blocks(vec ? k_w4_load<float, true> : k_w4_load<float, false>, blocks, stream, w4, s, group,
                       static_cast<float*>(w));
}
