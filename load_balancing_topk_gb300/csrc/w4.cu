// w4.cu -- weight matrices to 4 bits and back (mep_w4_save, mep_w4_load).
//
// One pass over memory, a CTA a block of 128 rows and 64 columns, which goes
// through shared memory: rows outside in 16-byte vectors, inside the 32 rows of
// two columns that a lane's pairs are of (w4.cuh). Rows that do not start on
// 16-byte boundaries are read and written element by element, coalesced over a
// row's 64 columns. What bounds it is what a lane has to issue for a weight.
//   save  Largest magnitudes first, of 32 rows of two columns a thread (bf16, in
//         packed maxima) or 64 of one; scales and their reciprocals, one thread
//         each; then the pairs. q = w / s is a division, as the format is defined
//         by it: a product by the correctly rounded 1 / s and corrections by the
//         remainder, two fused multiply-adds each, after which the quotient is
//         correctly rounded (Markstein, 1990: two from fp32; one from bf16, where
//         a quotient of two numbers of eight bits is 2^-9 or more from every half
//         step unless it is one, and one it meets exactly). 1.5 * 2^23 rounds to
//         a whole number, ties to even, and four of them become 16 bits of pairs
//         by multiply-adds. Scales below 2^-100, whose reciprocal or remainder
//         may leave fp32, divide, and keep within +-7, which others do anyway.
//         The scale is a product by fp32's 1/7, not a quotient: that is what
//         dividing a tensor by 7 is on the GPU in elementary tensor operations, whose
//         bytes these are then. The two round to different bf16 for 140 of 2^24
//         fp32 magnitudes, for none that a bf16 holds.
//   load  In bf16 two weights at once: the bits of q + 8 are a bf16 of q / 64
//         after one multiply-add (few.cu), and that times 64 s is rounded once.
//         Scales from 2^120 on go the other way, through fp32, like fp32 output.
//
// Measured, L2 flushed before: bf16 [64, 2048, 2816] saved in 254 us and loaded in
// 146, where 929 MB each way take 139 at the copy rate (55%, 95%); fp32 [16, 2048,
// 2816] 103 and 68 (416 MB, 62: 60%, 91%). Element by element, bf16 [16, 2047,
// 2817] 143 and 118 (232 MB, 35), fp32 169 and 112 (62): bound by the accesses, two
// or four bytes a lane; the aligned vectors that cover a row, shifted on their way
// through shared memory, are not built. Read by a lane from where its pairs' values lie, without the shared
// memory, the first took 1640 both ways; through it 558; with packed maxima,
// corrected quotients and pairs by multiply-adds 400.

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
#pragma unroll 32
    for (int i = 0; i < kW4Rows * kW4Cols / kThreads; ++i) {
      const int q = i * kThreads + threadIdx.x, r = q / kW4Cols, c = q % kW4Cols;
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

constexpr float kRoundShift = 12582912.f;  // 1.5 * 2^23

// q of x: x / s to the nearest whole number. `ONCE`: one correction is enough.
// (Two at a time in packed fp32 it took 279 us where this takes 255.)
template <bool ONCE> __device__ __forceinline__ float quotient(float x, float s, float inv) {
  float q = x * inv;
  q = fmaf(fmaf(-q, s, x), inv, q);
  if (!ONCE) q = fmaf(fmaf(-q, s, x), inv, q);
  return (q + kRoundShift) - kRoundShift;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) k_w4_save(const T* __restrict__ w, Matrices s, int group,
                                                      uint8_t* __restrict__ w4) {
  __shared__ __align__(16) T tile[kW4Rows * kPitch<T>];
  __shared__ uint32_t s_top[4][kW4Cols];  // of 32 rows: the largest magnitude's bits
  __shared__ float2 s_scale[4][kW4Cols];  // and the group's scale, and 1 / it
  pdl_launch_dependents();
  pdl_wait();
  const At a = at_block(s, blockIdx.x);
  rows_in<T, VEC>(w, a, tile);
  __syncthreads();
  const int tid = threadIdx.x;
  if (sizeof(T) == 2) {
    const __nv_bfloat162* in = reinterpret_cast<const __nv_bfloat162*>(tile) + (tid >> 5) * 32 * (kPitch<T> / 2) + (tid & 31);
    __nv_bfloat162 m = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll 16
    for (int r = 0; r < 32; ++r) m = __hmax2_nan(m, __habs2(in[r * (kPitch<T> / 2)]));
    s_top[tid >> 5][2 * (tid & 31)] = __float_as_uint(__bfloat162float(m.x));
    s_top[tid >> 5][2 * (tid & 31) + 1] = __float_as_uint(__bfloat162float(m.y));
  } else {
    const uint32_t* in = reinterpret_cast<const uint32_t*>(tile) + (tid >> 6) * 64 * kPitch<T> + (tid & 63);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      uint32_t m = 0;  // an infinity and then a NaN lie above all numbers
#pragma unroll 16
      for (int r = 0; r < 32; ++r) m = max(m, in[(32 * q + r) * kPitch<T>] & 0x7fffffffu);
      s_top[2 * (tid >> 6) + q][tid & 63] = m;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int q = 2 * (tid >> 6) + i, c = tid & 63, n = group / 32, q0 = q / n * n;
    uint32_t m = s_top[q0][c];
    for (int o = 1; o < n; ++o) m = max(m, s_top[q0 + o][c]);
    const float sc = m >= 0x7f800000u ? __uint_as_float(0x7fc00000u)
                                      : __bfloat162float(__float2bfloat16_rn(__uint_as_float(m) * (1.f / kW4Top)));
    s_scale[q][c] = make_float2(sc, sc > 0.f ? 1.f / sc : 0.f);  // 0: every q is 0
  }
  __syncthreads();
  const int c = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  uint8_t* out = w4 + (long long)blockIdx.x * w4_block_bytes(group);
  const T* mine = tile + 16 * c + g;
  bool slow = false;
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int l = 0; l < 2; ++l) {
      const float2 sc = s_scale[q][16 * c + 8 * l + g];
      slow |= !(sc.x == 0.f) && !(sc.x >= 0x1p-100f);  // NaN too: what it meets may not be a number
    }
  uint4* pairs = reinterpret_cast<uint4*>(out) + (c * 8 + g) * 4 + t;
  if (!slow) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t word[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 s0 = s_scale[2 * h + j / 2][16 * c + g], s1 = s_scale[2 * h + j / 2][16 * c + 8 + g];
        float byte[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const T* x = mine + row_of(h, j, r, t) * kPitch<T>;
          byte[r] = fmaf(quotient<sizeof(T) == 2>(to_f32(x[8]), s1.x, s1.y), 16.f,
                         quotient<sizeof(T) == 2>(to_f32(x[0]), s0.x, s0.y));
        }
        // + 136 in every byte, and the bits of a whole number
        const uint32_t low = __float_as_uint(fmaf(byte[1], 256.f, byte[0]) + (kRoundShift + 34952.f));
        const uint32_t high = __float_as_uint(fmaf(byte[3], 256.f, byte[2]) + (kRoundShift + 34952.f));
        word[j] = __byte_perm(low, high, 0x5410);
      }
      pairs[h * 128] = make_uint4(word[0], word[1], word[2], word[3]);
    }
  } else {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      const int h = i >> 2, j = i & 3;
      uint32_t word = 0;
#pragma unroll 1
      for (int o = 0; o < 8; ++o) {
        const int r = o >> 1, l = o & 1;
        const float2 sc = s_scale[2 * h + j / 2][16 * c + 8 * l + g];
        const float q = sc.x > 0.f ? rintf(to_f32(mine[row_of(h, j, r, t) * kPitch<T> + 8 * l]) / sc.x) : 0.f;
        word |= uint32_t(int(fminf(fmaxf(q, -kW4Top), kW4Top)) + 8) << (8 * r + 4 * l);
      }
      reinterpret_cast<uint32_t*>(pairs + h * 128)[j] = word;
    }
  }
  if (t < kW4Rows / group) {
    const int q = t * (group / 32);
    reinterpret_cast<__nv_bfloat162*>(out + kW4Pairs)[t * 32 + c * 8 + g] =
        __floats2bfloat162_rn(s_scale[q][16 * c + g].x, s_scale[q][16 * c + 8 + g].x);
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
  bool wide = false;
#pragma unroll
  for (int h = 0; h < 2; ++h) pairs[h] = __ldcs(reinterpret_cast<const uint4*>(in) + ((h * 4 + c) * 8 + g) * 4 + t);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    sc[q] = scales[(group == 32 ? q : group == 64 ? q / 2 : 0) * 32];
    wide |= !(__bfloat162float(sc[q].x) < 0x1p120f) || !(__bfloat162float(sc[q].y) < 0x1p120f);
  }
  if (sizeof(T) == 2 && !wide) {
    __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(mine);
    const __nv_bfloat162 k64 = __floats2bfloat162_rn(64.f, 64.f);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t word[4] = {pairs[h].x, pairs[h].y, pairs[h].z, pairs[h].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 s64 = __hmul2(sc[2 * h + j / 2], k64);
        uint32_t v = word[j];
#pragma unroll
        for (int i = 0; i < 2; ++i, v >>= 8)
#pragma unroll
          for (int l = 0; l < 2; ++l) {
            uint32_t q;
            asm("fma.rn.bf16x2 %0, %1, %2, %3;"
                : "=r"(q)
                : "r"(v & (l ? 0x00f000f0u : 0x000f000fu)), "r"(l ? 0x7d007d00u : 0x7f007f00u), "r"(0xbe00be00u));
            const __nv_bfloat162 x = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&q), l ? __high2bfloat162(s64) : __low2bfloat162(s64));
            // rows 8 i + 2 t and the next one
            o[row_of(h, j, i, t) * kPitch<T> + 8 * l] = x.x;
            o[row_of(h, j, i + 2, t) * kPitch<T> + 8 * l] = x.y;
          }
      }
    }
  } else {
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
