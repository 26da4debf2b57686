// ckpt.cuh -- the 8-bit checkpoint row shared by layer_norm.cu, act_ckpt.cu
// and grouped_wgrad.cu, and the element types of the training operators.
//
// A row of C columns: C signed bytes q, from byte align16(C) on one scale
// byte s per block of 128 columns, padding to a multiple of 32 bytes. A value
// is q * 2^(s - 127). Per block, with a = max |x|: k = max(floor(log2 a) - 6,
// -126), s = k + 127, q = rint(x * 2^-k) (ties to even) kept within +-127.
// a * 2^-k lies in [64, 128), so a bf16 x (8 significant bits: at most 127.5)
// is off by at most half a step, 2^(k-1). Every factor is a power of two:
// the rounding to q is the only one, and q * 2^k is exact in bf16, which is
// what lets a tensor-core product run on exactly the kept values. Fixed
// point rather than an 8-bit float: the step is a / 64 at most over the whole
// block, where a 3-bit mantissa is off by up to 1/16 of every large value.
// A block that holds an infinity or a NaN gets s = 255: its values come back
// as NaN, so that an overflow stays visible in the gradients.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "mep_common.cuh"
#include "vec.cuh"

namespace mep {
namespace {

constexpr int kCkptBlock = 128;   // columns that share one scale byte
constexpr int kCkptNan = 255;     // scale byte of a block with a non-finite value

__host__ __device__ __forceinline__ int ckpt_scale_at(int C) { return (C + 15) & ~15; }
__host__ __device__ __forceinline__ long long ckpt_row_bytes(long long C) {
  return (((C + 15) & ~15LL) + (C + kCkptBlock - 1) / kCkptBlock + 31) & ~31LL;
}

// Scale byte of a block from the bits of its largest magnitude (as unsigned
// integers, magnitudes compare as they do as numbers, with infinity and then
// NaN above them all).
__device__ __forceinline__ int ckpt_scale(uint32_t top) {
  const int e = int(top >> 23);  // biased exponent; 0 also for zero and subnormals
  return e == 255 ? kCkptNan : max(e - 6, 1);
}
// 2^-k and 2^k of a scale byte s = k + 127, 1 <= s <= 248; 0 and NaN for 255.
__device__ __forceinline__ float ckpt_inv_step(int s) {
  return s == kCkptNan ? 0.f : __uint_as_float(uint32_t(254 - s) << 23);
}
__device__ __forceinline__ float ckpt_step(int s) {
  return __uint_as_float(s == kCkptNan ? 0x7fc00000u : uint32_t(s) << 23);
}
// Signed byte j of w as a float: its bits under 2^23, less 2^23 + 128.
// (w here with its bytes' sign bits flipped.)
__device__ __forceinline__ float ckpt_byte(uint32_t w, int j) {
  return __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 + j));
}
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Where a tensor of `type` with these columns may start: rows of a multiple of
// 8 columns are read and written in 16-byte vectors, others element by element,
// so that any run of their rows is as good; checkpoint rows are whole vectors
// at any width.
inline bool may_start(const void* p, int type, long long columns) {
  const uintptr_t step = columns % 8 == 0 || type == MEP_CKPT8 ? 16 : type == MEP_BF16 ? 2 : 4;
  return reinterpret_cast<uintptr_t>(p) % step == 0;
}

// ---------------------------------------------------------------------------
// Two fp32 values in one 64-bit register, and operations on both at once, each
// rounded as the single form is.
struct F2 {
  unsigned long long v;
  __device__ __forceinline__ float x() const { return __uint_as_float(uint32_t(v)); }
  __device__ __forceinline__ float y() const { return __uint_as_float(uint32_t(v >> 32)); }
};
__device__ __forceinline__ F2 pair(float x, float y) {
  F2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d.v) : "f"(x), "f"(y));
  return d;
}
__device__ __forceinline__ F2 both(float v) { return pair(v, v); }
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return d;
}
// Two bf16 of a word, widened.
__device__ __forceinline__ F2 widen(uint32_t w) {
  return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// x * 2^-k + 1.5 * 2^23 in one rounding leaves x * 2^-k rounded to nearest-even
// in the low bits (a conversion instruction runs at an eighth of the rate). In
// a block with s = 255 every finite value becomes 0 (times 0), the others some
// byte that is never read as a value.
constexpr float kRound = 12582912.f;
__device__ __forceinline__ uint2 ckpt_bytes(const F2 (&r)[4]) {
  uint32_t q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) q[j] = __byte_perm(uint32_t(r[j].v), uint32_t(r[j].v >> 32), 0x0040);
  return make_uint2(__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410));
}

// ---------------------------------------------------------------------------
// Sixteen lanes share a block of 128 columns; each holds eight of them. VEC:
// columns [8l, 8l + 8) of the block, whole 16-byte vectors (rows of a multiple
// of 8 columns); else columns l, l + 16, ... one by one, which stay coalesced
// where rows start anywhere.
constexpr int kHalf = 16;

template <bool VEC> __device__ __forceinline__ int half_col(int block, int l, int j) {
  return block * kCkptBlock + (VEC ? 8 * l + j : l + kHalf * j);
}
// Bits of the largest magnitude of four words of two bf16, of four pairs of fp32.
// (a maximum that keeps a NaN; on the packed words with integer instructions
// the gated activation ran 4% slower)
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t top_of(const F2 (&v)[4]) {
  float t = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) t = max_nan(t, max_nan(fabsf(v[j].x()), fabsf(v[j].y())));
  return __float_as_uint(t);
}
__device__ __forceinline__ uint32_t top_of(const uint32_t (&w)[4]) {
  const F2 v[4] = {widen(w[0]), widen(w[1]), widen(w[2]), widen(w[3])};
  return top_of(v);
}

// Eight values of a row as they lie in memory (columns beyond C are 0).
template <int KIND> struct Pack;
template <> struct Pack<MEP_BF16> {
  uint32_t w[4];
  template <bool VEC>
  __device__ __forceinline__ void load(const void* base, long long row, int C, int block, int l) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + row * C;
    if (VEC) {
      const int c = half_col<true>(block, l, 0);
      const uint4 q = c < C ? ld_nc(reinterpret_cast<const uint4*>(p + c)) : make_uint4(0, 0, 0, 0);
      w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c0 = half_col<false>(block, l, 2 * j), c1 = half_col<false>(block, l, 2 * j + 1);
        w[j] = (c0 < C ? __ldg(p + c0) : 0u) | (c1 < C ? uint32_t(__ldg(p + c1)) << 16 : 0u);
      }
    }
  }
  __device__ __forceinline__ F2 at(int j) const {  // values 2j and 2j + 1
    return widen(w[j]);
  }
  __device__ __forceinline__ F2 plus(int j, F2 c) const { return add2(at(j), c); }  // at(j) + c
  __device__ __forceinline__ uint32_t top() const { return top_of(w); }
  __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0u; }
};
template <> struct Pack<MEP_F32> {
  float v[8];
  template <bool VEC>
  __device__ __forceinline__ void load(const void* base, long long row, int C, int block, int l) {
    const float* p = static_cast<const float*>(base) + row * C;
    if (VEC) {
      const int c = half_col<true>(block, l, 0);
      const bool in = c < C;
      const float4* q = reinterpret_cast<const float4*>(p + c);
      const float4 a = in ? __ldg(q) : make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 b = in ? __ldg(q + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = half_col<false>(block, l, j);
        v[j] = c < C ? __ldg(p + c) : 0.f;
      }
    }
  }
  __device__ __forceinline__ F2 at(int j) const { return pair(v[2 * j], v[2 * j + 1]); }
  __device__ __forceinline__ F2 plus(int j, F2 c) const { return add2(at(j), c); }
  __device__ __forceinline__ uint32_t top() const {
    const F2 a[4] = {at(0), at(1), at(2), at(3)};
    return top_of(a);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
  }
};
template <> struct Pack<MEP_CKPT8> {
  uint32_t w[2];
  float step;
  template <bool VEC>
  __device__ __forceinline__ void load(const void* base, long long row, int C, int block, int l) {
    const uint8_t* p = static_cast<const uint8_t*>(base) + row * ckpt_row_bytes(C);
    const bool in = half_col<VEC>(block, l, 0) < C;
    if (VEC) {
      const uint2 q = in ? __ldg(reinterpret_cast<const uint2*>(p + half_col<true>(block, l, 0)))
                         : make_uint2(0, 0);
      w[0] = q.x, w[1] = q.y;
    } else {
      w[0] = w[1] = 0u;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = half_col<false>(block, l, j);
        if (c < C) w[j >> 2] |= uint32_t(__ldg(p + c)) << (8 * (j & 3));
      }
    }
    step = in ? ckpt_step(__ldg(p + ckpt_scale_at(C) + block)) : 0.f;
  }
  __device__ __forceinline__ F2 q(int j) const {
    const uint32_t u = w[j >> 1] ^ 0x80808080u;
    const int b = 2 * (j & 1);
    return add2(pair(ckpt_byte(u, b), ckpt_byte(u, b + 1)), both(-8388736.f));
  }
  __device__ __forceinline__ F2 at(int j) const { return mul2(q(j), both(step)); }
  __device__ __forceinline__ F2 plus(int j, F2 c) const { return fma2(q(j), both(step), c); }
  __device__ __forceinline__ void clear() { w[0] = w[1] = 0u, step = 0.f; }
};

// Four pairs of values into the row at p, rounded to its type (FULL: the block
// is known to lie within the row; `in`: there is such a row); v becomes what
// was stored. Returns the bits of its largest magnitude.
template <typename T, bool VEC, bool FULL = false>
__device__ __forceinline__ uint32_t store8(T* p, int C, int block, int l, F2 (&v)[4], bool in = true) {
  if (sizeof(T) == 2) {
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[j].x(), v[j].y());
      o[j] = *reinterpret_cast<const uint32_t*>(&h);
      v[j] = widen(o[j]);
    }
    if (VEC) {
      const int c = half_col<true>(block, l, 0);
      if (in && (FULL || c < C)) *reinterpret_cast<uint4*>(p + c) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = half_col<false>(block, l, j);
        if (in && c < C) reinterpret_cast<uint16_t*>(p)[c] = uint16_t(j & 1 ? o[j >> 1] >> 16 : o[j >> 1]);
      }
    }
    return top_of(o);
  } else {
    if (VEC) {
      const int c = half_col<true>(block, l, 0);
      if (in && (FULL || c < C)) {
        // in one piece where it lies so (the same for all rows, as rows are whole
        // sectors): two pieces are two writes of every sector (norm forward of
        // [32768, 2048] 100 us, in one 89; loading it from 8 bits and saving it 127, 108)
        if (reinterpret_cast<uintptr_t>(p + c) % 32 == 0) {
          asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(p + c), "l"(v[0].v), "l"(v[1].v),
                       "l"(v[2].v), "l"(v[3].v)
                       : "memory");
        } else {
          float4* q = reinterpret_cast<float4*>(p + c);
          q[0] = make_float4(v[0].x(), v[0].y(), v[1].x(), v[1].y());
          q[1] = make_float4(v[2].x(), v[2].y(), v[3].x(), v[3].y());
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = half_col<false>(block, l, j);
        if (in && c < C) reinterpret_cast<float*>(p)[c] = j & 1 ? v[j >> 1].y() : v[j >> 1].x();
      }
    }
    return top_of(v);
  }
}

// n blocks on their way into checkpoint rows: for each its row, its number
// in the row, whether this half warp has it at all, the bits of this lane's
// largest magnitude, and this lane's values.
template <int n> struct Kept {
  uint8_t* row[n];
  int block[n];
  bool in[n];
  uint32_t top[n];
  F2 v[n][4];
};
// Writes them, all lanes of the warp together; the lanes of a row's last block
// also write its padding. The blocks go through each stage side by side: one by
// one, with their branches between them, hardly two of their instructions
// overlapped.
template <bool VEC, bool FULL = false, int n>
__device__ __forceinline__ void save8(Kept<n>& k, int C, int l) {
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) k.top[i] = max(k.top[i], __shfl_xor_sync(MEP_FULL_MASK, k.top[i], d));
  int s[n];
  bool cut = false;
#pragma unroll
  for (int i = 0; i < n; ++i) {
    s[i] = ckpt_scale(k.top[i]);
    const float inv = ckpt_inv_step(s[i]);
    cut |= __uint_as_float(k.top[i]) * inv >= 127.5f;
#pragma unroll
    for (int j = 0; j < 4; ++j) k.v[i][j] = fma2(k.v[i][j], both(inv), both(kRound));
  }
  if (cut) {  // only a block whose largest value is at least 127.5 steps can round to 128: one in a hundred
#pragma unroll
    for (int i = 0; i < n; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        k.v[i][j] = pair(fminf(fmaxf(k.v[i][j].x(), kRound - 127.f), kRound + 127.f),
                         fminf(fmaxf(k.v[i][j].y(), kRound - 127.f), kRound + 127.f));
  }
  const int at = ckpt_scale_at(C), nb = (C + kCkptBlock - 1) / kCkptBlock;
  bool last = false;
#pragma unroll
  for (int i = 0; i < n; ++i) {
    const uint2 q = ckpt_bytes(k.v[i]);
    if (VEC) {
      const int c = half_col<true>(k.block[i], l, 0);
      if (k.in[i] && (FULL || c < C)) *reinterpret_cast<uint2*>(k.row[i] + c) = q;
    } else if (k.in[i]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = half_col<false>(k.block[i], l, j);
        if (c < C) k.row[i][c] = uint8_t((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
      }
    }
    if (l == 0 && k.in[i]) k.row[i][at + k.block[i]] = uint8_t(s[i]);
    last |= k.block[i] == nb - 1;
  }
  if (last) {
    const int end = int(ckpt_row_bytes(C));
#pragma unroll
    for (int i = 0; i < n; ++i)
      if (k.in[i] && k.block[i] == nb - 1) {
        if (C + l < at) k.row[i][C + l] = 0;
        for (int e = at + nb + l; e < end; e += kHalf) k.row[i][e] = 0;
      }
  }
}

}  // namespace
}  // namespace mep
