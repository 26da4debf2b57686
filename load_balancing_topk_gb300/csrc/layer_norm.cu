// layer_norm.cu -- layer norm over the hidden width (mep_layer_norm) and its
// backward pass (mep_layer_norm_backward), with 8-bit checkpoint rows as a
// by-product of the first and as input of the second.
//
// Both are one pass over memory with the row in registers: a row belongs to W
// warps, whose half warps hold blocks of 128 columns, eight values a lane
// (the checkpoint's blocks, so that a block's largest magnitude is four
// shuffles away). Sums over a row go through shuffles and, for W > 1, a few
// words of shared memory.
// A row of a multiple of 8 columns is fetched ahead: every thread copies its
// own vectors of the rows of the next turns into its own slots of shared memory
// (cp.async), so that the next rows' loads are under way while a row's sums
// are, and no thread waits for another's copies. What a thread has to issue
// bounds them, most of all narrow rows. The backward pass of [65536, 7168] took
// 820 us with the rows in flight in registers, 665 copied ahead and in pairs of
// fp32, 444 with two rows of 16 columns a thread, 128 registers and addresses
// that step, and takes 437 now (95% of the copy rate); [32768, 2048] takes 49
// us forward (81%), 68 with y in 8 bits (73%), 70 backward from x in 8 bits (71%).
//   k_norm       every warp takes the mean of its part of a row, then the
//                squares around that mean; joined after one barrier, as
//                var H = sum of the warps' squares + n_w (mean_w - mean)^2.
//                All squares are of differences: a row far from zero loses
//                nothing to cancellation.
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
// Rows of other widths are loaded as they are used, value by value, but L2 is
// asked for them two turns before: [32768, 2047] bf16 forward 123 -> 100 us,
// backward 168 -> 122 (131 with one turn).
constexpr int kTurnsToL2 = 2;
// Turns whose rows are on their way: up to four, as many as fit `room` bytes of
// slots a thread.
__host__ __device__ constexpr int ahead_of(int bytes, int room) {
  return room / bytes >= 4 ? 4 : room / bytes > 1 ? room / bytes : 1;
}

// ---------------------------------------------------------------------------
// Barrier of one row group: W warps (of a CTA that may hold several groups).
__device__ __forceinline__ void group_sync(int group, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
}

// Eight parameters of a block; `none` without the tensor, 0 beyond H.
template <bool VEC>
__device__ __forceinline__ void load_params(const void* p, int type, int H, int block, int l,
                                            float none, F2 (&v)[4]) {
  if (p == nullptr) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = both(none);
  } else if (type == MEP_F32) {
    Pack<MEP_F32> q;
    q.load<VEC>(p, 0, H, block, l);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = q.at(j);
  } else {
    Pack<MEP_BF16> q;
    q.load<VEC>(p, 0, H, block, l);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = q.at(j);
  }
}

// Sums of n (2 or 4) values a thread over the W warps of a group. The lanes
// first share the values out among themselves (each step halves the values a
// lane still carries): 6 or 7 shuffles a warp, not 10 or 20. s holds n words a
// warp, not in use elsewhere before the group's next barrier but one.
template <int n> __device__ __forceinline__ float warp_sums(float (&v)[n]) {
  constexpr int lanes = 32 / n;  // that carry the same value in the end
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
  float t = v[0];
#pragma unroll
  for (int e = lanes / 2; e >= 1; e >>= 1) t += __shfl_xor_sync(MEP_FULL_MASK, t, e);
  return t;  // of value lane / lanes: the lane's bits 4, 3, ... chose it, high bit first
}
template <int n>
__device__ __forceinline__ void group_sums(float (&v)[n], float* s, int W, int warp, int group) {
  constexpr int lanes = 32 / n;
  const int lane = threadIdx.x & 31;
  float t = warp_sums<n>(v);
  if (W > 1) {
    const int mine = lane / lanes, k0 = lane % lanes;
    if (k0 == 0) s[warp * n + mine] = t;
    group_sync(group, 32 * W);
    t = 0.f;
    for (int k = k0; k < W; k += lanes) t += s[k * n + mine];
#pragma unroll
    for (int e = lanes / 2; e >= 1; e >>= 1) t += __shfl_xor_sync(MEP_FULL_MASK, t, e);
  }
#pragma unroll
  for (int i = 0; i < n; ++i) v[i] = __shfl_sync(MEP_FULL_MASK, t, i * lanes);
}

// ---------------------------------------------------------------------------
// A thread's slots. Piece i of thread t lies at (i * threads + t) * 16 bytes
// (8 for checkpoint bytes): neighbours side by side.
// Past L1 where a warp's 16-byte pieces lie side by side; through it where every
// other piece is another copy's (32 bytes a lane), or L2 is asked for each
// sector twice: [32768, 2048] fp32 forward 134 us past it, 100 through it,
// backward 207 and 135; bf16 forward 49 and 51.
template <bool L1> __device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  if (L1)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// All but the newest `left` groups of this thread's copies have landed.
template <int left> __device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(left) : "memory");
}

template <int KIND> struct Slot {
  static constexpr int bytes = KIND == MEP_BF16 ? 16 : KIND == MEP_F32 ? 32 : 8;  // per thread and block
  // Address of the eight columns from c of row 0, and the bytes from row to row.
  static __device__ __forceinline__ const char* at(const void* base, int c) {
    return static_cast<const char*>(base) + (long long)c * (bytes / 8);
  }
  static __device__ __forceinline__ long long pitch(int H) {
    return KIND == MEP_CKPT8 ? ckpt_row_bytes(H) : (long long)H * (bytes / 8);
  }
  static __device__ __forceinline__ void copy(uint32_t slot, int threads, const char* src) {
    const int t = threadIdx.x;
    if (KIND == MEP_CKPT8) {
      copy_async8(slot + t * 8, src);
    } else {
      copy_async16<KIND == MEP_F32>(slot + t * 16, src);
      if (KIND == MEP_F32) copy_async16<true>(slot + (threads + t) * 16, src + 16);
    }
  }
  static __device__ __forceinline__ void zero(uint32_t slot, int threads) {
    const int t = threadIdx.x;
    if (KIND == MEP_CKPT8) {
      asm volatile("st.shared.v2.b32 [%0], {%1, %1};" ::"r"(slot + t * 8), "r"(0) : "memory");
    } else {
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(slot + t * 16), "r"(0) : "memory");
      if (KIND == MEP_F32)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(slot + (threads + t) * 16), "r"(0)
                     : "memory");
    }
  }
  static __device__ __forceinline__ void put(uint32_t slot, int threads, const Pack<KIND>& p) {
    const int t = threadIdx.x;
    if constexpr (KIND == MEP_CKPT8) {
      asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(slot + t * 8), "r"(p.w[0]), "r"(p.w[1]) : "memory");
    } else if constexpr (KIND == MEP_BF16) {
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(slot + t * 16), "r"(p.w[0]), "r"(p.w[1]),
                   "r"(p.w[2]), "r"(p.w[3])
                   : "memory");
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(slot + (h * threads + t) * 16),
                     "f"(p.v[4 * h]), "f"(p.v[4 * h + 1]), "f"(p.v[4 * h + 2]), "f"(p.v[4 * h + 3])
                     : "memory");
    }
  }
  static __device__ __forceinline__ void fetch(uint32_t slot, int threads, Pack<KIND>& p) {
    const int t = threadIdx.x;
    if constexpr (KIND == MEP_CKPT8) {
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(p.w[0]), "=r"(p.w[1]) : "r"(slot + t * 8));
    } else if constexpr (KIND == MEP_BF16) {
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(p.w[0]), "=r"(p.w[1]), "=r"(p.w[2]), "=r"(p.w[3])
                   : "r"(slot + t * 16));
    } else {
      asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(p.v[0]), "=f"(p.v[1]), "=f"(p.v[2]), "=f"(p.v[3])
                   : "r"(slot + t * 16));
      asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(p.v[4]), "=f"(p.v[5]), "=f"(p.v[6]), "=f"(p.v[7])
                   : "r"(slot + (threads + t) * 16));
    }
  }
};

// Asks L2 for the rows from r on, U or as many as there are, of `pitch` bytes
// each, by the threads (t of n) of a group.
template <int U>
__device__ __forceinline__ void rows_to_l2(const void* p, unsigned r, unsigned N, long long pitch, int t, int n) {
  const char* row = static_cast<const char*>(p) + r * pitch;
  const long long end = (r >= N ? 0 : min(unsigned(U), N - r)) * pitch;
  for (long long o = 128ll * t; o < end; o += 128ll * n) prefetch_l2(row + o);
}

// An SM has 512 threads with 128 registers each, in CTAs of up to 512: what they
// wait for is copied ahead, and more of them with fewer registers issue more
// for the same work (forward [32768, 2048] with 1024 threads, one block a half
// warp: 62 us against 52, with y in 8 bits and that read back 131 against 115).
constexpr int kSmThreads = 512;
// Beyond two blocks a half warp the parameters have no room in registers: a
// thread keeps its own in shared memory, 32 bytes a block, beside the slots
// (from L2 they were more bytes than the rows: bf16 [16384, 12288] forward 280
// us, 191 so, backward 345 and 222).
template <int J> constexpr int kParamBytes = J > 2 ? 32 * J : 0;
template <int KIND, int J, int U> __host__ __device__ constexpr int norm_ahead() {
  return ahead_of(U * J * Slot<KIND>::bytes, 196608 / kSmThreads - 2 * kParamBytes<J>);
}
template <int KIND, int XKIND, int J, int U> __host__ __device__ constexpr int dx_ahead() {
  return ahead_of(U * J * (Slot<KIND>::bytes + Slot<XKIND>::bytes), 196608 / kSmThreads - kParamBytes<J>);
}
__device__ __forceinline__ void put_params(uint32_t at, int threads, const F2 (&v)[4]) {
  asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(at + threadIdx.x * 16), "l"(v[0].v), "l"(v[1].v) : "memory");
  asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(at + (threads + threadIdx.x) * 16), "l"(v[2].v), "l"(v[3].v)
               : "memory");
}
__device__ __forceinline__ void get_params(uint32_t at, int threads, F2 (&v)[4]) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v[0].v), "=l"(v[1].v) : "r"(at + threadIdx.x * 16));
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];"
               : "=l"(v[2].v), "=l"(v[3].v)
               : "r"(at + (threads + threadIdx.x) * 16));
}

// J blocks a half warp, W warps a row (2 J W >= blocks of a row; FULL: equal,
// and no block is cut), U rows a turn, KEEP: a checkpoint is written.
template <typename T, int KIND, bool VEC, bool FULL, bool KEEP, int J, int U>
__global__ void __launch_bounds__(kSmThreads)
    k_norm(const T* __restrict__ x, const void* __restrict__ w, const void* __restrict__ b, int p_type,
           float eps, unsigned N, int H, int W, T* __restrict__ y, float* __restrict__ mean,
           float* __restrict__ rstd, uint8_t* __restrict__ x_ckpt, uint8_t* __restrict__ y_ckpt) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int A = norm_ahead<KIND, J, U>();
  extern __shared__ __align__(16) float s_dyn[];  // slots
  __shared__ float2 s_part[2][kMaxWarps * 2];     // two rows' mean and squares of a warp, twice
  const int l = threadIdx.x % kHalf;
  const int group = (threadIdx.x >> 5) / W, groups = blockDim.x / (32 * W);
  const int warp = (threadIdx.x >> 5) - group * W, half = 2 * warp + ((threadIdx.x >> 4) & 1);
  const int nb = (H + kCkptBlock - 1) / kCkptBlock, threads = blockDim.x;
  const float inv_h = 1.f / H;
  const unsigned first = (blockIdx.x * groups + group) * U, step = gridDim.x * groups * U;
  const long long row_bytes = ckpt_row_bytes(H);
  uint32_t slots = 0;
  constexpr int turn_bytes = J * U * Slot<KIND>::bytes;  // a thread's, of all threads' turn
  const char* src = nullptr;
  long long src_step = 0;
  bool there[J];
#pragma unroll
  for (int i = 0; i < J; ++i) there[i] = FULL || half_col<VEC>(half + 2 * W * i, l, 0) < H;
  const auto ahead = [&](unsigned r, uint32_t slot) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (r + u < N) {
        const char* row = src + u * Slot<KIND>::pitch(H);
#pragma unroll
        for (int i = 0; i < J; ++i)
          if (there[i])
            Slot<KIND>::copy(slot + (u * J + i) * threads * Slot<KIND>::bytes, threads,
                             row + 2 * W * i * 16 * Slot<KIND>::bytes);
      }
    src += src_step;
    copy_async_commit();
  };
  if (VEC) {
    slots = uint32_t(__cvta_generic_to_shared(s_dyn));
    src = Slot<KIND>::at(x, half_col<true>(half, l, 0)) + first * Slot<KIND>::pitch(H);
    src_step = step * Slot<KIND>::pitch(H);
#pragma unroll
    for (int i = 0; i < J; ++i)
      if (!there[i])
        for (int k = 0; k < A * U; ++k) Slot<KIND>::zero(slots + (k * J + i) * threads * Slot<KIND>::bytes, threads);
    for (int k = 0; k < A; ++k) ahead(first + k * step, slots + k * turn_bytes * threads);
  }
  // columns of this warp, and of the warps whose parts this lane joins
  const auto columns = [&](int k) {
    int n = 0;
    for (int i = 0; i < J; ++i) n += max(0, min(2 * kCkptBlock, H - (2 * k + 2 * W * i) * kCkptBlock));
    return n;
  };
  const int k16 = threadIdx.x & 15;
  const float inv_mine = 1.f / max(1, columns(warp));
  const float n_a = k16 < W ? columns(k16) : 0, n_c = k16 + 16 < W ? columns(k16 + 16) : 0;
  F2 wv[J > 2 ? 1 : J][4], bv[J > 2 ? 1 : J][4];
  const uint32_t params = uint32_t(__cvta_generic_to_shared(s_dyn)) + (VEC ? A * turn_bytes * threads : 0);
#pragma unroll
  for (int i = 0; i < J; ++i) {
    const int k = J > 2 ? 0 : i;
    load_params<VEC>(w, p_type, H, half + 2 * W * i, l, 1.f, wv[k]);
    load_params<VEC>(b, p_type, H, half + 2 * W * i, l, 0.f, bv[k]);
    if (J > 2) {
      put_params(params + (2 * i) * threads * 32, threads, wv[k]);
      put_params(params + (2 * i + 1) * threads * 32, threads, bv[k]);
    }
  }
  T* out = y + (long long)first * H;
  uint8_t *xc = x_ckpt + first * row_bytes, *yc = y_ckpt + first * row_bytes;
  int at = 0, turn = 0;  // slot, sums
  for (unsigned r = first; r < N; r += step, turn ^= 1) {
    Pack<KIND> p[U][J];
    if (VEC) {
      const uint32_t slot = slots + at * turn_bytes * threads;
      copy_async_wait<A - 1>();
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < J; ++i)
          Slot<KIND>::fetch(slot + (u * J + i) * threads * Slot<KIND>::bytes, threads, p[u][i]);
      ahead(r + A * step, slot);
      at = at + 1 == A ? 0 : at + 1;
    } else {
      rows_to_l2<U>(x, r + kTurnsToL2 * step, N, Slot<KIND>::pitch(H), threadIdx.x - group * 32 * W, 32 * W);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < J; ++i) {
          if (r + u < N)
            p[u][i].template load<false>(x, r + u, H, half + 2 * W * i, l);
          else
            p[u][i].clear();
        }
    }
    float m[2] = {0.f, 0.f}, rs[2] = {0.f, 0.f};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      F2 sum = both(0.f);
#pragma unroll
      for (int i = 0; i < J; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum = add2(sum, p[u][i].at(j));
      m[u] = sum.x() + sum.y();
    }
    // lane's row of the two is lane / 16 from here on
    const float mw = warp_sums<2>(m) * inv_mine;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      m[u] = __shfl_sync(MEP_FULL_MASK, mw, 16 * u);
      F2 sq = both(0.f);
#pragma unroll
      for (int i = 0; i < J; ++i) {
        const int block = half + 2 * W * i;
        if (!there[i]) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          F2 c = add2(p[u][i].at(j), both(-m[u]));
          if (!VEC)
            c = pair(half_col<false>(block, l, 2 * j) < H ? c.x() : 0.f,
                     half_col<false>(block, l, 2 * j + 1) < H ? c.y() : 0.f);
          sq = fma2(c, c, sq);
        }
      }
      rs[u] = sq.x() + sq.y();
    }
    float sq = warp_sums<2>(rs), mean_all = mw;
    if (W > 1) {
      float2* s = &s_part[turn][group * W * 2];
      if ((threadIdx.x & 15) == 0) s[2 * warp + ((threadIdx.x >> 4) & 1)] = make_float2(mw, sq);
      group_sync(group, 32 * W);
      const int lane = threadIdx.x & 31, k = lane & 15;
      const float2 none = make_float2(0.f, 0.f);
      const float2 a = k < W ? s[2 * k + (lane >> 4)] : none, c = k + 16 < W ? s[2 * (k + 16) + (lane >> 4)] : none;
      float t = fmaf(a.x, n_a, c.x * n_c);
#pragma unroll
      for (int e = 8; e >= 1; e >>= 1) t += __shfl_xor_sync(MEP_FULL_MASK, t, e);
      mean_all = t * inv_h;
      const float da = a.x - mean_all, dc = c.x - mean_all;
      sq = (a.y + c.y) + fmaf(n_a * da, da, n_c * dc * dc);
#pragma unroll
      for (int e = 8; e >= 1; e >>= 1) sq += __shfl_xor_sync(MEP_FULL_MASK, sq, e);
    }
    const float rstd_all = 1.f / sqrtf(sq * inv_h + eps);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      m[u] = __shfl_sync(MEP_FULL_MASK, mean_all, 16 * u);
      rs[u] = __shfl_sync(MEP_FULL_MASK, rstd_all, 16 * u);
      if (threadIdx.x % (32 * W) == u && r + u < N) {
        mean[r + u] = m[u];
        rstd[r + u] = rs[u];
      }
    }
    constexpr int JJ = J < 2 ? J : 2;  // blocks side by side
#pragma unroll
    for (int i0 = 0; i0 < J; i0 += JJ) {
      Kept<JJ * U> k;
#pragma unroll
      for (int e = 0; e < JJ * U; ++e) {
        k.block[e] = half + 2 * W * (i0 + e / U);
        k.in[e] = (U == 1 || r + e % U < N) && (FULL || k.block[e] < nb);
      }
      if (KEEP && x_ckpt != nullptr) {
#pragma unroll
        for (int e = 0; e < JJ * U; ++e) {
          const Pack<KIND>& q = p[e % U][i0 + e / U];
          k.row[e] = xc + e % U * row_bytes;
          k.top[e] = q.top();
#pragma unroll
          for (int j = 0; j < 4; ++j) k.v[e][j] = q.at(j);
        }
        save8<VEC, FULL>(k, H, l);
      }
#pragma unroll
      for (int e = 0; e < JJ * U; ++e) {
        const int u = e % U, i = i0 + e / U;
        if (J > 2 && u == 0) {
          get_params(params + (2 * i) * threads * 32, threads, wv[0]);
          get_params(params + (2 * i + 1) * threads * 32, threads, bv[0]);
        }
        const F2(&wi)[4] = wv[J > 2 ? 0 : i], (&bi)[4] = bv[J > 2 ? 0 : i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          F2 v = fma2(mul2(add2(p[u][i].at(j), both(-m[u])), both(rs[u])), wi[j], bi[j]);
          if (!VEC)
            v = pair(half_col<false>(k.block[e], l, 2 * j) < H ? v.x() : 0.f,
                     half_col<false>(k.block[e], l, 2 * j + 1) < H ? v.y() : 0.f);
          else if (!there[i])
            v = both(0.f);
          k.v[e][j] = v;
        }
        k.row[e] = yc + u * row_bytes;
        k.top[e] = store8<T, VEC, FULL>(out + (long long)u * H, H, k.block[e], l, k.v[e], k.in[e]);
      }
      if (KEEP && y_ckpt != nullptr) save8<VEC, FULL>(k, H, l);
    }
    out += (long long)step * H;
    if (KEEP) {
      xc += step * row_bytes;
      yc += step * row_bytes;
    }
  }
}

template <typename T, int KIND, int XKIND, bool VEC, int J, int U>
__global__ void __launch_bounds__(kSmThreads)
    k_norm_dx(const T* __restrict__ dy, const void* __restrict__ x, const void* __restrict__ w,
              int p_type, const float* __restrict__ mean, const float* __restrict__ rstd, unsigned N,
              int H, int W, T* __restrict__ dx, float* __restrict__ ws) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int A = dx_ahead<KIND, XKIND, J, U>();
  extern __shared__ __align__(16) float s_dyn[];  // slots; at the end the groups' column sums
  __shared__ float s_sum[2][kMaxWarps * 2 * U];
  const int l = threadIdx.x % kHalf;
  const int group = (threadIdx.x >> 5) / W, groups = blockDim.x / (32 * W);
  const int warp = (threadIdx.x >> 5) - group * W, half = 2 * warp + ((threadIdx.x >> 4) & 1);
  const int threads = blockDim.x;
  const float inv_h = 1.f / H;
  F2 dw[J][4], db[J][4], held_w[J > 2 ? 1 : J][4];
  bool there[J];
  constexpr int piece = Slot<KIND>::bytes + Slot<XKIND>::bytes;  // a thread's bytes of a block
  const uint32_t slots = uint32_t(__cvta_generic_to_shared(s_dyn));
  const uint32_t params = slots + (VEC ? A : 1) * U * J * threads * piece;
  const auto weight = [&](int i) -> const F2(&)[4] {
    if (J > 2) get_params(params + i * threads * 32, threads, held_w[0]);
    return held_w[J > 2 ? 0 : i];
  };
#pragma unroll
  for (int i = 0; i < J; ++i) {
    there[i] = half_col<VEC>(half + 2 * W * i, l, 0) < H;
    load_params<VEC>(w, p_type, H, half + 2 * W * i, l, 1.f, held_w[J > 2 ? 0 : i]);
    if (J > 2) put_params(params + i * threads * 32, threads, held_w[0]);
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[i][j] = db[i][j] = both(0.f);
  }
  const unsigned first = (blockIdx.x * groups + group) * U, step = gridDim.x * groups * U;
  const char* dsrc = Slot<KIND>::at(dy, half_col<true>(half, l, 0)) + first * Slot<KIND>::pitch(H);
  const char* xsrc = Slot<XKIND>::at(x, half_col<true>(half, l, 0)) + first * Slot<XKIND>::pitch(H);
  const long long dstep = step * Slot<KIND>::pitch(H), xstep = step * Slot<XKIND>::pitch(H);
  const auto ahead = [&](unsigned r, uint32_t slot) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = r + u < N;
      if (in || u > 0) {  // (a row beyond the last beside one before it: zeros, so that no sum has to ask)
        const char *drow = dsrc + u * Slot<KIND>::pitch(H), *xrow = xsrc + u * Slot<XKIND>::pitch(H);
#pragma unroll
        for (int i = 0; i < J; ++i)
          if (there[i]) {
            const uint32_t s = slot + (u * J + i) * threads * piece, sx = s + threads * Slot<KIND>::bytes;
            if (u > 0 && !in) {
              Slot<KIND>::zero(s, threads);
              Slot<XKIND>::zero(sx, threads);
            } else {
              Slot<KIND>::copy(s, threads, drow + 2 * W * i * 16 * Slot<KIND>::bytes);
              Slot<XKIND>::copy(sx, threads, xrow + 2 * W * i * 16 * Slot<XKIND>::bytes);
            }
          }
      }
    }
    dsrc += dstep;
    xsrc += xstep;
    copy_async_commit();
  };
  // what is one value a row, a turn ahead in registers
  float m1[U], rs1[U];
  int sb1[U][J];
  const float *mp = mean + first, *rp = rstd + first;
  const uint8_t* sp = static_cast<const uint8_t*>(x) + first * ckpt_row_bytes(H) + ckpt_scale_at(H) + half;
  const auto scalars = [&](unsigned r) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = r + u < N;
      m1[u] = in ? __ldg(mp + u) : 0.f;
      rs1[u] = in ? __ldg(rp + u) : 0.f;
      if (XKIND == MEP_CKPT8)
#pragma unroll
        for (int i = 0; i < J; ++i)
          sb1[u][i] = in && there[i] ? __ldg(sp + u * ckpt_row_bytes(H) + 2 * W * i) : 1;
    }
    mp += step;
    rp += step;
    if (XKIND == MEP_CKPT8) sp += step * ckpt_row_bytes(H);
  };
  if (VEC) {
#pragma unroll
    for (int i = 0; i < J; ++i)
      if (!there[i])
        for (int k = 0; k < A * U; ++k) {
          const uint32_t s = slots + (k * J + i) * threads * piece;
          Slot<KIND>::zero(s, threads);
          Slot<XKIND>::zero(s + threads * Slot<KIND>::bytes, threads);
        }
    for (int k = 0; k < A; ++k) ahead(first + k * step, slots + k * U * J * threads * piece);
  }
  scalars(first);
  T* out = dx + (long long)first * H;
  int at = 0, turn = 0;  // slot, sums
  for (unsigned r = first; r < N; r += step, turn ^= 1) {
    const uint32_t slot = slots + at * U * J * threads * piece;
    float m[U], rs[U], sums[2 * U];
    int sb[U][J];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      m[u] = m1[u];
      rs[u] = rs1[u];
#pragma unroll
      for (int i = 0; i < J; ++i) sb[u][i] = sb1[u][i];
    }
    // both passes fetch a row's values anew from the slots (two loads a vector);
    // values that had to be loaded one by one are put there by the first (fp32
    // [32768, 2047] 195 -> 148 us)
    const auto fetch = [&](int u, int i, bool first_pass, Pack<KIND>& d, Pack<XKIND>& p) {
      const uint32_t s = slot + (u * J + i) * threads * piece, sx = s + threads * Slot<KIND>::bytes;
      if (VEC || !first_pass) {
        Slot<KIND>::fetch(s, threads, d);
        Slot<XKIND>::fetch(sx, threads, p);
        if constexpr (XKIND == MEP_CKPT8) p.step = ckpt_step(sb[u][i]);
      } else {
        d.template load<false>(dy, r + u, H, half + 2 * W * i, l);
        p.template load<false>(x, r + u, H, half + 2 * W * i, l);
        Slot<KIND>::put(s, threads, d);
        Slot<XKIND>::put(sx, threads, p);
      }
    };
    if (VEC) {
      copy_async_wait<A - 1>();
    } else {
      rows_to_l2<U>(dy, r + kTurnsToL2 * step, N, Slot<KIND>::pitch(H), threadIdx.x - group * 32 * W, 32 * W);
      rows_to_l2<U>(x, r + kTurnsToL2 * step, N, Slot<XKIND>::pitch(H), threadIdx.x - group * 32 * W, 32 * W);
    }
    scalars(r + step);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      F2 s1 = both(0.f), s2 = both(0.f);
      {
        const F2 k1 = both(rs[u]), k0 = both(-m[u]);
#pragma unroll
        for (int i = 0; i < J; ++i) {
          Pack<KIND> d;
          Pack<XKIND> p;
          fetch(u, i, true, d, p);
          const F2(&wv)[4] = weight(i);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // (x - mean) first: exact where the row is far from zero
            const F2 g = d.at(j), xhat = mul2(p.plus(j, k0), k1), t = mul2(g, wv[j]);
            s1 = add2(s1, t);
            s2 = fma2(t, xhat, s2);
            dw[i][j] = fma2(g, xhat, dw[i][j]);
            db[i][j] = add2(db[i][j], g);
          }
        }
      }
      sums[u] = s1.x() + s1.y();
      sums[U + u] = s2.x() + s2.y();
    }
    group_sums<2 * U>(sums, &s_sum[turn][group * W * 2 * U], W, warp, group);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      {
        // rs (t - c1 - xhat c2), with xhat rs = (x - m) rs^2
        const F2 k1 = both(rs[u]), k0 = both(-m[u]);
        const F2 a = both(-rs[u] * sums[u] * inv_h), c = both(-rs[u] * sums[U + u] * inv_h * rs[u]);
#pragma unroll
        for (int i = 0; i < J; ++i) {
          Pack<KIND> d;
          Pack<XKIND> p;
          fetch(u, i, false, d, p);
          const F2(&wv)[4] = weight(i);
          F2 v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            v[j] = fma2(p.plus(j, k0), c, fma2(mul2(d.at(j), wv[j]), k1, a));
          store8<T, VEC>(out + (long long)u * H, H, half + 2 * W * i, l, v, U == 1 || r + u < N);
        }
      }
    }
    out += (long long)step * H;
    if (VEC) {
      ahead(r + A * step, slot);
      at = at + 1 == A ? 0 : at + 1;
    }
  }
  if (ws == nullptr) return;
  // join the groups' column sums: laid out by thread, then by value
  const int mine = 32 * W, tid = threadIdx.x - group * mine, cols = mine * 8 * J;
  if (groups > 1) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int i = 0; i < J; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float* a = s_dyn + (2 * group) * cols + (8 * i + 2 * j) * mine + tid;
        a[0] = dw[i][j].x(), a[mine] = dw[i][j].y();
        a[cols] = db[i][j].x(), a[cols + mine] = db[i][j].y();
      }
    __syncthreads();
    if (group != 0) return;
    for (int g = 1; g < groups; ++g)
#pragma unroll
      for (int i = 0; i < J; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float* a = s_dyn + (2 * g) * cols + (8 * i + 2 * j) * mine + tid;
          dw[i][j] = add2(dw[i][j], pair(a[0], a[mine]));
          db[i][j] = add2(db[i][j], pair(a[cols], a[cols + mine]));
        }
  }
  float* part = ws + (long long)blockIdx.x * 2 * H;
#pragma unroll
  for (int i = 0; i < J; ++i) {
    store8<float, VEC>(part, H, half + 2 * W * i, l, dw[i]);
    store8<float, VEC>(part + H, H, half + 2 * W * i, l, db[i]);
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

// The default limit of 48 KB holds for dynamic and static shared memory together.
int allow_smem(const void* kernel, int bytes) {
  return set_max_dynamic_smem(kernel, bytes > 44 * 1024 && bytes <= 48 * 1024 ? 48 * 1024 + 1 : bytes);
}

// How a row is laid out: J blocks a half warp, W warps a row, U rows a turn,
// `groups` rows' worth of warps in a CTA.
struct Shape {
  int J, U, W, groups, threads, parts;
};
Shape shape_of(long long N, int H, int J, int U) {
  Shape s;
  s.J = J;
  s.U = U;
  s.W = ceil_div(ceil_div(H, kCkptBlock), 2 * J);
  // as many rows as fit 512 threads, but rather a CTA for every SM
  s.groups = s.W >= 16 ? 1 : 16 / s.W;
  while (s.groups > 1 && N < 152ll * U * s.groups) s.groups /= 2;
  s.threads = 32 * s.W * s.groups;
  return s;
}
// Blocks a half warp: one where a row has no more than two, else two, and four
// for rows of more than 8192 columns (backward [16384, 12288] 345 us before the
// weights went to shared memory; with two blocks, 1024 threads and half the
// registers 483). Four also (`four`) where a row would take 9 or 10 warps, 4097
// to 5120 columns, of which an SM has room for 16; at 12 warps, [20000, 6144],
// the bf16 backward pass from 8 bits took 152 us with four and 142 with two.
// Over those widths, of 20000 rows, in us with four and with two:
//   forward     bf16 84-91 and 88-113, fp32 115-133 and 147-162, odd widths
//               137-158 and 215-240; with one or two checkpoints alike
//   backward    bf16 103-115 and 111-125, from 8 bits 117-122 and 131-135,
//               odd widths 201-223 and 257-281, but from 8 bits 303-317 and
//               275-297: two
//               fp32 179-197 and 177-197, from 8 bits 193-211 and 162-177,
//               odd widths 255-332 and 234-262: two
int blocks_of(int H, bool four) {
  const int nb = ceil_div(H, kCkptBlock), warps = ceil_div(nb, 4);
  return nb <= 2 ? 1 : warps > 16 || (four && (warps == 9 || warps == 10)) ? 4 : 2;
}
// Two rows a turn in bf16, up to two blocks: their sums share one barrier and
// most of their shuffles (forward [32768, 2048] 49 us, one row a turn 62;
// backward [65536, 7168] 443 and 552). In fp32 a row is twice the bytes and two
// gain nothing (134 and 135 us). The number of CTAs must not depend on the
// device: the workspace is sized by it.
Shape backward_shape(long long N, int H, int type, int x_type) {
  const int J = blocks_of(H, type == MEP_BF16 && (H % 8 == 0 || x_type != MEP_CKPT8));
  Shape s = shape_of(N, H, J, type == MEP_BF16 && H % 8 == 0 && J <= 2 ? 2 : 1);
  const int want = ceil_div(N < 1 ? 1 : N, s.U * s.groups), cap = 152 * (kSmThreads / s.threads);
  s.parts = want < cap ? want : cap;
  return s;
}
// The most CTAs of any call of up to N rows. They are not most at N itself:
// with fewer rows a CTA holds fewer row groups, and up to three times as many
// CTAs fit. A workspace for the longest batch has to serve every shorter one.
int backward_parts(long long N, int H, int type, int x_type) {
  int most = 0;
  for (;;) {
    const Shape s = backward_shape(N, H, type, x_type);
    most = s.parts > most ? s.parts : most;
    if (s.groups == 1) return most;
    N = 152ll * s.U * s.groups - 1;  // the longest call of smaller CTAs: with as large ones, fewer rows take fewer
  }
}

template <typename T, int KIND, bool VEC, bool FULL, bool KEEP, int J, int U>
cudaError_t run_norm(const Shape& s, const void* x, const void* w, const void* b, int p_type, float eps,
                     unsigned N, int H, void* y, float* mean, float* rstd, uint8_t* xc, uint8_t* yc,
                     cudaStream_t st) {
  const int want = ceil_div(N, s.groups * U), cap = sm_count() * (kSmThreads / s.threads);
  const int smem = s.threads * ((VEC ? norm_ahead<KIND, J, U>() * U * J * Slot<KIND>::bytes : 0) + 2 * kParamBytes<J>);
  const auto kernel = k_norm<T, KIND, VEC, FULL, KEEP, J, U>;
  if (allow_smem(reinterpret_cast<const void*>(kernel), smem)) return cudaErrorInvalidValue;
  return launch_pdl(kernel, dim3(want < cap ? want : cap), dim3(s.threads), smem, st,
                    static_cast<const T*>(x), w, b, p_type, eps, N, H, s.W, static_cast<T*>(y), mean,
                    rstd, xc, yc);
}

template <typename T, int KIND, bool VEC>
cudaError_t pick_norm(const void* x, const void* w, const void* b, int p_type, float eps, unsigned N,
                      int H, void* y, float* mean, float* rstd, uint8_t* xc, uint8_t* yc,
                      cudaStream_t st) {
  constexpr int U = KIND == MEP_BF16 ? 2 : 1;
  const int J = blocks_of(H, true);
  const Shape s = shape_of(N, H, J, U);
  // Without the edge and checkpoint tests the forward pass issues a fifth less
  // ([32768, 2048] 61 -> 51 us, [65536, 7168] 404 -> 334 us); the backward
  // pass, which waits for memory, ran the same either way.
  const bool full = VEC && H == s.W * 2 * J * kCkptBlock, keep = xc != nullptr || yc != nullptr;
  const auto run = J == 1   ? run_norm<T, KIND, VEC, false, true, 1, U>
                   : J == 4 ? run_norm<T, KIND, VEC, false, true, 4, U>
                   : full   ? (keep ? run_norm<T, KIND, VEC, VEC, true, 2, U>
                                    : run_norm<T, KIND, VEC, VEC, false, 2, U>)
                            : run_norm<T, KIND, VEC, false, true, 2, U>;
  return run(s, x, w, b, p_type, eps, N, H, y, mean, rstd, xc, yc, st);
}

template <typename T, int KIND, int XKIND, bool VEC, int J, int U>
cudaError_t run_dx(const Shape& s, const void* dy, const void* x, const void* w, int p_type,
                   const float* mean, const float* rstd, unsigned N, int H, void* dx, float* ws,
                   cudaStream_t st) {
  const int threads = s.threads;
  const int slots = threads * ((VEC ? dx_ahead<KIND, XKIND, J, U>() : 1) * U * J *
                                   (Slot<KIND>::bytes + Slot<XKIND>::bytes) + kParamBytes<J>);
  const int join = s.groups > 1 ? 2 * threads * 8 * J * 4 : 0, smem = slots > join ? slots : join;
  const auto kernel = k_norm_dx<T, KIND, XKIND, VEC, J, U>;
  if (allow_smem(reinterpret_cast<const void*>(kernel), smem)) return cudaErrorInvalidValue;
  return launch_pdl(kernel, dim3(s.parts), dim3(threads), smem, st, static_cast<const T*>(dy), x, w,
                    p_type, mean, rstd, N, H, s.W, static_cast<T*>(dx), ws);
}

template <typename T, int KIND, int XKIND, bool VEC>
cudaError_t pick_dx(const Shape& s, const void* dy, const void* x, const void* w, int p_type,
                    const float* mean, const float* rstd, unsigned N, int H, void* dx, float* ws,
                    cudaStream_t st) {
  constexpr int U = KIND == MEP_BF16 && VEC ? 2 : 1;  // as backward_shape has it
  const auto run = s.J == 1   ? run_dx<T, KIND, XKIND, VEC, 1, U>
                   : s.J == 2 ? run_dx<T, KIND, XKIND, VEC, 2, U>
                              : run_dx<T, KIND, XKIND, VEC, 4, 1>;
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
  if (!may_start(x, x_type, H) || !may_start(y, x_type, H) || !may_start(weight, p_type, H) ||
      !may_start(bias, p_type, H) || !may_start(mean, MEP_F32, H) || !may_start(rstd, MEP_F32, H) ||
      !aligned16(x_ckpt) || !aligned16(y_ckpt))
    return MEP_ERR_INVALID_ARG;
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
  int most = 0;
  for (int type : {MEP_BF16, MEP_F32})
    for (int x_type : {type, MEP_CKPT8}) {
      const int n = backward_parts(N, int(H), type, x_type);
      most = n > most ? n : most;
    }
  *bytes = size_t(most) * 2 * H * sizeof(float);
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
  if (!may_start(dy, dy_type, H) || !may_start(x, x_type, H) || !may_start(dx, dy_type, H) ||
      !may_start(weight, p_type, H) || !may_start(mean, MEP_F32, H) || !may_start(rstd, MEP_F32, H) ||
      !may_start(dweight, MEP_F32, H) || !may_start(dbias, MEP_F32, H) || !aligned16(ws))
    return MEP_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Shape s = backward_shape(N, int(H), dy_type, x_type);
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
