// grouped_wgrad.cu -- the experts' weight gradients over the static buffer
// (mep_grouped_wgrad), on the sm_100-family tensor cores (tcgen05 + TMA).
//
// Source: "月之暗面开源MoonEP：面向MoE训练的专家并行通信库", section
// 内存契约与权重布局: the weights of one projection are one [E+B, H, H']
// tensor, gradients are fp32, those of the prefetch slots lie in a buffer of
// their own seen as [R, B, H, H'], which mep_reduce_grad folds into the home
// experts' gradients.
//
// dW_j[h, n] = sum over the rows of group j of x[row, h] * dy[row, n]: a
// product whose inner dimension is the ragged one. Both operands lie with the
// outer dimension contiguous (M- and N-major), so TMA boxes of 64 rows x 64
// columns are tensor-core operands as they come.
//
// Two launches on the caller's stream:
//   k_wgrad_groups  (1 CTA) checks every cu_seqlens row and lists the weight
//                   rows that have to be written, each with its row segments
//                   (one per rank that has rows of it);
//   k_wgrad_pair    persistent clusters of two CTAs, one per SM, 512 threads
//                   each, over units (weight row, 256 rows of H, 256 columns
//                   of H'), grid-stride. CTA r of a pair owns 128 of the 256
//                   rows of H. Per step of 64 buffer rows:
//     warp 0      TMA producer: this CTA's 128 columns of x (bf16 boxes, or
//                 the checkpoint's bytes and their 64 scale bytes) and its
//                 half of the 256 columns of dy, into a ring of stages;
//     warps 4..7  converter: checkpoint bytes to bf16 operand boxes (exact:
//                 q * 2^k has 8 significant bits), and zeros over the rows
//                 that a segment's last step takes from the next group, in
//                 both operands (a NaN there would survive a product with 0);
//     warp 1      of CTA 0 issues the pair MMAs (tcgen05.mma.cta_group::2,
//                 M = 256, N = 256 or 128, K = 16) into one of two TMEM
//                 accumulators, which changes every kChunk steps;
//     warps 8..15 add each finished accumulator to fp32 sums in registers
//                 (128 a thread), and at the end of the unit write them
//                 through shared memory with bulk tensor stores, or bulk
//                 tensor additions.
// The sums leave TMEM every kChunk * 64 rows because the tensor cores do not
// round their fp32 additions to nearest: over a long group the error of one
// accumulator grows with the number of steps, that of the registers' sums,
// rounded to nearest, with its root.
// Every wait is bounded as in grouped_gemm.cu.

#include "ckpt.cuh"
#include "tc.cuh"

#ifndef MEP_WGRAD_CHUNK
#define MEP_WGRAD_CHUNK 8
#endif

namespace mep {
namespace {

constexpr int kBM = 128;                 // rows of H per CTA
constexpr int kBN = 256;                 // columns of H' per pair
constexpr int kBK = 64;                  // buffer rows per step
constexpr int kBox = kBK * 64 * 2;       // one 64 x 64 bf16 box, 8 KB
constexpr int kOp = 2 * kBox;            // an operand's two boxes, 16 KB
constexpr int kQ = kBK * kBM;            // checkpoint bytes of a step, 8 KB
constexpr int kScale = kBK * 16;         // their scale bytes, in 16-byte rows
constexpr int kChunk = MEP_WGRAD_CHUNK;  // steps summed in TMEM
constexpr int kThreads = 512;
constexpr int kTmemCols = 2 * kBN;
constexpr int kGroupThreads = 1024;
constexpr int kStoreBox = 32 * 32 * 4;   // 32 rows x 32 fp32 columns
constexpr int kEpiWarps = 8;
constexpr int kPair = 2;

template <bool CKPT> struct Ring {
  static constexpr int stage = 2 * kOp + (CKPT ? kQ + kScale : 0);
  static constexpr int stages = CKPT ? 4 : 6;
  static constexpr int smem = 1024 /* alignment slack */ + stages * stage + kEpiWarps * kStoreBox + 512;
  static_assert(smem <= 232448, "the ring must fit in 227 KB of shared memory");
};

struct Smem {
  uint64_t full[6], ready[6], empty[6], tfull[2], tempty[2], drain;
  uint32_t tmem;
  int abort;
  int count;
};

// wait_phase for a whole warp, without a call (the roles hold their state in
// registers across it), with long tries and the same answer for all lanes.
template <bool HONOR = true>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                          int32_t* status) {
  bool ok = mbar_try_wait_long(bar, parity);
  uint64_t t0 = 0;
  while (!ok) {
#pragma unroll 1
    for (int i = 0; i < 16 && !ok; ++i) ok = mbar_try_wait_long(bar, parity);
    if (ok || (HONOR && *abort)) break;
    const uint64_t now = globaltimer();
    if (t0 == 0) {
      t0 = now;
    } else if (now - t0 > MEP_GEMM_TIMEOUT_NS) {
      *abort = 1;
      set_status(status, MEP_ERR_TIMEOUT);
      break;
    }
  }
  return __all_sync(MEP_FULL_MASK, ok);
}
// Lane 0's value: the same for the warp, and known to be.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(MEP_FULL_MASK, v, 0); }
// One lane of a converged warp.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, int x, int y, int z,
                                             uint32_t src) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];\n\t"
      "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(x), "r"(y), "r"(z), "r"(src)
      : "memory");
}
__device__ __forceinline__ void tma_add_3d(const CUtensorMap* map, int x, int y, int z,
                                           uint32_t src) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.bulk_group [%0, {%1, %2, %3}], [%4];\n\t"
      "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(x), "r"(y), "r"(z), "r"(src)
      : "memory");
}
// Arrival on a barrier of another CTA of the cluster, ordered after this
// thread's own work at CTA scope: what the other CTA's MMA issuer goes on to
// start reads this CTA's operands and TMEM on this CTA's own SM, and the
// writes to them were closed by fence.proxy.async or tcgen05.fence before. (A
// release at cluster scope waits for a round trip to L2: 1250 cycles, on a
// step of 512.)
__device__ __forceinline__ void mbar_arrive_remote(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}
__device__ __forceinline__ void bulk_wait_read_0() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// bf16 in, fp32 accumulate, A and B both with their outer dimension contiguous.
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
                            ((uint32_t)(kBN >> 3) << 17) | ((uint32_t)(256 >> 4) << 24);
constexpr uint32_t kIdescN = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
                             ((uint32_t)(128 >> 3) << 17) | ((uint32_t)(256 >> 4) << 24);

// ---------------------------------------------------------------------------
// The weight rows to write, weight row < E a home expert and E + r*B + b slot
// b of rank r: entries[2i] = {weight row, first segment, segments, steps},
// entries[2i + 1] = {first segment's first buffer row, its rows, 0, 0};
// segs[j] = {first buffer row, rows}. Without `accumulate` a home expert is
// listed even without rows (it is written as zero), a slot never is.
__global__ void __launch_bounds__(kGroupThreads)
    k_wgrad_groups(const int32_t* __restrict__ cu, int R, int E, int B, int SK, int accumulate,
                   int32_t* status, int* __restrict__ count, int4* __restrict__ entries,
                   int2* __restrict__ segs) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ int s_warp[33], s_entry[kGroupThreads + 1], s_seg[kGroupThreads + 1];
  __shared__ int s_bad, s_entries, s_segs, s_stat;
  const int G = E + B;
  if (threadIdx.x == 0) {
    s_bad = s_entries = s_segs = 0;
    s_stat = read_status(status);
  }
  __syncthreads();
  if (s_stat != 0) {
    if (threadIdx.x == 0) *count = 0;
    return;
  }
  for (long long p = threadIdx.x; p < (long long)R * G; p += blockDim.x) {
    const int j = int(p % G), v = cu[p], prev = j == 0 ? 0 : cu[p - 1];
    if (v < prev || (j == G - 1 && v != SK)) s_bad = 1;
  }
  __syncthreads();
  if (s_bad) {
    if (threadIdx.x == 0) {
      *count = 0;
      set_status(status, MEP_ERR_BAD_SEQLENS);
    }
    return;
  }
  const int W = E + R * B;
  for (int base = 0; base < W; base += blockDim.x) {
    const int w = base + threadIdx.x;
    const bool home = w < E;
    const int j = home ? w : (w < W ? E + (w - E) % B : 0);
    const int r0 = home ? 0 : (w < W ? (w - E) / B : 0), r1 = w < W ? (home ? R : r0 + 1) : r0;
    int nseg = 0, steps = 0;
    for (int r = r0; r < r1; ++r) {
      const long long p = (long long)r * G + j;
      const int len = cu[p] - (j == 0 ? 0 : cu[p - 1]);
      nseg += len > 0;
      steps += (len + kBK - 1) / kBK;
    }
    const bool listed = w < W && (nseg > 0 || (home && !accumulate));
    s_entry[threadIdx.x] = listed;
    s_seg[threadIdx.x] = nseg;
    __syncthreads();
    block_excl_scan(s_entry, s_entry, blockDim.x, s_warp, true);
    block_excl_scan(s_seg, s_seg, blockDim.x, s_warp, true);
    if (listed) {
      int at = s_segs + s_seg[threadIdx.x];
      int4* entry = entries + 2 * (s_entries + s_entry[threadIdx.x]);
      entry[0] = make_int4(w, at, nseg, steps);
      entry[1] = make_int4(0, 0, 0, 0);
      for (int r = r0; r < r1; ++r) {
        const long long p = (long long)r * G + j;
        const int lo = j == 0 ? 0 : cu[p - 1], len = cu[p] - lo;
        if (len > 0) {
          const int row = int((long long)r * SK + lo);
          if (entry[1].y == 0) entry[1] = make_int4(row, len, 0, 0);
          segs[at++] = make_int2(row, len);
        }
      }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      s_entries += s_entry[blockDim.x];
      s_segs += s_seg[blockDim.x];
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) *count = s_entries;
}

// Two signed bytes of w (chosen by sel) times a power of two, as two bf16.
// The bytes are placed under 0x43 (bf16 128 + low seven bits, or 256 + ...
// where the sign bit is set): v = 128 + low7, c = 128 or 256, v - c = q
// exactly, and q * step has 8 significant bits.
__device__ __forceinline__ uint32_t dequant2(uint32_t w, uint32_t sel, __nv_bfloat162 step) {
  const uint32_t x = __byte_perm(w, 0x43434343u, sel);
  const uint32_t v = x & 0xff7fff7fu, c = x & 0xff80ff80u;
  const __nv_bfloat162 q = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                   *reinterpret_cast<const __nv_bfloat162*>(&c));
  const __nv_bfloat162 r = __hmul2(q, step);
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ void lds64(uint32_t addr, uint32_t& a, uint32_t& b) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr));
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// The units of one CTA pair, in the order in which every role of both CTAs
// walks them (whole warps: what steers the loops is the same for all lanes,
// and known to be, so that addresses and descriptors stay in uniform
// registers). The next unit's entry is loaded while f works on this one's;
// f(entry, tile) returns false to stop.
struct Entry {
  int4 e;       // {weight row, first segment, segments, steps}
  int row, len; // the first segment
};
__device__ __forceinline__ Entry load_entry(const int4* __restrict__ entries, int i) {
  const int4 a = entries[2 * i], b = entries[2 * i + 1];
  return {a, b.x, b.y};
}
__device__ __forceinline__ Entry uniform(const Entry& e) {
  return {make_int4(uniform(e.e.x), uniform(e.e.y), uniform(e.e.z), uniform(e.e.w)), uniform(e.row),
          uniform(e.len)};
}
template <typename F>
__device__ __forceinline__ void for_units(const int4* __restrict__ entries, int count, int tiles, F f) {
  const int step = gridDim.x / 2;
  int i = (blockIdx.x / 2) / tiles, tile = (blockIdx.x / 2) % tiles;
  if (i >= count) return;
  Entry cur = uniform(load_entry(entries, i)), next = cur;
  for (;;) {
    const int t = tile + step, ni = i + t / tiles;
    if (ni < count) next = load_entry(entries, ni);
    if (!f(cur, tile) || ni >= count) return;
    cur = uniform(next);
    i = ni;
    tile = t % tiles;
  }
}
// The steps of one unit: f(first buffer row, rows left from it on) per step.
template <typename F>
__device__ __forceinline__ bool for_steps(const Entry& en, const int2* __restrict__ segs, F f) {
  int row = en.row, len = en.len;
  for (int g = 0; g < en.e.z; ++g) {
    if (g > 0) {
      const int2 seg = segs[en.e.y + g];
      row = uniform(seg.x);
      len = uniform(seg.y);
    }
    for (int k = 0; k < len; k += kBK)
      if (!f(row + k, len - k)) return false;
  }
  return true;
}
// A ring position: stage and the parity of its round.
struct Pos {
  uint32_t s = 0, parity = 0;
  template <int N> __device__ __forceinline__ void next() {
    if (++s == N) {
      s = 0;
      parity ^= 1u;
    }
  }
};

// ---------------------------------------------------------------------------
template <bool CKPT>
__global__ void __launch_bounds__(kThreads, 1)
    k_wgrad_pair(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_s,
                 const __grid_constant__ CUtensorMap map_dy, const __grid_constant__ CUtensorMap map_home,
                 const __grid_constant__ CUtensorMap map_slot, const int* __restrict__ count_ptr,
                 const int4* __restrict__ entries, const int2* __restrict__ segs, int32_t* status,
                 int E, int H, int Hp, int accumulate) {
  constexpr int kSt = Ring<CKPT>::stages, kStage = Ring<CKPT>::stage;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gen_base = smem_raw + (base - raw);
  const uint32_t out_box = base + kSt * kStage;
  Smem* S = reinterpret_cast<Smem*>(gen_base + kSt * kStage + kEpiWarps * kStoreBox);
  volatile int* abort_flag = &S->abort;

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int rank = uniform(int(cluster_rank()));
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kSt; ++s) {
      mbar_init(smem_u32(&S->full[s]), 1);   // this CTA's producer and its bytes
      mbar_init(smem_u32(&S->ready[s]), 8);  // CTA 0: four converter warps of each CTA
      mbar_init(smem_u32(&S->empty[s]), 1);  // CTA 0's multicast commit
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&S->tfull[a]), 1);
      mbar_init(smem_u32(&S->tempty[a]), 2 * kEpiWarps);
    }
    mbar_init(smem_u32(&S->drain), 1);
    S->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&S->tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  if (threadIdx.x == 0) S->count = read_status(status) != 0 ? 0 : *count_ptr;
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = uniform(S->tmem);
  const int nM = (H + 2 * kBM - 1) / (2 * kBM), nN = (Hp + kBN - 1) / kBN;
  const int tiles = nM * nN, count = uniform(S->count);

  // the four warpgroups' registers: 56 + 72 + 192 + 192 = 4 x 128 at launch
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      // ---------------- TMA producer ----------------
      Pos at;
      uint32_t issued = 0;
      for_units(entries, count, tiles, [&](const Entry& en, int t) {
        const int h0 = t / nN * 2 * kBM + rank * kBM, n0 = t % nN * kBN;
        const bool narrow = Hp - n0 <= 128;
        const int c0 = n0 + rank * (narrow ? 64 : 128);
        const int na = h0 >= H ? 0 : h0 + 64 < H ? 2 : 1;
        const int nb = c0 >= Hp ? 0 : !narrow && c0 + 64 < Hp ? 2 : 1;
        const uint32_t bytes = (CKPT ? (na > 0 ? kQ + kScale : 0) : na * kBox) + nb * kBox;
        const int sx = ckpt_scale_at(H) + ((h0 / kCkptBlock) & ~15);
        return for_steps(en, segs, [&](int row, int) {
          if (!warp_wait(smem_u32(&S->empty[at.s]), at.parity ^ 1u, abort_flag, status)) return false;
          const uint32_t bar = smem_u32(&S->full[at.s]), st = base + at.s * kStage;
          if (elected()) {
            mbar_expect_tx(bar, bytes);
            if (CKPT) {
              if (na > 0) {
                tma_load_2d(st + 2 * kOp, &map_x, h0, row, bar);
                tma_load_2d(st + 2 * kOp + kQ, &map_s, sx, row, bar);
              }
            } else {
              if (na > 0) tma_load_2d(st, &map_x, h0, row, bar);
              if (na > 1) tma_load_2d(st + kBox, &map_x, h0 + 64, row, bar);
            }
            if (nb > 0) tma_load_2d(st + kOp, &map_dy, c0, row, bar);
            if (nb > 1) tma_load_2d(st + kOp + kBox, &map_dy, c0 + 64, row, bar);
          }
          __syncwarp();
          at.template next<kSt>();
          ++issued;
          return true;
        });
      });
      // this CTA's copies have landed, and every commit aimed at it has arrived
      for (uint32_t j = issued > kSt ? issued - kSt : 0; j < issued; ++j) {
        warp_wait<false>(smem_u32(&S->full[j % kSt]), (j / kSt) & 1u, abort_flag, status);
        warp_wait<false>(smem_u32(&S->empty[j % kSt]), (j / kSt) & 1u, abort_flag, status);
      }
    } else if (warp == 1 && leader) {
      // ---------------- MMA issuer (CTA 0 only) ----------------
      Pos at, acc;  // stage; accumulator
      const uint64_t adesc = sdesc(base, kBox, 1024), bdesc = sdesc(base + kOp, kBox, 1024);
      for_units(entries, count, tiles, [&](const Entry& en, int t) {
        const uint32_t idesc = Hp - t % nN * kBN <= 128 ? kIdescN : kIdesc;
        int steps = en.e.w, in_chunk = 0;
        return for_steps(en, segs, [&](int, int left) {
          if (in_chunk == 0 &&
              !warp_wait(smem_u32(&S->tempty[acc.s]), acc.parity ^ 1u, abort_flag, status))
            return false;
          if (!warp_wait(smem_u32(&S->ready[at.s]), at.parity, abort_flag, status)) return false;
          tc_fence_after();
          const uint32_t d = tmem + acc.s * kBN;
          const uint64_t ad = adesc + (at.s * kStage >> 4), bd = bdesc + (at.s * kStage >> 4);
          const bool last = in_chunk == kChunk - 1 || steps == 1;
          if (elected()) {
            if (left > kBK - 16) {
#pragma unroll
              for (int kk = 0; kk < kBK / 16; ++kk)
                tc_mma2(d, ad + kk * 128, bd + kk * 128, kk > 0 ? 1u : (uint32_t)in_chunk, idesc);
            } else {
              for (int kk = 0; 16 * kk < left; ++kk)
                tc_mma2(d, ad + kk * 128, bd + kk * 128, uint32_t(kk + in_chunk), idesc);
            }
            tc_commit2_mc(smem_u32(&S->empty[at.s]), 3);
            if (last) tc_commit2_mc(smem_u32(&S->tfull[acc.s]), 3);
          }
          __syncwarp();
          at.template next<kSt>();
          --steps;
          ++in_chunk;
          if (last) {
            acc.template next<2>();
            in_chunk = 0;
          }
          return true;
        });
      });
      if (elected()) tc_commit2(smem_u32(&S->drain));
      __syncwarp();
      warp_wait<false>(smem_u32(&S->drain), 0u, abort_flag, status);
    }
  } else if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    // ---------------- converter ----------------
    // Thread t takes columns [8c, 8c + 8) and [64 + 8c, 64 + 8c + 8), c = t & 7,
    // of four rows: two 8-byte reads and two 16-byte stores, chunk c of either
    // operand box. All boxes are 128-byte swizzled. A quarter warp stores to
    // the eight chunks of one row; a half warp reads half of two rows that
    // differ in bit 2, whose swizzle puts them into different halves.
    const int t = threadIdx.x - 128, c8 = t & 7;
    const int row0 = (lane >> 4) + ((lane >> 3) & 1) * 4 + (warp & 1) * 2 + ((warp >> 1) & 1) * 8;
    Pos at;
    for_units(entries, count, tiles, [&](const Entry& en, int tile) {
      const int h0 = tile / nN * 2 * kBM + rank * kBM;
      const uint32_t sbyte = (uint32_t)(h0 / kCkptBlock) & 15u;
      return for_steps(en, segs, [&](int, int left) {
          if (!warp_wait(smem_u32(&S->full[at.s]), at.parity, abort_flag, status)) return false;
          const uint32_t st = base + at.s * kStage;
          const int valid = min(kBK, left), need = (valid + 15) & ~15;
          if (CKPT) {
            if (h0 < H) {
              const uint32_t q = st + 2 * kOp, sc = q + kQ;
              uint32_t v[4][4], sb[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int row = row0 + 16 * i;
#pragma unroll
                for (int half = 0; half < 2; ++half)
                  lds64(q + row * 128 + (((4 * half + (c8 >> 1)) ^ (row & 7)) << 4) + (c8 & 1) * 8,
                        v[i][2 * half], v[i][2 * half + 1]);
                asm volatile("ld.shared.u8 %0, [%1];" : "=r"(sb[i]) : "r"(sc + row * 16 + sbyte));
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int row = row0 + 16 * i;
                // rows of the next group: q times 0
                const uint32_t bits =
                    row < valid ? (sb[i] == (uint32_t)kCkptNan ? 0x7fffu : sb[i] << 7) * 0x10001u : 0u;
                const __nv_bfloat162 step = *reinterpret_cast<const __nv_bfloat162*>(&bits);
                const uint32_t dst = st + row * 128 + ((c8 ^ (row & 7)) << 4);
#pragma unroll
                for (int half = 0; half < 2; ++half)
                  sts128(dst + half * kBox, dequant2(v[i][2 * half], 0x4140, step),
                         dequant2(v[i][2 * half], 0x4342, step),
                         dequant2(v[i][2 * half + 1], 0x4140, step),
                         dequant2(v[i][2 * half + 1], 0x4342, step));
              }
            }
          }
          if (valid < need)  // whole rows: the swizzle stays within a row
            for (int i = t; i < (need - valid) * 32; i += 128) {
              const int row = valid + (i >> 5), piece = i & 31;
              if (CKPT && piece < 16) continue;
              sts128(st + (piece >> 3) * kBox + row * 128 + ((piece & 7) << 4), 0u, 0u, 0u, 0u);
            }
          if (CKPT || valid < need) fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(map_to_rank(smem_u32(&S->ready[at.s]), 0));
          at.template next<kSt>();
          return true;
      });
    });
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    // ---------------- sums and epilogue ----------------
    // Warp q + 4 * half holds TMEM lanes (rows of H) [32q, 32q + 32) and
    // columns [128 half, 128 half + 128) of the unit.
    const int q = warp & 3, half = (warp - 8) >> 2;
    const uint32_t box = out_box + (uint32_t)(warp - 8) * kStoreBox;
    Pos at;
    for_units(entries, count, tiles, [&](const Entry& en, int tile) {
      const int4 e = en.e;
      const int h = tile / nN * 2 * kBM + rank * kBM + 32 * q, n = tile % nN * kBN + 128 * half;
      const int chunks = (e.w + kChunk - 1) / kChunk;
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.f;
      for (int c = 0; c < chunks; ++c) {
        if (!warp_wait(smem_u32(&S->tfull[at.s]), at.parity, abort_flag, status)) return false;
        tc_fence_after();
        const uint32_t ta = tmem + at.s * kBN + 128 * half + ((uint32_t)(32 * q) << 16);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + 32 * i < Hp) {
            uint32_t v[32];
            tc_ld32_issue(ta + 32 * i, v);
            tc_ld_wait(v);
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[32 * i + j] += __uint_as_float(v[j]);
          }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(map_to_rank(smem_u32(&S->tempty[at.s]), 0));
        at.template next<2>();
      }
      const CUtensorMap* map = e.x < E ? &map_home : &map_slot;
      const int z = e.x < E ? e.x : e.x - E;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (h < H && n + 32 * i < Hp) {
          if (lane == 0) bulk_wait_read_0();
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            sts128(box + lane * 128 + ((j ^ (lane & 7)) << 4), __float_as_uint(acc[32 * i + 4 * j]),
                   __float_as_uint(acc[32 * i + 4 * j + 1]), __float_as_uint(acc[32 * i + 4 * j + 2]),
                   __float_as_uint(acc[32 * i + 4 * j + 3]));
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (accumulate)
              tma_add_3d(map, n + 32 * i, h, z, box);
            else
              tma_store_3d(map, n + 32 * i, h, z, box);
          }
        }
      return true;
    });
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (threadIdx.x == 0 && read_status(status) != 0) {
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 100000ull) {
    }
  }
  cluster_sync();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                 : "memory");
}

// ---------------------------------------------------------------------------
// host side
bool map_2d(CUtensorMap* m, CUtensorMapDataType type, const void* ptr, unsigned long long rows,
            unsigned long long cols, unsigned long long stride, unsigned box_cols, unsigned box_rows,
            CUtensorMapSwizzle swizzle) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {stride};
  const cuuint32_t box[2] = {box_cols, box_rows}, estr[2] = {1, 1};
  return fn(m, type, 2, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// fp32 [n, H, H'], boxes of 32 x 32: a third dimension keeps a box that
// hangs over the last rows of H out of the next matrix.
bool map_grad(CUtensorMap* m, float* ptr, unsigned long long n, unsigned long long H,
              unsigned long long Hp) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {Hp, H, n}, strides[2] = {Hp * 4, H * Hp * 4};
  const cuuint32_t box[3] = {32, 32, 1}, estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, ptr, dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool CKPT>
cudaError_t launch_wgrad(cudaStream_t st, const CUtensorMap& mx, const CUtensorMap& ms,
                         const CUtensorMap& md, const CUtensorMap& mh, const CUtensorMap& msl,
                         const int* count, const int4* entries, const int2* segs, int32_t* status,
                         int E, int H, int Hp, int accumulate) {
  static GridCache cache;
  void (*kernel)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, const int*,
                 const int4*, const int2*, int32_t*, int, int, int, int) = k_wgrad_pair<CKPT>;
  if (set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), Ring<CKPT>::smem))
    return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kPair;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Ring<CKPT>::smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int grid = 0;
  {
    std::lock_guard<std::mutex> lock(cache.mu);
    if (cache.grid[dev] == 0) {
      // The warpgroups share out 512 x 128 registers: with fewer at launch
      // setmaxnreg would wait for ever.
      cudaFuncAttributes fa;
      cudaError_t e = cudaFuncGetAttributes(&fa, reinterpret_cast<const void*>(kernel));
      if (e != cudaSuccess) return e;
      if (fa.numRegs != 128) return cudaErrorInvalidConfiguration;
      int nclusters = 0;
      cfg.gridDim = dim3(sm_count() / kPair * kPair);
      e = cudaOccupancyMaxActiveClusters(&nclusters, kernel, &cfg);
      if (e != cudaSuccess) return e;
      if (nclusters < 1) return cudaErrorInvalidConfiguration;
      cache.grid[dev] = (nclusters * kPair < sm_count() ? nclusters : sm_count() / kPair) * kPair;
    }
    grid = cache.grid[dev];
  }
  cfg.gridDim = dim3(grid);
  return cudaLaunchKernelEx(&cfg, kernel, mx, ms, md, mh, msl, count, entries, segs, status, E, H, Hp,
                            accumulate);
}

}  // namespace
}  // namespace mep

using namespace mep;

extern "C" int mep_grouped_wgrad_workspace_bytes(int R, int S, int K, int E, int B, size_t* bytes) {
  if (bytes == nullptr || R < 1 || S < 0 || K < 1 || E < 1 || B < 0) return MEP_ERR_INVALID_ARG;
  if (R > MEP_MAX_R || E > MEP_MAX_E || K > MEP_MAX_K || (long long)R * B > MEP_MAX_SLOTS)
    return MEP_ERR_INVALID_ARG;
  *bytes = 16 + 32 * ((size_t)E + (size_t)R * B) + 8 * (size_t)R * (E + B);
  return MEP_OK;
}

extern "C" int mep_grouped_wgrad(const void* x, int x_type, const mep_bf16* dy,
                                 const int32_t* cu_seqlens, int32_t* status, int R, int S, int K,
                                 int E, int B, int H, int Hp, int accumulate, void* ws,
                                 size_t ws_bytes, float* home_grad, float* slot_grad, void* stream) {
  size_t need = 0;
  if (mep_grouped_wgrad_workspace_bytes(R, S, K, E, B, &need) != MEP_OK) return MEP_ERR_INVALID_ARG;
  if (x_type != MEP_BF16 && x_type != MEP_CKPT8) return MEP_ERR_INVALID_ARG;
  if (H < 8 || H % 8 != 0 || Hp < 8 || Hp % 8 != 0 || H > MEP_MAX_CKPT_C || Hp > MEP_MAX_CKPT_C)
    return MEP_ERR_INVALID_ARG;
  const long long SK = (long long)S * K, rows = (long long)R * SK;
  const long long tiles = (long long)((H + 2 * kBM - 1) / (2 * kBM)) * ((Hp + kBN - 1) / kBN);
  if (rows > 0x7fffff00LL || tiles * ((long long)E + (long long)R * B) > 0x7fff0000LL)
    return MEP_ERR_INVALID_ARG;
  if (cu_seqlens == nullptr || home_grad == nullptr || ws == nullptr || ws_bytes < need ||
      (B > 0 && slot_grad == nullptr) || (rows > 0 && (x == nullptr || dy == nullptr)))
    return MEP_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(dy) || !aligned16(home_grad) || !aligned16(slot_grad) || !aligned16(ws))
    return MEP_ERR_INVALID_ARG;
  if ((rows > 0 && (!on_current_device(x) || !on_current_device(dy))) ||
      !on_current_device(home_grad) || (B > 0 && !on_current_device(slot_grad)))
    return MEP_ERR_INVALID_ARG;
  CUtensorMap mx, ms, md, mh, msl;
  if (!map_grad(&mh, home_grad, E, H, Hp)) return MEP_ERR_CUDA;
  msl = mh;  // never used without slots
  if (B > 0 && !map_grad(&msl, slot_grad, (unsigned long long)R * B, H, Hp)) return MEP_ERR_CUDA;
  mx = ms = md = mh;  // never used without rows
  if (rows > 0) {
    const unsigned long long rb = ckpt_row_bytes(H);
    bool ok = map_2d(&md, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dy, rows, Hp, 2ull * Hp, 64, kBK,
                     CU_TENSOR_MAP_SWIZZLE_128B);
    if (x_type == MEP_CKPT8)
      ok = ok &&
           map_2d(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, x, rows, H, rb, kBM, kBK, CU_TENSOR_MAP_SWIZZLE_128B) &&
           map_2d(&ms, CU_TENSOR_MAP_DATA_TYPE_UINT8, x, rows, rb, rb, 16, kBK, CU_TENSOR_MAP_SWIZZLE_NONE);
    else
      ok = ok && map_2d(&mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, rows, H, 2ull * H, 64, kBK,
                        CU_TENSOR_MAP_SWIZZLE_128B);
    if (!ok) return MEP_ERR_CUDA;
  }
  int* count = static_cast<int*>(ws);
  int4* entries = reinterpret_cast<int4*>(static_cast<char*>(ws) + 16);
  int2* segs = reinterpret_cast<int2*>(entries + 2 * ((size_t)E + (size_t)R * B));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t err = launch_pdl(k_wgrad_groups, dim3(1), dim3(kGroupThreads), 0, st, cu_seqlens, R, E,
                               B, int(SK), accumulate, status, count, entries, segs);
  if (err != cudaSuccess) return MEP_ERR_CUDA;
  err = x_type == MEP_CKPT8 ? launch_wgrad<true>(st, mx, ms, md, mh, msl, count, entries, segs, status,
                                                 E, H, Hp, accumulate)
                            : launch_wgrad<false>(st, mx, ms, md, mh, msl, count, entries, segs,
                                                  status, E, H, Hp, accumulate);
  return err == cudaSuccess ? MEP_OK : MEP_ERR_CUDA;
}
