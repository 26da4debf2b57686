// few.cu -- the whole layer for a few tokens (mep_expert_layer) and the product
// of a few rows with a matrix in 4 bits (mep_w4_product).
//
// What bounds both is the weights' bytes: 64 tokens of an expert still do less
// than the tensor cores can while its weights arrive. So everything is arranged
// around one stream of weights: one CTA an SM, whose producer warp keeps a ring
// of stages full of bulk copies and never waits for anything but room; the
// products, the joins and the barriers between the layer's two products happen
// behind it.
//
// A unit of work is 128 columns of one expert (64 gate and the 64 matching up
// columns, or 128 columns of the second product) times the expert's tokens; a
// step is a stage's share of a unit's sum. The steps of all units in a row are
// cut into equal runs, one a CTA, so that every SM reads as many bytes as the
// others whatever the number of experts and columns; a unit that is cut leaves
// a partial sum in each of its CTAs, in fp32 in the workspace, joined in order
// after a barrier of the grid (1.3 us, and the ring of the second product fills
// meanwhile). One cooperative launch for the layer: three barriers, in
//   products 1 | activation | products 2 | weighted sum over the token's experts.
// Which experts are in use and which tokens they have, every CTA finds out by
// itself from topk_idx (a 64-bit mask of tokens for each expert).
//
// Tensor cores: mma.sync m16n8k16 with the weights as the 16-row operand and
// eight tokens as the columns, fp32 sums. (tcgen05 takes its operands from
// shared memory or TMEM at M = 64 or 128, where bytes in flight and not the
// rate are short here; and weights in 4 bits have to pass through registers,
// where this instruction takes them.) Weights in bf16 are read from the
// swizzled stage by transposing ldmatrix; in 4 bits a lane's 16 bytes are its
// operand of four steps (w4.cuh): a shift and a logic operation put two of them
// behind bf16's 128, a packed subtraction of 136 leaves q exactly, and the
// scale multiplies the group's fp32 sums.
// The activation is kept as two bf16, the value rounded and what that left
// over, and the second product takes both: it is then off by 2^-17, not 2^-9.

#include <cooperative_groups.h>

#include "ckpt.cuh"
#include "tc.cuh"
#include "w4.cuh"

namespace mep {
namespace {

constexpr int kMaxCtas = 152;       // SMs of a GB300; more are not used, the workspace counts on it
constexpr int kM = 4;               // warps across a unit's columns, 32 each
constexpr int kUnit = 128;          // columns of a unit
constexpr int kPanelRow = 128;      // bytes of a stage's row of 64 bf16 columns
constexpr int kMaxStages = 16;
constexpr int kSmem = 225 * 1024;
constexpr int kChunk = 32;          // tokens of an expert that one unit takes in the layer

__host__ __device__ constexpr int step_rows(int fmt) { return fmt == MEP_BF16 ? 128 : 256; }
__host__ __device__ constexpr int threads_of(int slices) { return 32 * (kM * slices + 2); }

// ---------------------------------------------------------------------------
// A product's units and this CTA's run of steps.
struct Phase {
  uint32_t ks, nb;      // steps of a unit, units of an expert
  uint32_t per;         // steps of a CTA
  uint32_t parts;       // CTAs that a unit may be cut over
  uint32_t begin, n;    // this CTA's
};
// Units are cut where a CTA's run ends: unit u is in CTAs u * ks / per up to
// ((u + 1) * ks - 1) / per.
__host__ __device__ __forceinline__ uint32_t parts_of(uint32_t ks, uint32_t per) {
  const uint32_t p = (ks - 1) / per + 2;
  return p < ks ? p : ks;
}
__device__ __forceinline__ Phase make_phase(uint32_t experts, uint32_t nb, uint32_t ks) {
  Phase p;
  p.ks = ks, p.nb = nb;
  const uint32_t total = experts * nb * ks;
  p.per = max(1u, (total + gridDim.x - 1) / gridDim.x);
  p.parts = parts_of(ks, p.per);
  p.begin = min(total, blockIdx.x * p.per);
  p.n = min(total, p.begin + p.per) - p.begin;
  return p;
}
__device__ __forceinline__ uint32_t first_cta(const Phase& p, uint32_t unit) { return unit * p.ks / p.per; }
__device__ __forceinline__ uint32_t parts_in(const Phase& p, uint32_t unit) {
  return ((unit + 1) * p.ks - 1) / p.per - first_cta(p, unit) + 1;
}

// ---------------------------------------------------------------------------
// The ring of stages.
struct Ring {
  uint32_t full, empty;         // barriers, 8 bytes each
  uint32_t stage0, stage_bytes; // first stage
  uint32_t x_at, plane;         // of a stage: where the rows of x start; bytes of a plane of them
  int stages;
  volatile int* abort;
  int32_t* status;
};
struct Cursor {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++slot == stages) slot = 0, parity ^= 1;
  }
};
// Where a product's weights lie: expert e's first panel of unit j, and the second panel of the unit.
struct Weights {
  const CUtensorMap* map;                // bf16
  const uint8_t* w4;                     // 4 bits
  long long expert, panel, second;       //   bytes
  int col, col_second;                   // bf16: columns of the same
  int limit;                             // units whose j * 128 + 64 reaches it have no second panel
  int K;                                 // rows
};
// Rows of x: `planes` of them after one another (the activation's two).
struct Rows {
  const char* p;
  long long pitch;  // bytes
  int K;            // bf16 of a row
};
struct List {
  const uint16_t *expert, *start;  // of an entry: its expert, its first row
  const uint16_t* row;             // of a row: t * K + k
  int entries;
};

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void bulk(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

// One thread: weights of steps [from, to) of this CTA's run.
template <int FMT>
__device__ __forceinline__ void produce_weights(const Phase& p, uint32_t from, uint32_t to, const Ring& r, Cursor& c,
                                                const Weights& w, const uint16_t* expert, int block) {
  uint32_t s = (p.begin + from) % p.ks, u = (p.begin + from) / p.ks;
  uint32_t j = u % p.nb, e = u / p.nb;
  for (uint32_t i = from; i < to; ++i) {
    const uint32_t bar = r.full + 8 * c.slot, dst = r.stage0 + c.slot * r.stage_bytes;
    if (!wait_phase(r.empty + 8 * c.slot, c.parity ^ 1, r.abort, r.status)) return;
    const bool two = int(j * kUnit + kW4Cols) < w.limit;
    if (FMT == MEP_BF16) {
      const uint32_t bytes = step_rows(FMT) * kPanelRow;
      mbar_expect_tx(bar, two ? 2 * bytes : bytes);
      tma_3d(dst, w.map, j * w.col, s * step_rows(FMT), expert[e], bar);
      if (two) tma_3d(dst + bytes, w.map, j * w.col + w.col_second, s * step_rows(FMT), expert[e], bar);
    } else {
      const int left = (w.K + kW4Rows - 1) / kW4Rows - 2 * int(s);
      const uint32_t bytes = (left < 2 ? 1 : 2) * block;
      const uint8_t* src = w.w4 + expert[e] * w.expert + j * w.panel + (long long)s * (2 * block);
      mbar_expect_tx(bar, two ? 2 * bytes : bytes);
      bulk(dst, src, bytes, bar);
      if (two) bulk(dst + 2 * block, src + w.second, bytes, bar);
    }
    c.next(r.stages);
    if (++s == p.ks) {
      s = 0;
      if (++j == p.nb) j = 0, ++e;
    }
  }
}

// One warp: the rows of x of all steps of this CTA's run. ROW(entry's row number) -> row of x.
template <int FMT, int PLANES, typename RowOf>
__device__ __forceinline__ void produce_rows(const Phase& p, const Ring& r, Cursor& c, const Rows& x,
                                             const uint16_t* start, RowOf row_of) {
  constexpr int BK = step_rows(FMT), pitch = BK * 2 + 16;
  const int lane = threadIdx.x & 31;
  uint32_t s = p.begin % p.ks, u = p.begin / p.ks;
  uint32_t j = u % p.nb, e = u / p.nb;
  for (uint32_t i = 0; i < p.n; ++i) {
    const uint32_t bar = r.full + 8 * c.slot, dst = r.stage0 + c.slot * r.stage_bytes + r.x_at;
    const int first = start[e], m = start[e + 1] - first, k0 = s * BK, bytes = 2 * min(BK, x.K - k0);
    if (!__all_sync(MEP_FULL_MASK, wait_phase(r.empty + 8 * c.slot, c.parity ^ 1, r.abort, r.status))) return;
    if (bytes < 2 * BK) {  // beyond the sum's end the weights are zeros: what they meet must be numbers
      for (int q = lane; q < PLANES * m; q += 32) {
        const uint32_t d = dst + (q % PLANES) * r.plane + (q / PLANES) * pitch;
        for (int b = bytes; b < 2 * BK; b += 16)
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(d + b), "r"(0) : "memory");
      }
      fence_async();
      __syncwarp();
    }
    if (lane == 0) mbar_expect_tx(bar, PLANES * m * bytes);
    __syncwarp();
    for (int q = lane; q < PLANES * m; q += 32)
      bulk(dst + (q % PLANES) * r.plane + (q / PLANES) * pitch,
           x.p + (row_of(first + q / PLANES) * PLANES + q % PLANES) * x.pitch + 2 * k0, bytes, bar);
    c.next(r.stages);
    if (++s == p.ks) {
      s = 0;
      if (++j == p.nb) j = 0, ++e;
    }
  }
}

// ---------------------------------------------------------------------------
// Products.
__device__ __forceinline__ void ldmatrix4(uint32_t (&v)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&v)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// Operand of one step: two q at bits 4i and 16 + 4i of the word, behind the bits of bf16 128, less 136.
__device__ __forceinline__ void widen_q(uint32_t word, uint32_t (&a)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = ((word >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(a[i]) : "r"(v), "r"(0x43084308u));
  }
}

// This warp's share of a stage: 16 columns of either panel, slice `sl` of the rows.
template <int FMT, int SLICES, int NT, int PLANES>
__device__ __forceinline__ void stage_product(float (&acc)[2][NT][4], uint32_t stage, const Ring& r, int mi, int sl,
                                              int group, int block) {
  constexpr int BK = step_rows(FMT), pitch = BK * 2 + 16;
  const int lane = threadIdx.x & 31;
  const uint32_t xb = stage + r.x_at + (lane & 7) * pitch + (sl * (BK / SLICES) + 8 * (lane >> 3)) * 2;
  if (FMT == MEP_BF16) {
    const uint32_t wa = stage + (sl * (BK / SLICES) + (lane >> 4) * 8 + (lane & 7)) * kPanelRow +
                        (((2 * mi + ((lane >> 3) & 1)) ^ (lane & 7)) << 4);
#pragma unroll
    for (int k = 0; k < BK / SLICES; k += 32) {
      uint32_t a[2][2][4];
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int s = 0; s < 2; ++s) ldmatrix4_trans(a[q][s], wa + q * (BK * kPanelRow) + (k + 16 * s) * kPanelRow);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int pl = 0; pl < PLANES; ++pl) {
          uint32_t b[4];
          ldmatrix4(b, xb + pl * r.plane + n * (8 * pitch) + 2 * k);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            mma(acc[q][n], a[q][0], b[0], b[1]);
            mma(acc[q][n], a[q][1], b[2], b[3]);
          }
        }
    }
  } else {
    // 64 rows at a time: a lane's 16 bytes of either panel
#pragma unroll
    for (int k = 0; k < BK / SLICES; k += 64) {
      const int row = sl * (BK / SLICES) + k, b = row / kW4Rows, h = row / 64 % 2;
      const uint32_t wb = stage + b * block;
      uint4 words[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) words[q] = lds128(wb + q * 2 * block + ((h * 4 + mi) * 32 + lane) * 16);
      const uint32_t sb = wb + kW4Pairs + (mi * 8 + (lane >> 2)) * 4;
      // groups of 32 rows scale every 32, the others every 64 (128 is 64 twice, by the same scale)
      const uint32_t g0 = 64 * h / group * 128, g1 = (64 * h + 32) / group * 128;
      const bool split = group == 32;
      float sum[2][NT][4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (half == 0 || split) {
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int n = 0; n < NT; ++n) sum[q][n][0] = sum[q][n][1] = sum[q][n][2] = sum[q][n][3] = 0.f;
        }
        uint32_t a[2][2][4];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          widen_q(half ? words[q].z : words[q].x, a[q][0]);
          widen_q(half ? words[q].w : words[q].y, a[q][1]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int pl = 0; pl < PLANES; ++pl) {
            uint32_t bx[4];
            ldmatrix4(bx, xb + pl * r.plane + n * (8 * pitch) + 2 * (k + 32 * half));
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              mma(sum[q][n], a[q][0], bx[0], bx[1]);
              mma(sum[q][n], a[q][1], bx[2], bx[3]);
            }
          }
        if (half == 1 || split) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t sc = lds32(sb + q * 2 * block + (half ? g1 : g0));
            const float lo = __uint_as_float(sc << 16), hi = __uint_as_float(sc & 0xffff0000u);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              acc[q][n][0] = fmaf(lo, sum[q][n][0], acc[q][n][0]);
              acc[q][n][1] = fmaf(lo, sum[q][n][1], acc[q][n][1]);
              acc[q][n][2] = fmaf(hi, sum[q][n][2], acc[q][n][2]);
              acc[q][n][3] = fmaf(hi, sum[q][n][3], acc[q][n][3]);
            }
          }
        }
      }
    }
  }
}

// Steps of one unit, then its partial sum: slices joined through shared memory
// (in order), the first slice's warps write. PUT(panel, column of 64, token, value).
template <int FMT, int SLICES, int NT, int PLANES, typename Put>
__device__ __forceinline__ void unit_product(uint32_t steps, uint32_t s, int K, const Ring& r, Cursor& c, int m,
                                             int group, int block, float4* s_join, Put put) {
  constexpr int BK = step_rows(FMT);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mi = warp % kM, sl = warp / kM;
  float acc[2][NT][4];
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[q][n][0] = acc[q][n][1] = acc[q][n][2] = acc[q][n][3] = 0.f;
  for (; steps > 0; --steps, ++s) {
    if (!__all_sync(MEP_FULL_MASK, wait_phase(r.full + 8 * c.slot, c.parity, r.abort, r.status))) break;
    // a slice wholly beyond the sum's end has no weights (4 bits) or zeros
    if (int(s * BK) + sl * (BK / SLICES) / kW4Rows * kW4Rows < K)
      stage_product<FMT, SLICES, NT, PLANES>(acc, r.stage0 + c.slot * r.stage_bytes, r, mi, sl, group, block);
    __syncwarp();
    if (lane == 0)
      asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(r.empty + 8 * c.slot) : "memory");
    c.next(r.stages);
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (8 * n >= m) break;
    float4* mine = s_join + ((sl - 1) * kM + mi) * 64 + lane;
    if (sl > 0) {
      mine[0] = make_float4(acc[0][n][0], acc[0][n][1], acc[0][n][2], acc[0][n][3]);
      mine[32] = make_float4(acc[1][n][0], acc[1][n][1], acc[1][n][2], acc[1][n][3]);
    }
    asm volatile("bar.sync %0, %1;" ::"r"(1 + mi), "r"(32 * SLICES) : "memory");
    if (sl == 0) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float v[4] = {acc[q][n][0], acc[q][n][1], acc[q][n][2], acc[q][n][3]};
#pragma unroll
        for (int o = 1; o < SLICES; ++o) {
          const float4 f = s_join[((o - 1) * kM + mi) * 64 + 32 * q + lane];
          v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = 8 * n + 2 * (lane & 3) + (i & 1);
          if (t < m) put(q, 16 * mi + (lane >> 2) + 8 * (i >> 1), t, v[i]);
        }
      }
    }
    asm volatile("bar.sync %0, %1;" ::"r"(1 + mi), "r"(32 * SLICES) : "memory");
  }
}

// All units of this CTA's run. PUT(entry, unit of the expert, part, panel, column, token, value).
template <int FMT, int SLICES, int NTMAX, int PLANES, typename Put>
__device__ __forceinline__ void products(const Phase& p, int K, const Ring& r, Cursor& c, const uint16_t* start,
                                         int group, int block, float4* s_join, Put put) {
  uint32_t i = 0;
  while (i < p.n) {  // after a wait that gave up too: the joins' barriers want every warp
    const uint32_t at = p.begin + i, u = at / p.ks, s = at % p.ks, steps = min(p.ks - s, p.n - i);
    const uint32_t e = u / p.nb, j = u % p.nb, part = blockIdx.x - first_cta(p, u);
    const int m = start[e + 1] - start[e];
    const auto f = [&](int q, int col, int t, float v) { put(e, j, part, q, col, t, v); };
    if (m <= 8)
      unit_product<FMT, SLICES, 1, PLANES>(steps, s, K, r, c, m, group, block, s_join, f);
    else if (m <= 16)
      unit_product<FMT, SLICES, 2, PLANES>(steps, s, K, r, c, m, group, block, s_join, f);
    else if (NTMAX <= 4 || m <= 32)
      unit_product<FMT, SLICES, 4, PLANES>(steps, s, K, r, c, m, group, block, s_join, f);
    else
      unit_product<FMT, SLICES, NTMAX, PLANES>(steps, s, K, r, c, m, group, block, s_join, f);
    i += steps;
  }
}

// Stages for rows of up to m tokens (as many as a unit's instantiation computes).
template <int FMT, int PLANES>
__device__ __forceinline__ void size_ring(Ring& r, uint32_t room, int m, int block) {
  const int rows = m <= 8 ? 8 : m <= 16 ? 16 : m <= 32 ? 32 : 64;
  r.x_at = FMT == MEP_BF16 ? 2 * step_rows(FMT) * kPanelRow : 4 * block;
  r.plane = rows * (step_rows(FMT) * 2 + 16);
  r.stage_bytes = (r.x_at + PLANES * r.plane + 1023) / 1024 * 1024;
  r.stages = min(kMaxStages, int(room / r.stage_bytes));
}

struct Head {  // start of shared memory
  uint64_t full[kMaxStages], empty[kMaxStages];
  int warp_sums[32];
  int abort, bad, most, entries, rows, go;
};

__device__ __forceinline__ void init_ring(Ring& r, Head* h, int consumers, int32_t* status) {
  r.full = smem_u32(h->full), r.empty = smem_u32(h->empty);
  r.abort = &h->abort, r.status = status;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(r.full + 8 * i, 2);  // weights, rows
      mbar_init(r.empty + 8 * i, consumers);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    h->abort = h->bad = h->most = 0;
  }
}

// After a wait that gave up: copies may be under way still; they land before the CTA's memory is another's.
__device__ __forceinline__ void settle(const Ring& r) {
  __syncthreads();
  if (threadIdx.x == 0 && *r.abort) {
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 100000ull) {
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
struct LayerArgs {
  const __nv_bfloat16* x;
  const int32_t* idx;
  const float* topk_w;
  const uint8_t *w1, *w2;
  int32_t* status;
  int T, K, E, H, F, group;
  float *part1, *part2;
  __nv_bfloat16* act;
  __nv_bfloat16* out;
};

__host__ __device__ __forceinline__ int max_entries(int T, int K, int E) {
  return (E < T * K ? E : T * K) + T * K / kChunk;
}
__host__ __device__ __forceinline__ uint32_t list_bytes(int T, int K, int E) {
  return (2u * (2 * max_entries(T, K, E) + 1 + 3 * T * K) + 1023) / 1024 * 1024;
}
__host__ __device__ __forceinline__ uint32_t join_bytes(int slices) { return (slices - 1) * kM * 64 * 16; }
constexpr uint32_t kHeadBytes = 1024;
static_assert(sizeof(Head) <= kHeadBytes, "head");

// The experts in use in ascending order, each one's tokens in order, more than
// kChunk of them in several entries; where each assignment went.
__device__ __forceinline__ void make_list(const LayerArgs& a, Head* h, char* scratch, uint16_t* expert, uint16_t* start,
                                          uint16_t* row_entry, uint16_t* row_of, uint16_t* row_token) {
  unsigned long long* mask = reinterpret_cast<unsigned long long*>(scratch);
  uint16_t* e_start = reinterpret_cast<uint16_t*>(mask + a.E);
  uint16_t* e_entry = e_start + a.E;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, A = a.T * a.K;
  for (int e = tid; e < a.E; e += threads) mask[e] = 0;
  __syncthreads();
  for (int i = tid; i < A; i += threads) {
    const int e = a.idx[i];
    if (e >= 0 && e < a.E) {
      const unsigned long long bit = 1ull << (i / a.K);
      if (atomicOr(&mask[e], bit) & bit) h->bad = 1;
    } else if (e != -1) {
      h->bad = 1;
    }
  }
  __syncthreads();
  // entries and rows before each thread's experts, in one word
  const int per = (a.E + threads - 1) / threads, lo = min(a.E, tid * per), hi = min(a.E, lo + per);
  int sum = 0, most = 0;
  for (int e = lo; e < hi; ++e) {
    const int n = __popcll(mask[e]);
    sum += ((n + kChunk - 1) / kChunk << 16) + n;
    most = max(most, n);
  }
  const int incl = warp_incl_scan(sum);
  most = __reduce_max_sync(MEP_FULL_MASK, most);
  if (lane == 31) h->warp_sums[warp] = incl;
  if (lane == 0) atomicMax(&h->most, most);
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < threads / 32; ++w) {
    if (w < warp) before += h->warp_sums[w];
    all += h->warp_sums[w];
  }
  before += incl - sum;
  for (int e = lo; e < hi; ++e) {
    const int n = __popcll(mask[e]);
    int entry = before >> 16, row = before & 0xffff;
    e_start[e] = row, e_entry[e] = entry;
    for (int q = 0; q < n; q += kChunk, ++entry) expert[entry] = e, start[entry] = row + q;
    before += ((n + kChunk - 1) / kChunk << 16) + n;
  }
  if (tid == 0) {
    h->entries = all >> 16, h->rows = all & 0xffff;
    start[all >> 16] = all & 0xffff;
  }
  __syncthreads();
  for (int i = tid; i < A; i += threads) {
    const int e = a.idx[i];
    if (e < 0 || e >= a.E) {
      row_of[i] = 0xffff;
      continue;
    }
    const int t = i / a.K, rank = __popcll(mask[e] & ((1ull << t) - 1));
    const int row = e_start[e] + rank;
    row_of[i] = row;
    if (!h->bad) row_token[row] = t, row_entry[row] = e_entry[e] + rank / kChunk;
  }
  fence_async();  // the ring's copies come into the same memory
  __syncthreads();
}

template <int FMT, int SLICES>
__global__ void __launch_bounds__(threads_of(SLICES), 1)
    k_layer(const __grid_constant__ CUtensorMap map1, const __grid_constant__ CUtensorMap map2, const LayerArgs a) {
  extern __shared__ __align__(1024) char smem[];
  const auto grid = cooperative_groups::this_grid();
  constexpr int BK = step_rows(FMT), NTMAX = kChunk / 8, kConsumers = kM * SLICES;
  Head* h = reinterpret_cast<Head*>(smem);
  char* at = smem + kHeadBytes;
  float4* s_join = reinterpret_cast<float4*>(at);
  at += join_bytes(SLICES);
  const int cap = max_entries(a.T, a.K, a.E), A = a.T * a.K;
  uint16_t* expert = reinterpret_cast<uint16_t*>(at);
  uint16_t* start = expert + cap;
  uint16_t* row_entry = start + cap + 1;
  uint16_t* row_of = row_entry + A;
  uint16_t* row_token = row_of + A;
  at += list_bytes(a.T, a.K, a.E);
  Ring r;
  init_ring(r, h, kConsumers, a.status);
  const int block = FMT == MEP_W4 ? w4_block_bytes(a.group) : 0;
  if (threadIdx.x == 0) h->go = read_status(a.status) == 0;
  __syncthreads();
  make_list(a, h, at, expert, start, row_entry, row_of, row_token);
  const bool go = h->go && !h->bad;
  if (h->go && h->bad && threadIdx.x == 0) set_status(a.status, MEP_ERR_BAD_ROUTING);
  r.stage0 = smem_u32(at);
  size_ring<FMT, 2>(r, kSmem - uint32_t(at - smem), min(h->most, kChunk), block);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t experts = go ? h->entries : 0, rows = go ? h->rows : 0;
  const Phase p1 = make_phase(experts, (a.F + 63) / 64, (a.H + BK - 1) / BK);
  const Phase p2 = make_phase(experts, (a.H + kUnit - 1) / kUnit, (a.F + BK - 1) / BK);
  const long long m1 = FMT == MEP_W4 ? w4_matrix_bytes(a.H, a.F, a.group) : 0, q1 = FMT == MEP_W4 ? w4_panel_bytes(a.H, a.group) : 0;
  const long long m2 = FMT == MEP_W4 ? w4_matrix_bytes(a.F, a.H, a.group) : 0, q2 = FMT == MEP_W4 ? w4_panel_bytes(a.F, a.group) : 0;
  const Weights w1 = {&map1, a.w1, 2 * m1, q1, m1, 64, a.F, 0x7fffffff, a.H};
  const Weights w2 = {&map2, a.w2, m2, 2 * q2, q2, kUnit, 64, a.H, a.F};
  const Rows x1 = {reinterpret_cast<const char*>(a.x), 2LL * a.H, a.H};
  const Rows x2 = {reinterpret_cast<const char*>(a.act), 2LL * a.F, a.F};
  Cursor c;
  const uint32_t ahead = min(p2.n, uint32_t(r.stages));

  if (warp == kConsumers) {
    if (lane == 0) {
      produce_weights<FMT>(p1, 0, p1.n, r, c, w1, expert, block);
      produce_weights<FMT>(p2, 0, ahead, r, c, w2, expert, block);  // filling while the activation is computed
    }
    __syncwarp();
  } else if (warp == kConsumers + 1) {
    produce_rows<FMT, 1>(p1, r, c, x1, start, [&](int row) { return (long long)row_token[row]; });
  } else {
    products<FMT, SLICES, NTMAX, 1>(p1, a.H, r, c, start, a.group, block, s_join,
                                    [&](uint32_t e, uint32_t j, uint32_t part, int q, int col, int t, float v) {
                                      const int f = j * 64 + col;
                                      if (f < a.F)
                                        a.part1[((long long)(start[e] + t) * p1.parts + part) * (2 * a.F) + q * a.F + f] = v;
                                    });
  }
  grid.sync();
  {
    const uint32_t quads = a.F / 4, n = rows * quads, step = gridDim.x * blockDim.x;
    for (uint32_t i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) {
      const uint32_t row = i / quads, f = i % quads * 4;
      const uint32_t parts = parts_in(p1, row_entry[row] * p1.nb + f / 64);
      const float* in = a.part1 + (long long)row * p1.parts * (2 * a.F) + f;
      float g[4] = {}, u[4] = {};
#pragma unroll 4
      for (uint32_t q = 0; q < parts; ++q) {
        const float4 vg = *reinterpret_cast<const float4*>(in + q * (2LL * a.F));
        const float4 vu = *reinterpret_cast<const float4*>(in + q * (2LL * a.F) + a.F);
        g[0] += vg.x, g[1] += vg.y, g[2] += vg.z, g[3] += vg.w;
        u[0] += vu.x, u[1] += vu.y, u[2] += vu.z, u[3] += vu.w;
      }
      __nv_bfloat16 hi[4], lo[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float v = g[k] / (1.f + expf(-g[k])) * u[k];
        hi[k] = __float2bfloat16_rn(v);
        const float rest = v - __bfloat162float(hi[k]);
        lo[k] = __float2bfloat16_rn(isfinite(rest) ? rest : 0.f);  // an infinity stays one
      }
      __nv_bfloat16* o = a.act + (long long)row * 2 * a.F + f;
      *reinterpret_cast<uint2*>(o) = *reinterpret_cast<uint2*>(hi);
      *reinterpret_cast<uint2*>(o + a.F) = *reinterpret_cast<uint2*>(lo);
    }
    fence_async();
  }
  grid.sync();
  if (warp == kConsumers) {
    if (lane == 0) produce_weights<FMT>(p2, ahead, p2.n, r, c, w2, expert, block);
    __syncwarp();
  } else if (warp == kConsumers + 1) {
    fence_async();
    produce_rows<FMT, 2>(p2, r, c, x2, start, [&](int row) { return (long long)row; });
  } else {
    products<FMT, SLICES, NTMAX, 2>(p2, a.F, r, c, start, a.group, block, s_join,
                                    [&](uint32_t e, uint32_t j, uint32_t part, int q, int col, int t, float v) {
                                      const int n = j * kUnit + 64 * q + col;
                                      if (n < a.H) a.part2[((long long)(start[e] + t) * p2.parts + part) * a.H + n] = v;
                                    });
  }
  grid.sync();
  if (go) {
    // eight lanes share four outputs, each a part of the token's experts
    const uint32_t quads = a.H / 4, n = a.T * quads * 8, step = gridDim.x * blockDim.x;
    for (uint32_t i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) {
      const uint32_t o = i / 8, t = o / quads, col = o % quads * 4;
      float s[4] = {};
      for (int k = i % 8; k < a.K; k += 8) {
        const uint32_t row = row_of[t * a.K + k];
        if (row == 0xffff) continue;
        const uint32_t parts = parts_in(p2, row_entry[row] * p2.nb + col / kUnit);
        const float* in = a.part2 + (long long)row * p2.parts * a.H + col;
        float y[4] = {};
#pragma unroll 4
        for (uint32_t q = 0; q < parts; ++q) {
          const float4 v = *reinterpret_cast<const float4*>(in + q * (long long)a.H);
          y[0] += v.x, y[1] += v.y, y[2] += v.z, y[3] += v.w;
        }
        const float w = a.topk_w[t * a.K + k];
#pragma unroll
        for (int q = 0; q < 4; ++q) s[q] = fmaf(w, y[q], s[q]);
      }
      const unsigned lanes = 0xffu << (threadIdx.x & 24);
#pragma unroll
      for (int d = 4; d > 0; d >>= 1)
#pragma unroll
        for (int q = 0; q < 4; ++q) s[q] += __shfl_xor_sync(lanes, s[q], d);
      if (i % 8 == 0) {
        __nv_bfloat16 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = __float2bfloat16_rn(s[q]);
        *reinterpret_cast<uint2*>(a.out + (long long)t * a.H + col) = *reinterpret_cast<uint2*>(v);
      }
    }
  }
  settle(r);
}

// ---------------------------------------------------------------------------
struct ProductArgs {
  const __nv_bfloat16* x;
  const uint8_t* w4;
  int32_t* status;
  int T, K, N, group;
  __nv_bfloat16* padded;  // rows of x that are whole 16-byte vectors, where K is not a multiple of 8
  float* part;
  void* y;
};

template <int SLICES, int NTMAX, typename T>
__global__ void __launch_bounds__(threads_of(SLICES), 1) k_w4_product(const ProductArgs a) {
  extern __shared__ __align__(1024) char smem[];
  const auto grid = cooperative_groups::this_grid();
  constexpr int FMT = MEP_W4, BK = step_rows(FMT), kConsumers = kM * SLICES;
  Head* h = reinterpret_cast<Head*>(smem);
  uint16_t* start = reinterpret_cast<uint16_t*>(h + 1);  // one entry, all rows
  uint16_t* expert = start + 2;
  static_assert(sizeof(Head) + 8 <= kHeadBytes, "head");
  float4* s_join = reinterpret_cast<float4*>(smem + kHeadBytes);
  char* at = smem + kHeadBytes + join_bytes(SLICES);
  Ring r;
  init_ring(r, h, kConsumers, a.status);
  if (threadIdx.x == 0) {
    h->go = read_status(a.status) == 0;
    start[0] = 0, start[1] = a.T, expert[0] = 0;
  }
  __syncthreads();
  const bool go = h->go;
  const int block = w4_block_bytes(a.group);
  r.stage0 = smem_u32(at);
  size_ring<FMT, 1>(r, kSmem - uint32_t(at - smem), a.T, block);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Phase p = make_phase(go ? 1 : 0, (a.N + kUnit - 1) / kUnit, (a.K + BK - 1) / BK);
  const long long panel = w4_panel_bytes(a.K, a.group);
  const Weights w = {nullptr, a.w4, 0, 2 * panel, panel, 0, 0, a.N, a.K};
  const bool pad = a.K % 8 != 0;
  const int K8 = (a.K + 7) / 8 * 8;
  const Rows x = {reinterpret_cast<const char*>(pad ? a.padded : a.x), 2LL * K8, K8};
  Cursor c;
  const uint32_t ahead = min(p.n, uint32_t(r.stages));
  if (pad) {
    if (threadIdx.x == 32 * kConsumers) produce_weights<FMT>(p, 0, ahead, r, c, w, expert, block);
    __syncwarp();
    for (uint32_t i = blockIdx.x * blockDim.x + threadIdx.x; i < uint32_t(a.T * K8); i += gridDim.x * blockDim.x) {
      const uint32_t t = i / K8, k = i % K8;
      a.padded[i] = int(k) < a.K ? a.x[(long long)t * a.K + k] : __float2bfloat16_rn(0.f);
    }
    fence_async();
    grid.sync();
    fence_async();
  }
  if (warp == kConsumers) {
    if (lane == 0) produce_weights<FMT>(p, pad ? ahead : 0, p.n, r, c, w, expert, block);
    __syncwarp();
  } else if (warp == kConsumers + 1) {
    produce_rows<FMT, 1>(p, r, c, x, start, [&](int row) { return (long long)row; });
  } else {
    products<FMT, SLICES, NTMAX, 1>(p, a.K, r, c, start, a.group, block, s_join,
                                    [&](uint32_t, uint32_t j, uint32_t part, int q, int col, int t, float v) {
                                      const int n = j * kUnit + 64 * q + col;
                                      if (n < a.N) a.part[((long long)t * p.parts + part) * a.N + n] = v;
                                    });
  }
  grid.sync();
  if (go) {
    const uint32_t n = uint32_t(a.T) * a.N, step = gridDim.x * blockDim.x;
    for (uint32_t i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) {
      const uint32_t t = i / a.N, col = i % a.N, parts = parts_in(p, col / kUnit);
      const float* in = a.part + (long long)t * p.parts * a.N + col;
      float s = 0.f;
#pragma unroll 4
      for (uint32_t q = 0; q < parts; ++q) s += in[q * (long long)a.N];
      static_cast<T*>(a.y)[i] = from_f32<T>(s);
    }
  }
  settle(r);
}

// ---------------------------------------------------------------------------
// host side
template <typename... KArgs, typename... Args>
int launch_all(void (*kernel)(KArgs...), long long most, int threads, cudaStream_t st, const Args&... args) {
  if (set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), kSmem)) return MEP_ERR_CUDA;
  const int sms = sm_count() < kMaxCtas ? sm_count() : kMaxCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(most < 1 ? 1 : most < sms ? most : sms));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? MEP_OK : MEP_ERR_CUDA;
}
long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Most bytes of partial sums [rows][parts][columns] with 1 to `experts` of them
// in use: the fewer, the more CTAs share a unit, and the fewer rows there are.
size_t part_bytes(int experts, int T, int A, long long nb, long long ks, long long columns) {
  size_t top = 0;
  for (int n = 1; n <= experts; ++n) {
    const long long per = ceil_div(n * nb * ks, kMaxCtas), rows = (long long)T * n < A ? (long long)T * n : A;
    const size_t bytes = size_t(rows) * parts_of(uint32_t(ks), uint32_t(per)) * columns * 4;
    if (bytes > top) top = bytes;
  }
  return align256(top);
}

// 3D bf16 map over [E, K, N], box {64 columns, 128 rows, 1}, 128-byte swizzle; beyond a matrix's edges zeros.
bool make_map3(CUtensorMap* m, const void* p, long long E, long long K, long long N) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {cuuint64_t(N), cuuint64_t(K), cuuint64_t(E)};
  const cuuint64_t strides[2] = {cuuint64_t(N) * 2, cuuint64_t(N) * K * 2};
  const cuuint32_t box[3] = {64, cuuint32_t(step_rows(MEP_BF16)), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The layer's workspace: partial sums of the first product, the activation, partial sums of the second.
struct LayerSpace {
  size_t part1, act, part2;
  size_t all() const { return part1 + act + part2; }
};
bool layer_space(int T, int K, int E, long long H, long long F, int w_type, int group, LayerSpace* s) {
  if (T < 0 || T > MEP_MAX_FEW || K < 1 || K > MEP_MAX_K || E < 1 || E > MEP_MAX_E || H < 8 || F < 8 || H % 8 != 0 ||
      F % 8 != 0 || H > MEP_MAX_FEW_H || F > MEP_MAX_FEW_H / 2)
    return false;
  if (w_type != MEP_BF16 && (w_type != MEP_W4 || !w4_sizes_ok(H, F, group))) return false;
  // beyond K experts there are no more rows, only fewer parts
  const int A = T * K, experts = E < K ? E : K, bk = step_rows(w_type);
  s->part1 = part_bytes(T > 0 ? experts : 0, T, A, ceil_div(F, 64), ceil_div(H, bk), 2 * F);
  s->part2 = part_bytes(T > 0 ? experts : 0, T, A, ceil_div(H, kUnit), ceil_div(F, bk), H);
  s->act = align256(size_t(A) * F * 4);
  return true;
}

struct ProductSpace {
  size_t padded, part;
  size_t all() const { return padded + part; }
};
bool product_space(int T, long long K, long long N, int group, ProductSpace* s) {
  if (T < 0 || T > MEP_MAX_FEW || !w4_sizes_ok(K, N, group)) return false;
  s->padded = K % 8 == 0 ? 0 : align256(size_t(T) * ceil_div(K, 8) * 16);
  s->part = part_bytes(1, T, T, ceil_div(N, kUnit), ceil_div(K, step_rows(MEP_W4)), N);
  return true;
}

template <int FMT, int SLICES>
int launch_layer(const CUtensorMap& m1, const CUtensorMap& m2, const LayerArgs& a, cudaStream_t st) {
  const long long experts = max_entries(a.T, a.K, a.E), bk = step_rows(FMT);
  const long long n1 = experts * ceil_div(a.F, 64) * ceil_div(a.H, bk), n2 = experts * ceil_div(a.H, kUnit) * ceil_div(a.F, bk);
  return launch_all(k_layer<FMT, SLICES>, n1 > n2 ? n1 : n2, threads_of(SLICES), st, m1, m2, a);
}
template <typename T> int launch_product(const ProductArgs& a, cudaStream_t st) {
  const long long n = ceil_div(a.N, kUnit) * ceil_div(a.K, step_rows(MEP_W4));
  return a.T <= 32 ? launch_all(k_w4_product<4, 4, T>, n, threads_of(4), st, a)
                   : launch_all(k_w4_product<2, 8, T>, n, threads_of(2), st, a);
}

}  // namespace
}  // namespace mep

using namespace mep;

extern "C" int mep_w4_product_workspace_bytes(int T, int64_t K, int64_t N, int group, size_t* bytes) {
  ProductSpace s;
  if (bytes == nullptr || !product_space(T, K, N, group, &s)) return MEP_ERR_INVALID_ARG;
  *bytes = s.all();
  return MEP_OK;
}

extern "C" int mep_w4_product(const mep_bf16* x, const uint8_t* w4, int32_t* status, int T, int64_t K, int64_t N,
                              int group, void* ws, size_t ws_bytes, int y_type, void* y, void* stream) {
  ProductSpace s;
  if (!product_space(T, K, N, group, &s) || (y_type != MEP_BF16 && y_type != MEP_F32)) return MEP_ERR_INVALID_ARG;
  if (T == 0) return MEP_OK;
  if (x == nullptr || w4 == nullptr || y == nullptr || ws == nullptr || ws_bytes < s.all()) return MEP_ERR_INVALID_ARG;
  if (!aligned16(w4) || !aligned16(ws) || reinterpret_cast<uintptr_t>(x) % (K % 8 == 0 ? 16 : 2) != 0 ||
      reinterpret_cast<uintptr_t>(y) % (y_type == MEP_BF16 ? 2 : 4) != 0)
    return MEP_ERR_INVALID_ARG;
  char* p = static_cast<char*>(ws);
  const ProductArgs a = {reinterpret_cast<const __nv_bfloat16*>(x), w4, status, T, int(K), int(N), group,
                         reinterpret_cast<__nv_bfloat16*>(p), reinterpret_cast<float*>(p + s.padded), y};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return y_type == MEP_BF16 ? launch_product<__nv_bfloat16>(a, st) : launch_product<float>(a, st);
}

extern "C" int mep_expert_layer_workspace_bytes(int T, int K, int E, int64_t H, int64_t F, int w_type, int group,
                                                size_t* bytes) {
  LayerSpace s;
  if (bytes == nullptr || !layer_space(T, K, E, H, F, w_type, group, &s)) return MEP_ERR_INVALID_ARG;
  *bytes = s.all();
  return MEP_OK;
}

extern "C" int mep_expert_layer(const mep_bf16* x, const int32_t* topk_idx, const float* topk_w, const void* w1,
                                const void* w2, int w_type, int group, int32_t* status, int T, int K, int E, int64_t H,
                                int64_t F, void* ws, size_t ws_bytes, mep_bf16* out, void* stream) {
  LayerSpace s;
  if (!layer_space(T, K, E, H, F, w_type, group, &s)) return MEP_ERR_INVALID_ARG;
  if (T == 0) return MEP_OK;
  if (x == nullptr || topk_idx == nullptr || topk_w == nullptr || w1 == nullptr || w2 == nullptr || ws == nullptr ||
      out == nullptr || ws_bytes < s.all())
    return MEP_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w1) || !aligned16(w2) || !aligned16(ws) || !aligned16(out) ||
      reinterpret_cast<uintptr_t>(topk_idx) % 4 != 0 || reinterpret_cast<uintptr_t>(topk_w) % 4 != 0)
    return MEP_ERR_INVALID_ARG;
  char* p = static_cast<char*>(ws);
  const LayerArgs a = {reinterpret_cast<const __nv_bfloat16*>(x),
                       topk_idx,
                       topk_w,
                       static_cast<const uint8_t*>(w1),
                       static_cast<const uint8_t*>(w2),
                       status,
                       T,
                       K,
                       E,
                       int(H),
                       int(F),
                       group,
                       reinterpret_cast<float*>(p),
                       reinterpret_cast<float*>(p + s.part1 + s.act),
                       reinterpret_cast<__nv_bfloat16*>(p + s.part1),
                       reinterpret_cast<__nv_bfloat16*>(out)};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  CUtensorMap m1 = {}, m2 = {};
  if (w_type == MEP_W4) return launch_layer<MEP_W4, 4>(m1, m2, a, st);
  if (!on_current_device(w1) || !on_current_device(w2)) return MEP_ERR_INVALID_ARG;
  if (!make_map3(&m1, w1, E, H, 2 * F) || !make_map3(&m2, w2, E, F, H)) return MEP_ERR_CUDA;
  return launch_layer<MEP_BF16, 4>(m1, m2, a, st);
}
