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
// A unit of work is 256 columns of one expert (128 gate and the 128 matching up
// columns, or 256 columns of the second product) times the expert's tokens, up
// to 32 in the layer; a step is a stage's share of a unit's sum: 64 rows of bf16
// (32 KB), 256 of 4 bits (33 to 36 KB). The steps of all units in a row are cut
// into runs without regard to where units end, so that every SM reads about as
// many bytes as the others whatever the number of experts and columns (Phase);
// a unit that is cut leaves a partial sum for each of its runs, in fp32 in the
// workspace, joined in order after a barrier of the grid (1.3 us, and the ring of
// the second product fills meanwhile). One cooperative launch for the layer:
//   products 1 | activation | products 2 | weighted sum over the token's experts
// with a barrier at each stroke, and one more in front where runs are counted.
// Which experts are in use and which tokens they have, every CTA finds out by
// itself from topk_idx (a 64-bit mask of tokens for each expert; 2.8 us).
//
// Tensor cores: mma.sync m16n8k16 with the weights as the 16-row operand and
// eight tokens as the columns, fp32 sums. (tcgen05 takes its operands from
// shared memory or TMEM at M = 64 or 128, where bytes in flight and not the
// rate are short here; and weights in 4 bits have to pass through registers,
// where this instruction takes them.) Weights in bf16 are read from the
// swizzled stage by transposing ldmatrix; in 4 bits a lane's 16 bytes are its
// operand of four steps (w4.cuh): a mask and a packed multiply-add make two of
// them q / 64 exactly, and the scale multiplies the group's fp32 sums.
// The activation is kept as two bf16, the value rounded and what that left
// over, and the second product takes both: it is then off by 2^-17 of itself at
// most (below 2^-117 by 2^-134, half of bf16's smallest number), where one bf16
// would be off by 2^-8. bf16 x bf16 is exact in fp32. Of the results of 64 tokens of
// the large layer 0.46% round to the other side than the 64-bit value does, 0.15%
// with fp32 throughout; the error in the norm is 1.658e-3 for both, the rounding.
//
// Measured, as one node of a graph, L2 flushed before it (back to back):
//   64 tokens, 256 experts, 7168 x 1408, 8 each, bf16: 12.2 GB of weights in
//     1746 to 1790 us (1693 to 1750), 6.8 to 7.1 TB/s; the same without the products.
//   16 tokens of it in 4 bits: 1.24 GB in 260 us (244). Without the products the
//     copies take 226, and the products hide behind them but for a unit's start and
//     its sums: a stage's 65536 weights keep eight warps busy for some 1000 clocks,
//     in which they issue nine operations for eight weights to widen them. Sixteen
//     warps of half the columns each took 294, where eight took 283; both blocks of
//     a stage in one go 308, where one after another took 302.
//   1 token in 4 bits: 125 MB in 48 us (42); 1 token, 64 experts, 2048 x 1408, 6
//     each, bf16: 104 MB in 40 us (32). A launch with its first loads is some 5,
//     the list 2.8, a barrier 1.3; the rest is the stream with its start and its
//     slowest SM (some read a fifth slower than others).
//   A call of a few small experts 19 us (16): all latency. What helped there is
//     that the code is run through before its data is there (products(), k_layer).
//   [1, 7168] x [7168, 7168] in 4 bits 20 us (16.5), [64, 2048] x [2048, 65536]
//     74 us (70), without the products 40: at 64 rows they are 34 us of the
//     tensor pipe, and x comes from L2 once a step. In groups of 64 rows it takes
//     83, of 32 rows 91: more scales, and more registers than a thread has (88 to
//     200 bytes of them spilled).

#include <cooperative_groups.h>

#include "ckpt.cuh"
#include "tc.cuh"
#include "w4.cuh"

namespace mep {
namespace {

constexpr int kMaxCtas = 152;       // SMs of a GB300; more are not used, the workspace counts on it
constexpr int kWarps = 8;           // across a unit's columns: 16 of its first half and 16 of its second
constexpr int kThreads = 32 * (kWarps + 1);       // a producer's warp beside them
constexpr int kLayerThreads = 32 * (kWarps + 2);  // and one that runs ahead through the sums
constexpr int kUnit = 256;          // columns of a unit
constexpr int kPanels = kUnit / kW4Cols;
constexpr int kPanelRow = 128;      // bytes of a stage's row of 64 bf16 columns
constexpr int kMaxStages = 8;
constexpr int kSmem = 227 * 1024;
constexpr int kChunk = 32;          // tokens of an expert that one unit takes in the layer

// The kernels go by the weights' group: 0 for bf16, else 32, 64 or 128 rows of
// a column in 4 bits.
__host__ __device__ constexpr int step_rows(int group) { return group == 0 ? 64 : 256; }

// ---------------------------------------------------------------------------
// n / d by a product, n < 2^31: with 2^l >= d, m = floor(2^(31+l) / d) + 1 the
// product is off by too little to reach the next quotient.
struct Div {
  uint32_t m;
  int shift;
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return m == 0 ? n : __umulhi(n, m) >> shift; }
};
Div div_of(uint32_t d) {
  int l = 0;
  while ((1u << l) < d) ++l;
  return {d == 1 ? 0u : uint32_t((1ull << (31 + l)) / d + 1), l - 1};
}
// A product's sizes, known on the host: steps of a unit, units of an expert.
struct Shape {
  uint32_t ks, nb;
  Div by_ks, by_nb;
};
Shape shape_of(long long ks, long long nb) {
  return {uint32_t(ks), uint32_t(nb), div_of(uint32_t(ks)), div_of(uint32_t(nb))};
}
// Its units' steps in a row, cut into runs. Up to kOneRun steps a CTA: one run
// each, equal ones. More: runs of a power of two, sixteen to 32 a CTA, taken as
// they come, since some SMs are a fifth slower than others at reading (64 tokens
// of the large layer: 2.72 ms with equal shares, 2.32 this way). In 4 bits, whose
// panels are contiguous, three quarters of the steps are in one long run a CTA
// (16 tokens of the large layer 357 -> 341 us); in bf16, whose rows' pieces lie
// between the other columns', CTAs read faster side by side (1790 us; 1870 with
// long runs). Short runs are a sixteenth of a unit or more, which bounds the
// partial sums.
constexpr uint32_t kOneRun = 32;
struct Phase {
  uint32_t ks, nb;
  uint32_t total, run;       // steps; of a short run
  uint32_t q, first, runs;   // short runs in a CTA's own one, in all own ones; runs, the own ones counted as one each
  uint32_t parts;            // runs that a unit may be cut over
  uint32_t by_run, by_q;     // n / d: 2^32 / d + 1, exact for powers of two and for n * d < 2^32; 0: d is 1
  Div by_ks, by_nb;
};
__host__ __device__ __forceinline__ uint32_t least_run(uint32_t ks) {
  uint32_t run = 4;
  while (run * 16 < ks) run *= 2;
  return run;
}
__host__ __device__ __forceinline__ uint32_t run_of(uint32_t total, uint32_t ks) {
  const uint32_t per = (total + kMaxCtas - 1) / kMaxCtas;
  if (per <= kOneRun) return per > 1 ? per : 1;
  uint32_t run = least_run(ks);
  while (run * 32 <= per) run *= 2;
  return run;
}
// A unit is cut where runs end, into so many parts at most:
__host__ __device__ __forceinline__ uint32_t parts_of(uint32_t ks, uint32_t run) {
  const uint32_t p = (ks - 1) / run + 2;
  return p < ks ? p : ks;
}
__device__ __forceinline__ uint32_t divide(uint32_t n, uint32_t m) { return m == 0 ? n : __umulhi(n, m); }
__device__ __forceinline__ Phase make_phase(uint32_t experts, const Shape& s, bool long_run) {
  Phase p;
  p.ks = s.ks, p.nb = s.nb, p.by_ks = s.by_ks, p.by_nb = s.by_nb;
  p.total = experts * s.nb * s.ks;
  p.run = run_of(p.total, s.ks);
  p.by_run = 0xffffffffu / p.run + 1;
  const uint32_t shorts = divide(p.total + p.run - 1, p.by_run), each = p.total / (gridDim.x * p.run);
  p.q = long_run && each > 1 ? each * 3 / 4 : 1;
  p.by_q = 0xffffffffu / p.q + 1;
  p.first = gridDim.x * p.q;
  p.runs = shorts <= p.first ? divide(shorts + p.q - 1, p.by_q) : gridDim.x + shorts - p.first;
  p.parts = p.run % s.ks == 0 ? 1 : parts_of(s.ks, p.run);
  return p;
}
// Each run a unit: nothing is cut (and nothing asks run_at).
__device__ __forceinline__ void whole_units(Phase& p) {
  p.run = p.ks, p.q = 1, p.first = gridDim.x, p.runs = p.nb, p.parts = 1;
}
// The run of a step; the first step of a run.
__device__ __forceinline__ uint32_t run_at(const Phase& p, uint32_t step) {
  const uint32_t r = divide(step, p.by_run);
  return r < p.first ? divide(r, p.by_q) : gridDim.x + r - p.first;
}
__device__ __forceinline__ uint32_t run_start(const Phase& p, uint32_t run) {
  return min(p.total, (run < gridDim.x ? run * p.q : p.first + run - gridDim.x) * p.run);
}
// Unit u is in runs run_at(u * ks) up to run_at((u + 1) * ks - 1).
__device__ __forceinline__ uint32_t parts_in(const Phase& p, uint32_t unit) {
  return p.parts == 1 ? 1 : run_at(p, (unit + 1) * p.ks - 1) - run_at(p, unit * p.ks) + 1;
}

// ---------------------------------------------------------------------------
// What a CTA's warps have to know of a unit, or of the part of one that is in a
// run. The producer, which waits for room most of the time, works it out. Where
// each of the eight other warps did, a part began with 1100 clocks, now 400, and a
// step takes 1200 (16 tokens of the large layer in 4 bits 302 us, 285 this way).
struct __align__(16) Part {
  int steps, left, rows, columns;  // 0: the end; rows of the sum from its first step on; of x; columns of the unit on
  long long to;                    // its first sum's number
  long long none;
};
// The ring of stages.
struct Ring {
  uint32_t full, empty;         // barriers, 8 bytes each
  uint32_t stage0, stage_bytes; // first stage
  uint32_t x_at;                // of a stage: where the rows of x start
  int stages;
  struct Part* part;            // of a stage that a part starts with
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
// Where a product's weights lie. A unit's four panels of 64 columns are two and
// two: of the first and the second half of its columns.
struct Weights {
  const CUtensorMap* map;           // bf16
  const uint8_t* w4;                // 4 bits
  long long expert, panel, second;  //   bytes of an expert, of a panel; from a unit's first to its third panel
  int unit, col_second;             // panels from unit to unit; bf16: columns from the first to the third
  int columns;                      // of a half that there are (both products have the first panel of a unit)
  bool gated;                       // the halves are gate and up columns, each counted to `columns`
  int K;                            // rows
};
// Rows of x: `planes` of them after one another (the activation's two). They come
// in tiles of 64 columns, 128-byte swizzled: in the product all rows in one copy
// (x is the map's, its box the tile), in the layer from bf16 four rows of the list
// in one or, of the activation, whose rows are in the list's order, eight (a lane
// issues a copy in some 80 clocks: 64 tokens, 8 each of 32 experts, 7168 x 1408,
// row by row 515 us, so 370 to 376). In 4 bits, where a step has four times the columns
// and tiles would be four times as many copies, the layer copies row by row.
struct Rows {
  const CUtensorMap* map;
  const char* p;
  const uint16_t* token;  // row of x of a row of the list; NULL: the same
  long long pitch;        // bytes
  int K;                  // bf16 of a row
  int planes;
};
// Where a product's sums go: rows' parts of `pitch` of them.
struct Sums {
  uint32_t pitch;
  int unit, half;    // columns from unit to unit, from a unit's first half to its second
  int limit, inner;  // j * unit + column + (of the second half) inner is below limit where a column is there
};

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Four rows, 64 columns from x on.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, int x, const int (&y)[4], uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], "
      "[%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void bulk(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __noinline__ void grid_barrier() { cooperative_groups::this_grid().sync(); }
// Rows that a stage has room for (as many as a unit's instantiation computes).
__device__ __forceinline__ int tile_rows(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }" : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok;
}
// A whole warp waits; the same answer in every lane.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const Ring& r) {
  if (__all_sync(MEP_FULL_MASK, mbar_try_wait_long(bar, parity))) return true;
  return __all_sync(MEP_FULL_MASK, wait_phase(bar, parity, r.abort, r.status));
}

// ---------------------------------------------------------------------------
// The producer warp's side. A step's stage is full once its weights have come
// and its rows have: two arrivals. What a step needs is worked out where its
// unit begins; a step itself has to cost less than its bytes take to come (a
// stage of 32 KB in 0.75 us).
template <int G, bool TILES> struct Stream {
  static constexpr int BK = step_rows(G), pitch = BK * 2 + 16;
  const Ring& r;
  const uint16_t *expert, *start;
  static constexpr int block = G == 0 ? 0 : w4_block_bytes(G);
  Phase p;
  Weights w;
  Rows x;
  Sums o;
  uint32_t run_part = 0;       // which part of its unit the run starts with
  bool fresh = false;          // a part starts with this step
  uint32_t step = 0, end = 0;  // of the run
  uint32_t s, j, entry;        // step of the unit, unit of the expert, the expert's entry
  uint32_t tx;                 // bytes of a full step's weights
  int e, rows_n, panels;       // expert, rows of x; a bit for each panel that is there
  const uint8_t* unit_w;       // 4 bits: the unit's first panel
  const char* row[2];          // this lane's rows of x
  uint32_t at[2];              // and where they go in a stage
  int y[4];                    // rows of this lane's copy of a tile

  __device__ __forceinline__ Stream(const Ring& ring, const uint16_t* e_, const uint16_t* s_)
      : r(ring), expert(e_), start(s_) {}
  __device__ __forceinline__ void unit() {
    const int lane = threadIdx.x & 31, first = start[entry], panel = j * w.unit, pl = x.planes - 1;
    rows_n = (start[entry + 1] - first) << pl, e = expert[entry], fresh = true;
    if (TILES && G == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i)  // beyond the last row the last one again: products of a column that no one reads
        y[i] = x.token != nullptr ? x.token[first + min(4 * lane + i, rows_n - 1)] : 2 * first + 8 * lane;
    }
    if (TILES) rows_n = tile_rows(rows_n);
    const int count = (w.columns + kW4Cols - 1) / kW4Cols - panel;
    panels = w.gated ? (count > 1 ? 15 : 5) : count >= 4 ? 15 : (1 << count) - 1;
    tx = __popc(panels) * (G == 0 ? step_rows(G) * kPanelRow : 2 * block);
    if (G != 0) unit_w = w.w4 + e * w.expert + panel * w.panel;
#pragma unroll
    for (int i = 0; i < 2 && !TILES; ++i) {
      const int q = lane + 32 * i;
      at[i] = r.x_at + q * pitch;
      if (q < rows_n) {
        const int of = first + (q >> pl);
        row[i] = x.p + (((x.token == nullptr ? of : x.token[of]) << pl) + (q & pl)) * x.pitch;
      }
    }
  }
  __device__ __forceinline__ void seek(uint32_t run) {
    step = run_start(p, run), end = run_start(p, run + 1);
    if (step >= end) return;
    const uint32_t u = p.by_ks(step);
    s = step - u * p.ks, entry = p.by_nb(u), j = u - entry * p.nb;
    run_part = p.parts == 1 ? 0 : run - run_at(p, u * p.ks);
    unit();
  }
  __device__ __forceinline__ void own(const Phase& p_, const Weights& w_, const Rows& x_, const Sums& o_) {
    p = p_, w = w_, x = x_, o = o_;
    seek(blockIdx.x);
  }
  __device__ __forceinline__ void next() {
    fresh = false;
    if (++step == end || ++s < p.ks) return;
    s = 0, run_part = 0;
    if (++j == p.nb) j = 0, ++entry;
    unit();
  }
  __device__ __forceinline__ void weights(int slot) const {  // one lane
    const uint32_t bar = r.full + 8 * slot, dst = r.stage0 + slot * r.stage_bytes;
    if (fresh) {
      const int first = start[entry], n = (start[entry + 1] - first) * x.planes;
      Part part;
      part.steps = min(p.ks - s, end - step), part.left = w.K - int(s * BK), part.rows = n, part.columns = o.limit - int(j) * o.unit;
      part.to = ((long long)first * p.parts + run_part) * o.pitch + j * o.unit, part.none = 0;
      r.part[slot] = part;
    }
    if (G == 0) {
      constexpr uint32_t bytes = step_rows(G) * kPanelRow;
      const int col = j * w.unit * kW4Cols, k = s * BK;
      mbar_expect_tx(bar, tx);
#pragma unroll
      for (int q = 0; q < kPanels; ++q)
        if (panels >> q & 1) tma_3d(dst + q * bytes, w.map, col + (q & 1) * kW4Cols + (q >> 1) * w.col_second, k, e, bar);
    } else {
      const uint8_t* src = unit_w + s * (2 * block);
      const uint32_t half = 2 * int(s) + 1 == (w.K + kW4Rows - 1) / kW4Rows;  // the last step may have one block
      mbar_expect_tx(bar, tx >> half);
#pragma unroll
      for (int q = 0; q < kPanels; ++q)
        if (panels >> q & 1) bulk(dst + q * 2 * block, src + (q & 1) * w.panel + (q >> 1) * w.second, (2 * block) >> half, bar);
    }
  }
  __device__ __forceinline__ void rows(int slot) const {  // the warp
    const int lane = threadIdx.x & 31, k0 = s * BK, bytes = 2 * min(BK, x.K - k0);
    const uint32_t bar = r.full + 8 * slot, dst = r.stage0 + slot * r.stage_bytes;
    if (TILES && G == 0) {
      if (lane == 0) mbar_expect_tx(bar, rows_n * BK * 2);
      if (x.token != nullptr) {
        if (lane < rows_n / 4) tma_gather4(dst + r.x_at + lane * 512, x.map, k0, y, bar);
      } else {
        if (lane < rows_n / 8) tma_2d(dst + r.x_at + lane * 1024, x.map, k0, y[0], bar);
      }
      return;
    }
    if (TILES) {  // zeros beyond the rows and the sum's end
      if (lane == 0) {
        mbar_expect_tx(bar, rows_n * BK * 2);
#pragma unroll
        for (int i = 0; i < BK / 64; ++i) tma_2d(dst + r.x_at + i * rows_n * 128, x.map, k0 + 64 * i, 0, bar);
      }
      return;
    }
    if (bytes < 2 * BK) {  // beyond the sum's end the weights are zeros: what they meet must be numbers
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (lane + 32 * i < rows_n)
          for (int b = bytes; b < 2 * BK; b += 16)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + at[i] + b), "r"(0) : "memory");
      fence_async();
      __syncwarp();
    }
    if (lane == 0) mbar_expect_tx(bar, rows_n * bytes);
    // lanes' copies go out one after another: a branch leaves the others out
    if (lane < rows_n) bulk(dst + at[0], row[0] + 2 * k0, bytes, bar);
    if (rows_n > 32 && lane + 32 < rows_n) bulk(dst + at[1], row[1] + 2 * k0, bytes, bar);
  }
  // Before a barrier of the grid: the weights of as many steps of the CTA's own
  // run as the ring has room for, and their rows where these are there already.
  __device__ __forceinline__ void ahead(Cursor& c, bool with_rows) {
#pragma unroll 1
    for (int i = 0; i < r.stages && step < end; ++i) {
      if (!warp_wait(r.empty + 8 * c.slot, c.parity ^ 1, r)) break;
      if ((threadIdx.x & 31) == 0) weights(c.slot);
      if (with_rows) rows(c.slot);
      c.next(r.stages);
      next();
    }
  }
  // After it: the rows that are due, of the stages from `behind` on; the rest of
  // the own run, further runs off the counter, the end's mark.
  __device__ __forceinline__ void feed(Cursor& c, Cursor behind, bool due, uint32_t* counter) {
    const int lane = threadIdx.x & 31;
    const bool more = p.runs > gridDim.x;
    uint32_t taken = 0;
    if (more && lane == 0) taken = atomicAdd(counter, 1u);  // on its way while the run is fed
    if (due) {
      const uint32_t to = step, stop = end;
      seek(blockIdx.x);
      while (step < to) {
        rows(behind.slot);
        behind.next(r.stages);
        next();
      }
      end = stop;
    }
#pragma unroll 1
    while (true) {
      if (step == end) {
        const uint32_t run = more ? gridDim.x + __shfl_sync(MEP_FULL_MASK, taken, 0) : p.runs;
        if (run >= p.runs) break;
        seek(run);
        if (lane == 0) taken = atomicAdd(counter, 1u);
      }
      if (!warp_wait(r.empty + 8 * c.slot, c.parity ^ 1, r)) return;
      if (lane == 0) weights(c.slot);
      rows(c.slot);
      c.next(r.stages);
      next();
    }
    if (!warp_wait(r.empty + 8 * c.slot, c.parity ^ 1, r)) return;
    if (lane == 0) {
      r.part[c.slot].steps = 0;
      arrive(r.full + 8 * c.slot);
      arrive(r.full + 8 * c.slot);
    }
    c.next(r.stages);
    __syncwarp();
  }
};

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
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
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
// Operand of one step, over 64: the word's four pairs of q + 8 at bits 0, 4, 8
// and 12 of either half. Bits 0-7 of a bf16 without more are that whole number
// times 2^-133 (subnormal up to 127, the first binade above), so that one fused
// multiply-add takes a pair to q / 64, exactly, wherever in the byte it was.
__device__ __forceinline__ void widen_q(uint32_t word, uint32_t (&a)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i, word >>= 8) {
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(a[2 * i]) : "r"(word & 0x000f000fu), "r"(0x7f007f00u), "r"(0xbe00be00u));
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(a[2 * i + 1]) : "r"(word & 0x00f000f0u), "r"(0x7d007d00u), "r"(0xbe00be00u));
  }
}
constexpr float kQ = 64.f;

// This warp's share of a stage: 16 columns of either half.
template <int G, bool TILES, int NT>
__device__ __forceinline__ void stage_product(float (&acc)[2][NT][4], uint32_t stage, const Ring& r, int warp,
                                              int blocks, int tile) {
  constexpr int BK = step_rows(G), pitch = BK * 2 + 16;
  const int lane = threadIdx.x & 31;
  // eight rows of x from row 8 n on, 32 columns from k on: where this lane's part starts
  const auto x_at = [&](int n, int k) -> uint32_t {
    if (TILES)
      return stage + r.x_at + (k >> 6) * (tile * 128) + (8 * n + (lane & 7)) * 128 +
             ((((k >> 3 & 7) + (lane >> 3)) ^ (lane & 7)) << 4);
    return stage + r.x_at + (8 * n + (lane & 7)) * pitch + 16 * (lane >> 3) + 2 * k;
  };
  if (G == 0) {
    const uint32_t wa = stage + (warp >> 2) * (BK * kPanelRow) + ((lane >> 4) * 8 + (lane & 7)) * kPanelRow +
                        (((2 * (warp & 3) + ((lane >> 3) & 1)) ^ (lane & 7)) << 4);
#pragma unroll
    for (int k = 0; k < BK; k += 32) {
      uint32_t a[2][2][4];
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int s = 0; s < 2; ++s) ldmatrix4_trans(a[q][s], wa + q * (2 * BK * kPanelRow) + (k + 16 * s) * kPanelRow);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t b[4];
        ldmatrix4(b, x_at(n, k));
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int q = 0; q < 2; ++q) mma(acc[q][n], a[q][s], b[2 * s], b[2 * s + 1]);
      }
    }
  } else {
    // Everything that a block of 128 rows needs of the stage is asked for at once;
    // with more than 32 rows of x the block is gone through again. In the layer, where
    // that is rare, for every 16 of them: with 32 at once the registers ran short in
    // the instantiations for fewer rows too (16 tokens, 256 experts, 7168 x 1408: 281
    // us, 260 this way; 64 tokens, 6 each of 64, 2048 x 1408: 126 and 112). The
    // product, of which 64 rows are no rare case, takes 32 (74 us; 87 by 16).
    constexpr int NS = NT < 4 ? NT : NT == 8 && !TILES ? 2 : 4, block = w4_block_bytes(G > 0 ? G : 128), per = G > 0 ? G / 32 : 1;  // groups: per * 32 rows
    constexpr bool early = NT <= 2;                                                                       // x too
    uint4 w[2][2];
    uint32_t x[early ? 4 : 1][early ? NS : 1][4], scale[4][2];
#pragma unroll
    for (int i = 0; i < 2 * (NT / NS); ++i) {
      const int n0 = (i >> 1) * NS, b = i & 1;
      if (b >= blocks) continue;
      const uint32_t wb = stage + (warp >> 2) * 2 * block + b * block;
      const uint32_t at = wb + ((warp & 3) * 32 + lane) * 16, sb = wb + kW4Pairs + ((warp & 3) * 8 + (lane >> 2)) * 4;
#pragma unroll
      for (int h = 0; h < 2; ++h) w[h][0] = lds128(at + 2048 * h), w[h][1] = lds128(at + 2048 * h + 4 * block);
      if (early) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int n = 0; n < NS; ++n) ldmatrix4(x[k][n], x_at(n0 + n, 128 * b + 32 * k));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if ((k + 1) % per == 0)
#pragma unroll
          for (int q = 0; q < 2; ++q) scale[k][q] = lds32(sb + k / per * 128 + q * 4 * block);
      float sum[2][NS][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // 32 rows
        uint32_t a[2][2][4];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint4& v = w[k >> 1][q];
            widen_q(k & 1 ? (s ? v.w : v.z) : (s ? v.y : v.x), a[q][s]);
          }
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          if (!early) ldmatrix4(x[0][0], x_at(n0 + n, 128 * b + 32 * k));
          const uint32_t(&f)[4] = early ? x[k][n] : x[0][0];
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              if (s == 0 && k % per == 0)
                mma_first(sum[q][n], a[q][s], f[2 * s], f[2 * s + 1]);
              else
                mma(sum[q][n], a[q][s], f[2 * s], f[2 * s + 1]);
            }
        }
        if ((k + 1) % per == 0) {  // a group ends
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float lo = __uint_as_float(scale[k][q] << 16), hi = __uint_as_float(scale[k][q] & 0xffff0000u);
#pragma unroll
            for (int n = 0; n < NS; ++n) {
              float(&to)[4] = acc[q][n0 + n];
              to[0] = fmaf(lo, sum[q][n][0], to[0]);
              to[1] = fmaf(lo, sum[q][n][1], to[1]);
              to[2] = fmaf(hi, sum[q][n][2], to[2]);
              to[3] = fmaf(hi, sum[q][n][3], to[3]);
            }
          }
        }
      }
    }
  }
}

// The steps of a part, then their sums out. PUT(half, column of the half, row, two
// values: of this row of x and the next one). `dry`: see products().
template <int G, bool TILES, int NT, typename Put>
__device__ __forceinline__ bool unit_product(int steps, int left, const Ring& r, Cursor& c, int rows, bool dry, Put put) {
  constexpr int BK = step_rows(G);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float acc[2][NT][4];
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[q][n][0] = acc[q][n][1] = acc[q][n][2] = acc[q][n][3] = 0.f;
  bool there = true;  // the part's start has been waited for
#pragma unroll 1
  for (; steps > 0; --steps, left -= BK) {
    if (!dry && !__all_sync(MEP_FULL_MASK, there) && !warp_wait(r.full + 8 * c.slot, c.parity, r)) return false;
    Cursor after = c;
    after.next(r.stages);
    there = !dry && steps > 1 && mbar_test(r.full + 8 * after.slot, after.parity);  // asked for while this step is worked on
    const int blocks = G != 0 ? (left + kW4Rows - 1) / kW4Rows : 0;
    stage_product<G, TILES, NT>(acc, r.stage0 + c.slot * r.stage_bytes, r, warp, blocks, tile_rows(rows));
    __syncwarp();
    if (dry) continue;
    if (lane == 0) arrive(r.empty + 8 * c.slot);
    c.next(r.stages);
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (8 * n >= rows) break;
    const int row = 8 * n + 2 * (lane & 3);
    if (row < rows && !dry) {
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float f = G != 0 ? kQ : 1.f;
          put(q, 16 * warp + (lane >> 2) + 4 * i, row, f * acc[q][n][i], f * acc[q][n][i + 1]);
        }
    }
  }
  return true;
}

// All steps that this CTA is fed, of up to `most` rows of x a unit. PUT(part, and
// as above). What a kernel executes for the first time comes from far away, at
// some 25 ns an instruction: dry, the code is run through once, on whatever the
// first stage holds and to no effect, while that stage's bytes are on their way.
enum Run { kReal, kDry, kDryThenReal };
template <int G, bool TILES, int NTMAX, typename Put>
__device__ __forceinline__ void products(const Ring& r, Cursor& c, Run how, int most, Put put) {
  bool dry = how != kReal;
#pragma unroll 1
  while (true) {
    Part part = {1, step_rows(G), most, 0, 0, 0};
    if (!dry) {
      if (!warp_wait(r.full + 8 * c.slot, c.parity, r)) return;
      part = r.part[c.slot];
      if (part.steps == 0) break;
    }
    const auto f = [&](int q, int col, int row, float v0, float v1) { put(part, q, col, row, v0, v1); };
    bool ok;
    if (part.rows <= 8)
      ok = unit_product<G, TILES, 1>(part.steps, part.left, r, c, part.rows, dry, f);
    else if (part.rows <= 16)
      ok = unit_product<G, TILES, 2>(part.steps, part.left, r, c, part.rows, dry, f);
    else if (NTMAX <= 4 || part.rows <= 32)
      ok = unit_product<G, TILES, 4>(part.steps, part.left, r, c, part.rows, dry, f);
    else
      ok = unit_product<G, TILES, NTMAX>(part.steps, part.left, r, c, part.rows, dry, f);
    if (!ok || how == kDry) return;
    dry = false;
  }
  __syncwarp();
  if ((threadIdx.x & 31) == 0) arrive(r.empty + 8 * c.slot);
  c.next(r.stages);
}

// Stages for up to `rows` rows of x. Tiles start on a swizzle's boundary.
template <int G, bool TILES> __device__ __forceinline__ void size_ring(Ring& r, uint32_t room, int rows) {
  r.x_at = G == 0 ? kPanels * step_rows(G) * kPanelRow : kPanels * 2 * w4_block_bytes(G > 0 ? G : 128);
  if (TILES) r.x_at = (r.x_at + 1023) / 1024 * 1024;
  r.stage_bytes = (r.x_at + tile_rows(rows) * (step_rows(G) * 2 + (TILES ? 0 : 16)) + 1023) / 1024 * 1024;
  r.stages = min(kMaxStages, int(room / r.stage_bytes));
}

struct Head {  // start of shared memory
  uint64_t full[kMaxStages], empty[kMaxStages];
  Part part[kMaxStages];
  int warp_sums[32];
  int abort, bad, most, rows, go;
  Phase phase[2];
};
constexpr uint32_t kHeadBytes = 1024;

__device__ __forceinline__ void init_names(Ring& r, Head* h, int32_t* status) {
  r.full = smem_u32(h->full), r.empty = smem_u32(h->empty);
  r.part = h->part, r.abort = &h->abort, r.status = status;
}
__device__ __forceinline__ void init_ring(Ring& r, Head* h, int32_t* status) {
  init_names(r, h, status);
  if (threadIdx.x < kMaxStages) {
    mbar_init(r.full + 8 * threadIdx.x, 2);  // weights, rows
    mbar_init(r.empty + 8 * threadIdx.x, kWarps);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x == 0) h->abort = h->bad = h->most = 0;
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

// Items [0, n) over `warps` warps of every CTA, one CTA's after another's: a few items are on as many SMs.
struct Spread {
  uint32_t i, step;
};
__device__ __forceinline__ Spread spread(int warps) {
  return {((threadIdx.x >> 5) * gridDim.x + blockIdx.x) * 32 + (threadIdx.x & 31), warps * gridDim.x * 32};
}

// ---------------------------------------------------------------------------
struct LayerArgs {
  const __nv_bfloat16* x;
  const int32_t* idx;
  const float* topk_w;
  const uint8_t *w1, *w2;
  int32_t* status;
  int T, K, E, H, F;
  Shape s1, s2;
  int counted;  // the counters may be in use
  Div by_k;
  uint32_t* counters;
  float *part1, *part2;
  __nv_bfloat16* act;
  __nv_bfloat16* out;
};

__host__ __device__ __forceinline__ int max_entries(int T, int K, int E) {
  return (E < T * K ? E : T * K) + T * K / kChunk;
}
__host__ __device__ __forceinline__ uint32_t list_bytes(int T, int K, int E) {
  return (2u * (2 * max_entries(T, K, E) + 1 + 3 * T * K) + 4u * T * K + 1023) / 1024 * 1024;
}

struct Lists {              // in shared memory
  float* weight;            // of an assignment, as given
  uint16_t *expert, *start; // of an entry: its expert, its first row (one more at the end)
  uint16_t *entry, *token;  // of a row
  uint16_t* row;            // of an assignment; kNone
};
constexpr uint16_t kNone = 0xffff;

// The experts in use in ascending order, each one's tokens in order, more than
// kChunk of them in several entries; where each assignment went. What comes from
// memory is asked for at the start, the barriers' words are set up meanwhile.
// The warps that make it: four of the products' and the producer.
constexpr int kListWarps = 4;
__device__ __forceinline__ void list_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * (kListWarps + 1)) : "memory"); }

__device__ __forceinline__ void make_list(const LayerArgs& a, Ring& r, Head* h, char* scratch, const Lists& l, bool long_run) {
  unsigned long long* mask = reinterpret_cast<unsigned long long*>(scratch);
  uint32_t* e_at = reinterpret_cast<uint32_t*>(mask + a.E);  // entry and first row of an expert
  constexpr int threads = 32 * (kListWarps + 1);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5 == kWarps ? kListWarps : threadIdx.x >> 5;
  const int tid = 32 * warp + lane, A = a.T * a.K;
  const int mine = tid < A ? __ldg(a.idx + tid) : -1;
  const float weight = tid < A ? __ldg(a.topk_w + tid) : 0.f;
  const int held = tid == 0 ? read_status(a.status) : 0;
  init_ring(r, h, a.status);
  for (int e = tid; e < a.E; e += threads) mask[e] = 0;
  if (tid == 0 && blockIdx.x == 0) a.counters[0] = a.counters[1] = 0;
  list_sync();
  if (tid == 0) h->go = held == 0;
#pragma unroll 1
  for (int i = tid, e = mine; i < A;) {
    if (e >= 0 && e < a.E) {
      const unsigned long long bit = 1ull << a.by_k(i);
      if (atomicOr(&mask[e], bit) & bit) h->bad = 1;
    } else if (e != -1) {
      h->bad = 1;
    }
    if ((i += threads) < A) e = a.idx[i];
  }
  list_sync();
  // entries and rows before each thread's experts, in one word
  const int per = a.E <= threads ? 1 : (a.E + threads - 1) / threads, lo = min(a.E, tid * per), hi = min(a.E, lo + per);
  uint32_t sum = 0;
  int most = 0;
#pragma unroll 1
  for (int e = lo; e < hi; ++e) {
    const int n = __popcll(mask[e]);
    sum += ((n + kChunk - 1) / kChunk << 16) + n;
    most = max(most, n);
  }
  const uint32_t incl = warp_incl_scan(sum);
  most = __reduce_max_sync(MEP_FULL_MASK, most);
  if (lane == 31) h->warp_sums[warp] = incl;
  if (lane == 0 && most > 0) atomicMax(&h->most, most);
  list_sync();
  const uint32_t w = lane < threads / 32 ? h->warp_sums[lane] : 0;
  const uint32_t all = __reduce_add_sync(MEP_FULL_MASK, w);
  uint32_t before = __reduce_add_sync(MEP_FULL_MASK, lane < warp ? w : 0) + incl - sum;
#pragma unroll 1
  for (int e = lo; e < hi; ++e) {
    const int n = __popcll(mask[e]);
    int entry = before >> 16;
    const int row = before & 0xffff;
    e_at[e] = before;
    for (int q = 0; q < n; q += kChunk, ++entry) l.expert[entry] = e, l.start[entry] = row + q;
    before += ((n + kChunk - 1) / kChunk << 16) + n;
  }
  if (lane == 0 && warp < 2) {
    const bool run = h->go && !h->bad;
    h->phase[warp] = make_phase(run ? all >> 16 : 0, warp == 0 ? a.s1 : a.s2, long_run);
    if (warp == 0) {
      h->rows = run ? all & 0xffff : 0;
      l.start[all >> 16] = all & 0xffff;
    }
  }
  list_sync();
  if (!h->bad)
#pragma unroll 1
    for (int i = tid, e = mine; i < A;) {
      l.weight[i] = i == tid ? weight : a.topk_w[i];
      if (e < 0) {
        l.row[i] = kNone;
      } else {
        const int t = a.by_k(i), rank = __popcll(mask[e] & ((1ull << t) - 1)), row = (e_at[e] & 0xffff) + rank;
        l.row[i] = row, l.token[row] = t, l.entry[row] = (e_at[e] >> 16) + rank / kChunk;
      }
      if ((i += threads) < A) e = a.idx[i];
    }
  fence_async();  // the ring's copies come into the same memory
}

template <int G> __device__ __forceinline__ Weights first_weights(const LayerArgs& a, const CUtensorMap* map) {
  const long long m = G != 0 ? w4_matrix_bytes(a.H, a.F, G) : 0, q = G != 0 ? w4_panel_bytes(a.H, G) : 0;
  return {map, a.w1, 2 * m, q, m, 2, a.F, a.F, true, a.H};
}
__device__ __forceinline__ Sums first_sums(const LayerArgs& a) { return {2u * a.F, kUnit / 2, a.F, a.F, 0}; }
__device__ __forceinline__ Sums second_sums(const LayerArgs& a) { return {uint32_t(a.H), kUnit, kUnit / 2, a.H, kUnit / 2}; }
template <int G> __device__ __forceinline__ Weights second_weights(const LayerArgs& a, const CUtensorMap* map) {
  const long long m = G != 0 ? w4_matrix_bytes(a.F, a.H, G) : 0, q = G != 0 ? w4_panel_bytes(a.F, G) : 0;
  return {map, a.w2, m, q, 2 * q, 4, 2 * kW4Cols, a.H, false, a.F};
}

// silu(g) * u. Below -88, where e^-g leaves fp32, 1 + e^-g is e^-g to 2^-126: g *
// e^g * u, with e^g as the square of e^(g/2), u between the two factors, is what
// fp32 holds of it (g = -100 and u = 1e38 make -3.7e-4; a quotient flushed to 0).
__device__ __forceinline__ float silu_times(float g, float u) {
  if (g < -88.f) {
    const float h = expf(0.5f * g);
    return g * h * u * h;
  }
  return g / (1.f + expf(-g)) * u;
}

constexpr float kTopBf16 = 255.f * 0x1p120f;  // bf16's largest number

// The activation of n quads of columns: the first product's parts added up, in
// order, then silu(g) * u as two bf16.
__device__ __forceinline__ void activate(const LayerArgs& a, const Phase& p, const Lists& l, uint32_t n, Spread s, bool dry) {
  constexpr uint32_t quads = kUnit / 8;  // of a unit's gates
#pragma unroll 1
  for (; s.i < n; s.i += s.step) {
    const uint32_t unit = s.i / quads, row = p.by_nb(unit), j = unit - row * p.nb, col = j * (kUnit / 2) + s.i % quads * 4;
    if (int(col) >= a.F) continue;
    const uint32_t parts = parts_in(p, l.entry[row] * p.nb + j);
    const float* in = a.part1 + (long long)row * p.parts * (2 * a.F) + col;
    float g[4] = {}, u[4] = {};
#pragma unroll 4
    for (uint32_t q = 0; q < parts; ++q, in += 2 * a.F) {
      const float4 vg = __ldcg(reinterpret_cast<const float4*>(in));
      const float4 vu = __ldcg(reinterpret_cast<const float4*>(in + a.F));
      g[0] += vg.x, g[1] += vg.y, g[2] += vg.z, g[3] += vg.w;
      u[0] += vu.x, u[1] += vu.y, u[2] += vu.z, u[3] += vu.w;
    }
    __nv_bfloat16 hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float v = silu_times(g[k], u[k]);
      const bool beyond = fabsf(v) > kTopBf16 && !isinf(v);  // a number in fp32, which rounding might make an infinity
      hi[k] = __float2bfloat16_rn(beyond ? copysignf(kTopBf16, v) : v);
      const float rest = v - __bfloat162float(hi[k]);
      lo[k] = __float2bfloat16_rn(isfinite(rest) ? rest : 0.f);  // an infinity stays one
    }
    __nv_bfloat16* o = a.act + (long long)row * 2 * a.F + col;
    if (!dry) {
      *reinterpret_cast<uint2*>(o) = *reinterpret_cast<uint2*>(hi);
      *reinterpret_cast<uint2*>(o + a.F) = *reinterpret_cast<uint2*>(lo);
    }
  }
}

// n lanes' items of the output: eight lanes share 16 columns, each a part of the
// token's experts, whose parts are added up in order.
__device__ __forceinline__ void combine(const LayerArgs& a, const Phase& p, const Lists& l, uint32_t n, Spread s, bool dry) {
  constexpr uint32_t items = kUnit / 16 * 8;
#pragma unroll 1
  for (; s.i < n; s.i += s.step) {
    const uint32_t u = s.i / items, t = p.by_nb(u), j = u - t * p.nb, col = j * kUnit + s.i % items / 8 * 16;
    if (int(col) >= a.H) continue;
    const bool full = int(col) + 16 <= a.H;  // else eight columns
    float v[16] = {};
#pragma unroll 1
    for (int k = s.i % 8; k < a.K; k += 8) {
      const uint32_t row = l.row[t * a.K + k];
      if (row == kNone) continue;
      const float w = l.weight[t * a.K + k];
      const uint32_t parts = parts_in(p, l.entry[row] * p.nb + j);
      const float* in = a.part2 + (long long)row * p.parts * a.H + col;
      float y[16] = {};
#pragma unroll 2
      for (uint32_t q = 0; q < parts; ++q, in += a.H) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i >= 2 && !full) break;
          const float4 f = __ldcg(reinterpret_cast<const float4*>(in) + i);
          y[4 * i] += f.x, y[4 * i + 1] += f.y, y[4 * i + 2] += f.z, y[4 * i + 3] += f.w;
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = fmaf(w, y[i], v[i]);
    }
    // halves of the lanes' sums change hands: eight lanes end with two outputs each
    const unsigned lanes = 0xffu << (threadIdx.x & 24);
    const int lane = threadIdx.x & 7;
#pragma unroll
    for (int d = 4, left = 8; d > 0; d >>= 1, left >>= 1)
#pragma unroll
      for (int i = 0; i < left; ++i) {
        const bool up = lane & d;
        const float mine = up ? v[left + i] : v[i], other = up ? v[i] : v[left + i];
        v[i] = mine + __shfl_xor_sync(lanes, other, d);
      }
    const int at = (lane & 4 ? 8 : 0) + (lane & 2 ? 4 : 0) + (lane & 1 ? 2 : 0);
    if ((full || at < 8) && !dry)
      *reinterpret_cast<__nv_bfloat162*>(a.out + (long long)t * a.H + col + at) = __floats2bfloat162_rn(v[0], v[1]);
  }
}

template <int G>
__global__ void __launch_bounds__(kLayerThreads, 1)
    k_layer(const __grid_constant__ CUtensorMap map1, const __grid_constant__ CUtensorMap map2,
            const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_act, const LayerArgs a) {
  constexpr bool TILES = G == 0;
  extern __shared__ __align__(1024) char smem[];
  Head* h = reinterpret_cast<Head*>(smem);
  Lists l;
  {
    const int cap = max_entries(a.T, a.K, a.E), A = a.T * a.K;
    l.weight = reinterpret_cast<float*>(smem + kHeadBytes);
    l.expert = reinterpret_cast<uint16_t*>(l.weight + A);
    l.start = l.expert + cap;
    l.entry = l.start + cap + 1;
    l.token = l.entry + A;
    l.row = l.token + A;
  }
  const uint32_t used = kHeadBytes + list_bytes(a.T, a.K, a.E);
  const int warp = threadIdx.x >> 5;
  Ring r;
  // The list is made by some of the warps. The others meanwhile run through the
  // product, dry; all meet at a barrier, where each has got to. Then the last warp
  // runs through the two sums, dry (before, their first instructions took 2 to 4
  // us each, most of it after a barrier when nothing else was under way).
  if (warp < kListWarps || warp == kWarps) {
    make_list(a, r, h, smem + used, l, G != 0);
  } else {
    r.stage0 = smem_u32(smem + used), r.stage_bytes = r.x_at = 0, r.stages = 1;
  }
  const auto list_made = [&]() {
    asm volatile("barrier.sync 0;" ::: "memory");
    init_names(r, h, a.status);
    r.stage0 = smem_u32(smem + used);
    size_ring<G, TILES>(r, kSmem - used, 2 * min(h->most, kChunk));
  };
  // How many barriers there are does not depend on what is read: every CTA comes
  // to all of them, whatever another stream does to the status word meanwhile.
  const bool counted = a.counted;
  Cursor c;
  if (warp == kWarps) {
    list_made();
    if (h->go && h->bad && threadIdx.x == 32 * kWarps) set_status(a.status, MEP_ERR_BAD_ROUTING);
    const Phase &p1 = h->phase[0], &p2 = h->phase[1];
    Stream<G, TILES> t(r, l.expert, l.start);
    Cursor behind;
    t.own(p1, first_weights<G>(a, &map1), {&map_x, reinterpret_cast<const char*>(a.x), l.token, 2LL * a.H, a.H, 1},
          first_sums(a));
    t.ahead(c, true);
    if (counted) grid_barrier();
#pragma unroll 1
    for (int phase = 0; phase < 2; ++phase) {
      t.feed(c, behind, phase == 1, a.counters + phase);
      if (phase == 0) {  // the ring fills while the activation is computed
        behind = c;
        t.own(p2, second_weights<G>(a, &map2), {&map_act, reinterpret_cast<const char*>(a.act), nullptr, 2LL * a.F, a.F, 2},
              second_sums(a));
        t.ahead(c, false);
        grid_barrier();
      }
      grid_barrier();
      fence_async();
    }
  } else {
    // Two turns of product and sum; -1: the product, dry; -3, -2: the sums, dry.
    const bool helper = warp > kWarps;
    int phase = -1;
    if (helper || warp < kListWarps) {
      list_made();
      if (counted) grid_barrier();
      phase = !helper ? 0 : h->rows > 0 ? -3 : -1;
    }
#pragma unroll 1
    for (; phase < (helper ? -1 : 2); ++phase) {
      const bool dry = phase < -1, second = dry ? phase == -2 : phase == 1;
      const Phase& p = h->phase[second];
      if (!dry) {
        const Sums o = second ? second_sums(a) : first_sums(a);
        float* out = second ? a.part2 : a.part1;
        const uint32_t pitch = p.parts * o.pitch;
        products<G, TILES, kChunk / 4>(r, c, phase < 0 ? kDry : kReal, 1,
                                       [&](const Part& part, int q, int col, int row, float v0, float v1) {
                                         if (col + q * o.inner >= part.columns) return;
                                         // the two rows: the activation's two of one token; else two tokens. An
                                         // infinite weight makes the first one's sum what it is to be, and the
                                         // second's anything (infinity times 0 or times the other sign)
                                         float* to = out + part.to + (long long)(second ? row >> 1 : row) * pitch + q * o.half + col;
                                         *to = second && isfinite(v0) ? v0 + v1 : v0;
                                         if (!second && row + 1 < part.rows) to[pitch] = v1;
                                       });
        if (phase < 0) {
          list_made();
          if (counted) grid_barrier();
          continue;
        }
        grid_barrier();
      }
      Spread s = spread(kWarps);
      if (dry) s.i = threadIdx.x & 31, s.step = 0x40000000;
      if (!second) {
        activate(a, p, l, dry ? 32 : h->rows * p.nb * (kUnit / 8), s, dry);
        if (!dry) {
          fence_async();
          grid_barrier();
        }
      } else if (h->go && !h->bad) {
        combine(a, p, l, dry ? 32 : a.T * p.nb * (kUnit / 16 * 8), s, dry);
      }
    }
    if (helper)
      for (int i = 0; i < 3; ++i) grid_barrier();
  }
  settle(r);
}

// ---------------------------------------------------------------------------
struct ProductArgs {
  const __nv_bfloat16* x;
  const uint8_t* w4;
  int32_t* status;
  int T, K, N, y_type;
  Shape shape;
  int whole;  // a run is a unit
  uint32_t* counter;
  __nv_bfloat16* padded;  // rows of x that are whole 16-byte vectors, where K is not a multiple of 8
  float* part;
  void* y;
};

__device__ __forceinline__ void put_y(const ProductArgs& a, long long at, float v) {
  if (a.y_type == MEP_BF16)
    static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(a.y)[at] = v;
}

template <int G, int NTMAX>
__global__ void __launch_bounds__(kThreads, 1) k_w4_product(const __grid_constant__ CUtensorMap map_x, const ProductArgs a) {
  extern __shared__ __align__(1024) char smem[];
  Head* h = reinterpret_cast<Head*>(smem);
  uint16_t* start = reinterpret_cast<uint16_t*>(h + 1);  // one entry, all rows
  uint16_t* expert = start + 2;
  static_assert(sizeof(Head) + 8 <= kHeadBytes, "head");
  constexpr uint32_t used = kHeadBytes;
  const bool producer = threadIdx.x >> 5 == kWarps;
  Ring r;
  const int held = threadIdx.x == 0 ? read_status(a.status) : 0;
  init_ring(r, h, a.status);
  if (threadIdx.x == 0) {
    start[0] = 0, start[1] = a.T, expert[0] = 0;
    if (blockIdx.x == 0) *a.counter = 0;
    h->go = held == 0;
  }
  __syncthreads();
  const bool go = h->go;
  r.stage0 = smem_u32(smem + used);
  size_ring<G, true>(r, kSmem - used, a.T);
  Phase p = make_phase(1, a.shape, true);
  if (a.whole) whole_units(p);
  const bool pad = a.K % 8 != 0;
  // as in k_layer: no barrier goes by the status word
  const bool first_barrier = pad || p.runs > gridDim.x, joined = p.parts > 1;
  if (!go) p.total = p.runs = 0;
  const int K8 = (a.K + 7) / 8 * 8;
  const auto copy_rows = [&]() {  // to whole vectors
    for (uint32_t i = blockIdx.x * blockDim.x + threadIdx.x; i < uint32_t(a.T * K8); i += gridDim.x * blockDim.x) {
      const uint32_t t = i / K8, k = i % K8;
      a.padded[i] = int(k) < a.K ? a.x[(long long)t * a.K + k] : __float2bfloat16_rn(0.f);
    }
    fence_async();
  };
  const Sums o = {uint32_t(a.N), kUnit, kUnit / 2, a.N, kUnit / 2};
  Cursor c;
  if (producer) {
    Stream<G, true> t(r, expert, start);
    const Cursor behind;
    const long long panel = w4_panel_bytes(a.K, G);
    t.own(p, {nullptr, a.w4, 0, panel, 2 * panel, 4, 0, a.N, false, a.K}, {&map_x, nullptr, nullptr, 0, K8, 1}, o);
    t.ahead(c, !pad);
    if (pad) copy_rows();
    if (first_barrier) grid_barrier();
    fence_async();
    t.feed(c, behind, pad, a.counter);
  } else {
    if (pad) copy_rows();
    if (first_barrier) grid_barrier();
    const long long pitch = (long long)p.parts * a.N;
    products<G, true, NTMAX>(r, c, kDryThenReal, a.T, [&](const Part& part, int q, int col, int row, float v0, float v1) {
      if (col + q * o.inner >= part.columns) return;
      const long long at = part.to + row * pitch + q * o.half + col;
      if (!joined) {
        put_y(a, at, v0);
        if (row + 1 < part.rows) put_y(a, at + pitch, v1);
      } else {
        a.part[at] = v0;
        if (row + 1 < part.rows) a.part[at + pitch] = v1;
      }
    });
  }
  // The parts' sums. The producer, which is done before the products, runs through
  // them once ahead, dry, where runs are long enough to hide it ([1, 7168] x [7168,
  // 7168], 6 steps: 21.1 us without, 19.1 with; [5, 1001] x [1001, 1407], 1 step: 15.0
  // and 16.0).
  if (joined) {
#pragma unroll 1
    for (int pass = producer && p.run >= 4 ? 0 : 1; pass < 2; ++pass) {
      const bool dry = pass == 0;
      if (!dry) grid_barrier();
      if (!go) continue;
      const uint32_t quads = (a.N + 3) / 4, n = dry ? min(32u, quads) : uint32_t(a.T) * quads;
      const bool vec = a.N % 4 == 0;
      Spread s = spread(kWarps + 1);
      if (dry) s.i = threadIdx.x & 31;
#pragma unroll 1
      for (; s.i < n; s.i += s.step) {
        const uint32_t t = s.i / quads, col = (s.i - t * quads) * 4, parts = parts_in(p, col / kUnit);
        const float* in = a.part + (long long)t * p.parts * a.N + col;
        float v[4] = {};
#pragma unroll 4
        for (uint32_t q = 0; q < parts; ++q, in += a.N) {
          if (vec) {
            const float4 f = __ldcg(reinterpret_cast<const float4*>(in));
            v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += int(col) + i < a.N ? __ldcg(in + i) : 0.f;
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (int(col) + i < a.N && !dry) put_y(a, (long long)t * a.N + col + i, v[i]);
      }
    }
  }
  settle(r);
}

// ---------------------------------------------------------------------------
// host side
int ctas() { return sm_count() < kMaxCtas ? sm_count() : kMaxCtas; }

template <typename... KArgs, typename... Args>
int launch_all(void (*kernel)(KArgs...), long long most, int threads, cudaStream_t st, const Args&... args) {
  if (set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), kSmem)) return MEP_ERR_CUDA;
  const int sms = ctas();
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

// Most bytes of partial sums [rows][parts][columns] with any number of entries
// up to `most`, and T rows an entry at most, A in all. One run a CTA: the more
// entries the longer the runs and the fewer the parts, and beyond `full` entries
// no more rows. Several runs a CTA: the least run's parts.
size_t part_bytes(int most, int full, int T, int A, long long nb, long long ks, long long columns) {
  size_t top = 0;
  for (int n = 1; n <= full && n <= most; ++n) {
    const uint32_t per = uint32_t(ceil_div(n * nb * ks, kMaxCtas));
    if (per > kOneRun) break;
    const long long rows = (long long)T * n < A ? (long long)T * n : A;
    const size_t values = size_t(rows) * parts_of(uint32_t(ks), per) * columns;
    if (values > top) top = values;
  }
  if (ceil_div(most * nb * ks, kMaxCtas) > kOneRun) {
    const size_t values = size_t(A) * parts_of(uint32_t(ks), least_run(uint32_t(ks))) * columns;
    if (values > top) top = values;
  }
  return align256(4 * top);
}

// 3D bf16 map over [E, K, N], box {64 columns, a step's rows, 1}, 128-byte swizzle; beyond a matrix's edges zeros.
bool make_map3(CUtensorMap* m, const void* p, long long E, long long K, long long N) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {cuuint64_t(N), cuuint64_t(K), cuuint64_t(E)};
  const cuuint64_t strides[2] = {cuuint64_t(N) * 2, cuuint64_t(N) * K * 2};
  const cuuint32_t box[3] = {64, cuuint32_t(step_rows(0)), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2D bf16 map over [rows, columns], box {64 columns, box_rows}, 128-byte swizzle; beyond the edges zeros.
bool make_map2(CUtensorMap* m, const void* p, long long rows, long long columns, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {cuuint64_t(columns), cuuint64_t(rows)}, strides[1] = {cuuint64_t(columns) * 2};
  const cuuint32_t box[2] = {64, cuuint32_t(box_rows)}, estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t kCounters = 256;  // bytes at the start

// The layer's workspace: counters, partial sums of the first product, the activation, partial sums of the second.
struct LayerSpace {
  size_t part1, act, part2;
  size_t all() const { return kCounters + part1 + act + part2; }
};
bool layer_space(int T, int K, int E, long long H, long long F, int w_type, int group, LayerSpace* s) {
  if (T < 0 || T > MEP_MAX_FEW || K < 1 || K > MEP_MAX_K || E < 1 || E > MEP_MAX_E || H < 8 || F < 8 || H % 8 != 0 ||
      F % 8 != 0 || H > MEP_MAX_FEW_H || F > MEP_MAX_FEW_H / 2)
    return false;
  if (w_type != MEP_BF16 && (w_type != MEP_W4 || !w4_sizes_ok(H, F, group))) return false;
  const int A = T * K, most = max_entries(T, K, E), bk = step_rows(w_type == MEP_W4 ? group : 0);
  s->part1 = part_bytes(most, K, T, A, ceil_div(F, kUnit / 2), ceil_div(H, bk), 2 * F);
  s->part2 = part_bytes(most, K, T, A, ceil_div(H, kUnit), ceil_div(F, bk), H);
  s->act = align256(size_t(A) * F * 4);
  return true;
}

// Whether a product's runs are its units: where that leaves no more than a fifth
// of the SMs idle in the last round, for partial sums cost a write and a read of
// the output and a barrier ([64, 2048] x [2048, 65536]: 99 us with them, 74
// without).
bool whole_product(long long N) {
  const long long units = ceil_div(N, kUnit), rounds = ceil_div(units, kMaxCtas);
  return rounds * kMaxCtas * 4 <= units * 5;
}
struct ProductSpace {
  size_t padded, part;
  size_t all() const { return kCounters + padded + part; }
};
bool product_space(int T, long long K, long long N, int group, ProductSpace* s) {
  if (T < 0 || T > MEP_MAX_FEW || !w4_sizes_ok(K, N, group)) return false;
  s->padded = K % 8 == 0 ? 0 : align256(size_t(T) * ceil_div(K, 8) * 16);
  s->part = T == 0 || whole_product(N) ? 0 : part_bytes(1, 1, T, T, ceil_div(N, kUnit), ceil_div(K, step_rows(128)), N);
  return true;
}

struct Maps {
  CUtensorMap w1, w2, x, act;
};
template <int G>
int launch_layer(const Maps& m, const LayerArgs& a, cudaStream_t st) {
  const long long experts = max_entries(a.T, a.K, a.E), bk = step_rows(G);
  const long long n1 = experts * ceil_div(a.F, kUnit / 2) * ceil_div(a.H, bk), n2 = experts * ceil_div(a.H, kUnit) * ceil_div(a.F, bk);
  return launch_all(k_layer<G>, n1 > n2 ? n1 : n2, kLayerThreads, st, m.w1, m.w2, m.x, m.act, a);
}
template <int G> int launch_product(const CUtensorMap& x, const ProductArgs& a, cudaStream_t st) {
  const long long n = ceil_div(a.N, kUnit) * ceil_div(a.K, step_rows(G));
  return a.T <= 32 ? launch_all(k_w4_product<G, 4>, n, kThreads, st, x, a) : launch_all(k_w4_product<G, 8>, n, kThreads, st, x, a);
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
  char* p = static_cast<char*>(ws) + kCounters;
  const ProductArgs a = {reinterpret_cast<const __nv_bfloat16*>(x), w4, status, T, int(K), int(N), y_type,
                         shape_of(ceil_div(K, step_rows(128)), ceil_div(N, kUnit)), whole_product(N), static_cast<uint32_t*>(ws),
                         reinterpret_cast<__nv_bfloat16*>(p), reinterpret_cast<float*>(p + s.padded), y};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  CUtensorMap map = {};
  const void* from = K % 8 == 0 ? static_cast<const void*>(x) : p;
  if (!on_current_device(from)) return MEP_ERR_INVALID_ARG;
  if (!make_map2(&map, from, T, ceil_div(K, 8) * 8, T <= 8 ? 8 : T <= 16 ? 16 : T <= 32 ? 32 : 64)) return MEP_ERR_CUDA;
  return group == 32   ? launch_product<32>(map, a, st)
         : group == 64 ? launch_product<64>(map, a, st)
                       : launch_product<128>(map, a, st);
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
  char* p = static_cast<char*>(ws) + kCounters;
  const int bk = step_rows(w_type == MEP_W4 ? group : 0);
  const long long steps1 = ceil_div(H, bk) * ceil_div(F, kUnit / 2), steps2 = ceil_div(F, bk) * ceil_div(H, kUnit);
  // fewer SMs take the runs that are sized for kMaxCtas as they come
  const int counted = ctas() < kMaxCtas || max_entries(T, K, E) * (steps1 > steps2 ? steps1 : steps2) > kOneRun * (long long)kMaxCtas;
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
                       shape_of(ceil_div(H, bk), ceil_div(F, kUnit / 2)),
                       shape_of(ceil_div(F, bk), ceil_div(H, kUnit)),
                       counted,
                       div_of(K),
                       static_cast<uint32_t*>(ws),
                       reinterpret_cast<float*>(p),
                       reinterpret_cast<float*>(p + s.part1 + s.act),
                       reinterpret_cast<__nv_bfloat16*>(p + s.part1),
                       reinterpret_cast<__nv_bfloat16*>(out)};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Maps m = {};
  if (w_type == MEP_W4)
    return group == 32   ? launch_layer<32>(m, a, st)
           : group == 64 ? launch_layer<64>(m, a, st)
                         : launch_layer<128>(m, a, st);
  if (!on_current_device(w1) || !on_current_device(w2) || !on_current_device(x) || !on_current_device(ws)) return MEP_ERR_INVALID_ARG;
  if (!make_map3(&m.w1, w1, E, H, 2 * F) || !make_map3(&m.w2, w2, E, F, H) || !make_map2(&m.x, x, T, H, 1) ||
      !make_map2(&m.act, a.act, 2LL * T * K, F, 8))
    return MEP_ERR_CUDA;
  return launch_layer<0>(m, a, st);
}
