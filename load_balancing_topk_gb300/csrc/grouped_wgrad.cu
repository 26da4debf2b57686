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
//                   (one per rank that has rows of it), cut into parts where
//                   a group is long next to all the work, the longest first;
//   k_wgrad_pair    persistent clusters of two CTAs, one per SM, 512 threads
//                   each, over units (part of a weight row's group, 256 rows
//                   of H, 256 columns of H'), to and fro over the pairs. CTA r
//                   of a pair owns 128 of the 256 rows of H. Per step of 64
//                   buffer rows (128 from checkpoint rows):
//     warps 0, 2  TMA producers: this CTA's 128 columns of x (bf16 boxes, or
//                 the checkpoint's bytes and the rows' scale bytes), and its
//                 half of the 256 columns of dy, into a ring of stages;
//     warps 4..7  converter: checkpoint bytes to a bf16 operand A in TMEM (exact:
//                 q * 2^k has 8 significant bits), and zeros over the rows
//                 that a segment's last step takes from the next group, in
//                 both operands (a NaN there would survive a product with 0);
//     warp 1      of CTA 0 issues the pair MMAs (tcgen05.mma.cta_group::2,
//                 M = 256, N = 256 or 128, K = 16; A from shared memory, or
//                 from TMEM) into an accumulator in TMEM: one of two in turn,
//                 or the only one where A takes the room of the other;
//     warps 8..15 add each accumulator, once Ring::chunk steps are in it, to
//                 fp32 sums in registers (128 a thread), and at the end of
//                 the unit write them through shared memory with bulk tensor
//                 stores, or bulk tensor additions.
//
// Why the sums leave TMEM: the tensor cores do not round their fp32 additions
// to nearest, and the error of one accumulator grows with the number of
// steps. Over some 3000 rows of normal bf16 values it was 3.2e-6 of the result
// with a single accumulator, and 0.9, 0.5 and 0.2e-6 with sums moved (and then
// rounded to nearest) every 1024, 512 and 256 rows; fp32 products are off by
// 0.2 to 0.4e-6. 512 cost 3% over 1024 and saves 6% over 256. A checkpoint's
// bytes have fewer bits to lose: 1.7, 2.6 and 3.5e-7 at 1024, 1536 and 2048
// rows (5.4e-7 with a single accumulator). The longer a chunk, the less often
// the MMAs wait for the one accumulator to empty: 724, 707 and 702 us on the
// medium layer (696). 1536 has most of that.
//
// What bounds it, on the medium layer ([196608, 2048] x [196608, 1408], 67
// groups). Back to back the power limit: from bf16 rows 778 to 788 us (1440 to
// 1460 TFLOP/s) at an SM clock of 1470 MHz, from checkpoint rows 798 to 819
// (1385 to 1420) at 1590, a dense library product of the size 790 at 1670. So a
// pass from checkpoint rows takes 12% more cycles, of which the power they do
// not draw gives back all but 3%.
// In single passes the cycles: 672 to 759 us from bf16 rows by the GPU, 707 to
// 749 from checkpoint rows (1494 to 1688 and 1515 to 1605 TFLOP/s; the library
// product 1694 to 1739). From bf16 rows they are the feed: per step an SM takes
// in 32 KB and its MMAs read as much of shared memory, all of its 128 bytes a
// cycle. From checkpoint rows, of the 1310 cycles of a step of 128 rows (1024
// of MMAs) a converter warp works 825 and waits 160 for the copies, and the
// MMAs wait 135 for the sums to leave the one accumulator.
// The large workload's layer ([524288, 7168] x [524288, 1408], 256 experts)
// takes 6.28 ms from bf16 rows and 6.48 from checkpoint rows in single passes
// (1686 and 1635 TFLOP/s), 7.35 and 7.62 back to back.
// What it took to get there: the operand in TMEM (through shared memory 940
// us), 128 rows a step, for what each step costs a converter to start (847 ->
// 823 us; with the ring below, 750 against 893 at 64), a fourth stage, so that
// copies, conversion and products of a stage may follow each other without
// holding up the next (825 -> 752), and seven instructions for four bytes
// instead of ten (762 -> 740). Loading a step's bytes before converting any,
// or a step ahead, ran slower (773, 1007).
// Waiting with short tries cost 7%, addresses in ordinary instead of uniform
// registers 4%, a release at cluster scope per step half.
// Every wait is bounded as in grouped_gemm.cu.

#include "ckpt.cuh"
#include "tc.cuh"

namespace mep {
namespace {

constexpr int kBM = 128;                 // rows of H per CTA
constexpr int kBN = 256;                 // columns of H' per pair
constexpr int kBK = 64;                  // buffer rows that the list of parts counts in
constexpr int kThreads = 512;
constexpr int kTmemCols = 2 * kBN;
constexpr int kGroupThreads = 1024;
constexpr int kEpiWarps = 8;
constexpr int kPair = 2;
// How long groups are cut into parts (k_wgrad_groups). At H 512, H' 512 one
// group of 4096 rows took 31 us whole, 31 in parts of 8 steps and 28 in parts
// of 16, which is no loss at 1024 rows either (18 against 22 us); two groups of
// 16384 rows at 256 x 256 took 156 us whole, 59 in four parts, 47 in eight and
// 50 in sixteen (the last of them adds all up).
constexpr int kPairs = 76;  // a fixed number, so that the parts do not depend on the device
constexpr int kLeastSteps = 16;
constexpr int kMostParts = 8;
constexpr int kMostPartials = 2 * kPairs;  // parts * tiles of all entries with several parts: see partials_of
constexpr int kTile = 2 * kBM * kBN;       // fp32 values of a partial sum

// A step of K buffer rows and its stage: from bf16 rows the operands A and B;
// from checkpoint rows B and the bytes, which become an A in TMEM, in steps of
// 128 rows, with output boxes half as large, for a fourth stage.
template <bool CKPT> struct Ring {
  static constexpr int K = CKPT ? 128 : 64;
  static constexpr int box = K * 64 * 2, op = 2 * box;      // a bf16 box of 64 columns; an operand's two
  static constexpr int q = K * kBM, scales = K * 16;        // checkpoint bytes; scale bytes, in 16-byte rows
  static constexpr int stage = op + (CKPT ? q + scales : op), stages = CKPT ? 4 : 6;
  static constexpr int out = CKPT ? 16 : 32, out_box = 32 * out * 4;  // an output box: columns; bytes of 32 rows
  static constexpr int b0 = CKPT ? 0 : op;                  // B within a stage
  static constexpr int accs = CKPT ? 1 : 2;                 // accumulators
  static constexpr int a_cols = K / 2;                      // TMEM columns of an A
  static constexpr int chunk = CKPT ? 12 : 8;               // steps summed in TMEM
  static constexpr int smem = 1024 /* alignment slack */ + stages * stage + kEpiWarps * out_box + 512;
  static_assert(smem <= 232448, "the ring must fit in 227 KB of shared memory");
  static_assert(accs * kBN + (CKPT ? stages * a_cols : 0) <= kTmemCols, "TMEM");
};

struct Smem {
  uint64_t full[8], ready[8], empty[8], tfull[2], tempty[2], drain;
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
// b of rank r, in parts: parts[2i] = {weight row, first segment, 0, steps},
// parts[2i + 1] = {first buffer row, rows from there to the segment's end,
// parts of this weight row + 256 * number of this one, index of the weight
// row's first partial sum}; segs[j] = {first buffer row, rows}, R places for a
// home expert and one for a slot. Without `accumulate` a home expert is listed
// even without rows (it is written as zero), a slot never is.
//
// A part is at most what a pair has to do in all, so that few, uneven groups
// still fill the pairs (half of that cost more in joins than it evened out: 58
// against 48 us at 22220 rows in 18 groups, 1160 x 520); a group has at most
// kMostParts (the last of them adds the partial sums of all up), and only one
// of more than kLeastSteps is cut. The longest come first. A thread has one weight row, reads its group
// ends once (together the threads read, and check, all of cu_seqlens), and
// places its parts by counting over the others' lengths in shared memory. With
// more weight rows than threads, empty slots among them, the list is in their
// order and nothing is cut. That serves calls whose rows are spread (64 ranks
// of 2 experts and 1000 rows, each with a slot in use, at 512 x 512: 117 us
// with 16 slots a rank, 1152 weight rows; 187 with 14, 1024 weight rows, of
// which the counting is some 90), but not those with one expert hot (the same
// with 64600 rows of one expert: 357 and 212).
__device__ __forceinline__ int ceil_div(long long a, long long b) { return int((a + b - 1) / b); }

struct Row {  // a weight row's group
  int segments = 0, steps = 0;
  int2 first = {0, 0};  // its first segment
  bool bad = false;
};
// Reads the group ends of weight row w, checks them, lists the segments.
__device__ __forceinline__ Row read_row(const int32_t* __restrict__ cu, int w, int R, int E, int B, int SK,
                                        int2* __restrict__ segs) {
  Row row;
  const int G = E + B;
  const bool home = w < E;
  const int j = home ? w : E + (w - E) % B, r0 = home ? 0 : (w - E) / B, r1 = home ? R : r0 + 1;
  int2* to = segs + (home ? (long long)w * R : (long long)E * R + (w - E));
#pragma unroll 4
  for (int r = r0; r < r1; ++r) {
    const long long p = (long long)r * G + j;
    // (compared, not subtracted: the difference of two ends of a corrupt row may wrap)
    const int hi = cu[p], lo = j == 0 ? 0 : cu[p - 1];
    const bool bad = lo < 0 || hi < lo || hi > SK || (j == G - 1 && hi != SK);
    row.bad |= bad;
    const int len = bad ? 0 : hi - lo;
    if (len > 0) {
      const int2 seg = make_int2(int((long long)r * SK + lo), len);
      if (row.segments == 0) row.first = seg;
      to[row.segments++] = seg;
      row.steps += ceil_div(len, kBK);
    }
  }
  return row;
}

__global__ void __launch_bounds__(kGroupThreads)
    k_wgrad_groups(const int32_t* __restrict__ cu, int R, int E, int B, int SK, int tiles, int accumulate,
                   int32_t* status, int* __restrict__ count, int4* __restrict__ parts,
                   int2* __restrict__ segs, int* __restrict__ arrived) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ int s_warp[33], s_listed[kGroupThreads + 1];
  __shared__ int2 s_rows[kGroupThreads];  // {steps of a part, parts}
  __shared__ int s_steps;
  const int W = E + R * B, t = threadIdx.x;
  const auto seg0 = [&](int w) { return w < E ? w * R : E * R + (w - E); };
  if (t == 0) s_steps = 0;
  const int stat = read_status(status);
  if (W <= int(blockDim.x)) {
    const Row row = t < W ? read_row(cu, t, R, E, B, SK, segs) : Row();
    const int stop = __syncthreads_or((stat != 0 ? 2 : 0) | (row.bad ? 1 : 0));
    if (stop) {  // (what is read from a malformed table is not used)
      if (t == 0) {
        *count = 0;
        if (stat == 0) set_status(status, MEP_ERR_BAD_SEQLENS);
      }
      return;
    }
    const int warp_steps = __reduce_add_sync(MEP_FULL_MASK, row.steps);
    if ((t & 31) == 0 && warp_steps > 0) atomicAdd(&s_steps, warp_steps);
    __syncthreads();
    const int most = max(kLeastSteps, ceil_div((long long)s_steps * tiles, kPairs)), s = row.steps;
    const bool listed = t < W && (s > 0 || (t < E && !accumulate));
    const int len = s > most ? max(ceil_div(s, kMostParts), ceil_div(s, ceil_div(s, most))) : s;
    const int np = !listed ? 0 : s > 0 ? ceil_div(s, len) : 1;
    if (t < W) s_rows[t] = make_int2(len, np);
    __syncthreads();
    int pos = 0, partial = 0, all = 0, partials = 0;
    for (int j = 0; j < W; ++j) {
      const int2 o = s_rows[j];
      all += o.y;
      if (o.x > len || (o.x == len && j < t)) pos += o.y;
      if (o.y > 1) {
        partials += o.y;
        if (j < t) partial += o.y;
      }
    }
    if (t == 0) *count = all;
    for (int i = t; i < partials * tiles * 2 * kEpiWarps; i += blockDim.x) arrived[i] = 0;
    int g = seg0(t), done = 0;  // segment, its steps that are behind
    int2 seg = row.first;
    for (int k = 0; k < np; ++k) {
      const int steps = min(len, s - k * len);
      parts[2 * (pos + k)] = make_int4(t, g, 0, steps);
      parts[2 * (pos + k) + 1] = make_int4(seg.x + done * kBK, seg.y - done * kBK, np + 256 * k, partial);
      for (int left = k + 1 < np ? steps : 0; left > 0;) {  // on to the next part's first step
        const int here = ceil_div(seg.y, kBK) - done;
        if (left < here) {
          done += left;
          left = 0;
        } else {
          left -= here;
          done = 0;
          seg = segs[++g];
        }
      }
    }
    return;
  }
  int bad = 0, listed_before = 0;
  for (int base = 0; base < W; base += blockDim.x) {
    const int w = base + t;
    const Row row = w < W ? read_row(cu, w, R, E, B, SK, segs) : Row();
    bad |= row.bad;
    const bool listed = w < W && (row.steps > 0 || (w < E && !accumulate));
    s_listed[t] = listed;
    __syncthreads();
    block_excl_scan(s_listed, s_listed, blockDim.x, s_warp, true);
    if (listed) {
      int4* part = parts + 2 * (listed_before + s_listed[t]);
      part[0] = make_int4(w, seg0(w), 0, row.steps);
      part[1] = make_int4(row.first.x, row.first.y, 1, 0);
    }
    listed_before += s_listed[blockDim.x];
    __syncthreads();
  }
  bad = __syncthreads_or(bad);
  if (t == 0) {
    *count = bad || stat != 0 ? 0 : listed_before;
    if (bad && stat == 0) set_status(status, MEP_ERR_BAD_SEQLENS);
  }
}

// Four TMEM columns of A for 16 rows, eight times over (16x128b): thread T of the
// warp writes register 2i to row T / 4, column 4i + T % 4, register 2i + 1 to
// the row eight further.
__device__ __forceinline__ void tc_st16x128(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// The pair MMA with A (each CTA's 128 rows) in TMEM.
__device__ __forceinline__ void tc_mma2_ta(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc,
                                           uint32_t accumulate, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Four 8 x 8 matrices of 16-bit elements, transposed: thread T gets of each the
// elements of column T / 4 in rows 2 (T % 4) and the next. Lane l gives the
// address of row l % 8 of matrix l / 8.
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(addr)
               : "memory");
}

// The four signed bytes q of w times a power of two each, as bf16: bytes 0 and
// 2 by the halves of `step` (which holds it times 2^6) into even, bytes 1 and 3
// into odd. With its sign bit flipped a byte is u = q + 128, and sixteen bits
// that hold u alone are bf16 u * 2^-133, below and above the smallest normal
// number alike (u = 128) as its spacing stays the same. u * 2^127 in one step
// less 2 is q * 2^-6, which has eight bits, and so has q times the power of two.
__device__ __forceinline__ uint32_t dequant2(uint32_t u, __nv_bfloat162 step) {
  constexpr uint32_t kUp = 0x7f007f00u, kBack = 0xc000c000u;  // 2^127, -2
  const uint32_t up = kUp, back = kBack;
  const __nv_bfloat162 q = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&u),
                                   *reinterpret_cast<const __nv_bfloat162*>(&up),
                                   *reinterpret_cast<const __nv_bfloat162*>(&back));
  const __nv_bfloat162 r = __hmul2(q, step);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ void dequant4(uint32_t w, __nv_bfloat162 step, uint32_t& even, uint32_t& odd) {
  const uint32_t u = w ^ 0x80808080u;
  even = dequant2(__byte_perm(u, 0u, 0x4240), step);
  odd = dequant2(__byte_perm(u, 0u, 0x4341), step);
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// The units of one CTA pair, in the order in which every role of both CTAs
// walks them (whole warps: what steers the loops is the same for all lanes,
// and known to be, so that addresses and descriptors stay in uniform
// registers): round by round over the pairs, to and fro, since the list goes
// from long to short. The next unit's part is loaded while f works on this
// one's; f(part, tile) returns false to stop.
struct Part {
  int w, seg, steps;  // weight row, first segment
  int row, len;       // first row, rows to the segment's end
  int of, partial;
};
__device__ __forceinline__ Part load_part(const int4* __restrict__ parts, int i) {
  const int4 a = parts[2 * i], b = parts[2 * i + 1];
  return {a.x, a.y, a.w, b.x, b.y, b.z, b.w};
}
__device__ __forceinline__ Part uniform(const Part& p) {
  return {uniform(p.w), uniform(p.seg), uniform(p.steps), uniform(p.row), uniform(p.len), uniform(p.of),
          uniform(p.partial)};
}
template <typename F>
__device__ __forceinline__ void for_units(const int4* __restrict__ parts, int count, int tiles, F f) {
  const int pairs = gridDim.x / 2, units = count * tiles, me = blockIdx.x / 2;
  int base = 0, u = me;
  if (u >= units) return;
  Part cur = uniform(load_part(parts, u / tiles)), next = cur;
  for (;;) {
    base += pairs;
    const int nu = base / pairs % 2 == 0 ? base + me : base + pairs - 1 - me;
    const bool more = nu < units;
    if (more) next = load_part(parts, nu / tiles);
    if (!f(cur, u % tiles) || !more) return;  // (only the last round is short)
    cur = uniform(next);
    u = nu;
  }
}
// The steps of one unit, of up to K rows: f(first buffer row, rows left from it
// on, whether it is the unit's last).
template <int K, typename F>
__device__ __forceinline__ bool for_steps(const Part& part, const int2* __restrict__ segs, F f) {
  int row = part.row, len = part.len, g = part.seg;
  for (int steps = part.steps; steps > 0;) {
    if (len <= 0) {
      const int2 seg = segs[++g];
      row = uniform(seg.x);
      len = uniform(seg.y);
    }
    const int left = min(len, steps * kBK);
    steps -= K > kBK && left > kBK ? 2 : 1;
    if (!f(row, left, steps == 0)) return false;
    row += K;
    len -= K;
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
                 const int4* __restrict__ parts, const int2* __restrict__ segs, int* __restrict__ arrived,
                 float4* __restrict__ partials, int32_t* status, int E, int H, int Hp, int accumulate) {
  using Rg = Ring<CKPT>;
  constexpr int kSt = Rg::stages, kStage = Rg::stage;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gen_base = smem_raw + (base - raw);
  const uint32_t out_box = base + kSt * kStage;
  Smem* S = reinterpret_cast<Smem*>(gen_base + kSt * kStage + kEpiWarps * Rg::out_box);
  volatile int* abort_flag = &S->abort;

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int rank = uniform(int(cluster_rank()));
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kSt; ++s) {
      mbar_init(smem_u32(&S->full[s]), 2);   // this CTA's producers and their bytes
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
  const uint32_t tmem = uniform(S->tmem), a_ring = tmem + Rg::accs * kBN;
  const int nM = (H + 2 * kBM - 1) / (2 * kBM), nN = (Hp + kBN - 1) / kBN;
  const int tiles = nM * nN, count = uniform(S->count);

  // the four warpgroups' registers: 56 + 72 + 192 + 192 = 4 x 128 at launch
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 || warp == 2) {
      // ---------------- TMA producers: x, dy ----------------
      const bool of_x = warp == 0;
      Pos at;
      uint32_t issued = 0;
      for_units(parts, count, tiles, [&](const Part& en, int t) {
        const int h0 = t / nN * 2 * kBM + rank * kBM, n0 = t % nN * kBN;
        const bool narrow = Hp - n0 <= 128;
        const int c0 = n0 + rank * (narrow ? 64 : 128);
        const int na = h0 >= H ? 0 : h0 + 64 < H ? 2 : 1;
        const int nb = c0 >= Hp ? 0 : !narrow && c0 + 64 < Hp ? 2 : 1;
        const uint32_t bytes = !of_x ? nb * Rg::box : !CKPT ? na * Rg::box : na > 0 ? Rg::q + Rg::scales : 0;
        const int sx = ckpt_scale_at(H) + ((h0 / kCkptBlock) & ~15);
        return for_steps<Rg::K>(en, segs, [&](int row, int, bool) {
          if (!warp_wait(smem_u32(&S->empty[at.s]), at.parity ^ 1u, abort_flag, status)) return false;
          const uint32_t bar = smem_u32(&S->full[at.s]), st = base + at.s * kStage;
          if (elected()) {
            mbar_expect_tx(bar, bytes);
            if (!of_x) {
              if (nb > 0) tma_load_2d(st + Rg::b0, &map_dy, c0, row, bar);
              if (nb > 1) tma_load_2d(st + Rg::b0 + Rg::box, &map_dy, c0 + 64, row, bar);
            } else if (CKPT) {
              if (na > 0) tma_load_2d(st + Rg::op, &map_x, h0, row, bar);
              if (na > 0) tma_load_2d(st + Rg::op + Rg::q, &map_s, sx, row, bar);
            } else {
              if (na > 0) tma_load_2d(st, &map_x, h0, row, bar);
              if (na > 1) tma_load_2d(st + Rg::box, &map_x, h0 + 64, row, bar);
            }
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
      const uint64_t adesc = sdesc(base, Rg::box, 1024), bdesc = sdesc(base + Rg::b0, Rg::box, 1024);
      for_units(parts, count, tiles, [&](const Part& en, int t) {
        // A in TMEM has its rows in its lanes: not transposed (bit 15)
        const uint32_t idesc = (Hp - t % nN * kBN <= 128 ? kIdescN : kIdesc) & (CKPT ? ~(1u << 15) : ~0u);
        int in_chunk = 0;
        return for_steps<Rg::K>(en, segs, [&](int, int left, bool end) {
          if (in_chunk == 0 &&
              !warp_wait(smem_u32(&S->tempty[acc.s]), acc.parity ^ 1u, abort_flag, status))
            return false;
          if (!warp_wait(smem_u32(&S->ready[at.s]), at.parity, abort_flag, status)) return false;
          tc_fence_after();
          const uint32_t d = tmem + acc.s * kBN;
          const uint64_t ad = adesc + (at.s * kStage >> 4), bd = bdesc + (at.s * kStage >> 4);
          const uint32_t at_col = a_ring + at.s * Rg::a_cols;
          const bool last = in_chunk == Rg::chunk - 1 || end;
          if (elected()) {
            if (left > Rg::K - 16) {
#pragma unroll
              for (int kk = 0; kk < Rg::K / 16; ++kk) {
                if (CKPT)
                  tc_mma2_ta(d, at_col + kk * 8, bd + kk * 128, kk > 0 ? 1u : (uint32_t)in_chunk, idesc);
                else
                  tc_mma2(d, ad + kk * 128, bd + kk * 128, kk > 0 ? 1u : (uint32_t)in_chunk, idesc);
              }
            } else {
              for (int kk = 0; 16 * kk < left; ++kk) {
                if (CKPT)
                  tc_mma2_ta(d, at_col + kk * 8, bd + kk * 128, uint32_t(kk + in_chunk), idesc);
                else
                  tc_mma2(d, ad + kk * 128, bd + kk * 128, uint32_t(kk + in_chunk), idesc);
              }
            }
            tc_commit2_mc(smem_u32(&S->empty[at.s]), 3);
            if (last) tc_commit2_mc(smem_u32(&S->tfull[acc.s]), 3);
          }
          __syncwarp();
          at.template next<kSt>();
          ++in_chunk;
          if (last) {
            acc.template next<Rg::accs>();
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
    // Warp q makes the TMEM lanes [32q, 32q + 32) of A, 16 at a time. Of the
    // bytes [64 rows][128 columns] (128-byte swizzled) it reads 8 rows x 16
    // columns as an 8 x 8 matrix of byte pairs, transposed: a thread's word
    // holds columns 2c and 2c + 1 (c = lane / 4) of two consecutive rows --
    // and a TMEM word of A is two consecutive steps of K, here rows. So the
    // bytes go from registers to TMEM without an exchange between threads
    // or a way through shared memory. Column 2c becomes lane c of the 16,
    // column 2c + 1 lane 8 + c: the epilogue puts the rows of D right.
    const int t = threadIdx.x - 128, q4 = warp & 3;
    Pos at;
    for_units(parts, count, tiles, [&](const Part& en, int tile) {
      const int h0 = tile / nN * 2 * kBM + rank * kBM;
      const uint32_t sbyte = (uint32_t)(h0 / kCkptBlock) & 15u;
      return for_steps<Rg::K>(en, segs, [&](int, int left, bool) {
          if (!warp_wait(smem_u32(&S->full[at.s]), at.parity, abort_flag, status)) return false;
          const uint32_t st = base + at.s * kStage;
          const int valid = min(Rg::K, left), need = (valid + 15) & ~15;
          if (CKPT && h0 < H) {
            const uint32_t q = st + Rg::op, sc = q + Rg::q;
            tc_fence_after();  // the MMAs that read this A last are done: `empty` let the producer go on
            // lane l has the steps of rows 2l and 2l + 1 (0 for rows of the next group: q times 0)
#pragma unroll
            for (int k0 = 0; k0 < Rg::K; k0 += 64) {
              if (k0 >= valid) break;
              uint32_t s0, s1, v[16];
              asm volatile("ld.shared.u8 %0, [%1];" : "=r"(s0) : "r"(sc + (k0 + 2 * lane) * 16 + sbyte));
              asm volatile("ld.shared.u8 %0, [%1];" : "=r"(s1) : "r"(sc + (k0 + 2 * lane + 1) * 16 + sbyte));
#pragma unroll
              for (int i = 0; i < 16; i += 4) {  // eight words for either 16 columns
                const int row = k0 + 8 * ((i & 7) + (lane >> 3)) + (lane & 7);
                ldsm4_trans(q + row * 128 + (((2 * q4 + (i >> 3)) ^ (row & 7)) << 4), v[i], v[i + 1], v[i + 2],
                            v[i + 3]);
              }
              s0 = k0 + 2 * lane >= valid ? 0u : s0 == (uint32_t)kCkptNan ? 0x7fffu : (s0 + 6) << 7;
              s1 = k0 + 2 * lane + 1 >= valid ? 0u : s1 == (uint32_t)kCkptNan ? 0x7fffu : (s1 + 6) << 7;
              const uint32_t pairs = s0 | s1 << 16;
              uint32_t step[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) step[i] = __shfl_sync(MEP_FULL_MASK, pairs, 4 * i + (lane & 3));
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                uint32_t o[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const __nv_bfloat162 f = *reinterpret_cast<const __nv_bfloat162*>(&step[i]);
                  dequant4(v[8 * half + i], f, o[2 * i], o[2 * i + 1]);
                }
                tc_st16x128(a_ring + at.s * Rg::a_cols + k0 / 2 + ((uint32_t)(32 * q4 + 16 * half) << 16), o);
              }
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before();
          }
          if (valid < need)  // whole rows: the swizzle stays within a row
            for (int i = t; i < (need - valid) * 32; i += 128) {
              const int row = valid + (i >> 5), piece = i & 31;
              if (CKPT && piece >= 16) continue;  // there B alone lies in shared memory
              sts128(st + (piece >> 3) * Rg::box + row * 128 + ((piece & 7) << 4), 0u, 0u, 0u, 0u);
            }
          if (valid < need) fence_async_smem();
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
    const uint32_t box = out_box + (uint32_t)(warp - 8) * Rg::out_box;
    // the row of H, of these 32, in this lane: the converter's order
    const int row = CKPT ? (lane & 16) + ((lane & 7) << 1) + ((lane >> 3) & 1) : lane;
    Pos at;
    for_units(parts, count, tiles, [&](const Part& en, int tile) {
      const int h = tile / nN * 2 * kBM + rank * kBM + 32 * q, n = tile % nN * kBN + 128 * half;
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.f;
      int in_chunk = 0;
      const bool ok = for_steps<Rg::K>(en, segs, [&](int, int, bool end) {
        if (++in_chunk < Rg::chunk && !end) return true;
        in_chunk = 0;
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
        at.template next<Rg::accs>();
        return true;
      });
      if (!ok) return false;
      if ((en.of & 255) > 1 && h < H && n < Hp) {
        // This part's sums go to the workspace, in the order of the threads
        // that will read them; the warp that comes last adds up all parts', in
        // their order: the same bits whoever is last.
        const int np = en.of & 255, mine = (rank * kEpiWarps + warp - 8) * 32 * 32 + lane;
        const long long part0 = (long long)en.partial * tiles + tile;
        float4* own = partials + (part0 + (long long)(en.of >> 8) * tiles) * (kTile / 4) + mine;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          __stcg(own + 32 * i, make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]));
        __threadfence();
        __syncwarp();
        int before = 0;
        if (lane == 0) before = atomicAdd(arrived + part0 * 2 * kEpiWarps + rank * kEpiWarps + warp - 8, 1);
        if (uniform(before) != np - 1) return true;
        __threadfence();
#pragma unroll
        for (int i = 0; i < 128; ++i) acc[i] = 0.f;
        for (int k = 0; k < np; ++k) {
          const float4* from = partials + (part0 + (long long)k * tiles) * (kTile / 4) + mine;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float4 v = __ldcg(from + 32 * i);
            acc[4 * i] += v.x;
            acc[4 * i + 1] += v.y;
            acc[4 * i + 2] += v.z;
            acc[4 * i + 3] += v.w;
          }
        }
      }
      const CUtensorMap* map = en.w < E ? &map_home : &map_slot;
      const int z = en.w < E ? en.w : en.w - E;
#pragma unroll
      for (int i = 0; i < 128 / Rg::out; ++i)
        if (h < H && n + Rg::out * i < Hp) {
          if (lane == 0) bulk_wait_read_0();
          __syncwarp();
#pragma unroll
          for (int j = 0; j < Rg::out / 4; ++j) {
            const float* v = &acc[Rg::out * i + 4 * j];
            sts128(box + row * (4 * Rg::out) + ((j ^ (Rg::out == 32 ? row & 7 : (row >> 1) & 3)) << 4),
                   __float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (accumulate)
              tma_add_3d(map, n + Rg::out * i, h, z, box);
            else
              tma_store_3d(map, n + Rg::out * i, h, z, box);
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

// fp32 [n, H, H'], boxes of 32 x `cols`: a third dimension keeps a box that
// hangs over the last rows of H out of the next matrix.
bool map_grad(CUtensorMap* m, float* ptr, unsigned long long n, unsigned long long H,
              unsigned long long Hp, unsigned cols) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {Hp, H, n}, strides[2] = {Hp * 4, H * Hp * 4};
  const cuuint32_t box[3] = {cols, 32, 1}, estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, ptr, dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, cols == 32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool CKPT>
cudaError_t launch_wgrad(cudaStream_t st, const CUtensorMap& mx, const CUtensorMap& ms,
                         const CUtensorMap& md, const CUtensorMap& mh, const CUtensorMap& msl,
                         const int* count, const int4* parts, const int2* segs, int* arrived,
                         float4* partials, int32_t* status, int E, int H, int Hp, int accumulate) {
  static GridCache cache;
  void (*kernel)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, const int*,
                 const int4*, const int2*, int*, float4*, int32_t*, int, int, int, int) = k_wgrad_pair<CKPT>;
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
  return cudaLaunchKernelEx(&cfg, kernel, mx, ms, md, mh, msl, count, parts, segs, arrived, partials, status,
                            E, H, Hp, accumulate);
}

// The workspace: count | parts | arrivals | segments | partial sums.
struct Layout {
  size_t parts, arrived, segs, partials, bytes;
};
long long tiles_of(int H, int Hp) {
  return (long long)((H + 2 * kBM - 1) / (2 * kBM)) * ((Hp + kBN - 1) / kBN);
}
// Partial sums at most: an entry of s steps is cut into at most s / most + 1 <=
// 2 s / most parts, and most >= steps * tiles / kPairs over all entries; only
// entries of more than kLeastSteps steps are cut, into at most s / 8 parts; and
// every segment of rows has one step that is not full.
long long partials_of(int R, long long rows, int G, int H, int Hp) {
  const long long segments = rows < (long long)R * G ? rows : (long long)R * G;
  const long long steps = rows / kBK + segments;
  if (steps <= kLeastSteps) return 0;
  const long long by_steps = tiles_of(H, Hp) * (steps / 8 + 1);
  return by_steps < kMostPartials ? by_steps : kMostPartials;
}
Layout layout_of(int R, long long SK, int E, int B, int H, int Hp) {
  const auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
  const size_t W = (size_t)E + (size_t)R * B;
  const long long np = partials_of(R, (long long)R * SK, E + B, H, Hp);
  Layout l;
  l.parts = 16;
  l.arrived = l.parts + 32 * (W + kMostPartials);
  l.segs = l.arrived + 4 * (size_t)np * 2 * kEpiWarps;
  l.partials = up(l.segs + 8 * (size_t)R * (E + B));
  l.bytes = l.partials + 4 * (size_t)np * kTile;
  return l;
}

}  // namespace
}  // namespace mep

using namespace mep;

extern "C" int mep_grouped_wgrad_workspace_bytes(int R, int S, int K, int E, int B, int H, int Hp,
                                                 size_t* bytes) {
  if (bytes == nullptr || R < 1 || S < 0 || K < 1 || E < 1 || B < 0) return MEP_ERR_INVALID_ARG;
  if (R > MEP_MAX_R || E > MEP_MAX_E || K > MEP_MAX_K || (long long)R * B > MEP_MAX_SLOTS)
    return MEP_ERR_INVALID_ARG;
  if (H < 8 || H % 8 != 0 || Hp < 8 || Hp % 8 != 0 || H > MEP_MAX_CKPT_C || Hp > MEP_MAX_CKPT_C)
    return MEP_ERR_INVALID_ARG;
  const long long SK = (long long)S * K;
  if (R * SK > 0x7fffff00LL ||
      tiles_of(H, Hp) > 0x7fff0000LL / (2 * kMostPartials + (long long)E + (long long)R * B))
    return MEP_ERR_INVALID_ARG;
  *bytes = layout_of(R, SK, E, B, H, Hp).bytes;
  return MEP_OK;
}

extern "C" int mep_grouped_wgrad(const void* x, int x_type, const mep_bf16* dy,
                                 const int32_t* cu_seqlens, int32_t* status, int R, int S, int K,
                                 int E, int B, int H, int Hp, int accumulate, void* ws,
                                 size_t ws_bytes, float* home_grad, float* slot_grad, void* stream) {
  size_t need = 0;
  if (mep_grouped_wgrad_workspace_bytes(R, S, K, E, B, H, Hp, &need) != MEP_OK) return MEP_ERR_INVALID_ARG;
  if (x_type != MEP_BF16 && x_type != MEP_CKPT8) return MEP_ERR_INVALID_ARG;
  const long long SK = (long long)S * K, rows = (long long)R * SK;
  if (cu_seqlens == nullptr || home_grad == nullptr || ws == nullptr || ws_bytes < need ||
      (B > 0 && slot_grad == nullptr) || (rows > 0 && (x == nullptr || dy == nullptr)))
    return MEP_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(dy) || !aligned16(home_grad) || !aligned16(slot_grad) || !aligned16(ws))
    return MEP_ERR_INVALID_ARG;
  if ((rows > 0 && (!on_current_device(x) || !on_current_device(dy))) ||
      !on_current_device(home_grad) || (B > 0 && !on_current_device(slot_grad)))
    return MEP_ERR_INVALID_ARG;
  CUtensorMap mx, ms, md, mh, msl;
  const unsigned out_cols = x_type == MEP_CKPT8 ? Ring<true>::out : Ring<false>::out;
  if (!map_grad(&mh, home_grad, E, H, Hp, out_cols)) return MEP_ERR_CUDA;
  msl = mh;  // never used without slots
  if (B > 0 && !map_grad(&msl, slot_grad, (unsigned long long)R * B, H, Hp, out_cols)) return MEP_ERR_CUDA;
  mx = ms = md = mh;  // never used without rows
  if (rows > 0) {
    const unsigned long long rb = ckpt_row_bytes(H);
    bool ok = map_2d(&md, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dy, rows, Hp, 2ull * Hp, 64,
                     x_type == MEP_CKPT8 ? Ring<true>::K : Ring<false>::K, CU_TENSOR_MAP_SWIZZLE_128B);
    if (x_type == MEP_CKPT8)
      ok = ok &&
           map_2d(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, x, rows, H, rb, kBM, Ring<true>::K, CU_TENSOR_MAP_SWIZZLE_128B) &&
           map_2d(&ms, CU_TENSOR_MAP_DATA_TYPE_UINT8, x, rows, rb, rb, 16, Ring<true>::K,
                  CU_TENSOR_MAP_SWIZZLE_NONE);
    else
      ok = ok && map_2d(&mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, rows, H, 2ull * H, 64, Ring<false>::K,
                        CU_TENSOR_MAP_SWIZZLE_128B);
    if (!ok) return MEP_ERR_CUDA;
  }
  const Layout l = layout_of(R, SK, E, B, H, Hp);
  char* p = static_cast<char*>(ws);
  int *count = reinterpret_cast<int*>(p), *arrived = reinterpret_cast<int*>(p + l.arrived);
  int4* parts = reinterpret_cast<int4*>(p + l.parts);
  int2* segs = reinterpret_cast<int2*>(p + l.segs);
  float4* partials = reinterpret_cast<float4*>(p + l.partials);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // a small block: its barriers are most of what this kernel takes
  const int W = E + R * B, group_threads = W >= kGroupThreads ? kGroupThreads : W < 128 ? 128 : (W + 31) / 32 * 32;
  cudaError_t err =
      launch_pdl(k_wgrad_groups, dim3(1), dim3(group_threads), 0, st, cu_seqlens, R, E, B, int(SK),
                 int(tiles_of(H, Hp)), accumulate, status, count, parts, segs, arrived);
  if (err != cudaSuccess) return MEP_ERR_CUDA;
  err = x_type == MEP_CKPT8 ? launch_wgrad<true>(st, mx, ms, md, mh, msl, count, parts, segs, arrived,
                                                 partials, status, E, H, Hp, accumulate)
                            : launch_wgrad<false>(st, mx, ms, md, mh, msl, count, parts, segs, arrived,
                                                  partials, status, E, H, Hp, accumulate);
  return err == cudaSuccess ? MEP_OK : MEP_ERR_CUDA;
}
