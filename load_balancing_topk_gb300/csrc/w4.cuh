// w4.cuh -- the 4-bit weight matrix shared by w4.cu and few.cu.
//
// A matrix [K, N]: panels of 64 columns, each a run of blocks of 128 rows
// (K and N filled up with zeros). A block is 4096 bytes of pairs and then
// 128 / group rows of 64 bf16 scales. Row k = 64 h + 16 j + 8 i + 2 t + e of a
// block and column n = 16 c + 8 l + g of a panel: q + 8 is half l of byte
// ((((4 h + c) * 8 + g) * 4 + t) * 4 + j) * 4 + 2 e + i; the scale is number
// 16 c + 2 g + l of its group's 64.
// So lane (g, t) of a warp finds in its 16 bytes of (h, c) columns g and g + 8
// at the rows that the A operand of four m16n8k16 products wants of it: word j
// is step j, and its halves' nibbles i, l the operand's four registers, an even
// row in the lower half word and the next in the upper. One panel's blocks are
// one contiguous run, scales beside the pairs they belong to, so that a column
// of the product is one bulk copy after another.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "mep_common.cuh"

namespace mep {
namespace {

constexpr int kW4Rows = 128, kW4Cols = 64;          // of a block
constexpr int kW4Pairs = kW4Rows * kW4Cols / 2;     // bytes of pairs
constexpr float kW4Top = 7.f;                       // largest |q|

__host__ __device__ constexpr int w4_block_bytes(int group) {
  return kW4Pairs + kW4Rows / group * kW4Cols * 2;
}
__host__ __device__ __forceinline__ long long w4_panel_bytes(long long K, int group) {
  return (K + kW4Rows - 1) / kW4Rows * w4_block_bytes(group);
}
__host__ __device__ __forceinline__ long long w4_matrix_bytes(long long K, long long N, int group) {
  return (N + kW4Cols - 1) / kW4Cols * w4_panel_bytes(K, group);
}
inline bool w4_sizes_ok(long long K, long long N, int group) {
  return K >= 1 && K <= MEP_MAX_W4 && N >= 1 && N <= MEP_MAX_W4 && (group == 32 || group == 64 || group == 128);
}

}  // namespace
}  // namespace mep
