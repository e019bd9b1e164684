// The 4-bit form of a tensor (moe_mx4 in moe.h) on the device: where codes and
// scales lie.
#pragma once

#include "common.h"

namespace moe {

constexpr int kMxBlock = 32;   // values that share a scale
constexpr int kMxTile = 128;   // contraction length of a tile: 16 columns x 128 = 1 KiB of codes
constexpr int kMxGroup = 512;  // contraction length of a word of scales

__host__ __device__ constexpr int mx_groups(int64_t k) { return int((k + kMxGroup - 1) / kMxGroup); }

// Of a strip of 16 columns of a weight matrix [k, cols], lane (g, c) = (lane / 16,
// lane % 16) holds the 32 values from 32g on of column c of each tile: 16 bytes of
// codes, and a byte of the word of scales of four tiles.  This is its share of the
// row operand of a 16 x 16 x 128 matrix instruction.
// Words of 16 bytes of codes, and words of scales, before strip `strip` (over all matrices).
__device__ __forceinline__ int64_t mx_strip_codes(int64_t strip, int64_t k) { return strip * (k / kMxTile) * kWave; }
__device__ __forceinline__ int64_t mx_strip_scales(int64_t strip, int64_t k) { return strip * mx_groups(k) * kWave; }

}  // namespace moe
