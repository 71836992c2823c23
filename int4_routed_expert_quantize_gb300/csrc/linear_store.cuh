// The device layout of 4-bit weights (coli_linear.h), which both kernels read.
//
// 8 rows x 128 columns are a block: 32 lanes x 16 bytes of codes (+ 8, so that they are unsigned), then each row's
// scales of the block's groups.  A tile of 8 rows is its blocks one after another.  Lane (n = lane / 4, c = lane % 4) holds 4 words of 8
// columns of row n, all of one group for all c: groups of 128 take columns 32 c + 8 j (word j), of 64 columns
// 64 (j / 2) + 16 c + 8 (j % 2), of 32 columns 32 j + 8 c.  Nibble i of a word is column 2 i (i < 4) or 2 i - 7, so that masks take
// pairs of neighbours.
#pragma once

#include "attn_device.cuh"
#include "bulk.cuh"

namespace coli {

constexpr int kBlockCodes = 512;

__host__ __device__ constexpr int block_bytes(int group) { return kBlockCodes + 16 * (128 / group); }

// column of a lane's word j within a block
template <int G>
__host__ __device__ constexpr int word_col(int c, int j) {
  return G == 128 ? 32 * c + 8 * j : G == 64 ? 64 * (j >> 1) + 16 * c + 8 * (j & 1) : 32 * j + 8 * c;
}

struct LinearParams {
  const uint8_t* store;
  const uint16_t* x;
  uint16_t* y;
  int64_t x_stride, y_stride;
  int n_tokens, rows, cols;
  int tiles, blocks;  // of the whole matrix
  int part;           // blocks of a CTA of the cluster (the last one may have fewer)
  int kw, rw;         // warps that share a tile, tiles' worth of warps: a step is rw * step_tiles tiles
  int slots;
  int* status;
};

// more than 16 tokens, groups of 128
cudaError_t configure_linear_many();
cudaError_t launch_linear_many(const LinearParams& p, int dtype, int num_sms, cudaStream_t stream);

}  // namespace coli
