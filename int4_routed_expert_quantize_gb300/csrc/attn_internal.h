// Internal types of the paged-cache attention (coli_attn.h): what the kernels get, the workspace
// and the launchers.  Not part of the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "coli_attn.h"

namespace coli {

constexpr int kAttnMaxSeqs = 4096;
constexpr int kAttnMaxGroup = 64;     // query heads per key head
constexpr int kAttnPrefixRows = 8;    // tokens per sequence the prefix workspace is sized for
constexpr int kAttnMaxPairs = 64;     // rotated pairs of a head
constexpr int kAttnNoWindow = 1 << 30;
// AttnParams::unit_cost of the two kernels.  Geometric mean over 23 batches, us, with 1 / 2 / 3 for the split kernel:
// 32.1 / 31.7 / 31.7; with 1 / 2 / 3 / 4 / 6 for the tensor-memory kernel: 31.7 / 31.4 / 31.7 / 32.0 / 32.9.
constexpr int kSplitUnitCost = 2;
constexpr int kTileUnitCost = 2;
constexpr int kSplitMaxRows = 32;     // rows of a block of the split kernel, and of a sequence it takes
constexpr int kSplitKeys = 64;        // keys per tile of the split kernel
constexpr int kTileKeys = 128;        // keys per tile of the tensor-memory kernel
constexpr int kTileRows = 256;        // query rows per block of the tensor-memory kernel (2 x 128)

// A unit of attention work is one block of query tokens of one sequence with one key head; a list of all
// units' key tiles is cut into equal stretches, one per CTA.  A unit cut by a stretch's end leaves
// one partial result per CTA in the workspace: the first part in slot 1 of its CTA, the others in slot 0
// of theirs.  Its record, at the index of the CTA with the second part, tells the combine kernel.
struct AttnRec {
  int first_cta, last_cta;  // CTAs with a part of the unit; first_cta < 0: no record
  int token0, tokens;       // the unit's query tokens
  int head;                 // key head
};

struct AttnParams {
  const void* q;
  int64_t q_stride;
  void* out;
  int64_t out_stride;
  bool out_sectors;  // every head of out starts on a 32-byte boundary (otherwise on a 16-byte one)
  float* lse;
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* table;
  int64_t table_stride;
  int n_seqs, n_tokens, max_pages;  // n_seqs 0: the shared prefix alone
  int max_q;  // new tokens of a sequence at most (from more, rows of cut units go missing, which is reported)
  // the shared prefix, or nullptr: one more sequence (number n_seqs) with all n_tokens queries, each of which
  // sees all its keys
  const int32_t* pre_len;
  const int32_t* pre_table;
  int pre_pages;
  int n_q, n_kv, group, head_dim;
  int page_shift, n_pages;
  int window, sinks;  // window >= kAttnNoWindow: none (and sinks 0)
  float scale_log2;   // scale * log2(e)
  int block_tokens;   // query tokens per block
  int late_wait;      // the launch before this one belongs to the same call and is not read: wait for it at the end
  int unit_cost;      // list positions of a unit besides its tiles
  // workspace
  float* part_o;     // [2 * CTAs][rows per block][head_dim] unnormalised partial outputs
  float2* part_ml;   // [2 * CTAs][rows per block] their maximum (log2 units) and sum
  AttnRec* rec;      // [CTAs]
  uint32_t* seq_pos;  // [n_seqs + 3] first list position of each sequence, the total, the stretch; or nullptr
  // prefix calls only: rows of uncut units go here, unnormalised, by (token, head); [0] those of the sequences'
  // own keys, [1] those of the prefix
  float* dense_o[2];
  float2* dense_ml[2];
  uint8_t* redo;   // [max_tokens][n_kv] rows the joining kernel computes again (flag_unit), zero otherwise
  int* redo_any;   // [0] some are; [1] blocks of that kernel that are done
  int64_t k_page, k_head, k_slot, v_page, v_head, v_slot;  // cache strides, for those units
  const void *kc, *vc;
  int* status;
};

struct AttnKvMaps {  // boxes of 64 values x min(page, box) slots, 128-byte swizzle
  CUtensorMap k64, v64;    // box 64 slots: split kernel
  CUtensorMap k128, v128;  // box 128 slots: tensor-memory kernel
};

struct AttnAppend {
  const void *q, *k, *v;
  void *q_out, *kc, *vc;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  int64_t kp, kh, ks, vp, vh, vs;  // cache strides in elements
  const int32_t *q_start, *kv_len, *table;
  int64_t table_stride;
  int n_seqs, n_tokens, max_pages, n_pages, page_shift;
  int n_q, n_kv, head_dim, rot, interleaved;
  const int32_t* pos_base;  // added to every position for the rotation, or nullptr
  const uint64_t* turn;  // [rot/2] turns per position as a fraction of 2^64
  int* status;
};

int split_rows(int64_t rows);  // rows per block of the split kernel for sequences of up to `rows` rows
int split_grid(int num_sms);  // CTAs
cudaError_t configure_attn_split();
cudaError_t launch_attn_split(const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v,
                              int rows, int dtype, int num_sms, cudaStream_t stream);
int tile_block_tokens(int group);  // tokens per block of the tensor-memory kernel
cudaError_t configure_attn_tile();
cudaError_t launch_attn_tile(const AttnParams& p, const CUtensorMap& q, const CUtensorMap& k,
                             const CUtensorMap& v, int dtype, int num_sms, cudaStream_t stream);
// merges the partials of cut units into out / lse; the launch before had `ctas` CTAs and blocks of `rows` rows, of
// which at most `live` are in use
cudaError_t launch_attn_combine(const AttnParams& p, int rows, int live, int ctas, int dtype, cudaStream_t stream);
// merges, for every row, the sequence's own and the prefix's results into out / lse; same_list: one launch, with blocks of
// own_rows rows, made both; else the split kernel made the sequences' and the tensor-memory kernel the prefix's
cudaError_t launch_attn_join(const AttnParams& own, int own_rows, const AttnParams& shared, bool same_list,
                             int shared_ctas, int dtype, cudaStream_t stream);
cudaError_t launch_attn_append(const AttnAppend& a, int dtype, int num_sms, cudaStream_t stream);

}  // namespace coli
