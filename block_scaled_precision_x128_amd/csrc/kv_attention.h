// How one fp8_kv_attention call is laid out: the split of the positions and
// the parts of the workspace, shared by the kernels of the call.
#pragma once

#include "attention.h"
#include "device_common.h"
#include "paging.h"

namespace fp8blk {

// Rows (query tokens x heads of a kv head) that the decode kernel takes: two
// tiles of 16, one for heads of 256, whose second tile does not fit the
// registers.
constexpr int decode_rows(int head_dim) { return head_dim == 256 ? 16 : 32; }

struct KvPlan {
  FastDiv page, group;        // by block_size, by heads / kv_heads
  int head_waves;             // decode: kv heads of a workgroup, a power of two up to 4
  int splits, split_len;      // positions [s split_len, (s + 1) split_len) go to split s
  float* part_o;              // [splits, part_rows, D]: sum of p v of a split, without the value scales
  v2f* part_ml;               // [splits, part_rows]: its maximum (powers of two) and sum of p
  int64_t part_rows;          // q_tokens * heads
  float* lse;                 // the caller's, or the workspace's where a chunk's weights need one
  float* scores;              // decode with weights: [batch, kv_heads, score_rows, score_ld], powers of two
  int64_t score_rows, score_ld;
  void* queries;              // chunk with weights: the rows' operands and factors, null otherwise
  float* factors;
  int64_t row_tiles;          // tiles of 32 rows of a (sequence, kv head)
};

// Waves of a workgroup of the chunk kernel, 32 rows each, and the workgroups
// that cover the rows.  (Eight waves for 256 rows or more, staging a tile for
// twice the rows: 1189 us against 1118 at 2048 new tokens on 32k positions, 64
// against 60 at 8 x 64 on 4k, 219 against 224 at 2 x 512 on 8k.)
constexpr int kChunkWaves = 4;
inline int64_t kv_chunk_tiles(int64_t heads, int64_t kv_heads, int64_t max_q) {
  return (max_q * (heads / kv_heads) + 32 * kChunkWaves - 1) / (32 * kChunkWaves);
}

// The split of max_kv positions over `units` workgroups each.
void plan_splits(int64_t units, int64_t groups, int64_t least, int64_t grain, int64_t max_kv, KvPlan& p);
// Joins the splits into a.out and p.lse.
void launch_join(const KvAttnArgs& a, const KvPlan& p, int head_dim, hipStream_t st);

void launch_kv_decode(const KvAttnArgs& a, const KvPlan& p, int head_dim, hipStream_t st);
void launch_kv_chunk(const KvAttnArgs& a, const KvPlan& p, int head_dim, hipStream_t st);
// weights_out of a chunk, after p.lse has been written.
void launch_kv_chunk_weights(const KvAttnArgs& a, const KvPlan& p, int head_dim, hipStream_t st);

}  // namespace fp8blk
