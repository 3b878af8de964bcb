// The specialised attention kernels, as hc_attn.cu dispatches them.
#pragma once

#include "hc_attn.cuh"
#include "hc_internal.h"

namespace hc {

// Up to 16 rows to a key head (hc_attn_rows.cu). `single`: every sequence has one
// new token; `aligned`: 16-byte accesses are possible everywhere.
bool attn_rows_supported(int dtype, int dim, bool single, int group, bool aligned);
// Its own split of sequences of one new token: CTAs beside one for each tile, and
// pieces (of all sequences) at most; none where splits by the host are as good.
// `keys`: the longest sequence's.
struct RowsSchedule {
  int spare_ctas, units;
  bool clusters;  // no pieces, but a cluster to a sequence
};
RowsSchedule attn_rows_schedule(int64_t seqs, int kv_heads, int64_t keys, int num_sms);
cudaError_t launch_attn_rows(const AttnArgs& a, int dtype, int64_t slots, cudaStream_t s);

// float32, tiles of 64 rows (hc_attn_f32.cu).
bool attn_f32_supported(int dtype, int dim, bool aligned);
cudaError_t launch_attn_f32(const AttnArgs& a, int64_t slots, cudaStream_t s);

// Any number of rows, on tcgen05 (hc_attn_tile.cu); takes a workspace of its
// own and needs no splits.
bool attn_tile_supported(int dtype, int dim, int page, float scale, bool aligned);
size_t attn_tile_workspace(int64_t tokens, int group, int seqs, int dim, int num_sms);
cudaError_t launch_attn_tile(const AttnArgs& a, int dtype, void* workspace, int num_sms, cudaStream_t s);

}  // namespace hc
