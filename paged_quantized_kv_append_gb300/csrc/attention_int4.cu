// Paged attention instantiations for 4-bit codes with a scale per group of 32
// values (kept in its own translation unit so the formats compile in parallel).
#include "attention_launch.cuh"

namespace pqkv {

cudaError_t launch_attention_int4_group(const AttnParams& p, const CUtensorMap& map, int grid,
                                      int nt, bool pair, cudaStream_t stream) {
  if (p.num_splits == 0) return launch_int4_umma_plain(p, grid, nt, stream);
  return launch_attention_dtype<PQKV_KV_INT4_GROUP>(p, map, grid, nt, pair, stream);
}

int attention_blocks_per_sm_int4_group(int nt, bool pair, int num_seqs) {
  return blocks_per_sm_dtype<PQKV_KV_INT4_GROUP>(nt, pair, num_seqs);
}

cudaError_t launch_attention_partial_int4_group(const AttnPartialParams& p, const CUtensorMap& map,
                                              int grid, int nt, bool pair, cudaStream_t stream) {
  if (p.num_splits == 0) return launch_int4_umma_partial(p, grid, nt, stream);
  return launch_attention_partial_dtype<PQKV_KV_INT4_GROUP>(p, map, grid, nt, pair, stream);
}

cudaError_t launch_attention_window_int4_group(const AttnWindowParams& p, const CUtensorMap& map,
                                             int grid, int nt, cudaStream_t stream) {
  if (p.num_splits == 0) return launch_int4_umma_window(p, grid, nt, stream);
  return launch_attention_window_dtype<PQKV_KV_INT4_GROUP>(p, map, grid, nt, stream);
}

}  // namespace pqkv
