// Paged attention over 4-bit codes with a scale per group of 32 values: balanced calls run
// on tcgen05 (int4_umma.cuh), fixed splits, whose blocks each take one partition, in the
// kernel that the other formats use.
#include "attention_launch.cuh"

namespace pqkv {

cudaError_t launch_attention_int4_group(const AttnParams& p, const CUtensorMap& map, int grid,
                                      int nt, bool pair, cudaStream_t stream) {
  if (p.num_splits == 0) return launch_int4_umma_plain(p, grid, nt, stream);
  return launch_attention_dtype<PQKV_KV_INT4_GROUP>(p, map, grid, nt, pair, stream);
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
