// Shared-prefix attention instantiations for one KV format (kept in its own
// translation unit so the formats compile in parallel).
#include "shared_umma.cuh"

namespace pqkv {

cudaError_t launch_shared_fp16(const SharedParams& p, const CUtensorMap& prefix_map,
                             const CUtensorMap& map, cudaStream_t st) {
  const cudaError_t e = launch_private_dtype<PQKV_KV_FP16>(p, map, p.suf_rp / 8, st);
  if (e != cudaSuccess) return e;
  return launch_shared_umma_t<PQKV_KV_FP16>(p, prefix_map, st);
}

}  // namespace pqkv
