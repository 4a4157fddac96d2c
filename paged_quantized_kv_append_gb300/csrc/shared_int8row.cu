// Shared-prefix attention instantiations for one KV format (kept in its own
// translation unit so the formats compile in parallel).
#include "shared_prefix.cuh"

namespace pqkv {

cudaError_t launch_shared_int8_row(const SharedParams& p, const CUtensorMap& map, cudaStream_t st) {
  return launch_shared_dtype<PQKV_KV_INT8_ROW>(p, map, st);
}

}  // namespace pqkv
