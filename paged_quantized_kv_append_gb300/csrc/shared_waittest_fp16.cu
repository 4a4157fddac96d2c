// Shared-prefix attention of one KV format in the test mode of its bounded waits (see
// pqkv_testing.h): kernels of its own, so that the production ones are compiled as
// without it.
#include "shared_umma.cuh"

namespace pqkv {

cudaError_t launch_shared_wait_test_fp16(const SharedWaitTestParams& p, const CUtensorMap& prefix_map,
                                       const CUtensorMap& map, cudaStream_t st) {
  const cudaError_t e = launch_private_t<PQKV_KV_FP16, 3>(p, map, st);
  if (e != cudaSuccess) return e;
  return launch_shared_umma_t<PQKV_KV_FP16>(p, prefix_map, st);
}

}  // namespace pqkv
