// Test instantiation of the 4-bit tcgen05 kernel for its bounded waits (see
// pqkv_testing.h): 24 rows, one tile's copies never issued, waits of about 1 ms.
#include "int4_umma.cuh"

namespace pqkv {

cudaError_t launch_int4_umma_wait_test(const AttnWaitTestParams& p, int grid, cudaStream_t stream) {
  return launch_int4_umma_t<3>(p, grid, stream);
}

}  // namespace pqkv
