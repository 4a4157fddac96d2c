// The tcgen05 attention kernels of 4-bit pools, one call each per mode (in a translation
// unit of its own, so that the formats compile in parallel).
#include "int4_umma.cuh"

namespace pqkv {

cudaError_t launch_int4_umma_plain(const AttnParams& p, int grid, int nt, cudaStream_t stream) {
  return launch_int4_umma(p, grid, nt, stream);
}
cudaError_t launch_int4_umma_partial(const AttnPartialParams& p, int grid, int nt,
                                     cudaStream_t stream) {
  return launch_int4_umma(p, grid, nt, stream);
}
cudaError_t launch_int4_umma_window(const AttnWindowParams& p, int grid, int nt,
                                    cudaStream_t stream) {
  return launch_int4_umma(p, grid, nt, stream);
}

}  // namespace pqkv
