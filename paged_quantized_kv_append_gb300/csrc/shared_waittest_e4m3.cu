// Shared-prefix attention of one KV format in the test mode of its bounded waits (see
// pqkv_testing.h): kernels of its own, so that the production ones are compiled as
// without it.
#include "pqkv_testing.h"
#include "shared_umma.cuh"

namespace pqkv {

cudaError_t launch_shared_wait_test_e4m3(const SharedWaitTestParams& p, const CUtensorMap& prefix_map,
                                       const CUtensorMap& map, cudaStream_t st) {
  const cudaError_t e = launch_private_t<PQKV_KV_FP8_E4M3, 3>(p, map, st);
  if (e != cudaSuccess) return e;
  return launch_shared_umma_t<PQKV_KV_FP8_E4M3>(p, prefix_map, st);
}

cudaError_t launch_shared_wait_test_fp16(const SharedWaitTestParams& p,
                                         const CUtensorMap& prefix_map, const CUtensorMap& map,
                                         cudaStream_t st);

}  // namespace pqkv

using namespace pqkv;

extern "C" int pqkv_testing_shared_prefix_wait_timeout(
    const void* q, void* out, const void* pages, int64_t num_pages, const int32_t* block_table,
    int32_t max_pages_per_seq, const int32_t* seq_lens, int32_t num_seqs,
    const int32_t* group_offsets, const int32_t* prefix_lens, int32_t num_groups, int32_t q_len,
    int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
    int32_t kv_dtype, const float* k_scale, const float* v_scale, int32_t scale_per_head,
    int32_t max_seq_len, int32_t max_prefix_len, void* workspace, size_t workspace_bytes,
    int32_t* status, void* stream, int32_t skip_block, int32_t skip_part, int32_t skip_tile) {
  AttnArgs a{q, pages, num_pages, block_table, max_pages_per_seq, seq_lens, num_seqs, q_len,
             num_q_heads, num_kv_heads, head_dim, page_size, kv_dtype, k_scale, v_scale,
             scale_per_head, 0, max_seq_len};
  const SharedArgs sa{group_offsets, prefix_lens, num_groups, max_prefix_len};
  CUtensorMap map, prefix_map;
  int sms = 0;
  const int rc = bind_shared_prefix(&a, sa, out, workspace, workspace_bytes, status, &prefix_map,
                                    &map, &sms);
  if (rc || num_seqs == 0) return rc;
  SharedWaitTestParams p;
  static_cast<SharedParams&>(p) = shared_params(a, sa, out, workspace, sms, status);
  p.skip_block = skip_block;
  p.skip_part = skip_part;
  p.skip_tile = skip_tile;
  if (p.suf_rp != 24 || (kv_dtype != PQKV_KV_FP16 && kv_dtype != PQKV_KV_FP8_E4M3))
    return PQKV_EUNSUPPORTED;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_shared_plan(p, st);
  if (e == cudaSuccess)
    e = kv_dtype == PQKV_KV_FP16 ? launch_shared_wait_test_fp16(p, prefix_map, map, st)
                                 : launch_shared_wait_test_e4m3(p, prefix_map, map, st);
  if (e == cudaSuccess) e = launch_shared_merge(p, kv_dtype, st);
  return e == cudaSuccess ? PQKV_OK : PQKV_ECUDA;
}
