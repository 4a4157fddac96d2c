// Attention of a batch whose sequences share prefixes: decode / verify
// attention with the result of pqkv_paged_attention, in which the keys of a
// shared prefix are read once for all the sequences that share it.
//
// With p_g the shared pages of group g, the keys of a sequence s of the group
// are split in two: the prefix, keys [0, 16 p_g), which every query row of the
// group sees whole, and the private keys [16 p_g, L_s).  Softmax over a union
// of key sets needs only (m, l, O) of each set,
//     m = max score,  l = sum_j 2^{s_j - m},  O = sum_j 2^{s_j - m} V_j
// (scores in log2 units), and
//     out = sum_p 2^{m_p - M} O_p / sum_p 2^{m_p - M} l_p,   M = max_p m_p.
// So the prefix is one product of all the group's rows (n_g * q_len * G of a
// kv-head) with its keys, the private part is attention over a short cache,
// and a merge joins them.
#pragma once

#include "pqkv_common.cuh"

namespace pqkv {

// What the plan kernel leaves in the workspace for the kernels after it
// (int32 each; N = num_seqs, M = num_groups).
struct SharedPlan {
  int32_t* len;       // [N]     tokens of the sequence, clamped into its row
  int32_t* group;     // [N]     its group
  int32_t* page0;     // [N]     its first private page = its group's shared pages
  int32_t* spre;      // [N + 1] units of the sequences before it, see kSegmentCost
  // four rows of M + 1: the group's first sequence, its shared pages, the row
  // tiles of a kv-head in the groups before it, and those tiles' cost
  int32_t* groups;
  __host__ __device__ int32_t* goff() const { return groups; }
  __host__ __device__ int32_t* gpages(int M) const { return groups + (M + 1); }
  __host__ __device__ int32_t* gtiles(int M) const { return groups + 2 * (M + 1); }
  __host__ __device__ int32_t* gcost(int M) const { return groups + 3 * (M + 1); }
};

struct SharedParams {
  const uint16_t* q;        // fp16 bits [B*q_len][Hq][128]
  uint16_t* out;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* group_offsets;
  const int32_t* prefix_lens;
  const float* k_scale;     // INT8_ROW: the fp16 row scales after the pool's codes
  const float* v_scale;
  int32_t* status;
  SharedPlan plan;
  float* pre_o;             // prefix fragments: [slots][RP][128] unnormalised O
  float* pre_ml;            // [slots][3][RP] m (log2 units), and l of either half's keys
  float* suf_o;             // private fragments, the same
  float* suf_ml;            // [slots][2][RP] m and l
  int64_t num_pages;
  int32_t bt_stride;
  int32_t num_seqs;
  int32_t num_groups;
  int32_t q_len;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t group;            // num_q_heads / num_kv_heads
  int32_t rows;             // group * q_len: query rows of a (sequence, kv-head)
  int32_t scale_per_head;
  int32_t pre_rp;           // rows of a prefix fragment's slot
  int32_t suf_rp;           // padded rows of a private fragment
  int32_t max_prefix;       // bound of the prefixes that are shared
  int32_t pre_workers;      // CTAs of the prefix launch (0: nothing to share, no launch)
  int32_t split_cost;       // of a key tile for a row tile of at most 128 rows; see kFullCost
  int32_t suf_workers;      // warps of the private-key launch
  float sm_scale_log2;      // log2(e) / sqrt(head_dim)
};

// Test mode of the bounded waits: one copy is never issued, and waits give up after
// about 1 ms.  Built only into the testing entry point.
struct SharedWaitTestParams : SharedParams {
  int32_t skip_block;       // CTA of the prefix launch, or warp of the private keys' launch
  int32_t skip_part;        // 0: a key tile of K, 1: of V, 2: a private page
  int32_t skip_tile;        // which one of the block's (warp's) share
};
constexpr long long kTestWaitCycles = 1ll << 21;

// Equal contiguous shares of U units over at most `most` workers, at least
// `min_share` units each (fewer, larger shares where there is little to do: each
// share ends in a partial result that the merge has to read).  Every share is
// non-empty, so the workers holding units of [a, b) are owner(a)..owner(b-1).
struct Shares {
  int64_t U;
  int n;
  __device__ __forceinline__ Shares(int64_t units, int most, int min_share) : U(units) {
    const int64_t want = div(units, min_share);
    n = (int)(want < most ? (units > 0 && want < 1 ? 1 : want) : most);
  }
  static __device__ __forceinline__ int64_t div(int64_t a, int64_t b) {
    if (((uint64_t)a | (uint64_t)b) <= 0xFFFFFFFFull) return (uint32_t)a / (uint32_t)b;
    return a / b;
  }
  __device__ __forceinline__ int64_t start(int w) const { return div((int64_t)w * U, n); }
  __device__ __forceinline__ int owner(int64_t x) const { return (int)div((x + 1) * n - 1, U); }
};

constexpr int kUmmaRows = 256;      // rows of a full row tile
constexpr int kUmmaKeys = 128;      // keys of a key tile
constexpr int kUmmaPages = kUmmaKeys / kPageSize;

// Work of the prefix: (row tile, key tile) pairs of a kv-head.  The row tiles of a
// kv-head are full ones, then the rest.  A key tile costs a row tile of more than
// 128 rows kFullCost, a smaller one (half the products, the same codes to widen)
// split_cost.  For E4M3 and INT8, where widening decides a small row tile, 3
// (cycles per key tile: 2940 against 2350; decode of 256: 111 us, with 2: 116).  For
// FP16, with nothing to widen (2620 against 1500), and INT8_ROW, whose scores cost the
// softmax more, 2 (verification of 4 groups: 112 us, with 3: 120).
constexpr int kFullCost = 4;
__host__ __device__ __forceinline__ int umma_tiles(int rows) {
  return (rows + kUmmaRows - 1) / kUmmaRows;
}
__host__ __device__ __forceinline__ int umma_weight(int rows, int split_cost) {
  const int rem = rows % kUmmaRows;
  return kFullCost * (rows / kUmmaRows) + (rem > 128 ? kFullCost : (rem > 0 ? split_cost : 0));
}
// Work of the private keys: the units of a (sequence, kv-head) segment are its pages,
// then kSegmentCost that stand for its query rows and its partial result: a share in
// sequences of one or two private pages holds many segments, and by pages alone one SM
// worked 99K cycles where the others took 61K (13 us of a call: fp16 verification of
// 32 x 8; with 1 119 us, 2 116, 6 117, E4M3 decode of 256 113, 111 and 113).
constexpr int kSegmentCost = 2;
constexpr int kPrivateShare = 2;             // units, the least of a warp
constexpr int kPrefixShare = kFullCost;      // a key tile, the least of a CTA

// The steps of one validated call: its parameters (queues nothing), the plan and the
// merge.
SharedParams shared_params(const AttnArgs& a, const SharedArgs& sa, void* out, void* workspace,
                           int sms, int32_t* status);
cudaError_t launch_shared_plan(const SharedParams& p, cudaStream_t stream);
cudaError_t launch_shared_merge(const SharedParams& p, int kv_dtype, cudaStream_t stream);

// A call's two halves, per KV format (shared_<format>.cu).  prefix_map: see
// encode_prefix_map; map: the attention's own.
cudaError_t launch_shared_fp16(const SharedParams& p, const CUtensorMap& prefix_map,
                               const CUtensorMap& map, cudaStream_t st);
cudaError_t launch_shared_e4m3(const SharedParams& p, const CUtensorMap& prefix_map,
                               const CUtensorMap& map, cudaStream_t st);
cudaError_t launch_shared_int8(const SharedParams& p, const CUtensorMap& prefix_map,
                               const CUtensorMap& map, cudaStream_t st);
cudaError_t launch_shared_int8_row(const SharedParams& p, const CUtensorMap& prefix_map,
                                   const CUtensorMap& map, cudaStream_t st);

// Blocks per SM of the private-key launch for rows padded to 8 nt: two where registers
// and shared memory hold them (8 rows; an fp16 block's ring takes 128 KB, and a grid of
// two for an SM that holds one made two waves: 64 fp16 sequences of 4K shared and up to
// 1K private tokens 75.9 us, with one 71.3).
constexpr int private_blocks_per_sm(int kv_dtype, int nt) {
  return nt == 1 && kv_dtype != PQKV_KV_FP16 ? 2 : 1;
}

}  // namespace pqkv
