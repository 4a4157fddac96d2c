// Shared-prefix attention: the plan (which keys are shared, who has how many
// pages), the merge of the partial results, and the launch of one call.  The
// attention over the prefix is in shared_umma.cuh, over the private keys in
// shared_private.cuh.
#include <algorithm>
#include <cmath>

#include "attention_impl.cuh"
#include "block_scan.cuh"
#include "shared_prefix.cuh"

namespace pqkv {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanEach = PQKV_MAX_SEQS / kPlanThreads;

// One block, 3 us: three dependent rounds of loads and two scans.  Every later kernel
// needs all of it, so it is worth a launch of its own: repeated by each of 152 CTAs
// it would cost them the same 3 us.  The shared pages of group g are the whole pages of
// min(prefix_lens[g], min_s(L_s - q_len)): keys before every query of the
// group, so no row needs a mask in the prefix, and every sequence keeps at
// least its q_len new tokens private.
__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const SharedParams p) {
  __shared__ int s_off[PQKV_MAX_SEQS + 1];
  __shared__ int s_min[PQKV_MAX_SEQS];
  grid_dependency_wait();
  grid_dependents_launch();
  const int tid = threadIdx.x, B = p.num_seqs, M = p.num_groups;
  // -- everything that is read, at once
  const int per = (B + kPlanThreads - 1) / kPlanThreads, gper = (M + kPlanThreads - 1) / kPlanThreads;
  int len[kPlanEach], want[kPlanEach];
#pragma unroll
  for (int i = 0; i < kPlanEach; ++i) {
    const int s = tid * per + i, g = tid * gper + i;
    len[i] = i < per && s < B ? p.seq_lens[s] : 0;
    want[i] = i < gper && g < M ? p.prefix_lens[g] : 0;
  }
  // -- the groups: contiguous, in order, every sequence in one.  Offsets that
  //    are not are reported, and nothing is shared then
  bool ok = true;
  for (int g = tid; g <= M; g += kPlanThreads) {
    const int v = p.group_offsets[g];
    const int prev = g > 0 ? p.group_offsets[g - 1] : 0;
    ok = ok && (g > 0 ? v >= prev : v == 0) && (g < M || v == B);
    s_off[g] = v;
    if (g < M) s_min[g] = 0x7fffffff;
  }
  ok = __syncthreads_and(ok);
  if (!ok) {
    if (tid == 0) report(p.status, PQKV_DEV_SEQ_RANGE);
    for (int g = tid; g <= M; g += kPlanThreads) s_off[g] = g == 0 ? 0 : B;
    __syncthreads();
  }
  // -- the sequences' lengths, and the shortest of each group
  int grp[kPlanEach];
#pragma unroll
  for (int i = 0; i < kPlanEach; ++i) {
    const int s = tid * per + i;
    grp[i] = 0;
    if (i >= per || s >= B) continue;
    const int Lmax = p.bt_stride * kPageSize;
    if (len[i] < p.q_len || len[i] > Lmax) {
      report(p.status, PQKV_DEV_SEQ_RANGE);
      len[i] = max(p.q_len, min(len[i], Lmax));
    }
    grp[i] = last_at_most(s_off, M, s);
    atomicMin(&s_min[grp[i]], len[i] - p.q_len);
  }
  __syncthreads();
  // -- the groups' shared pages, row tiles and costs
  int tiles[kPlanEach], costs[kPlanEach], tsum = 0, psum = 0;
#pragma unroll
  for (int i = 0; i < kPlanEach; ++i) {
    const int g = tid * gper + i;
    tiles[i] = costs[i] = 0;
    if (i >= gper || g >= M) continue;
    const int n = s_off[g + 1] - s_off[g];
    int pages = 0;
    if (n > 0 && ok) {
      if (want[i] < 0 || want[i] > s_min[g] + p.q_len) report(p.status, PQKV_DEV_SEQ_RANGE);
      pages = max(0, min(min(want[i], s_min[g]), p.max_prefix)) / kPageSize;
    }
    p.plan.gpages(M)[g] = pages;
    p.plan.goff()[g] = s_off[g];
    tiles[i] = pages > 0 ? umma_tiles(n * p.rows) : 0;
    costs[i] = umma_weight(n * p.rows, p.split_cost) * ((pages + kUmmaPages - 1) / kUmmaPages);
    tsum += tiles[i];
    psum += costs[i];
    s_min[g] = pages;
  }
  int at_t = tsum, at_p = psum, total_t, total_p;
  block_scan2<kPlanThreads>(at_t, at_p, total_t, total_p);
#pragma unroll
  for (int i = 0; i < kPlanEach; ++i) {
    const int g = tid * gper + i;
    if (i >= gper || g >= M) continue;
    p.plan.gtiles(M)[g] = at_t;
    p.plan.gcost(M)[g] = at_p;
    at_t += tiles[i];
    at_p += costs[i];
  }
  if (tid == 0) {
    p.plan.gtiles(M)[M] = total_t;
    p.plan.gcost(M)[M] = total_p;
    p.plan.goff()[M] = B;
  }
  __syncthreads();
  // -- the private pages
  int at = 0, none = 0, total_s, total_none;
#pragma unroll
  for (int i = 0; i < kPlanEach; ++i) {
    const int s = tid * per + i;
    if (i >= per || s >= B) continue;
    at += (len[i] + kPageSize - 1) / kPageSize - s_min[grp[i]] + kSegmentCost;
  }
  block_scan2<kPlanThreads>(at, none, total_s, total_none);
#pragma unroll
  for (int i = 0; i < kPlanEach; ++i) {
    const int s = tid * per + i;
    if (i >= per || s >= B) continue;
    p.plan.len[s] = len[i];
    p.plan.group[s] = grp[i];
    p.plan.page0[s] = s_min[grp[i]];
    p.plan.spre[s] = at;
    at += (len[i] + kPageSize - 1) / kPageSize - s_min[grp[i]] + kSegmentCost;
  }
  if (tid == 0) p.plan.spre[B] = total_s;
}

struct MergeRow {
  int64_t pre_slot, suf_slot;   // its first results
  int n_pre, per;               // the prefix's results, `per` of a CTA
  int total;                    // with the private ones; 0: no row
  int pre_r, suf_r;             // its row in either's
  int h, out;                   // kv-head, output row
};

// What a row has to join.  A thread per row finds it for the row's warps: about 600
// instructions, mostly divisions, that each warp spent beside some 300 for its sums
// (64 x 5 rows: 2 us more a call).
__device__ __forceinline__ MergeRow merge_row(const SharedParams& p, int64_t row) {
  MergeRow m = {};
  const int H = p.num_kv_heads, M = p.num_groups;
  if (row >= (int64_t)p.num_seqs * p.q_len * p.num_q_heads) return m;
  const int hq = (int)(row % p.num_q_heads);
  const int tok = (int)(row / p.num_q_heads);
  const int s = tok / p.q_len, i = tok % p.q_len, gq = hq % p.group;
  const int h = hq / p.group;
  m.h = h;
  m.out = (int)row;
  const int g = p.plan.group[s];
  const int a0 = p.plan.spre[s], n = p.plan.spre[s + 1] - a0;
  const int units = p.plan.spre[p.num_seqs], costs = p.plan.gcost(M)[M];
  // -- the prefix's fragments: CTAs c0 .. c0 + n_pre / per - 1, `per` results each
  const int np = p.plan.gpages(M)[g], first = p.plan.goff()[g];
  const int behind = p.plan.goff()[g + 1];
  const int tiles = p.plan.gtiles(M)[g], nt = p.plan.gtiles(M)[g + 1] - tiles;
  const int cost = p.plan.gcost(M)[g], C = p.plan.gcost(M)[g + 1] - cost;
  if (np > 0) {
    const int nrows = (behind - first) * p.rows;
    const int R = (s - first) * p.rows + i * p.group + gq;
    const int rt = R / kUmmaRows, T = (np + kUmmaPages - 1) / kUmmaPages;
    const bool dual = nrows - rt * kUmmaRows > 128;
    const int w = dual ? kFullCost : p.split_cost;
    const int64_t a = (int64_t)cost * H + (int64_t)h * C + (int64_t)rt * kFullCost * T;
    const Shares sh((int64_t)costs * H, p.pre_workers, kPrefixShare);
    const int c0 = sh.owner(a);
    m.per = dual ? 1 : 2;
    m.n_pre = (sh.owner(a + (int64_t)w * (T - 1)) - c0 + 1) * m.per;
    m.pre_slot = (int64_t)tiles * H + h * nt + rt + c0;
    m.pre_r = R % kUmmaRows;
  }
  // -- the private ones
  const int64_t a = (int64_t)a0 * H + (int64_t)h * n;
  const Shares sh((int64_t)units * H, p.suf_workers, kPrivateShare);
  const int w0 = sh.owner(a);
  m.total = m.n_pre + sh.owner(a + n - kSegmentCost - 1) - w0 + 1;
  m.suf_slot = (int64_t)s * H + h + w0;
  m.suf_r = i * p.group + gq;
  return m;
}

// kWarps warps per output row.  The row's fragments, the prefix's first, are dealt
// to the row's warps; a warp loads four at once and folds them in with a running
// maximum, and the warps' results are joined in order (a fixed order throughout,
// so the result is deterministic).  A lane owns four dims.  Bound by the latency of its
// loads out of L2 in three or four waves of blocks: 10240 rows with 8 results each (42
// MB) take about 10 us behind the prefix's kernel, 17 from cold caches.  A block per
// sequence and head that walked its rows in one wave was slower (64 x 5: 6 us): the
// rows' loads then wait for the join before them.
template <int kWarps>
__global__ void __launch_bounds__(256) shared_merge_kernel(const SharedParams p, int scaled) {
  __shared__ float4 s_acc[kWarps > 1 ? 8 : 1][32];
  __shared__ float2 s_ml[8];
  __shared__ MergeRow s_row[8 / kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % kWarps;
  grid_dependency_wait();
  grid_dependents_launch();
  if (threadIdx.x < 8 / kWarps)
    s_row[threadIdx.x] = merge_row(p, (int64_t)blockIdx.x * (8 / kWarps) + threadIdx.x);
  __syncthreads();
  const MergeRow row = s_row[warp / kWarps];
  const bool in = row.total > 0;
  float top = kNoScore, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (in) {
    for (int k0 = sub; k0 < row.total; k0 += 4 * kWarps) {
      float m[4], lw[4];
      float4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + j * kWarps;
        m[j] = kNoScore;
        lw[j] = 0.f;
        v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < row.n_pre) {
          const int64_t slot = row.pre_slot + (k >> (row.per - 1));
          const int r = row.pre_r + (row.per > 1 ? (k & 1) * (p.pre_rp / 2) : 0);
          const float* ml = p.pre_ml + slot * 3 * p.pre_rp + r;
          m[j] = __ldg(ml);
          lw[j] = __ldg(ml + p.pre_rp) + __ldg(ml + 2 * p.pre_rp);
          v[j] = __ldg(reinterpret_cast<const float4*>(p.pre_o + (slot * p.pre_rp + r) * kHeadDim) +
                       lane);
        } else if (k < row.total) {
          const int64_t slot = row.suf_slot + (k - row.n_pre);
          const float* ml = p.suf_ml + slot * 2 * p.suf_rp + row.suf_r;
          m[j] = __ldg(ml);
          lw[j] = __ldg(ml + p.suf_rp);
          v[j] = __ldg(reinterpret_cast<const float4*>(p.suf_o +
                                                       (slot * p.suf_rp + row.suf_r) * kHeadDim) +
                       lane);
        }
      }
      const float mn = fmaxf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), top);
      const float f = ex2(top - mn);
      l *= f;
      acc.x *= f;
      acc.y *= f;
      acc.z *= f;
      acc.w *= f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float w = ex2(m[j] - mn);
        l += w * lw[j];
        acc.x += w * v[j].x;
        acc.y += w * v[j].y;
        acc.z += w * v[j].z;
        acc.w += w * v[j].w;
      }
      top = mn;
    }
  }
  if constexpr (kWarps > 1) {
    s_acc[warp][lane] = acc;
    if (lane == 0) s_ml[warp] = make_float2(top, l);
    __syncthreads();
    if (sub) return;
#pragma unroll
    for (int j = 1; j < kWarps; ++j) {
      const float2 ml = s_ml[warp + j];
      const float4 v = s_acc[warp + j][lane];
      const float mn = fmaxf(top, ml.x);
      const float f0 = ex2(top - mn), f1 = ex2(ml.x - mn);
      l = l * f0 + ml.y * f1;
      acc.x = acc.x * f0 + v.x * f1;
      acc.y = acc.y * f0 + v.y * f1;
      acc.z = acc.z * f0 + v.z * f1;
      acc.w = acc.w * f0 + v.w * f1;
      top = mn;
    }
  }
  if (!in) return;
  float inv = l > 0.f ? 1.f / l : 0.f;
  if (scaled) inv *= __ldg(p.v_scale + (p.scale_per_head ? row.h : 0));
  __half2 h01 = __floats2half2_rn(acc.x * inv, acc.y * inv);
  __half2 h23 = __floats2half2_rn(acc.z * inv, acc.w * inv);
  uint2 pk;
  pk.x = *reinterpret_cast<uint32_t*>(&h01);
  pk.y = *reinterpret_cast<uint32_t*>(&h23);
  *reinterpret_cast<uint2*>(p.out + (int64_t)row.out * kHeadDim + 4 * lane) = pk;
}

template <int kWarps>
cudaError_t launch_merge_t(const SharedParams& p, int scaled, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.num_seqs * p.q_len * p.num_q_heads;
  const int per_block = 8 / kWarps;
  return launch_pdl(shared_merge_kernel<kWarps>, (unsigned)((rows + per_block - 1) / per_block), 256,
                    0, stream, p, scaled);
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

constexpr int kMaxSms = 160;   // the workspace holds the partial results of this many SMs

// Sizes of a call, and where its arrays lie in the workspace.
struct SharedLayout {
  int pre_rp, suf_rp, pre_workers, suf_workers;
  size_t pre_o, pre_ml, suf_o, suf_ml, total;   // offsets

  SharedLayout(int B, int M, int q_len, int hq, int hkv, int kv_dtype, int sms) {
    const int rows = hq / hkv * q_len;
    // a slot holds a row tile, or twice a tile of at most 128 rows
    pre_rp = (int)std::min<int64_t>(kUmmaRows, 2 * (((int64_t)B * rows + 7) / 8 * 8));
    suf_rp = rows_padded(rows);
    sms = std::min(sms, kMaxSms);
    pre_workers = sms;
    suf_workers = sms * private_blocks_per_sm(kv_dtype, suf_rp / 8) * 8;
    // (groups without a sequence have no row tile)
    const int64_t pre_slots =
        (int64_t)(umma_tiles(B * rows) + std::min(M, B)) * hkv + pre_workers;
    const int64_t suf_slots = (int64_t)B * hkv + suf_workers;
    size_t at = up256((size_t)(4 * (B + 1) + 4 * (M + 1)) * 4);
    auto take = [&](size_t bytes) {
      const size_t here = at;
      at += up256(bytes);
      return here;
    };
    pre_o = take((size_t)pre_slots * pre_rp * kHeadDim * 4);
    pre_ml = take((size_t)pre_slots * 3 * pre_rp * 4);
    suf_o = take((size_t)suf_slots * suf_rp * kHeadDim * 4);
    suf_ml = take((size_t)suf_slots * 2 * suf_rp * 4);
    total = at;
  }
};

}  // namespace

cudaError_t launch_shared_plan(const SharedParams& p, cudaStream_t stream) {
  return launch_pdl(shared_plan_kernel, 1, kPlanThreads, 0, stream, p);
}

// Warps per row by the partial results a row may have: one warp folds four in the
// time of one load, so more warps pay from about eight results on.
cudaError_t launch_shared_merge(const SharedParams& p, int kv_dtype, cudaStream_t stream) {
  const int scaled = kv_dtype == PQKV_KV_FP8_E4M3 || kv_dtype == PQKV_KV_INT8;
  const int64_t rows = (int64_t)p.num_seqs * p.rows;         // of a kv-head
  const int64_t segs = (int64_t)umma_tiles((int)rows) * p.num_kv_heads;
  const int64_t results = (p.pre_workers / segs + 1) * (rows <= 128 ? 2 : 1) +
                          p.suf_workers / ((int64_t)p.num_seqs * p.num_kv_heads) + 1;
  if (results > 32) return launch_merge_t<8>(p, scaled, stream);
  if (results > 16) return launch_merge_t<4>(p, scaled, stream);
  if (results > 8) return launch_merge_t<2>(p, scaled, stream);
  return launch_merge_t<1>(p, scaled, stream);
}

size_t shared_prefix_workspace(int32_t num_seqs, int32_t num_groups, int32_t q_len, int32_t hq,
                               int32_t hkv) {
  // of any format: of one with the most blocks
  return SharedLayout(num_seqs, num_groups, q_len, hq, hkv, PQKV_KV_INT8, kMaxSms).total;
}

SharedParams shared_params(const AttnArgs& a, const SharedArgs& sa, void* out, void* workspace,
                           int sms, int32_t* status) {
  const int B = a.num_seqs, M = sa.num_groups;
  const SharedLayout lay(B, M, a.q_len, a.num_q_heads, a.num_kv_heads, a.kv_dtype, sms);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  SharedParams p = {};
  p.q = static_cast<const uint16_t*>(a.q);
  p.out = static_cast<uint16_t*>(out);
  p.block_table = a.block_table;
  p.seq_lens = a.seq_lens;
  p.group_offsets = sa.group_offsets;
  p.prefix_lens = sa.prefix_lens;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.status = status;
  int32_t* at = reinterpret_cast<int32_t*>(ws);
  auto take = [&](int n) {
    int32_t* here = at;
    at += n;
    return here;
  };
  p.plan.len = take(B);
  p.plan.group = take(B);
  p.plan.page0 = take(B);
  p.plan.spre = take(B + 1);
  p.plan.groups = take(4 * (M + 1));
  p.pre_o = reinterpret_cast<float*>(ws + lay.pre_o);
  p.pre_ml = reinterpret_cast<float*>(ws + lay.pre_ml);
  p.suf_o = reinterpret_cast<float*>(ws + lay.suf_o);
  p.suf_ml = reinterpret_cast<float*>(ws + lay.suf_ml);
  p.num_pages = a.num_pages;
  p.bt_stride = a.max_pages_per_seq;
  p.num_seqs = B;
  p.num_groups = M;
  p.q_len = a.q_len;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.group = a.num_q_heads / a.num_kv_heads;
  p.rows = p.group * a.q_len;
  p.scale_per_head = a.scale_per_head ? 1 : 0;
  p.pre_rp = lay.pre_rp;
  p.suf_rp = lay.suf_rp;
  // no more CTAs than the caller's bounds leave work for
  const int cap = a.max_pages_per_seq * kPageSize;
  const int longest = a.max_seq_len > 0 ? std::min(a.max_seq_len, cap) : cap;
  p.max_prefix = sa.max_prefix_len > 0 ? std::min(sa.max_prefix_len, longest) : longest;
  const int64_t tiles = (int64_t)(p.max_prefix / kPageSize + kUmmaPages - 1) / kUmmaPages *
                        (umma_tiles(B * p.rows) + M) * a.num_kv_heads;
  p.pre_workers = (int)std::min<int64_t>(lay.pre_workers, tiles);
  const int64_t units = (int64_t)B * a.num_kv_heads *
                        ((longest + kPageSize - 1) / kPageSize + kSegmentCost);
  p.suf_workers =
      (int)std::min<int64_t>(lay.suf_workers, (units / kPrivateShare + 7) / 8 * 8);
  p.split_cost = a.kv_dtype == PQKV_KV_FP8_E4M3 || a.kv_dtype == PQKV_KV_INT8 ? 3 : 2;
  p.sm_scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)a.head_dim));
  return p;
}

cudaError_t launch_shared_prefix(const AttnArgs& a, const SharedArgs& sa, void* out,
                                 const CUtensorMap& prefix_map, const CUtensorMap& map,
                                 void* workspace, int sms, int32_t* status, cudaStream_t stream) {
  const SharedParams p = shared_params(a, sa, out, workspace, sms, status);
  cudaError_t e = launch_shared_plan(p, stream);
  if (e != cudaSuccess) return e;
  switch (a.kv_dtype) {
    case PQKV_KV_FP16: e = launch_shared_fp16(p, prefix_map, map, stream); break;
    case PQKV_KV_FP8_E4M3: e = launch_shared_e4m3(p, prefix_map, map, stream); break;
    case PQKV_KV_INT8_ROW: e = launch_shared_int8_row(p, prefix_map, map, stream); break;
    default: e = launch_shared_int8(p, prefix_map, map, stream); break;
  }
  if (e != cudaSuccess) return e;
  return launch_shared_merge(p, a.kv_dtype, stream);
}

}  // namespace pqkv
