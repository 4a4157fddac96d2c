// The private keys of a shared-prefix batch: short caches of many sequences.
// One warp per share: the fragments of a contiguous range of units (the pages of
// (sequence, kv-head) segments, and what a segment costs besides), each streamed by the warp alone (no barrier between warps, so a
// sequence with a few pages costs a few pages).  Per page the products are the
// attention kernel's: S^T = K Q^T with the page's tokens as M and the G*q_len
// query rows as N, O^T = V^T P^T.
//
// What bounds it: the instructions between a page's products (about 780 a page for 32
// rows) with two warps a scheduler to hide their latencies, which is what the register
// file holds at 24 and 32 rows (a third of the issue slots used, DRAM 25 %, the tensor
// pipe 20 % of the time).  2168 E4M3 pages x 8 heads for 20 rows (71 MB) take 32 us
// from cold caches, 1494 fp16 pages x 8 for 32 rows (98 MB) 35.  It runs before the
// prefix's kernel, whose blocks set themselves up on the SMs that it leaves and then
// wait for its end: with the prefix first a call took up to 5 us longer (64 x 5 rows:
// 182 against 179.5 us, 45 x 5 of INT8_ROW 116.5 against 111).
#pragma once

#include <atomic>

#include "attention_launch.cuh"
#include "shared_prefix.cuh"

namespace pqkv {

template <int KVT, int NT>
struct WarpCfg {
  static constexpr int kW = 8;
  static constexpr int kMinBlocks = private_blocks_per_sm(KVT, NT);
  static constexpr int kThreads = kW * 32;
  static constexpr int kTileBytes = (KVT == PQKV_KV_FP16) ? 8192 : 4096;
  static constexpr int kStages = (KVT == PQKV_KV_FP16 || NT == 1) ? 2 : 4;   // per warp
  static constexpr int kRP = 8 * NT;
  static constexpr bool kRowScaled = (KVT == PQKV_KV_INT8_ROW);
  static constexpr int kQOff = kW * kStages * kTileBytes;
  static constexpr int kQBytes = 4 * NT * 32 * 16;                            // per warp
  static constexpr int kScOff = kQOff + kW * kQBytes;
  static constexpr int kScBytes = kRowScaled ? kW * kStages * 64 : 0;
  static constexpr int kBarOff = kScOff + kScBytes;
  static constexpr int kTabOff = kBarOff + kW * kStages * 8 + 8;
  static __host__ __device__ constexpr int smem_bytes(int n) {
    return kTabOff + (2 * n + 1) * 4 + 1024;
  }
  static_assert(smem_bytes(PQKV_MAX_SEQS) <= 232448, "shared memory of the largest launch");
};

template <int KVT, int NT, class PP = SharedParams>
__global__ void __launch_bounds__(WarpCfg<KVT, NT>::kThreads, WarpCfg<KVT, NT>::kMinBlocks)
    private_kernel(const __grid_constant__ CUtensorMap map, const PP p) {
  using Cfg = WarpCfg<KVT, NT>;
  static_assert(Cfg::kMinBlocks * (Cfg::smem_bytes(PQKV_MAX_SEQS) + 1024) <= 228 * 1024,
                "the blocks that the launch counts on, with the 1 KB that each takes besides");
  constexpr bool kWaitTest = std::is_same<PP, SharedWaitTestParams>::value;
  constexpr uint64_t kLimitNs = kWaitTest ? kTestWaitLimitNs : kWaitLimitNs;
  constexpr int W = Cfg::kW, S = Cfg::kStages, RP = Cfg::kRP;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::kBarOff);
  const int N = p.num_seqs;
  int* pre = reinterpret_cast<int*>(smem + Cfg::kTabOff);   // [N + 1] units before
  int* page0 = pre + N + 1;                                 // [N] first private page
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int H = p.num_kv_heads;

  if (tid < W * S) {
    mbar_init(&bars[tid], 1);
    fence_barrier_init();
  }
  if (tid == 0) prefetch_tensormap(&map);
  grid_dependency_wait();
  grid_dependents_launch();
  for (int i = tid; i <= N; i += Cfg::kThreads) {
    pre[i] = p.plan.spre[i];
    if (i < N) page0[i] = p.plan.page0[i];
  }
  __syncthreads();

  const int64_t U = (int64_t)pre[N] * H;
  const Shares sh(U, p.suf_workers, kPrivateShare);
  const int worker = warp * gridDim.x + blockIdx.x;     // neighbouring shares on different SMs
  if (worker >= sh.n) return;
  int64_t x0 = sh.start(worker);
  const int64_t x1 = sh.start(worker + 1);

  auto sequence_of = [&](int64_t x) {
    int lo = 0, hi = N - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)pre[mid] * H <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
  };
  // unit x: sequence s, kv-head h, page `pg` of its np private ones (or behind them)
  auto unit = [&](int64_t x, int& s, int& h, int& pg, int& np) {
    s = sequence_of(x);
    const int n = pre[s + 1] - pre[s];
    const int64_t off = x - (int64_t)pre[s] * H, seg = Shares::div(off, n);
    h = (int)seg;
    pg = (int)(off - seg * n);
    np = n - kSegmentCost;
  };
  int s0, h0;
  {                                     // the first page
    int pg, np;
    unit(x0, s0, h0, pg, np);
    if (pg >= np) {
      x0 += np + kSegmentCost - pg;
      if (x0 >= x1) return;
      unit(x0, s0, h0, pg, np);
    }
  }
  const int ntot = (int)(x1 - x0);
  uint8_t* ring = smem + warp * S * Cfg::kTileBytes;
  uint64_t* full = bars + warp * S;
  uint16_t* scales = reinterpret_cast<uint16_t*>(smem + Cfg::kScOff) + warp * S * 32;
  uint4* sQ = reinterpret_cast<uint4*>(smem + Cfg::kQOff + warp * Cfg::kQBytes);
  const uint64_t policy = l2_evict_first_policy();
  uint64_t scale_policy = policy;
  if constexpr (Cfg::kRowScaled) scale_policy = l2_evict_last_policy();

  // the page of unit u of the share, and its kv-head: -1 where there is no page
  auto lookup = [&](int u, int& id, int& h) {
    id = 0;
    h = -1;
    if (u >= ntot) return;
    int s, pg, np, hs;
    unit(x0 + u, s, hs, pg, np);
    if (pg >= np) return;
    h = hs;
    id = __ldg(p.block_table + (int64_t)s * p.bt_stride + page0[s] + pg);
    if (id < 0 || (int64_t)id >= p.num_pages) report(p.status, PQKV_DEV_PAGE_RANGE);
  };
  // -- query rows: lane (g, t) holds, of row 8 nt + g, the values that its own
  // fragment-table entries take
  int q_off[NT];                        // of the row, from the sequence's and head's first
  uint32_t q_pos = 0;                   // 4 bits each: query position of rows 8 nt + 2 t + c
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = 8 * nt + g;
    q_off[nt] = r < p.rows ? (r / p.group * p.num_q_heads + r % p.group) * kHeadDim : -1;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int rr = 8 * nt + 2 * t + c;     // (rows behind the last see what the last sees)
      q_pos |= (uint32_t)(min(rr, p.rows - 1) / p.group) << (4 * (2 * nt + c));
    }
  }
  uint4 qv[NT][4];
  auto fetch_q = [&](int s, int h) {
    const uint16_t* src =
        p.q + ((int64_t)s * p.q_len * p.num_q_heads + (int64_t)h * p.group) * kHeadDim;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k2 = 0; k2 < 4; ++k2)
        qv[nt][k2] = q_off[nt] >= 0 ? __ldg(reinterpret_cast<const uint4*>(
                                          src + q_off[nt] + k_dim_base<KVT>(t, 2 * k2)))
                                    : make_uint4(0, 0, 0, 0);
  };
  fetch_q(s0, h0);                      // the first segment's, under the look-ups below
  int cur_id, cur_h, nxt_id, nxt_h, ubase = 0;
  lookup(lane, cur_id, cur_h);
  lookup(32 + lane, nxt_id, nxt_h);
  int issued = 0, consumed = 0, u = 0;
  auto issue_next = [&]() {
    int h = -1, at = 0;
    while (h < 0) {
      if (u >= ntot) return;
      if (u - ubase >= 32) {
        cur_id = nxt_id;
        cur_h = nxt_h;
        ubase += 32;
        lookup(ubase + 32 + lane, nxt_id, nxt_h);
      }
      at = u - ubase;
      h = __shfl_sync(0xffffffffu, cur_h, at);
      u += 1;
    }
    const int id = __shfl_sync(0xffffffffu, cur_id, at);
    bool copy = true;
    if constexpr (kWaitTest)
      copy = worker != p.skip_block || p.skip_part != 2 || issued != p.skip_tile;
    if (copy && lane == 0) {
      const int stage = issued % S;
      const bool id_ok = id >= 0 && (int64_t)id < p.num_pages;
      if constexpr (Cfg::kRowScaled) {
        // as in the attention kernel: the page's row scales on the tile's barrier
        uint16_t* dst = scales + stage * 32;
        if (!id_ok) {
#pragma unroll
          for (int k = 0; k < 4; ++k) reinterpret_cast<uint4*>(dst)[k] = make_uint4(0, 0, 0, 0);
        }
        mbar_arrive_expect_tx(&full[stage], Cfg::kTileBytes + (id_ok ? 64 : 0));
        tma_load_4d(ring + stage * Cfg::kTileBytes, &map, &full[stage], 0, 0, h, id, policy);
        if (id_ok)
          bulk_load(dst,
                    reinterpret_cast<const uint16_t*>(p.k_scale) +
                        ((int64_t)id * p.num_kv_heads + h) * 32,
                    64, &full[stage], scale_policy);
      } else {
        mbar_arrive_expect_tx(&full[stage], Cfg::kTileBytes);
        tma_load_4d(ring + stage * Cfg::kTileBytes, &map, &full[stage], 0, 0, h, id, policy);
      }
    }
    issued += 1;
  };
#pragma unroll 1
  for (int k = 0; k < S; ++k) issue_next();

  QFrags<NT> qf;
  qf.tab = sQ;
  bool dead = false;
  for (int64_t x = x0; x < x1;) {
    int s, h, pg0, np;
    unit(x, s, h, pg0, np);
    const int npg = (int)min((int64_t)(np - pg0), x1 - x);
    const int L = p.plan.len[s], lim_min = L - p.q_len;
    const int key0 = (page0[s] + pg0) * kPageSize;
    // ---- the segment's query rows, in fragment order (a lane's own entries)
    if (x > x0) fetch_q(s, h);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k2 = 0; k2 < 4; ++k2) sQ[(k2 * NT + nt) * 32 + lane] = qv[nt][k2];
    float qk_scale = p.sm_scale_log2;
    if constexpr (KVT != PQKV_KV_FP16 && KVT != PQKV_KV_INT8_ROW) {
      const int hs = p.scale_per_head ? h : 0;
      const float ks = __ldg(p.k_scale + hs), vs = __ldg(p.v_scale + hs);
      if (!(ks > 0.f && ks <= 3.4e38f && vs > 0.f && vs <= 3.4e38f))
        report(p.status, PQKV_DEV_BAD_SCALE);
      qk_scale = ks * p.sm_scale_log2;
    }
    float o[8][NT][4];
    float mref[NT][2], lsum[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        mref[nt][c] = kNoScore;
        lsum[nt][c] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[mt][nt][k] = 0.f;
    }
    __syncwarp();
    for (int j = 0; j < npg; ++j) {
      const int stage = consumed % S;
      if (!dead) {
        bool ok = mbar_wait<kLimitNs>(&full[stage], (consumed / S) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          dead = true;
          if (lane == 0) report(p.status, PQKV_DEV_TIMEOUT);
        }
      }
      if (dead) break;
      const uint8_t* T = ring + stage * Cfg::kTileBytes;
      const int pos0 = key0 + j * kPageSize;
      float sc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) sc[nt][k] = 0.f;
      page_qk<KVT, NT>(T, g, t, lane, qf, sc);
      if constexpr (Cfg::kRowScaled) {
        const float2 ks = __half22float2(
            *reinterpret_cast<const __half2*>(scales + stage * 32 + g * 4));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          sc[nt][0] *= ks.x;
          sc[nt][1] *= ks.x;
          sc[nt][2] *= ks.y;
          sc[nt][3] *= ks.y;
        }
      }
      if (pos0 + kPageSize - 1 > lim_min) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int tok = pos0 + g + ((k & 2) ? 8 : 0);
            const int at = (q_pos >> (4 * (2 * nt + (k & 1)))) & 15;
            if (tok > lim_min + at) sc[nt][k] = -INFINITY;
          }
      }
      // the reference maximum moves only past 2^8 (see attention_impl.cuh)
      bool raise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          raise |= fmaf(fmaxf(sc[nt][c], sc[nt][c + 2]), qk_scale, -mref[nt][c]) > 8.f;
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float m = fmaxf(sc[nt][c], sc[nt][c + 2]);
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
            m *= qk_scale;
            if (m > mref[nt][c] + 8.f) {
              const float f = ex2(mref[nt][c] - m);
              mref[nt][c] = m;
              lsum[nt][c] *= f;
#pragma unroll
              for (int mt = 0; mt < 8; ++mt) {
                o[mt][nt][c] *= f;
                o[mt][nt][c + 2] *= f;
              }
            }
          }
      }
      const bool tail = pos0 + kPageSize > L;
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float pr[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) pr[k] = ex2(fmaf(sc[nt][k], qk_scale, -mref[nt][k & 1]));
        lsum[nt][0] += pr[0] + pr[2];
        lsum[nt][1] += pr[1] + pr[3];
        if constexpr (Cfg::kRowScaled) {
          const float2 vs = __half22float2(
              *reinterpret_cast<const __half2*>(scales + stage * 32 + g * 4 + 2));
          const float v0 = !tail || pos0 + g < L ? vs.x : 0.f;
          const float v8 = !tail || pos0 + g + 8 < L ? vs.y : 0.f;
          pr[0] *= v0;
          pr[1] *= v0;
          pr[2] *= v8;
          pr[3] *= v8;
        }
        pb[nt][0] = movmatrix_trans(pack_half2(pr[0], pr[1]));
        pb[nt][1] = movmatrix_trans(pack_half2(pr[2], pr[3]));
      }
      VMask vm;
      vm.init(t, L - pos0);
      page_pv<KVT, NT>(T, g, t, pb, tail, vm, o, []() {});
      __syncwarp();
      fence_proxy_async_smem();
      consumed += 1;
      issue_next();
    }
    if (dead) break;
    // ---- the fragment's O, m, l
    const int64_t slot = (int64_t)s * H + h + worker;
    float* dst_o = p.suf_o + slot * RP * kHeadDim;
    float* dst_ml = p.suf_ml + slot * 2 * RP;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float l = lsum[nt][c];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const int r = 8 * nt + 2 * t + c;
        if (r >= p.rows) continue;
        if (g == 0) {
          dst_ml[r] = mref[nt][c];
          dst_ml[RP + r] = l;
        }
        float4* d4 = reinterpret_cast<float4*>(dst_o + r * kHeadDim + 16 * g);
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4)
          d4[k4] = make_float4(o[2 * k4][nt][c], o[2 * k4][nt][c + 2], o[2 * k4 + 1][nt][c],
                               o[2 * k4 + 1][nt][c + 2]);
      }
    __syncwarp();
    x += npg + kSegmentCost;            // (behind x1 where the share ends inside)
  }
  // after a wait that ran out: never leave with a copy in flight
  if (dead && lane == 0)
    for (int u = consumed; u < issued; ++u) {
      if constexpr (kWaitTest)
        if (worker == p.skip_block && p.skip_part == 2 && u == p.skip_tile) continue;
      (void)mbar_wait(&full[u % S], (u / S) & 1);
    }
}

template <int KVT, int NT, class PP>
cudaError_t launch_private_t(const PP& p, const CUtensorMap& map, cudaStream_t stream) {
  using Cfg = WarpCfg<KVT, NT>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = opt_in_smem(private_kernel<KVT, NT, PP>,
                                    Cfg::smem_bytes(PQKV_MAX_SEQS), done);
  if (e != cudaSuccess) return e;
  return launch_pdl(private_kernel<KVT, NT, PP>, p.suf_workers / Cfg::kW, Cfg::kThreads,
                    Cfg::smem_bytes(p.num_seqs), stream, map, p);
}

template <int KVT>
cudaError_t launch_private_dtype(const SharedParams& p, const CUtensorMap& map, int nt,
                                     cudaStream_t stream) {
  switch (nt) {
    case 1: return launch_private_t<KVT, 1>(p, map, stream);
    case 2: return launch_private_t<KVT, 2>(p, map, stream);
    case 3: return launch_private_t<KVT, 3>(p, map, stream);
    case 4: return launch_private_t<KVT, 4>(p, map, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pqkv
