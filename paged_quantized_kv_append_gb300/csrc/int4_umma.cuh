// Attention over a 4-bit pool on the fifth-generation tensor cores: the balanced decode,
// verify, sliding-window and partial calls of INT4_GROUP.
//
// With a tile of 128 keys of a (sequence, kv-head) as the products' long side and the
// segment's R = G * q_len query rows (padded to N = 16 or 32) as the short one,
//     S^T = K Q^T   (128 x N x 128, K in TMEM, Q in shared memory, S in TMEM)
//     P^T = 2^(S^T c - m)   (fp16, shared memory)
//     O^T += V^T P^T   (128 dims x N x 128 keys, V and P in shared memory, O in TMEM)
// so a row of the short side costs next to nothing, and the work is what 4 bits need: the
// codes of a tile become 32768 fp16 values (each exact), 11 instructions for eight.
//
// One CTA per SM takes a contiguous share of the tiles of all segments.  Warps: 0-3 the
// softmax (a key per thread), 4-7 and 8-11 widen K and V (a key per thread: K's row goes
// to the thread's TMEM lane, V's to shared memory), 12-15 bring a fragment's query rows
// and write its O, m and l (and merge a segment's partial results, when the CTA is the
// segment's last), 16 and 19 the copies, 17 the products, 18 the fragments of the share.
// Every stage is two deep, the codes five to seven tiles, so a fragment's end overlaps the
// next one.
//
// What bounds it: the instructions around a tile, in two chains.  The 18432 bytes of a tile
// are 780 cycles of an SM's share of the memory; a tile takes 1500 (8 x 131072 keys, 8 heads,
// 20 rows: 343 us, 3.52 TB/s, 52 % of the measured copy; 32 rows 45 %; one row of 16 heads
// 51 %).  K's and V's warps work all of that time: four turns, each of 145 cycles for a group's
// 32 values a thread and 130 to 180 for their store.  And a kernel without any widening still
// took 250 us, 1090 cycles a tile: a tile's scores landed, their load out of TMEM, the vote of
// the four softmax warps, the probabilities' store and V's product follow one another.
// The register split below was measured with 24 rows alone.  It leaves the softmax warps of
// 8 and 16 rows registers to spare, and the 32-row kernels spill 88 to 112 bytes a thread.
// Tried and slower: a second group of warps each for K and V
// (355 us), a second softmax for every other tile (460), waits by one warp of a group and a
// barrier (400), one warp for the scores' products and one for V's (365), K and V in one loop
// (393), and their rows unrolled in full (600): a scheduler's warps run a code each, and
// what does not fit its instruction cache together is fetched again for every tile.
#pragma once

#include "attention_launch.cuh"
#include "tcgen05.cuh"

namespace pqkv {

constexpr int kI4Keys = 128;                    // keys of a tile
constexpr int kI4Pages = kI4Keys / kPageSize;
constexpr int kI4PageBytes = 2 * kInt4Tile;
// A row's reference is raised when a score passes it by more than this (log2), and all rows'
// to their largest scores then: probabilities stay <= 2^15.9, within fp16's 2^16, and the
// largest key's is 1 or more, so each is off by half a step, 2^-11 of it or, under 2^-14,
// 2^-25 of the largest at most.  With 8 a verify of 8 x 131072 took 350 us instead of 343, one
// of 524288 208 instead of 200: a raise costs a tile about 1500 cycles.
constexpr float kI4Raise = 15.9f;

// A fragment of the CTA's share: tiles of one segment.
struct I4Frag {
  int nt;             // tiles; 0: the share is done
  int s, h;           // sequence, kv-head
  int page0, pages;   // first logical page, pages to read
  int L;              // cached tokens of the sequence
  int lim;            // position of query 0: row r sees keys up to lim + r / G
  int seg, cnt;       // segment, its number of partial results
  int first;          // the CTA of its first one
  int slot;           // of this one
  int pad;
};
static_assert(sizeof(I4Frag) == 48, "three 16-byte words");

template <int NT>
struct I4Cfg {
  static constexpr int kThreads = 20 * 32;
  // registers per thread of the launch, and of the softmax, the widening, the queries'
  // and results' and the other warps
  static constexpr int kRegLaunch = 96;
  static constexpr int kRegSoftmax = 160, kRegWiden = 80, kRegOut = 96, kRegOther = 56;
  static_assert(kRegSoftmax + 2 * kRegWiden + kRegOut + kRegOther <= 5 * kRegLaunch,
                "registers of the launch");
  static constexpr int kRP = 8 * NT;                     // rows that are computed
  static constexpr int kN = NT <= 2 ? 16 : 32;           // columns of the products
  static constexpr int kMaxStages = 7;                   // of the codes, as far as they fit
  static constexpr int kSlab = kI4Pages * kI4PageBytes;  // a tile's codes and scales
  static constexpr int kVTile = 2 * 128 * 128;           // two halves: 128 rows of 64 values
  static constexpr int kPTile = 128 * 64;                // 128 rows of up to 32 values
  static constexpr int kQHalf = kN * 128;                // N rows of 64 values
  static constexpr int kFrags = 4;
  static constexpr int kReaders = 19;                    // warps that read fragments
  static constexpr int kVOff = 0;
  static constexpr int kPOff = kVOff + 2 * kVTile;
  static constexpr int kQOff = kPOff + 2 * kPTile;
  static constexpr int kFragOff = kQOff + 2 * 2 * kQHalf;
  static constexpr int kMaxOff = kFragOff + kFrags * (int)sizeof(I4Frag);   // [32][4]
  static constexpr int kMlOff = kMaxOff + 32 * 4 * 4;    // [2][5][32]: m, and l of 4 warps
  static constexpr int kBarOff = kMlOff + 2 * 5 * 32 * 4;
  static constexpr int kBars = 2 * kMaxStages + 2 * kFrags + 23;
  static constexpr int kMiscOff = kBarOff + ((kBars * 8 + 15) & ~15);
  static constexpr int kSlabOff = (kMiscOff + 32 + 127) & ~127;
  // the stages, and behind them three ints a sequence
  static __host__ __device__ constexpr int pre_bytes(int num_seqs) { return (3 * num_seqs + 1) * 4; }
  static __host__ __device__ constexpr int stages(int num_seqs) {
    const int fit = (232448 - kSlabOff - pre_bytes(num_seqs)) / kSlab;
    return fit < kMaxStages ? fit : kMaxStages;
  }
  static __host__ __device__ constexpr int smem_bytes(int num_seqs) {
    return kSlabOff + stages(num_seqs) * kSlab + pre_bytes(num_seqs);
  }
  // (odd numbers too: each of the two copying warps steps over every other stage, and comes to
  // the rest of them when it wraps)
  static_assert(stages(1) == kMaxStages && stages(PQKV_MAX_SEQS) == (kN == 16 ? 6 : 5),
                "shared memory of the smallest and of the largest launch");
  // TMEM columns
  static constexpr uint32_t kTmemK = 0, kTmemS = 128, kTmemO = 192;
  // kind::f16, fp32 D, M 128; S: A and B with their values along K; O: both along M and N
  static constexpr uint32_t kIdescS = (1u << 4) | ((uint32_t)(kN >> 3) << 17) | ((128u >> 4) << 24);
  static constexpr uint32_t kIdescO = kIdescS | (1u << 15) | (1u << 16);
};

__device__ __forceinline__ void tmem_alloc_256(uint32_t* dst) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;" ::"r"(
                   smem_u32(dst))
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free_256(uint32_t base) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(base));
}
__device__ __forceinline__ void tmem_ld8(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(
                   r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tmem_landed8(uint32_t* r) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7])::"memory");
}

__device__ __forceinline__ __half lds_half(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return __ushort_as_half(v);
}

// maximum over the warp
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// P as B: rows of 64 bytes (32 values along N), 64-byte swizzle (a 16-byte chunk's index is
// XORed with row / 2 & 3); the 8-row groups are 512 bytes apart, a k-step of 16 rows 1 KB.
__device__ __forceinline__ uint64_t i4_p_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(512 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(4) << 61);
}

template <int NT, class PP>
__global__ void __launch_bounds__(I4Cfg<NT>::kThreads, 1) int4_umma_kernel(const PP p) {
  using Cfg = I4Cfg<NT>;
  constexpr bool kPartial = IsPartial<PP>::value;
  constexpr bool kWin = IsWindow<PP>::value;
  constexpr bool kWaitTest = IsWaitTest<PP>::value;
  // looks of a wait: each takes some 100 ns, with the nap behind it.  (A look that finds
  // nothing returns at once, and the warps' looks share a unit: without naps they made the
  // satisfied waits cost 280 cycles.)
  constexpr uint32_t kLooks = kWaitTest ? 1u << 13 : 1u << 23;
  constexpr int RP = Cfg::kRP, N = Cfg::kN, F = Cfg::kFrags;
  const uint32_t S = (uint32_t)Cfg::stages(p.num_seqs);
  extern __shared__ __align__(1024) uint8_t smem[];       // the swizzle's atoms are 1 KB
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::kBarOff);
  uint64_t* slab_full = bars;             // [S] a tile's codes have landed
  uint64_t* slab_empty = bars + Cfg::kMaxStages;   // [S] they are in registers
  uint64_t* k_full = bars + 2 * Cfg::kMaxStages;        // [2] K in TMEM
  uint64_t* pv_full = k_full + 2;         // [2] V and the probabilities in shared memory
  uint64_t* s_full = k_full + 4;          // [2] scores in TMEM (K is read)
  uint64_t* pv_done = k_full + 6;         // [2] V and the probabilities are read
  // per fragment, two deep: queries in place, O complete, O read, m and l written, read
  uint64_t* q_full = k_full + 8;
  uint64_t* o_done = k_full + 10;
  uint64_t* o_empty = k_full + 12;
  uint64_t* l_full = k_full + 14;
  uint64_t* l_empty = k_full + 16;
  uint64_t* vote = k_full + 18;           // the softmax warps have said whether to raise
  uint64_t* raised = k_full + 19;         // and their rows' maxima
  uint64_t* written = k_full + 20;        // a partial result is written
  uint64_t* ticket_in = k_full + 21;      // and its ticket drawn
  uint64_t* drain = k_full + 22;
  uint64_t* frag_full = k_full + 23;      // [F]
  uint64_t* frag_empty = frag_full + F;   // [F]
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::kMiscOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::kMiscOff + 4);
  volatile int* merge_flag = reinterpret_cast<volatile int*>(smem + Cfg::kMiscOff + 8);
  volatile uint32_t* raise_at = reinterpret_cast<volatile uint32_t*>(smem + Cfg::kMiscOff + 16);
  I4Frag* frags = reinterpret_cast<I4Frag*>(smem + Cfg::kFragOff);
  float* sMax = reinterpret_cast<float*>(smem + Cfg::kMaxOff);
  float* sMl = reinterpret_cast<float*>(smem + Cfg::kMlOff);
  int* pre = reinterpret_cast<int*>(smem + Cfg::kSlabOff + S * Cfg::kSlab);   // [B + 1] tiles before
  int* slen = pre + p.num_seqs + 1;                          // [B]
  int* sfp = slen + p.num_seqs;                              // [B] first page read (window)

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = p.num_seqs, H = p.num_kv_heads;
  if (tid == 0) {
    for (uint32_t i = 0; i < S; ++i) {
      mbar_init(&slab_full[i], 1);
      mbar_init(&slab_empty[i], 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 4);
      mbar_init(&pv_full[i], 8);
      mbar_init(&s_full[i], 1);
      mbar_init(&pv_done[i], 1);
      mbar_init(&q_full[i], 4);
      mbar_init(&o_done[i], 1);
      mbar_init(&o_empty[i], 4);
      mbar_init(&l_full[i], 4);
      mbar_init(&l_empty[i], 4);
    }
    for (int i = 0; i < F; ++i) {
      mbar_init(&frag_full[i], 1);
      mbar_init(&frag_empty[i], Cfg::kReaders);
    }
    mbar_init(vote, 4);
    mbar_init(raised, 4);
    mbar_init(written, 4);
    mbar_init(ticket_in, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    raise_at[0] = raise_at[1] = 0;
    fence_barrier_init();
    pre[0] = 0;
  }
  if (warp == 17) tmem_alloc_256(tmem_slot);
  // columns of P behind the computed rows stay 0
  for (int i = tid; i < 2 * Cfg::kPTile / 16; i += Cfg::kThreads)
    reinterpret_cast<uint4*>(smem + Cfg::kPOff)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  grid_dependency_wait();
  grid_dependents_launch();
  // -- per-sequence lengths, clamped into their rows, and tiles
  for (int s = tid; s < B; s += Cfg::kThreads) {
    int L = p.seq_lens[s];
    const int Lmax = p.bt_stride * kPageSize, Lmin = kPartial ? 0 : p.q_len;
    if (L < Lmin || L > Lmax) {
      if (blockIdx.x == 0) report(p.status, PQKV_DEV_SEQ_RANGE);
      L = max(Lmin, min(L, Lmax));
    }
    slen[s] = L;
    int np = (L + kPageSize - 1) / kPageSize;
    if constexpr (kWin) {
      const int fp = max(0, L - p.q_len - p.window + 1) / kPageSize;
      sfp[s] = fp;
      np -= fp;
    }
    pre[s + 1] = (np + kI4Pages - 1) / kI4Pages;
  }
  __syncthreads();
  if (warp == 0) {
    int run = 0;
    for (int base = 0; base < B; base += 32) {
      int v = base + lane < B ? pre[base + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      if (base + lane < B) pre[base + lane + 1] = run + v;
      run += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  if constexpr (kPartial) {
    // rows of sequences with no local keys: O = 0, LSE = -inf
    for (int s = blockIdx.x; s < B; s += gridDim.x) {
      if (slen[s] != 0) continue;
      const int64_t r0 = (int64_t)s * p.q_len * p.num_q_heads;
      const int nr = p.q_len * p.num_q_heads;
      for (int i = tid; i < nr * kHeadDim; i += Cfg::kThreads) p.out_o[r0 * kHeadDim + i] = 0.f;
      for (int i = tid; i < nr; i += Cfg::kThreads) p.out_lse[r0 + i] = -INFINITY;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  // Bounded wait (about a second of looks; the kernel's end reports it): when one runs out the
  // whole CTA stops at its next waits.  Called by whole warps; every lane gets the same answer.
  auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t nap = 20) -> bool {
#pragma unroll 1
    for (uint32_t n = kLooks; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity)); --n) {
      if (n == 0) *abort_flag = 1;
      if (*abort_flag) return false;
      __nanosleep(nap);
    }
    return true;
  };
  auto frag_at = [&](uint32_t n, I4Frag& f) -> bool {
    if (!wait(&frag_full[n % F], (n / F) & 1)) return false;
    const uint4* src = reinterpret_cast<const uint4*>(frags + n % F);
    uint4* dst = reinterpret_cast<uint4*>(&f);
#pragma unroll
    for (int i = 0; i < 3; ++i) dst[i] = src[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(&frag_empty[n % F]);
    f.nt = __shfl_sync(0xffffffffu, f.nt, 0);      // (warp-uniform to the compiler)
    return f.nt > 0;
  };
  const int key = tid & 127;                 // of a tile, where threads have one

  if (warp < 4) {
    // ================= softmax: a key per thread =================
    regs_up<Cfg::kRegSoftmax>();
    const uint32_t lane_sel = (uint32_t)(warp * 32) << 16;
    const float c = p.sm_scale_log2;
    uint32_t tl = 0;                                     // tiles so far
    uint32_t raises = 0;
    // the rows' query positions, 4 bits each (rows behind the last see what it sees)
    uint32_t q_pos[NT];
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      q_pos[k] = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        q_pos[k] |= (uint32_t)(min(8 * k + j, p.rows - 1) / p.group) << (4 * j);
    }
    I4Frag f;
    bool ok = true;
    for (uint32_t n = 0; ok && frag_at(n, f); ++n) {
      float ref[RP], l[RP];
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        ref[r] = kNoScore;
        l[r] = 0.f;
      }
#pragma unroll 1
      for (int i = 0; i < f.nt; ++i, ++tl) {
        const uint32_t b = tl & 1, par = (tl >> 1) & 1;
        if (!(ok = wait(&s_full[b], par))) break;
        tc_fence_after();
        uint32_t x[RP];
        const uint32_t tS = tmem + lane_sel + Cfg::kTmemS + b * 32;
#pragma unroll
        for (int k = 0; k < RP; k += 8) tmem_ld8(tS + k, x + k);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < RP; k += 8) tmem_landed8(x + k);
        const int pos0 = (f.page0 + i * kI4Pages) * kPageSize, pos = pos0 + key;
        if (pos0 + kI4Keys - 1 > min(f.lim, f.L - 1)) {
#pragma unroll
          for (int r = 0; r < RP; ++r)
            if (pos >= f.L || pos > f.lim + (int)((q_pos[r / 8] >> (4 * (r & 7))) & 15))
              x[r] = 0xff800000u;
        }
        if constexpr (kWin) {
          if (pos0 <= f.lim + p.q_len - 1 - p.window) {
#pragma unroll
            for (int r = 0; r < RP; ++r)
              if (pos <= f.lim + (int)((q_pos[r / 8] >> (4 * (r & 7))) & 15) - p.window)
                x[r] = 0xff800000u;
          }
        }
        // (the largest exponent as it is formed below: no probability can be more)
        float top[4] = {kNoScore, kNoScore, kNoScore, kNoScore};
#pragma unroll
        for (int r = 0; r < RP; r += 2) {
          const float a = fmaf(__uint_as_float(x[r]), c, -ref[r]);
          const float d = fmaf(__uint_as_float(x[r + 1]), c, -ref[r + 1]);
          top[(r >> 1) & 3] = max3(top[(r >> 1) & 3], a, d);
        }
        const bool raise = fmaxf(max3(top[0], top[1], top[2]), top[3]) > kI4Raise;
        // The warps agree: the note of a tile is its number + 1 (a buffer's older notes are
        // smaller, and its next one comes after a vote that this warp is still to cast).
        // The probabilities are formed under the vote, and again if it raises.
        if (__any_sync(0xffffffffu, raise) && lane == 0) raise_at[b] = tl + 1;
        __syncwarp();
        if (lane == 0) mbar_arrive(vote);
        float pr[RP];
#pragma unroll
        for (int r = 0; r < RP; ++r) pr[r] = ex2(fmaf(__uint_as_float(x[r]), c, -ref[r]));
        if (!(ok = wait(vote, tl & 1))) break;
        if (__builtin_expect(raise_at[b] == tl + 1, 0)) {
          // every row's reference to its largest score so far; O follows
#pragma unroll
          for (int r = 0; r < RP; ++r) {
            const float m = warp_max(__uint_as_float(x[r]));
            if (lane == 0) sMax[r * 4 + warp] = m;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(raised);
          if (!(ok = wait(raised, raises & 1))) break;
          raises += 1;
          float fct[RP];
#pragma unroll
          for (int r = 0; r < RP; ++r) {
            const float4 m = *reinterpret_cast<const float4*>(sMax + r * 4);
            const float nref = fmaxf(ref[r], fmaxf(fmaxf(m.x, m.y), fmaxf(m.z, m.w)) * c);
            fct[r] = ex2(ref[r] - nref);
            ref[r] = nref;
            l[r] *= fct[r];
            pr[r] = ex2(fmaf(__uint_as_float(x[r]), c, -nref));
          }
          if (i > 0) {
            // O is still when the last product with V is done
            if (!(ok = wait(&pv_done[b ^ 1], ((tl - 1) >> 1) & 1))) break;
            tc_fence_after();
            const uint32_t tO = tmem + lane_sel + Cfg::kTmemO + (n & 1) * 32;
#pragma unroll
            for (int k = 0; k < RP; k += 8) {
              uint32_t o[8];
              tmem_ld8(tO + k, o);
              tmem_wait_ld();
              tmem_landed8(o);
#pragma unroll
              for (int j = 0; j < 8; ++j)
                o[j] = __float_as_uint(__uint_as_float(o[j]) * fct[k + j]);
              tmem_st8(tO + k, o);
            }
            tmem_wait_st();
            tc_fence_before();
          }
        }
        uint32_t ph[RP / 2];
#pragma unroll
        for (int r = 0; r < RP; r += 2) {
          l[r] += pr[r];
          l[r + 1] += pr[r + 1];
          ph[r / 2] = pack_half2(pr[r], pr[r + 1]);
        }
        // (P's buffer was last read for tile tl - 2, before this tile's scores were formed)
        const uint32_t dst = sbase + Cfg::kPOff + b * Cfg::kPTile + key * 64;
#pragma unroll
        for (int k = 0; k < NT; ++k)
          sts128(dst + ((k ^ ((key >> 1) & 3)) << 4), ph[4 * k], ph[4 * k + 1], ph[4 * k + 2],
                 ph[4 * k + 3]);
        fence_proxy_async_smem();
        tc_fence_before();               // the scores are read, too
        __syncwarp();
        if (lane == 0) mbar_arrive(&pv_full[b]);
      }
      if (!ok) break;
      // ---- m and l of the fragment
      if (n >= 2 && !(ok = wait(&l_empty[n & 1], (n / 2 + 1) & 1))) break;
      float* ml = sMl + (n & 1) * 5 * 32;
#pragma unroll
      for (int g = 0; g < NT; ++g) {
        // eight rows' sums over the lanes: each exchange halves the rows a lane holds
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = l[8 * g + k];
#pragma unroll
        for (int o = 16, w = 4; w > 0; o >>= 1, w >>= 1) {
          const bool up = lane & o;
#pragma unroll
          for (int k = 0; k < w; ++k) {
            const float send = up ? v[k] : v[k + w], keep = up ? v[k + w] : v[k];
            v[k] = keep + __shfl_xor_sync(0xffffffffu, send, o);
          }
        }
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
        if ((lane & 3) == 0)
          ml[(1 + warp) * 32 + 8 * g + ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 +
             ((lane >> 2) & 1)] = v[0];
        if (warp == 0 && lane < 8) {
          float m = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (lane == k) m = ref[8 * g + k];
          ml[8 * g + lane] = m;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&l_full[n & 1]);
    }
  } else if (warp < 12) {
    // ================= widen the codes of K, and of V =================
    regs_down<Cfg::kRegWiden>();
    const int kv = warp >= 8;
    // the thread's row of a tile's slab: chunk of its group 0, scale of its group 0
    const int line = (key & 15) >> 1;
    const uint32_t row = sbase + Cfg::kSlabOff + (key >> 4) * kI4PageBytes + kv * kInt4Tile;
    const uint32_t chunk0 =
        row + line * 128 + ((((key & 1) * 4) ^ (((line & 1) * 5) ^ (line & 2))) << 4);
    const uint32_t scale0 = row + kInt4Codes + (key & 15) * 2;
    const uint32_t to_k = tmem + ((uint32_t)((warp & 3) * 32) << 16) + Cfg::kTmemK;
    const uint32_t to_v = sbase + Cfg::kVOff + key * 128 + ((key & 7) << 4);
    uint32_t tl = 0, stage = 0, phase = 0;
    I4Frag f;
    bool ok = true;
    for (uint32_t n = 0; ok && frag_at(n, f); ++n) {
      int pos = f.page0 * kPageSize + key;
#pragma unroll 1
      for (int i = 0; i < f.nt; ++i, ++tl, pos += kI4Keys) {
        const uint32_t b = tl & 1;
        // the codes have landed, and the buffer is free: a barrier per lane
        const bool second = (lane & 1) && tl >= 2;
        if (!(ok = wait(second ? (kv ? pv_done : s_full) + b : slab_full + stage,
                         (second ? (tl >> 1) + 1 : phase) & 1)))
          break;
        const uint32_t from = stage * Cfg::kSlab;
        const uint32_t at = chunk0 + from, scale = scale0 + from;
        // tokens behind the end may be anything, and 0 times V has to be 0 there: a scale
        // of 0 makes it so (K's scores are masked)
        const bool live = kv == 0 || pos < f.L;
        // the thread's TMEM lane, or chunk 0 of its 128-byte row of V's first half (chunk k
        // is at `^ 16 k`)
        const uint32_t to = kv == 0 ? to_k + b * 64 : to_v + b * Cfg::kVTile;
        tc_fence_after();
        // A group a turn, the next one's codes read ahead (the last turn's are not used).  The
        // slab may be filled again when the turns are done: what its loads brought has been
        // used.
        if (kv == 0) {
          uint4 x = lds128u(at);
          __half sc = lds_half(scale);
#pragma unroll 2
          for (int g = 0; g < 4; ++g) {
            const Int4Scale s(__half2half2(sc));
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            x = lds128u(at ^ ((g + 1) << 4 & 48));
            sc = lds_half(scale + ((g + 1) & 3) * 2 * kPageSize);
            uint32_t o[16];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t v[4];
              int4_word(w[k], s, v);
#pragma unroll
              for (int j = 0; j < 4; ++j) o[4 * k + j] = v[j];
            }
            tmem_st16(to + g * 16, o);
          }
          tmem_wait_st();
          tc_fence_before();
        } else {
          uint4 x = lds128u(at);
          __half sc = lds_half(scale);
#pragma unroll 2
          for (int g = 0; g < 4; ++g) {
            const Int4Scale s(__half2half2(live ? sc : __ushort_as_half(0)));
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            x = lds128u(at ^ ((g + 1) << 4 & 48));
            sc = lds_half(scale + ((g + 1) & 3) * 2 * kPageSize);
            uint32_t o[16];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t v[4];
              int4_word(w[k], s, v);
#pragma unroll
              for (int j = 0; j < 4; ++j) o[4 * k + j] = v[j];
            }
            const uint32_t half = (to + (g >> 1) * 16384) ^ ((g & 1) << 6);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              sts128(half ^ (k << 4), o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive((kv ? pv_full : k_full) + b);
          mbar_arrive(&slab_empty[stage]);
        }
        if (++stage == S) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp < 16) {
    // ================= query rows in, O out =================
    static_assert(Cfg::kRegOut == Cfg::kRegLaunch, "these warps keep theirs");
    const int wq = warp & 3, t = tid & 127;              // t: the thread's dim of O^T
    const uint32_t lane_sel = (uint32_t)(wq * 32) << 16;
    auto load_q = [&](const I4Frag& f, uint32_t n) {
      // row r, 16-byte chunk cc of its 16; rows behind the last are zeros
      for (int i = t; i < N * 16; i += 128) {
        const int r = i >> 4, cc = i & 15;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < p.rows) {
          const int64_t row = ((int64_t)f.s * p.q_len + r / p.group) * p.num_q_heads +
                              f.h * p.group + r % p.group;
          v = __ldg(reinterpret_cast<const uint4*>(p.q + row * kHeadDim) + cc);
        }
        sts128(sbase + Cfg::kQOff + (n & 1) * 2 * Cfg::kQHalf + (cc >> 3) * Cfg::kQHalf + r * 128 +
                   (((cc & 7) ^ (r & 7)) << 4),
               v.x, v.y, v.z, v.w);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[n & 1]);
    };
    I4Frag cur, nxt;
    bool have = frag_at(0, cur);
    bool ok = true;
    uint32_t tickets = 0;
    if (have) load_q(cur, 0);
    for (uint32_t n = 0; have; ++n) {
      // the next fragment's rows: their buffer was last read by the scores of fragment
      // n - 1, whose O is done
      const bool more = frag_at(n + 1, nxt);
      if (more) load_q(nxt, n + 1);
      if (!(ok = wait(&l_full[n & 1], (n / 2) & 1, 100))) break;
      if (!(ok = wait(&o_done[n & 1], (n / 2) & 1))) break;
      tc_fence_after();
      uint32_t o[RP];
      const uint32_t tO = tmem + lane_sel + Cfg::kTmemO + (n & 1) * 32;
#pragma unroll
      for (int k = 0; k < RP; k += 8) tmem_ld8(tO + k, o + k);
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < RP; k += 8) tmem_landed8(o + k);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_empty[n & 1]);
      const float* ml = sMl + (n & 1) * 5 * 32;
      const int64_t out_row0 = (int64_t)cur.s * p.q_len;
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        if (r >= p.rows) continue;
        const float l = (ml[32 + r] + ml[64 + r]) + (ml[96 + r] + ml[128 + r]);
        const float val = __uint_as_float(o[r]);
        if (cur.cnt == 1) {
          const int64_t orow =
              (out_row0 + r / p.group) * p.num_q_heads + cur.h * p.group + r % p.group;
          const float res = l == 0.f ? 0.f : val / l;
          if constexpr (kPartial) {
            p.out_o[orow * kHeadDim + t] = res;
            if (t == 0) p.out_lse[orow] = row_lse(ml[r], l);
          } else {
            p.out[orow * kHeadDim + t] = __half_as_ushort(__float2half_rn(res));
          }
        } else {
          p.part_o[((size_t)cur.slot * RP + r) * kHeadDim + t] = val;
          if (t == 0) {
            p.part_ml[(size_t)cur.slot * 2 * RP + r] = ml[r];
            p.part_ml[(size_t)cur.slot * 2 * RP + RP + r] = l;
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&l_empty[n & 1]);
      if (cur.cnt > 1) {
        // the segment's last CTA (an acquire-release ticket) merges its partial results
        __syncwarp();
        if (lane == 0) mbar_arrive(written);
        if (wq == 0) {
          if (!(ok = wait(written, tickets & 1))) break;
          if (lane == 0) {
            int ticket;
            asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                         : "=r"(ticket)
                         : "l"(p.counters + cur.seg)
                         : "memory");
            *merge_flag = ticket == cur.cnt - 1;
            mbar_arrive(ticket_in);
          }
          __syncwarp();
        }
        if (!(ok = wait(ticket_in, tickets & 1))) break;
        tickets += 1;
        if (*merge_flag) {
          // in the order of the CTAs: eight results a step, folded with a running rescale
          const int first = cur.first;
          for (int it = t; it < p.rows * 32; it += 128) {
            const int r = it >> 5, dq = it & 31;
            float M = kNoScore, l = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int q0 = 0; q0 < cur.cnt; q0 += 8) {
              float mq[8], lq[8];
              float4 vq[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const bool in = q0 + k < cur.cnt;
                const size_t sl = cur.seg + first + (in ? q0 + k : 0);
                mq[k] = in ? __ldcg(p.part_ml + sl * 2 * RP + r) : kNoScore;
                lq[k] = in ? __ldcg(p.part_ml + sl * 2 * RP + RP + r) : 0.f;
                vq[k] = in ? __ldcg(reinterpret_cast<const float4*>(
                                        p.part_o + (sl * RP + r) * kHeadDim) + dq)
                           : make_float4(0.f, 0.f, 0.f, 0.f);
              }
              float Mn = M;
#pragma unroll
              for (int k = 0; k < 8; ++k) Mn = fmaxf(Mn, mq[k]);
              const float fc = ex2(M - Mn);
              l *= fc;
              acc.x *= fc;
              acc.y *= fc;
              acc.z *= fc;
              acc.w *= fc;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float wk = ex2(mq[k] - Mn);
                l += wk * lq[k];
                acc.x += wk * vq[k].x;
                acc.y += wk * vq[k].y;
                acc.z += wk * vq[k].z;
                acc.w += wk * vq[k].w;
              }
              M = Mn;
            }
            const float inv = row_inv(l, 1.f);
            const int64_t orow =
                (out_row0 + r / p.group) * p.num_q_heads + cur.h * p.group + r % p.group;
            if constexpr (kPartial) {
              *reinterpret_cast<float4*>(p.out_o + orow * kHeadDim + 4 * dq) =
                  make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
              if (dq == 0) p.out_lse[orow] = row_lse(M, l);
            } else {
              uint2 pk;
              pk.x = pack_half2(acc.x * inv, acc.y * inv);
              pk.y = pack_half2(acc.z * inv, acc.w * inv);
              *reinterpret_cast<uint2*>(p.out + orow * kHeadDim + 4 * dq) = pk;
            }
          }
          if (t == 0) p.counters[cur.seg] = 0;
        }
      }
      cur = nxt;
      have = more;
    }
  } else {
  regs_down<Cfg::kRegOther>();
  if (warp == 16 || warp == 19) {
    // ================= copies: of the even and of the odd tiles =================
    const uint64_t policy = l2_evict_first_policy();
    const uint8_t* pool = reinterpret_cast<const uint8_t*>(p.k_scale);
    const int64_t page_bytes = (int64_t)H * kI4PageBytes;
    const uint32_t turn = warp == 19;
    uint32_t tl = 0, stage = turn, phase = 0;
    I4Frag f;
    bool ok = true;
    for (uint32_t n = 0; ok && frag_at(n, f); ++n) {
      const int32_t* row = p.block_table + (int64_t)f.s * p.bt_stride + f.page0;
      const uint8_t* src = pool + (int64_t)f.h * kI4PageBytes;
      // lane = page of the warp's next four tiles (every other one), looked up four ahead;
      // -2: no page
      auto lookup = [&](int i) -> int {
        const int pg = (i + 2 * (lane >> 3)) * kI4Pages + (lane & 7);
        if (pg >= f.pages) return -2;
        const int id = __ldg(row + pg);
        if (id < 0 || (int64_t)id >= p.num_pages) {
          report(p.status, PQKV_DEV_PAGE_RANGE);
          return -1;
        }
        return id;
      };
      int i = (int)((turn ^ tl) & 1);
      int ids = lookup(i), next = lookup(i + 8);
      int at = 0;                                            // the tile's first lane
#pragma unroll 1
      for (; i < f.nt; i += 2) {
        if (at == 32) {
          at = 0;
          ids = next;
          next = lookup(i + 8);
        }
        const uint32_t me = tl + i;
        if (me >= S && !(ok = wait(&slab_empty[stage], phase ^ 1, 40))) break;
        uint8_t* dst = smem + Cfg::kSlabOff + stage * Cfg::kSlab;
        const uint32_t bad = (__ballot_sync(0xffffffffu, ids < 0) >> at) & 0xFFu;
        bool copy = true;
        if constexpr (kWaitTest)
          copy = (int)blockIdx.x != p.skip_block || (int)me != p.skip_page;
        if (copy && bad == 0) {
          int id[kI4Pages];
#pragma unroll
          for (int k = 0; k < kI4Pages; ++k) id[k] = __shfl_sync(0xffffffffu, ids, at + k);
          // (issued by one elected thread: by eight lanes, a copy took 110 cycles)
          if (elect_one()) {
            mbar_arrive_expect_tx(&slab_full[stage], Cfg::kSlab);
#pragma unroll
            for (int k = 0; k < kI4Pages; ++k)
              bulk_load(dst + k * kI4PageBytes, src + id[k] * page_bytes, kI4PageBytes,
                        &slab_full[stage], policy);
          }
        } else if (copy) {
          // a segment's last tile, or pages outside the pool, which read as zeros
          const int here = min(kI4Pages, f.pages - i * kI4Pages);
#pragma unroll 1
          for (int k = 0; k < here; ++k)
            for (int z = lane; (bad >> k & 1) && z < kI4PageBytes / 16; z += 32)
              reinterpret_cast<uint4*>(dst + k * kI4PageBytes)[z] = make_uint4(0, 0, 0, 0);
          __syncwarp();
          const uint32_t good = ~bad & ((1u << here) - 1);
          if (lane == 0) mbar_arrive_expect_tx(&slab_full[stage], __popc(good) * kI4PageBytes);
          __syncwarp();
#pragma unroll 1
          for (int k = 0; k < here; ++k) {
            const int id = __shfl_sync(0xffffffffu, ids, at + k);
            if (lane == 0 && (good >> k & 1))
              bulk_load(dst + k * kI4PageBytes, src + id * page_bytes, kI4PageBytes,
                        &slab_full[stage], policy);
          }
        }
        __syncwarp();
        at += kI4Pages;
        stage += 2;
        if (stage >= S) {
          stage -= S;
          phase ^= 1;
        }
      }
      tl += ok ? f.nt : i;
    }
    // no copy may be in flight when the CTA ends, after a wait that ran out either
    if (lane == 0)
      for (uint32_t k = tl > S ? tl - S : 0; k < tl; ++k) {
        if ((k & 1) != turn) continue;
        if constexpr (kWaitTest)
          if ((int)blockIdx.x == p.skip_block && (int)k == p.skip_page) continue;
        (void)mbar_wait(&slab_full[k % S], (k / S) & 1);
      }
  } else if (warp == 17) {
    // ================= products =================
    uint32_t tl = 0;
    I4Frag f;
    bool ok = true;
    const uint64_t q_desc = tc_desc(sbase + Cfg::kQOff, 16),
                   v_desc = tc_desc(sbase + Cfg::kVOff, 16384),
                   p_desc = i4_p_desc(sbase + Cfg::kPOff);
    // O^T += V^T P^T on tile `at`; acc: not the fragment's first; last: its last
    auto pv = [&](uint32_t at, uint32_t n, bool acc, bool last) -> bool {
      const uint32_t b = at & 1, par = (at >> 1) & 1;
      if (!acc && n >= 2 && !wait(&o_empty[n & 1], (n / 2 + 1) & 1)) return false;
      if (!wait(&pv_full[b], par)) return false;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t va = v_desc + (uint64_t)(b * (Cfg::kVTile >> 4)),
                       pb = p_desc + (uint64_t)(b * (Cfg::kPTile >> 4));
#pragma unroll
        for (int k = 0; k < 8; ++k)
          tc_mma_ss(tmem + Cfg::kTmemO + (n & 1) * 32, va + k * 128, pb + k * 64, Cfg::kIdescO,
                    acc || k > 0);
        tc_commit(&pv_done[b]);
        if (last) tc_commit(&o_done[n & 1]);
      }
      __syncwarp();
      return true;
    };
    // a tile's scores are issued before the product with V of the tile before it
    bool pend = false, pend_acc = false, pend_last = false;
    uint32_t pend_n = 0;
    for (uint32_t n = 0; ok && frag_at(n, f); ++n) {
      if (!(ok = wait(&q_full[n & 1], (n / 2) & 1))) break;
      const int nt = f.nt;
#pragma unroll 1
      for (int i = 0; i < nt; ++i, ++tl) {
        const uint32_t b = tl & 1, par = (tl >> 1) & 1;
        // (the scores of tile tl - 2 are read: their probabilities' product is issued)
        if (!(ok = wait(&k_full[b], par))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t q = q_desc + (uint64_t)((n & 1) * (2 * Cfg::kQHalf >> 4));
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tc_mma_ts(tmem + Cfg::kTmemS + b * 32, tmem + Cfg::kTmemK + b * 64 + 8 * k,
                      q + (uint64_t)(((k >> 2) * Cfg::kQHalf + (k & 3) * 32) >> 4), Cfg::kIdescS,
                      k > 0);
          tc_commit(&s_full[b]);
        }
        __syncwarp();
        if (pend && !(ok = pv(tl - 1, pend_n, pend_acc, pend_last))) break;
        pend = true;
        pend_n = n;
        pend_acc = i > 0;
        pend_last = i + 1 == nt;
      }
    }
    if (ok && pend) (void)pv(tl - 1, pend_n, pend_acc, pend_last);
    // products in flight end before the TMEM is freed, after a wait that ran out too
    if (elect_one()) tc_commit(drain);
    (void)mbar_wait(drain, 0);
  } else if (warp == 18) {
    // ================= the share's fragments =================
    if (lane == 0) {
      SplitT<false> sp;
      sp.pre = pre;
      sp.B = B;
      sp.H = H;
      sp.P = (int64_t)pre[B] * H;
      // (no empty shares: a segment's partial results are those of neighbouring CTAs)
      sp.C = (int)min((int64_t)gridDim.x, sp.P);
      sp.k = 0;
      // units [x, e) of the share, and the first one's sequence (by halving: a walk over the
      // sequences before it, and divisions in 64 bits, took 4 us of a call for 256 sequences)
      const auto div = [](int64_t n, int64_t d) { return SplitT<false>::udiv(n, d); };
      int64_t x = 0, e = 0;
      int s = 0;
      if ((int)blockIdx.x < sp.C) {
        x = div((int64_t)blockIdx.x * sp.P, sp.C);
        e = div((int64_t)(blockIdx.x + 1) * sp.P, sp.C);
        for (int hi = B - 1; s < hi;) {
          const int mid = (s + hi) >> 1;
          if ((int64_t)pre[mid + 1] * H > x) hi = mid; else s = mid + 1;
        }
      }
      for (uint32_t n = 0;; ++n) {
        I4Frag f = {};
        if (x < e) {
          while ((int64_t)pre[s + 1] * H <= x) ++s;
          const int np = pre[s + 1] - pre[s];
          const int64_t base = (int64_t)pre[s] * H;
          f.s = s;
          f.h = (int)div(x - base, np);
          f.seg = s * H + f.h;
          const int64_t seg_a = base + (int64_t)f.h * np, seg_b = seg_a + np;
          const int t0 = (int)(x - seg_a);
          f.nt = (int)(min(e, seg_b) - x);
          x += f.nt;
          f.L = slen[s];
          const int fp = kWin ? sfp[s] : 0;
          f.page0 = fp + t0 * kI4Pages;
          f.pages = min((f.L + kPageSize - 1) / kPageSize, fp + (t0 + f.nt) * kI4Pages) - f.page0;
          // (bounded, so that positions may be added to it)
          if constexpr (kPartial) f.lim = max(-(1 << 30), min(p.q_pos[s], 1 << 30));
          else f.lim = f.L - p.q_len;
          f.cnt = sp.count_fast(f.seg, seg_a, seg_b, f.first);
          f.slot = f.seg + (int)blockIdx.x;
        }
        if (n >= F) {
          bool there;
          uint32_t looks = kLooks;
          while (!(there = mbar_try_wait(&frag_empty[n % F], (n / F + 1) & 1)) && looks-- > 0 &&
                 !*abort_flag)
            __nanosleep(200);
          if (!there) break;
        }
        frags[n % F] = f;
        mbar_arrive(&frag_full[n % F]);
        if (f.nt == 0) break;
      }
    }
    __syncwarp();
  }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && *abort_flag) report(p.status, PQKV_DEV_TIMEOUT);
  if (warp == 17) tmem_free_256(tmem);
}

template <int NT, class PP>
cudaError_t launch_int4_umma_t(const PP& p, int grid, cudaStream_t stream) {
  using Cfg = I4Cfg<NT>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e =
      opt_in_smem(int4_umma_kernel<NT, PP>, 232448, done);
  if (e != cudaSuccess) return e;
  // the register split counts on the registers that the launch bounds allow; a build that
  // used fewer would wait for them forever
  static const int regs = [] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, int4_umma_kernel<NT, PP>) == cudaSuccess ? at.numRegs : 0;
  }();
  if (regs < Cfg::kRegLaunch) return cudaErrorLaunchOutOfResources;
  return launch_pdl(int4_umma_kernel<NT, PP>, grid, Cfg::kThreads, Cfg::smem_bytes(p.num_seqs),
                    stream, p);
}

template <class PP>
cudaError_t launch_int4_umma(const PP& p, int grid, int nt, cudaStream_t stream) {
  switch (nt) {
    case 1: return launch_int4_umma_t<1>(p, grid, stream);
    case 2: return launch_int4_umma_t<2>(p, grid, stream);
    case 3: return launch_int4_umma_t<3>(p, grid, stream);
    case 4: return launch_int4_umma_t<4>(p, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pqkv
