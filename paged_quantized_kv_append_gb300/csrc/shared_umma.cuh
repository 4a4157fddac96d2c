// The shared prefix on the fifth-generation tensor cores: all the rows of a
// group's kv-head against the prefix's keys.
//
// One CTA per SM works on a contiguous share of (row tile, key tile) pairs of
// 256 rows and 128 keys.  With X = the tile's rows as A and the keys as B,
//     S = Q K^T   (128 x 128 x 128, A and B in shared memory, S in TMEM)
//     P = 2^(S c - m)   (fp16, over S's own TMEM columns)
//     O += P V    (128 x 128 x 128, A in TMEM, B in shared memory, O in TMEM)
// Two streams of 128 rows take turns on the tensor cores, so that one's softmax
// runs under the other's products: the two halves of a 256-row tile, or, where
// a tile has at most 128 rows, the even and the odd key tiles of the same rows
// (two partial results, joined by the merge like any others).
//
// Warps: 0-3 and 4-7 the softmax of stream 0 and 1 (a thread per row), 8-11
// widen the 8-bit codes to fp16 (exact; TMA writes the fp16 pool's rows into
// place itself), 12 issues the copies, 13 and 14 the products of a stream each.
//
// The running maximum of a row is only raised when a score passes it by more
// than 8 (probabilities stay <= 2^8 in fp16), so O is rescaled rarely, by the
// softmax warps themselves, between two products of their stream.
#pragma once

#include "shared_private.cuh"

namespace pqkv {

// ---------------------------------------------------------------------------
// tcgen05
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc_512(uint32_t* dst) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                   smem_u32(dst))
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}

__device__ __forceinline__ void tmem_free_512(uint32_t base) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(base));
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// the barrier completes its phase's arrival when the products issued so far are done
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}

// D (TMEM) = A (shared) B (shared) + (acc ? D : 0)
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}

// D (TMEM) = A (TMEM) B (shared) + (acc ? D : 0)
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}

// True in one thread of a converged warp.  The products are issued under it from
// warp-uniform control flow: their operands then stay in uniform registers
// (issued by a lane of a divergent branch, an instruction cost about 100 cycles,
// more than the 64 that its product takes).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}"
               : "=r"(p));
  return p != 0;
}

#define PQKV_R32(F) \
  F(0), F(1), F(2), F(3), F(4), F(5), F(6), F(7), F(8), F(9), F(10), F(11), F(12), F(13), F(14), \
      F(15), F(16), F(17), F(18), F(19), F(20), F(21), F(22), F(23), F(24), F(25), F(26), F(27), \
      F(28), F(29), F(30), F(31)

// 32 columns of the thread's TMEM row into (from) registers
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
#define PQKV_OUT(i) "=r"(r[i])
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
      "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : PQKV_R32(PQKV_OUT)
      : "r"(addr)
      : "memory");
#undef PQKV_OUT
}

__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
#define PQKV_IN(i) "r"(r[i])
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
      "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::PQKV_R32(PQKV_IN),
      "r"(addr)
      : "memory");
#undef PQKV_IN
}

__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// 16 columns, for the rare rescale of O beside a row of scores in registers
__device__ __forceinline__ void tmem_ld16_wait(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
// The loads are asynchronous: after the wait, mark the registers as written
// here, so that nothing that reads them is scheduled before it.
__device__ __forceinline__ void tmem_landed32(uint32_t* r) {
#define PQKV_IO(i) "+r"(r[i])
  asm volatile("" : PQKV_R32(PQKV_IO)::"memory");
#undef PQKV_IO
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Shared-memory operand of 128 rows of 64 fp16 values per 16 KB half, rows of
// 128 bytes, 128-byte swizzle (a 16-byte chunk's index is XORed with row & 7).
// The rows run along M or N and the values along K (Q, K): the 8-row groups
// are 1 KB apart, a k-step of 16 values is 32 bytes further.
// The rows run along K and the values along N (V): the two 64-value halves are
// 16 KB apart, the 8-row groups 1 KB, a k-step of 16 rows is 2 KB further.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t half_stride) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)(half_stride >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// kind::f16, fp16 A and B, fp32 D, M 128, N 64 (keys) and 128 (dims); B with
// its rows along K for V
constexpr uint32_t kIdescQK = (1u << 4) | ((64u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kIdescPV = (1u << 4) | (1u << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);

__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unf2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}
// 32 bytes, a whole sector per lane
__device__ __forceinline__ void stg256(float* dst, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ uint4 lds128u(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

// TMA of one page's K or V rows into place
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                            int c0, int c1, int c2, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4),
      "r"(smem_u32(bar))
      : "memory");
}

// ---------------------------------------------------------------------------
// Work
// ---------------------------------------------------------------------------
struct UmmaFrag {
  int g, h, rt;       // group, kv-head, row tile
  int u0, u1;         // key tiles [u0, u1)
  int row0, nrows;    // first row of the tile, rows of the group's kv-head
  int pages;          // shared pages of the group
  int seg;            // segment: row tiles in order over groups and kv-heads
  bool dual;          // more than 128 rows: the streams split the rows
};

// The CTA's fragments in order.  Segment (g, h, rt) covers the costs
// [a, a + w T) of its T key tiles (w = 2 or 1); key tile i belongs to the share
// that holds cost a + w i.
struct UmmaIter {
  const int* tab;     // the plan's rows of groups
  int stride;         // entries per row
  int64_t x, e;

  __device__ int goff(int g) const { return tab[g]; }
  __device__ int gpages(int g) const { return tab[stride + g]; }
  __device__ int gtiles(int g) const { return tab[2 * stride + g]; }
  __device__ int gcost(int g) const { return tab[3 * stride + g]; }

  // M groups, H kv-heads, `rows` rows of a (sequence, kv-head)
  __device__ bool next(UmmaFrag& f, int M, int H, int rows) {
    while (x < e) {
      int lo = 0, hi = M - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int64_t)gcost(mid) * H <= x) lo = mid; else hi = mid - 1;
      }
      const int g = lo, C = gcost(g + 1) - gcost(g);
      const int T = (gpages(g) + kUmmaPages - 1) / kUmmaPages;
      const int64_t off = x - (int64_t)gcost(g) * H;
      f.g = g;
      f.h = (int)Shares::div(off, C);
      const int in = (int)(off - (int64_t)f.h * C);
      f.rt = in / (2 * T);
      f.nrows = (goff(g + 1) - goff(g)) * rows;
      f.row0 = f.rt * kUmmaRows;
      f.dual = f.nrows - f.row0 > 128;
      const int w = f.dual ? 2 : 1;
      const int64_t a = x - (in - f.rt * 2 * T);
      f.u0 = (int)((x - a + w - 1) / w);
      f.u1 = (int)min((int64_t)T, (e - a + w - 1) / w);
      f.pages = gpages(g);
      f.seg = gtiles(g) * H + f.h * (gtiles(g + 1) - gtiles(g)) + f.rt;
      x = min(e, a + (int64_t)w * T);
      if (f.u0 < f.u1) return true;
    }
    return false;
  }
};

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int KVT>
struct UmmaCfg {
  static constexpr bool kWide = KVT == PQKV_KV_FP16;      // rows need no widening
  static constexpr bool kRowScaled = KVT == PQKV_KV_INT8_ROW;
  static constexpr int kThreads = 512;
  static constexpr long long kWaitCycles = 1ll << 31;     // 1.04 s at 2.07 GHz
  // A row's reference maximum is raised when a score passes it by more than
  // this (log2): probabilities stay <= 2^14, within fp16's 2^16, and the fewer
  // rescales of O the better (8 as in the decode kernel: 300 cycles a step on
  // scores with outliers).  Row-scaled V: p times a scale of up to 2^8 has to
  // fit too.
  static constexpr float kRaise = kRowScaled ? 8.f : 14.f;
  static constexpr int kHalf = 128 * 128;                 // 16 KB: 128 rows of 64 values
  static constexpr int kTile = 2 * kHalf;
  static constexpr int kQOff = 0;                         // 2 streams
  static constexpr int kKOff = kQOff + 2 * kTile;         // 2 stages
  static constexpr int kVOff = kKOff + 2 * kTile;         // 2 stages
  static constexpr int kCodeOff = kVOff + 2 * kTile;      // staged codes: slabs of 128 rows
  static constexpr int kSlab = 128 * 128;
  static constexpr int kSlabs = kWide ? 0 : 2;
  static constexpr int kScOff = kCodeOff + kSlabs * kSlab;  // fp16 row scales: 3 stages of K and V
  static constexpr int kScBytes = kRowScaled ? 3 * 2 * 128 * 2 : 0;
  static constexpr int kBarOff = kScOff + kScBytes;
  static constexpr int kBars = 4 + 8 + 14 + 2;
  // the plan of up to kTabGroups groups is copied to shared memory (more are
  // read from L2: a search per fragment)
  static constexpr int kTabGroups = kRowScaled ? 15 : 48;
  static constexpr int kTabOff = kBarOff + kBars * 8 + 8;
  static constexpr int kSmemBytes = kTabOff + 4 * (kTabGroups + 1) * 4 + 1024;
  static_assert(kSmemBytes <= 232448, "shared memory of a block");
  // registers per thread of the softmax, widening and issuing warps, of the
  // 128 * 512 that the block is launched with
  static constexpr int kRegSoftmax = 152, kRegWiden = 120, kRegIssue = 88;
  static_assert(2 * kRegSoftmax + kRegWiden + kRegIssue <= 4 * 128, "registers of the launch");
};

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------
template <int KVT>
__global__ void __launch_bounds__(512, 1)
    shared_umma_kernel(const __grid_constant__ CUtensorMap map, const SharedParams p) {
  using Cfg = UmmaCfg<KVT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::kBarOff);
  uint64_t* code_full = bars;          // [2] a slab of codes has landed
  uint64_t* code_empty = bars + 2;     // [2] it has been widened
  uint64_t* k_full = bars + 4;         // [2] a stage's fp16 rows are in place
  uint64_t* k_empty = bars + 6;        // [2] the products have read them
  uint64_t* v_full = bars + 8;
  uint64_t* v_empty = bars + 10;
  uint64_t* q_ready = bars + 12;       // [stream] the fragment's query rows are in place
  uint64_t* s_full = bars + 14;        // [stream][half] 64 keys' scores in TMEM
  uint64_t* p_ready = bars + 18;       // [stream][half] their probabilities, and O rescaled
  uint64_t* o_done = bars + 22;        // [stream] their product with V is done
  uint64_t* o_last = bars + 24;        // [stream] the fragment's last product with V is done
  uint64_t* drain = bars + 26;         // [stream] after a wait that ran out
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::kBarOff + Cfg::kBars * 8);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::kBarOff + Cfg::kBars * 8 + 4);
  const int M = p.num_groups, H = p.num_kv_heads;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&code_full[i], 1);
      mbar_init(&code_empty[i], 4);
      mbar_init(&k_full[i], Cfg::kWide ? 1 : 4);
      mbar_init(&k_empty[i], 2);
      mbar_init(&v_full[i], Cfg::kWide ? 1 : 4);
      mbar_init(&v_empty[i], 2);
      mbar_init(&q_ready[i], 4);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_full[2 + i], 1);
      mbar_init(&p_ready[i], 4);
      mbar_init(&p_ready[2 + i], 4);
      mbar_init(&o_done[i], 1);
      mbar_init(&o_last[i], 1);
      mbar_init(&drain[i], 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 13) tmem_alloc_512(tmem_slot);
  if (warp == 12 && lane == 0) prefetch_tensormap(&map);
  grid_dependency_wait();
  grid_dependents_launch();
  UmmaIter it;
  it.tab = p.plan.groups;
  it.stride = M + 1;
  if (M <= Cfg::kTabGroups) {
    int* tab = reinterpret_cast<int*>(smem + Cfg::kTabOff);
    for (int i = tid; i < 4 * (M + 1); i += Cfg::kThreads) tab[i] = p.plan.groups[i];
    it.tab = tab;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const Shares sh((int64_t)it.gcost(M) * H, p.pre_workers);
  it.x = it.e = 0;
  if ((int)blockIdx.x < sh.n) {
    it.x = sh.start(blockIdx.x);
    it.e = sh.start(blockIdx.x + 1);
  }
  UmmaFrag f;

  // Bounded wait (about 1 s).  When one runs out the whole CTA stops at its next waits.
  // Called by whole warps; every lane gets the same answer.
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const long long t0 = clock64();
    for (uint32_t n = 1;; ++n) {
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
      if ((n & 63u) == 0) {
        const bool late = clock64() - t0 > Cfg::kWaitCycles;
        if (__any_sync(0xffffffffu, late || *abort_flag)) {
          if (lane == 0) {
            if (!*abort_flag) report(p.status, PQKV_DEV_TIMEOUT);
            *abort_flag = 1;
          }
          return false;
        }
      }
    }
  };

  if (warp < 8) {
    // ================= softmax: thread = row =================
    regs_up<Cfg::kRegSoftmax>();
    const int st = warp >> 2, wq = warp & 3, r = wq * 32 + lane;
    const uint32_t lane_sel = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + lane_sel + st * 128, tO = tmem + lane_sel + 256 + st * 128;
    uint32_t n_step = 0;             // steps of this stream so far (a key tile: two halves)
    uint32_t n_frag = 0;             // its fragments with a step
    uint32_t n_tile = 0;             // key tiles of the CTA so far (row scales' stages)
    // the fragment's row of this thread, or -1; its query row into shared memory
    auto load_row = [&]() -> int {
      const int row = f.row0 + (f.dual ? st * 128 : 0) + r;
      const int steps = f.dual ? f.u1 - f.u0 : (f.u1 - f.u0 + 1 - st) / 2;
      const bool live = row < f.nrows;
      if (steps > 0) {
        const int64_t tok = (int64_t)it.goff(f.g) * p.q_len + row / p.group;
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + (tok * p.num_q_heads + f.h * p.group + row % p.group) * kHeadDim);
        const uint32_t dst = sbase + Cfg::kQOff + st * Cfg::kTile + r * 128;
        uint4 v[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) v[c] = live ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int c = 0; c < 16; ++c)
          sts128(dst + (c >> 3) * Cfg::kHalf + (((c & 7) ^ (r & 7)) << 4), v[c].x, v[c].y, v[c].z,
                 v[c].w);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_ready[st]);
      }
      return live ? row : -1;
    };
    bool ok = it.next(f, M, H, p.rows);
    int my_row = ok ? load_row() : -1;
    while (ok) {
      float scale = p.sm_scale_log2;
      if constexpr (KVT == PQKV_KV_FP8_E4M3 || KVT == PQKV_KV_INT8) {
        const int hs = p.scale_per_head ? f.h : 0;
        const float ks = __ldg(p.k_scale + hs), vs = __ldg(p.v_scale + hs);
        if (!(ks > 0.f && ks <= 3.4e38f && vs > 0.f && vs <= 3.4e38f))
          report(p.status, PQKV_DEV_BAD_SCALE);
        scale *= ks;
      }
      const int nt = f.u1 - f.u0, steps = f.dual ? nt : (nt + 1 - st) / 2;
      const int keys = f.pages * kPageSize - f.u0 * kUmmaKeys;     // of the fragment, and behind
      const bool dual = f.dual;
      const bool warp_live = __any_sync(0xffffffffu, my_row >= 0);
      const int64_t slot = (int64_t)f.seg + blockIdx.x;
      const int at = st * (p.pre_rp / 2) + r;
      float ref = kNoScore, l = 0.f;
#pragma unroll 1
      for (int i = 0; ok && i < steps; ++i) {
        const int u = dual ? i : 2 * i + st;
        const uint32_t sc = sbase + Cfg::kScOff + (n_tile + u) % 3 * 512;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          if (!wait(&s_full[2 * st + half], n_step & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (warp_live) {
            const uint32_t tH = tS + 64 * half;
            uint32_t s[64];
            tmem_ld32(tH, s);
            tmem_ld32(tH + 32, s + 32);
            tmem_wait_ld();
            tmem_landed32(s);
            tmem_landed32(s + 32);
            const uint32_t sch = sc + 128 * half;          // 64 fp16 scales of K, of V 256 bytes on
            if constexpr (Cfg::kRowScaled) {
#pragma unroll
              for (int c = 0; c < 64; c += 8) {
                const uint4 k8 = lds128u(sch + c * 2);
                const uint32_t kk[4] = {k8.x, k8.y, k8.z, k8.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float2 ks = __half22float2(*reinterpret_cast<const __half2*>(&kk[j]));
                  s[c + 2 * j] = __float_as_uint(__uint_as_float(s[c + 2 * j]) * ks.x);
                  s[c + 2 * j + 1] = __float_as_uint(__uint_as_float(s[c + 2 * j + 1]) * ks.y);
                }
              }
            }
            const int valid = keys - u * kUmmaKeys - 64 * half;
            if (valid < 64) {
#pragma unroll
              for (int c = 0; c < 64; ++c)
                if (c >= valid) s[c] = 0xff800000u;            // -inf
            }
            float mx4[4] = {kNoScore, kNoScore, kNoScore, kNoScore};
#pragma unroll
            for (int c = 0; c < 64; c += 2)
              mx4[(c >> 1) & 3] = max3(mx4[(c >> 1) & 3], __uint_as_float(s[c]),
                                       __uint_as_float(s[c + 1]));
            const float m2 = max3(fmaxf(mx4[0], mx4[1]), mx4[2], mx4[3]) * scale;
            const bool raise = m2 > ref + Cfg::kRaise;
            if (__any_sync(0xffffffffu, raise)) {
              const float nref = raise ? m2 : ref;
              const float fct = ex2(ref - nref);
              ref = nref;
              l *= fct;
              if (i + half > 0) {                              // O holds something
                // the half before this one (the one before that is done: this
                // half's scores were issued behind its product)
                if (!wait(&o_done[st], (half + 1) & 1)) {
                  ok = false;
                  break;
                }
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < 128; c += 16) {
                  uint32_t o[16];
                  tmem_ld16_wait(tO + c, o);
#pragma unroll
                  for (int k = 0; k < 16; ++k)
                    o[k] = __float_as_uint(__uint_as_float(o[k]) * fct);
                  tmem_st16(tO + c, o);
                }
              }
            }
            const uint64_t scale2 = f2(scale, scale), ref2 = f2(-ref, -ref);
            uint64_t sum[4] = {0, 0, 0, 0};
            uint32_t ph[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              float a, b;
              unf2(fma2(f2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), scale2, ref2),
                   a, b);
              a = ex2(a);
              b = ex2(b);
              sum[c & 3] = add2(sum[c & 3], f2(a, b));
              if constexpr (Cfg::kRowScaled) {
                // p * (V row scale), rounded once: the fp32 product
                uint32_t w;
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(sch + 256 + c * 4));
                const float2 vs = __half22float2(*reinterpret_cast<const __half2*>(&w));
                a *= vs.x;
                b *= vs.y;
              }
              ph[c] = pack_half2(a, b);
            }
            tmem_st32(tH, ph);
            float a, b;
            unf2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), a, b);
            l += a + b;
            tmem_wait_st();
          }
          // (a warp without a row: its probabilities feed rows that nobody reads)
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_ready[2 * st + half]);
        }
        n_step += 1;
      }
      n_tile += nt;
      if (!ok) break;
      // ---- the next fragment's query row (this one's scores are done), so that
      // its first product runs under what follows
      const bool live = my_row >= 0;
      ok = it.next(f, M, H, p.rows);
      if (ok) my_row = load_row();
      // ---- O, m and l of the fragment
      if (steps > 0) {
        if (!wait(&o_last[st], n_frag & 1)) break;
        n_frag += 1;
        tc_fence_after();
      }
      if (warp_live) {
        float* dst = p.pre_o + (slot * p.pre_rp + at) * kHeadDim;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          if (steps > 0) {
            tmem_ld32(tO + 32 * c, o);
            tmem_wait_ld();
            tmem_landed32(o);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0;
          }
          if (live) {
#pragma unroll
            for (int k = 0; k < 32; k += 8) stg256(dst + 32 * c + k, o + k);
          }
        }
        if (live) {
          p.pre_ml[slot * 2 * p.pre_rp + at] = ref;
          p.pre_ml[slot * 2 * p.pre_rp + p.pre_rp + at] = l;
        }
      }
      tc_fence_before();
    }
  } else if (warp < 12) {
    // ================= widen the codes =================
    regs_down<Cfg::kRegWiden>();
    if constexpr (!Cfg::kWide) {
      const int wt = tid - 256;
      uint32_t n_slab = 0, n_tile = 0;
      bool ok = true;
      // INT8_ROW: K and V row scale (fp16 bits) of this thread's token of key
      // tile u; 0 behind the prefix and for pages outside the pool
      auto row_scale = [&](int u) -> ushort2 {
        const int tok = u * kUmmaKeys + wt, pg = tok / kPageSize, rr = tok % kPageSize;
        if (pg >= f.pages) return make_ushort2(0, 0);
        const int id = __ldg(p.block_table + (int64_t)it.goff(f.g) * p.bt_stride + pg);
        if (id < 0 || (int64_t)id >= p.num_pages) return make_ushort2(0, 0);
        const uint16_t* src = reinterpret_cast<const uint16_t*>(p.k_scale) +
                              (((int64_t)id * H + f.h) * 8 + (rr & 7)) * 4 + (rr >> 3);
        return make_ushort2(__ldg(src), __ldg(src + 2));
      };
      ushort2 ahead = make_ushort2(0, 0);
      while (ok && it.next(f, M, H, p.rows)) {
        for (int u = f.u0; ok && u < f.u1; ++u, ++n_tile) {
          if constexpr (Cfg::kRowScaled) {
            // The tile's fp16 row scales, a token per thread, read a tile ahead.
            // Stage n % 3 was last read by the softmax of tile n - 3, whose
            // product with V the V stage's release for tile n - 1 came after.
            uint16_t* dst = reinterpret_cast<uint16_t*>(smem + Cfg::kScOff + n_tile % 3 * 512);
            dst[wt] = u == f.u0 ? row_scale(u).x : ahead.x;
            dst[128 + wt] = u == f.u0 ? row_scale(u).y : ahead.y;
            if (u + 1 < f.u1) ahead = row_scale(u + 1);
          }
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv, ++n_slab) {
            const int slot = n_slab % Cfg::kSlabs, stage = n_tile & 1;
            uint64_t* empty = (kv ? v_empty : k_empty) + stage;
            if (!wait(&code_full[slot], (n_slab / Cfg::kSlabs) & 1) ||
                (n_tile >= 2 && !wait(empty, ((n_tile >> 1) + 1) & 1))) {
              ok = false;
              break;
            }
            const uint32_t src = sbase + Cfg::kCodeOff + slot * Cfg::kSlab;
            const uint32_t dst = sbase + (kv ? Cfg::kVOff : Cfg::kKOff) + stage * Cfg::kTile;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int idx = i * 128 + wt, row = idx >> 3, j = idx & 7;
              const uint4 c = lds128u(src + row * 128 + ((j ^ (row & 7)) << 4));
              uint32_t w[8];
              dequant_word<KVT>(c.x, w[0], w[1]);
              dequant_word<KVT>(c.y, w[2], w[3]);
              dequant_word<KVT>(c.z, w[4], w[5]);
              dequant_word<KVT>(c.w, w[6], w[7]);
              // the row's 16 values are chunks 2 (j & 3) and the next of half
              // j >> 2; the halves' lanes take the two in opposite order, so
              // that a row's eight lanes store to eight different chunks
              const uint32_t at = dst + (j >> 2) * Cfg::kHalf + row * 128;
              const int c0 = 2 * (j & 3) + (j >> 2), c1 = c0 ^ 1;
              const bool up = j >> 2;
              sts128(at + ((c0 ^ (row & 7)) << 4), up ? w[4] : w[0], up ? w[5] : w[1],
                     up ? w[6] : w[2], up ? w[7] : w[3]);
              sts128(at + ((c1 ^ (row & 7)) << 4), up ? w[0] : w[4], up ? w[1] : w[5],
                     up ? w[2] : w[6], up ? w[3] : w[7]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive((kv ? v_full : k_full) + stage);
              mbar_arrive(&code_empty[slot]);
            }
          }
        }
      }
    }
  } else {
  regs_down<Cfg::kRegIssue>();
  if (warp == 12) {
    // ================= copies =================
    uint32_t n = 0, n_tile = 0;      // copies (K or V of a key tile) and key tiles so far
    bool ok = true;
    while (ok && it.next(f, M, H, p.rows)) {
      const int32_t* row = p.block_table + (int64_t)it.goff(f.g) * p.bt_stride;
      for (int u = f.u0; ok && u < f.u1; ++u, ++n_tile) {
        // lane = page of the tile; pages behind the prefix read as zeros
        // (a page id one past the pool: the copy's bounds fill them)
        int id = (int)p.num_pages;
        const int pg = u * kUmmaPages + lane;
        if (lane < kUmmaPages && pg < f.pages) {
          id = __ldg(row + pg);
          if (id < 0 || (int64_t)id >= p.num_pages) report(p.status, PQKV_DEV_PAGE_RANGE);
        }
        for (int kv = 0; kv < 2; ++kv) {
          if constexpr (Cfg::kWide) {
            const int stage = n_tile & 1;
            uint64_t* full = (kv ? v_full : k_full) + stage;
            ok = n_tile < 2 || wait((kv ? v_empty : k_empty) + stage, ((n_tile >> 1) + 1) & 1);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(full, Cfg::kTile);
            __syncwarp();
            if (lane < kUmmaPages) {
              const uint32_t dst =
                  sbase + (kv ? Cfg::kVOff : Cfg::kKOff) + stage * Cfg::kTile + lane * 2048;
              tma_load_5d(dst, &map, full, 0, 0, kv * kPageSize, f.h, id);
              tma_load_5d(dst + Cfg::kHalf, &map, full, 0, 1, kv * kPageSize, f.h, id);
            }
            ++n;
          } else {
            const int slot = n % Cfg::kSlabs;
            ok = n < Cfg::kSlabs || wait(&code_empty[slot], ((n / Cfg::kSlabs) + 1) & 1);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&code_full[slot], Cfg::kSlab);
            __syncwarp();
            if (lane < kUmmaPages)
              tma_load_5d(sbase + Cfg::kCodeOff + slot * Cfg::kSlab + lane * 2048, &map,
                          &code_full[slot], 0, 0, kv * kPageSize, f.h, id);
            ++n;
          }
        }
      }
    }
    // after a wait that ran out: no copy may be in flight when the CTA ends
    __syncwarp();
    if (!ok && lane == 0) {
      if constexpr (Cfg::kWide) {
        for (uint32_t i = n > 4 ? n - 4 : 0; i < n; ++i)     // copy i: K or V of tile i / 2
          (void)mbar_wait((i & 1 ? v_full : k_full) + ((i >> 1) & 1), (i >> 2) & 1);
      } else {
        for (uint32_t i = n > Cfg::kSlabs ? n - Cfg::kSlabs : 0; i < n; ++i)
          (void)mbar_wait(&code_full[i % Cfg::kSlabs], (i / Cfg::kSlabs) & 1);
      }
    }
  } else if (warp < 15) {
    // ================= products: a warp per stream =================
    // The tensor pipe takes few products ahead of the one it works on, so a
    // wait between two products of a warp leaves it idle; with a warp for each
    // stream the other stream's products fill the gap.
    const int st = warp - 13;
    uint32_t n_tile = 0, n_q = 0, n_step = 0;
    bool ok = true;
    const uint64_t q_desc = tc_desc(sbase + Cfg::kQOff + st * Cfg::kTile, 16),
                   k_desc = tc_desc(sbase + Cfg::kKOff, 16),
                   v_desc = tc_desc(sbase + Cfg::kVOff, Cfg::kHalf);
    const uint32_t tS = tmem + st * 128, tO = tmem + 256 + st * 128;
    while (ok && it.next(f, M, H, p.rows)) {
      const int nt = f.u1 - f.u0;
      const bool dual = f.dual;
      const int steps = dual ? nt : (nt + 1 - st) / 2;
      // S = Q K^T on half a key tile.  A stage is free again when both streams
      // are done with it, or after its one stream's second arrival.
      auto qk = [&](uint32_t tl, int half) -> bool {
        const uint32_t stage = tl & 1;
        if (!half && !wait(&k_full[stage], (tl >> 1) & 1)) return false;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t b = k_desc + (uint64_t)((stage * Cfg::kTile + half * 8192) >> 4);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint64_t off = (uint64_t)(((k >> 2) * Cfg::kHalf + (k & 3) * 32) >> 4);
            tc_mma_ss(tS + 64 * half, q_desc + off, b + off, kIdescQK, k > 0);
          }
          tc_commit(&s_full[2 * st + half]);
          if (half) {
            tc_commit(&k_empty[stage]);
            if (!dual) tc_commit(&k_empty[stage]);
          }
        }
        __syncwarp();
        return true;
      };
      // O += P V on half a key tile
      auto pv = [&](uint32_t tl, int half, bool acc, bool last) -> bool {
        const uint32_t stage = tl & 1;
        if (!half && !wait(&v_full[stage], (tl >> 1) & 1)) return false;
        if (!wait(&p_ready[2 * st + half], n_step & 1)) return false;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t b = v_desc + (uint64_t)((stage * Cfg::kTile + half * 8192) >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_ts(tO, tS + 64 * half + k * 8, b + (uint64_t)(k * 2048 >> 4), kIdescPV,
                      acc || k > 0);
          tc_commit(&o_done[st]);
          if (half) {
            tc_commit(&v_empty[stage]);
            if (!dual) tc_commit(&v_empty[stage]);
            if (last) tc_commit(&o_last[st]);
          }
        }
        __syncwarp();
        return true;
      };
      // Half h's next scores go over its probabilities, right behind the product
      // that reads them (products of one thread run in order), so that they are
      // there when the softmax is done with the other half.
      if (steps > 0) {
        const uint32_t tl = n_tile + (dual ? 0 : st);
        ok = wait(&q_ready[st], n_q & 1) && qk(tl, 0) && qk(tl, 1);
        n_q += 1;
      }
#pragma unroll 1
      for (int i = 0; ok && i < steps; ++i) {
        const uint32_t tl = n_tile + (dual ? i : 2 * i + st), next = tl + (dual ? 1 : 2);
        const bool more = i + 1 < steps;
        ok = pv(tl, 0, i > 0, false) && (!more || qk(next, 0)) && pv(tl, 1, true, !more) &&
             (!more || qk(next, 1));
        n_step += 1;
      }
      n_tile += nt;
    }
    if (!ok) {                       // products in flight end before the TMEM is freed
      if (elect_one()) tc_commit(&drain[st]);
      (void)mbar_wait(&drain[st], 0);
    }
  }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 13) tmem_free_512(tmem);
}

template <int KVT>
cudaError_t launch_shared_umma_t(const SharedParams& p, const CUtensorMap& map,
                                 cudaStream_t stream) {
  using Cfg = UmmaCfg<KVT>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = opt_in_smem(shared_umma_kernel<KVT>, Cfg::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  // the register split needs the 128 registers per thread that the launch
  // bounds allow; a build that used fewer would wait for them forever
  static const int regs = [] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, shared_umma_kernel<KVT>) == cudaSuccess ? at.numRegs : 0;
  }();
  if (regs < 128) return cudaErrorLaunchOutOfResources;
  return launch_pdl(shared_umma_kernel<KVT>, p.pre_workers, Cfg::kThreads, Cfg::kSmemBytes, stream,
                    map, p);
}

}  // namespace pqkv
