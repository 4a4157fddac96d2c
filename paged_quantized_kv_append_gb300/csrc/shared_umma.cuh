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
// Warps: 0-7 and 8-15 the softmax of stream 0 and 1 (two threads per row, each
// with 64 of a tile's 128 keys), 16-19 and 20-23 widen the 8-bit codes of K and of
// V to fp16 (exact; TMA writes the fp16 pool's rows into place itself), 24 and
// 26 issue the copies of K and V, 25 the products, 27 announces the share's
// fragments.
//
// A row's reference m is one of its scores and follows the largest loosely (see kRaise),
// so O is rescaled now and then, by the softmax warps themselves, between two products of their
// stream.
//
// What bounds it: a stream's chain of scores, softmax and product with V.  The 32
// products of a tile of 256 rows take 2048 cycles (64 each); a tile takes 2840 for
// fp16, 3200 for E4M3 and INT8 (whose widening shares the softmax's issue slots) and
// more for INT8_ROW, which scales scores and probabilities; TMEM holds no third stream (128 columns
// of scores and 128 of O each).  1280 rows a head against 32768 keys of E4M3, 8 heads
// (172 GFLOP): 135 us from cold caches, 1.3 PFLOP/s; 134 MB of codes are read up to
// five times, out of L2.  A CTA's first scores begin 6 to 7 us after it does (plan,
// page ids, copies, widening), its second fragment's 4 us after the first one's last.
// Slower when measured: the codes fetched by the widening warps themselves, a page
// prefetch into L2, the products issued by a warp per stream, 64 keys a step.
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
// one column
__device__ __forceinline__ uint32_t tmem_ld1_wait(uint32_t addr) {
  uint32_t v;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\t"
               "tcgen05.wait::ld.sync.aligned;"
               : "=r"(v)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void tmem_st1(uint32_t addr, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(addr), "r"(v) : "memory");
}
// 16 columns
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
// The loads are asynchronous: after the wait, mark the registers as written
// here, so that nothing that reads them is scheduled before it.
__device__ __forceinline__ void tmem_landed16(uint32_t* r) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
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

// kind::f16, fp16 A and B, fp32 D, M 128, N 128; B with its rows along K for V
constexpr uint32_t kIdescQK = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kIdescPV = kIdescQK | (1u << 16);

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

// barrier of 64 threads (two warps); pair_any also ORs their predicates
__device__ __forceinline__ void pair_sync(int id) {
  asm volatile("barrier.sync.aligned %0, 64;" ::"r"(id) : "memory");
}
__device__ __forceinline__ bool pair_any(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\t"
      "barrier.red.or.pred.aligned q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)v)
      : "memory");
  return r != 0;
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
// A fragment of the CTA's share: key tiles [u0, u0 + nt) of one row tile.
struct UmmaFrag {
  int nt;             // key tiles; 0: the share is done
  int dual;           // more than 128 rows: the streams split the rows
  int h;              // kv-head
  int seq0;           // the group's first sequence
  int row0, nrows;    // first row of the tile, rows of the group's kv-head
  int page0, pages;   // first page of the fragment, shared pages of the group
  int slot;           // of the partial result
  int pad[3];
};
static_assert(sizeof(UmmaFrag) == 48, "three 16-byte words");

// The CTA's fragments in order.  Segment (g, h, rt) covers the costs
// [a, a + w T) of its T key tiles (w a tile's cost); key tile i belongs to the share
// that holds cost a + w i.
struct UmmaIter {
  const SharedParams& p;
  int64_t x, e;

  __device__ UmmaFrag next(int cta) {
    const int M = p.num_groups, H = p.num_kv_heads;
    const int32_t *goff = p.plan.goff(), *gpages = p.plan.gpages(M), *gtiles = p.plan.gtiles(M),
                  *gcost = p.plan.gcost(M);
    UmmaFrag f = {};
    while (x < e) {
      int g = 0, hi = M - 1;
      while (g < hi) {
        const int mid = (g + hi + 1) >> 1;
        if ((int64_t)gcost[mid] * H <= x) g = mid; else hi = mid - 1;
      }
      const int C = gcost[g + 1] - gcost[g];
      const int T = (gpages[g] + kUmmaPages - 1) / kUmmaPages;
      const int64_t off = x - (int64_t)gcost[g] * H;
      f.h = (int)Shares::div(off, C);
      const int in = (int)(off - (int64_t)f.h * C);
      const int rt = in / (kFullCost * T);
      f.seq0 = goff[g];
      f.nrows = (goff[g + 1] - f.seq0) * p.rows;
      f.row0 = rt * kUmmaRows;
      f.dual = f.nrows - f.row0 > 128;
      const int w = f.dual ? kFullCost : p.split_cost;
      const int64_t a = x - (in - rt * kFullCost * T);
      const int u0 = (int)((x - a + w - 1) / w);
      f.nt = (int)min((int64_t)T, (e - a + w - 1) / w) - u0;
      f.page0 = u0 * kUmmaPages;
      f.pages = gpages[g];
      f.slot = gtiles[g] * H + f.h * (gtiles[g + 1] - gtiles[g]) + rt + cta;
      x = min(e, a + (int64_t)w * T);
      if (f.nt > 0) return f;
    }
    f.nt = 0;
    return f;
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
  static constexpr int kThreads = 896;
  static constexpr int kRegLaunch = 72;
  static constexpr long long kWaitCycles = 1ll << 31;     // 1.04 s at 2.07 GHz
  // A row's reference is raised when a score passes it by more than kRaise (log2), to
  // that score: probabilities stay <= 2^15.9, within fp16's 2^16 (with 8: times a row
  // scale of V of up to 2^8), and the largest key's is 1 or more.  So each is off by half a
  // step, 2^-11 of it or, under 2^-14 (INT8_ROW: with its scale), 2^-25 of the largest
  // at most, as in the other attention calls.  A raise holds its stream up by about 500
  // cycles and takes all rows of its warps to their largest scores, so that they need
  // none soon (64 x 5 rows of scores with outliers: 181.8 us a call; only the rows that
  // passed kRaise 185.3, and with 15 186.5).  With the reference 3 above the score it was
  // 181.5, but what a large score leaves of the others was rounded eight times as
  // coarsely: a tail 2^-22 under it was lost.
  static constexpr float kRaise = kRowScaled ? 8.f : 15.9f;
  static constexpr int kHalf = 128 * 128;                 // 16 KB: 128 rows of 64 values
  static constexpr int kTile = 2 * kHalf;
  static constexpr int kQOff = 0;                         // 2 streams
  static constexpr int kKOff = kQOff + 2 * kTile;         // 2 stages
  static constexpr int kVOff = kKOff + 2 * kTile;         // 2 stages
  static constexpr int kCodeOff = kVOff + 2 * kTile;      // staged codes: slabs of 128 rows
  static constexpr int kSlab = 128 * 128;
  static constexpr int kSlabs = kWide ? 0 : 2;
  static constexpr int kScOff = kCodeOff + kSlabs * kSlab;  // fp16 row scales: 4 stages of K and V
  static constexpr int kScBytes = kRowScaled ? 4 * 2 * 128 * 2 : 0;
  static constexpr int kBarOff = kScOff + kScBytes;
  static constexpr int kBars = 4 + 8 + 12 + 8;
  // fragments announced by the scheduling warp: a ring of kFrags
  static constexpr int kFrags = 4;
  static constexpr int kReaders = kWide ? 19 : 27;         // warps that read them
  static constexpr int kLeftOff = kBarOff + kBars * 8 + 8;  // softmax warps' last meetings
  static constexpr int kFragOff = kLeftOff + 16 * 4;
  static constexpr int kSmemBytes = kFragOff + kFrags * (int)sizeof(UmmaFrag);
  static_assert(kSmemBytes <= 232448, "shared memory of a block");
  // registers per thread of the softmax, widening and issuing warps, of the
  // 72 * 896 that the block is launched with
  static constexpr int kRegSoftmax = 80, kRegWiden = 56, kRegIssue = 72;
  static_assert(4 * kRegSoftmax + 2 * kRegWiden + kRegIssue <= 7 * kRegLaunch,
                "registers of the launch");
};

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------
template <int KVT, class PP = SharedParams>
__global__ void __launch_bounds__(896, 1)
    shared_umma_kernel(const __grid_constant__ CUtensorMap map, const PP p) {
  using Cfg = UmmaCfg<KVT>;
  constexpr bool kWaitTest = std::is_same<PP, SharedWaitTestParams>::value;
  constexpr long long kWaitCycles = kWaitTest ? kTestWaitCycles : Cfg::kWaitCycles;
  extern __shared__ __align__(1024) uint8_t smem[];       // the swizzle's atoms are 1 KB
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::kBarOff);
  uint64_t* code_full = bars;          // [2] a slab of codes has landed
  uint64_t* code_empty = bars + 2;     // [2] it has been widened
  uint64_t* k_full = bars + 4;         // [2] a stage's fp16 rows are in place
  uint64_t* k_empty = bars + 6;        // [2] the products have read them
  uint64_t* v_full = bars + 8;
  uint64_t* v_empty = bars + 10;
  uint64_t* q_ready = bars + 12;       // [stream] the fragment's query rows are in place
  uint64_t* s_full = bars + 14;        // [stream] scores in TMEM
  uint64_t* p_ready = bars + 16;       // [stream][part] probabilities (32 of a thread's 64 keys)
  uint64_t* o_last = bars + 20;        // [stream] the fragment's last product with V is done
  uint64_t* drain = bars + 22;         // all products are done
  uint64_t* frag_full = bars + 24;     // [kFrags]
  uint64_t* frag_empty = bars + 28;    // [kFrags]
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::kBarOff + Cfg::kBars * 8);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::kBarOff + Cfg::kBars * 8 + 4);
  const int H = p.num_kv_heads;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&code_full[i], 1);
      mbar_init(&code_empty[i], 4);
      mbar_init(&k_full[i], Cfg::kWide ? 1 : 4);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], Cfg::kWide ? 1 : 4);
      mbar_init(&v_empty[i], 1);
      mbar_init(&q_ready[i], 8);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], 8);
      mbar_init(&p_ready[2 + i], 8);
      mbar_init(&o_last[i], 1);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < Cfg::kFrags; ++i) {
      mbar_init(&frag_full[i], 1);
      mbar_init(&frag_empty[i], Cfg::kReaders);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (tid < 16) reinterpret_cast<int*>(smem + Cfg::kLeftOff)[tid] = 0;
  if (warp == 25) tmem_alloc_512(tmem_slot);
  if (warp == 24 && lane == 0) prefetch_tensormap(&map);
  // The wait is for the private keys' kernel, of which this one needs nothing but that
  // the plan, and what the caller wrote, is visible: only this wait promises that.  An
  // order of starts does not (without it, and with the merge's plan reads before its
  // own, a call took 3 to 5 us less of 40 to 180).
  grid_dependency_wait();
  grid_dependents_launch();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Bounded wait (about 1 s).  When one runs out the whole CTA stops at its next waits.
  // Called by whole warps; every lane gets the same answer.
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const long long t0 = clock64();
    for (uint32_t n = 1;; ++n) {
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
      if ((n & 63u) == 0) {
        const bool late = clock64() - t0 > kWaitCycles;
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

  // Fragment n of the CTA's share (waits until it is announced; false after a
  // wait that ran out), and the warp's word that it is done with it.
  const UmmaFrag* frags = reinterpret_cast<const UmmaFrag*>(smem + Cfg::kFragOff);
  auto frag_at = [&](uint32_t n, const UmmaFrag*& f) -> bool {
    f = frags + n % Cfg::kFrags;
    return wait(&frag_full[n % Cfg::kFrags], (n / Cfg::kFrags) & 1);
  };
  auto frag_done = [&](uint32_t n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&frag_empty[n % Cfg::kFrags]);
  };

  if (warp < 16) {
    // ================= softmax: two threads per row =================
    regs_up<Cfg::kRegSoftmax>();
    const int st = warp >> 3, half = (warp >> 2) & 1, wq = warp & 3, r = wq * 32 + lane;
    const uint32_t lane_sel = (uint32_t)(wq * 32) << 16;
    // this thread's 64 scores, over them its 64 probabilities, and 64 values of O
    const uint32_t tS = tmem + lane_sel + st * 128 + half * 64;
    const uint32_t tO = tmem + lane_sel + 256 + st * 128 + half * 64;
    // Barrier of the row's two warps: meeting k is step k's, if the fragment has a row
    // for them.  A warp that leaves, for whatever reason, notes the meeting that would
    // come next, as its last, and joins one more; the other finds the note there and
    // leaves as well.  A note of a later meeting is not for this one: the other wrote it
    // after it had passed here.  So every meeting has both warps or is both's last, and a
    // warp waits at one no longer than the other's own waits last.
    const int pair = 1 + st * 4 + wq;
    volatile uint32_t* left = reinterpret_cast<volatile uint32_t*>(smem + Cfg::kLeftOff);
    bool alone = true;               // the last meeting is still to come
    const uint32_t tPeer = tS + 31 + (half ? -64 : 64);     // the other half's maximum
    uint32_t n_step = 0;             // steps of this stream so far
    uint32_t n_last = 0;             // its fragments with a step
    uint32_t n_tile = 0;             // key tiles of the CTA so far (row scales' stages)
    uint32_t n = 0;                  // fragments
    const UmmaFrag* f;
    // whether fragment f has a row for this thread; half of it into shared memory
    auto load_row = [&]() -> bool {
      const int nt = f->nt, dual = f->dual, row = f->row0 + (dual ? st * 128 : 0) + r;
      const bool live = row < f->nrows;
      if (dual || nt > st) {
        const int64_t tok = (int64_t)f->seq0 * p.q_len + row / p.group;
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + (tok * p.num_q_heads + f->h * p.group + row % p.group) * kHeadDim + half * 64);
        const uint32_t dst = sbase + Cfg::kQOff + st * Cfg::kTile + half * Cfg::kHalf + r * 128;
        uint4 v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = live ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          sts128(dst + ((c ^ (r & 7)) << 4), v[c].x, v[c].y, v[c].z, v[c].w);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_ready[st]);
      }
      return live;
    };
    // 16 scores from column c on, once landed: scaled by their rows' scales, -inf
    // behind the prefix
    auto dress = [&](uint32_t* s, int c, int valid, uint32_t sc) {
      if constexpr (Cfg::kRowScaled) {
#pragma unroll
        for (int k = 0; k < 16; k += 8) {
          const uint4 k8 = lds128u(sc + (c + k) * 2);
          const uint32_t kk[4] = {k8.x, k8.y, k8.z, k8.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 ks = __half22float2(*reinterpret_cast<const __half2*>(&kk[j]));
            float a, b;
            unf2(mul2(f2(__uint_as_float(s[k + 2 * j]), __uint_as_float(s[k + 2 * j + 1])),
                      f2(ks.x, ks.y)),
                 a, b);
            s[k + 2 * j] = __float_as_uint(a);
            s[k + 2 * j + 1] = __float_as_uint(b);
          }
        }
      }
      if (valid < 64) {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (c + k >= valid) s[k] = 0xff800000u;
      }
    };
    bool ok = frag_at(n, f) && f->nt > 0;
    bool live = ok && load_row();
    while (ok) {
      float scale = p.sm_scale_log2;
      if constexpr (KVT == PQKV_KV_FP8_E4M3 || KVT == PQKV_KV_INT8) {
        const int hs = p.scale_per_head ? f->h : 0;
        const float ks = __ldg(p.k_scale + hs), vs = __ldg(p.v_scale + hs);
        if (!(ks > 0.f && ks <= 3.4e38f && vs > 0.f && vs <= 3.4e38f))
          report(p.status, PQKV_DEV_BAD_SCALE);
        scale *= ks;
      }
      const int nt = f->nt, dual = f->dual, slot = f->slot;
      const int steps = dual ? nt : (nt + 1 - st) / 2;
      // keys of the prefix from this thread's first on
      int valid = (f->pages - f->page0) * kPageSize - half * 64 - (dual ? 0 : st * kUmmaKeys);
      const bool warp_live = __any_sync(0xffffffffu, live);
      float ref = kNoScore, l = 0.f;
#pragma unroll 1
      for (int i = 0; i < steps; ++i) {
        if (!wait(&s_full[st], n_step & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (warp_live) {
          // INT8_ROW: the 64 fp16 scales of K, of V 256 bytes on
          const uint32_t sc = sbase + Cfg::kScOff + half * 128 +
                              (n_tile + (dual ? i : 2 * i + st)) % 4 * 512;
          // -- the maximum.  The first 32 scores stay in registers, the others are
          // read again below (registers are short)
          uint32_t s[32];
          float top;
          {
            uint32_t v[32];
            tmem_ld32(tS, s);
            tmem_ld32(tS + 32, v);
            tmem_wait_ld();
            tmem_landed32(s);
            tmem_landed32(v);
            float m[4] = {kNoScore, kNoScore, kNoScore, kNoScore};
#pragma unroll
            for (int c = 0; c < 32; c += 16) {
              dress(v + c, 32 + c, valid, sc);
              dress(s + c, c, valid, sc);
            }
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              m[k & 2] = max3(m[k & 2], __uint_as_float(v[k]), __uint_as_float(v[k + 1]));
              m[1 + (k & 2)] = max3(m[1 + (k & 2)], __uint_as_float(s[k]), __uint_as_float(s[k + 1]));
            }
            top = max3(fmaxf(m[0], m[1]), m[2], m[3]);
          }
          // (the largest exponent as it will be formed below: no probability can be more)
          if (pair_any(pair, fmaf(top, scale, -ref) > Cfg::kRaise)) {
            const uint32_t last = left[warp ^ 4];
            if (last && last <= n_step + 1) {        // the other warp has left
              ok = alone = false;
              break;
            }
            // -- raise, of every row to its largest score so far: the two warps tell each
            // other their rows' maxima (over the last of the scores that are in
            // registers) and rescale half of O each.
            // O is still: the last product with V came before these scores
            top *= scale;
            tmem_st1(tS + 31, __float_as_uint(top));
            tmem_wait_st();
            tc_fence_before();
            pair_sync(pair);
            tc_fence_after();
            const float nref = max3(ref, top, __uint_as_float(tmem_ld1_wait(tPeer)));
            const float fct = ex2(ref - nref);
            ref = nref;
            l *= fct;
            if (i > 0) {
#pragma unroll 1
              for (int c = 0; c < 64; c += 32) {
                uint32_t o[32];
                tmem_ld32(tO + c, o);
                tmem_wait_ld();
                tmem_landed32(o);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * fct);
                tmem_st32(tO + c, o);
              }
            }
            tc_fence_before();
            pair_sync(pair);                 // both maxima are read: P may go over them
            tc_fence_after();
          }
          // -- the probabilities, 16 keys at a time; the first 32 are handed over
          // while the others are formed
          const uint64_t scale2 = f2(scale, scale), ref2 = f2(-ref, -ref);
          uint64_t sum[2] = {0, 0};
          [[maybe_unused]] uint4 vs8;
          uint32_t ph[16];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t* x = s + 16 * (c & 1);
            if (c >= 2) {
              tmem_wait_ld();
              tmem_landed16(x);
              if (c == 2) tmem_ld16(tS + 48, s + 16);
              dress(x, 16 * c, valid, sc);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              float a, b;
              unf2(fma2(f2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), scale2, ref2),
                   a, b);
              a = ex2(a);
              b = ex2(b);
              sum[k & 1] = add2(sum[k & 1], f2(a, b));
              if constexpr (Cfg::kRowScaled) {
                // p * (V row scale) in fp32, rounded once.  As fp16(code * scale) in
                // the widening the error grew by a half (for 3 us of 106)
                if (k % 4 == 0) vs8 = lds128u(sc + 256 + (16 * c + 2 * k) * 2);
                const uint32_t w = k % 4 == 0 ? vs8.x : k % 4 == 1 ? vs8.y
                                                      : k % 4 == 2 ? vs8.z : vs8.w;
                const float2 vs = __half22float2(*reinterpret_cast<const __half2*>(&w));
                unf2(mul2(f2(a, b), f2(vs.x, vs.y)), a, b);
              }
              ph[8 * (c & 1) + k] = pack_half2(a, b);
            }
            if (c == 0) tmem_ld16(tS + 32, s);         // lands under the second 16
            if (c == 1) {
              tmem_st16(tS, ph);
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&p_ready[2 * st]);
            }
          }
          tmem_st16(tS + 16, ph);
          float a, b;
          unf2(add2(sum[0], sum[1]), a, b);
          l += a + b;
          tmem_wait_st();
        } else if (lane == 0) {
          mbar_arrive(&p_ready[2 * st]);
        }
        // (a warp without a row: its probabilities feed rows that nobody reads)
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[2 * st + 1]);
        n_step += 1;
        valid -= dual ? kUmmaKeys : 2 * kUmmaKeys;
      }
      n_tile += nt;
      if (!ok) break;
      // ---- the next fragment's query row (this one's scores are done), so that
      // its first product runs under what follows
      frag_done(n);
      n += 1;
      const bool store = live;
      if (!frag_at(n, f)) break;
      ok = f->nt > 0;
      live = ok && load_row();
      // ---- O, m and l of the fragment
      if (steps > 0) {
        if (!wait(&o_last[st], n_last & 1)) break;
        n_last += 1;
        tc_fence_after();
      }
      if (warp_live) {
        const int at = st * (p.pre_rp / 2) + r;
        float* dst = p.pre_o + ((int64_t)slot * p.pre_rp + at) * kHeadDim + half * 64;
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          uint32_t o[32];
          if (steps > 0) {
            tmem_ld32(tO + c, o);
            tmem_wait_ld();
            tmem_landed32(o);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0;
          }
          if (store) {
#pragma unroll
            for (int k = 0; k < 32; k += 8) stg256(dst + c + k, o + k);
          }
        }
        if (store) {                                           // m, and l of either half
          float* ml = p.pre_ml + (int64_t)slot * 3 * p.pre_rp + at;
          if (half == 0) ml[0] = ref;
          ml[(1 + half) * p.pre_rp] = l;
        }
      }
      tc_fence_before();
    }
    if (alone) {
      if (lane == 0) left[warp] = n_step + 1;
      __syncwarp();
      (void)pair_any(pair, true);
    }
  } else if (warp < 24) {
    // ================= widen the codes =================
    regs_down<Cfg::kRegWiden>();
    if constexpr (!Cfg::kWide) {
      const int kv = (warp - 16) >> 2, wt = (tid - 512) & 127;       // K or V
      uint64_t *full = kv ? v_full : k_full, *empty = kv ? v_empty : k_empty;
      const uint32_t src = sbase + Cfg::kCodeOff + kv * Cfg::kSlab;
      uint32_t n_tile = 0;
      bool ok = true;
      const UmmaFrag* f;
      // INT8_ROW: K and V row scale (fp16 bits) of this thread's token of key
      // tile u; 0 behind the prefix and for pages outside the pool
      auto row_scale = [&](int u) -> ushort2 {
        const int pg = f->page0 + u * kUmmaPages + wt / kPageSize, rr = wt % kPageSize;
        if (pg >= f->pages) return make_ushort2(0, 0);
        const int id = __ldg(p.block_table + (int64_t)f->seq0 * p.bt_stride + pg);
        if (id < 0 || (int64_t)id >= p.num_pages) return make_ushort2(0, 0);
        const uint16_t* from = reinterpret_cast<const uint16_t*>(p.k_scale) +
                               (((int64_t)id * H + f->h) * 8 + (rr & 7)) * 4 + (rr >> 3);
        return make_ushort2(__ldg(from), __ldg(from + 2));
      };
      ushort2 ahead = make_ushort2(0, 0);
      for (uint32_t n = 0; ok; ++n) {
        if (!frag_at(n, f)) break;
        const int nt = f->nt;
        if (nt == 0) break;
#pragma unroll 1
        for (int u = 0; u < nt; ++u, ++n_tile) {
          const uint32_t stage = n_tile & 1;
          if constexpr (Cfg::kRowScaled)
            if (kv == 0 && u == 0) ahead = row_scale(0);
          // the codes have landed and the stage is free: a barrier per lane
          const bool odd = (lane & 1) && n_tile >= 2;
          if (!wait(odd ? empty + stage : &code_full[kv], (odd ? (n_tile >> 1) + 1 : n_tile) & 1)) {
            ok = false;
            break;
          }
          if constexpr (Cfg::kRowScaled) {
            // The tile's row scales, a token per thread, read a tile ahead, for the
            // softmax, which applies them to the fp32 scores and probabilities (and
            // may do so before V is widened: so V's come from K's warps as well).
            // Stage n % 4 was last read for tile n - 4, whose probabilities went into
            // their product before the scores of tile n - 2, waited for above, were
            // formed.
            if (kv == 0) {
              uint16_t* to = reinterpret_cast<uint16_t*>(smem + Cfg::kScOff + n_tile % 4 * 512);
              to[wt] = ahead.x;
              to[128 + wt] = ahead.y;
              if (u + 1 < nt) ahead = row_scale(u + 1);
            }
          }
          const uint32_t dst = sbase + (kv ? Cfg::kVOff : Cfg::kKOff) + stage * Cfg::kTile;
          // the slab into registers, and it may be filled again
          uint4 c[8];
          const int j = wt & 7;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = i * 16 + (wt >> 3);
            c[i] = lds128u(src + row * 128 + ((j ^ (row & 7)) << 4));
          }
          // (the fence: the loads above are done before a copy may write there.  Without
          // it a fast copy, out of L2, overtook loads that the products held up.)
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&code_empty[kv]);
          // A row's 16 values are chunks 2 (j & 3) and the next of half j >> 2; the
          // halves' lanes take the two in opposite order, so that a row's eight
          // lanes store to eight different chunks.
          const int c0 = 2 * (j & 3) + (j >> 2), c1 = c0 ^ 1;
          const bool up = j >> 2;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = i * 16 + (wt >> 3);
            const uint32_t at = dst + (j >> 2) * Cfg::kHalf + row * 128;
            uint32_t w[8];
            dequant_word<KVT>(up ? c[i].z : c[i].x, w[0], w[1]);
            dequant_word<KVT>(up ? c[i].w : c[i].y, w[2], w[3]);
            dequant_word<KVT>(up ? c[i].x : c[i].z, w[4], w[5]);
            dequant_word<KVT>(up ? c[i].y : c[i].w, w[6], w[7]);
            sts128(at + ((c0 ^ (row & 7)) << 4), w[0], w[1], w[2], w[3]);
            sts128(at + ((c1 ^ (row & 7)) << 4), w[4], w[5], w[6], w[7]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&full[stage]);
          }
        }
        if (ok) frag_done(n);
      }
    }
  } else {
  regs_down<Cfg::kRegIssue>();
  if (warp == 24 || warp == 26) {
    // ================= copies: of K and of V =================
    // One elected thread issues a tile's copies from warp-uniform code: by eight
    // lanes, a page each, a copy took 110 cycles, and the 16 (fp16: 32) of a tile
    // took longer than its products.
    const int kv = warp == 26;
    uint64_t *full = Cfg::kWide ? (kv ? v_full : k_full) : code_full + kv,
             *empty = Cfg::kWide ? (kv ? v_empty : k_empty) : code_empty + kv;
    constexpr uint32_t kStages = Cfg::kWide ? 2 : 1;
    constexpr uint32_t kBytes = Cfg::kWide ? Cfg::kTile : Cfg::kSlab;
    const uint32_t base =
        sbase + (Cfg::kWide ? (kv ? Cfg::kVOff : Cfg::kKOff) : Cfg::kCodeOff + kv * Cfg::kSlab);
    uint32_t n_tile = 0;
    bool ok = true;
    const UmmaFrag* f;
    for (uint32_t nf = 0; ok; ++nf) {
      if (!(ok = frag_at(nf, f))) break;
      const int nt = f->nt, h = f->h;
      if (nt == 0) break;
      const int32_t* row = p.block_table + (int64_t)f->seq0 * p.bt_stride + f->page0;
      const int left = f->pages - f->page0;
      // lane = page of the tile, looked up a tile ahead; pages behind the prefix
      // read as zeros (a page id one past the pool: the copy's bounds fill them)
      auto page_id = [&](int u) -> int {
        const int pg = u * kUmmaPages + lane;
        return lane < kUmmaPages && u < nt && pg < left ? __ldg(row + pg) : (int)p.num_pages;
      };
      int next_id = page_id(0);
#pragma unroll 1
      for (int u = 0; u < nt; ++u, ++n_tile) {
        const int id = next_id;
        next_id = page_id(u + 1);
        if (kv == 0 && lane < kUmmaPages && u * kUmmaPages + lane < left &&
            (id < 0 || (int64_t)id >= p.num_pages))
          report(p.status, PQKV_DEV_PAGE_RANGE);
        int ids[kUmmaPages];
#pragma unroll
        for (int i = 0; i < kUmmaPages; ++i) ids[i] = __shfl_sync(0xffffffffu, id, i);
        const uint32_t stage = n_tile % kStages;
        ok = n_tile < kStages || wait(empty + stage, (n_tile / kStages + 1) & 1);
        if (!ok) break;
        bool copy = true;
        if constexpr (kWaitTest)
          copy = (int)blockIdx.x != p.skip_block || kv != p.skip_part || (int)n_tile != p.skip_tile;
        if (copy && elect_one()) {
          mbar_arrive_expect_tx(full + stage, kBytes);
#pragma unroll
          for (int i = 0; i < kUmmaPages; ++i)
#pragma unroll
            for (int part = 0; part < (Cfg::kWide ? 2 : 1); ++part)
              tma_load_5d(base + stage * kBytes + part * Cfg::kHalf + i * 2048, &map, full + stage, 0,
                          part, kv * kPageSize, h, ids[i]);
        }
        __syncwarp();
      }
      if (ok) frag_done(nf);
    }
    // no copy may be in flight when the CTA ends, after a wait that ran out either
    if (lane == 0)
      for (uint32_t i = n_tile > kStages ? n_tile - kStages : 0; i < n_tile; ++i) {
        if constexpr (kWaitTest)
          if ((int)blockIdx.x == p.skip_block && kv == p.skip_part && (int)i == p.skip_tile) continue;
        (void)mbar_wait(full + i % kStages, (i / kStages) & 1);
      }
  } else if (warp == 25) {
    // ================= products =================
    // The streams take turns: a stream's product with V and its next scores, then
    // the other's.  Issued by a warp each, the streams' products mixed, both had
    // their scores at the same time and then the tensor cores idle.
    // counters of stream 0 and 1: fragments begun, steps
    uint32_t n_tile = 0, q0 = 0, q1 = 0, s0 = 0, s1 = 0;
    bool ok = true;
    const uint64_t q_desc = tc_desc(sbase + Cfg::kQOff, 16), k_desc = tc_desc(sbase + Cfg::kKOff, 16),
                   v_desc = tc_desc(sbase + Cfg::kVOff, Cfg::kHalf);
    // S = Q K^T of stream st on K stage `stage` (one thread)
    auto qk = [&](auto stream, uint32_t stage, bool release) {
      constexpr int st = decltype(stream)::value;
      const uint64_t a = q_desc + (uint64_t)(st * (Cfg::kTile >> 4)),
                     b = k_desc + (uint64_t)(stage * (Cfg::kTile >> 4));
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint64_t off = (uint64_t)(((k >> 2) * Cfg::kHalf + (k & 3) * 32) >> 4);
        tc_mma_ss(tmem + st * 128, a + off, b + off, kIdescQK, k > 0);
      }
      tc_commit(&s_full[st]);
      if (release) tc_commit(&k_empty[stage]);
    };
    // a stream's first scores of a fragment, on key tile tl
    auto begin = [&](auto stream, uint32_t tl, uint32_t& nq, bool release) -> bool {
      constexpr int st = decltype(stream)::value;
      if (!wait(lane & 1 ? &k_full[tl & 1] : &q_ready[st], (lane & 1 ? tl >> 1 : nq) & 1))
        return false;
      nq += 1;
      tc_fence_after();
      if (elect_one()) qk(stream, tl & 1, release);
      __syncwarp();
      return true;
    };
    // O += P V on key tile tl, P over the scores (32 columns for either half's 64
    // keys); then the stream's next scores (key tile `next`), over P: products of
    // one thread run in order.  The lanes look at a wait's two barriers at once.
    auto step = [&](auto stream, uint32_t tl, uint32_t next, bool more, bool acc, bool release,
                    uint32_t& ns) -> bool {
      constexpr int st = decltype(stream)::value;
      const uint32_t stage = tl & 1;
      const uint64_t b = v_desc + (uint64_t)(stage * (Cfg::kTile >> 4));
      const uint32_t tS = tmem + st * 128, tO = tmem + 256 + st * 128;
      // (a part: 32 keys of either half)
      if (!wait(lane & 1 ? &v_full[stage] : &p_ready[2 * st], (lane & 1 ? tl >> 1 : ns) & 1))
        return false;
      tc_fence_after();
      if (elect_one()) {
        tc_mma_ts(tO, tS, b, kIdescPV, acc);
        tc_mma_ts(tO, tS + 8, b + 128, kIdescPV, true);
        tc_mma_ts(tO, tS + 64, b + 512, kIdescPV, true);
        tc_mma_ts(tO, tS + 72, b + 640, kIdescPV, true);
      }
      __syncwarp();
      const bool odd = (lane & 1) && more;
      if (!wait(odd ? &k_full[next & 1] : &p_ready[2 * st + 1], (odd ? next >> 1 : ns) & 1))
        return false;
      ns += 1;
      tc_fence_after();
      if (elect_one()) {
        tc_mma_ts(tO, tS + 16, b + 256, kIdescPV, true);
        tc_mma_ts(tO, tS + 24, b + 384, kIdescPV, true);
        tc_mma_ts(tO, tS + 80, b + 768, kIdescPV, true);
        tc_mma_ts(tO, tS + 88, b + 896, kIdescPV, true);
        if (release) tc_commit(&v_empty[stage]);
        if (more) qk(stream, next & 1, release);
        else tc_commit(&o_last[st]);
      }
      __syncwarp();
      return true;
    };
    const std::integral_constant<int, 0> A;
    const std::integral_constant<int, 1> B;
    const UmmaFrag* f;
    for (uint32_t nf = 0; ok; ++nf) {
      if (!(ok = frag_at(nf, f))) break;
      const int nt = __shfl_sync(0xffffffffu, f->nt, 0);
      if (nt == 0) break;
      if (__shfl_sync(0xffffffffu, f->dual, 0)) {
        // both streams on every key tile
        ok = begin(A, n_tile, q0, false) && begin(B, n_tile, q1, true);
#pragma unroll 1
        for (int u = 0; ok && u < nt; ++u) {
          const uint32_t tl = n_tile + u;
          ok = step(A, tl, tl + 1, u + 1 < nt, u > 0, false, s0) &&
               step(B, tl, tl + 1, u + 1 < nt, u > 0, true, s1);
        }
      } else {
        // the even key tiles are stream 0's, the odd ones stream 1's
        ok = begin(A, n_tile, q0, true) && (nt < 2 || begin(B, n_tile + 1, q1, true));
#pragma unroll 1
        for (int u = 0; ok && u < nt; u += 2) {
          const uint32_t tl = n_tile + u;
          ok = step(A, tl, tl + 2, u + 2 < nt, u > 0, true, s0) &&
               (u + 1 >= nt || step(B, tl + 1, tl + 3, u + 3 < nt, u > 0, true, s1));
        }
      }
      n_tile += nt;
      if (ok) frag_done(nf);
    }
    // products in flight end before the TMEM is freed, after a wait that ran out too
    if (elect_one()) tc_commit(drain);
    (void)mbar_wait(drain, 0);
  } else {
    // ================= the share's fragments =================
    const Shares sh((int64_t)p.plan.gcost(p.num_groups)[p.num_groups] * H, p.pre_workers, kPrefixShare);
    UmmaIter it{p, 0, 0};
    if ((int)blockIdx.x < sh.n) {
      it.x = sh.start(blockIdx.x);
      it.e = sh.start(blockIdx.x + 1);
    }
    UmmaFrag* out = reinterpret_cast<UmmaFrag*>(smem + Cfg::kFragOff);
    for (uint32_t n = 0;; ++n) {
      const UmmaFrag f = it.next(blockIdx.x);
      if (n >= Cfg::kFrags && !wait(&frag_empty[n % Cfg::kFrags], (n / Cfg::kFrags + 1) & 1)) break;
      if (lane == 0) {
        out[n % Cfg::kFrags] = f;
        mbar_arrive(&frag_full[n % Cfg::kFrags]);
      }
      if (f.nt == 0) break;
    }
  }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 25) tmem_free_512(tmem);
}

template <int KVT, class PP>
cudaError_t launch_shared_umma_t(const PP& p, const CUtensorMap& map, cudaStream_t stream) {
  using Cfg = UmmaCfg<KVT>;
  if (p.pre_workers == 0) return cudaSuccess;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = opt_in_smem(shared_umma_kernel<KVT, PP>, Cfg::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  // the register split needs the 72 registers per thread that the launch
  // bounds allow; a build that used fewer would wait for them forever
  static const int regs = [] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, shared_umma_kernel<KVT, PP>) == cudaSuccess ? at.numRegs : 0;
  }();
  if (regs < Cfg::kRegLaunch) return cudaErrorLaunchOutOfResources;
  return launch_pdl(shared_umma_kernel<KVT, PP>, p.pre_workers, Cfg::kThreads, Cfg::kSmemBytes,
                    stream, map, p);
}

}  // namespace pqkv
