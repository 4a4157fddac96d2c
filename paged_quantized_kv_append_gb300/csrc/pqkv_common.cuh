// Device helpers shared by the append and attention kernels: inline PTX for
// mbarriers, TMA tile loads, warp-level mma / movmatrix, and the 8-bit KV code
// conversions.  sm_103a only.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

#include "pqkv_internal.h"

namespace pqkv {

// ---------------------------------------------------------------------------
// status word
// ---------------------------------------------------------------------------
__device__ __forceinline__ void report(int32_t* status, int bit) {
  if (status) atomicOr(status, bit);
}

// ---------------------------------------------------------------------------
// programmatic dependent launch
// ---------------------------------------------------------------------------
// The kernels of this library (all but one attention instantiation, see
// attention_impl.cuh) are launched with programmatic stream serialization
// allowed, so their blocks may become resident while the kernel before them
// in the stream is still running.  Such a kernel waits, before its first
// global-memory access, until that kernel has completed and its writes are
// visible (at once when there is none), and then lets the next kernel's
// blocks be scheduled: what is saved is the launch latency between kernels,
// not any ordering.
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void grid_dependents_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Host side: launch `kernel` with programmatic stream serialization allowed.
template <class... KArgs, class... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// ---------------------------------------------------------------------------
// thread-block clusters (distributed shared memory)
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}

__device__ __forceinline__ uint32_t cluster_ctarank() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(n));
  return n;
}

// every thread of every block of the cluster; orders this block's shared
// writes before the other blocks' reads that follow their wait
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// the address of shared variable `a` of block `rank` of the cluster
__device__ __forceinline__ uint32_t cluster_map(uint32_t a, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// Host side: launch with a cluster of `cluster` blocks (and programmatic
// stream serialization when `pdl`)
template <class... KArgs, class... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                           cudaStream_t stream, unsigned cluster, bool pdl, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// ---------------------------------------------------------------------------
// shared-memory addresses and mbarriers
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count)
               : "memory");
}

__device__ __forceinline__ void fence_barrier_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ uint64_t globaltimer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// Wait until the phase of the given parity has completed.  Gives up after
// kLimitNs of wall time (1 s unless a test instantiation lowers it) and
// returns false; the caller reports PQKV_DEV_TIMEOUT and stops.
constexpr uint64_t kWaitLimitNs = 1000000000ull;  // 1 s

template <uint64_t kLimitNs = kWaitLimitNs>
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t n = 1;; ++n) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((n & 255u) == 0 && globaltimer_ns() - t0 > kLimitNs) return false;
  }
}

// ---------------------------------------------------------------------------
// TMA: 4-D tiled load of one (page, kv-head) K+V tile into shared memory
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int c0, int c1, int c2, int c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
      "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// Untiled bulk copy of `bytes` (a multiple of 16; both addresses 16-byte
// aligned) from global to shared memory, completing on `bar` like a TMA tile.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1], %2, [%3], %4;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// The same without a cache hint, to a shared-memory address (what other blocks read again).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ uint64_t l2_evict_last_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  return p;
}

__device__ __forceinline__ uint64_t l2_evict_first_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}

__device__ __forceinline__ void prefetch_tensormap(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// ---------------------------------------------------------------------------
// warp-level tensor-core products
// ---------------------------------------------------------------------------
// D = A(16x16, row) * B(16x8, col) + D ; fp16 inputs, fp32 accumulators
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose an 8x8 matrix of 16-bit elements held one row-pair per lane.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// 32 bytes, a whole sector per lane
__device__ __forceinline__ void stg256(void* dst, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// ---------------------------------------------------------------------------
// 8-bit code -> fp16 conversions (exact: every E4M3 value and every integer
// in [-127, 127] is an fp16 value)
// ---------------------------------------------------------------------------
// E4M3: 4 codes of a word -> (d0,d1), (d2,d3); the halves of the word feed
// the conversions directly
__device__ __forceinline__ void e4m3_word(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// INT8: code c becomes the fp16 1024 + (c + 128) by placing (c ^ 0x80) under
// the fp16 exponent byte 0x64; 1152 is then subtracted exactly.
// t = [c0, ?, c1, ?] (raw codes in bytes 0 and 2) -> f16x2 (c0, c1)
__device__ __forceinline__ uint32_t i8pair(uint32_t t) {
  uint32_t u = (t & 0x00FF00FFu) ^ 0x64806480u;
  __half2 h = *reinterpret_cast<__half2*>(&u);
  h = __hsub2(h, __half2(__half(1152.0f), __half(1152.0f)));
  return *reinterpret_cast<uint32_t*>(&h);
}

// INT8: 4 codes of a word -> (d0,d1), (d2,d3).  The sign bits are flipped
// once for the whole word; one byte permute per pair then places two codes
// under the exponent byte 0x64 (1024 + (c + 128)), and 1152 is subtracted.
__device__ __forceinline__ void int8_word(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t x = w ^ 0x80808080u;
  uint32_t l = __byte_perm(x, 0x64646464u, 0x4140), h = __byte_perm(x, 0x64646464u, 0x4342);
  const __half2 off = __half2(__half(1152.0f), __half(1152.0f));
  __half2 hl = __hsub2(*reinterpret_cast<__half2*>(&l), off);
  __half2 hh = __hsub2(*reinterpret_cast<__half2*>(&h), off);
  lo = *reinterpret_cast<uint32_t*>(&hl);
  hi = *reinterpret_cast<uint32_t*>(&hh);
}

// ---------------------------------------------------------------------------
// 4-bit codes -> fp16 (include/pqkv.h: PQKV_KV_INT4_GROUP)
// ---------------------------------------------------------------------------
constexpr int kInt4Group = 32;        // values that share a scale
constexpr int kInt4Codes = 1024;      // bytes of a K or V tile's codes; its scales follow
constexpr int kInt4Tile = 1152;       // bytes of a K or V tile

// Where row `line` * 2 + odd of a 4-bit K or V tile keeps the 16 bytes of its group c.
// The chunks of a 128-byte line (two rows) are turned by f = 0, 5, 2, 7 from line to
// line: the eight lanes of a phase then read eight different chunks both where they
// share a line (K here), where they hold rows of four lines at one group (a row per
// thread), and where they read 8 bytes of two groups in four lines (V here).
__device__ __forceinline__ int int4_chunk(int line, int odd, int c) {
  const int f = ((line & 1) * 5) ^ (line & 2);
  return line * 128 + (((odd * 4 + c) ^ f) << 4);
}

// The value of code c under the scale s is c s: c has 3 bits and a sign, s 8 bits, so
// the product is an fp16 value.  A field of the word, n = c + 8, placed in the upper
// mantissa bits under the exponent of 16 reads as 16 + n, and (16 + n) s - 24 s = c s is one
// fused multiply-add without a rounding (24 s has at most 10 bits, and s at most 2720
// keeps it finite).
struct Int4Scale {
  __half2 s, b;                       // s and -24 s
  __device__ __forceinline__ explicit Int4Scale(__half2 scale) : s(scale) {
    b = __hmul2(scale, __half2(__half(-24.0f), __half(-24.0f)));
  }
};

__device__ __forceinline__ uint32_t int4_field(uint32_t w, const Int4Scale& sc) {
  const uint32_t v = (w & 0x03C003C0u) | 0x4C004C00u;
  const __half2 h = __hfma2(*reinterpret_cast<const __half2*>(&v), sc.s, sc.b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The four fields of a word: field f of its halves is values 2 f and 2 f + 1 of the
// word's eight (or, with halves of two rows' words, one value of either row).  Fields 0
// to 2 lie at bits 6, 2 and 10 of a half, field 3 at bits 14, 15, 0, 1, so that swapping
// the half's bytes (`swapped`) puts it at bit 6 and field 2 at bit 2.  Both shifts are to the
// left, which the multipliers can do where the logic unit is the busier one (a shift to
// the right for field 2: 1 to 2 % slower attention).
__device__ __forceinline__ void int4_pair(uint32_t w, uint32_t swapped, const Int4Scale& sc,
                                          uint32_t (&out)[4]) {
  out[0] = int4_field(w, sc);
  out[1] = int4_field(w << 4, sc);
  out[2] = int4_field(swapped << 4, sc);
  out[3] = int4_field(swapped, sc);
}

__device__ __forceinline__ void int4_word(uint32_t w, const Int4Scale& sc, uint32_t (&out)[4]) {
  int4_pair(w, __byte_perm(w, 0, 0x2301), sc, out);
}

}  // namespace pqkv
