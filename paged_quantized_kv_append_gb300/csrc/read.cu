// kv_read: the tokens of requests out of the pool, as contiguous fp16 rows (a request's
// cached context for a dense attention over it, or for another pool or machine).
//
// Output row t of K and of V is the token at position first_pos[s] + t - token_offsets[s]
// of the request s with token_offsets[s] <= t < token_offsets[s + 1]; its value is
//     E4M3, INT8: fp16(dec(code) * scale)    INT8_ROW: fp16(code * row scale)
//     INT4_GROUP: code * group scale (an fp16 value)    FP16: the bits
// each rounded once, to nearest even, from the exact product (fp32 holds it for INT8_ROW;
// E4M3's and INT8's product with an fp32 scale is rounded to fp32 first).
//
// A copy that widens: per (token, kv-head) 512 bytes are written and 144 to 512 read, so
// DRAM bounds it (131072 E4M3 tokens of 8 heads: 5.7 TB/s, 84 % of the measured copy; 178000
// at 4 bits: 6.0, 89 %; tiny calls 2.7 us).  A thread takes 16 values (4 bits: 32, a group):
// a block's threads lie along a token's K heads, then its V heads, then the next token, so
// that stores run over whole rows (32 or 64 bytes a lane) and the request and page are looked
// up for neighbouring tokens.
#include "block_scan.cuh"
#include "pqkv_common.cuh"

namespace pqkv {

constexpr int kReadThreads = 256;
// a piece: its stored bytes (8-bit 16, fp16 32, 4-bit 16) and their scale
template <int KVT>
struct ReadPiece {
  static constexpr int kValues = KVT == PQKV_KV_INT4_GROUP ? 32 : 16;
  static constexpr int kLoads = KVT == PQKV_KV_FP16 ? 2 : 1;      // of 16 bytes
  uint4 w[kLoads];
  float scale;
  uint16_t* out;                       // null: the row is left as it is
};

// U pieces of a thread have their loads in flight at once
template <int KVT, int U>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const ReadParams p) {
  using Piece = ReadPiece<KVT>;
  constexpr int kElem = KVT == PQKV_KV_FP16 ? 2 : 1;
  constexpr bool kInt4 = KVT == PQKV_KV_INT4_GROUP;
  constexpr int64_t kTile = kInt4 ? kInt4Tile : (int64_t)kPageSize * kHeadDim * kElem;
  __shared__ int off[PQKV_MAX_SEQS + 1];
  grid_dependency_wait();
  grid_dependents_launch();
  const int B = p.num_seqs, H = p.num_kv_heads;
  for (int i = threadIdx.x; i <= B; i += kReadThreads) off[i] = p.token_offsets[i];
  __syncthreads();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= B; i += kReadThreads)
      if (i == 0 ? off[0] != 0 : off[i] < off[i - 1]) report(p.status, PQKV_DEV_SEQ_RANGE);
  constexpr int kRow = kHeadDim / Piece::kValues;              // pieces of a row
  const int per_token = 2 * H * kRow;
  const int live = min(off[B], p.num_tokens);
  if (blockIdx.x == 0 && threadIdx.x == 0 && off[B] > p.num_tokens)
    report(p.status, PQKV_DEV_SEQ_RANGE);
  const int64_t total = (int64_t)live * per_token;

  for (int64_t i0 = (int64_t)blockIdx.x * kReadThreads * U; i0 < total;
       i0 += (int64_t)gridDim.x * kReadThreads * U) {
    const int t0 = (int)(i0 / per_token);
    const uint32_t j0 = (uint32_t)(i0 - (int64_t)t0 * per_token);
    int s = last_at_most(off, B, t0);
    Piece x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t at = j0 + u * kReadThreads + threadIdx.x, dt = at / (uint32_t)per_token;
      const int64_t t = (int64_t)t0 + dt;
      const int j = (int)(at - dt * per_token);
      x[u].out = nullptr;
      if (t >= live) continue;
      while (s + 1 < B && off[s + 1] <= t) ++s;
      const int c = j % kRow, kvh = j / kRow, kv = kvh >= H, h = kv ? kvh - H : kvh;
      const int64_t pos = (int64_t)(p.first_pos ? __ldg(p.first_pos + s) : 0) + t - off[s];
      if (t < off[s] || t >= off[s + 1] || pos < 0 || pos >= (int64_t)p.bt_stride * kPageSize) {
        if (j == 0) report(p.status, PQKV_DEV_SEQ_RANGE);
        continue;
      }
      float scale = 1.f;
      if constexpr (KVT == PQKV_KV_FP8_E4M3 || KVT == PQKV_KV_INT8) {
        scale = __ldg((kv ? p.v_scale : p.k_scale) + (p.scale_per_head ? h : 0));
        if (!(scale > 0.f && scale <= 3.4e38f)) {
          if (c == 0) report(p.status, PQKV_DEV_BAD_SCALE);
          continue;
        }
      }
      x[u].out = (kv ? p.v + t * p.v_stride : p.k + t * p.k_stride) + h * kHeadDim +
                 c * Piece::kValues;
      x[u].scale = scale;
      const int id = __ldg(p.block_table + (int64_t)s * p.bt_stride + (int)pos / kPageSize);
      const int r = (int)pos % kPageSize;
      if (id < 0 || (int64_t)id >= p.num_pages) {
        if (j == 0) report(p.status, PQKV_DEV_PAGE_RANGE);
        x[u].scale = 0.f;
#pragma unroll
        for (int k = 0; k < Piece::kLoads; ++k) x[u].w[k] = make_uint4(0, 0, 0, 0);
        continue;
      }
      const uint8_t* tile = p.pages + (((int64_t)id * H + h) * 2 + kv) * kTile;
      if constexpr (kInt4) {
        x[u].w[0] = __ldcs(reinterpret_cast<const uint4*>(tile + int4_chunk(r >> 1, r & 1, c)));
        x[u].scale =
            __half2float(__ldg(reinterpret_cast<const __half*>(tile + kInt4Codes) + c * kPageSize + r));
      } else {
        const uint4* src = reinterpret_cast<const uint4*>(tile + (r * kHeadDim + c * 16) * kElem);
#pragma unroll
        for (int k = 0; k < Piece::kLoads; ++k) x[u].w[k] = __ldcs(src + k);
        if constexpr (KVT == PQKV_KV_INT8_ROW)     // [i][K row i, K row i + 8, V row i, ...]
          x[u].scale = __half2float(__ushort_as_half(__ldg(
              p.row_scales + (((int64_t)id * H + h) * 8 + (r & 7)) * 4 + kv * 2 + (r >> 3))));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!x[u].out) continue;
      const uint32_t w[4] = {x[u].w[0].x, x[u].w[0].y, x[u].w[0].z, x[u].w[0].w};
      uint32_t o[8];
      if constexpr (kInt4) {
        const Int4Scale sc(__half2half2(__float2half_rn(x[u].scale)));     // (exact)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t f[4];
            int4_word(w[2 * half + k], sc, f);
#pragma unroll
            for (int m = 0; m < 4; ++m) o[4 * k + m] = f[m];
          }
          stg256(x[u].out + 16 * half, o);
        }
        continue;
      }
      if constexpr (KVT == PQKV_KV_FP16) {
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = w[k];
        o[4] = x[u].w[Piece::kLoads - 1].x;
        o[5] = x[u].w[Piece::kLoads - 1].y;
        o[6] = x[u].w[Piece::kLoads - 1].z;
        o[7] = x[u].w[Piece::kLoads - 1].w;
      } else if constexpr (!kInt4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t lo, hi;
          if constexpr (KVT == PQKV_KV_FP8_E4M3) e4m3_word(w[k], lo, hi);
          else int8_word(w[k], lo, hi);
          const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
          const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
          o[2 * k] = pack_half2(a.x * x[u].scale, a.y * x[u].scale);
          o[2 * k + 1] = pack_half2(b.x * x[u].scale, b.y * x[u].scale);
        }
      }
      stg256(x[u].out, o);
    }
  }
}

template <int KVT>
cudaError_t launch_read_t(const ReadParams& p, int sms, cudaStream_t stream) {
  const int64_t pieces =
      (int64_t)p.num_tokens * p.num_kv_heads * 2 * (kHeadDim / ReadPiece<KVT>::kValues);
  // Four pieces a thread where that fills the SMs, one where it does not (at 4 bits, 2048 tokens
  // of 8 heads: 6.6 us, with four 8.0; 178000 tokens: 155 us, with one 179; E4M3, 131072: 142, 187).
  const int64_t most = (int64_t)sms * 8;
  if (pieces < most * kReadThreads)
    return launch_pdl(read_kernel<KVT, 1>, (unsigned)((pieces + kReadThreads - 1) / kReadThreads),
                      kReadThreads, 0, stream, p);
  const int64_t want = (pieces + 4 * kReadThreads - 1) / (4 * kReadThreads);
  return launch_pdl(read_kernel<KVT, 4>, (unsigned)(want < most ? want : most), kReadThreads, 0,
                    stream, p);
}

cudaError_t launch_read(const ReadParams& p, int kv_dtype, int sms, cudaStream_t stream) {
  switch (kv_dtype) {
    case PQKV_KV_FP16: return launch_read_t<PQKV_KV_FP16>(p, sms, stream);
    case PQKV_KV_FP8_E4M3: return launch_read_t<PQKV_KV_FP8_E4M3>(p, sms, stream);
    case PQKV_KV_INT8: return launch_read_t<PQKV_KV_INT8>(p, sms, stream);
    case PQKV_KV_INT8_ROW: return launch_read_t<PQKV_KV_INT8_ROW>(p, sms, stream);
    case PQKV_KV_INT4_GROUP: return launch_read_t<PQKV_KV_INT4_GROUP>(p, sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pqkv
