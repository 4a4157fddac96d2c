// Block tables grown and shortened on the GPU from the requests' lengths.
//
// pqkv_extend_block_tables: request s holds L_s tokens and gets n_s more.  With
//   have_s = ceil(L_s / 16),  need_s = ceil((L_s + n_s) / 16) - have_s,
//   upto_s = need_0 + ... + need_s
// the request is served when need_s == 0 or upto_s <= free_count, and its j-th
// new page is free_pages[free_count - 1 - (upto_s - need_s + j)] (the stack's
// top first).  The sums run over every request, the refused ones included, so
// the served requests that need pages are the leading ones and they take the
// top upto_s entries of the stack without a gap.
// pqkv_truncate_block_tables: the pages [max(ceil(keep_s / 16), owned_s),
// ceil(L_s / 16)) of each request are pushed, requests in order, pages in
// order: the place of a page on the stack is free_count + an exclusive sum.
//
// Every block repeats the scan over the requests (at most 2048, 8 to 16 KB out
// of L2) into shared memory and then takes its slice of the tokens (of the
// pages); a token finds its request by binary search in the scanned offsets.
// That costs each block about a microsecond and saves a second launch with its
// round trip through memory.  The state (seq_lens, free_count) may be updated
// in place: where another block could still read what is written, the state is
// written by a second launch of one block, which reads everything before it
// writes.
//
// Nothing here is near the memory's rate: the bytes of the largest step (777 prompts,
// 1.0 M tokens, 12.6 MB of slots and positions) take 1.9 us of it, of the others
// nothing.  What is left is a launch and the scan's chain of loads and barriers: a call
// (the next one queued behind it) takes 9.7 us for 8 requests of one token, 9.9 to 12
// for 2048 of 5, 10.8 for the 777 prompts, 8.4 to 8.9 for a truncation, of which the
// host's part is about 7.
#include <algorithm>

#include "block_scan.cuh"
#include "pqkv_common.cuh"

namespace pqkv {
namespace {

constexpr int kThreads = 512;
constexpr int kPerThread = PQKV_MAX_SEQS / kThreads;
static_assert(kPerThread * kThreads == PQKV_MAX_SEQS, "whole requests per thread");

__device__ __forceinline__ int page_count(int tokens) {
  return (int)(((unsigned)tokens + (kPageSize - 1)) / kPageSize);
}

__device__ __forceinline__ int checked_count(const int32_t* free_count, int cap, bool tell,
                                             int32_t* status) {
  const int fc = *free_count;
  if (fc >= 0 && fc <= cap) return fc;
  if (tell) report(status, PQKV_DEV_SLOT_RANGE);
  return fc < 0 ? 0 : cap;
}

__global__ void __launch_bounds__(kThreads) extend_tables_kernel(const ExtendParams p) {
  __shared__ int s_off[PQKV_MAX_SEQS];     // first token of each request in the step's batch
  __shared__ int s_len[PQKV_MAX_SEQS];     // tokens held, or -1 for a refused request
  __shared__ int s_page[PQKV_MAX_SEQS];    // pages taken by the requests before it
  grid_dependency_wait();
  grid_dependents_launch();
  const int tid = threadIdx.x, B = p.num_seqs, T = p.num_tokens;
  const bool first = blockIdx.x == 0;
  const int fc = checked_count(p.free_count, p.max_free, first && p.write_tokens, p.status);
  const int64_t cap = (int64_t)p.max_pages_per_seq * kPageSize;

  // -- every request's tokens and pages, summed.  One scan does both: from the
  // first request on whose tokens do not fit the step's batch, no later one
  // that brings tokens fits either, so counting their pages moves nothing.
  const int per = (B + kThreads - 1) / kThreads;
  int L[kPerThread], n[kPerThread], need[kPerThread];
  bool ok[kPerThread];
  int64_t tok = 0, tok_total;
  int pages = 0, pages_total, bits = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int s = tid * per + i;
    const bool in = i < per && s < B;
    L[i] = in ? p.seq_lens[s] : 0;
    n[i] = in ? p.new_tokens[s] : 0;
    ok[i] = L[i] >= 0 && n[i] >= 0 && (int64_t)L[i] + n[i] <= cap;
    if (!ok[i]) bits |= PQKV_DEV_SEQ_RANGE;
    n[i] = max(n[i], 0);
    need[i] = ok[i] ? page_count(L[i] + n[i]) - page_count(L[i]) : 0;
    tok += n[i];
    pages += need[i];
  }
  block_scan2<kThreads>(tok, pages, tok_total, pages_total);
  const bool tell = first && p.write_tokens, state = first && p.write_state;
  int taken = 0;                                     // pages of this thread's served requests
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int s = tid * per + i;
    const int off = (int)min(tok, (int64_t)T), before = pages;
    tok += n[i];
    pages += need[i];
    bool served = ok[i];
    if (served && n[i] > 0 && tok > T) {
      served = false;
      bits |= PQKV_DEV_SEQ_RANGE;
    }
    if (served && need[i] > 0 && pages > fc) {
      served = false;
      bits |= PQKV_DEV_SLOT_RANGE;
    }
    if (served) taken += need[i];
    if (i < per && s < B) {
      s_off[s] = off;
      s_len[s] = served ? L[i] : -1;
      s_page[s] = before;
      if (tell && p.token_offsets) p.token_offsets[s] = off;
      if (state) p.seq_lens_out[s] = served ? L[i] + n[i] : L[i];
    }
  }
  if (tell) {
    if (bits) report(p.status, bits);
    if (tid == 0 && p.token_offsets) p.token_offsets[B] = (int)min(tok_total, (int64_t)T);
  }
  if (state) {
    __shared__ int s_taken;
    if (tid == 0) s_taken = 0;
    __syncthreads();
    if (taken) atomicAdd(&s_taken, taken);
    __syncthreads();
    if (tid == 0) *p.free_count_out = fc - s_taken;
  }
  if (!p.write_tokens) return;
  __syncthreads();

  // -- this block's tokens
  const int live = (int)min(tok_total, (int64_t)T);
  int bad = 0;
  for (int64_t t64 = (int64_t)blockIdx.x * kThreads + tid; t64 < T;
       t64 += (int64_t)gridDim.x * kThreads) {
    const int t = (int)t64;
    int64_t slot = -1;
    int pos = -1;
    if (t < live) {
      const int s = last_at_most(s_off, B, t);
      const int len = s_len[s];
      if (len >= 0) {
        const int at = len + (t - s_off[s]);
        const int j = at / kPageSize, have = page_count(len);
        int32_t* entry = p.block_table + (int64_t)s * p.max_pages_per_seq + j;
        int page;
        if (j < have) {
          page = *entry;
        } else {
          page = p.free_pages[fc - 1 - (s_page[s] + j - have)];
          if (at % kPageSize == 0) *entry = page;    // the page's first token
        }
        if (page >= 0 && (int64_t)page < p.num_pages) {
          slot = (int64_t)page * kPageSize + at % kPageSize;
          pos = at;
        } else {
          bad = 1;
        }
      }
    }
    p.slot_mapping[t] = slot;
    if (p.positions) p.positions[t] = pos;
  }
  if (bad) report(p.status, PQKV_DEV_PAGE_RANGE);
}

__global__ void __launch_bounds__(kThreads) truncate_tables_kernel(const TruncateParams p) {
  __shared__ int s_off[PQKV_MAX_SEQS];     // pages pushed by the requests before it
  __shared__ int s_first[PQKV_MAX_SEQS];   // first page pushed
  grid_dependency_wait();
  grid_dependents_launch();
  const int tid = threadIdx.x, B = p.num_seqs;
  const bool first = blockIdx.x == 0;
  const int fc = checked_count(p.free_count, p.max_free, first && p.write_pages, p.status);
  const int64_t cap = (int64_t)p.max_pages_per_seq * kPageSize;
  const int per = (B + kThreads - 1) / kThreads;
  int gone[kPerThread], from[kPerThread], len_out[kPerThread];
  int pages = 0, bits = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int s = tid * per + i;
    gone[i] = from[i] = len_out[i] = 0;
    if (i >= per || s >= B) continue;
    const int L = p.seq_lens[s], keep = p.keep_lens[s];
    const int owned = p.owned_pages ? max(p.owned_pages[s], 0) : 0;
    len_out[i] = L;
    if (keep < 0 || keep > L || L > cap) {           // left as it is
      bits |= PQKV_DEV_SEQ_RANGE;
      continue;
    }
    len_out[i] = keep;
    from[i] = max(page_count(keep), owned);
    gone[i] = max(page_count(L) - from[i], 0);
    pages += gone[i];
  }
  int unused = 0, unused_total, total;
  block_scan2<kThreads>(unused, pages, unused_total, total);
  const int room = p.max_free - fc;                  // places left on the stack
  const int pushed = min(total, room);
  const bool state = first && p.write_state;
  int run = pages;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int s = tid * per + i;
    if (i < per && s < B) {
      s_off[s] = run;
      s_first[s] = from[i];
      if (state) p.seq_lens_out[s] = len_out[i];
    }
    run += gone[i];
  }
  if (first && p.write_pages) {
    if (tid == 0 && total > room) bits |= PQKV_DEV_SLOT_RANGE;
    if (bits) report(p.status, bits);
  }
  __syncthreads();                                   // also: every read precedes the next write
  if (state && tid == 0) *p.free_count_out = fc + pushed;
  if (!p.write_pages) return;
  int bad = 0;
  for (int64_t e64 = (int64_t)blockIdx.x * kThreads + tid; e64 < pushed;
       e64 += (int64_t)gridDim.x * kThreads) {
    const int e = (int)e64;
    const int s = last_at_most(s_off, B, e);
    const int page = p.block_table[(int64_t)s * p.max_pages_per_seq + s_first[s] + (e - s_off[s])];
    p.free_pages[fc + e] = page;
    if (page < 0) bad = 1;
  }
  if (bad) report(p.status, PQKV_DEV_PAGE_RANGE);
}

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + bn && y < x + an;
}

// Whether the state that a launch writes overlaps what its other blocks read.
bool in_place(const void* lens_out, const void* count_out, size_t row, const void* a,
              const void* b, const void* c, const void* count) {
  const void* rows[3] = {a, b, c};
  for (const void* r : rows)
    if (overlap(lens_out, row, r, row) || overlap(count_out, 4, r, row)) return true;
  return overlap(lens_out, row, count, 4) || overlap(count_out, 4, count, 4);
}

}  // namespace

cudaError_t launch_extend_tables(ExtendParams p, int sms, cudaStream_t stream) {
  const int64_t want = ((int64_t)p.num_tokens + kThreads - 1) / kThreads;
  const int grid = (int)std::min<int64_t>(std::max<int64_t>(want, 1), 2 * sms);
  const bool again = grid > 1 && in_place(p.seq_lens_out, p.free_count_out,
                                          (size_t)p.num_seqs * 4, p.seq_lens, p.new_tokens,
                                          nullptr, p.free_count);
  p.write_tokens = 1;
  p.write_state = !again;
  const cudaError_t e = launch_pdl(extend_tables_kernel, grid, kThreads, 0, stream, p);
  if (e != cudaSuccess || !again) return e;
  p.write_tokens = 0;
  p.write_state = 1;
  return launch_pdl(extend_tables_kernel, 1, kThreads, 0, stream, p);
}

cudaError_t launch_truncate_tables(TruncateParams p, int sms, cudaStream_t stream) {
  // the pages that come back are known on the device only: at most all of the
  // stack's places, and no more than the tables hold
  const int64_t most = std::min<int64_t>(p.max_free, (int64_t)p.num_seqs * p.max_pages_per_seq);
  const int64_t want = (most + kThreads - 1) / kThreads;
  const int grid = (int)std::min<int64_t>(std::max<int64_t>(want, 1), sms);
  const bool again = grid > 1 && in_place(p.seq_lens_out, p.free_count_out,
                                          (size_t)p.num_seqs * 4, p.seq_lens, p.keep_lens,
                                          p.owned_pages, p.free_count);
  p.write_pages = 1;
  p.write_state = !again;
  const cudaError_t e = launch_pdl(truncate_tables_kernel, grid, kThreads, 0, stream, p);
  if (e != cudaSuccess || !again) return e;
  p.write_pages = 0;
  p.write_state = 1;
  return launch_pdl(truncate_tables_kernel, 1, kThreads, 0, stream, p);
}

}  // namespace pqkv
