// fa_paged_common.cuh -- what the kernels of libfa_paged.so share: the cache's view on the
// device, a packed token's sequence, a sequence's checked lengths.
#pragma once

#include "fa_band.cuh"
#include "sm100.cuh"

namespace fa {

constexpr int kStatusInvalid = -1;  // == FA_ERR_INVALID

struct PagedView {
  const int* table;
  const int* cu_q;
  const int* seq_k;
  int table_row, table_width;
  int num_pages, page_shift;
  int heads;
  int batch, tokens;
};

struct SeqInfo {
  int begin;  // first packed row
  int n;      // new tokens
  int nk;     // cached keys, new tokens included
  bool ok;    // the lengths are consistent; otherwise the sequence is left out
};

// A sequence's lengths, checked: its rows lie within the packed rows, it has at most max_q
// new tokens, and its keys fit the page table.
__device__ __forceinline__ SeqInfo seq_info(const PagedView& c, int b, int max_q) {
  SeqInfo s;
  s.begin = c.cu_q[b];
  const int end = c.cu_q[b + 1];
  s.nk = c.seq_k[b];
  s.ok = s.begin >= 0 && end >= s.begin && end <= c.tokens && end - s.begin <= max_q &&
         s.nk >= 0 &&
         s.nk <= (static_cast<long long>(c.table_width) << c.page_shift);
  s.n = s.ok ? end - s.begin : 0;
  return s;
}

// The last b < batch with cu_q[b] <= t, or -1; called by a whole warp. Each round probes 32
// places of what is left, so a batch of up to 1024 takes two dependent loads.
__device__ __forceinline__ int owner_of(const int* cu_q, int batch, int t, int lane) {
  int lo = 0, count = batch;  // candidates lo .. lo + count - 1; cu_q is taken as ascending
  if (batch <= 0 || cu_q[0] > t) return -1;
  while (count > 1) {
    const int step = (count + 31) / 32;
    const int at = lane * step;
    const unsigned hit =
        __ballot_sync(0xffffffffu, at < count && cu_q[lo + (at < count ? at : 0)] <= t);
    const int best = 31 - __clz(hit | 1u);
    lo += best * step;
    count = min(step, count - best * step);
  }
  return lo;
}

}  // namespace fa
