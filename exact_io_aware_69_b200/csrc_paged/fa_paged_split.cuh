// fa_paged_split.cuh -- how the attention kernels share a ragged batch out.
//
// An item is what one pass over keys serves: up to `tpi` consecutive new tokens of one
// sequence, all query heads of one key head. Its cost is the key tiles (128 keys) that its
// rows see, plus kItemCost for starting and finishing it. The items, ordered by (sequence,
// key head, place in the sequence), lie end to end on a line of cost, and CTA c of C takes
// the stretch [W c / C, W (c + 1) / C) of it: every CTA gets the same work whatever the
// lengths, an item that crosses a boundary is computed in parts, and each CTA has at most
// two parts (its first item's end, its last item's beginning). A boundary within an
// item's first kItemCost units moves to the item's start, so that no part is empty.
//
// The split depends only on the lengths, the mask and the grid, so the parts and the order
// in which they are joined -- and with them every rounding -- are the same on every call.
// Every CTA finds its two boundaries itself (a pass over the batch's lengths, no launch of
// its own, nothing to keep in step with the lengths): split_bounds below.
#pragma once

#ifdef __CUDACC__
#include "fa_paged_common.cuh"
#endif

namespace fa {

constexpr int kKeyTile = 128;
// One tile's time, about: an item's first scores wait for its first keys, and its last
// product is followed by the sums and the store.
constexpr int kItemCost = 1;

struct KeyRange {
  int lo, hi;        // keys that some row of the item sees (lo > hi: none)
  int first, count;  // their tiles
};

// Keys and tiles of the item of tokens [p * tpi, min(n, (p + 1) * tpi)).
__host__ __device__ inline KeyRange item_keys(int p, int tpi, int n, int nk, int wl, int wr) {
  const int off = nk - n;
  const int t0 = p * tpi;
  const int t1 = (t0 + tpi < n ? t0 + tpi : n) - 1;
  KeyRange r;
  r.lo = t0 + off - wl > 0 ? t0 + off - wl : 0;
  r.hi = t1 + off + wr < nk - 1 ? t1 + off + wr : nk - 1;
  r.first = r.lo <= r.hi ? r.lo / kKeyTile : 0;
  r.count = r.lo <= r.hi ? r.hi / kKeyTile - r.first + 1 : 0;
  return r;
}
__host__ __device__ inline int items_of(int n, int tpi) { return (n + tpi - 1) / tpi; }
__host__ __device__ inline int item_cost(const KeyRange& r) { return r.count + kItemCost; }

// CTAs of an attention launch: one per SM of a B200. A fixed count keeps the split the
// same everywhere, and divisions by it are multiplications.
constexpr int kSplitGrid = 148;
// A CTA's share of cost W: an even part of it, at least `least`. (Every CTA computes it in
// its prologue, where a 64-bit division by a variable is 400 cycles of latency.)
__host__ __device__ inline long long split_share(long long W, int least) {
  const long long even = (W + kSplitGrid - 1) / kSplitGrid;
  return even > least ? even : least;
}
// Start of CTA c's stretch.
__host__ __device__ inline long long split_start(long long W, int c, long long share) {
  return c * share < W ? c * share : W;
}
// a / b of non-negative numbers, 32 bits wide where they fit.
__host__ __device__ inline long long quotient(long long a, long long b) {
  return (a | b) >> 32 ? a / b : static_cast<unsigned>(a) / static_cast<unsigned>(b);
}
// The tile at which a boundary `r` units into an item cuts it (0: before the item).
__host__ __device__ inline int split_tile(long long r) {
  return r <= kItemCost ? 0 : static_cast<int>(r - kItemCost);
}

// Before tile j of the item (sequence b, key head h, place p).
struct Bound {
  int b, h, p, j;
};

#ifdef __CUDACC__
// A CTA's stretch: from `at` to before `end`; `seq` is at's sequence.
struct Stretch {
  Bound at, end;
  SeqInfo seq;
};

// Called by all threads of the block. `costs`: shared scratch of 8 bytes per sequence;
// *out: shared. Reports sequences with inconsistent lengths. Ends with a __syncthreads.
template <bool ONE_ITEM>
__device__ __forceinline__ void split_bounds(const PagedView& c, int tpi, int max_q, int wl,
                                             int wr, int least, long long* costs, Stretch* out) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int warps = blockDim.x >> 5;
  // cost per key head of every sequence
  if (ONE_ITEM) {
    for (int b = threadIdx.x; b < c.batch; b += blockDim.x) {
      const SeqInfo s = seq_info(c, b, max_q);
      if (!s.ok && blockIdx.x == 0) atomicExch(&g_fa_status, kStatusInvalid);
      costs[b] = s.n > 0 ? item_cost(item_keys(0, tpi, s.n, s.nk, wl, wr)) : 0;
    }
  } else {
    for (int b = warp; b < c.batch; b += warps) {
      const SeqInfo s = seq_info(c, b, max_q);
      if (!s.ok && blockIdx.x == 0 && lane == 0) atomicExch(&g_fa_status, kStatusInvalid);
      const int items = items_of(s.n, tpi);
      long long sum = 0;
      for (int p = lane; p < items; p += 32)
        sum += item_cost(item_keys(p, tpi, s.n, s.nk, wl, wr));
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (lane == 0) costs[b] = sum;
    }
  }
  __syncthreads();
  if (warp < 2) {  // warp w finds the start of CTA blockIdx.x + w
    const int per = (c.batch + 31) / 32;
    const int b0 = min(c.batch, lane * per), b1 = min(c.batch, b0 + per);
    long long own = 0;
    for (int b = b0; b < b1; ++b) own += costs[b];
    long long upto = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += v;
    }
    const long long W = __shfl_sync(0xffffffffu, upto, 31) * c.heads;
    const long long x =
        split_start(W, static_cast<int>(blockIdx.x) + warp, split_share(W, least));
    Bound at{c.batch, 0, 0, 0};
    SeqInfo s{};
    if (x < W) {
      // the lane whose sequences hold x, then the sequence
      const long long before = (upto - own) * c.heads;
      const unsigned hit = __ballot_sync(0xffffffffu, before <= x && x < upto * c.heads);
      const int from = __ffs(hit) - 1;
      int b = b0;
      long long rem = x - before;
      if (lane == from)
        while (rem >= costs[b] * c.heads) rem -= costs[b++] * c.heads;
      b = __shfl_sync(0xffffffffu, b, from);
      rem = __shfl_sync(0xffffffffu, rem, from);
      const long long w = costs[b];
      at.b = b;
      at.h = static_cast<int>(quotient(rem, w));
      rem -= at.h * w;
      s = seq_info(c, b, max_q);
      if (!ONE_ITEM) {
        for (int p0 = 0;; p0 += 32) {  // ends: rem < w, the sum over all items
          const int p = p0 + lane;
          const bool real = p < items_of(s.n, tpi);
          const int cost = real ? item_cost(item_keys(p, tpi, s.n, s.nk, wl, wr)) : 0;
          int sum = cost;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d) sum += v;
          }
          const unsigned in = __ballot_sync(0xffffffffu, real && rem < sum);
          if (in) {
            const int l = __ffs(in) - 1;
            at.p = p0 + l;
            rem -= __shfl_sync(0xffffffffu, sum - cost, l);
            break;
          }
          if (!__any_sync(0xffffffffu, real)) break;
          rem -= __shfl_sync(0xffffffffu, sum, 31);
        }
      }
      at.j = split_tile(rem);
    }
    if (lane == 0) {
      if (warp == 0) {
        out->at = at;
        out->seq = s;
      } else {
        out->end = at;
      }
    }
  }
  fence_async_smem();  // the scratch may be written by TMA next
  __syncthreads();
}

// A CTA's items in order. Every role of the CTA walks them by itself.
struct Walk {
  Bound at, end;
  SeqInfo seq;
  KeyRange keys;
  int j0, j1;  // this CTA's tiles of the item, counted from keys.first
  bool more;

  __device__ __forceinline__ Walk(const PagedView& c, int tpi, int max_q, int wl, int wr,
                                  const Stretch& s)
      : at(s.at), end(s.end), seq(s.seq) {
    j0 = at.j;
    more = at.b < c.batch;
    settle(c, tpi, wl, wr);
  }
  __device__ __forceinline__ bool at_end() const {
    return at.b == end.b && at.h == end.h && at.p == end.p;
  }
  __device__ __forceinline__ void settle(const PagedView& c, int tpi, int wl, int wr) {
    if (more && at_end() && end.j <= j0) more = false;
    if (!more) return;
    keys = item_keys(at.p, tpi, seq.n, seq.nk, wl, wr);
    j1 = at_end() ? end.j : keys.count;
  }
  __device__ __forceinline__ void next(const PagedView& c, int tpi, int max_q, int wl, int wr) {
    if (at_end()) {
      more = false;
      return;
    }
    j0 = 0;
    if ((++at.p) * tpi >= seq.n) {
      at.p = 0;
      if (++at.h == c.heads) {
        at.h = 0;
        do {
          if (++at.b >= c.batch) {
            more = false;
            return;
          }
          seq = seq_info(c, at.b, max_q);
        } while (seq.n == 0);
      }
    }
    settle(c, tpi, wl, wr);
  }
};

// What CTA c left in parts, for the kernel that joins them. Slot 2 c holds the end (or
// the middle) of an item that an earlier CTA began, slot 2 c + 1 the beginning of one that
// a later CTA goes on with.
struct PartInfo {
  int begins;    // slot 2 c + 1 is in use
  int token0;    // ... its item's first packed row,
  int tokens;    //     its tokens,
  int head;      //     its key head
  int goes_on;   // slot 2 c is in use and does not finish its item
  int pad[3];
};

__device__ __forceinline__ void write_part_info(const PagedView& c, int tpi, int max_q,
                                                const Stretch& stretch, PartInfo* parts) {
  const Bound a = stretch.at, e = stretch.end;
  PartInfo info{};
  const bool same = a.b == e.b && a.h == e.h && a.p == e.p;
  if (a.b < c.batch && e.b < c.batch && e.j > 0 && !(same && e.j <= a.j)) {
    if (same && a.j > 0) {
      info.goes_on = 1;
    } else {
      const SeqInfo s = seq_info(c, e.b, max_q);
      info.begins = 1;
      info.token0 = s.begin + e.p * tpi;
      info.tokens = min(tpi, s.n - e.p * tpi);
      info.head = e.h;
    }
  }
  parts[blockIdx.x] = info;
}
#endif

}  // namespace fa
