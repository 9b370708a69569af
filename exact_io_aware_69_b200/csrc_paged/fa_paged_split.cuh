// fa_paged_split.cuh -- how the attention kernels share a ragged batch out.
//
// An item is what one pass over keys serves: up to `tpi` consecutive new tokens of one
// sequence, all query heads of one key head. Its cost is the key tiles (128 keys) that its
// rows see, plus `start` tiles for starting and finishing it. The items, ordered by (sequence,
// key head, place in the sequence), lie end to end on a line of cost, and CTA c of C takes
// the stretch [W c / C, W (c + 1) / C) of it: every CTA gets the same work whatever the
// lengths, an item that crosses a boundary is computed in parts, and each CTA has at most
// two parts (its first item's end, its last item's beginning). A boundary within an
// item's first `start` units moves to the item's start, so that no part is empty.
//
// The split depends only on the lengths, the mask and the grid, so the parts and the order
// in which they are joined -- and with them every rounding -- are the same on every call.
// One warp of every CTA, the scheduler, finds the CTA's stretch from the batch's lengths (no
// launch of its own, nothing to keep in step with the lengths) and hands the items to the
// other warps through a ring in shared memory.
#pragma once

#ifdef __CUDACC__
#include "fa_paged_common.cuh"
#endif

namespace fa {

constexpr int kKeyTile = 128;
// Starting and finishing an item in key tiles' time: its first scores wait for its first
// keys, and its last product is followed by the sums and the store. 64 single tokens over
// 300 to 16,384 keys take 160 / 163 / 165 us with 2 / 3 / 4; prompts of 100 to 2000 tokens
// with and without single tokens 73.7 / 73.9 / 72.2 and 113 / 103 / 107 us (d = 64),
// 117 / 115 / 118 and 135 / 130 / 136 (d = 128).
constexpr int kStepItemCost = 2;
constexpr int kChunkItemCost = 3;

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
__host__ __device__ inline int item_cost(const KeyRange& r, int start) { return r.count + start; }

// CTAs of an attention launch: one per SM of a B200. A fixed count keeps the split the
// same everywhere, and divisions by it are multiplications.
constexpr int kSplitGrid = 148;
// Start of CTA c's stretch of cost W: even stretches, but none shorter than `least`. (The
// host keeps W below kMaxCost, so that 32 bits hold every sum here.)
constexpr long long kMaxCost = 1LL << 31;
__host__ __device__ inline unsigned split_start(unsigned W, unsigned c, unsigned least) {
  const unsigned even = W / kSplitGrid, rest = W - even * kSplitGrid;
  const unsigned x = even >= least ? c * even + (c < rest ? c : rest) : c * least;
  return x < W ? x : W;
}
// The tile at which a boundary `r` units into an item cuts it (0: before the item).
__host__ __device__ inline int split_tile(unsigned r, int start) {
  return r <= static_cast<unsigned>(start) ? 0 : static_cast<int>(r) - start;
}

// An item, or the part of it that falls to a CTA: tiles [first + j0, first + j1).
struct __align__(16) Item {
  int begin, n, nk, b;  // its sequence: first packed row, new tokens, keys, index
  int h, p;             // key head, place in the sequence
  KeyRange keys;
  int j0, j1;
};

#ifdef __CUDACC__
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

// The ring: kItemSlots items, a barrier each for "filled" (one arrival) and "read" (one
// arrival per reading warp).
constexpr int kItemSlots = 3;
struct ItemRing {
  uint32_t items;  // shared address of Item[kItemSlots]
  uint32_t full, empty;
  int slot;
  uint32_t phase;  // of the slot's pass; readers wait for `phase`, the scheduler for its flip

  __device__ __forceinline__ ItemRing(uint32_t items_, uint32_t bars)
      : items(items_), full(bars), empty(bars + 8 * kItemSlots), slot(0), phase(0) {}
  __device__ __forceinline__ void step() {
    if (++slot == kItemSlots) {
      slot = 0;
      phase ^= 1;
    }
  }
  // By one thread.
  __device__ __forceinline__ bool put(const Item& it, volatile int* abort_flag) {
    if (!mbar_wait(empty + 8 * slot, phase ^ 1, abort_flag)) return false;
    const uint32_t at = items + slot * static_cast<uint32_t>(sizeof(Item));
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(it.begin), "r"(it.n),
                 "r"(it.nk), "r"(it.b)
                 : "memory");
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + 16), "r"(it.h), "r"(it.p),
                 "r"(it.keys.lo), "r"(it.keys.hi)
                 : "memory");
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + 32), "r"(it.keys.first),
                 "r"(it.keys.count), "r"(it.j0), "r"(it.j1)
                 : "memory");
    mbar_arrive(full + 8 * slot);
    step();
    return true;
  }
  // By a thread, or by all lanes of a warp. False: there is none left, or the wait gave up
  // (*ok turns false). read() tells the scheduler, once per warp.
  __device__ __forceinline__ bool get(Item* it, bool* ok, volatile int* abort_flag) {
    if (!mbar_wait(full + 8 * slot, phase, abort_flag)) {
      *ok = false;
      return false;
    }
    const uint32_t at = items + slot * static_cast<uint32_t>(sizeof(Item));
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(it->begin), "=r"(it->n), "=r"(it->nk), "=r"(it->b)
                 : "r"(at)
                 : "memory");
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(it->h), "=r"(it->p), "=r"(it->keys.lo), "=r"(it->keys.hi)
                 : "r"(at + 16)
                 : "memory");
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(it->keys.first), "=r"(it->keys.count), "=r"(it->j0), "=r"(it->j1)
                 : "r"(at + 32)
                 : "memory");
    return it->begin >= 0;
  }
  __device__ __forceinline__ void read(bool speaker) {
    if (speaker) mbar_arrive(empty + 8 * slot);
    step();
  }
};
__device__ __forceinline__ void item_ring_init(uint32_t bars, int readers) {
  for (int i = 0; i < kItemSlots; ++i) {
    mbar_init(bars + 8 * i, 1);
    mbar_init(bars + 8 * (kItemSlots + i), static_cast<uint32_t>(readers));
  }
}

// The scheduler: one warp. locate() reads the batch's lengths and finds the CTA's stretch;
// run() puts its items into the ring and writes its PartInfo. ONE_ITEM: every sequence has
// at most tpi new tokens. A CTA's first key waits for locate(), whose instructions come
// cold from L2 at about 17 cycles each: few of them matter more than their kind.
template <bool ONE_ITEM>
struct Scheduler {
  static constexpr int kStart = ONE_ITEM ? kStepItemCost : kChunkItemCost;
  const PagedView& c;
  const int tpi, max_q, wl, wr, lane;
  int base;       // lane i holds sequence base + i
  SeqInfo seq;
  unsigned x0, x1;  // the stretch
  int b, h, p;      // the item at x0
  unsigned at;      // where it starts

  __device__ __forceinline__ Scheduler(const PagedView& c_, int tpi_, int max_q_, int wl_, int wr_)
      : c(c_), tpi(tpi_), max_q(max_q_), wl(wl_), wr(wr_), lane(threadIdx.x & 31) {}

  __device__ __forceinline__ void load(int from) {
    base = from;
    const int i = from + lane;
    seq = SeqInfo{0, 0, 0, true, false};
    if (i < c.batch) seq = seq_info(c, i, max_q);
  }
  __device__ __forceinline__ unsigned cost_of(int place, int n, int nk) const {
    return static_cast<unsigned>(item_cost(item_keys(place, tpi, n, nk, wl, wr), kStart));
  }
  // Cost per key head of this lane's sequence.
  __device__ __forceinline__ unsigned seq_cost() const {
    if (ONE_ITEM) return seq.n > 0 ? cost_of(0, seq.n, seq.nk) : 0;
    // short ones each by its lane, long ones by the warp, one after the other (a lane's turn
    // is ~60 cycles, a sequence's ~400)
    unsigned sum = 0;
    const bool own = seq.n <= 16 * tpi;
    for (int i = 0; own && i * tpi < seq.n; ++i) sum += cost_of(i, seq.n, seq.nk);
    for (unsigned todo = __ballot_sync(0xffffffffu, !own); todo; todo &= todo - 1) {
      const int l = __ffs(todo) - 1;
      const int n = __shfl_sync(0xffffffffu, seq.n, l), nk = __shfl_sync(0xffffffffu, seq.nk, l);
      unsigned part = 0;
      for (int i = lane; i * tpi < n; i += 32) part += cost_of(i, n, nk);
      part = __reduce_add_sync(0xffffffffu, part);
      if (lane == l) sum = part;
    }
    return sum;
  }

  __device__ __forceinline__ void locate(unsigned least) {
    unsigned per_head = 0, own = 0;
    bool falls = false;
    for (int i = 0; i < c.batch; i += 32) {
      load(i);
      falls = falls || seq.falls;
      if (!seq.ok && blockIdx.x == 0) atomicExch(&g_fa_status, kStatusInvalid);
      own = seq_cost();
      per_head += __reduce_add_sync(0xffffffffu, own);
    }
    // With a cu_q that decreases, the sequences may have more rows than the packed ones, by
    // which the host has bounded the sums here: nothing is shared out.
    const unsigned W = __any_sync(0xffffffffu, falls) ? 0 : per_head * c.heads;
    x0 = split_start(W, blockIdx.x, least);
    x1 = split_start(W, blockIdx.x + 1, least);
    at = x0;
    b = c.batch;
    h = p = 0;
    if (x0 >= x1) return;
    // the sequence that holds x0 (one does, unless the lengths change meanwhile)
    unsigned before = 0;
    for (int i = 0; i < c.batch; i += 32) {
      if (c.batch > 32) {
        load(i);
        own = seq_cost();
      }
      unsigned upto = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const unsigned v = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, x0 < before + upto * c.heads);
      if (hit) {
        const int l = __ffs(hit) - 1;
        b = i + l;
        const unsigned w = __shfl_sync(0xffffffffu, own, l);
        unsigned r = x0 - before - (__shfl_sync(0xffffffffu, upto, l) - w) * c.heads;
        if (r >= w) {
          h = static_cast<int>(r / w);
          r -= h * w;
        }
        if (!ONE_ITEM) r = locate_item(l, r);
        at = x0 - r;
        return;
      }
      before += __shfl_sync(0xffffffffu, upto, 31) * c.heads;
    }
  }
  // Sets p to the item of lane l's sequence that holds r; returns the rest.
  __device__ __forceinline__ unsigned locate_item(int l, unsigned r) {
    const int n = __shfl_sync(0xffffffffu, seq.n, l), nk = __shfl_sync(0xffffffffu, seq.nk, l);
    for (int i = lane; (i - lane) * tpi < n; i += 32) {  // finds it: r is below the sum
      unsigned sum = i * tpi < n ? cost_of(i, n, nk) : 0;
      const unsigned cost = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const unsigned v = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += v;
      }
      const unsigned in = __ballot_sync(0xffffffffu, r < sum);
      const int k = in ? __ffs(in) - 1 : 31;
      if (in) {
        p = i - lane + k;
        return r - __shfl_sync(0xffffffffu, sum - cost, k);
      }
      r -= __shfl_sync(0xffffffffu, sum, 31);
    }
    return 0;
  }

  __device__ __forceinline__ void run(ItemRing& ring, volatile int* abort_flag, PartInfo* parts) {
    PartInfo info{};
    Item it;
    bool ok = true;
    while (ok && b < c.batch) {
      // all lanes hold the same item
      it.begin = __shfl_sync(0xffffffffu, seq.begin, b - base);
      it.n = __shfl_sync(0xffffffffu, seq.n, b - base);
      it.nk = __shfl_sync(0xffffffffu, seq.nk, b - base);
      it.b = b;
      bool more = it.n > 0;
      for (; ok && more; p = 0, more = ++h < c.heads) {
        it.h = h;
        for (; ok && more && p * tpi < it.n; ++p) {
          it.p = p;
          it.keys = item_keys(p, tpi, it.n, it.nk, wl, wr);
          const unsigned cost = item_cost(it.keys, kStart);
          it.j0 = at < x0 ? split_tile(x0 - at, kStart) : 0;
          it.j1 = at + cost <= x1 ? it.keys.count : split_tile(x1 - at, kStart);
          if (it.j1 > it.j0 || (it.keys.count == 0 && at + cost <= x1)) {
            if (it.j1 < it.keys.count && blockIdx.x + 1 < kSplitGrid) {  // a later CTA goes on
              info.goes_on = it.j0 > 0;
              info.begins = it.j0 == 0;
              info.token0 = it.begin + p * tpi;
              info.tokens = min(tpi, it.n - p * tpi);
              info.head = h;
            }
            ok = lane != 0 || ring.put(it, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
          }
          at += cost;
          if (at >= x1) more = false;
        }
        if (!more) break;
      }
      if (at >= x1) break;
      h = p = 0;
      if (++b == base + 32 && b < c.batch) load(b);
    }
    if (lane == 0) {
      it.begin = -1;
      if (ok) ring.put(it, abort_flag);
      parts[blockIdx.x] = info;
    }
  }
};
#endif

}  // namespace fa
