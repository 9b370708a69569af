// fa_paged_common.cuh -- what the kernels of libfa_paged.so share: the cache's view on the
// device, a packed token's sequence, a sequence's checked lengths.
#pragma once

#include "fa_band.cuh"
#include "sm100.cuh"

namespace fa {

constexpr int kStatusInvalid = -1;  // == FA_ERR_INVALID

// Dependent launch: a kernel's launch overlaps the end of the one before it, and nothing of
// what that one wrote (or still reads) is touched before dependency_wait. Every thread
// waits, so a kernel has ended only when all before it have.
__device__ __forceinline__ void dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void dependents_may_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

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
  bool falls; // cu_q decreases: other sequences may claim the same rows
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
  s.falls = end < s.begin;
  return s;
}

// max of three, NaN if any of them is
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int s = 16; s >= 1; s >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, s));
  return x;
}
// Reduces C (16 or 32) columns over the 32 lanes at once: v[q] is this lane's value of
// column q; the result is that of column lane % C. Each round halves the columns a lane
// keeps, so C columns take about C shuffles instead of 5 C.
struct MaxOf {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct SumOf {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
template <int C, class Op>
__device__ __forceinline__ float reduce_columns(float* v, int lane, Op op) {
#pragma unroll
  for (int s = C / 2; s >= 1; s >>= 1) {
    const bool upper = (lane & s) != 0;
#pragma unroll
    for (int i = 0; i < s; ++i) {
      const float send = upper ? v[i] : v[i + s];
      const float keep = upper ? v[i + s] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, s));
    }
  }
  if (C == 16) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
  return v[0];
}
// MMAs issued by a whole converged warp, one lane of it elected. A shared-memory descriptor
// is two words of which only the low one (address and leading offset) moves: kept apart
// and the same in all lanes, they can live in uniform registers, where the instruction
// wants them; from a branch of lane 0 every descriptor of every MMA is moved there first.
struct SmemDesc {
  uint32_t lo, hi;
};
// 128-byte swizzle; byte offsets of the leading and the stride dimension.
__device__ __forceinline__ SmemDesc smem_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return {(saddr >> 4 & 0x3FFFu) | (lbo >> 4) << 16, (sbo >> 4) | 1u << 14 | 2u << 29};
}
__device__ __forceinline__ void warp_mma_ss(uint32_t d, SmemDesc a, uint32_t a_bytes, SmemDesc b,
                                            uint32_t b_bytes, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 da, {%1, %2};\n\t"
      "mov.b64 db, {%3, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}\n" ::"r"(d),
      "r"(a.lo + (a_bytes >> 4)), "r"(a.hi), "r"(b.lo + (b_bytes >> 4)), "r"(b.hi), "r"(idesc),
      "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void warp_mma_ts(uint32_t d, uint32_t a, SmemDesc b, uint32_t b_bytes,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 db;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b.lo + (b_bytes >> 4)), "r"(b.hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void warp_mma_commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(
          bar)
      : "memory");
}
// A 4-D tiled load by a whole converged warp (all arguments the same in every lane).
__device__ __forceinline__ void warp_tma_load_4d(uint32_t dst, const CUtensorMap* map, int x,
                                                 int y, int z, int w, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];\n\t}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
// A wait by a whole warp: the same answer in every lane.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}

// Four consecutive 32-bit TMEM columns of this warp's lanes.
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
  tmem_wait_ld();
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]));
}
// Named barrier over `count` threads that tells each whether any of them passed true.
__device__ __forceinline__ bool named_bar_or(int id, int count, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "bar.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(id), "r"(count), "r"(static_cast<uint32_t>(v))
      : "memory");
  return r != 0;
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

// Pages of one sequence as a warp reads them ahead: lane i holds the indexes of pages
// base + i and base + 32 + i, so the table is read one coalesced load at a time, a window
// ahead of its use. Indexes outside the pool become num_pages, whose rows the tensor maps
// read as zeros; *bad is set.
struct PageWindow {
  const int* row;  // the sequence's table row
  int width, pages;
  int base, now, then;
  bool bad;

  __device__ __forceinline__ int fetch(int i) {
    if (i >= width) return pages;
    const int p = row[i];
    return p;
  }
  __device__ __forceinline__ void start(const PagedView& c, int b, int first, int lane) {
    row = c.table + static_cast<long>(b) * c.table_row;
    width = c.table_width;
    pages = c.num_pages;
    base = first;
    now = fetch(base + lane);
    then = fetch(base + 32 + lane);
  }
  // Moves on until page `first` is in the window (calls ascend).
  __device__ __forceinline__ void advance(int first, int lane) {
    while (first >= base + 32) {
      base += 32;
      now = then;
      then = fetch(base + 32 + lane);
    }
  }
  // Page i of the sequence, of the window; the same i in every lane.
  __device__ __forceinline__ int get(int i) {
    int p = __shfl_sync(0xffffffffu, now, (i - base) & 31);
    if (static_cast<unsigned>(p) >= static_cast<unsigned>(pages)) {
      p = pages;
      bad = true;
    }
    return p;
  }
};

}  // namespace fa
