// fa_paged_chunk.cuh -- attention of longer chunks of new tokens over a paged cache.
//
// The pass is bound by the tensor cores and the exponentials: R query rows do 4 R d
// operations per key, so every K and V tile brought on chip serves as many rows as tensor
// memory holds, 2 x 128. Query rows are packed: row r of a 128-row tile is token
// r / group and query head r % group of one key head's group, so that heads which share
// keys share their tiles too, and a causal chunk's masked corner stays small (256 rows are
// 256 / group tokens). When the group does not divide 128 the last rows of a tile are
// zeros.
//
// Work is shared out along the keys (fa_paged_split.cuh): one persistent CTA per SM, all
// with the same number of key tiles, whatever the mix of long chunks and single tokens; a
// chunk's heavy last rows, or a long context behind a short chunk, cannot leave SMs idle.
//
// Warp roles (at launch every thread holds the same number of registers, then the last
// warpgroup hands some to the others; warps counted from it):
//   softmax         thread r of a warpgroup owns row r of its query tile (TMEM lane r), so its
//                   maximum needs no exchange. A tile's keys go in two halves of 64. At d =
//                   128 a warpgroup per query tile takes them in turn (384 threads), at d =
//                   64 there is one for each half (640 threads).
//   warp 0          K producer: the item's two Q tiles, then K tiles into 2 stages.
//   warp 2          V producer, 2 stages. Both walk the page table by themselves, a window
//                   of pages ahead, one box per page and 64 columns.
//   warp 3          scheduler: the CTA's items.
//   warp 1          MMA issuer. With S_g,h the scores of query tile g and half h of the tile
//                   and PV_g,h their weights' product, it issues for each tile
//                     PV_0,0 S_0,0  PV_1,0 S_1,0  PV_0,1 S_0,1  PV_1,1 S_1,1
//                   each PV that of the tile before. The order runs on across items: the
//                   next item's first scores are computed while this one's outputs leave.
//
// TMEM (512 columns): 64 columns of scores per (g, h) at 128 g + 64 h, whose first 32 the
// weights P take over; behind them O of g, at d = 64 of (g, h). Because a half's scores wait
// only for the product of the half two before, they are there when the softmax has finished
// the half in between: it never waits for the tensor core's round trip, which with
// whole-tile buffers was half of its time. Products into an O run in order; it may be
// rescaled once the product before has landed (a barrier, waited for only when a row's
// reference moves past 2^8, and at the item's end).
//
// The two halves apart at d = 64: the exponentials bound that size (a tile's products take
// half as long as at d = 128, its softmax as long), and two softmax warps per scheduler left
// their unit idle 39 % of the time; with four, 2048 tokens over 16k keys (32 heads) took 306
// us for 365 (310 now, 815 TFLOP/s). Each has a reference, a sum and an O of its own, joined at an
// item's end. At d = 128 tensor memory has no room for four O.
//
// An item with one query tile (a single token among chunks, a short draft, a chunk's last
// tokens) would leave one half of the warps idle and the tensor core waiting for the other.
// There the two groups take the key tiles in turn, both with query tile 0, and the first
// warpgroup joins the partial outputs out of tensor memory by their references and sums.
// Warps none of whose rows is a real query skip the softmax.
//
// Scores are in base 2. One row sum, of the unrounded weights, gives L and normalises O, while
// the product multiplies weights rounded to 16 bits: O is off by at most half a step of its
// keys' values on top of its own rounding. A second sum, of the rounded weights, would make O
// an exact average with them, so that the rounding of a weight that dominates its row
// cancels. For rows of 2000 random keys with scores of standard deviation 1 / 3 / 6 / 10 the mean
// relative error in bf16 (before O is rounded) is 0.0017 / 0.0013 / 0.0011 / 0.0008 with one
// sum and 0.0017 / 0.0012 / 0.0007 / 0.0004 with two, the largest 0.0039 and 0.0034. The loop
// is bound by its instructions, of which the second sum is three of eight per pair: 2048
// tokens over 16k keys take 459 us for 435 at d = 128, 351 for 311 at d = 64. V rows of keys
// that no row of the item sees are zeroed in shared memory before they are multiplied by
// weights of 0.
#pragma once

#include "fa_paged_step.cuh"

namespace fa {

// Warps by head size.
template <int D>
struct ChunkRoles {
  static constexpr int kHalves = D == 64 ? 2 : 1;  // softmax warpgroups per query tile
  static constexpr int kSoftmaxWarps = 8 * kHalves;
  static constexpr int kK = kSoftmaxWarps, kMma = kK + 1, kV = kK + 2, kScheduler = kK + 3;
  static constexpr int kThreads = 32 * (kSoftmaxWarps + 4);
  // Registers per thread at launch (the most that many threads can have), then those of
  // the softmax warpgroups and of the last one; the sums must be equal.
  static constexpr int kLaunchRegs = D == 64 ? 96 : 168;
  static constexpr int kSoftmaxRegs = D == 64 ? 104 : 216;
  static constexpr int kSmallRegs = D == 64 ? 64 : 72;
  static_assert(2 * kHalves * kSoftmaxRegs + kSmallRegs == (2 * kHalves + 1) * kLaunchRegs,
                "register split");
};
constexpr float kChunkRescaleSlack = 8.0f;
constexpr int kChunkRows = 256;  // rows of an item
constexpr int kChunkKStages = 2;
constexpr int kChunkVStages = 2;

template <int D>
struct ChunkLayout {
  static constexpr uint32_t kTileBytes = kKeyTile * D * 2;
  static constexpr uint32_t kChunkBytes = kKeyTile * 128;  // 128 rows x 64 values
  static constexpr uint32_t kQ = 0;                        // 2 tiles
  static constexpr uint32_t kK = kQ + 2 * kTileBytes;
  static constexpr uint32_t kV = kK + kChunkKStages * kTileBytes;
  static constexpr uint32_t kOut = kV + kChunkVStages * kTileBytes;  // 4 KB per softmax warp
  static constexpr uint32_t kItems = kOut + 8 * 4096;  // (of the warps that store)
  // [warpgroup - 1][row] (reference, sum) of the softmax warpgroups that do not store
  static constexpr uint32_t kJoin = kItems + kItemSlots * sizeof(Item);
  static constexpr uint32_t kBar = kJoin + (2 * ChunkRoles<D>::kHalves - 1) * 128 * 8;
  static constexpr int bQFull = 0, bQEmpty = 1, bKFull = 2, bKEmpty = bKFull + kChunkKStages,
                       bVFull = bKEmpty + kChunkKStages, bVEmpty = bVFull + kChunkVStages,
                       bSFull = bVEmpty + kChunkVStages,  // + 2 g + h, as the next two
                       bPFull = bSFull + 4, bDone = bPFull + 4, bJoin = bDone + 4,
                       bJoined = bJoin + 1,
                       bPair = bJoined + 1, bPaired = bPair + 2,  // + group
                       bItems = bPaired + 2,
                       kNumBars = bItems + 2 * kItemSlots;
  static constexpr uint32_t kTmemSlot = kBar + kNumBars * 8;
  static constexpr uint32_t kAbort = kTmemSlot + 8;
  static constexpr uint32_t kBytes = kAbort + 8 + 1024;
  // at least 120 KB, so that one CTA and its 512 TMEM columns sit on each SM
  static constexpr uint32_t kSmem = kBytes > 120 * 1024 ? kBytes : 120 * 1024;
  static constexpr uint32_t tS = 0;    // + 128 * warpgroup + 64 * half
  static constexpr uint32_t tO = 256;  // + D * group, or 64 * (2 * group + half) at d = 64
};

// The key tiles that each warpgroup of an item takes part in, within the CTA's part.
struct ChunkTiles {
  bool one;          // one query tile: group g takes tiles first + g, first + g + 2, ...
  int lo[2], hi[2];  // otherwise query tile g takes [lo, hi); lo >= hi: none
  int first, last;   // the union, [first, last)

  __device__ __forceinline__ ChunkTiles(const Item& w, int tpt, int wl, int wr) {
    first = w.keys.first + w.j0;
    last = w.keys.first + w.j1;
    one = (2 * w.p + 1) * tpt >= w.n;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const KeyRange r = one ? KeyRange{0, 0, first + g, last - first - g}
                             : item_keys(2 * w.p + g, tpt, w.n, w.nk, wl, wr);
      lo[g] = max(first, r.first);
      hi[g] = min(last, r.first + r.count);
    }
  }
  __device__ __forceinline__ int step() const { return one ? 2 : 1; }
  __device__ __forceinline__ bool in(int g, int tile) const {
    const int l = g ? lo[1] : lo[0], h = g ? hi[1] : hi[0];
    return tile >= l && tile < h && (!one || ((tile - l) & 1) == 0);
  }
  __device__ __forceinline__ bool last_of(int g, int tile) const {
    return tile + step() >= (g ? hi[1] : hi[0]);
  }
  __device__ __forceinline__ bool any(int g) const { return g ? lo[1] < hi[1] : lo[0] < hi[0]; }
};

template <int D, bool BF16>
__global__ void __launch_bounds__(ChunkRoles<D>::kThreads, 1)
    fa_paged_chunk_kernel(const __grid_constant__ CUtensorMap tmQ,
                          const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ CUtensorMap tmO,
                          const __grid_constant__ CUtensorMap tmPart, const PagedView c,
                          uint16_t* __restrict__ O, Strides so, float* __restrict__ L,
                          float* __restrict__ Lpart,
                          PartInfo* __restrict__ parts, int group, int max_q, int wl, int wr,
                          int least,
                          float scale_log2) {
  using Lay = ChunkLayout<D>;
  using Roles = ChunkRoles<D>;
  constexpr bool kOwn = Roles::kHalves == 2;  // a half of the keys has an O of its own
  // Of every 16 exponential pairs, kPolyPairs go to the FMA pipe: 2048 tokens over 16k keys
  // (32 heads) take 446 / 451 / 429 / 435 / 464 us at d = 128 with 0 / 1 / 2 / 4 / 8 of them,
  // 324 / 317 / 310 / 311 / 342 at d = 64. The polynomial clamps its argument at -125, where it
  // gives exactly kPolyLeast; that is taken off again, so that a masked score's weight is 0:
  // 2^-125 is a bf16 number, and a large value of a key that the row does not see would show
  // in O. (A weight above 2^-101 loses nothing by it, others less than 2^-125. Masked tiles
  // wholly on the exponential unit, as in the forward, cost two loops: 447 us for 439.)
  constexpr int kPolyPairs = 2;
  constexpr int kPolyStride = 16 / kPolyPairs;
  constexpr float kPolyLeast = kExp2C0 * 0x1p-125f;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t pad = ((raw_base + 1023u) & ~1023u) - raw_base;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw_base + pad;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // uniform
  const int lane = threadIdx.x & 31;
  const int tpt = kKeyTile / group;  // tokens of a query tile
  // x / group for x < 128: ceil(2^16 / group) errs by less than 128 / 2^16 of a unit
  const int by_group = (65535 + group) / group;
  const int tpi = 2 * tpt;           // tokens of an item
  auto bar = [&](int i) -> uint32_t { return sbase + Lay::kBar + 8u * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::kAbort);

  dependents_may_launch();
  if (threadIdx.x == 0) {
    mbar_init(bar(Lay::bQFull), 1);
    mbar_init(bar(Lay::bQEmpty), 1);
    for (int s = 0; s < kChunkKStages; ++s) {
      mbar_init(bar(Lay::bKFull + s), 1);
      mbar_init(bar(Lay::bKEmpty + s), 1);
    }
    for (int s = 0; s < kChunkVStages; ++s) {
      mbar_init(bar(Lay::bVFull + s), 1);
      mbar_init(bar(Lay::bVEmpty + s), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(Lay::bSFull + i), 1);
      mbar_init(bar(Lay::bPFull + i), 128);
      mbar_init(bar(Lay::bDone + i), 1);
    }
    mbar_init(bar(Lay::bJoin), 128 * (2 * Roles::kHalves - 1));
    mbar_init(bar(Lay::bJoined), 128);
    for (int g = 0; g < 2; ++g) {
      mbar_init(bar(Lay::bPair + g), 128);
      mbar_init(bar(Lay::bPaired + g), 128);
    }
    item_ring_init(bar(Lay::bItems), Roles::kSoftmaxWarps + 3);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == Roles::kMma) {
    tmem_alloc(sbase + Lay::kTmemSlot, 512);
    tmem_relinquish();
  }
  // rows of the Q tiles that no box fills stay zero
  if (tpt * group < kKeyTile)
    for (uint32_t i = threadIdx.x; i < 2 * Lay::kTileBytes / 16; i += Roles::kThreads)
      *reinterpret_cast<uint4*>(smem + Lay::kQ + i * 16) = make_uint4(0u, 0u, 0u, 0u);
  fence_async_smem();
  dependency_wait();
  Scheduler<false> schedule(c, tpi, max_q, wl, wr);
  if (warp == Roles::kScheduler) schedule.locate(least);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + Lay::kTmemSlot);
  ItemRing ring(sbase + Lay::kItems, bar(Lay::bItems));
  Item w;
  bool ok = true;

  if (warp >= Roles::kSoftmaxWarps) setmaxnreg_dec<Roles::kSmallRegs>();  // the last warpgroup
  if (warp == Roles::kScheduler) {
    schedule.run(ring, abort_flag, parts);
  } else if (warp == Roles::kK || warp == Roles::kV) {
    // ---------------------------------------------------------------- producers
    const bool is_k = warp == Roles::kK;
    const CUtensorMap* map = is_k ? &tmK : &tmV;
    const int stages = is_k ? kChunkKStages : kChunkVStages;
    const uint32_t tiles = sbase + (is_k ? Lay::kK : Lay::kV);
    const int full = is_k ? Lay::bKFull : Lay::bVFull, empty = is_k ? Lay::bKEmpty : Lay::bVEmpty;
    if (lane == 0) {
      tma_prefetch(map);
      if (is_k) tma_prefetch(&tmQ);
    }
    __syncwarp();
    int st = 0, item = 0;
    uint32_t phase = 1;  // of the stage's empty barrier: the first pass finds it free
    PageWindow win;
    win.bad = false;
    while (ok && __all_sync(0xffffffffu, ring.get(&w, &ok, abort_flag))) {
      ring.read(lane == 0);
      if (w.j0 >= w.j1) continue;
      const int first = w.keys.first + w.j0;
      win.start(c, w.b, first * kKeyTile >> c.page_shift, lane);
      if (is_k) {
        ok = item == 0 ||
             mbar_wait(bar(Lay::bQEmpty), static_cast<uint32_t>(item - 1) & 1, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          // both tiles, or the only one
          const int q_tiles = (2 * w.p + 1) * tpt >= w.n ? 1 : 2;
          mbar_expect_tx(bar(Lay::bQFull), static_cast<uint32_t>(q_tiles * tpt * group) * D * 2);
          for (int g = 0; g < q_tiles; ++g)
            for (int i = 0; i < D / 64; ++i)
              tma_load_4d(sbase + Lay::kQ + g * Lay::kTileBytes + i * Lay::kChunkBytes, &tmQ,
                          i * 64, 0, w.begin + (2 * w.p + g) * tpt, w.h, bar(Lay::bQFull));
        }
        __syncwarp();
        ++item;
      }
      for (int tile = first; tile < w.keys.first + w.j1; ++tile) {
        const TilePages pages(tile, w.keys, c.page_shift);
        ok = mbar_wait(bar(empty + st), phase, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        if (lane == 0)
          mbar_expect_tx(bar(full + st),
                         static_cast<uint32_t>(pages.count * pages.rows) * D * 2);
        __syncwarp();
        load_tile_pages<D>(pages, tile, c.page_shift, win, map, tiles + st * Lay::kTileBytes,
                           bar(full + st), w.h, lane);
        if (++st == stages) {
          st = 0;
          phase ^= 1;
        }
      }
    }
    if (win.bad) atomicExch(&g_fa_status, kStatusInvalid);
  } else if (warp == Roles::kMma) {
    // -------------------------------------------------------------- MMA issuer
    {
      constexpr uint32_t idesc_s = idesc_f16_f32(kKeyTile, 64, BF16, false, false);
      constexpr uint32_t idesc_o = idesc_f16_f32(kKeyTile, D, BF16, false, true);
      // Where every (g, h) owes a product and sees the tile -- all but an item's edges -- the
      // turns are laid out straight: this one thread feeds the tensor core, and with run-time
      // g and h its own instructions take twice the time of what it issues. All other cases
      // share one body with run-time g and h: copies for each made this warp's code 16 KB,
      // and it and the softmax warps' kept pushing each other out of the instruction cache,
      // at three times the cost for all code that runs once an item.
      int ks = 0, item = 0;
      uint32_t kphase = 0, pphase = 0;  // pphase: bit 2 g + h
      // what (g, h) owes: 0 nothing, else 1 (an item's first product: O is overwritten) or 2,
      // + 4 times the V tile's index among the CTA's
      uint32_t owed[4] = {0, 0, 0, 0};
      uint32_t vi = 0;  // V tiles before this one
      bool more = true;
      while (ok && more) {
        more = __all_sync(0xffffffffu, ring.get(&w, &ok, abort_flag));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (more) ring.read(lane == 0);
        // First the products that the item before is owed, its softmax warps wait for them
        // before they read on: a turn without scores. It is all that an item without tiles,
        // like the end, is read for.
        const bool work = __all_sync(0xffffffffu, more && w.j0 < w.j1);
        ChunkTiles t(w, tpt, wl, wr);
        t.one = __all_sync(0xffffffffu, t.one);
        t.first = __shfl_sync(0xffffffffu, t.first, 0);
        t.last = __shfl_sync(0xffffffffu, t.last, 0);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          t.lo[g] = __shfl_sync(0xffffffffu, t.lo[g], 0);
          t.hi[g] = __shfl_sync(0xffffffffu, t.hi[g], 0);
        }
        const int last = work ? t.last : t.first;
        const bool owing = (owed[0] | owed[1] | owed[2] | owed[3]) != 0;
        for (int tile = owing ? t.first - 1 : t.first; ok && tile < last; ++tile) {
          if (!t.one && tile > t.first && owed[0] && owed[1] && owed[2] && owed[3] &&
              t.in(0, tile) && t.in(1, tile)) {
            const uint32_t v = vi - 1;  // owed by all four
            const uint32_t vs = v % kChunkVStages;
            const SmemDesc dv =
                smem_desc(sbase + Lay::kV + vs * Lay::kTileBytes, Lay::kChunkBytes, 1024);
            const SmemDesc dk = smem_desc(sbase + Lay::kK + ks * Lay::kTileBytes, 16, 1024);
#pragma unroll
            for (int turn = 0; turn < 4; ++turn) {
              const int h = turn >> 1, g = turn & 1, i = 2 * g + h;
              const uint32_t d_s = tmem + Lay::tS + g * 128 + h * 64, d_o = tmem + Lay::tO + (kOwn ? i : g) * D;
              ok = warp_wait(bar(Lay::bPFull + i), pphase >> i & 1u, abort_flag) &&
                   (turn > 0 || (warp_wait(bar(Lay::bVFull + vs), (v / kChunkVStages) & 1,
                                           abort_flag) &&
                                 warp_wait(bar(Lay::bKFull + ks), kphase, abort_flag)));
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int k = 0; k < 4; ++k)
                warp_mma_ts(d_o, d_s + k * 8, dv, h * 8192 + k * 2048, idesc_o,
                       k > 0 ? 1u : (owed[i] & 3u) - 1u);
              warp_mma_commit(bar(Lay::bDone + i));
              const SmemDesc dq = smem_desc(sbase + Lay::kQ + g * Lay::kTileBytes, 16, 1024);
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const uint32_t koff = (k >> 2) * Lay::kChunkBytes + (k & 3) * 32;
                warp_mma_ss(d_s, dq, koff, dk, h * 8192 + koff, idesc_s,
                       k > 0 ? 1u : 0u);
              }
              warp_mma_commit(bar(Lay::bSFull + i));
              owed[i] = 2u + 4u * vi;
            }
            if (!ok) break;
            warp_mma_commit(bar(Lay::bVEmpty + vs));
            warp_mma_commit(bar(Lay::bKEmpty + ks));
            pphase ^= 15u;
            ++vi;
            if (++ks == kChunkKStages) {
              ks = 0;
              kphase ^= 1;
            }
            continue;
          }
          const bool alone = t.one && tile > t.first;
          bool k_waited = false;
#pragma unroll 1
          for (int turn = 0; turn < 4; ++turn) {
            const int h = turn >> 1, g = turn & 1, i = 2 * g + h;
            if (alone && g != ((tile - t.first) & 1)) continue;
            const uint32_t what = g ? (h ? owed[3] : owed[2]) : (h ? owed[1] : owed[0]);
            const uint32_t d_s = tmem + Lay::tS + g * 128 + h * 64;
            uint32_t next = 0;
            if (what != 0) {
              const uint32_t v = what >> 2;
              const uint32_t vs = v % kChunkVStages;
              ok = warp_wait(bar(Lay::bPFull + i), pphase >> i & 1u, abort_flag) &&
                   warp_wait(bar(Lay::bVFull + vs), (v / kChunkVStages) & 1, abort_flag);
              if (!ok) break;
              tc_fence_after();
              const SmemDesc dv = smem_desc(sbase + Lay::kV + vs * Lay::kTileBytes + h * 8192,
                                              Lay::kChunkBytes, 1024);
              const uint32_t d_o = tmem + Lay::tO + (kOwn ? i : g) * D;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                warp_mma_ts(d_o, d_s + k * 8, dv, k * 2048, idesc_o,
                       k > 0 ? 1u : (what & 3u) - 1u);
              warp_mma_commit(bar(Lay::bDone + i));
              pphase ^= 1u << i;
              // the V tile is released with the last product that is owed for it
              bool others = false;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                others = others || (k != i && owed[k] != 0 && owed[k] >> 2 == v);
              if (!others) warp_mma_commit(bar(Lay::bVEmpty + vs));
            }
            if (t.in(g, tile)) {
              if (tile == t.first)
                ok = warp_wait(bar(Lay::bQFull), static_cast<uint32_t>(item) & 1, abort_flag);
              if (ok && !k_waited) ok = warp_wait(bar(Lay::bKFull + ks), kphase, abort_flag);
              if (!ok) break;
              k_waited = true;
              tc_fence_after();
              const SmemDesc dq =
                  smem_desc(sbase + Lay::kQ + (t.one ? 0 : g) * Lay::kTileBytes, 16, 1024);
              const SmemDesc dk =
                  smem_desc(sbase + Lay::kK + ks * Lay::kTileBytes + h * 8192, 16, 1024);
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const uint32_t koff = (k >> 2) * Lay::kChunkBytes + (k & 3) * 32;
                warp_mma_ss(d_s, dq, koff, dk, koff, idesc_s, k > 0 ? 1u : 0u);
              }
              warp_mma_commit(bar(Lay::bSFull + i));
              next = ((kOwn || h == 0) && tile == (g ? t.lo[1] : t.lo[0]) ? 1u : 2u) + 4u * vi;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) owed[k] = k == i ? next : owed[k];
          }
          if (!ok) break;
          if (tile < t.first) continue;
          warp_mma_commit(bar(Lay::bKEmpty + ks));
          ++vi;
          if (++ks == kChunkKStages) {
            ks = 0;
            kphase ^= 1;
          }
        }
        if (!ok) break;
        if (work) {
          warp_mma_commit(bar(Lay::bQEmpty));
          ++item;
        }
      }
    }
  } else if (warp < Roles::kSoftmaxWarps) {
    // ----------------------------------------------------------------- softmax
    setmaxnreg_inc<Roles::kSoftmaxRegs>();
    const int g = warp / (4 * Roles::kHalves);
    const int half = kOwn ? warp >> 2 & 1 : 0;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;  // row of the query tile = TMEM lane
    const int tr = r * by_group >> 16;  // its token in the tile (tpt or more: a row of zeros)
    const int head_in = r - tr * group;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t o_cols = Lay::tO + (kOwn ? 2 * g + half : g) * D;
    const uint64_t c2 = f2_pack(scale_log2, scale_log2);
    uint32_t used = 0;  // tiles of this group before: phases of its S, P and product barriers
    uint32_t jphase = 0, pair_phase = 0;
    int vi = 0;  // V tiles of the CTA before this item
    while (ok) {
      if (!__all_sync(0xffffffffu, ring.get(&w, &ok, abort_flag))) break;
      ring.read(lane == 0);
      const int off = w.nk - w.n;
      bool one;
      int lo, hi, first;
      {
        const ChunkTiles t(w, tpt, wl, wr);
        one = t.one;
        lo = g ? t.lo[1] : t.lo[0];
        hi = g ? t.hi[1] : t.hi[0];
        first = t.first;
      }
      const int step = one ? 2 : 1;
      const int tok0 = (2 * w.p + (one ? 0 : g)) * tpt;  // first token of the query tile
      // whether any row of this warp is a query
      const bool busy = quarter * 32 < min(tpt, w.n - tok0) * group;
      // keys that every row of the query tile sees, and this thread's row
      const int all_lo = min(tok0 + tpt, w.n) - 1 + off - wl;
      const int all_hi = min(w.nk - 1, tok0 + off + wr);
      const int mid = tok0 + tr + off;
      const int row_lo = mid - wl, row_hi = min(w.nk - 1, mid + wr);
      float m = -INFINITY;  // running reference, base-2 scaled units
      float l = 0.f;        // row sum of p
      for (int tile = lo; ok && tile < hi; tile += step, ++used) {
#pragma unroll 1
        for (int h = half; h < (kOwn ? half + 1 : 2); ++h) {
          const uint32_t bars = 2 * g + h;
          ok = __all_sync(0xffffffffu, mbar_wait(bar(Lay::bSFull + bars), used & 1, abort_flag));
          if (!ok) break;
          tc_fence_after();
          const uint32_t s_cols = Lay::tS + g * 128 + h * 64;
          const int key0 = tile * kKeyTile + h * 64;
          const bool edge = key0 < all_lo || key0 + 63 > all_hi;
          if (edge && (key0 < w.keys.lo || key0 + 63 > w.keys.hi)) {
            // keys that no row of the item sees: their V rows become zeros (by all warps)
            const int v = vi + tile - first;
            ok = __all_sync(0xffffffffu,
                            mbar_wait(bar(Lay::bVFull + v % kChunkVStages),
                                      static_cast<uint32_t>(v / kChunkVStages) & 1, abort_flag));
            if (!ok) break;
            const int key = key0 + (r & 63);
            if (key < w.keys.lo || key > w.keys.hi) {  // rows r and r + 64: half the columns each
              const uint32_t row = sbase + Lay::kV + (v % kChunkVStages) * Lay::kTileBytes +
                                   (key - tile * kKeyTile) * 128;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                const int at = i + (r >> 6) * (D / 16);  // 16-byte piece of the row
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                 row + (at >> 3) * Lay::kChunkBytes + (at & 7) * 16),
                             "r"(0)
                             : "memory");
              }
            }
            fence_async_smem();
          }
          if (!busy) {
            tc_fence_before();
            mbar_arrive(bar(Lay::bPFull + bars));
            continue;
          }
          // An edge of the mask: columns [first_col, last_col] of the row are visible, the
          // others become -inf in tensor memory. 32 columns at a time in a loop, off the main
          // path: unrolled on the registers below it tripled an edge tile's time, most of it
          // spent fetching instructions that few tiles run.
          if (edge) {
            const int first_col = row_lo - key0, last_col = row_hi - key0;
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
              const int lo_bit = first_col - 32 * i, hi_bit = last_col - 32 * i;
              uint32_t seen = hi_bit < 0 ? 0u : 0xffffffffu >> (31 - min(hi_bit, 31));
              seen &= lo_bit > 31 ? 0u : 0xffffffffu << max(lo_bit, 0);
              if (__all_sync(0xffffffffu, seen == 0xffffffffu)) continue;
              uint32_t x[32];
              tmem_ld32(lane_base + s_cols + i * 32, x);
              tmem_wait_ld();
              reg_fence32(x);
#pragma unroll
              for (int k = 0; k < 32; ++k) x[k] = seen >> k & 1 ? x[k] : 0xff800000u;
              tmem_st32(lane_base + s_cols + i * 32, x);
            }
            tmem_wait_st();
          }
          // row maximum over four independent chains; at d = 64 the upper half of the scores is
          // read again for its exponentials, so that 32 stay in registers
          constexpr int kHeld = kOwn ? 32 : 64;
          float s[kHeld];
          float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int part = 64 - kHeld; part >= 0; part -= kHeld) {
            uint32_t sr[kHeld];
#pragma unroll
            for (int i = 0; i < kHeld; i += 32) tmem_ld32(lane_base + s_cols + part + i, sr + i);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < kHeld; i += 32) reg_fence32(sr + i);
#pragma unroll
            for (int e = 0; e < kHeld; ++e) s[e] = __uint_as_float(sr[e]);
#pragma unroll
            for (int i = 0; i < kHeld; i += 8) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mq[k] = fmax3_nan(mq[k], s[i + 2 * k], s[i + 2 * k + 1]);
            }
          }
          const float mx = fmax3_nan(fmax3_nan(mq[0], mq[1], mq[2]), mq[3], mq[3]);
          const float cand = mx * scale_log2;
          const float m_new = (cand > m + kChunkRescaleSlack) ? cand : m;
          // a row that has seen no key keeps m = -inf: alpha = 1, and 0 is subtracted
          const bool empty_row = m_new == -INFINITY;
          const float alpha = empty_row ? 1.f : ex2_approx(m - m_new);  // 0 at first
          const float m_sub = empty_row ? 0.f : m_new;
          const uint64_t nm2 = f2_pack(-m_sub, -m_sub);
          uint64_t sum2[2] = {0, 0};  // packed +0.0f
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t pk[16];
            if (kOwn && j == 1) {
              uint32_t sr[32];
              tmem_ld32(lane_base + s_cols + 32, sr);
              tmem_wait_ld();
              reg_fence32(sr);
#pragma unroll
              for (int e = 0; e < 32; ++e) s[e] = __uint_as_float(sr[e]);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int e = j * (kHeld - 32) + 2 * i;
              float x0, x1;
              f2_unpack(f2_fma(f2_pack(s[e], s[e + 1]), c2, nm2), x0, x1);
              float p0, p1;
              if (i % kPolyStride == kPolyStride - 1) {
                ex2_poly_pair(x0, x1, p0, p1);
                f2_unpack(f2_add(f2_pack(p0, p1), f2_pack(-kPolyLeast, -kPolyLeast)), p0, p1);
              } else {
                p0 = ex2_approx(x0);
                p1 = ex2_approx(x1);
              }
              pk[i] = pack2<BF16>(p0, p1);
              sum2[i & 1] = f2_add(sum2[i & 1], f2_pack(p0, p1));
            }
            tmem_st16(lane_base + s_cols + j * 16, pk);
          }
          float a0, a1;
          f2_unpack(f2_add(sum2[0], sum2[1]), a0, a1);
          // a NaN score comes by the maximum: the polynomial's clamp drops it
          l = l * alpha + (isnan(mx) ? mx : a0 + a1);
          // a reference moved, and O holds products: once the last of them has landed (that
          // of the half before; the one before that landed ahead of these scores)
          if ((tile > lo || (!kOwn && h > 0)) && __any_sync(0xffffffffu, alpha != 1.f)) {
            ok = __all_sync(0xffffffffu, mbar_wait(bar(Lay::bDone + (kOwn ? bars : bars ^ 1)),
                                                   (!kOwn && h ? used : used - 1) & 1,
                                                   abort_flag));
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int i = 0; i < D; i += 32) {
              uint32_t o[32];
              tmem_ld32(lane_base + o_cols + i, o);
              tmem_wait_ld();
              reg_fence32(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(lane_base + o_cols + i, o);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(bar(Lay::bPFull + bars));
          m = m_new;
        }
      }
      vi += w.j1 - w.j0;
      const bool some = lo < hi;
      ok = __all_sync(
          0xffffffffu,
          ok && (!some || (mbar_wait(bar(Lay::bDone + 2 * g + half), (used - 1) & 1, abort_flag) &&
                           (kOwn || mbar_wait(bar(Lay::bDone + 2 * g + 1), (used - 1) & 1,
                                              abort_flag)))));
      tc_fence_after();
      // Warpgroups that share a query tile -- all where it is the item's only one, else, at d =
      // 64, the two halves of its keys -- join their sums; the first of them stores.
      const int me = kOwn ? 2 * g + half : g;
      const int sharing = one ? 2 * Roles::kHalves : Roles::kHalves;
      const bool stores = me % sharing == 0;
      float2* sums = reinterpret_cast<float2*>(smem + Lay::kJoin) + r;
      float top = m;
      if (sharing > 1 && ok) {
        const uint32_t told = bar(one ? Lay::bJoin : Lay::bPair + g);
        if (!stores) {
          sums[(me - 1) * 128] = make_float2(m, l);
          mbar_arrive(told);
        } else {
          ok = __all_sync(0xffffffffu, mbar_wait(told, one ? jphase : pair_phase, abort_flag));
          tc_fence_after();
#pragma unroll 1
          for (int i = me + 1; i < me + sharing; ++i) top = fmaxf(top, sums[(i - 1) * 128].x);
        }
      }
      // Rows that see no key keep the reference -inf and sums of 0: O = 0, L = -inf. A NaN
      // among the scores is in the sum and makes O and L NaN.
      const float top_sub = top == -INFINITY ? 0.f : top;
      float inv_l = ex2_approx(m - top_sub);
      if (stores) {
        l *= inv_l;
#pragma unroll 1
        for (int i = me + 1; i < me + sharing; ++i) {
          const float2 other = sums[(i - 1) * 128];
          const float f = ex2_approx(other.x - top_sub);
          l = fmaf(other.y, f, l);
          sums[(i - 1) * 128].x = f;  // read again by this thread, with that warpgroup's O
        }
      }
      const float L2 = top_sub + log2f(l);
      const float inv_sum = l == 0.f ? 0.f : 1.f / l;
      inv_l *= inv_sum;
      // O / l: a thread holds a row, a store wants rows' neighbours side by side, so 128
      // bytes of each row (64 columns, or 32 of a part in fp32) at a time go through the
      // warp's 4 KB of shared memory, 128-byte-swizzled, and leave in one TMA store (of a
      // part's rows, or of whole tokens when 32 rows are that) or, at a sequence's ragged end,
      // as four rows an instruction. (Straight from the rows' threads an item's store took
      // 3000 to 8000 cycles.)
      if (ok && busy && stores) {
        const bool whole = w.j0 == 0 && w.j1 == w.keys.count;
        const bool other_some = one && first + 1 < w.keys.first + w.j1;
        const int rows = min(tpt, w.n - tok0) * group;  // of the query tile
        const int row0 = quarter * 32;
        const int tok_row0 = row0 * by_group >> 16;  // token of the warp's first row
        const int slot_row = (w.j0 > 0 ? 2 * blockIdx.x : 2 * blockIdx.x + 1) * kChunkRows +
                             (one ? 0 : g * kKeyTile);
        const bool by_tma = !whole || (32 % group == 0 && row0 + 32 <= rows);
        const uint32_t stage = sbase + Lay::kOut + (4 * g + quarter) * 4096;
#pragma unroll 1
        for (int i = 0; i < D; i += 32) {
          float x[32];
          uint32_t o[32];
          if (some) {  // without a key tile O was never written
            tmem_ld32(lane_base + o_cols + i, o);
            tmem_wait_ld();
            reg_fence32(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(o[e]) * inv_l;
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = 0.f;
          }
#pragma unroll 1
          for (int k = me + 1; k < me + sharing; ++k) {
            if (!(one && k >= Roles::kHalves ? other_some : some)) break;
            const float f = sums[(k - 1) * 128].x * inv_sum;
            tmem_ld32(lane_base + Lay::tO + k * D + i, o);
            tmem_wait_ld();
            reg_fence32(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = fmaf(__uint_as_float(o[e]), f, x[e]);
          }
          // the bytes before, of this item or the last, have left
          if (lane == 0 && (!whole || (i & 32) == 0)) bulk_wait_read_all();
          __syncwarp();
          if (whole) {  // half of the row's 128 bytes; they leave after the second half
            const int half = (i >> 5) & 1;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                               stage + lane * 128 + (((half * 4 + e) ^ (lane & 7)) << 4)),
                           "r"(pack2<BF16>(x[8 * e], x[8 * e + 1])),
                           "r"(pack2<BF16>(x[8 * e + 2], x[8 * e + 3])),
                           "r"(pack2<BF16>(x[8 * e + 4], x[8 * e + 5])),
                           "r"(pack2<BF16>(x[8 * e + 6], x[8 * e + 7]))
                           : "memory");
            if (!half) continue;
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                               stage + lane * 128 + ((e ^ (lane & 7)) << 4)),
                           "f"(x[4 * e]), "f"(x[4 * e + 1]), "f"(x[4 * e + 2]), "f"(x[4 * e + 3])
                           : "memory");
          }
          if (by_tma) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (whole)
                tma_store_4d(&tmO, stage, i - 32, 0, w.begin + tok0 + tok_row0, w.h);
              else
                tma_store_2d(&tmPart, stage, i, slot_row + row0);
              bulk_commit();
            }
          } else {
            __syncwarp();
#pragma unroll 1
            for (int e = lane >> 3; e < min(32, rows - row0); e += 4) {
              const int row = row0 + e;
              uint4 y;
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w)
                           : "r"(stage + e * 128 + (((lane & 7) ^ (e & 7)) << 4))
                           : "memory");
              if (row < rows) {
                const int t = row * by_group >> 16;
                *reinterpret_cast<uint4*>(O + static_cast<long>(w.begin + tok0 + t) * so.sn +
                                          (w.h * group + row - t * group) * so.sh + (i - 32) +
                                          (lane & 7) * 8) = y;
              }
            }
            __syncwarp();
          }
        }
        if (r < rows) {
          if (whole)
            L[static_cast<long>(w.h * group + head_in) * c.tokens + w.begin + tok0 + tr] =
                L2 * 0.69314718055994530942f;
          else
            Lpart[slot_row + r] = L2;
        }
      }
      tc_fence_before();
      if (sharing > 1 && ok) {  // the others' sums and O have been read
        const uint32_t read = bar(one ? Lay::bJoined : Lay::bPaired + g);
        if (stores)
          mbar_arrive(read);
        else
          ok = __all_sync(0xffffffffu, mbar_wait(read, one ? jphase : pair_phase, abort_flag));
        if (one)
          jphase ^= 1;
        else
          pair_phase ^= 1;
      }
    }
    if (lane == 0) bulk_wait_all();  // what left by TMA is out before the CTA ends
  }

  tc_fence_before();
  __syncthreads();
  if (warp == Roles::kMma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace fa
