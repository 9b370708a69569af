// fa_paged_step.cuh -- attention of a few new tokens per sequence over a paged cache: the
// decode step and the check of drafted tokens (up to 24 rows per key head, a row being one
// token's query head).
//
// The pass is bound by reading K and V from HBM once: with R rows it does 4 R d
// operations per 4 d bytes of a key. So the work is laid out along the keys
// (fa_paged_split.cuh: one persistent CTA per SM, each with the same number of key tiles),
// a producer warp streams the pages' tiles through a ring without a pause across items,
// and both products go to the tensor cores with the keys on the 128-row side, where a tile
// of them fills an MMA whatever R is:
//   S^T_j = K_j Q^T            M = 128 keys, N = NQ query columns, K = d
//   O^T  += V_j^T P_j^T        M = d (128), N = NQ, K = 128 keys; A = V_j read M-major,
//                              B = P_j^T from shared memory (NQ rows x 128 keys, 16-bit)
// At d = 64 the second MMA keeps M = 128 (its A then reaches into the K tile behind V in
// the stage): lanes 64-127 of O^T hold products nobody reads.
//
// Column q of an item is token q / group and query head q % group of its key head's group,
// so all query heads that share a key head share one pass over it. Columns beyond the
// item's rows hold whatever lies in shared memory: a column's values meet no other's.
//
// Softmax: thread r owns key r of the tile and all query columns. The reference m of a
// column moves only when a score exceeds it by more than 2^8; whether any does is one
// barrier-vote per tile, and only then are the tile's maxima exchanged and O^T rescaled.
// Columns beyond the item's rows are skipped in fours. Two sums per column: of the 16-bit
// weights, which normalises O, and of the unrounded ones, which gives L.
//
// V rows of keys that no row of the item sees -- behind the sequence's end, before its
// window, or in pages that are not loaded -- are zeroed in shared memory, since 0 times
// whatever an unwritten row holds need not be 0.
//
// Warps: four softmax warps, two TMA producers (Q and K, V), the MMA issuer, the scheduler.
#pragma once

#include "fa_paged_split.cuh"

namespace fa {

constexpr float kStepRescaleSlack = 8.0f;

template <int D, int NQ>
struct StepLayout {
  static constexpr int kSoftmax = 128;
  static constexpr int kThreads = kSoftmax + 128;
  static constexpr uint32_t kTileBytes = kKeyTile * D * 2;
  static constexpr uint32_t kChunkBytes = kKeyTile * 128;  // 128 rows x 64 values
  static constexpr uint32_t kStageBytes = 2 * kTileBytes;  // V tile, then K tile
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr uint32_t kQChunk = NQ * 128;  // NQ rows x 64 values
  static constexpr uint32_t kQBytes = kQChunk * (D / 64);
  static constexpr uint32_t kPBytes = NQ * 256;  // NQ rows x 128 keys
  static constexpr uint32_t kQ = kStages * kStageBytes;   // 2 buffers
  static constexpr uint32_t kP = kQ + 2 * kQBytes;        // 2 buffers
  static constexpr uint32_t kRed = kP + 2 * kPBytes;      // [column][warp] maxima
  static constexpr uint32_t kSums = kRed + 4 * NQ * 4;    // [2][column][warp]
  static constexpr uint32_t kRef = kSums + 8 * NQ * 4;    // [column] reference
  static constexpr uint32_t kTok = kRef + NQ * 4;         // [column] token of a column
  static constexpr uint32_t kItems = kTok + NQ;
  static constexpr uint32_t kBar = kItems + kItemSlots * sizeof(Item);
  static constexpr int kNumBars = 2 * kStages + 10 + 2 * kItemSlots;
  static constexpr uint32_t kTmemSlot = kBar + kNumBars * 8;
  static constexpr uint32_t kAbort = kTmemSlot + 8;
  static constexpr uint32_t kBytes = kAbort + 8 + 1024;
  // TMEM: S^T buffers at 0 and NQ, O^T at 2 NQ
  static constexpr uint32_t tO = 2 * NQ;
  static constexpr uint32_t kTmemCols = NQ == 16 ? 64 : 128;
  // barriers
  static constexpr int bFull = 0, bEmpty = kStages, bQFull = 2 * kStages, bQEmpty = bQFull + 2,
                       bSFull = bQEmpty + 2, bPFull = bSFull + 2,
                       bDone = bPFull + 2,  // the product of a P buffer has landed
                       bItems = bDone + 2;
};

// Byte of (row, key) in an NQ-row, 128-byte-swizzled tile of 128 16-bit columns.
template <int NQ>
__device__ __forceinline__ uint32_t step_swz(int row, int col) {
  const int byte = (col & 63) * 2;
  return static_cast<uint32_t>((col >> 6) * NQ * 128 + row * 128 +
                               ((((byte >> 4) ^ (row & 7)) << 4) | (byte & 15)));
}

template <int C>
__device__ __forceinline__ void tmem_ld_cols(uint32_t addr, uint32_t* r) {
  if constexpr (C == 16) {
    tmem_ld16(addr, r);
    tmem_wait_ld();
    reg_fence16(r);
  } else {
    tmem_ld32(addr, r);
    tmem_wait_ld();
    reg_fence32(r);
  }
}

// The pages of tile `tile` that hold keys of [keys.lo, keys.hi]: up to 8, of which a box of
// `rows` rows and 64 columns each is loaded.
struct TilePages {
  int first, count;  // pages of the sequence
  int rows;          // of a page in this tile
  __device__ __forceinline__ TilePages(int tile, const KeyRange& keys, int shift) {
    const int k0 = max(tile * kKeyTile, keys.lo), k1 = min(tile * kKeyTile + kKeyTile - 1, keys.hi);
    first = k0 >> shift;
    count = (k1 >> shift) - first + 1;
    rows = min(1 << shift, kKeyTile);
  }
};
// Issued box by box by the converged warp: with a box per lane each took ~85 cycles (its
// operands go to uniform registers one lane at a time), a tile of 16-row pages 1400.
template <int D>
__device__ __forceinline__ void load_tile_pages(const TilePages& t, int tile, int shift,
                                                PageWindow& win, const CUtensorMap* map,
                                                uint32_t dst, uint32_t bar, int head, int lane) {
  win.advance(t.first, lane);
#pragma unroll 1
  for (int i = 0; i < t.count; ++i) {
    const int page = win.get(t.first + i);
    const int key = max((t.first + i) << shift, tile * kKeyTile);  // first key of the box
    const uint32_t at = dst + static_cast<uint32_t>(key - tile * kKeyTile) * 128u;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      warp_tma_load_4d(at + c * kKeyTile * 128, map, c * 64, key & ((1 << shift) - 1), head, page,
                       bar);
  }
}

template <int D, int NQ, bool BF16>
__global__ void __launch_bounds__(StepLayout<D, NQ>::kThreads, 1)
    fa_paged_step_kernel(const __grid_constant__ CUtensorMap tmQ,
                         const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const PagedView c,
                         uint16_t* __restrict__ O, Strides so, float* __restrict__ L,
                         float* __restrict__ Opart, float* __restrict__ Lpart,
                         PartInfo* __restrict__ parts, int group, int max_q, int wl, int wr,
                         int least, float scale_log2) {
  using Lay = StepLayout<D, NQ>;
  constexpr int S = Lay::kStages;
  constexpr int C = NQ;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t pad = ((raw_base + 1023u) & ~1023u) - raw_base;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw_base + pad;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // uniform
  const int lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return sbase + Lay::kBar + 8u * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::kAbort);
  uint8_t* tok = smem + Lay::kTok;
  constexpr int kProducer = Lay::kSoftmax / 32, kMma = kProducer + 2,
                kScheduler = kMma + 1;

  dependents_may_launch();
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(bar(Lay::bFull + s), 2);  // K and V
      mbar_init(bar(Lay::bEmpty + s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(Lay::bQFull + b), 1);
      mbar_init(bar(Lay::bQEmpty + b), 1);
      mbar_init(bar(Lay::bSFull + b), 1);
      mbar_init(bar(Lay::bPFull + b), Lay::kSoftmax);
      mbar_init(bar(Lay::bDone + b), 1);
    }
    item_ring_init(bar(Lay::bItems), kProducer + 3);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kScheduler) {
    dependency_wait();
    Scheduler<true> schedule(c, max_q, max_q, wl, wr);
    schedule.locate(least);
    __syncthreads();
    ItemRing ring(sbase + Lay::kItems, bar(Lay::bItems));
    schedule.run(ring, abort_flag, parts);
    __syncthreads();
    return;
  }
  if (warp == kMma) {
    tmem_alloc(sbase + Lay::kTmemSlot, Lay::kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x < NQ) tok[threadIdx.x] = static_cast<uint8_t>(threadIdx.x / group);
  dependency_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + Lay::kTmemSlot);
  ItemRing ring(sbase + Lay::kItems, bar(Lay::bItems));
  Item w;
  bool ok = true;

  if (warp == kProducer || warp == kProducer + 1) {
    // --------------------------------------- TMA producers: Q and K, V
    const bool is_k = warp == kProducer;
    const CUtensorMap* map = is_k ? &tmK : &tmV;
    if (lane == 0) {
      tma_prefetch(map);
      if (is_k) tma_prefetch(&tmQ);
    }
    __syncwarp();
    const uint32_t q_bytes = static_cast<uint32_t>(group) * max_q * D * 2;
    const uint32_t at = sbase + (is_k ? Lay::kTileBytes : 0);
    int it = 0, item = 0;
    PageWindow win;
    win.bad = false;
    while (ok && __all_sync(0xffffffffu, ring.get(&w, &ok, abort_flag))) {
      ring.read(lane == 0);
      if (w.j0 >= w.j1) continue;
      win.start(c, w.b, (w.keys.first + w.j0) * kKeyTile >> c.page_shift, lane);
      if (is_k) {
        const int qb = item & 1;
        ok = item < 2 || mbar_wait(bar(Lay::bQEmpty + qb),
                                   static_cast<uint32_t>(item / 2 - 1) & 1, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (lane == 0) {
          mbar_expect_tx(bar(Lay::bQFull + qb), q_bytes);
          for (int i = 0; i < D / 64; ++i)
            tma_load_4d(sbase + Lay::kQ + qb * Lay::kQBytes + i * Lay::kQChunk, &tmQ, i * 64, 0,
                        w.begin, w.h, bar(Lay::bQFull + qb));
        }
        __syncwarp();
        ++item;
      }
      for (int j = w.j0; j < w.j1; ++j, ++it) {
        const int st = it % S;
        const int tile = w.keys.first + j;
        const TilePages pages(tile, w.keys, c.page_shift);
        ok = it < S || mbar_wait(bar(Lay::bEmpty + st), static_cast<uint32_t>(it / S - 1) & 1,
                                 abort_flag);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        if (lane == 0)
          mbar_expect_tx(bar(Lay::bFull + st),
                         static_cast<uint32_t>(pages.count * pages.rows) * D * 2);
        __syncwarp();
        load_tile_pages<D>(pages, tile, c.page_shift, win, map, at + st * Lay::kStageBytes,
                           bar(Lay::bFull + st), w.h, lane);
      }
    }
    if (win.bad) atomicExch(&g_fa_status, kStatusInvalid);
  } else if (warp == kMma) {
    // -------------------------------------------------------------- MMA issuer
    {
      constexpr uint32_t id_s = idesc_f16_f32(kKeyTile, NQ, BF16, false, false);
      constexpr uint32_t id_o = idesc_f16_f32(128, NQ, BF16, true, false);
      // O^T += V^T P^T of tile t of the CTA's tiles (accumulate: not an item's first)
      auto product = [&](int t, bool accumulate) -> bool {
        const int st = t % S, pb = t & 1;
        if (!warp_wait(bar(Lay::bPFull + pb), static_cast<uint32_t>(t >> 1) & 1, abort_flag))
          return false;
        tc_fence_after();
        const SmemDesc dv = smem_desc(sbase + st * Lay::kStageBytes, Lay::kChunkBytes, 1024);
        const SmemDesc dp = smem_desc(sbase + Lay::kP + pb * Lay::kPBytes, 16, 1024);
#pragma unroll
        for (int k = 0; k < kKeyTile / 16; ++k)
          warp_mma_ss(tmem + Lay::tO, dv, k * 2048, dp, (k >> 2) * Lay::kQChunk + (k & 3) * 32,
                      id_o, (accumulate || k > 0) ? 1u : 0u);
        warp_mma_commit(bar(Lay::bEmpty + st));
        warp_mma_commit(bar(Lay::bDone + pb));
        return true;
      };
      int it = 0, item = 0;
      bool owed = false, last_accumulates = false;  // the product of tile it - 1
      while (ok && __all_sync(0xffffffffu, ring.get(&w, &ok, abort_flag))) {
        ring.read(lane == 0);
        const int j0 = __shfl_sync(0xffffffffu, w.j0, 0), j1 = __shfl_sync(0xffffffffu, w.j1, 0);
        if (j0 >= j1) {
          // an item without tiles: the softmax warps wait for the item before's last product
          // before they read on
          if (owed) ok = product(it - 1, last_accumulates);
          owed = false;
          continue;
        }
        const int qb = item & 1;
        ok = warp_wait(bar(Lay::bQFull + qb), static_cast<uint32_t>(item >> 1) & 1, abort_flag);
        const SmemDesc dq = smem_desc(sbase + Lay::kQ + qb * Lay::kQBytes, 16, 1024);
        for (int j = j0; ok && j < j1; ++j, ++it) {
          const int st = it % S;
          ok = warp_wait(bar(Lay::bFull + st), static_cast<uint32_t>(it / S) & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const SmemDesc dk =
              smem_desc(sbase + st * Lay::kStageBytes + Lay::kTileBytes, 16, 1024);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            warp_mma_ss(tmem + (it & 1) * NQ, dk, (k >> 2) * Lay::kChunkBytes + (k & 3) * 32, dq,
                        (k >> 2) * Lay::kQChunk + (k & 3) * 32, id_s, k > 0 ? 1u : 0u);
          warp_mma_commit(bar(Lay::bSFull + (it & 1)));
          if (j == j1 - 1) warp_mma_commit(bar(Lay::bQEmpty + qb));
          if (owed) ok = product(it - 1, last_accumulates);
          owed = true;
          last_accumulates = j > j0;
        }
        ++item;
      }
      if (ok && owed) product(it - 1, last_accumulates);
    }
  } else {
    // ----------------------------------------------------------------- softmax
    const int r = threadIdx.x;  // key of the tile = TMEM lane
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    float* red = reinterpret_cast<float*>(smem + Lay::kRed);
    float* sums = reinterpret_cast<float*>(smem + Lay::kSums);
    float* refs = reinterpret_cast<float*>(smem + Lay::kRef);
    constexpr int gbar = 1;  // the softmax warps' named barrier
    // a column that has seen no key: below every finite score, and -inf - kNone = -inf
    constexpr float kNone = -3.402823466e38f;
    int it = 0;
    while (true) {
      const bool more = ring.get(&w, &ok, abort_flag);
      __syncwarp();
      // all leave together; and the last item's sums have been read
      if (!named_bar_and(gbar, 128, more)) break;
      ring.read(lane == 0);
      const int cols = w.n * group;
      const int off = w.nk - w.n;
      // keys that every row sees
      const int all_lo = w.n - 1 + off - wl, all_hi = min(w.nk - 1, off + wr);
      float m[C], l[C], l_o[C];
#pragma unroll
      for (int q = 0; q < C; ++q) {
        m[q] = kNone;
        l[q] = 0.f;  // this thread's (key's) share of the sums
        l_o[q] = 0.f;
      }
      for (int j = w.j0; j < w.j1; ++j, ++it) {
        const int b = it & 1;
        const int key0 = (w.keys.first + j) * kKeyTile;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(Lay::bSFull + b),
                                               static_cast<uint32_t>(it >> 1) & 1, abort_flag));
        float s[C];
        bool raise = !ok;
        if (ok) {
          tc_fence_after();
          uint32_t sr[C];
          tmem_ld_cols<C>(lane_base + b * NQ, sr);
#pragma unroll
          for (int q = 0; q < C; ++q) s[q] = __uint_as_float(sr[q]);
          if (key0 < all_lo || key0 + kKeyTile - 1 > all_hi) {  // an edge of the mask
            const int key = key0 + r;
#pragma unroll
            for (int q = 0; q < C; ++q) {
              if ((q & 3) == 0 && q >= cols) break;
              const int mid = tok[q] + off;
              if (key > min(w.nk - 1, mid + wr) || key < mid - wl) s[q] = -INFINITY;
            }
            if (key < w.keys.lo || key > w.keys.hi) {
              const uint32_t v = sbase + (it % S) * Lay::kStageBytes + r * 128;
              // the stage has landed: its K has been multiplied
#pragma unroll
              for (int i = 0; i < D / 8; ++i)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                 v + (i >> 3) * Lay::kChunkBytes + (i & 7) * 16),
                             "r"(0)
                             : "memory");
            }
          }
#pragma unroll
          for (int q = 0; q < C; ++q) {
            if ((q & 3) == 0 && q >= cols) break;
            raise = raise || fmaf(s[q], scale_log2, -m[q]) > kStepRescaleSlack;
          }
        }
        if (named_bar_or(gbar, 128, raise)) {
          ok = named_bar_and(gbar, 128, ok);
          if (!ok) break;
          {
            float v[C];
#pragma unroll
            for (int q = 0; q < C; ++q) v[q] = s[q];
            const float top = reduce_columns<C>(v, lane, MaxOf());
            if (lane < C) red[lane * 4 + warp] = top * scale_log2;
          }
          named_bar_sync(gbar, 128);
          // O^T holds products: it is rescaled, once the last of them has landed
          const bool rescale = j > w.j0;
          if (rescale) {
            ok = __all_sync(0xffffffffu,
                            mbar_wait(bar(Lay::bDone + (b ^ 1)),
                                      static_cast<uint32_t>((it - 1) >> 1) & 1, abort_flag));
            tc_fence_after();
          }
#pragma unroll
          for (int q4 = 0; q4 < C; q4 += 4) {
            if (q4 >= cols) break;
            float alpha[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int q = q4 + k;
              const float4 t = *reinterpret_cast<const float4*>(red + q * 4);
              const float top = fmaxf(fmaxf(t.x, t.y), fmaxf(t.z, t.w));
              const float m_new = top > m[q] + kStepRescaleSlack ? top : m[q];
              alpha[k] = ex2_approx(m[q] - m_new);  // 0 at first
              m[q] = m_new;
              l[q] *= alpha[k];
              l_o[q] *= alpha[k];
            }
            if (rescale && ok) {
              uint32_t o[4];
              tmem_ld4(lane_base + Lay::tO + q4, o);
              tmem_st4(lane_base + Lay::tO + q4,
                       __float_as_uint(__uint_as_float(o[0]) * alpha[0]),
                       __float_as_uint(__uint_as_float(o[1]) * alpha[1]),
                       __float_as_uint(__uint_as_float(o[2]) * alpha[2]),
                       __float_as_uint(__uint_as_float(o[3]) * alpha[3]));
            }
          }
          if (rescale) tmem_wait_st();
        }
        // P_j^T into buffer b, once the product before last has read it
        if (ok && it >= 2)
          ok = __all_sync(0xffffffffu,
                          mbar_wait(bar(Lay::bDone + b),
                                    static_cast<uint32_t>((it - 2) >> 1) & 1, abort_flag));
        uint8_t* pt = smem + Lay::kP + b * Lay::kPBytes;
#pragma unroll
        for (int q = 0; q < C; ++q) {
          if ((q & 3) == 0 && q >= cols) break;  // those rows of P are never read as a result
          const float p = ex2_approx(fmaf(s[q], scale_log2, -m[q]));
          const uint32_t pk = pack2<BF16>(p, 0.f);
          float pr, unused;
          unpack2<BF16>(pk, pr, unused);
          l[q] += p;
          l_o[q] += pr;
          *reinterpret_cast<uint16_t*>(pt + step_swz<NQ>(q, r)) =
              static_cast<uint16_t>(pk & 0xFFFFu);
        }
        fence_async_smem();
        tc_fence_before();
        mbar_arrive(bar(Lay::bPFull + b));
        // a wait that gave up in one warp reaches the others at the next vote
      }
      // sums over the tile's 128 keys, while the item's last product runs
      {
        const float a = reduce_columns<C>(l, lane, SumOf());
        const float e = reduce_columns<C>(l_o, lane, SumOf());
        if (lane < C) {
          sums[lane * 8 + warp] = a;
          sums[lane * 8 + 4 + warp] = e;
        }
        if (r == 0) {
#pragma unroll
          for (int q = 0; q < C; ++q) refs[q] = m[q];
        }
      }
      const bool some = w.j1 > w.j0;
      ok = __all_sync(0xffffffffu,
                      ok && (!some || mbar_wait(bar(Lay::bDone + ((it - 1) & 1)),
                                                static_cast<uint32_t>((it - 1) >> 1) & 1,
                                                abort_flag)));
      ok = named_bar_and(gbar, 128, ok);
      if (!ok) break;
      tc_fence_after();
      const bool whole = w.j0 == 0 && w.j1 == w.keys.count;
      const long slot = w.j0 > 0 ? 2L * blockIdx.x : 2L * blockIdx.x + 1;
      // thread r: row r of the d columns (lane r of O^T) of every query column ...
#pragma unroll 1
      for (int q4 = 0; q4 < cols; q4 += 4) {
        uint32_t o[4];
        tmem_ld4(lane_base + Lay::tO + q4, o);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int q = q4 + k;
          if (q >= cols || (D < 128 && r >= D)) break;
          const float4 t = *reinterpret_cast<const float4*>(sums + q * 8 + 4);
          const float e = (t.x + t.y) + (t.z + t.w);
          // no key seen: O = 0 (and O^T may not have been written at all)
          const float val = e == 0.f ? 0.f : __fdividef(__uint_as_float(o[k]), e);
          if (whole) {
            const int tq = tok[q];
            const int head = w.h * group + q - tq * group;
            O[(w.begin + tq) * so.sn + head * so.sh + r] =
                static_cast<uint16_t>(pack2<BF16>(val, 0.f) & 0xFFFFu);
          } else {
            Opart[(slot * NQ + q) * D + r] = val;
          }
        }
      }
      // ... and L of query column r
      if (r < cols) {
        const float4 t = *reinterpret_cast<const float4*>(sums + r * 8);
        const float a = (t.x + t.y) + (t.z + t.w);
        const float L2 = a == 0.f ? -INFINITY : refs[r] + log2f(a);
        if (whole) {
          const int tq = tok[r];
          const int head = w.h * group + r - tq * group;
          L[static_cast<long>(head) * c.tokens + w.begin + tq] =
              L2 * 0.69314718055994530942f;
        } else {
          Lpart[slot * NQ + r] = L2;
        }
      }
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, Lay::kTmemCols);
  }
}

}  // namespace fa
