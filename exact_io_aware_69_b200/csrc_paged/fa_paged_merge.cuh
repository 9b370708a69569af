// fa_paged_merge.cuh -- joins the parts of items that the split cut: with the parts'
// normalised outputs O_s and base-2 log-sum-exps L_s,
//   L = log2 sum_s 2^(L_s),   O = sum_s 2^(L_s - L) O_s,
// the recurrence of the online softmax applied to whole parts, in the order of the CTAs
// that computed them (a block's warps first each take every eighth part, then join theirs).
//
// Bound by latency: a chain of a few dependent reads, whatever the batch. So the launch
// overlaps the attention kernel's, every block finds the rows to join by itself from the
// CTAs' part records, and the rows are dealt evenly to the blocks: one row to a block and
// its parts to the warps while there are few rows (a decode step may have a part per SM for
// each of a handful), else a row to a warp. (The parts are written while this kernel is on the
// device already: their pointers must not be __restrict__ to const, which would allow loads
// through the cache for data that stays constant.)
//
// A part's rows come in tiles of `tile_tokens` tokens, `tile_rows` rows apart; row q of
// token t of a tile is t * group + q.
#pragma once

#include "fa_paged_split.cuh"

namespace fa {

constexpr int kMergeThreads = 256;
constexpr int kMergeWarps = kMergeThreads / 32;
static_assert(kMergeThreads >= kSplitGrid, "one thread per CTA of the split");

template <int D, bool BF16>
__global__ void __launch_bounds__(kMergeThreads)
    fa_paged_merge_kernel(const float* Opart, const float* Lpart, const PartInfo* parts,
                          int rows_per_slot, int tile_tokens, int tile_rows, int group,
                          uint16_t* __restrict__ O, Strides so, float* __restrict__ L,
                          int tokens) {
  constexpr int CPL = D / 32;
  __shared__ int first_row[kSplitGrid];       // of the item that CTA c began, among all rows
  __shared__ int2 item_of[kSplitGrid];        // its token0 and key head
  __shared__ unsigned ends[kMergeWarps];      // bit c: CTA c does not go on with its first item
  __shared__ int warp_rows[kMergeWarps];
  __shared__ float s_m[kMergeWarps], s_l[kMergeWarps], s_o[kMergeWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int me = threadIdx.x;
  dependents_may_launch();
  dependency_wait();
  // rows of the items that CTA `me` began and others went on with
  const bool real = me < kSplitGrid;
  const int4 head = real ? *reinterpret_cast<const int4*>(parts + me) : make_int4(0, 0, 0, 0);
  const bool end = !real || parts[me].goes_on == 0;
  const int rows = head.x ? head.z * group : 0;
  int upto = rows;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += v;
  }
  const unsigned bits = __ballot_sync(0xffffffffu, end);
  if (lane == 31) {
    warp_rows[warp] = upto;
    ends[warp] = bits;
  }
  __syncthreads();
  int total = 0, before = 0;
#pragma unroll
  for (int i = 0; i < kMergeWarps; ++i) {
    before = i == warp ? total : before;
    total += warp_rows[i];
  }
  if (real) {
    first_row[me] = before + upto - rows;
    item_of[me] = make_int2(head.y, head.w);
  }
  __syncthreads();
  const int blocks = static_cast<int>(gridDim.x);
  const bool shared_row = total <= blocks;  // a row's parts over the block's warps
  const int wpr = shared_row ? kMergeWarps : 1;
  const int w = shared_row ? warp : 0;
  for (int row = shared_row ? blockIdx.x : blockIdx.x * kMergeWarps + warp; row < total;
       row += blocks * (shared_row ? 1 : kMergeWarps)) {
    // the last CTA whose item starts at or before the row (those after it that began
    // nothing start at the same row as the next)
    int c = 0;
#pragma unroll
    for (int step = 128; step >= 1; step >>= 1)
      if (c + step < kSplitGrid && first_row[c + step] <= row) c += step;
    const int2 item = item_of[c];
    // parts: slot 2 c + 1, then 2 (c + 1), 2 (c + 2), ... up to the first CTA that ends it
    int last = c + 1;
    for (int i = last >> 5; i < kMergeWarps; ++i) {
      const unsigned after = ends[i] & (i == last >> 5 ? 0xffffffffu << (last & 31) : 0xffffffffu);
      if (after) {
        last = 32 * i + __ffs(after) - 1;
        break;
      }
    }
    const int n = last - c + 1;
    const int r = row - first_row[c];
    const int t = r / group;
    const int q = r - t * group;
    const int tile = t / tile_tokens;
    const int in_slot = tile * tile_rows + (t - tile * tile_tokens) * group + q;
    auto row_of = [&](int s) -> long {
      return (s == 0 ? 2L * c + 1 : 2L * (c + s)) * rows_per_slot + in_slot;
    };
    float M = -INFINITY, tot = 0.f, o[CPL];
#pragma unroll
    for (int i = 0; i < CPL; ++i) o[i] = 0.f;
    for (int s = w + lane * wpr; s < n; s += 32 * wpr) M = fmaxf(M, Lpart[row_of(s)]);
    M = warp_max(M);
    const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll 4
    for (int s = w; s < n; s += wpr) {
      const long at = row_of(s);
      const float f = ex2_approx(Lpart[at] - ref);  // 0 for a part whose rows saw no key
      tot += f;
      if constexpr (CPL == 4) {
        const float4 v = *reinterpret_cast<const float4*>(Opart + at * D + lane * 4);
        o[0] = fmaf(f, v.x, o[0]);
        o[1] = fmaf(f, v.y, o[1]);
        o[2] = fmaf(f, v.z, o[2]);
        o[3] = fmaf(f, v.w, o[3]);
      } else {
        const float2 v = *reinterpret_cast<const float2*>(Opart + at * D + lane * 2);
        o[0] = fmaf(f, v.x, o[0]);
        o[1] = fmaf(f, v.y, o[1]);
      }
    }
    if (shared_row) {
      if (lane == 0) {
        s_m[warp] = M;
        s_l[warp] = tot;
      }
#pragma unroll
      for (int i = 0; i < CPL; ++i) s_o[warp][lane * CPL + i] = o[i];
      __syncthreads();
      if (warp == 0) {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kMergeWarps; ++i) top = fmaxf(top, s_m[i]);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < CPL; ++i) o[i] = 0.f;
        const float from = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int i = 0; i < kMergeWarps; ++i) {
          const float f = ex2_approx(s_m[i] - from);
          sum = fmaf(f, s_l[i], sum);
#pragma unroll
          for (int k = 0; k < CPL; ++k) o[k] = fmaf(f, s_o[i][lane * CPL + k], o[k]);
        }
        M = top;
        tot = sum;
      }
    }
    if (!shared_row || warp == 0) {
      const float inv = tot == 0.f ? 0.f : 1.f / tot;
      const int head_q = item.y * group + q;
      uint16_t* dst = O + (item.x + t) * so.sn + head_q * so.sh + lane * CPL;
      if constexpr (CPL == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<BF16>(o[0] * inv, o[1] * inv),
                                                    pack2<BF16>(o[2] * inv, o[3] * inv));
      else
        *reinterpret_cast<uint32_t*>(dst) = pack2<BF16>(o[0] * inv, o[1] * inv);
      if (lane == 0)
        L[static_cast<long>(head_q) * tokens + item.x + t] =
            tot == 0.f ? -INFINITY : (M + log2f(tot)) * 0.69314718055994530942f;
    }
    // (a shared row is its block's only one: s_m, s_l and s_o are written once)
  }
}

}  // namespace fa
