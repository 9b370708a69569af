// fa_paged_merge.cuh -- joins the parts of items that the split cut: with the parts'
// normalised outputs O_s and base-2 log-sum-exps L_s,
//   L = log2 sum_s 2^(L_s),   O = sum_s 2^(L_s - L) O_s,
// the recurrence of the online softmax applied to whole parts, in the order of the CTAs
// that computed them.
//
// A part's rows come in tiles of `tile_tokens` tokens, `tile_rows` rows apart; row q of
// token t of a tile is t * group + q.
//
// Block (c, y) serves rows of the item whose first part is CTA c's slot 2 c + 1; it ends at
// once when there is none. WPR warps share a row's parts: eight for a decode step, whose
// few rows may have up to a part per SM, one for chunks, whose many rows have few. Bound
// by the latency of its dependent reads, so the launch overlaps the attention kernel's
// (programmatic dependent launch) and a warp keeps several parts' loads in flight.
#pragma once

#include "fa_paged_split.cuh"

namespace fa {

constexpr int kMergeThreads = 256;
static_assert(kMergeThreads >= kSplitGrid, "one thread per CTA of the split");

template <int D, int WPR, bool BF16>
__global__ void __launch_bounds__(kMergeThreads)
    fa_paged_merge_kernel(const float* __restrict__ Opart, const float* __restrict__ Lpart,
                          const PartInfo* __restrict__ parts, int rows_per_slot, int tile_tokens,
                          int tile_rows, int group, uint16_t* __restrict__ O, Strides so, float* __restrict__ L,
                          int tokens) {
  constexpr int CPL = D / 32;
  constexpr int kRows = kMergeThreads / 32 / WPR;  // rows of a block
  __shared__ int last;                             // the CTA of the item's last part
  __shared__ float s_m[8], s_l[8], s_o[8][D];
  const int c = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) last = kSplitGrid - 1;
  dependents_may_launch();
  dependency_wait();
  const int i = c + 1 + static_cast<int>(threadIdx.x);
  const bool goes_on = i < kSplitGrid && parts[i].goes_on;  // loaded beside the next line's
  const PartInfo info = parts[c];
  if (!info.begins) return;
  __syncthreads();
  if (i < kSplitGrid && !goes_on) atomicMin(&last, i);
  __syncthreads();
  const int n = last - c + 1;  // parts: slot 2 c + 1, then slots 2 (c + 1), 2 (c + 2), ...
  const int r = blockIdx.y * kRows + warp / WPR;
  const bool live = r < info.tokens * group;
  const int w = warp % WPR;
  float M = -INFINITY, tot = 0.f, o[CPL];
#pragma unroll
  for (int i = 0; i < CPL; ++i) o[i] = 0.f;
  const int t = r / group;
  const int q = r - t * group;
  const int tile = t / tile_tokens;
  const int in_slot = tile * tile_rows + (t - tile * tile_tokens) * group + q;
  auto row_of = [&](int s) -> long {
    return (s == 0 ? 2L * c + 1 : 2L * (c + s)) * rows_per_slot + in_slot;
  };
  if (live) {
    for (int s = w + lane * WPR; s < n; s += 32 * WPR) M = fmaxf(M, Lpart[row_of(s)]);
    M = warp_max(M);
    if (M != -INFINITY) {
#pragma unroll 4
      for (int s = w; s < n; s += WPR) {
        const long row = row_of(s);
        const float f = ex2_approx(Lpart[row] - M);  // 0 for a part whose rows saw no key
        tot += f;
        if constexpr (CPL == 4) {
          const float4 v = *reinterpret_cast<const float4*>(Opart + row * D + lane * 4);
          o[0] = fmaf(f, v.x, o[0]);
          o[1] = fmaf(f, v.y, o[1]);
          o[2] = fmaf(f, v.z, o[2]);
          o[3] = fmaf(f, v.w, o[3]);
        } else {
          const float2 v = *reinterpret_cast<const float2*>(Opart + row * D + lane * 2);
          o[0] = fmaf(f, v.x, o[0]);
          o[1] = fmaf(f, v.y, o[1]);
        }
      }
    }
  }
  if constexpr (WPR > 1) {
    if (lane == 0) {
      s_m[warp] = M;
      s_l[warp] = tot;
    }
#pragma unroll
    for (int i = 0; i < CPL; ++i) s_o[warp][lane * CPL + i] = o[i];
    __syncthreads();
    if (w != 0) return;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < WPR; ++i) top = fmaxf(top, s_m[warp + i]);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < CPL; ++i) o[i] = 0.f;
    if (top != -INFINITY) {
#pragma unroll
      for (int i = 0; i < WPR; ++i) {
        const float f = ex2_approx(s_m[warp + i] - top);
        sum = fmaf(f, s_l[warp + i], sum);
#pragma unroll
        for (int k = 0; k < CPL; ++k) o[k] = fmaf(f, s_o[warp + i][lane * CPL + k], o[k]);
      }
    }
    M = top;
    tot = sum;
  }
  if (!live) return;
  const float inv = tot > 0.f ? 1.f / tot : 0.f;
  const int head = info.head * group + q;
  uint16_t* dst = O + (info.token0 + t) * so.sn + head * so.sh + lane * CPL;
  if constexpr (CPL == 4)
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(pack2<BF16>(o[0] * inv, o[1] * inv), pack2<BF16>(o[2] * inv, o[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack2<BF16>(o[0] * inv, o[1] * inv);
  if (lane == 0)
    L[static_cast<long>(head) * tokens + info.token0 + t] =
        tot > 0.f ? (M + log2f(tot)) * 0.69314718055994530942f : -INFINITY;
}

}  // namespace fa
