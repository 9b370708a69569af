// fa_paged_simple.cuh -- exact attention over a paged cache, one CTA per (token, query
// head) on CUDA cores: the plain online softmax with the keys dealt to four warps.
#pragma once

#include "fa_paged_common.cuh"

namespace fa {

constexpr int kSimpleThreads = 128;

struct PagedKv {
  const uint16_t* k;
  const uint16_t* v;
  Strides sk, sv;  // sb: page, sh: head, sn: row
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kSimpleThreads)
    fa_paged_simple_kernel(const PagedView c, const PagedKv kv, const uint16_t* Q, Strides sq,
                           uint16_t* O, Strides so, float* L, int Hq, int max_q, int wl, int wr,
                           float scale_log2) {
  constexpr int CPL = D / 32;
  __shared__ float q[D];
  __shared__ float ms[4], ls[4], os[4][D];
  const int t = blockIdx.x, h = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = owner_of(c.cu_q, c.batch, t, lane);
  if (b < 0 || t >= c.cu_q[c.batch]) return;
  const SeqInfo s = seq_info(c, b, max_q);
  if (!s.ok || t >= s.begin + s.n) {
    if (threadIdx.x == 0) atomicExch(&g_fa_status, kStatusInvalid);
    return;
  }
  const int hk = h / (Hq / c.heads);
  for (int i = threadIdx.x; i < D / 2; i += kSimpleThreads) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(Q + t * sq.sn + h * sq.sh + 2 * i);
    unpack2<BF16>(u, q[2 * i], q[2 * i + 1]);
  }
  __syncthreads();
  const int mid = t - s.begin + s.nk - s.n;
  const int lo = max(0, mid - wl), hi = min(s.nk - 1, mid + wr);
  float m = -INFINITY, l = 0.f, o[CPL];
  for (int i = 0; i < CPL; ++i) o[i] = 0.f;
  for (int j0 = lo + warp * 32; j0 <= hi; j0 += kSimpleThreads) {
    const int j = j0 + lane;
    float x = -INFINITY;
    long voff = -1;
    if (j <= hi) {
      const int page = c.table[static_cast<long>(b) * c.table_row + (j >> c.page_shift)];
      const int row = j & ((1 << c.page_shift) - 1);
      if (static_cast<unsigned>(page) < static_cast<unsigned>(c.num_pages)) {
        const uint16_t* kr = kv.k + page * kv.sk.sb + hk * kv.sk.sh + row * kv.sk.sn;
        voff = page * kv.sv.sb + hk * kv.sv.sh + row * kv.sv.sn;
        x = 0.f;
        for (int i = 0; i < D; i += 2) {
          float a, e;
          unpack2<BF16>(*reinterpret_cast<const uint32_t*>(kr + i), a, e);
          x = fmaf(q[i], a, fmaf(q[i + 1], e, x));
        }
      } else {
        atomicExch(&g_fa_status, kStatusInvalid);
        x = 0.f;
      }
      x *= scale_log2;
    }
    float mx = x;
    for (int k = 16; k >= 1; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
    const float mn = fmaxf(m, mx);
    const float alpha = exp2f(m - mn);
    const float p = exp2f(x - mn);
    l = l * alpha + p;
    m = mn;
    for (int i = 0; i < CPL; ++i) o[i] *= alpha;
    for (int k = 0; k < 32; ++k) {
      const float pk = __shfl_sync(0xffffffffu, p, k);
      const long vo = __shfl_sync(0xffffffffu, voff, k);
      if (vo >= 0)
        for (int i = 0; i < CPL; i += 2) {
          float a, e;
          unpack2<BF16>(*reinterpret_cast<const uint32_t*>(kv.v + vo + lane * CPL + i), a, e);
          o[i] = fmaf(pk, a, o[i]);
          o[i + 1] = fmaf(pk, e, o[i + 1]);
        }
    }
  }
  for (int k = 16; k >= 1; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
  if (lane == 0) ms[warp] = m, ls[warp] = l;
  for (int i = 0; i < CPL; ++i) os[warp][lane * CPL + i] = o[i];
  __syncthreads();
  if (warp == 0) {
    const float M = fmaxf(fmaxf(ms[0], ms[1]), fmaxf(ms[2], ms[3]));
    float tot = 0.f, r[CPL];
    for (int i = 0; i < CPL; ++i) r[i] = 0.f;
    for (int w = 0; w < 4; ++w) {
      const float f = ms[w] == -INFINITY ? 0.f : exp2f(ms[w] - M);
      tot += f * ls[w];
      for (int i = 0; i < CPL; ++i) r[i] += f * os[w][lane * CPL + i];
    }
    const float inv = tot > 0.f ? 1.f / tot : 0.f;
    uint16_t* dst = O + t * so.sn + h * so.sh + lane * CPL;
    for (int i = 0; i < CPL; i += 2)
      *reinterpret_cast<uint32_t*>(dst + i) = pack2<BF16>(r[i] * inv, r[i + 1] * inv);
    if (lane == 0)
      L[static_cast<long>(h) * c.tokens + t] =
          tot > 0.f ? (M + log2f(tot)) * 0.69314718055994530942f : -INFINITY;
  }
}

}  // namespace fa
