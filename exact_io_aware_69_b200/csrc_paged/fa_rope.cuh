// fa_rope.cuh -- rotary positions, and the append of new tokens to a paged cache with the
// rotation applied on the way: one kernel, since both move rows of heads once and turn
// some of them.
//
// Pair i of a row at position pos is turned by a = pos * freqs[i]. The product and its
// reduction by whole turns are 64-bit (at pos = 10^6 a 32-bit product is off by 0.06 rad);
// sine and cosine of the reduced angle, the rotation and the magnitude are 32-bit, and the
// result is rounded once to 16 bits.
//
// The pass is bound by HBM: every element is read and written once. So a block takes a few
// tokens and computes their rot_dim / 2 sines and cosines once into shared memory (a token's
// angles serve all its heads; per thread and head they would cost more instructions than
// the rotation); its threads then stream rows: a thread owns two 16-byte vectors of a row,
// half the rotated (or half the copied) columns apart, so that in the half form it holds
// both columns of its pairs, neighbouring threads hold neighbouring vectors in both forms,
// and every store covers whole sectors; it keeps its angles in registers over the heads of
// its token. Threads of a warp run over the heads of a token or over tokens, whichever lie
// closer together in memory.
//
// Small blocks and two rows in flight per thread carry the most bandwidth: 2 x 8192 tokens of
// 32 + 8 heads, d 128, bf16 (336 MB) take 55.4 us (6.06 TB/s, 0.93 of the copy rate); 256
// threads with 2 / 4 / 5 rows 56.2 / 57.6 / 65.2, loading the first rows before the angles are
// there 57.7 to 65.
#pragma once

#include "fa_paged_common.cuh"

namespace fa {

constexpr int kRopeThreads = 128;
constexpr int kRopeRows = 2;          // rows in flight per thread
constexpr int kRopeMaxTokens = 4;     // tokens of a block
constexpr int kRopeMaxDim = 1024;

struct RopeRows {
  const uint16_t* src;
  uint16_t* dst;
  Strides ss, sd;
  int heads;
};

struct RopeArgs {
  RopeRows kinds[3];  // Q and K, which are rotated, and (append only) V, which is copied
  const int* positions;
  long pos_row;
  const double* freqs;
  int rot, d;
  float magnitude, sign;  // sign: -1 turns back
  int N;                  // rows per batch (rope), packed rows (append: one batch)
  long rows;              // B * N
  int tokens_per_block;
  bool tokens_first;      // neighbouring threads take neighbouring tokens, not heads
  PagedView cache;        // append only; its pages are the destination of k and v
};

__device__ __forceinline__ void sincos_of(int pos, double freq, float* s, float* c) {
  const double turns2 = static_cast<double>(pos) * freq * 0.31830988618379067154;  // angle / pi
  const double r = turns2 - 2.0 * rint(0.5 * turns2);                             // in [-1, 1]
  sincospif(static_cast<float>(r), s, c);
}

template <bool BF16>
__device__ __forceinline__ void rotate16(uint4& a, uint4& b, const float* cs, const float* sn,
                                         bool interleaved) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (interleaved) {  // pair i in word i
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x0, x1;
      unpack2<BF16>(w[i], x0, x1);
      w[i] = pack2<BF16>(x0 * cs[i] - x1 * sn[i], x1 * cs[i] + x0 * sn[i]);
    }
  } else {  // pair i: value i of the first vector with value i of the second
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x0, x1, y0, y1;
      unpack2<BF16>(w[i], x0, y0);
      unpack2<BF16>(w[4 + i], x1, y1);
      const int p = 2 * i;
      w[i] = pack2<BF16>(x0 * cs[p] - x1 * sn[p], y0 * cs[p + 1] - y1 * sn[p + 1]);
      w[4 + i] = pack2<BF16>(x1 * cs[p] + x0 * sn[p], y1 * cs[p + 1] + y0 * sn[p + 1]);
    }
  }
  a = make_uint4(w[0], w[1], w[2], w[3]);
  b = make_uint4(w[4], w[5], w[6], w[7]);
}

template <bool PAGED, bool BF16>
__global__ void __launch_bounds__(kRopeThreads) fa_rope_kernel(const RopeArgs a,
                                                               const bool interleaved) {
  extern __shared__ __align__(16) float rope_smem[];  // [tokens][rot / 2] cos, then sin
  __shared__ int s_pos[kRopeMaxTokens];
  __shared__ int s_owner[kRopeMaxTokens];  // append: -1 = the token belongs to nobody
  __shared__ int s_page[kRopeMaxTokens];   // append: destination page (-1: not written)
  __shared__ int s_row[kRopeMaxTokens];

  dependents_may_launch();
  dependency_wait();
  const int tpb = a.tokens_per_block;
  const long t0 = static_cast<long>(blockIdx.x) * tpb;
  const int nt = static_cast<int>(min(static_cast<long>(tpb), a.rows - t0));
  const int half = a.rot / 2;

  // thread = (token, row lane, pair of vectors), vectors fastest
  const int groups = a.d / 16;
  const int rlanes = kRopeThreads / groups / tpb;  // threads' rows of one token per pass
  const int g = threadIdx.x % groups;
  const int rest = threadIdx.x / groups;
  const int ti = a.tokens_first ? rest % tpb : rest / rlanes;
  const int rl = a.tokens_first ? rest / tpb : rest - ti * rlanes;
  const bool active = ti < nt && rl < rlanes;
  const long t = t0 + ti;
  const long b = PAGED ? 0 : t / a.N;
  const long n = PAGED ? t : t - b * a.N;
  const bool turns = g < a.rot / 16;
  // the columns of the thread's two vectors
  const int c0 = turns ? 8 * g : a.rot + 8 * (g - a.rot / 16);
  const int c1 = c0 + (turns ? half : (a.d - a.rot) / 2);
  if constexpr (PAGED) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = warp; i < nt; i += kRopeThreads / 32) {
      const PagedView& c = a.cache;
      const int tok = static_cast<int>(t0) + i;
      const int seq = owner_of(c.cu_q, c.batch, tok, lane);
      if (lane == 0) {
        int owner = -1, page = -1, row = 0, pos = 0;
        if (seq >= 0 && tok < c.cu_q[c.batch]) {
          const SeqInfo s = seq_info(c, seq, c.tokens);
          pos = s.nk - s.n + (tok - s.begin);
          if (s.ok && s.n <= s.nk && tok < s.begin + s.n) {
            owner = seq;
            page = c.table[static_cast<long>(seq) * c.table_row + (pos >> c.page_shift)];
            row = pos & ((1 << c.page_shift) - 1);
            if (static_cast<unsigned>(page) >= static_cast<unsigned>(c.num_pages)) page = -1;
          }
          if (owner < 0 || page < 0) atomicExch(&g_fa_status, kStatusInvalid);
        }
        s_owner[i] = owner;
        s_page[i] = page;
        s_row[i] = row;
        s_pos[i] = a.positions != nullptr && owner >= 0 ? a.positions[tok] : pos;
      }
    }
  } else {
    if (threadIdx.x < nt) {
      const long tok = t0 + threadIdx.x;
      const long bb = tok / a.N;
      const int nn = static_cast<int>(tok - bb * a.N);
      s_pos[threadIdx.x] = a.positions != nullptr ? a.positions[bb * a.pos_row + nn] : nn;
    }
  }
  __syncthreads();
  float* cosines = rope_smem;
  float* sines = rope_smem + tpb * half;
  for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
    float s, c;
    sincos_of(s_pos[i / half], a.freqs[i % half], &s, &c);
    cosines[i] = c * a.magnitude;
    sines[i] = s * a.magnitude * a.sign;
  }
  __syncthreads();
  if (active && (!PAGED || s_owner[ti] >= 0)) {
    float cs[8], sn[8];
    if (turns) {
      // pairs of the first vector and of the second: the same eight, or four and four
      const float* c = cosines + ti * half + (interleaved ? 4 * g : 8 * g);
      const float* s = sines + ti * half + (interleaved ? 4 * g : 8 * g);
      const int second = interleaved ? half / 2 : 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cs[i] = c[i];
        sn[i] = s[i];
        cs[4 + i] = c[second + i];
        sn[4 + i] = s[second + i];
      }
    }
#pragma unroll 1
    for (int kind = 0; kind < (PAGED ? 3 : 2); ++kind) {
      const RopeRows& rows = a.kinds[kind];
      // append: K and V rows go to row s_row of page s_page (sb: the page stride), if it is one
      const bool paged = PAGED && kind > 0;
      if (paged && s_page[ti] < 0) break;
      const uint16_t* src = rows.src + b * rows.ss.sb + n * rows.ss.sn;
      uint16_t* dst = rows.dst + (paged ? s_page[ti] : b) * rows.sd.sb +
                      (paged ? s_row[ti] : n) * rows.sd.sn;
      const bool rotate = turns && kind < 2;
#pragma unroll 1
      for (int h0 = rl; h0 < rows.heads; h0 += kRopeRows * rlanes) {
        uint4 x[kRopeRows], y[kRopeRows];
#pragma unroll
        for (int u = 0; u < kRopeRows; ++u) {
          const int h = h0 + u * rlanes;
          if (h < rows.heads) {
            const uint16_t* at = src + h * rows.ss.sh;
            x[u] = *reinterpret_cast<const uint4*>(at + c0);
            y[u] = *reinterpret_cast<const uint4*>(at + c1);
          }
        }
#pragma unroll
        for (int u = 0; u < kRopeRows; ++u) {
          const int h = h0 + u * rlanes;
          if (h < rows.heads) {
            if (rotate) rotate16<BF16>(x[u], y[u], cs, sn, interleaved);
            uint16_t* at = dst + h * rows.sd.sh;
            *reinterpret_cast<uint4*>(at + c0) = x[u];
            *reinterpret_cast<uint4*>(at + c1) = y[u];
          }
        }
      }
    }
  }
  // lengths that no row led to
  if (PAGED && blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.cache.batch; i += kRopeThreads) {
      const SeqInfo s = seq_info(a.cache, i, a.cache.tokens);
      if (!s.ok || (s.n > 0 && s.n > s.nk)) atomicExch(&g_fa_status, kStatusInvalid);
    }
}

}  // namespace fa
