// fa_paged_api.cu -- the C ABI declared in include/fa_paged.h: argument checks and kernel
// launches. All device work is in the .cuh kernels beside it.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "fa_paged.h"
#include "fa_paged_common.cuh"
#include "fa_paged_simple.cuh"
#include "fa_rope.cuh"

namespace {

constexpr float kLog2e = 1.4426950408889634074f;

bool aligned(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}
bool ok_ptr(const void* p, uintptr_t bytes = 16) { return p != nullptr && aligned(p, bytes); }

// Rows are moved in 16-byte pieces, so every stride is a multiple of 8 elements.
bool ok_strides(const fa_strides* s) {
  return s != nullptr && s->b >= 0 && s->h >= 0 && s->n >= 0 && (s->b | s->h | s->n) % 8 == 0;
}
fa::Strides strides(const fa_strides& s) {
  return {static_cast<long>(s.b), static_cast<long>(s.h), static_cast<long>(s.n)};
}

int launch_status() { return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// ------------------------------------------------------------------ rotation
int check_rotation(int d, int rot_dim, float magnitude, const double* freqs) {
  if (!ok_ptr(freqs, 8) || !isfinite(magnitude)) return FA_ERR_INVALID;
  if (rot_dim < 16 || rot_dim > d) return FA_ERR_INVALID;
  return rot_dim % 16 == 0 ? FA_OK : FA_ERR_UNSUPPORTED;
}

// Tokens of a block: one while that gives every SM at most a block or two (a token's rows
// then finish soonest), up to eight for long inputs, whose rows keep a thread's angles in
// registers for longer.
int rope_tokens_per_block(long rows, int groups) {
  int t = 1;
  while (t < fa::kRopeMaxTokens && rows / (2 * t) >= 148 * 2 &&
         fa::kRopeThreads / groups / (2 * t) >= 1)
    t *= 2;
  return t;
}

template <bool PAGED>
int launch_rope(fa::RopeArgs& a, bool interleaved, int dtype, cudaStream_t stream) {
  a.tokens_per_block = rope_tokens_per_block(a.rows, a.d / 16);
  const long blocks = (a.rows + a.tokens_per_block - 1) / a.tokens_per_block;
  if (blocks >= (1L << 31)) return FA_ERR_UNSUPPORTED;
  const size_t smem = static_cast<size_t>(a.tokens_per_block) * a.rot * sizeof(float);
  if (dtype == FA_BF16)
    fa::fa_rope_kernel<PAGED, true>
        <<<static_cast<unsigned>(blocks), fa::kRopeThreads, smem, stream>>>(a, interleaved);
  else
    fa::fa_rope_kernel<PAGED, false>
        <<<static_cast<unsigned>(blocks), fa::kRopeThreads, smem, stream>>>(a, interleaved);
  return launch_status();
}

fa::RopeRows rope_rows(const void* x, const fa_strides& xs, void* y, const fa_strides& ys,
                       int heads) {
  return {static_cast<const uint16_t*>(x), static_cast<uint16_t*>(y), strides(xs), strides(ys),
          heads};
}

// --------------------------------------------------------------------- cache
int check_cache(const fa_paged_cache* c, bool attention) {
  if (c == nullptr) return FA_ERR_INVALID;
  if (c->batch < 0 || c->tokens < 0 || c->heads <= 0 || c->d <= 0 || c->num_pages < 0 ||
      c->table_width < 0 || c->table_row < 0)
    return FA_ERR_INVALID;
  if (c->dtype != FA_BF16 && c->dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
    return FA_ERR_UNSUPPORTED;
  if (attention ? c->d != 64 && c->d != 128 : c->d % 16 != 0 || c->d > fa::kRopeMaxDim)
    return FA_ERR_UNSUPPORTED;
  if (c->batch > 16384 || c->heads > 1024 || c->tokens > (1 << 28) ||
      static_cast<long long>(c->table_width) * c->page_size > (1 << 28))
    return FA_ERR_UNSUPPORTED;
  if (c->batch == 0 || c->tokens == 0) return FA_OK;
  if (!ok_ptr(c->cu_q, 4) || !ok_ptr(c->seq_k, 4)) return FA_ERR_INVALID;
  if (c->table_width > 0 && !ok_ptr(c->table, 4)) return FA_ERR_INVALID;
  if (c->num_pages > 0 && (!ok_ptr(c->k_pages) || !ok_ptr(c->v_pages))) return FA_ERR_INVALID;
  const fa_strides k{c->k_page, c->k_head, c->k_row}, v{c->v_page, c->v_head, c->v_row};
  if (!ok_strides(&k) || !ok_strides(&v)) return FA_ERR_INVALID;
  return FA_OK;
}

fa::PagedView view_of(const fa_paged_cache& c) {
  int shift = 0;
  while ((1 << shift) < c.page_size) ++shift;
  return {c.table,     c.cu_q, c.seq_k, c.table_row, c.table_width,
          c.num_pages, shift,  c.heads, c.batch,     c.tokens};
}

// An edge that bounds nothing becomes fa::kUnbounded.
int edge(int w) { return w < 0 || w >= fa::kUnbounded ? fa::kUnbounded : w; }

template <int D, bool BF16>
int launch_simple(const fa_paged_cache& c, const void* Q, const fa_strides& xq, void* O,
                  const fa_strides& xo, float* L, int Hq, int max_q, int wl, int wr, float scale,
                  cudaStream_t stream) {
  const fa::PagedKv kv{static_cast<const uint16_t*>(c.k_pages),
                       static_cast<const uint16_t*>(c.v_pages),
                       {static_cast<long>(c.k_page), static_cast<long>(c.k_head),
                        static_cast<long>(c.k_row)},
                       {static_cast<long>(c.v_page), static_cast<long>(c.v_head),
                        static_cast<long>(c.v_row)}};
  const dim3 grid(static_cast<unsigned>(c.tokens), static_cast<unsigned>(Hq));
  fa::fa_paged_simple_kernel<D, BF16><<<grid, fa::kSimpleThreads, 0, stream>>>(
      view_of(c), kv, static_cast<const uint16_t*>(Q), strides(xq), static_cast<uint16_t*>(O),
      strides(xo), L, Hq, max_q, edge(wl), edge(wr), scale * kLog2e);
  return launch_status();
}

}  // namespace

extern "C" {

int fa_rope(const void* Xq, const fa_strides* xq, void* Yq, const fa_strides* yq, int Hq,
            const void* Xk, const fa_strides* xk, void* Yk, const fa_strides* yk, int Hk,
            const int* positions, long long pos_row, const double* freqs, int rot_dim,
            float magnitude, int interleaved, int inverse, int B, int N, int d, int dtype,
            void* stream) {
  if (B < 0 || N < 0 || Hq < 0 || Hk < 0 || d <= 0 || pos_row < 0) return FA_ERR_INVALID;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
  if (d % 16 != 0 || d > fa::kRopeMaxDim) return FA_ERR_UNSUPPORTED;
  const int st = check_rotation(d, rot_dim, magnitude, freqs);
  if (st != FA_OK) return st;
  if (static_cast<long long>(B) * N == 0 || Hq + Hk == 0) return FA_OK;
  if (Hq > 0 && (!ok_ptr(Xq) || !ok_ptr(Yq) || !ok_strides(xq) || !ok_strides(yq)))
    return FA_ERR_INVALID;
  if (Hk > 0 && (!ok_ptr(Xk) || !ok_ptr(Yk) || !ok_strides(xk) || !ok_strides(yk)))
    return FA_ERR_INVALID;
  if (!aligned(positions, 4)) return FA_ERR_INVALID;
  const fa_strides none{0, 0, 0};
  fa::RopeArgs a{};
  a.q = rope_rows(Xq, Hq ? *xq : none, Yq, Hq ? *yq : none, Hq);
  a.k = rope_rows(Xk, Hk ? *xk : none, Yk, Hk ? *yk : none, Hk);
  a.positions = positions;
  a.pos_row = static_cast<long>(pos_row);
  a.freqs = freqs;
  a.rot = rot_dim;
  a.d = d;
  a.magnitude = magnitude;
  a.sign = inverse ? -1.f : 1.f;
  a.N = N;
  a.rows = static_cast<long>(B) * N;
  return launch_rope<false>(a, interleaved != 0, dtype, static_cast<cudaStream_t>(stream));
}

int fa_paged_append(const fa_paged_cache* cache, const void* K, const fa_strides* xk,
                    const void* V, const fa_strides* xv, const void* Xq, const fa_strides* xq,
                    void* Yq, const fa_strides* yq, int Hq, const int* positions,
                    const double* freqs, int rot_dim, float magnitude, int interleaved,
                    void* stream) {
  int st = check_cache(cache, false);
  if (st != FA_OK) return st;
  if (Hq < 0 || (Hq > 0 && freqs == nullptr)) return FA_ERR_INVALID;
  if (freqs != nullptr && (st = check_rotation(cache->d, rot_dim, magnitude, freqs)) != FA_OK)
    return st;
  if (cache->batch == 0 || cache->tokens == 0) return FA_OK;
  if (!ok_ptr(K) || !ok_ptr(V) || !ok_strides(xk) || !ok_strides(xv)) return FA_ERR_INVALID;
  if (Hq > 0 && (!ok_ptr(Xq) || !ok_ptr(Yq) || !ok_strides(xq) || !ok_strides(yq)))
    return FA_ERR_INVALID;
  if (!aligned(positions, 4)) return FA_ERR_INVALID;
  if (cache->num_pages == 0 || cache->table_width == 0) return FA_ERR_INVALID;
  const fa_strides none{0, 0, 0}, kp{cache->k_page, cache->k_head, cache->k_row},
      vp{cache->v_page, cache->v_head, cache->v_row};
  fa::RopeArgs a{};
  a.q = rope_rows(Xq, Hq ? *xq : none, Yq, Hq ? *yq : none, Hq);
  a.k = rope_rows(K, *xk, cache->k_pages, kp, cache->heads);
  a.v = rope_rows(V, *xv, cache->v_pages, vp, cache->heads);
  a.positions = positions;
  a.freqs = freqs;
  a.rot = freqs != nullptr ? rot_dim : 0;
  a.d = cache->d;
  a.magnitude = magnitude;
  a.sign = 1.f;
  a.N = cache->tokens;
  a.rows = cache->tokens;
  a.cache = view_of(*cache);
  return launch_rope<true>(a, interleaved != 0, cache->dtype, static_cast<cudaStream_t>(stream));
}

size_t fa_paged_workspace_size(int tokens, int max_q, int Hq, int heads, int d) {
  if (tokens < 0 || max_q < 0 || Hq < 0 || heads <= 0 || d < 0) return static_cast<size_t>(-1);
  return 0;
}

int fa_paged_attention(const fa_paged_cache* cache, const void* Q, const fa_strides* xq, void* O,
                       const fa_strides* xo, float* L, int Hq, int max_q, int window_left,
                       int window_right, float scale, void* workspace, size_t workspace_bytes,
                       void* stream) {
  const int st = check_cache(cache, true);
  if (st != FA_OK) return st;
  if (Hq < 0 || Hq % cache->heads != 0 || max_q < 0) return FA_ERR_INVALID;
  if (!(scale > 0.f) || !isfinite(scale)) return FA_ERR_INVALID;
  if (Hq / cache->heads > 128) return FA_ERR_UNSUPPORTED;
  if (cache->batch == 0 || cache->tokens == 0 || Hq == 0) return FA_OK;
  if (!ok_ptr(Q) || !ok_ptr(O) || !ok_ptr(L) || !ok_strides(xq) || !ok_strides(xo))
    return FA_ERR_INVALID;
  const size_t need =
      fa_paged_workspace_size(cache->tokens, max_q, Hq, cache->heads, cache->d);
  if (need > 0 && (!ok_ptr(workspace, 256) || workspace_bytes < need)) return FA_ERR_INVALID;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf = cache->dtype == FA_BF16;
  if (cache->d == 64)
    return bf ? launch_simple<64, true>(*cache, Q, *xq, O, *xo, L, Hq, max_q, window_left,
                                        window_right, scale, s)
              : launch_simple<64, false>(*cache, Q, *xq, O, *xo, L, Hq, max_q, window_left,
                                         window_right, scale, s);
  return bf ? launch_simple<128, true>(*cache, Q, *xq, O, *xo, L, Hq, max_q, window_left,
                                       window_right, scale, s)
            : launch_simple<128, false>(*cache, Q, *xq, O, *xo, L, Hq, max_q, window_left,
                                        window_right, scale, s);
}

int fa_paged_device_status(void* stream) {
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return FA_ERR_CUDA;
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, fa::g_fa_status, sizeof(int)) != cudaSuccess) return FA_ERR_CUDA;
  if (v != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(fa::g_fa_status, &zero, sizeof(int)) != cudaSuccess)
      return FA_ERR_CUDA;
  }
  return v;
}

}  // extern "C"
