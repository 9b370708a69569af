// fa_paged_api.cu -- the C ABI declared in include/fa_paged.h: argument checks and kernel
// launches. All device work is in the .cuh kernels beside it.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "fa_paged.h"
#include "fa_paged_common.cuh"
#include "fa_paged_chunk.cuh"
#include "fa_paged_merge.cuh"
#include "fa_paged_step.cuh"
#include "fa_rope.cuh"

namespace {

constexpr float kLog2e = 1.4426950408889634074f;

bool aligned(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}
bool ok_ptr(const void* p, uintptr_t bytes = 16) { return p != nullptr && aligned(p, bytes); }

// Rows are moved in 16-byte pieces, so every stride is a multiple of 8 elements.
bool ok_strides(const fa_strides& s) {
  return s.b >= 0 && s.h >= 0 && s.n >= 0 && (s.b | s.h | s.n) % 8 == 0;
}
fa::Strides strides(const fa_strides& s) {
  return {static_cast<long>(s.b), static_cast<long>(s.h), static_cast<long>(s.n)};
}

// Launches a kernel so that it may begin before the one ahead of it in the stream has
// ended: every kernel here waits for that end itself before it touches memory.
template <typename... Params, typename... Args>
int launch(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
           const Args&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// ------------------------------------------------------------------ rotation
int check_rotation(int d, int rot_dim, float magnitude, const double* freqs) {
  if (!ok_ptr(freqs, 8) || !isfinite(magnitude)) return FA_ERR_INVALID;
  if (rot_dim < 16 || rot_dim > d) return FA_ERR_INVALID;
  return rot_dim % 16 == 0 ? FA_OK : FA_ERR_UNSUPPORTED;
}

// Tokens of a block: one while that gives every SM at most a few blocks (a token's rows
// then finish soonest), more for long inputs.
int rope_tokens_per_block(long rows, int groups) {
  int t = 1;
  while (t < fa::kRopeMaxTokens && rows / (2 * t) >= 148 * 4 &&
         fa::kRopeThreads / groups / (2 * t) >= 1)
    t *= 2;
  return t;
}

template <bool PAGED>
int launch_rope(fa::RopeArgs& a, bool interleaved, int dtype, cudaStream_t stream) {
  a.tokens_per_block = rope_tokens_per_block(a.rows, a.d / 16);
  const fa::RopeRows& most = a.kinds[a.kinds[0].heads > 0 ? 0 : 1];
  a.tokens_first = most.ss.sn < most.ss.sh;
  const long blocks = (a.rows + a.tokens_per_block - 1) / a.tokens_per_block;
  if (blocks >= (1L << 31)) return FA_ERR_UNSUPPORTED;
  const size_t smem = static_cast<size_t>(a.tokens_per_block) * a.rot * sizeof(float);
  const dim3 grid(static_cast<unsigned>(blocks));
  return launch(dtype == FA_BF16 ? fa::fa_rope_kernel<PAGED, true>
                                 : fa::fa_rope_kernel<PAGED, false>,
                grid, fa::kRopeThreads, smem, stream, a, interleaved);
}

// A stride of 0 over more than one row aliases rows: no tensor map describes them, and
// writing them would leave whichever came last.
bool steps(long long stride, long long rows) { return rows <= 1 || stride > 0; }
bool cache_steps(const fa_paged_cache& c) {
  return steps(c.k_row, c.page_size) && steps(c.k_head, c.heads) && steps(c.k_page, c.num_pages) &&
         steps(c.v_row, c.page_size) && steps(c.v_head, c.heads) && steps(c.v_page, c.num_pages);
}

// Rows of heads to rotate, `n` of each of `batch`. In place the strides have to be the same:
// a thread reads the columns of a row that it writes, before it writes them, and no others.
int check_rows(const fa_rope_rows& r, int batch, int n) {
  if (r.heads == 0) return FA_OK;
  if (!ok_ptr(r.x) || !ok_ptr(r.y) || !ok_strides(r.xs) || !ok_strides(r.ys))
    return FA_ERR_INVALID;
  if (!steps(r.ys.b, batch) || !steps(r.ys.h, r.heads) || !steps(r.ys.n, n))
    return FA_ERR_UNSUPPORTED;
  if (r.x == r.y && ((batch > 1 && r.xs.b != r.ys.b) || (r.heads > 1 && r.xs.h != r.ys.h) ||
                     (n > 1 && r.xs.n != r.ys.n)))
    return FA_ERR_INVALID;
  return FA_OK;
}
fa::RopeRows rope_rows(const fa_rope_rows& r) {
  return {static_cast<const uint16_t*>(r.x), static_cast<uint16_t*>(r.y), strides(r.xs),
          strides(r.ys), r.heads};
}

// --------------------------------------------------------------------- cache
int check_cache(const fa_paged_cache* c, bool attention) {
  if (c->batch < 0 || c->tokens < 0 || c->heads <= 0 || c->d <= 0 || c->num_pages < 0 ||
      c->table_width < 0 || c->table_row < 0)
    return FA_ERR_INVALID;
  if (c->dtype != FA_BF16 && c->dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
    return FA_ERR_UNSUPPORTED;
  if (attention ? c->d != 64 && c->d != 128 : c->d % 16 != 0 || c->d > fa::kRopeMaxDim)
    return FA_ERR_UNSUPPORTED;
  if (c->batch > 8192 || c->heads > 1024 || c->tokens > (1 << 28) ||
      static_cast<long long>(c->table_width) * c->page_size > (1 << 28))
    return FA_ERR_UNSUPPORTED;
  if (c->batch == 0 || c->tokens == 0) return FA_OK;
  if (!ok_ptr(c->cu_q, 4) || !ok_ptr(c->seq_k, 4)) return FA_ERR_INVALID;
  if (c->table_width > 0 && !ok_ptr(c->table, 4)) return FA_ERR_INVALID;
  if (c->num_pages > 0 && (!ok_ptr(c->k_pages) || !ok_ptr(c->v_pages))) return FA_ERR_INVALID;
  const fa_strides k{c->k_page, c->k_head, c->k_row}, v{c->v_page, c->v_head, c->v_row};
  if (!ok_strides(k) || !ok_strides(v)) return FA_ERR_INVALID;
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

// ----------------------------------------------------------------- attention
constexpr int kGrid = fa::kSplitGrid;
constexpr size_t kMaxDynSmem = 232448;  // 227 KB per block on sm_100

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// A 16-bit tensor of four dimensions (columns first, dense) with element strides of the
// other three; boxes of 64 columns x box1 x box2, 128-byte swizzle, zeros outside.
bool make_tmap(CUtensorMap* map, const void* ptr, int dtype, const long long (&dims)[4],
               const long long (&elems)[3], int box1, int box2) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  cuuint64_t size[4], strides[3];
  for (int i = 0; i < 4; ++i) size[i] = static_cast<cuuint64_t>(dims[i]);
  // a dimension of one is never stepped over: any valid stride does
  for (int i = 0; i < 3; ++i)
    strides[i] = static_cast<cuuint64_t>(dims[i + 1] == 1 ? dims[0] : elems[i]) * 2;
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box1), static_cast<cuuint32_t>(box2), 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  return enc(map,
             dtype == FA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                              : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
             4, const_cast<void*>(ptr), size, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The parts' outputs, fp32 rows of d columns, in boxes of 32 columns x 32 rows.
bool make_part_tmap(CUtensorMap* map, const float* ptr, int d, int rows) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  const cuuint64_t size[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows)};
  const cuuint64_t stride[1] = {static_cast<cuuint64_t>(d) * 4};
  const cuuint32_t box[2] = {32, 32}, step[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<float*>(ptr), size, stride, box,
             step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Rows (tokens x query heads of a key head) that the step kernel takes for one pass; the
// chunk kernel takes more. 24 sequences with 500 to 8000 keys, 32 heads over 8, step and
// chunk: 20 / 24 / 28 / 32 rows 60 / 64 / 67 / 70 and 64 / 64 / 64 / 64 us at d = 128 (96
// sequences, a key head for each query head: 20 rows 194 and 210, 28 rows 212 and 212),
// 20-32 rows 63 and 54 us at d = 64 (a tile there has half the bytes and the same softmax).
int step_max_rows(int d) { return d == 128 ? 24 : 16; }

// Workspace: a PartInfo per CTA, then base-2 log-sum-exps and normalised outputs (fp32) of
// two parts per CTA, `rows` rows each.
struct Workspace {
  int rows;
  size_t l_at, o_at, bytes;
};
Workspace workspace_for(int max_q, int group, int d) {
  Workspace w;
  const long long rows = static_cast<long long>(max_q) * group;
  w.rows = rows <= 16 ? 16 : rows <= step_max_rows(d) ? 32 : fa::kChunkRows;
  w.l_at = kGrid * sizeof(fa::PartInfo);
  w.o_at = w.l_at + 2ull * kGrid * w.rows * sizeof(float);
  w.bytes = w.o_at + 2ull * kGrid * w.rows * d * sizeof(float);
  return w;
}

struct AttentionArgs {
  const fa_paged_cache* c;
  const void* Q;
  fa_strides xq;
  void* O;
  fa_strides xo;
  float* L;
  int group, max_q, wl, wr;
  float scale;
  Workspace ws;
  uint8_t* workspace;
  cudaStream_t stream;

  fa::PartInfo* parts() const { return reinterpret_cast<fa::PartInfo*>(workspace); }
  float* lpart() const { return reinterpret_cast<float*>(workspace + ws.l_at); }
  float* opart() const { return reinterpret_cast<float*>(workspace + ws.o_at); }
};

// Tensor maps of the queries (column, head of a group, token, key head) and of the pages
// (column, row, key head, page). `tokens`: of a query box.
bool make_maps(const AttentionArgs& a, int tokens, CUtensorMap* q, CUtensorMap* k,
               CUtensorMap* v) {
  const fa_paged_cache& c = *a.c;
  const int rows = c.page_size < fa::kKeyTile ? c.page_size : fa::kKeyTile;
  return make_tmap(q, a.Q, c.dtype, {c.d, a.group, c.tokens, c.heads},
                   {a.xq.h, a.xq.n, a.xq.h * a.group}, a.group, tokens) &&
         make_tmap(k, c.k_pages, c.dtype, {c.d, c.page_size, c.heads, c.num_pages},
                   {c.k_row, c.k_head, c.k_page}, rows, 1) &&
         make_tmap(v, c.v_pages, c.dtype, {c.d, c.page_size, c.heads, c.num_pages},
                   {c.v_row, c.v_head, c.v_page}, rows, 1);
}

// Joins the parts of items whose query tiles have `tile_tokens` tokens, with `per_sm` blocks
// for each SM.
template <int D, bool BF16>
int launch_merge(const AttentionArgs& a, int tile_tokens, unsigned per_sm) {
  return launch(fa::fa_paged_merge_kernel<D, BF16>, dim3(kGrid * per_sm), fa::kMergeThreads, 0,
                a.stream, static_cast<const float*>(a.opart()),
                static_cast<const float*>(a.lpart()),
                static_cast<const fa::PartInfo*>(a.parts()), a.ws.rows, tile_tokens, fa::kKeyTile,
                a.group, static_cast<uint16_t*>(a.O), strides(a.xo), a.L, a.c->tokens);
}

// A kernel's shared-memory limit, set on every call: it is the current context's.
template <typename Kernel>
bool allow_smem(Kernel kernel, size_t smem) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(smem)) == cudaSuccess;
}

// The least cost (in key tiles, those for starting an item included) that is worth a CTA of its
// own: one token over 1000 keys (32 heads over 8) takes 9.2 / 9.5 / 9.9 / 10.7 / 13.3 us
// with 1 / 2 / 3 / 4 / 8, over 4000 keys 11.2 / 10.7 / 10.8 / 11.2 / 13.6, a prompt of 300
// tokens 18.2 / 21.5 / 25.4 / 30.3 with 2 / 4 / 6 / 8.
constexpr int kLeastCost = 2;

template <int D, int NQ, bool BF16>
int launch_step(const AttentionArgs& a) {
  using Lay = fa::StepLayout<D, NQ>;
  static_assert(Lay::kBytes <= kMaxDynSmem, "shared memory");
  auto kern = fa::fa_paged_step_kernel<D, NQ, BF16>;
  if (!allow_smem(kern, Lay::kBytes)) return FA_ERR_CUDA;
  CUtensorMap q, k, v;
  if (!make_maps(a, a.max_q, &q, &k, &v)) return FA_ERR_CUDA;
  const int st = launch(kern, dim3(kGrid), Lay::kThreads, Lay::kBytes, a.stream, q, k, v,
                        view_of(*a.c), static_cast<uint16_t*>(a.O), strides(a.xo), a.L, a.opart(),
                        a.lpart(), a.parts(), a.group, a.max_q, a.wl, a.wr, kLeastCost,
                        a.scale * kLog2e);
  return st != FA_OK ? st : launch_merge<D, BF16>(a, a.max_q, 2);
}

template <int D, bool BF16>
int launch_chunk(const AttentionArgs& a) {
  using Lay = fa::ChunkLayout<D>;
  static_assert(Lay::kSmem <= kMaxDynSmem, "shared memory");
  auto kern = fa::fa_paged_chunk_kernel<D, BF16>;
  // The kernel moves registers between warpgroups (setmaxnreg); its split adds up to
  // exactly this many registers per thread at launch (the build fails otherwise too).
  static std::atomic<bool> counted{false};
  if (!counted.load(std::memory_order_relaxed)) {
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, kern) != cudaSuccess) return FA_ERR_CUDA;
    if (attr.numRegs != fa::ChunkRoles<D>::kLaunchRegs) return FA_ERR_UNSUPPORTED;
    counted.store(true, std::memory_order_relaxed);
  }
  if (!allow_smem(kern, Lay::kSmem)) return FA_ERR_CUDA;
  CUtensorMap q, k, v;
  const int tpt = fa::kKeyTile / a.group;
  // a warp's 32 rows of the output, where those are whole tokens (the kernel asks the same)
  const int out_tokens = 32 % a.group == 0 ? 32 / a.group : 1;
  CUtensorMap o, part;
  if (!make_maps(a, tpt, &q, &k, &v) ||
      !make_tmap(&o, a.O, a.c->dtype, {a.c->d, a.group, a.c->tokens, a.c->heads},
                 {a.xo.h, a.xo.n, a.xo.h * a.group}, a.group, out_tokens) ||
      !make_part_tmap(&part, a.opart(), D, 2 * kGrid * a.ws.rows))
    return FA_ERR_CUDA;
  const int st = launch(kern, dim3(kGrid), fa::ChunkRoles<D>::kThreads, Lay::kSmem, a.stream, q, k, v,
                        o, part, view_of(*a.c), static_cast<uint16_t*>(a.O), strides(a.xo), a.L,
                        a.lpart(), a.parts(), a.group, a.max_q, a.wl, a.wr, kLeastCost,
                        a.scale * kLog2e);
  return st != FA_OK ? st : launch_merge<D, BF16>(a, tpt, 8);
}

template <int D, bool BF16>
int launch_attention(const AttentionArgs& a) {
  switch (a.ws.rows) {
    case 16: return launch_step<D, 16, BF16>(a);
    case 32:
      if constexpr (D == 128) return launch_step<D, 32, BF16>(a);
      break;
  }
  return launch_chunk<D, BF16>(a);
}

}  // namespace

extern "C" {

int fa_rope(const fa_rope_args* args, void* stream) {
  if (args == nullptr) return FA_ERR_INVALID;
  const fa_rope_args& r = *args;
  if (r.batch < 0 || r.rows < 0 || r.q.heads < 0 || r.k.heads < 0 || r.d <= 0 || r.pos_row < 0)
    return FA_ERR_INVALID;
  if (r.dtype != FA_BF16 && r.dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
  if (r.d % 16 != 0 || r.d > fa::kRopeMaxDim) return FA_ERR_UNSUPPORTED;
  int st = check_rotation(r.d, r.rot_dim, r.magnitude, r.freqs);
  if (st != FA_OK) return st;
  if (static_cast<long long>(r.batch) * r.rows == 0 || r.q.heads + r.k.heads == 0) return FA_OK;
  if ((st = check_rows(r.q, r.batch, r.rows)) != FA_OK) return st;
  if ((st = check_rows(r.k, r.batch, r.rows)) != FA_OK) return st;
  if (!aligned(r.positions, 4)) return FA_ERR_INVALID;
  fa::RopeArgs a{};
  a.kinds[0] = rope_rows(r.q);
  a.kinds[1] = rope_rows(r.k);
  a.positions = r.positions;
  a.pos_row = static_cast<long>(r.pos_row);
  a.freqs = r.freqs;
  a.rot = r.rot_dim;
  a.d = r.d;
  a.magnitude = r.magnitude;
  a.sign = r.inverse ? -1.f : 1.f;
  a.N = r.rows;
  a.rows = static_cast<long>(r.batch) * r.rows;
  return launch_rope<false>(a, r.interleaved != 0, r.dtype, static_cast<cudaStream_t>(stream));
}

int fa_paged_append(const fa_paged_append_args* args, void* stream) {
  if (args == nullptr) return FA_ERR_INVALID;
  const fa_paged_append_args& r = *args;
  const fa_paged_cache& c = r.cache;
  int st = check_cache(&c, false);
  if (st != FA_OK) return st;
  if (r.q.heads < 0 || (r.q.heads > 0 && r.freqs == nullptr)) return FA_ERR_INVALID;
  if (r.freqs != nullptr &&
      (st = check_rotation(c.d, r.rot_dim, r.magnitude, r.freqs)) != FA_OK)
    return st;
  if (c.batch == 0 || c.tokens == 0) return FA_OK;
  if (!ok_ptr(r.k) || !ok_ptr(r.v) || !ok_strides(r.ks) || !ok_strides(r.vs) ||
      !aligned(r.positions, 4))
    return FA_ERR_INVALID;
  if ((st = check_rows(r.q, 1, c.tokens)) != FA_OK) return st;
  if (c.num_pages == 0 || c.table_width == 0) return FA_ERR_INVALID;
  if (!cache_steps(c)) return FA_ERR_UNSUPPORTED;
  const fa_strides kp{c.k_page, c.k_head, c.k_row}, vp{c.v_page, c.v_head, c.v_row};
  fa::RopeArgs a{};
  a.kinds[0] = rope_rows(r.q);
  a.kinds[1] = rope_rows({r.k, c.k_pages, r.ks, kp, c.heads, 0});
  a.kinds[2] = rope_rows({r.v, c.v_pages, r.vs, vp, c.heads, 0});
  a.positions = r.positions;
  a.freqs = r.freqs;
  a.rot = r.freqs != nullptr ? r.rot_dim : 0;
  a.d = c.d;
  a.magnitude = r.magnitude;
  a.sign = 1.f;
  a.N = c.tokens;
  a.rows = c.tokens;
  a.cache = view_of(c);
  return launch_rope<true>(a, r.interleaved != 0, c.dtype, static_cast<cudaStream_t>(stream));
}

size_t fa_paged_workspace_size(int tokens, int max_q, int heads_q, int heads, int d) {
  if (tokens < 0 || max_q < 0 || heads_q < 0 || heads <= 0 || d < 0 || heads_q % heads != 0)
    return static_cast<size_t>(-1);
  if (tokens == 0 || max_q == 0 || heads_q == 0) return 0;
  return workspace_for(max_q < tokens ? max_q : tokens, heads_q / heads, d).bytes;
}

int fa_paged_attention(const fa_paged_attention_args* args, void* stream) {
  if (args == nullptr) return FA_ERR_INVALID;
  const fa_paged_attention_args& r = *args;
  const fa_paged_cache& c = r.cache;
  const int st = check_cache(&c, true);
  if (st != FA_OK) return st;
  if (r.heads_q < 0 || r.heads_q % c.heads != 0 || r.max_q < 0) return FA_ERR_INVALID;
  if (!(r.scale > 0.f) || !isfinite(r.scale)) return FA_ERR_INVALID;
  const int group = r.heads_q / c.heads;
  if (group > 128) return FA_ERR_UNSUPPORTED;
  if (c.batch == 0 || c.tokens == 0 || r.heads_q == 0 || r.max_q == 0) return FA_OK;
  if (!ok_ptr(r.q) || !ok_ptr(r.out) || !ok_ptr(r.lse, 4) || !ok_strides(r.qs) ||
      !ok_strides(r.os))
    return FA_ERR_INVALID;
  if (c.num_pages == 0 || c.table_width == 0) return FA_ERR_INVALID;
  if (!steps(r.qs.h, r.heads_q) || !steps(r.qs.n, c.tokens) || !steps(r.os.h, r.heads_q) ||
      !steps(r.os.n, c.tokens) || !cache_steps(c))
    return FA_ERR_UNSUPPORTED;
  const int max_q = r.max_q < c.tokens ? r.max_q : c.tokens;
  // the split counts key tiles of items in 32 bits
  const Workspace ws = workspace_for(max_q, group, c.d);
  const int tpi = ws.rows == fa::kChunkRows ? 2 * (fa::kKeyTile / group) : max_q;
  const long long items = c.tokens / tpi + c.batch;
  const long long tiles = static_cast<long long>(c.table_width) * c.page_size / fa::kKeyTile + 2;
  if (items * c.heads > fa::kMaxCost / (tiles + fa::kChunkItemCost)) return FA_ERR_UNSUPPORTED;
  if (!ok_ptr(r.workspace, 256) || r.workspace_bytes < ws.bytes) return FA_ERR_INVALID;
  const AttentionArgs a{&c,
                        r.q,
                        r.qs,
                        r.out,
                        r.os,
                        r.lse,
                        group,
                        max_q,
                        edge(r.window_left),
                        edge(r.window_right),
                        r.scale,
                        ws,
                        static_cast<uint8_t*>(r.workspace),
                        static_cast<cudaStream_t>(stream)};
  const bool bf = c.dtype == FA_BF16;
  if (c.d == 64) return bf ? launch_attention<64, true>(a) : launch_attention<64, false>(a);
  return bf ? launch_attention<128, true>(a) : launch_attention<128, false>(a);
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
