/*
 * fa_paged.h -- C ABI of libfa_paged.so: rotary positions, a paged key/value cache and
 * exact attention over it, for B200 (sm_100a). It stands beside fa.h: the same status
 * codes, 16-bit types, masks and ownership rules, in a library of its own.
 *
 * Rotary positions. The first rot_dim columns of a head are r/2 pairs (r = rot_dim), pair
 * i being columns (i, i + r/2) in the half form and (2 i, 2 i + 1) in the interleaved
 * form. A row at position pos turns pair i by the angle a = pos * freqs[i]:
 *     y0 = magnitude * (x0 cos a - x1 sin a),   y1 = magnitude * (x1 cos a + x0 sin a);
 * the other columns are copied. The angle is formed in 64 bits, the rotation in 32, and
 * the result is rounded once.
 *
 * Paged cache. Key j of sequence b is row j % page_size of page table[b][j / page_size];
 * K and V have pages of the same shape in two arrays with their own strides (so both may
 * be views of one pool). Tokens of a ragged batch are packed: sequence b owns the rows
 * cu_q[b] .. cu_q[b+1] - 1 of Q, K, V and O, its n = cu_q[b+1] - cu_q[b] new tokens, and
 * holds seq_k[b] cached keys, the new tokens included as its last n. Rows behind
 * cu_q[batch] belong to no sequence and are neither read nor written.
 *
 * Masks are fa.h's: with off = seq_k[b] - n, query i of a sequence sees key j iff
 * i + off - window_left <= j <= i + off + window_right (negative edge: unbounded);
 * (-1, 0) is causal. Query head h reads key head h / (Hq / heads). A row that sees no key
 * gets O = 0 and L = -inf. V rows of keys that no query of the attention tile at hand sees
 * are never multiplied, whatever they hold, nor are pages that only such keys lie in read.
 * V rows that some of a tile's queries see must be finite (a weight of 0 for the others
 * does not take a NaN or an infinity away); a NaN score, or one of +infinity, makes its own
 * row's O and L NaN.
 *
 * Lengths, tables and positions are read on the device, so a captured graph follows what
 * they hold when it runs. What the host cannot check is checked there: a sequence whose
 * lengths are inconsistent (cu_q decreasing or above the packed rows, more keys than the
 * table's width holds, fewer keys than new tokens in an append) is left out, by an attention
 * the whole batch if cu_q decreases anywhere (rows might belong to two sequences), and a page
 * index outside [0, num_pages) reads as zeros and is not written; each makes the next
 * fa_paged_device_status return FA_ERR_INVALID.
 *
 * Pointers are device pointers of the current device, 16-byte aligned (4 for the 32-bit
 * integer arrays, 8 for freqs); strides are in elements, the last dimension is dense, and
 * the other strides are multiples of 8 elements. Every call only enqueues work on
 * `stream`, with launches that overlap the end of the kernel before them; none reads or
 * writes memory before that kernel has ended. The caller owns every buffer; two calls that
 * may run at the same time need workspaces of their own. Outputs must not overlap inputs
 * except where a call says so.
 *
 * Errors are fa.h's codes, returned before anything is enqueued: FA_ERR_INVALID for null or
 * misaligned pointers, negative sizes, strides that are negative or no multiple of 8, bad
 * scales, magnitudes or rotation sizes, a workspace that is too small; FA_ERR_UNSUPPORTED
 * for dtypes, head dims, page sizes and group sizes other than named below, more than 8192
 * sequences, 1024 key heads or 2^28 packed rows or keys per sequence, a stride of 0 over
 * more than one row in an attention or in what a call writes, or a batch of 2^31 and more
 * (item, key tile) pairs by its bounds (tokens, batch, table_width); FA_ERR_CUDA when CUDA
 * refuses a launch.
 */
#ifndef FA_PAGED_H_
#define FA_PAGED_H_

#include <stddef.h>

#include "fa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element strides of a [B][H][N][d] tensor in whatever order it lies in memory. */
typedef struct {
    long long b, h, n;
} fa_strides;

typedef struct {
    void *k_pages;                     /* page p, head h, row j: p*k_page + h*k_head + j*k_row */
    void *v_pages;
    long long k_page, k_head, k_row;   /* element strides */
    long long v_page, v_head, v_row;
    const int *table;                  /* [batch][table_row], the first table_width used */
    const int *cu_q;                   /* [batch + 1] */
    const int *seq_k;                  /* [batch] */
    int table_row, table_width;
    int num_pages, page_size;          /* page_size: a power of two, 16 .. 1024 */
    int heads, d;                      /* key heads; d = 64 or 128 (append: see there) */
    int batch, tokens;                 /* sequences (up to 8192); packed rows of Q, K, V, O */
    int dtype;                         /* FA_BF16 or FA_FP16 */
    int reserved;
} fa_paged_cache;

/* Rows of heads that are rotated from x to y; heads = 0: none, the rest is not looked at. */
typedef struct {
    const void *x;
    void *y;
    fa_strides xs, ys;
    int heads;
    int reserved;
} fa_rope_rows;

/*
 * Rotates q [batch][q.heads][rows][d] and k [batch][k.heads][rows][d] in one launch;
 * `inverse` = 1 turns by -a instead, which is the gradient of the rotation (same
 * magnitude). Row n of batch b is at positions[b * pos_row + n] (pos_row = 0: the same for
 * every batch), or at n when positions is NULL. y may be x with the same strides (in
 * place; FA_ERR_INVALID with others); otherwise they must not overlap. d and rot_dim are multiples of 16,
 * 16 <= rot_dim <= d <= 1024.
 */
typedef struct {
    fa_rope_rows q, k;
    const int *positions;
    long long pos_row;
    const double *freqs;               /* [rot_dim / 2] */
    int rot_dim, interleaved, inverse;
    int batch, rows, d, dtype;
    float magnitude;
} fa_rope_args;
int fa_rope(const fa_rope_args *args, void *stream);

/*
 * Writes the new tokens' keys and values, k and v [tokens][heads][d] (strides h and n),
 * into their pages: V as it is, K rotated (freqs not NULL) or as it is (freqs NULL). Token
 * i of a sequence takes position seq_k[b] - n + i; `positions` [tokens], if given, replaces
 * it in the rotation only. With q.heads > 0 it also rotates q [tokens][q.heads][d] (strides
 * h and n) in the same launch; that needs freqs. Here d is any multiple of 16 up to 1024.
 * Tokens of sequences that share a page row race for it.
 */
typedef struct {
    fa_paged_cache cache;
    const void *k, *v;
    fa_strides ks, vs;
    fa_rope_rows q;
    const int *positions;
    const double *freqs;
    int rot_dim, interleaved;
    float magnitude;
    int reserved;
} fa_paged_append_args;
int fa_paged_append(const fa_paged_append_args *args, void *stream);

/*
 * Exact attention of the packed queries q [tokens][heads_q][d] (strides h and n) over the
 * cache: out [tokens][heads_q][d] and lse [heads_q][tokens] (fp32, natural log). heads_q is
 * a multiple of cache.heads, heads_q / cache.heads <= 128. max_q bounds the new tokens of
 * any sequence (one with more is left out, as above); it picks the kernel: up to 16 rows
 * (tokens x query heads of a key head; 24 at d = 128) are a step, more are a chunk. Work is
 * shared out evenly over the SMs by key tiles, so a sequence's keys may be split between
 * CTAs; the parts are joined by their log-sum-exps in a fixed order. Results are the same
 * bits on every call with the same lengths (the split, and so the rounding, of a sequence
 * depends on the lengths of the others). The weights are rounded to the 16-bit type for
 * their product with V, relative to about the largest so far: in fp16 those below 2^-14 of
 * it lose digits and those below 2^-25 vanish. A step divides the product by the sum of the
 * rounded weights, a chunk by that of the unrounded ones: there the rounding of a weight that
 * dominates its row stays in O, up to half a step of its key's value, and weights that
 * vanish still count in the sum. With max_q = 0 nothing is done. The workspace is 256-byte
 * aligned; its contents do not matter. Two launches.
 */
typedef struct {
    fa_paged_cache cache;
    const void *q;
    void *out;
    float *lse;
    fa_strides qs, os;
    int heads_q, max_q, window_left, window_right;
    float scale;
    int reserved;
    void *workspace;
    size_t workspace_bytes;
} fa_paged_attention_args;
size_t fa_paged_workspace_size(int tokens, int max_q, int heads_q, int heads, int d);
int fa_paged_attention(const fa_paged_attention_args *args, void *stream);

/* fa_get_device_status for the kernels of this library: synchronises `stream`, returns
 * and clears the current device's error word (FA_ERR_INVALID: see above). */
int fa_paged_device_status(void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_PAGED_H_ */
