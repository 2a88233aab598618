/*
 * snip_kv.h -- attention over a key/value cache held in 4 bits, in the same
 * library as snip.h (libsnip): appending keys and values to a paged cache
 * with the position rotation on the way, attention of the new tokens over the
 * cache (decode steps, drafted tokens, prompts), and reading cached tokens back.
 *
 * Conventions are those of snip_ops.h (caller-owned buffers, validation before
 * any HIP call, int status, snip_last_error(), work enqueued on `stream`;
 * element types SNIPOP_BF16 / SNIPOP_F32, leading dimensions in elements,
 * 16-byte aligned matrices). A matrix here has a row for each new token and
 * heads * head_dim columns.
 *
 * The cache is made of pages that the caller hands to sequences. A head's
 * values of a token are E2M1 codes, two to a byte, low nibble first, with a
 * scale for each block of 16 (NVFP4: E4M3) or 32 (MXFP4: E8M0) dimensions.
 * Within a page they lie in the order that the attention reads them in, p, s, v
 * being the bytes of a key's piece, of its scales and of a value's piece:
 *   k_codes  [pages][kv_heads][page_size/16][head_dim/2/p][16 tokens][p]
 *   k_scales [pages][kv_heads][page_size/16][head_dim/block/s][16 tokens][s]
 *   v_codes  [pages][kv_heads][page_size/4][head_dim/2/v][4 tokens][v]
 *   v_scales [pages][kv_heads][page_size/4][head_dim/block][4 tokens]
 *   p = 16, v = 4 (head_dim 64: 8 and 2); s = 2p/block, at least 1.
 */
#ifndef SNIP_KV_H
#define SNIP_KV_H

#include "snip_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* launch kinds in the timing records (snip_timing_*), next to SNIPOP_LAUNCH_* */
#define SNIPKV_LAUNCH_APPEND  8   /* append, gather; work: elements                       */
#define SNIPKV_LAUNCH_ATTN    9   /* attention; work: 4 * tokens * q_heads * head_dim     */
#define SNIPKV_LAUNCH_JOIN   10   /* joining split sequences; work: the same              */

#define SNIPKV_MAX_PAGE_SIZE 4096

typedef struct snipkv_cache {
  int32_t format;       /* SNIP_NVFP4 or SNIP_MXFP4                                     */
  int32_t page_size;    /* tokens of a page: a power of two, 16 .. SNIPKV_MAX_PAGE_SIZE */
  int32_t kv_heads;     /* 1 .. 1024                                                    */
  int32_t head_dim;     /* 64, 128 or 256                                               */
  int64_t pages;        /* pages that the buffers hold, 1 .. 2^31 - 1                   */
  void* k_codes;        /* device, 16-byte aligned, as laid out above                   */
  void* k_scales;
  void* v_codes;
  void* v_scales;
  const int32_t* texp;  /* NVFP4: device [2], the power of two that all keys, and all
                           values, are stored under: x = code * scale * 2^texp. The
                           caller's choice, made once (the smallest e with
                           max|x| <= 2688 * 2^e); unused for MXFP4                      */
} snipkv_cache;

/* The sequences of a call and their new tokens, which are each sequence's last.
 * Row t of the call's matrices is a token of sequence b if cu[b] <= t < cu[b+1]
 * (without cu: t == b); its position is lens[b] - (cu[b+1] - t), and the tokens
 * at page_size * i .. lie in page table[b][i]. A position below 0, one behind the
 * table, and one whose table entry is outside 0 .. pages - 1 (a page that was
 * given back, say) is not mapped: nothing is written there, and its key takes
 * no part. Rows from cu[seqs] on belong to nobody: what they hold does not
 * matter and they are not written, so a captured call may hold more rows than it
 * uses. A call has 1 .. 2^20 tokens; attention takes SHAPE for more than 2^24
 * tiles of 16 rows (a kv head's tokens times its query heads, and one a sequence)
 * or 2^30 over all kv heads. */
typedef struct snipkv_batch {
  const int32_t* table;  /* device [seqs][table_ld], max_pages entries used              */
  int64_t table_ld;
  int64_t max_pages;     /* >= 1; max_pages * page_size <= 2^30                          */
  const int32_t* lens;   /* device [seqs], the call's tokens included                    */
  const int32_t* cu;     /* device [seqs + 1], ascending from 0, or NULL: a token each   */
  int64_t seqs;          /* 1 .. 2^20                                                    */
} snipkv_batch;

/* Rotates queries and keys and appends keys and values:
 *   pair (a, b) at position p, angle row (c, s) = (cos[p][i], sin[p][i]):
 *   a' = a c - b s,  b' = b c + a s      (fp32, each operation rounded)
 * over the first rot_dim dimensions of a head, pairs (i, i + rot_dim/2), or
 * (2i, 2i + 1) where interleaved; then keys and values are quantized to nearest
 * as snip_quantize would a tensor with rows of head_dim, under the cache's texp.
 * A block's maximum is that of its finite elements; an infinity is stored as the
 * block's largest code, or as zero where the maximum is zero (NVFP4: or too small
 * for a scale above zero), NaN as zero.
 *   q         device [tokens][q_heads * head_dim], type `type`, ldq; NULL: none.
 *   k, v      device [tokens][kv_heads * head_dim], `type`, ldk, ldv. NULL (both):
 *             queries alone.
 *   cos, sin  device fp32 [angles][rot_dim / 2], 16-byte aligned; rot_dim = 0: no
 *             rotation. rot_dim a multiple of 64 up to head_dim.
 *   pos       device int32 [tokens], the row of the angles, or NULL: the token's
 *             position. Taken as 0 below 0 and as angles - 1 from there on.
 *   q_out     device bf16, ldqo (with q). May be q itself where that is bf16.
 * The positions of the rows must lie in different places: where two sequences
 * of a call share a page and write the same place, what is stored there is a mix
 * of the two.
 * Errors: NULL, SHAPE, ALIGN, FORMAT, HIP. */
int snipkv_append(const void* q, int64_t ldq, int64_t q_heads, const void* k, int64_t ldk, const void* v, int64_t ldv,
                  int type, int64_t tokens, const float* cos, const float* sin, int64_t angles, int64_t rot_dim,
                  int interleaved, const int32_t* pos, const snipkv_cache* cache, const snipkv_batch* batch,
                  void* q_out, int64_t ldqo, void* stream);

/* The cached keys and values of the rows' tokens in bf16 (exact but for the
 * ends of bf16's range); zeros where a position is not mapped.
 *   k, v      device bf16 [tokens][kv_heads * head_dim], ldk, ldv; one may be NULL.
 * Errors: NULL, SHAPE, ALIGN, FORMAT, HIP. */
int snipkv_gather(const snipkv_cache* cache, const snipkv_batch* batch, int64_t tokens, void* k, int64_t ldk,
                  void* v, int64_t ldv, void* stream);

/* Attention of the new tokens over the cache, which holds them already:
 *   s_j = scale * q . k_j  over the mapped positions j <= p, and j > p - window
 *   where window > 0;   out = sum_j softmax(s)_j v_j;   lse = log sum_j exp s_j
 * for every row and query head; head h reads kv head h / (q_heads / kv_heads).
 * A row with no key at all: out = 0, lse = -infinity. fp32 throughout, but the
 * softmax's terms, which enter the matrix product in fp16 (MXFP4: in two parts
 * of bf16); out is rounded once. Not defined for scores past 2e38 (NVFP4: nor for
 * rows where scale * 2^texp[0] * max|q| is, whatever the keys; MXFP4: nor for a
 * q . k_j that is, whatever the scale), values past 1e30, and scales of NaN (which
 * append never stores) in places that a row of the call sees: other rows of the
 * call may become NaN. The same inputs give the same bits.
 *   q         device bf16 [tokens][q_heads * head_dim], ldq.
 *   scale     > 0, up to 2e38.
 *   window    0: none; else >= 1.
 *   out       device bf16, ldo. May be q itself.
 *   lse       device fp32 [tokens][q_heads] or NULL.
 *   ws        device, 16-byte aligned, snipkv_attn_workspace() bytes, which may
 *             hold anything; calls that run at the same time need their own.
 * Errors: NULL, SHAPE, ALIGN, FORMAT, WORKSPACE, HIP. */
int snipkv_attn(const void* q, int64_t ldq, int64_t q_heads, int64_t tokens, const snipkv_cache* cache,
                const snipkv_batch* batch, float scale, int64_t window, void* out, int64_t ldo, float* lse,
                void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes of snipkv_attn (0 on invalid arguments). */
size_t snipkv_attn_workspace(int64_t tokens, int64_t seqs, int64_t q_heads, int64_t kv_heads, int64_t head_dim);

#ifdef __cplusplus
}
#endif

#endif /* SNIP_KV_H */
