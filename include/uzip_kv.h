/*
 * uzip_kv.h -- KV-cache operators next to the codec of uzip.h, for AMD
 * Instinct MI355X (gfx950): what a serving step does to a cache before it is
 * encoded for its transfer and after it is decoded.
 *
 *   uzip_kv_rope    rotary positions of a tensor, or the inverse rotation
 *   uzip_kv_append  rotary positions of new queries and keys; keys and values
 *                   written into the cache
 *   uzip_kv_attend  attention of each sequence's drafted tokens (one token, a
 *                   chain or a tree) over its cache and over each other; the
 *                   attention weight each cached token received, added up
 *   uzip_kv_evict   the cache cut to a number of tokens per head by that
 *                   weight, in the layout uzip_encode takes
 *
 * Conventions are those of uzip.h: device pointers (d_* and the pointers in
 * the structures below) are memory that the caller owns, 16-byte aligned
 * unless a comment says otherwise; the library allocates no device memory and
 * keeps no state between calls; calls only enqueue work on stream s;
 * arguments are checked on the host first, and a failed check returns a
 * negative UZIP_E* code and enqueues nothing. Workspaces are scratch: two
 * calls that may overlap (two streams, two graphs replayed at once) need two.
 * Values in device memory (lengths, page tables, positions) cannot be checked
 * on the host: whatever they hold, no kernel reads or writes outside the
 * described tensors (see each field).
 *
 * All strides are in elements. The head dim is contiguous and a multiple of 8
 * up to 256; every stride of a q, k, v or output tensor is a multiple of 8,
 * not negative, and a token stride is below 2^26.
 */
#ifndef UZIP_KV_H
#define UZIP_KV_H

#include "uzip.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types */
#define UZIP_KV_BF16 0u
#define UZIP_KV_F16  1u
#define UZIP_KV_E5M2 2u       /* caches only */

/* A cache of keys and values.
 * Contiguous (table NULL): element (sequence b, token t, head h, dim d) of the
 * keys is k[b * k_stride[0] + t * k_stride[1] + h * k_stride[2] + d], t <
 * tokens. In pages (table not NULL): token t of sequence b is row t % page of
 * page table[b * table_stride + t / page], and stride [0] is the one between
 * pages; page is a power of two, at least 16, and tokens is the table's
 * entries per sequence times page. A table entry outside [0, pages) is an
 * absent page: its tokens are seen by no query, appended tokens that fall
 * into it are dropped and evicted rows of it are zeros. */
typedef struct uzip_kv_cache {
    void          *k;
    void          *v;
    const int32_t *table;       /* 4-byte aligned */
    int64_t        k_stride[3];
    int64_t        v_stride[3];
    int64_t        table_stride;
    uint32_t       dtype;
    uint32_t       seqs;
    uint32_t       heads;       /* key/value heads */
    uint32_t       dim;
    uint32_t       tokens;
    uint32_t       page;
    uint32_t       pages;
    uint32_t       reserved;    /* 0 */
} uzip_kv_cache_t;

/* Rotary positions. With half = rot / 2 pairs, pair i is elements (i, half +
 * i) of the head, or (2i, 2i + 1) with UZIP_KV_INTERLEAVED; elements from rot
 * on are left as they are. At position p pair i turns by p * freq[i] turns
 * (the product and its fraction in binary64) and is multiplied by amplitude:
 *   (a, b) -> amplitude * (a cos - b sin, b cos + a sin)
 * in binary32, rounded once to the output's type. UZIP_KV_INVERSE turns the
 * other way: the gradient of the rotation, or a move to earlier positions.
 * freq NULL (with rot 0): no rotation. */
#define UZIP_KV_INTERLEAVED 0x1u
#define UZIP_KV_INVERSE     0x2u
typedef struct uzip_kv_rope {
    const double  *freq;        /* device, rot / 2 turns per position, 8-byte aligned */
    const int32_t *pos;         /* device, position of token t of sequence b at b * pos_stride + t;
                                   NULL (append only): length[b] + t */
    int64_t        pos_stride;
    uint32_t       rot;         /* even, at most the head dim */
    uint32_t       flags;
    float          amplitude;
    uint32_t       reserved;    /* 0 */
} uzip_kv_rope_t;

/* A tensor of tokens: [sequences, tokens, heads, dim]. */
typedef struct uzip_kv_tensor {
    void   *data;
    int64_t stride[3];          /* sequence, token, head */
} uzip_kv_tensor_t;

/* async. y = the rotation of x, both [seqs, tokens, heads, dim] of dtype BF16
 * or F16. y may be x with the same strides; otherwise they do not overlap. */
int uzip_kv_rope(const uzip_kv_tensor_t *x, const uzip_kv_tensor_t *y, uint32_t dtype, uint32_t seqs,
                 uint32_t tokens, uint32_t heads, uint32_t dim, const uzip_kv_rope_t *rope, hipStream_t s);

/* async. Token t of sequence b, t < tokens: q_out = the rotation of q (as
 * uzip_kv_rope; both may be NULL), and, when t < drafted[b] (all t when
 * drafted is NULL), the rotation of k and v itself are rounded to the cache's
 * type (to nearest even; values past E5M2's range become infinities) and
 * written to the cache's token length[b] + t. Tokens outside the cache's
 * capacity or in an absent page are dropped; nothing else in the cache is
 * written. q, k and v have the dtype BF16 or F16, and it is the cache's unless
 * the cache is E5M2. length is not changed. No two sequences may share a page
 * that is written. q_out may be q with the same strides; otherwise nothing that
 * is written overlaps anything else: not q_out and k or v, nor the two caches. */
typedef struct uzip_kv_append_args {
    uzip_kv_tensor_t q, q_out, k, v;
    const int32_t   *length;    /* device, one per sequence */
    const int32_t   *drafted;
    uint32_t         dtype;
    uint32_t         tokens;
    uint32_t         heads;     /* query heads */
    uint32_t         reserved;  /* 0 */
} uzip_kv_append_args_t;
int uzip_kv_append(const uzip_kv_cache_t *cache, const uzip_kv_append_args_t *a, const uzip_kv_rope_t *rope,
                   hipStream_t s);

/* async. Attention of tokens drafted for each sequence over its cache, which
 * holds length[b] earlier tokens and behind them the keys and values of the
 * drafted ones (uzip_kv_append). Query token i of sequence b, i < drafted[b],
 * sees every cached token below length[b], and drafted token j < drafted[b]
 * where tree[b * tree_stride[0] + i * tree_stride[1] + j] is not zero; without
 * a tree, where j <= i. Query head a uses key/value head a / (heads /
 * cache->heads). With s = scale q.k over the seen keys:
 *   lse = log sum exp s,  out = sum exp(s - lse) v,
 *   score[b, kv head, key] += sum over tokens i and the heads of that kv head
 *                             of exp(s - lse)
 * A query that sees nothing, or only keys with s = -inf, gives zeros and lse
 * -inf; so does a token i >= drafted[b]. Keys and values that a query does not
 * see have no effect on it, whatever they hold. A seen value that is not finite
 * leaves its element of the other queries' output not finite, an infinity or
 * NaN, also where the weight of its key rounds to zero. Lengths are clamped to the
 * cache's capacity. Products are exact in binary32 sums. Weights are multiplied
 * with the values in two terms of the cache's type (F16 beside E5M2), so that
 * little but the output's rounding shows; in one, rounded to half a step, where
 * more than 64 rows (tokens * heads / cache->heads) share keys over much work,
 * and for BF16 queries of an E5M2 cache. What score adds is taken with lse as
 * binary32 holds it, so it is off by 2^-23 |lse| of itself: of use below |lse|
 * of about 2^16. lse and score may be NULL. scale is in [2^-60, 2^60]. The result depends on
 * nothing but the inputs: no atomics. Outputs overlap no input. */
typedef struct uzip_kv_attend_args {
    uzip_kv_tensor_t q, out;
    float           *lse;       /* [seqs, tokens, heads], contiguous; 4-byte aligned */
    float           *score;     /* 4-byte aligned */
    int64_t          score_stride[2];  /* sequence, kv head; keys are contiguous */
    const int32_t   *length;
    const int32_t   *drafted;   /* NULL: all */
    const uint8_t   *tree;      /* NULL: a chain */
    int64_t          tree_stride[2];   /* sequence (0: one tree for all), row */
    uint32_t         dtype;     /* of q and out: BF16 or F16; the cache's unless that is E5M2 */
    uint32_t         tokens;
    uint32_t         heads;     /* query heads: a multiple of the cache's */
    float            scale;
    uint32_t         score_tokens;     /* keys a row of score holds, at most cache->tokens: later ones are not added */
    uint32_t         reserved;  /* 0 */
} uzip_kv_attend_args_t;
int uzip_kv_attend(const uzip_kv_cache_t *cache, const uzip_kv_attend_args_t *a, void *d_ws, uint64_t ws_bytes,
                   hipStream_t s);

/* Workspace of uzip_kv_attend for these shapes; 0 when they are invalid. */
uint64_t uzip_kv_attend_workspace_bytes(uint32_t seqs, uint32_t kv_heads, uint32_t dim, uint32_t cache_tokens,
                                        uint32_t tokens, uint32_t heads);

/* async. Cuts a cache to `keep` tokens per sequence and head. With n =
 * length[b] (clamped to [0, score_tokens]), head h keeps min(n, keep) of its
 * tokens: the first min(sink, n), the last min(recent, n), and of the others
 * those with the largest score, ties to the lower token; NaN ranks with -inf.
 * Kept tokens stay in order: slot j of out holds token index[b, h, j]; slots
 * from min(n, keep) on are zeros with index -1. out is contiguous (table
 * NULL), with cache's seqs, heads, dim and dtype and tokens = keep; its memory
 * does not overlap the cache, nor its keys its values. score_out (the kept tokens' scores, 0 behind
 * them) and length_out (min(n, keep)) may be NULL. sink + recent <= keep. */
typedef struct uzip_kv_evict_args {
    const float   *score;
    int64_t        score_stride[2];
    const int32_t *length;
    int32_t       *index;       /* [seqs, heads, keep], contiguous */
    float         *score_out;   /* [seqs, heads, keep], contiguous */
    int32_t       *length_out;  /* [seqs] */
    uint32_t       keep;
    uint32_t       sink;
    uint32_t       recent;
    uint32_t       score_tokens;       /* scores a row holds, at most cache->tokens: the cache is taken to end there */
} uzip_kv_evict_args_t;
int uzip_kv_evict(const uzip_kv_cache_t *cache, const uzip_kv_cache_t *out, const uzip_kv_evict_args_t *a,
                  void *d_ws, uint64_t ws_bytes, hipStream_t s);

/* Workspace of uzip_kv_evict, cache_tokens the scores a row holds; 0 when it
 * needs none (d_ws may then be NULL) or the shapes are invalid. */
uint64_t uzip_kv_evict_workspace_bytes(uint32_t seqs, uint32_t kv_heads, uint32_t cache_tokens);

#ifdef __cplusplus
}
#endif

#endif /* UZIP_KV_H */
