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
 * and, where a small model drafts what the large one answers with:
 *
 *   uzip_kv_append_scaled, uzip_kv_attend_scaled
 *                   the same over a cache in 8 bits with a scale for each
 *                   block of tokens and head
 *   uzip_kv_verify  which drafted tokens the target's probabilities accept
 *   uzip_kv_accept  the accepted tokens of a tree moved up in the cache
 *   uzip_kv_fork, uzip_kv_compact, uzip_kv_copy_pages
 *                   the page table of the next step, and the pages it moves
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
#define UZIP_KV_F32  2u       /* probabilities only */
#define UZIP_KV_E4M3 3u       /* caches with scales only: no infinities, largest value 448 */
#define UZIP_KV_I8   4u       /* caches with scales only: integers, -128 too though none is written */

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

/* Scales of an 8-bit cache: `block` tokens (a power of two from 16 to 65536, at
 * most the page) of a head share one for their keys and one for their values,
 * and an element stands for itself times it. That of token t of sequence b,
 * head h: k[b * k_stride[0] + t / block * k_stride[1] + h * k_stride[2]]; in
 * pages, of row r of page p: k[p * k_stride[0] + r / block * k_stride[1] + ...].
 * Strides are any that are not negative and lead to no element 2^30; 4-byte
 * aligned. Scales of blocks that are seen are positive, in [2^-80, 2^80]: sums of
 * 2^30 weights, each up to 2^8, times values then fit binary32. */
typedef struct uzip_kv_scales {
    float   *k;
    float   *v;
    int64_t  k_stride[3];
    int64_t  v_stride[3];
    uint32_t block;
    uint32_t reserved;          /* 0 */
} uzip_kv_scales_t;

/* async. uzip_kv_append for a cache of E4M3 or I8. The new tokens that a block
 * of a head receives (before they are rounded to any other type) have a largest
 * finite magnitude a, and MAX is 448 or 127. If the block has earlier tokens
 * (below length[b]) and a <= scale * MAX, its scale stays; otherwise it becomes
 * the smallest power of two, at least 2^-60, with a <= scale * MAX, and earlier
 * tokens of the block are rounded to it, each element times old scale / new
 * scale. An element is x / scale rounded to nearest even in binary32; beyond
 * MAX it is MAX with its sign, and NaN is NaN in E4M3, 0 in I8. Of a block that
 * receives nothing nothing is written. A magnitude above 2^80 MAX gets the scale
 * that holds it, beyond the range above: attention over it may be infinite.
 * Drafted tokens that are rejected later have had their part in a scale: it
 * stays, and what rounding to it cost the block's earlier tokens too. */
int uzip_kv_append_scaled(const uzip_kv_cache_t *cache, const uzip_kv_scales_t *scales, const uzip_kv_append_args_t *a,
                          const uzip_kv_rope_t *rope, hipStream_t s);

/* async. uzip_kv_attend over a cache of E4M3 or I8, with queries of BF16 or
 * F16. Weights times the values' scales are multiplied with the values in two
 * terms of BF16, whatever the shapes. uzip_kv_evict and uzip_kv_accept take no
 * such cache: a token that changes its block would have to be rounded again. */
int uzip_kv_attend_scaled(const uzip_kv_cache_t *cache, const uzip_kv_scales_t *scales, const uzip_kv_attend_args_t *a,
                          void *d_ws, uint64_t ws_bytes, hipStream_t s);

/* Workspace of uzip_kv_attend_scaled for these shapes; 0 when they are invalid. */
uint64_t uzip_kv_attend_scaled_workspace_bytes(uint32_t seqs, uint32_t kv_heads, uint32_t dim, uint32_t cache_tokens,
                                               uint32_t tokens, uint32_t heads);

/* async. Which drafted tokens the target accepts. Each sequence has a tree of
 * nodes: node 0 is its last token, node i > 0 is a drafted token tokens[b, i]
 * that follows node parent[b, i] < i (without parent, node i - 1); the children
 * of a node are tried in their order. target[b, i] holds the target's
 * probabilities of the token behind node i. draft[b, i], if there, holds those
 * that the children of node i were drawn from, each anew; without draft they
 * were chosen, not drawn. With c = 0 and mass = 1 at a node's first child, x =
 * tokens[b, i] and u = uniform[b, i] in [0, 1):
 *   with draft     child i is accepted if u q(x) mass < max(p(x) - c q(x), 0);
 *                  else c += mass, and mass = sum max(p - c q, 0)
 *   without        child i is accepted if u mass < p(x), of a token not tried
 *                  there before; else mass -= p(x), and x is taken out of p
 * and the walk goes on at an accepted child. Where none is, the next token is
 * the first one t with sum_{i <= t} left(i) > uniform[b, 0] sum left, left(i) =
 * max(p(i) - c q(i), 0), or p without what was taken out; or p itself if that
 * leaves nothing. All in binary64. The tokens are then distributed as the
 * target's.
 *   path[b]    the accepted nodes in order, node 0 first; -1 behind them
 *   count[b]   how many they are
 *   token[b]   the next token; -1 where there is no probability at all
 * Sequences with drafted[b] = 0 have count 0 and token -1. Probabilities that
 * are not finite or not positive count as 0; nodes with a parent or token that
 * is none are passed over. */
typedef struct uzip_kv_verify_args {
    const void    *target;      /* [seqs, nodes, vocab] of dtype; a row is contiguous */
    const void    *draft;       /* likewise, or NULL */
    int64_t        target_stride[2];   /* sequence, node */
    int64_t        draft_stride[2];
    const int32_t *tokens;      /* [seqs, nodes], rows contiguous, as the next three */
    const int32_t *parent;      /* or NULL: a chain */
    const int32_t *drafted;     /* nodes of each sequence, node 0 among them; NULL: all */
    const float   *uniform;
    int64_t        tokens_stride;
    int64_t        parent_stride;      /* 0: one tree for all */
    int64_t        uniform_stride;
    int32_t       *path;        /* [seqs, nodes], contiguous */
    int32_t       *count;
    int32_t       *token;
    uint32_t       dtype;       /* BF16, F16 or F32 */
    uint32_t       seqs;
    uint32_t       nodes;       /* at most 1024 */
    uint32_t       vocab;
    uint64_t       reserved;    /* 0 */
} uzip_kv_verify_args_t;
int uzip_kv_verify(const uzip_kv_verify_args_t *a, void *d_ws, uint64_t ws_bytes, hipStream_t s);

/* Workspace of uzip_kv_verify for these shapes; 0 when they are invalid. */
uint64_t uzip_kv_verify_workspace_bytes(uint32_t seqs, uint32_t nodes, uint32_t vocab);

/* async. Moves token length[b] + path[b, j] of sequence b to length[b] + j, for
 * j < count[b]: what a tree's accepted nodes appended is then what a chain would
 * have. path[b] increases, as uzip_kv_verify's does; entries with path[b, j] <=
 * j or >= nodes, tokens outside the cache and absent pages are passed over.
 * length is not changed. A cache without scales. */
typedef struct uzip_kv_accept_args {
    const int32_t *length;
    const int32_t *path;        /* [seqs, nodes], rows contiguous */
    int64_t        path_stride;
    const int32_t *count;
    uint32_t       nodes;       /* at most 1024 */
    uint32_t       reserved;    /* 0 */
} uzip_kv_accept_args_t;
int uzip_kv_accept(const uzip_kv_cache_t *cache, const uzip_kv_accept_args_t *a, hipStream_t s);

/* The page table of the next step. A page is in use if a sequence's table has
 * it for its tokens, or if held[page] is not zero; all others are free. Entries
 * of the tables behind the tokens are not looked at. */
typedef struct uzip_kv_pages {
    const int32_t *table;       /* [rows, entries], rows contiguous */
    int64_t        table_stride;
    const int32_t *length;      /* [rows] */
    const int32_t *parent;      /* [seqs]; fork only */
    const uint8_t *held;        /* [pages], or NULL */
    int32_t       *out_table;   /* [seqs, entries], contiguous; not the table */
    int32_t       *out_length;  /* [seqs]; fork only; not length */
    int32_t       *moves;       /* fork: [seqs, 2]; compact: [min(seqs * entries, pages / 2), 2]; (from, to), -1 where there is none */
    int32_t       *left;        /* fork: pages still free, or, negative, those that were lacking; compact: pages in use */
    uint32_t       rows;
    uint32_t       seqs;        /* compact: rows */
    uint32_t       entries;
    uint32_t       pages;
    uint32_t       page;        /* tokens: a power of two, at least 16 */
    uint32_t       room;        /* fork only */
    uint64_t       reserved;    /* 0 */
} uzip_kv_pages_t;

/* async. Sequence b goes on where row parent[b] of the table is: it has its
 * tokens, and pages for `room` more as far as the table has entries. A parent
 * outside [0, rows) leaves an empty sequence; rows that are no parent are
 * freed. Whole pages are shared. Of the sequences that have the same partly
 * filled last page the first one keeps it, unless it is held or whole for
 * another; the others get a copy (moves, for uzip_kv_copy_pages). New pages are
 * the lowest free ones, in the order of sequences and entries; entries for which
 * none is left are -1 (absent), and a copy that is not made loses its tokens.
 * Absent pages stay absent. */
int uzip_kv_fork(const uzip_kv_pages_t *a, void *d_ws, uint64_t ws_bytes, hipStream_t s);

/* async. Moves pages so that those in use, n of them, are the first n of the
 * pool: the tables' pages from n on go to the free ones below n, lowest to
 * lowest. Held pages stay where they are, so with those above n some below it
 * stay free. */
int uzip_kv_compact(const uzip_kv_pages_t *a, void *d_ws, uint64_t ws_bytes, hipStream_t s);

/* Workspace of both; 0 when the shapes are invalid. */
uint64_t uzip_kv_pages_workspace_bytes(uint32_t pages, uint32_t seqs, uint32_t entries);

/* A tensor of pages: byte address of a page's part (i, j), i < n[0], j < n[1]:
 * data + page * page_stride + i * stride[0] + j * stride[1], each `run` bytes. */
typedef struct uzip_kv_pool {
    void    *data;
    int64_t  page_stride;       /* bytes, as the others */
    int64_t  stride[2];
    uint32_t n[2];
    uint32_t run;
    uint32_t reserved;          /* 0 */
} uzip_kv_pool_t;

/* async. Copies page moves[i, 0] to page moves[i, 1] in each of n <= 8 pools,
 * i < count. Entries outside [0, pages) are passed over. Pages that are copied
 * to are distinct and none of those that are copied from. */
int uzip_kv_copy_pages(const int32_t *moves, uint32_t count, const uzip_kv_pool_t *pools, uint32_t n, uint32_t pages, hipStream_t s);

#ifdef __cplusplus
}
#endif

#endif /* UZIP_KV_H */
