/*
 * tb_serve.h -- C ABI of what a serving step does around the paged cache of
 * tb_cache.h: verification of drafted tokens, attention over a window of the
 * context, and a cache whose keys and values are held in 4 bits.
 *
 * Conventions are those of tb_cache.h: nothing is read back, nothing is
 * allocated, every call may be captured into a HIP graph, and no index from
 * device memory makes a kernel touch memory outside the arrays described here.
 */
#ifndef TB_SERVE_H
#define TB_SERVE_H

#include <stdint.h>

#include "tb_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- verification of drafted tokens ------------------------------------- */

/* Element type of probabilities, beside TB_BF16 and TB_FP16. */
enum { TB_FP32 = 2 };

/* Most entries of the vocabulary. */
#define TB_VERIFY_MAX_VOCAB (1u << 24)
/* Most entries of all sequences' vocabularies together, batch * vocab. */
#define TB_VERIFY_MAX_ENTRIES (1ull << 38)

/*
 * For each sequence b a tree of drafted tokens, node 0 its root: the last token
 * that holds already.  Node t > 0 proposes tokens[b][t] to follow its parent's,
 * parents[b][t] < t.  p = probs[b][t] is the target's distribution of what
 * follows node t, q = draft_probs[b][t] the one that the draft drew t's children
 * from, independently of each other; draft_probs NULL: the children were
 * not drawn but chosen.
 *
 * The walk begins at the root with w = p of the root and z = 1.  The children of
 * the current node are tried in the order of their numbers.  With x the child's
 * token and u = uniform[b][child], it is accepted if
 *     u q(x) z < w(x)      (u z < w(x) without draft_probs)
 * and is the current node then, with w = its p and z = 1.  If not, what it
 * stood for is taken off:
 *     w = max(w - z q, 0), z = sum w      (w(x) = 0, z = z - w(x) without)
 * When no child is left, the next token is drawn from w: the first x with
 *     w(0) + ... + w(x) > uniform[b][0] * sum w,
 * or from the current node's p if w is zero everywhere, which rounding can do.
 * The accepted tokens and the next one are then distributed as the target's.
 * Sums and comparisons are in 64 bits.
 *
 * Probabilities are finite and not negative, random numbers in [0, 1).  Others
 * give some path and some token of the vocabulary, or -1.  A node whose parent
 * is not below it, or whose token is outside the vocabulary, is passed over.
 * Without draft_probs a token that an earlier sibling had is never accepted.
 */
typedef struct tb_verify {
    const void *probs;            /* device, [batch][nodes][vocab]                                 */
    const void *draft_probs;      /* device, likewise, or NULL                                     */
    uint64_t probs_stride[2];     /* elements between sequences and nodes (any; vocab is contiguous) */
    uint64_t draft_stride[2];
    const int32_t *tokens;        /* device, [batch][nodes]; the root's is not read                */
    const int32_t *parents;       /* device, [batch][nodes], or NULL: chains, parent t - 1         */
    const float *uniform;         /* device, [batch][nodes]                                        */
    const int32_t *tree_nodes;    /* device, [batch]: how many of the nodes are real; NULL: all    */
    uint32_t batch, nodes, vocab; /* batch <= 2^16, nodes <= 2^12, vocab <= TB_VERIFY_MAX_VOCAB,
                                     batch * vocab <= TB_VERIFY_MAX_ENTRIES                        */
    uint32_t dtype;               /* TB_BF16, TB_FP16 or TB_FP32, of both distributions            */
    int32_t *count;               /* device, [batch]: accepted nodes, the root among them          */
    int32_t *path;                /* device, [batch][nodes]: their numbers, then -1                */
    int32_t *token;               /* device, [batch]: the next token; -1 where there is none       */
    /* What a cache of tb_cache.h then needs; seqs NULL: none of it, and the others are not used.  */
    const int32_t *seqs;          /* device, [batch]: rows of the cache; out of range: no sequence */
    const int32_t *lens;          /* device, [max_seqs]: the cache's                               */
    uint32_t max_seqs;
    int32_t *new_lens;            /* device, [batch]: lens + count, for tb_page_resize             */
    int32_t *append_seqs;         /* device, [batch * nodes] each: lists for tb_page_append, whose */
    int32_t *append_positions;    /* row is b * nodes + node; entry b * nodes + i is the i-th      */
    int32_t *append_index;        /* accepted node, -1, 0, 0 past the last                         */
    void *workspace;              /* device, tb_verify_workspace() bytes, 16-byte aligned          */
    uint64_t workspace_bytes;
} tb_verify;

/*
 * A sequence with no nodes (tree_nodes 0, or seqs out of range) has count 0 and token -1;
 * new_lens is its length then, or 0.  Two kernels.
 */
int tb_verify_drafts(const tb_verify *v, void *stream);

/* Bytes of workspace of a call; reads batch, vocab of `v` only.  Its content is of no matter. */
int tb_verify_workspace(const tb_verify *v, uint64_t *bytes_out);

/* ---- a cache held in 4 bits --------------------------------------------- */

/*
 * A head of head_dim elements (a multiple of 32) is held as blocks of 32: each
 * element as a sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (codes 0 .. 7, the
 * sign is bit 3), two to a byte, the first one low; after head_dim / 2 such bytes
 * one byte for each block, the power of two, less 127, that the block is
 * multiplied by; then zeros up to a multiple of four bytes.  The cache's
 * head_bytes is TB_FP4_HEAD_BYTES(head_dim), its pools and page_stride are
 * multiples of 4 bytes; all calls of tb_cache.h but the attention work on it.
 *
 * Rounding: the block's power is the smallest e with max |x| < 7 * 2^e, so that
 * no element is off by more than half of the widest step; each element goes to
 * the nearest value, of two the one with the even code.  e is
 * at least -23 and at most 13 for fp16, -126 and 125 for bf16, so that every
 * value is a number of the type; larger magnitudes than those are held as 6 * 2^e.  A
 * block with an element that is not finite is NaN (byte 255).
 */
#define TB_FP4_BLOCK 32
#define TB_FP4_HEAD_BYTES(head_dim) ((head_dim) / 2 + ((head_dim) / TB_FP4_BLOCK + 3) / 4 * 4)

/*
 * tb_page_append of rows of `dtype` (TB_BF16 or TB_FP16), heads * head_dim elements each, row_stride and
 * pool_stride in bytes and multiples of 2, to a cache held in 4 bits: they are rounded on the way.  The same position
 * twice leaves codes and powers of either row, and so numbers that may be of neither.
 */
int tb_fp4_append(const tb_cache *cache, uint32_t dtype, uint32_t head_dim, const void *rows, uint64_t nrows,
                  uint64_t row_stride, uint64_t pool_stride, const int32_t *seqs, const int32_t *positions,
                  const int32_t *index, uint32_t n, void *stream);

/*
 * The way back: row i of out, [npools][n][heads * head_bytes] with row_stride bytes
 * between rows and pool_stride between pools, is what position positions[i] of
 * sequence seqs[i] holds in pool first_pool + p.  A negative sequence reads as zeros; so
 * does what is out of range, with TB_CACHE_RANGE.  Rows of out lie apart: row_stride holds a row, and
 * pool_stride n rows (whichever of the two is larger holds the other's reach).
 */
int tb_page_read(const tb_cache *cache, uint32_t first_pool, uint32_t npools, void *out, uint64_t row_stride,
                 uint64_t pool_stride, const int32_t *seqs, const int32_t *positions, uint32_t n, void *stream);

/* The same of a cache held in 4 bits, as elements of dtype; out and its strides are multiples of 2 bytes. */
int tb_fp4_read(const tb_cache *cache, uint32_t dtype, uint32_t head_dim, uint32_t first_pool, uint32_t npools,
                void *out, uint64_t row_stride, uint64_t pool_stride, const int32_t *seqs,
                const int32_t *positions, uint32_t n, void *stream);

/* ---- attention over a window, or over a cache held in 4 bits ------------- */

/*
 * What tb_view_attention sees of the context.  A node's position is the
 * sequence's length plus its depth; with a window it sees what lies less than
 * `window` positions before its own, and the first `sinks` tokens of the sequence,
 * in the context and among the drafted nodes alike:
 *   token j of n:          j < sinks or n + depth - j < window
 *   node u (if its mask     n + depth_u < sinks or
 *   bit is set):            depth - depth_u < window
 * so that window 1 is the node by itself.  What is not seen has no effect, whatever it
 * holds, and what no node sees is not read.
 */
typedef struct tb_attn_view {
    uint32_t window;              /* 0: the whole context                                          */
    uint32_t sinks;
    const int32_t *depths;        /* device, [batch][nodes], each taken within 0 .. the tree's nodes - 1;
                                     NULL: node t's is t, for chains (a mask with a window needs them) */
    uint32_t fp4;                 /* 1: the cache is held in 4 bits (TB_FP4_HEAD_BYTES(head_dim)); the batch
                                     rounded up to a multiple of 8, times cache->heads is < 2^24   */
} tb_attn_view;

/* Largest pool held in 4 bits that tb_view_attention reads: page_stride * num_pages. */
#define TB_ATTN_MAX_POOL_FP4 (1ull << 34)

/* Bytes of workspace, as tb_tree_attention_workspace; of `view` only fp4 is read. */
int tb_view_attention_workspace(const tb_tree_attn *attn, const tb_attn_view *view, const tb_cache *cache,
                                uint64_t *bytes_out);

/* tb_tree_attention of what `view` says.  attn->dtype is the type of q, k, v, out. */
int tb_view_attention(const tb_tree_attn *attn, const tb_attn_view *view, const tb_cache *cache, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TB_SERVE_H */
