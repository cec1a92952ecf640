/*
 * tb_cache.h -- C ABI of the paged key/value cache in libtb: the pages that
 * the batched copy of tb.h fills, who holds them, and the attention of drafted
 * tokens over them.
 *
 * A cache is a set of pools (the keys and the values of each layer), each an
 * array of num_pages pages of page_tokens tokens, and one table that says
 * which page holds which tokens of which sequence; page p means the same
 * tokens in every pool.  All bookkeeping lives in device memory, so a serving
 * step (append, attention, fork, resize) enqueues without reading anything
 * back, and every call below may be captured into a HIP graph.
 *
 * Conventions are those of tb.h (status codes, streams, ownership, launch
 * events), and:
 *   - The library allocates nothing here: scratch and workspace are the
 *     caller's.  Calls on one cache change its bookkeeping and share its
 *     scratch, so the caller orders them (one stream, or events);
 *     tb_tree_attention and tb_page_append only read the bookkeeping (append
 *     may raise a flag).  Attention calls that can overlap in time need a
 *     workspace each.
 *   - Index lists are int32 arrays in device memory.  A negative sequence or
 *     page number is padding and skipped.  What cannot be done for a listed
 *     entry (a number out of range, say) is skipped and raises a bit of
 *     counts[1]; the rest of the list is still done.  No index makes a kernel
 *     touch memory outside the arrays described here.
 *   - Index lists, and what a call writes, overlap nothing else that the call
 *     reads or writes (a list is no part of the cache's own arrays, out is not q).
 *   - A call of several kernels carries the timing hook's start event on its
 *     first kernel and the stop event on its last.
 */
#ifndef TB_CACHE_H
#define TB_CACHE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Most pools of one cache: keys and values of 128 layers. */
#define TB_MAX_POOLS 256

/* How a page lies in memory: page_tokens x heads x head_bytes, or heads x
 * page_tokens x head_bytes, contiguous either way. */
enum { TB_CACHE_TOKEN_MAJOR = 0, TB_CACHE_HEAD_MAJOR = 1 };

/* Bits of counts[1].  They stay set until the caller clears them. */
enum {
    TB_CACHE_SHORT = 1,   /* too few free pages: no fork, or no growth, of that call was made     */
    TB_CACHE_RANGE = 2,   /* an entry's sequence, page, position or length was out of range        */
    TB_CACHE_BUSY = 4,    /* a fork's child already holds tokens, or is its own parent             */
    TB_CACHE_TWICE = 8,   /* a sequence came again in one list (the first entry counts)            */
    TB_CACHE_SHARED = 16  /* an appended token lies in a page that another sequence also refers to,
                             or a sequence was to grow in one                                      */
};

typedef struct tb_cache {
    const void *const *pools; /* HOST array of npools device addresses, read during the call only */
    uint32_t npools;          /* 0 .. TB_MAX_POOLS                                                */
    uint32_t layout;          /* TB_CACHE_TOKEN_MAJOR or TB_CACHE_HEAD_MAJOR                      */
    uint32_t num_pages;       /* pages of each pool, 1 .. 2^30                                    */
    uint32_t page_tokens;     /* tokens of a page, 1 .. 2^16                                      */
    uint32_t heads;           /* key/value heads, 1 .. 2^16                                       */
    uint32_t head_bytes;      /* bytes of one token's head, >= 1; of a token at most 2^26         */
    uint64_t page_stride;     /* bytes between pages, >= page_tokens * heads * head_bytes, which is
                                 at most 2^30                                                      */
    uint32_t max_seqs;        /* rows of the table, >= 1                                          */
    uint32_t max_pages;       /* pages of a row, >= 1; max_pages * page_tokens < 2^31             */
    int32_t *table;           /* device, [max_seqs][max_pages]: a sequence's pages in order; only the
                                 first ceil(lens / page_tokens) of a row are read, the others kept  */
    int32_t *lens;            /* device, [max_seqs]: tokens of each sequence                      */
    int32_t *refs;            /* device, [num_pages]: table entries that refer to the page, 0: free */
    int32_t *free_list;       /* device, [num_pages]: the free pages, a stack whose top is the last
                                 of its first counts[0]; what lies above is kept as it was         */
    int32_t *counts;          /* device, [4]: free pages, flags, two words unused                 */
    void *scratch;            /* device, tb_cache_scratch_bytes(), 16-byte aligned; cleared by
                                 tb_cache_init (or by the caller, to zero), then the library's      */
} tb_cache;

/*
 * Bytes of scratch for a cache of num_pages pages and max_seqs rows (host
 * only).  Errors: TB_ERR_INVALID for NULL or a size out of range.
 */
int tb_cache_scratch_bytes(uint32_t num_pages, uint32_t max_seqs, uint64_t *bytes_out);

/*
 * Empty cache: every length and reference 0, every page free with page 0 on
 * top of the stack, flags and scratch cleared.  The table and the pools are
 * not written.  One kernel.
 */
int tb_cache_init(const tb_cache *cache, void *stream);

/*
 * Copy n whole pages in every pool: dst pool p, page dst_pages[i] = src pool
 * p, page src_pages[i].  src may be the same cache or another of the same
 * npools, layout, page_tokens, heads and head_bytes; only the pools and
 * geometry of both are used (tables and the other fields may be NULL).  As
 * for tb_batched_copy, destinations must be pairwise disjoint and disjoint
 * from every source, else their bytes are unspecified (not checked: the lists
 * are in device memory).  A page number of either list outside its cache is
 * skipped; nothing raises a flag.  n == 0 or npools == 0 is a no-op.
 */
int tb_page_copy(const tb_cache *dst, const tb_cache *src, const int32_t *dst_pages, const int32_t *src_pages,
                 uint32_t n, void *stream);

/*
 * Write n tokens' keys and values: in pool p, position positions[i] of
 * sequence seqs[i] receives row index[i] of rows, a device array
 * [npools][nrows][heads * head_bytes] with row_stride bytes between rows and
 * pool_stride between pools.  index NULL: row i.  This is how a prompt's
 * tokens enter the cache, and how the accepted ones of a draft do: the caller
 * grows the sequence (tb_page_resize) and names the drafted rows.
 * Skipped with a flag: a position at or past the sequence's length or a row
 * at or past nrows (TB_CACHE_RANGE), a page with more than one reference
 * (TB_CACHE_SHARED: another sequence would see the write).  The same position
 * twice gives bytes of either row.
 */
int tb_page_append(const tb_cache *cache, const void *rows, uint64_t nrows, uint64_t row_stride,
                   uint64_t pool_stride, const int32_t *seqs, const int32_t *positions, const int32_t *index,
                   uint32_t n, void *stream);

/*
 * Fork n sequences: children[i] becomes a copy of parents[i].  The parent's
 * full pages are shared (one reference more); its last page, where it is only
 * partly used, is copied in every pool into a page of the child's own, its
 * used tokens only, so that both can grow.  New pages come off the stack in
 * list order.  A child must be an empty row (length 0), else TB_CACHE_BUSY;
 * lengths are those before the call, so a child cannot be a parent of the same
 * call to any effect.  One parent may have several children; a child listed
 * again is TB_CACHE_TWICE.  With too few free pages nothing is done
 * (TB_CACHE_SHORT).  n <= max_seqs.
 */
int tb_page_fork(const tb_cache *cache, const int32_t *parents, const int32_t *children, uint32_t n, void *stream);

/*
 * Set the lengths of n sequences: seqs[i] gets lens[i] tokens, 0 freeing it.
 * Shrinking releases the pages behind the new end; those that nothing refers
 * to any more are pushed in descending order of their number (the lowest comes
 * off first).  Then growing sequences take their new pages off the stack, in
 * list order and in order of position; with too few, no sequence that needs one
 * grows (TB_CACHE_SHORT) while the released pages stay released and the others
 * get their lengths.  Page contents are not touched.
 * A sequence whose last page is partly used and, after the call's releases,
 * referred to by another one as well (it was cut back into a page that a fork
 * shares) does not grow: the new tokens would be the other's too.  It is
 * skipped and raises TB_CACHE_SHARED; tb_page_fork to an empty row copies the
 * used tokens to a page of that row's own, which then can grow.
 * n <= max_seqs.
 */
int tb_page_resize(const tb_cache *cache, const int32_t *seqs, const int32_t *lens, uint32_t n, void *stream);

/*
 * Move the pages in use to the lowest numbers: with L pages in use, the i-th
 * free page below L receives, in every pool, the i-th page in use at or above
 * L (both ascending), tables and references follow, and the free pages become
 * L .. num_pages - 1 with L on top of the stack.  Pages at or above L keep
 * their bytes.
 */
int tb_page_compact(const tb_cache *cache, void *stream);

/* Largest pool that tb_tree_attention reads: page_stride * num_pages. */
#define TB_ATTN_MAX_POOL (1ull << 36)

/* Element types of tb_tree_attention. */
enum { TB_BF16 = 0, TB_FP16 = 1 };

/*
 * Attention of drafted tokens over the cache.  Sequence b of the batch has
 * the context in row seqs[b] of the cache's table and a tree of up to `nodes`
 * drafted tokens, whose keys and values k, v are not in the cache.  Node t of
 * b attends to the whole context and to the drafted nodes u with bit u % 64
 * of mask[b][t][u / 64] set:
 *   s_j = scale * (q . k_j),  out = sum_j exp(s_j) v_j / sum_j exp(s_j),
 *   lse = log sum_j exp(s_j)
 * for each of heads_q query heads, query head h reading key/value head
 * h / (heads_q / cache->heads).  mask NULL is a chain: node t sees nodes
 * u <= t (so nodes = 1 is ordinary decoding of one token).  tree_nodes (NULL:
 * all `nodes`) gives each tree's size; nodes past it neither see nor are seen,
 * their keys and values are not read, and their rows are written as for a
 * row that sees nothing: out 0, lse -infinity.  A sequence whose seqs entry is
 * negative or out of range has no context and no nodes.  Keys and values that
 * a row does not see have no effect on it, whatever they hold.
 * Products are of 16-bit inputs with fp32 sums, softmax statistics and sums are
 * fp32, probabilities are rounded to the element type for the second product, in
 * fp16 with steps of 2^-31 of the row's largest or finer, so that the small ones of a long context still
 * count together.
 */
typedef struct tb_tree_attn {
    const void *q;             /* device, [batch][nodes][heads_q][head_dim]                       */
    const void *k, *v;         /* device, [batch][nodes][heads][head_dim]                         */
    void *out;                 /* device, as q                                                    */
    float *lse;                /* device, [batch][nodes][heads_q] contiguous, or NULL             */
    uint64_t q_stride[3], k_stride[3], v_stride[3], out_stride[3]; /* elements between sequences, nodes, heads: */
                               /* multiples of 8; head_dim itself is contiguous.  Rows of out must
                                  lie apart: from the smallest stride up, each steps over all that
                                  the smaller ones reach                                          */
    const int32_t *seqs;       /* device, [batch]                                                 */
    const uint64_t *mask;      /* device, [batch][nodes][ceil(nodes / 64)], or NULL               */
    const int32_t *tree_nodes; /* device, [batch], or NULL                                        */
    uint32_t batch, nodes;     /* batch <= 2^16, nodes <= 2^12, batch * nodes * heads_q < 2^24     */
    uint32_t heads_q;          /* a multiple of cache->heads, at most 2^10                        */
    uint32_t head_dim;         /* 64, 96, 128 or 256; cache->head_bytes = 2 * head_dim            */
    uint32_t dtype;            /* TB_BF16 or TB_FP16, of q, k, v, out and the cache               */
    uint32_t k_pool, v_pool;   /* which pools hold this layer's keys and values                   */
    float scale;               /* finite, at most 1e30 either way                                 */
    void *workspace;           /* device, tb_tree_attention_workspace() bytes, 16-byte aligned    */
    uint64_t workspace_bytes;
} tb_tree_attn;

/*
 * Bytes of workspace a call needs; depends on batch, nodes, heads and head_dim
 * and not on the lengths (room for a share of every sequence beside those of the workgroups: 579 MB for 256
 * sequences of 64 nodes, 64 query heads of 128 over 8 key heads); 0 for no batch or no nodes.  Only those fields
 * of `attn` and heads of `cache` are read.  Errors: TB_ERR_INVALID; TB_ERR_HIP if the device cannot be queried.
 */
int tb_tree_attention_workspace(const tb_tree_attn *attn, const tb_cache *cache, uint64_t *bytes_out);

/* Errors: TB_ERR_INVALID for a bad argument (nothing enqueued), TB_ERR_HIP. */
int tb_tree_attention(const tb_tree_attn *attn, const tb_cache *cache, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TB_CACHE_H */
