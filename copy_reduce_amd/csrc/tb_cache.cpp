// tb_cache.cpp -- host half of the paged cache: argument checks and launches.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "tb_cache.h"
#include "tb_cache_internal.h"
#include "tb_internal.h"
#include "tb_launch.h"
#include "tb_serve.h"

using tbh::hip_fail;

// Checks that tb_serve.cpp makes as well.
namespace tbh {

constexpr uint32_t kMaxPages = 1u << 30;

bool aligned(const void *p, uint64_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

uint64_t token_bytes(const tb_cache *c) { return (uint64_t)c->heads * c->head_bytes; }
uint64_t page_bytes(const tb_cache *c) { return c->page_tokens * token_bytes(c); }

// The pools and the shape of a page.
bool pools_ok(const tb_cache *c) {
    if (c == nullptr || c->npools > TB_MAX_POOLS || c->layout > TB_CACHE_HEAD_MAJOR || c->num_pages == 0 ||
        c->num_pages > kMaxPages || c->page_tokens == 0 || c->page_tokens > (1u << 16) || c->heads == 0 ||
        c->heads > (1u << 16) || c->head_bytes == 0 || token_bytes(c) > (1u << 26) || page_bytes(c) > (1u << 30) ||
        c->page_stride < page_bytes(c) || c->page_stride > UINT64_MAX / c->num_pages)
        return false;
    if (c->npools > 0 && c->pools == nullptr)
        return false;
    const uint64_t span = c->page_stride * c->num_pages;
    for (uint32_t p = 0; p < c->npools; p++)
        if (c->pools[p] == nullptr || reinterpret_cast<uintptr_t>(c->pools[p]) > UINTPTR_MAX - span)
            return false;
    return true;
}

static bool sizes_ok(uint32_t num_pages, uint32_t max_seqs) {
    return num_pages >= 1 && num_pages <= kMaxPages && max_seqs >= 1 && max_seqs <= (1u << 30);
}

// The bookkeeping.
bool state_ok(const tb_cache *c) {
    return c != nullptr && sizes_ok(c->num_pages, c->max_seqs) && c->page_tokens >= 1 &&
           c->page_tokens <= (1u << 16) && c->max_pages >= 1 &&
           (uint64_t)c->max_pages * c->page_tokens < (1ull << 31) && c->table != nullptr && c->lens != nullptr &&
           c->refs != nullptr && c->free_list != nullptr && c->counts != nullptr && c->scratch != nullptr &&
           aligned(c->table, 4) && aligned(c->lens, 4) && aligned(c->refs, 4) && aligned(c->free_list, 4) &&
           aligned(c->counts, 4) && aligned(c->scratch, 16);
}

bool list_ok(const int32_t *p) { return p != nullptr && aligned(p, 4); }

tbk::CacheState state_of(const tb_cache *c) {
    tbk::CacheState s;
    s.table = c->table;
    s.lens = c->lens;
    s.refs = c->refs;
    s.free_list = c->free_list;
    s.counts = c->counts;
    s.num_pages = c->num_pages;
    s.page_tokens = c->page_tokens;
    s.max_seqs = c->max_seqs;
    s.max_pages = c->max_pages;
    (void)tbk::scratch_words(c->num_pages, c->max_seqs, static_cast<uint32_t *>(c->scratch), &s.w);
    return s;
}

}  // namespace tbh

namespace {

using namespace tbh;

// Whether every page begins at a multiple of `bytes`.
bool pages_aligned(const tb_cache *c, uint64_t bytes) {
    if (c->page_stride % bytes != 0)
        return false;
    for (uint32_t p = 0; p < c->npools; p++)
        if (!aligned(c->pools[p], bytes))
            return false;
    return true;
}

// Calls launch_one(pools, npools, shape, piece, last) for the pools of both caches, kPoolsPerLaunch at a time (once,
// with none, for caches without pools).  `parts`: the used tokens of a head-major page are a stretch a head.
template <typename Launch>
hipError_t for_pools(const tb_cache *dst, const tb_cache *src, bool parts, Launch launch_one) {
    const bool whole = !parts;
    tbk::PageShape g;
    g.src_stride = src->page_stride;
    g.dst_stride = dst->page_stride;
    g.src_pages = src->num_pages;
    g.dst_pages = dst->num_pages;
    g.page_tokens = dst->page_tokens;
    parts = parts && dst->layout == TB_CACHE_HEAD_MAJOR;
    g.runs = parts ? dst->heads : 1;
    g.token_bytes = (uint32_t)(parts ? dst->head_bytes : token_bytes(dst));
    uint32_t piece = 1;
    for (uint32_t w : {4u, 16u})
        if ((whole ? page_bytes(dst) : g.token_bytes) % w == 0 && pages_aligned(dst, w) && pages_aligned(src, w))
            piece = w;
    if (dst->npools == 0) {   // what rides along with the copy has to run all the same; no page is in range
        g.src_pages = g.dst_pages = 0;
        const tbk::Pools none = {};
        return launch_one(none, 1, g, 16u, true);
    }
    uint32_t p0 = 0;
    do {
        const uint32_t n = dst->npools - p0 < tbk::kPoolsPerLaunch ? dst->npools - p0 : tbk::kPoolsPerLaunch;
        tbk::Pools pools;
        for (uint32_t p = 0; p < n; p++) {
            pools.src[p] = reinterpret_cast<uintptr_t>(src->pools[p0 + p]);
            pools.dst[p] = reinterpret_cast<uintptr_t>(dst->pools[p0 + p]);
        }
        p0 += n;
        const hipError_t e = launch_one(pools, n, g, piece, p0 == dst->npools);
        if (e != hipSuccess)
            return e;
    } while (p0 < dst->npools);
    return hipSuccess;
}

}  // namespace

extern "C" {

int tb_cache_scratch_bytes(uint32_t num_pages, uint32_t max_seqs, uint64_t *bytes_out) {
    if (bytes_out == nullptr || !sizes_ok(num_pages, max_seqs))
        return TB_ERR_INVALID;
    *bytes_out = 4 * tbk::scratch_words(num_pages, max_seqs, nullptr, nullptr);
    return TB_OK;
}

int tb_cache_init(const tb_cache *cache, void *stream) {
    if (!state_ok(cache))
        return TB_ERR_INVALID;
    const hipError_t e = tbk::launch_cache_init(state_of(cache), static_cast<hipStream_t>(stream));
    return e == hipSuccess ? TB_OK : hip_fail(e, "cache init launch");
}

int tb_page_copy(const tb_cache *dst, const tb_cache *src, const int32_t *dst_pages, const int32_t *src_pages,
                 uint32_t n, void *stream) {
    if (!pools_ok(dst) || !pools_ok(src) || dst->npools != src->npools || dst->layout != src->layout ||
        dst->page_tokens != src->page_tokens || dst->heads != src->heads || dst->head_bytes != src->head_bytes ||
        n > (1u << 30))
        return TB_ERR_INVALID;
    if (n == 0 || dst->npools == 0)
        return TB_OK;
    if (!list_ok(dst_pages) || !list_ok(src_pages))
        return TB_ERR_INVALID;
    tbk::PagePairs pairs = {src_pages, dst_pages, nullptr, nullptr, n};
    tbk::LaunchSeq seq;
    const hipError_t e = for_pools(dst, src, false, [&](const tbk::Pools &pools, uint32_t np, const tbk::PageShape &g,
            uint32_t piece, bool last) {
        if (last)
            seq.last();
        return tbk::launch_page_copy(pools, np, g, pairs, piece, static_cast<hipStream_t>(stream));
    });
    return e == hipSuccess ? TB_OK : hip_fail(e, "page copy launch");
}

int tb_page_append(const tb_cache *cache, const void *rows, uint64_t nrows, uint64_t row_stride,
                   uint64_t pool_stride, const int32_t *seqs, const int32_t *positions, const int32_t *index,
                   uint32_t n, void *stream) {
    if (!pools_ok(cache) || !state_ok(cache) || n > (1u << 30))
        return TB_ERR_INVALID;
    if (n == 0 || cache->npools == 0)
        return TB_OK;
    const uint64_t bytes = token_bytes(cache);
    if (rows == nullptr || nrows == 0 || nrows > (1ull << 31) || row_stride < bytes || !list_ok(seqs) ||
        !list_ok(positions) || (index != nullptr && !aligned(index, 4)) ||
        (uint64_t)n * bytes > (1ull << 38) || row_stride > (UINT64_MAX >> 34) || pool_stride > (UINT64_MAX >> 10))
        return TB_ERR_INVALID;
    tbk::AppendArgs a;
    const bool token_major = cache->layout == TB_CACHE_TOKEN_MAJOR;
    a.seqs = seqs;
    a.positions = positions;
    a.index = index;
    a.nrows = nrows;
    a.row_stride = row_stride;
    a.pool_stride = pool_stride;
    a.page_stride = cache->page_stride;
    a.heads = token_major ? 1 : cache->heads;   // a token's stretches in the page
    a.head_bytes = (uint32_t)(token_major ? bytes : cache->head_bytes);
    a.token_step = a.head_bytes;
    a.head_step = (uint64_t)cache->page_tokens * cache->head_bytes;
    a.n = n;
    uint32_t piece = 1;
    for (uint32_t w : {4u, 16u})
        if (a.head_bytes % w == 0 && pages_aligned(cache, w) && aligned(rows, w) && row_stride % w == 0
                && pool_stride % w == 0)
            piece = w;
    const tbk::CacheState s = state_of(cache);
    tbk::LaunchSeq seq;
    for (uint32_t p0 = 0; p0 < cache->npools; p0 += tbk::kPoolsPerLaunch) {
        const uint32_t m = cache->npools - p0 < tbk::kPoolsPerLaunch ? cache->npools - p0 : tbk::kPoolsPerLaunch;
        tbk::Pools pools;
        memset(&pools, 0, sizeof(pools));
        for (uint32_t p = 0; p < m; p++)
            pools.dst[p] = reinterpret_cast<uintptr_t>(cache->pools[p0 + p]);
        a.rows = reinterpret_cast<uintptr_t>(rows) + p0 * pool_stride;
        if (p0 + m == cache->npools)
            seq.last();
        const hipError_t e =
            tbk::launch_append(pools, m, s, a, piece, static_cast<hipStream_t>(stream));
        if (e != hipSuccess)
            return hip_fail(e, "page append launch");
    }
    return TB_OK;
}

int tb_page_fork(const tb_cache *cache, const int32_t *parents, const int32_t *children, uint32_t n, void *stream) {
    if (!pools_ok(cache) || !state_ok(cache) || n > cache->max_seqs)
        return TB_ERR_INVALID;
    if (n == 0)
        return TB_OK;
    if (!list_ok(parents) || !list_ok(children))
        return TB_ERR_INVALID;
    const tbk::CacheState s = state_of(cache);
    hipStream_t st = static_cast<hipStream_t>(stream);
    tbk::LaunchSeq seq;
    hipError_t e = tbk::launch_fork_plan(s, parents, children, n, st);
    const tbk::PagePairs pairs = {s.w.from, s.w.to, s.w.aux, nullptr, n};
    if (e == hipSuccess)
        e = for_pools(cache, cache, true, [&](const tbk::Pools &pools, uint32_t np, const tbk::PageShape &g,
                uint32_t piece, bool last) {
            if (last)
                seq.last();
            return tbk::launch_fork_copy(pools, np, g, pairs, piece, s, parents, children, n, last, st);
        });
    return e == hipSuccess ? TB_OK : hip_fail(e, "page fork launch");
}

int tb_page_resize(const tb_cache *cache, const int32_t *seqs, const int32_t *lens, uint32_t n, void *stream) {
    if (!state_ok(cache) || n > cache->max_seqs)
        return TB_ERR_INVALID;
    if (n == 0)
        return TB_OK;
    if (!list_ok(seqs) || !list_ok(lens))
        return TB_ERR_INVALID;
    const hipError_t e = tbk::launch_resize(state_of(cache), seqs, lens, n, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? TB_OK : hip_fail(e, "page resize launch");
}

int tb_page_compact(const tb_cache *cache, void *stream) {
    if (!pools_ok(cache) || !state_ok(cache))
        return TB_ERR_INVALID;
    const tbk::CacheState s = state_of(cache);
    hipStream_t st = static_cast<hipStream_t>(stream);
    tbk::LaunchSeq seq;
    hipError_t e = tbk::launch_compact_plan(s, st);
    const tbk::PagePairs pairs = {s.w.from, s.w.to, nullptr, s.w.pairs, cache->num_pages / 2};
    if (e == hipSuccess)
        e = for_pools(cache, cache, false, [&](const tbk::Pools &pools, uint32_t np, const tbk::PageShape &g,
                uint32_t piece, bool last) {
            if (last)
                seq.last();
            return tbk::launch_compact_copy(pools, np, g, pairs, piece, s, last, st);
        });
    return e == hipSuccess ? TB_OK : hip_fail(e, "page compact launch");
}

// Whether rows of `row` elements, laid out in three dimensions, share none: taken from the smallest stride up, each
// one has to step over all that the smaller ones reach.
static bool rows_apart(const uint64_t (&stride)[3], const uint32_t (&extent)[3], uint32_t row) {
    uint64_t reach = row;   // strides are at most 2^40, extents 2^16
    uint32_t below = 0;     // dimensions taken
    for (int k = 0; k < 3; k++) {
        int next = -1;
        for (int j = 0; j < 3; j++)
            if (extent[j] > 1 && (below >> j & 1) == 0 && (next < 0 || stride[j] < stride[next]))
                next = j;
        if (next < 0)
            break;
        if (stride[next] < reach)
            return false;
        reach += stride[next] * (extent[next] - 1);
        below |= 1u << next;
    }
    return true;
}

static bool attn_sizes_ok(const tb_tree_attn *a, const tb_cache *c) {
    return a != nullptr && c != nullptr && a->batch <= (1u << 16) && a->nodes <= (1u << 12) && c->heads > 0 &&
           a->heads_q > 0 && a->heads_q <= (1u << 10) && a->heads_q % c->heads == 0 &&
           (uint64_t)a->batch * a->nodes * a->heads_q < (1u << 24) &&   // a workgroup of 256 threads a row at most
           (a->head_dim == 64 || a->head_dim == 96 || a->head_dim == 128 || a->head_dim == 256);
}

static int attention_workspace(const tb_tree_attn *a, const tb_cache *c, uint64_t *bytes_out) {
    if (bytes_out == nullptr || !attn_sizes_ok(a, c))
        return TB_ERR_INVALID;
    *bytes_out = 0;
    if (a->batch == 0 || a->nodes == 0)
        return TB_OK;
    int cus = 0;
    const int rc = tbh::cu_count_of_device(&cus);
    if (rc == TB_OK)
        *bytes_out = tbk::tree_attention_workspace(*a, c->heads, cus);
    return rc;
}

static int attention(const tb_tree_attn *a, const tb_attn_view &view, const tb_cache *c, void *stream) {
    const bool fp4 = view.fp4 != 0;
    if (!attn_sizes_ok(a, c) || !pools_ok(c) || !state_ok(c) || a->dtype > TB_FP16 ||
        !(fabsf(a->scale) <= 1e30f) || c->head_bytes != (fp4 ? TB_FP4_HEAD_BYTES(a->head_dim) : 2 * a->head_dim)
                || a->k_pool >= c->npools || a->v_pool >= c->npools)
        return TB_ERR_INVALID;
    if (a->batch == 0 || a->nodes == 0)
        return TB_OK;
    // few rows deal sequences to the 8 XCDs, a workgroup of 256 threads a head and sequence
    if (fp4 && ((uint64_t)a->batch + 7) / 8 * 8 * c->heads >= (1u << 24))
        return TB_ERR_INVALID;
    const uint64_t piece = fp4 ? 4 : 16;
    if (!aligned(c->pools[a->k_pool], piece) || !aligned(c->pools[a->v_pool], piece) || c->page_stride % piece != 0 ||
        c->page_stride * c->num_pages > (fp4 ? TB_ATTN_MAX_POOL_FP4 : TB_ATTN_MAX_POOL) || a->q == nullptr
                || a->k == nullptr || a->v == nullptr || a->out == nullptr || !aligned(a->q, 16) ||
        !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->out, 16) || !aligned(a->lse, 4) ||
        !list_ok(a->seqs) || !aligned(a->mask, 8) || !aligned(a->tree_nodes, 4) || !aligned(view.depths, 4)
                || (view.window != 0 && a->mask != nullptr && view.depths == nullptr))
        return TB_ERR_INVALID;
    // strides over an extent of one are never used
    tb_tree_attn args = *a;
    const uint32_t extent_q[3] = {a->batch, a->nodes, a->heads_q}, extent_kv[3] = {a->batch, a->nodes, c->heads};
    for (int k = 0; k < 3; k++) {
        if (extent_q[k] == 1)
            args.q_stride[k] = args.out_stride[k] = 0;
        if (extent_kv[k] == 1)
            args.k_stride[k] = args.v_stride[k] = 0;
        for (uint64_t stride : {args.q_stride[k], args.k_stride[k], args.v_stride[k], args.out_stride[k]})
            if (stride % 8 != 0 || stride > (1ull << 40))
                return TB_ERR_INVALID;
    }
    if (!rows_apart(args.out_stride, extent_q, a->head_dim) || a->workspace == nullptr || !aligned(a->workspace, 16))
        return TB_ERR_INVALID;
    int cus = 0;
    const int rc = tbh::cu_count_of_device(&cus);
    if (rc != TB_OK)
        return rc;
    if (a->workspace_bytes < tbk::tree_attention_workspace(args, c->heads, cus))
        return TB_ERR_INVALID;
    const hipError_t e = tbk::launch_tree_attention(args, view, *c, cus, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? TB_OK : hip_fail(e, "tree attention launch");
}

int tb_tree_attention_workspace(const tb_tree_attn *a, const tb_cache *c, uint64_t *bytes_out) {
    return attention_workspace(a, c, bytes_out);
}

int tb_tree_attention(const tb_tree_attn *a, const tb_cache *c, void *stream) {
    return attention(a, tb_attn_view{0, 0, nullptr, 0}, c, stream);
}

int tb_view_attention_workspace(const tb_tree_attn *a, const tb_attn_view *view, const tb_cache *c,
                                uint64_t *bytes_out) {
    if (view == nullptr || view->fp4 > 1)
        return TB_ERR_INVALID;
    return attention_workspace(a, c, bytes_out);
}

int tb_view_attention(const tb_tree_attn *a, const tb_attn_view *view, const tb_cache *c, void *stream) {
    if (view == nullptr || view->fp4 > 1)
        return TB_ERR_INVALID;
    return attention(a, *view, c, stream);
}

}  // extern "C"
