// tb_serve.cpp -- host half of what a serving step does around the paged cache: argument checks and launches of the
// verification of drafted tokens, and of tokens written to and read from a cache held in 4 bits.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include "tb_cache_internal.h"
#include "tb_internal.h"
#include "tb_launch.h"
#include "tb_serve.h"

using namespace tbh;

namespace {

// Whether the pools hold heads of head_dim elements in 4 bits, at multiples of 4 bytes.
bool fp4_ok(const tb_cache *c, uint32_t dtype, uint32_t head_dim) {
    if (dtype > TB_FP16 || head_dim == 0 || head_dim % TB_FP4_BLOCK != 0 || head_dim > (1u << 16)
            || c->head_bytes != TB_FP4_HEAD_BYTES(head_dim) || c->page_stride % 4 != 0)
        return false;
    for (uint32_t p = 0; p < c->npools; p++)
        if (!aligned(c->pools[p], 4))
            return false;
    return true;
}

// Rows of `row` bytes, n to a pool, that do not overlap.
bool rows_apart(uint64_t row, uint64_t row_stride, uint64_t pool_stride, uint32_t n, uint32_t npools) {
    if (row_stride > (UINT64_MAX >> 34) || pool_stride > (UINT64_MAX >> 10) || (n > 1 && row_stride < row))
        return false;
    if (npools < 2)
        return true;
    const uint64_t of_pool = n > 1 ? (n - 1) * row_stride + row : row;
    if (pool_stride >= of_pool)
        return true;
    return n > 1 && pool_stride >= row && row_stride >= (npools - 1) * pool_stride + row;
}

tbk::Fp4Args fp4_args(const tb_cache *c, uint32_t head_dim, const void *rows, uint64_t nrows, uint64_t row_stride,
                      uint64_t pool_stride, const int32_t *seqs, const int32_t *positions, const int32_t *index,
                      uint32_t n) {
    tbk::Fp4Args a;
    const bool token_major = c->layout == TB_CACHE_TOKEN_MAJOR;
    a.seqs = seqs;
    a.positions = positions;
    a.index = index;
    a.rows = reinterpret_cast<uintptr_t>(rows);
    a.nrows = nrows;
    a.row_stride = row_stride;
    a.pool_stride = pool_stride;
    a.page_stride = c->page_stride;
    a.head_step = token_major ? c->head_bytes : (uint64_t)c->page_tokens * c->head_bytes;
    a.token_step = token_major ? token_bytes(c) : c->head_bytes;
    a.heads = c->heads;
    a.dim = head_dim;
    a.n = n;
    return a;
}

// Calls launch_one(pools, how many, first) for the cache's pools first .. first + npools - 1, kPoolsPerLaunch at a time.
template <typename Launch>
hipError_t for_pools(const tb_cache *c, uint32_t first, uint32_t npools, Launch launch_one) {
    tbk::LaunchSeq seq;
    for (uint32_t p0 = 0; p0 < npools; p0 += tbk::kPoolsPerLaunch) {
        const uint32_t m = npools - p0 < tbk::kPoolsPerLaunch ? npools - p0 : tbk::kPoolsPerLaunch;
        tbk::Pools pools;
        memset(&pools, 0, sizeof(pools));
        for (uint32_t p = 0; p < m; p++)
            pools.dst[p] = reinterpret_cast<uintptr_t>(c->pools[first + p0 + p]);
        if (p0 + m == npools)
            seq.last();
        const hipError_t e = launch_one(pools, m, p0);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

}  // namespace

extern "C" {

int tb_fp4_append(const tb_cache *cache, uint32_t dtype, uint32_t head_dim, const void *rows, uint64_t nrows,
                  uint64_t row_stride, uint64_t pool_stride, const int32_t *seqs, const int32_t *positions,
                  const int32_t *index, uint32_t n, void *stream) {
    if (!pools_ok(cache) || !state_ok(cache) || !fp4_ok(cache, dtype, head_dim) || n > (1u << 30))
        return TB_ERR_INVALID;
    if (n == 0 || cache->npools == 0)
        return TB_OK;
    const uint64_t bytes = 2ull * cache->heads * head_dim;
    if (rows == nullptr || !aligned(rows, 2) || nrows == 0 || nrows > (1ull << 31) || row_stride < bytes ||
        row_stride % 2 != 0 || pool_stride % 2 != 0 || !list_ok(seqs) || !list_ok(positions) ||
        (index != nullptr && !aligned(index, 4)) || (uint64_t)n * bytes > (1ull << 38)
            || row_stride > (UINT64_MAX >> 34) || pool_stride > (UINT64_MAX >> 10))
        return TB_ERR_INVALID;
    tbk::Fp4Args a = fp4_args(cache, head_dim, rows, nrows, row_stride, pool_stride, seqs, positions, index, n);
    const tbk::CacheState s = state_of(cache);
    const hipError_t e = for_pools(cache, 0, cache->npools, [&](const tbk::Pools &pools, uint32_t m, uint32_t p0) {
        a.rows = reinterpret_cast<uintptr_t>(rows) + p0 * pool_stride;
        return tbk::launch_fp4_append(pools, m, s, a, dtype, static_cast<hipStream_t>(stream));
    });
    return e == hipSuccess ? TB_OK : hip_fail(e, "4-bit append launch");
}

int tb_page_read(const tb_cache *cache, uint32_t first_pool, uint32_t npools, void *out, uint64_t row_stride,
                 uint64_t pool_stride, const int32_t *seqs, const int32_t *positions, uint32_t n, void *stream) {
    if (!pools_ok(cache) || !state_ok(cache) || n > (1u << 30) || first_pool > cache->npools ||
        npools > cache->npools - first_pool)
        return TB_ERR_INVALID;
    if (n == 0 || npools == 0)
        return TB_OK;
    const uint64_t bytes = token_bytes(cache);
    if (out == nullptr || !list_ok(seqs) || !list_ok(positions) || (uint64_t)n * bytes > (1ull << 38) ||
        !rows_apart(bytes, row_stride, pool_stride, n, npools))
        return TB_ERR_INVALID;
    tbk::AppendArgs a;
    const bool token_major = cache->layout == TB_CACHE_TOKEN_MAJOR;
    a.seqs = seqs;
    a.positions = positions;
    a.index = nullptr;
    a.nrows = n;
    a.row_stride = row_stride;
    a.pool_stride = pool_stride;
    a.page_stride = cache->page_stride;
    a.heads = token_major ? 1 : cache->heads;   // a token's stretches in the page
    a.head_bytes = (uint32_t)(token_major ? bytes : cache->head_bytes);
    a.token_step = a.head_bytes;
    a.head_step = (uint64_t)cache->page_tokens * cache->head_bytes;
    a.n = n;
    uint32_t piece = 1;
    for (uint32_t w : {4u, 16u}) {
        bool fits = a.head_bytes % w == 0 && cache->page_stride % w == 0 && aligned(out, w)
                && (n == 1 || row_stride % w == 0) && (npools == 1 || pool_stride % w == 0);
        for (uint32_t p = 0; p < npools; p++)
            fits = fits && aligned(cache->pools[first_pool + p], w);
        if (fits)
            piece = w;
    }
    const tbk::CacheState s = state_of(cache);
    const hipError_t e = for_pools(cache, first_pool, npools, [&](const tbk::Pools &pools, uint32_t m, uint32_t p0) {
        a.rows = reinterpret_cast<uintptr_t>(out) + p0 * pool_stride;
        return tbk::launch_read(pools, m, s, a, piece, static_cast<hipStream_t>(stream));
    });
    return e == hipSuccess ? TB_OK : hip_fail(e, "page read launch");
}

int tb_fp4_read(const tb_cache *cache, uint32_t dtype, uint32_t head_dim, uint32_t first_pool, uint32_t npools,
                void *out, uint64_t row_stride, uint64_t pool_stride, const int32_t *seqs, const int32_t *positions,
                uint32_t n, void *stream) {
    if (!pools_ok(cache) || !state_ok(cache) || !fp4_ok(cache, dtype, head_dim) || n > (1u << 30) ||
        first_pool > cache->npools || npools > cache->npools - first_pool)
        return TB_ERR_INVALID;
    if (n == 0 || npools == 0)
        return TB_OK;
    const uint64_t bytes = 2ull * cache->heads * head_dim;
    if (out == nullptr || !aligned(out, 2) || row_stride % 2 != 0 || pool_stride % 2 != 0 || !list_ok(seqs) ||
        !list_ok(positions) || (uint64_t)n * bytes > (1ull << 38) ||
        !rows_apart(bytes, row_stride, pool_stride, n, npools))
        return TB_ERR_INVALID;
    tbk::Fp4Args a = fp4_args(cache, head_dim, out, n, row_stride, pool_stride, seqs, positions, nullptr, n);
    const tbk::CacheState s = state_of(cache);
    const hipError_t e = for_pools(cache, first_pool, npools, [&](const tbk::Pools &pools, uint32_t m, uint32_t p0) {
        a.rows = reinterpret_cast<uintptr_t>(out) + p0 * pool_stride;
        return tbk::launch_fp4_read(pools, m, s, a, dtype, static_cast<hipStream_t>(stream));
    });
    return e == hipSuccess ? TB_OK : hip_fail(e, "4-bit read launch");
}

static bool verify_sizes_ok(const tb_verify *v) {
    return v != nullptr && v->batch <= (1u << 16) && v->vocab >= 1 && v->vocab <= TB_VERIFY_MAX_VOCAB;
}

int tb_verify_workspace(const tb_verify *v, uint64_t *bytes_out) {
    if (bytes_out == nullptr || !verify_sizes_ok(v))
        return TB_ERR_INVALID;
    *bytes_out = v->batch == 0 ? 0 : tbk::verify_workspace(v->batch, v->vocab);
    return TB_OK;
}

int tb_verify_drafts(const tb_verify *v, void *stream) {
    // more entries and the second kernel's grid would pass 2^32 threads, after the first one has run
    if (!verify_sizes_ok(v) || v->nodes < 1 || v->nodes > (1u << 12) || v->dtype > TB_FP32 ||
        (uint64_t)v->batch * v->vocab > TB_VERIFY_MAX_ENTRIES)
        return TB_ERR_INVALID;
    if (v->batch == 0)
        return TB_OK;
    const uint64_t size = v->dtype == TB_FP32 ? 4 : 2;
    for (uint64_t stride : {v->probs_stride[0], v->probs_stride[1], v->draft_stride[0], v->draft_stride[1]})
        if (stride > (1ull << 40))
            return TB_ERR_INVALID;
    if (v->probs == nullptr || !aligned(v->probs, size) || !aligned(v->draft_probs, size) || !list_ok(v->tokens) ||
        !aligned(v->parents, 4) || v->uniform == nullptr || !aligned(v->uniform, 4) || !aligned(v->tree_nodes, 4) ||
        !list_ok(v->count) || !list_ok(v->path) || !list_ok(v->token) || v->workspace == nullptr ||
        !aligned(v->workspace, 16) || v->workspace_bytes < tbk::verify_workspace(v->batch, v->vocab))
        return TB_ERR_INVALID;
    if (v->seqs != nullptr &&
        (!list_ok(v->seqs) || !list_ok(v->lens) || !list_ok(v->new_lens) || !list_ok(v->append_seqs) ||
         !list_ok(v->append_positions) || !list_ok(v->append_index) || (uint64_t)v->batch * v->nodes > (1u << 30)))
        return TB_ERR_INVALID;
    const hipError_t e = tbk::launch_verify(*v, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? TB_OK : hip_fail(e, "verification launch");
}

}  // extern "C"
