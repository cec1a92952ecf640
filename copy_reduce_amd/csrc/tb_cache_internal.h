// tb_cache_internal.h -- declarations shared by the host half (tb_cache.cpp) and
// the kernels (tb_cache_kernels.hip, tb_attention.hip) of the paged cache.  Not
// part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tb_cache.h"

namespace tbk {

// Page numbers of one chunk of the compaction's scan: one workgroup's share.
constexpr uint32_t kScanChunk = 4096;

// The library's scratch in a cache.  `bits` is all zero between calls; the rest is
// written by a call before it is read.
struct Scratch32 {
    uint32_t *bits;    // [ceil(num_pages / 32)] pages whose last reference went
    int32_t *from;     // [max(num_pages, max_seqs)] plans of the call under way
    int32_t *to;       // [max(num_pages, max_seqs)]
    int32_t *rank;     // [num_pages] number of a moving page among those that move
    int32_t *aux;      // [max_seqs]
    int32_t *claim;    // [max_seqs]
    uint32_t *chunk;   // [2 * chunks] free pages below / used pages above the border, by chunk
    uint32_t *pairs;   // [1] pages that the compaction moves
    uint32_t *top;     // [1] free pages before a resize
};

inline uint64_t scratch_words(uint32_t num_pages, uint32_t max_seqs, uint32_t *base, Scratch32 *out) {
    const uint64_t p = num_pages, s = max_seqs, most = p > s ? p : s;
    const uint64_t sizes[8] = {(p + 31) / 32, most, most, p, s, s, 2 * ((p + kScanChunk - 1) / kScanChunk), 2};
    uint64_t at[9] = {0};
    for (int k = 0; k < 8; k++)
        at[k + 1] = (at[k] + sizes[k] + 3) / 4 * 4;   // 16-byte steps
    if (out != nullptr) {
        out->bits = base + at[0];
        out->from = reinterpret_cast<int32_t *>(base + at[1]);
        out->to = reinterpret_cast<int32_t *>(base + at[2]);
        out->rank = reinterpret_cast<int32_t *>(base + at[3]);
        out->aux = reinterpret_cast<int32_t *>(base + at[4]);
        out->claim = reinterpret_cast<int32_t *>(base + at[5]);
        out->chunk = base + at[6];
        out->pairs = base + at[7];
        out->top = base + at[7] + 1;
    }
    return at[8];
}

// The bookkeeping of a cache as the kernels see it.
struct CacheState {
    int32_t *table;
    int32_t *lens;
    int32_t *refs;
    int32_t *free_list;
    int32_t *counts;
    uint32_t num_pages;
    uint32_t page_tokens;
    uint32_t max_seqs;
    uint32_t max_pages;
    Scratch32 w;
};

// Pools of one launch (a call over more of them makes several launches).
constexpr uint32_t kPoolsPerLaunch = 128;
struct Pools {
    uint64_t src[kPoolsPerLaunch];
    uint64_t dst[kPoolsPerLaunch];
};

// Bytes of a page: `runs` contiguous stretches of run_tokens * token_bytes, one
// for a token-major page, one a head for a head-major one.
struct PageShape {
    uint64_t src_stride;   // bytes between pages
    uint64_t dst_stride;
    uint32_t src_pages;
    uint32_t dst_pages;
    uint32_t runs;
    uint32_t page_tokens;
    uint32_t token_bytes;  // of one run
};

// Which pages are copied: n pairs, or *n_dev of them.  tokens (may be null): the
// pair's used tokens are tokens[i] % page_tokens, 0 or negative meaning no copy.
struct PagePairs {
    const int32_t *src;
    const int32_t *dst;
    const int32_t *tokens;
    const uint32_t *n_dev;   // null: n
    uint32_t n;
};

struct AppendArgs {
    const int32_t *seqs;
    const int32_t *positions;
    const int32_t *index;
    uint64_t rows;
    uint64_t nrows;
    uint64_t row_stride;
    uint64_t pool_stride;
    uint64_t page_stride;
    uint32_t heads;
    uint32_t head_bytes;
    uint64_t token_step;   // bytes between a page's tokens
    uint64_t head_step;    // and between a token's heads
    uint32_t n;
};

hipError_t launch_cache_init(const CacheState &s, hipStream_t stream);
hipError_t launch_page_copy(const Pools &pools, uint32_t npools, const PageShape &shape, const PagePairs &pairs,
                            bool aligned16, hipStream_t stream);
// piece: 16, 4 or 1 bytes, what every address and a head are multiples of.
hipError_t launch_append(const Pools &pools, uint32_t npools, const CacheState &s, const AppendArgs &a,
                         uint32_t piece, hipStream_t stream);
// A fork: its plan, then its pages (pairs over the plan) and, with the launch that has `rows`, its rows.
hipError_t launch_fork_plan(const CacheState &s, const int32_t *parents, const int32_t *children, uint32_t n,
                            hipStream_t stream);
hipError_t launch_fork_copy(const Pools &pools, uint32_t npools, const PageShape &shape, const PagePairs &pairs,
                            bool aligned16, const CacheState &s, const int32_t *parents, const int32_t *children,
                            uint32_t n, bool rows, hipStream_t stream);
hipError_t launch_resize(const CacheState &s, const int32_t *seqs, const int32_t *lens, uint32_t n,
                         hipStream_t stream);
// A compaction: its plan, then its pages and, with the launch that has `apply`, its tables.
hipError_t launch_compact_plan(const CacheState &s, hipStream_t stream);
hipError_t launch_compact_copy(const Pools &pools, uint32_t npools, const PageShape &shape, const PagePairs &pairs,
                               bool aligned16, const CacheState &s, bool apply, hipStream_t stream);

// The attention's share of a stream of `units`: a `budget`-th, rounded up.  A division of 32 bits where that is enough,
// as it nearly always is.
__host__ __device__ inline uint64_t units_of_share(uint64_t units, uint32_t budget) {
    const uint64_t most = units + budget - 1;
    return most <= 0xffffffffu ? (uint32_t)most / budget : most / budget;
}

hipError_t launch_tree_attention(const tb_tree_attn &a, const tb_cache &c, int cu_count, hipStream_t stream);
uint64_t tree_attention_workspace(const tb_tree_attn &a, uint32_t heads, int cu_count);

}  // namespace tbk
