// tb_cache_kernels.hip -- gfx950 kernels of the paged cache's bookkeeping and
// of the copies that go with it.
//
// Page numbers, lengths and positions come from device memory, so every one is
// checked against its array before it is used as an index: a wrong number is
// skipped (and flagged where the header says so), never followed.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tb_cache_internal.h"
#include "tb_launch.h"

namespace tbk {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(1))) u32x4 gu32x4;
typedef __attribute__((address_space(1))) uint8_t gu8;

__device__ __forceinline__ void raise(const CacheState &s, int32_t bit) { atomicOr(&s.counts[1], bit); }

__device__ __forceinline__ int32_t pages_of(int32_t tokens, uint32_t page_tokens) {
    return (int32_t)(((uint32_t)tokens + page_tokens - 1) / page_tokens);
}

// A row's length, within what the row can hold.
__device__ __forceinline__ int32_t length_of(const CacheState &s, int32_t seq) {
    const int32_t most = (int32_t)(s.max_pages * s.page_tokens), n = s.lens[seq];
    return n < 0 ? 0 : (n < most ? n : most);
}

// Values that another workgroup of this call, or an atomic, wrote: read past the L1.
__device__ __forceinline__ int32_t fresh(const int32_t *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint32_t fresh(const uint32_t *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Exclusive sum of v over the workgroup's threads in order, *total the whole
// sum; lds holds one word a wave and is free again after the next barrier.
template <int BS>
__device__ __forceinline__ uint32_t block_sum(uint32_t v, uint32_t *total, uint32_t *lds) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t x = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t y = __shfl_up(x, d);
        if (lane >= d)
            x += y;
    }
    __syncthreads();
    if (lane == 63)
        lds[wave] = x;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int k = 0; k < BS / 64; k++) {
        const uint32_t t = lds[k];
        before += k < wave ? t : 0;
        all += t;
    }
    *total = all;
    return before + x - v;
}

// ---- init --------------------------------------------------------------------

__global__ __launch_bounds__(256) void cache_init_kernel(CacheState s) {
    const uint32_t n = gridDim.x * 256, at = blockIdx.x * 256 + threadIdx.x;
    for (uint32_t i = at; i < s.num_pages; i += n) {
        s.refs[i] = 0;
        s.free_list[i] = (int32_t)(s.num_pages - 1 - i);
    }
    for (uint32_t i = at; i < (s.num_pages + 31) / 32; i += n)
        s.w.bits[i] = 0;
    for (uint32_t i = at; i < s.max_seqs; i += n)
        s.lens[i] = 0;
    if (at < 4)
        s.counts[at] = at == 0 ? (int32_t)s.num_pages : 0;
}

hipError_t launch_cache_init(const CacheState &s, hipStream_t stream) {
    const uint32_t most = s.num_pages > s.max_seqs ? s.num_pages : s.max_seqs;
    const uint32_t grid = (most + 255) / 256;
    return launch(cache_init_kernel, grid < 1024 ? grid : 1024, 256, stream, nullptr, s);
}

// ---- page copy -----------------------------------------------------------------

// One workgroup copies up to kCopyBlock bytes of one run of one page in one pool: x is
// the place in the page, y the pool, z the pair (strided).
constexpr uint32_t kCopyBlock = 256 * 16 * 4;

template <int E>
__global__ __launch_bounds__(256) void page_copy_kernel(Pools pools, PageShape g, PagePairs pairs, uint32_t blocks) {
    const uint32_t run = blockIdx.x / blocks, block = blockIdx.x % blocks;
    const uint64_t run_step = (uint64_t)g.page_tokens * g.token_bytes;
    const uint64_t src0 = pools.src[blockIdx.y], dst0 = pools.dst[blockIdx.y];
    const uint32_t n = pairs.n_dev != nullptr ? *pairs.n_dev : pairs.n;
    for (uint32_t i = blockIdx.z; i < n; i += gridDim.z) {
        const uint32_t a = (uint32_t)pairs.src[i], b = (uint32_t)pairs.dst[i];
        if (a >= g.src_pages || b >= g.dst_pages)
            continue;
        uint64_t bytes = run_step;
        if (pairs.tokens != nullptr) {
            const int32_t t = pairs.tokens[i];
            bytes = t > 0 ? (uint64_t)((uint32_t)t % g.page_tokens) * g.token_bytes : 0;
        }
        const uint64_t src = src0 + a * g.src_stride + run * run_step, dst = dst0 + b * g.dst_stride + run * run_step;
        if constexpr (E == 16) {
            u32x4 v[4];
            const uint64_t at = (uint64_t)block * kCopyBlock + threadIdx.x * 16;
#pragma unroll
            for (int u = 0; u < 4; u++)
                if (at + u * 4096 < bytes)
                    v[u] = *(const gu32x4 *)(src + at + u * 4096);
#pragma unroll
            for (int u = 0; u < 4; u++)
                if (at + u * 4096 < bytes)
                    *(gu32x4 *)(dst + at + u * 4096) = v[u];
        } else {
            for (uint64_t at = (uint64_t)block * kCopyBlock + threadIdx.x; at < bytes && at < (uint64_t)(block + 1) * kCopyBlock; at += 256)
                *(gu8 *)(dst + at) = *(const gu8 *)(src + at);
        }
    }
}

hipError_t launch_page_copy(const Pools &pools, uint32_t npools, const PageShape &g, const PagePairs &pairs,
                            bool aligned16, hipStream_t stream) {
    const uint64_t run = (uint64_t)g.page_tokens * g.token_bytes;
    const uint32_t blocks = (uint32_t)((run + kCopyBlock - 1) / kCopyBlock);
    const dim3 grid(blocks * g.runs, npools, pairs.n < 65535 ? pairs.n : 65535);
    return launch(aligned16 ? page_copy_kernel<16> : page_copy_kernel<1>, grid, 256, stream, nullptr, pools, g, pairs,
                  blocks);
}

// ---- append --------------------------------------------------------------------

// One thread moves E bytes of one token in one pool (x: token and place, y: pool).
template <int E>
__global__ __launch_bounds__(256) void append_kernel(Pools pools, CacheState s, AppendArgs a, uint32_t parts) {
    const uint64_t at = (uint64_t)blockIdx.x * 256 + threadIdx.x;
    const uint64_t i = at / parts;
    if (i >= a.n)
        return;
    const uint32_t off = (uint32_t)(at % parts) * E;
    const int32_t q = a.seqs[i];
    if (q < 0)
        return;
    const int32_t pos = a.positions[i];
    const uint64_t row = a.index != nullptr ? (uint64_t)(int64_t)a.index[i] : i;
    if ((uint32_t)q >= s.max_seqs || pos < 0 || pos >= length_of(s, q) || row >= a.nrows) {
        if (off == 0 && blockIdx.y == 0)
            raise(s, TB_CACHE_RANGE);
        return;
    }
    const uint32_t j = (uint32_t)pos / s.page_tokens, in_page = (uint32_t)pos % s.page_tokens;
    const uint32_t page = (uint32_t)s.table[(uint64_t)q * s.max_pages + j];
    if (page >= s.num_pages || s.refs[page] > 1) {
        if (off == 0 && blockIdx.y == 0)
            raise(s, page >= s.num_pages ? TB_CACHE_RANGE : TB_CACHE_SHARED);
        return;
    }
    const uint64_t src = a.rows + blockIdx.y * a.pool_stride + row * a.row_stride + off;
    const uint64_t dst = pools.dst[blockIdx.y] + page * a.page_stride + in_page * a.token_step +
                         (off / a.head_bytes) * a.head_step + off % a.head_bytes;
    if constexpr (E == 16)
        *(gu32x4 *)dst = *(const gu32x4 *)src;
    else
        *(gu8 *)dst = *(const gu8 *)src;
}

hipError_t launch_append(const Pools &pools, uint32_t npools, const CacheState &s, const AppendArgs &a,
                         bool aligned16, hipStream_t stream) {
    const uint32_t parts = a.heads * a.head_bytes / (aligned16 ? 16 : 1);
    const dim3 grid((uint32_t)(((uint64_t)a.n * parts + 255) / 256), npools, 1);
    return launch(aligned16 ? append_kernel<16> : append_kernel<1>, grid, 256, stream, nullptr, pools, s, a, parts);
}

// ---- fork ----------------------------------------------------------------------

// One workgroup plans the whole call: which entries count, who gets which new
// page.  from[i], to[i]: the tail's page and its copy's; aux[i]: the length, or
// -1 for an entry that is skipped.
__global__ __launch_bounds__(1024) void fork_plan_kernel(CacheState s, const int32_t *parents, const int32_t *children,
                                                         uint32_t n) {
    __shared__ uint32_t lds[16];
    const uint32_t t = threadIdx.x;
    for (uint32_t i = t; i < n; i += 1024)
        if ((uint32_t)children[i] < s.max_seqs)
            s.w.claim[children[i]] = 0x7fffffff;
    __syncthreads();
    for (uint32_t i = t; i < n; i += 1024)
        if ((uint32_t)children[i] < s.max_seqs && parents[i] >= 0)
            atomicMin(&s.w.claim[children[i]], (int32_t)i);
    __syncthreads();
    uint32_t need_all = 0;
    for (uint32_t i0 = 0; i0 < n; i0 += 1024) {
        const uint32_t i = i0 + t;
        uint32_t need = 0, total;
        if (i < n) {
            const int32_t p = parents[i], c = children[i];
            int32_t len = -1;
            if (p >= 0 && c >= 0) {
                if ((uint32_t)p >= s.max_seqs || (uint32_t)c >= s.max_seqs)
                    raise(s, TB_CACHE_RANGE);
                else if (fresh(&s.w.claim[c]) != (int32_t)i)
                    raise(s, TB_CACHE_TWICE);
                else if (p == c || s.lens[c] != 0)
                    raise(s, TB_CACHE_BUSY);
                else
                    len = length_of(s, p);
            }
            need = len > 0 && (uint32_t)len % s.page_tokens != 0;
            s.w.aux[i] = len;
        }
        const uint32_t before = block_sum<1024>(need, &total, lds);
        if (i < n)
            s.w.to[i] = need ? (int32_t)(need_all + before) : -1;
        need_all += total;
    }
    const int32_t top = s.counts[0];
    const bool enough = top >= 0 && (uint32_t)top <= s.num_pages && need_all <= (uint32_t)top;
    __syncthreads();
    for (uint32_t i = t; i < n; i += 1024) {   // the same thread wrote aux[i] and to[i]
        const int32_t len = s.w.aux[i], k = s.w.to[i];
        int32_t from = -1, to = -1;
        if (!enough)
            s.w.aux[i] = -1;
        else if (len >= 0) {
            if (k >= 0) {
                from = s.table[(uint64_t)parents[i] * s.max_pages + (uint32_t)len / s.page_tokens];
                to = s.free_list[top - 1 - k];
            }
            s.lens[children[i]] = len;
        }
        s.w.from[i] = from;
        s.w.to[i] = to;
    }
    if (t == 0) {
        if (enough)
            s.counts[0] = top - (int32_t)need_all;
        else
            raise(s, TB_CACHE_SHORT);
    }
}

// The children's rows and the references: x is the place in the row, y the entry (strided).
__global__ __launch_bounds__(256) void fork_rows_kernel(CacheState s, const int32_t *parents, const int32_t *children,
                                                        uint32_t n) {
    const uint32_t j = blockIdx.x * 256 + threadIdx.x;
    for (uint32_t i = blockIdx.y; i < n; i += gridDim.y) {
        const int32_t len = s.w.aux[i];
        if (len <= 0)
            continue;
        const uint32_t full = (uint32_t)len / s.page_tokens;
        const uint64_t to = (uint64_t)children[i] * s.max_pages;
        if (j < full) {
            const int32_t page = s.table[(uint64_t)parents[i] * s.max_pages + j];
            s.table[to + j] = page;
            if ((uint32_t)page < s.num_pages)
                atomicAdd(&s.refs[page], 1);
        } else if (j == full && (uint32_t)len % s.page_tokens != 0) {
            const int32_t page = s.w.to[i];
            s.table[to + j] = page;
            if ((uint32_t)page < s.num_pages)
                s.refs[page] = 1;
        }
    }
}

hipError_t launch_fork_tables(const CacheState &s, const int32_t *parents, const int32_t *children, uint32_t n,
                              hipStream_t stream) {
    hipError_t e = launch(fork_plan_kernel, 1, 1024, stream, nullptr, s, parents, children, n);
    if (e != hipSuccess)
        return e;
    return launch(fork_rows_kernel, dim3((s.max_pages + 255) / 256, n < 65535 ? n : 65535), 256, stream, nullptr, s,
                  parents, children, n);
}

// ---- resize --------------------------------------------------------------------

// Release: one workgroup an entry.  from[i]: pages the row had, -1 for an
// entry that is skipped; to[i]: pages it is to have.
__global__ __launch_bounds__(256) void release_kernel(CacheState s, const int32_t *seqs, const int32_t *lens) {
    __shared__ int again;
    const uint32_t i = blockIdx.x;
    const int32_t q = seqs[i], len = lens[i];
    if (threadIdx.x == 0)
        again = 0;
    __syncthreads();
    bool ok = q >= 0;
    if (ok && ((uint32_t)q >= s.max_seqs || len < 0 || (uint32_t)len > s.max_pages * s.page_tokens)) {
        ok = false;
        if (threadIdx.x == 0)
            raise(s, TB_CACHE_RANGE);
    }
    if (ok) {
        for (uint32_t k = threadIdx.x; k < i; k += 256)
            if (seqs[k] == q)
                again = 1;
    }
    __syncthreads();
    if (ok && again) {
        ok = false;
        if (threadIdx.x == 0)
            raise(s, TB_CACHE_TWICE);
    }
    if (!ok) {
        if (threadIdx.x == 0)
            s.w.from[i] = -1;
        return;
    }
    const int32_t had = pages_of(length_of(s, q), s.page_tokens), has = pages_of(len, s.page_tokens);
    if (threadIdx.x == 0) {
        s.w.from[i] = had;
        s.w.to[i] = has;
    }
    for (int32_t j = has + (int32_t)threadIdx.x; j < had; j += 256) {
        const uint32_t page = (uint32_t)s.table[(uint64_t)q * s.max_pages + j];
        if (page < s.num_pages && atomicSub(&s.refs[page], 1) == 1)
            atomicOr(&s.w.bits[page >> 5], 1u << (page & 31));
    }
}

// One workgroup pushes the released pages and deals the new ones.
__global__ __launch_bounds__(1024) void restack_kernel(CacheState s, const int32_t *seqs, const int32_t *lens, uint32_t n) {
    __shared__ uint32_t lds[16];
    const uint32_t t = threadIdx.x, words = (s.num_pages + 31) / 32;
    uint32_t top = (uint32_t)s.counts[0];
    if (top > s.num_pages)
        top = s.num_pages;
    // words in descending order
    for (uint32_t w0 = 0; w0 < words; w0 += 1024) {
        const uint32_t k = w0 + t;
        uint32_t word = 0, total;
        if (k < words) {
            word = s.w.bits[words - 1 - k];
            if (word != 0)
                s.w.bits[words - 1 - k] = 0;
        }
        uint32_t at = top + block_sum<1024>(__popc(word), &total, lds);
        while (word != 0) {
            const int b = 31 - __clz((int)word);
            word &= ~(1u << b);
            if (at < s.num_pages)
                s.free_list[at++] = (int32_t)((words - 1 - k) * 32 + b);
        }
        top += total;
    }
    if (top > s.num_pages)
        top = s.num_pages;
    uint32_t need_all = 0;
    for (uint32_t i0 = 0; i0 < n; i0 += 1024) {
        const uint32_t i = i0 + t;
        uint32_t need = 0, total;
        if (i < n && s.w.from[i] >= 0 && s.w.to[i] > s.w.from[i])
            need = (uint32_t)(s.w.to[i] - s.w.from[i]);
        const uint32_t before = block_sum<1024>(need, &total, lds);
        if (i < n)
            s.w.aux[i] = (int32_t)top - 1 - (int32_t)(need_all + before);
        need_all += total;
    }
    const bool enough = need_all <= top;
    for (uint32_t i = t; i < n; i += 1024) {
        if (s.w.from[i] < 0)
            continue;
        if (!enough && pages_of(lens[i], s.page_tokens) > s.w.from[i]) {
            s.w.from[i] = -1;
            continue;
        }
        s.lens[seqs[i]] = lens[i];
    }
    if (t == 0) {
        s.counts[0] = (int32_t)(enough ? top - need_all : top);
        if (!enough)
            raise(s, TB_CACHE_SHORT);
    }
}

__global__ __launch_bounds__(256) void grow_kernel(CacheState s, const int32_t *seqs) {
    const uint32_t i = blockIdx.x;
    const int32_t had = s.w.from[i];
    if (had < 0)
        return;
    const int32_t has = s.w.to[i], first = s.w.aux[i];
    for (int32_t j = had + (int32_t)threadIdx.x; j < has; j += 256) {
        const int32_t page = s.free_list[first - (j - had)];
        s.table[(uint64_t)seqs[i] * s.max_pages + j] = page;
        if ((uint32_t)page < s.num_pages)
            s.refs[page] = 1;
    }
}

hipError_t launch_resize(const CacheState &s, const int32_t *seqs, const int32_t *lens, uint32_t n,
                         hipStream_t stream) {
    LaunchSeq seq;
    hipError_t e = launch(release_kernel, n, 256, stream, nullptr, s, seqs, lens);
    if (e == hipSuccess)
        e = launch(restack_kernel, 1, 1024, stream, nullptr, s, seqs, lens, n);
    seq.last();
    if (e == hipSuccess)
        e = launch(grow_kernel, n, 256, stream, nullptr, s, seqs);
    return e;
}

// ---- compact -------------------------------------------------------------------

__device__ __forceinline__ uint32_t border_of(const CacheState &s) {
    const int32_t top = s.counts[0];
    return top < 0 ? s.num_pages : ((uint32_t)top > s.num_pages ? 0 : s.num_pages - (uint32_t)top);
}

// Free pages below the border L and used ones at or above it, by chunk of pages.
__global__ __launch_bounds__(256) void compact_count_kernel(CacheState s) {
    __shared__ uint32_t lds[4];
    const uint32_t live = border_of(s);
    uint32_t holes = 0, movers = 0, total;
    for (uint32_t k = threadIdx.x; k < kScanChunk; k += 256) {
        const uint32_t p = blockIdx.x * kScanChunk + k;
        if (p < s.num_pages) {
            const bool used = s.refs[p] > 0;
            holes += p < live && !used;
            movers += p >= live && used;
        }
    }
    (void)block_sum<256>(holes, &total, lds);
    if (threadIdx.x == 0)
        s.w.chunk[2 * blockIdx.x] = total;
    (void)block_sum<256>(movers, &total, lds);
    if (threadIdx.x == 0)
        s.w.chunk[2 * blockIdx.x + 1] = total;
}

// to[r]: the r-th hole; from[r]: the r-th mover; rank[p]: r of mover p.
__global__ __launch_bounds__(256) void compact_rank_kernel(CacheState s, uint32_t chunks) {
    __shared__ uint32_t lds[4];
    const uint32_t live = border_of(s);
    uint32_t holes = 0, movers = 0, total;
    for (uint32_t k = threadIdx.x; k < blockIdx.x; k += 256) {
        holes += s.w.chunk[2 * k];
        movers += s.w.chunk[2 * k + 1];
    }
    (void)block_sum<256>(holes, &total, lds);
    holes = total;
    (void)block_sum<256>(movers, &total, lds);
    movers = total;
    for (uint32_t k0 = 0; k0 < kScanChunk; k0 += 256) {
        const uint32_t p = blockIdx.x * kScanChunk + k0 + threadIdx.x;
        const bool in = p < s.num_pages, used = in && s.refs[p] > 0;
        const bool hole = in && p < live && !used, mover = in && p >= live && used;
        uint32_t r = holes + block_sum<256>(hole, &total, lds);
        holes += total;
        if (hole)
            s.w.to[r] = (int32_t)p;
        r = movers + block_sum<256>(mover, &total, lds);
        movers += total;
        if (mover) {
            s.w.from[r] = (int32_t)p;
            s.w.rank[p] = (int32_t)r;
        }
    }
    // pairs that exist on both sides (all of them, in a cache that is in order)
    if (blockIdx.x == chunks - 1 && threadIdx.x == 0)
        *s.w.pairs = holes < movers ? holes : movers;
}

__global__ __launch_bounds__(256) void compact_apply_kernel(CacheState s) {
    const uint32_t live = border_of(s), pairs = *s.w.pairs;
    const uint32_t n = gridDim.x * 256, at = blockIdx.x * 256 + threadIdx.x;
    const uint64_t entries = (uint64_t)s.max_seqs * s.max_pages;
    for (uint64_t k = at; k < entries; k += n) {
        const uint32_t q = (uint32_t)(k / s.max_pages), j = (uint32_t)(k % s.max_pages);
        if ((int32_t)j >= pages_of(length_of(s, (int32_t)q), s.page_tokens))
            continue;
        const uint32_t page = (uint32_t)s.table[k];
        if (page < live || page >= s.num_pages)
            continue;
        const uint32_t r = (uint32_t)s.w.rank[page];
        if (r < pairs && s.w.from[r] == (int32_t)page)
            s.table[k] = s.w.to[r];
    }
    for (uint32_t r = at; r < pairs; r += n) {
        s.refs[s.w.to[r]] = s.refs[s.w.from[r]];
        s.refs[s.w.from[r]] = 0;
    }
    for (uint32_t k = at; k < s.num_pages - live; k += n)
        s.free_list[k] = (int32_t)(s.num_pages - 1 - k);
}

hipError_t launch_compact_plan(const CacheState &s, hipStream_t stream) {
    const uint32_t chunks = (s.num_pages + kScanChunk - 1) / kScanChunk;
    hipError_t e = launch(compact_count_kernel, chunks, 256, stream, nullptr, s);
    if (e == hipSuccess)
        e = launch(compact_rank_kernel, chunks, 256, stream, nullptr, s, chunks);
    return e;
}

hipError_t launch_compact_apply(const CacheState &s, hipStream_t stream) {
    return launch(compact_apply_kernel, 1024, 256, stream, nullptr, s);
}

}  // namespace tbk
