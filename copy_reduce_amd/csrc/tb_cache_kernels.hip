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
template <int BS, typename N>
__device__ __forceinline__ N block_sum(N v, N *total, N *lds) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    N x = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const N y = __shfl_up(x, d);
        if (lane >= d)
            x += y;
    }
    __syncthreads();
    if (lane == 63)
        lds[wave] = x;
    __syncthreads();
    N before = 0, all = 0;
#pragma unroll
    for (int k = 0; k < BS / 64; k++) {
        const N t = lds[k];
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

// Raw buffer resource over [base, base + bytes): accesses outside are not made (the hardware checks).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_over(uint64_t base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(base), (short)0, (int)bytes, 0x00020000);
}

// What the bookkeeping still has to do while a fork's or a compaction's pages are copied: it goes
// by the same plan and touches nothing that the copy does, so it rides along in the same launch.
enum { kAlone = 0, kWithFork = 1, kWithCompact = 2 };
struct Rider {
    CacheState s;
    const int32_t *parents, *children;
    uint32_t n;
};
__device__ void fork_rows(const Rider &r, uint32_t block, uint32_t blocks);
__device__ void compact_apply(const Rider &r, uint32_t block, uint32_t blocks);

// One workgroup copies TH * U * 16 bytes of one run of one page in one pool: x is the place
// in the page, y the pool, z the pair (strided).  The bytes are only moved, so HBM bounds it: whole pages with
// one load in flight a thread, streaming past the caches (nt; nt sc0 sc1 for the stores), 400 pages of
// 16 KiB in 64 pools in 147 us, 5.7 TB/s, against 162 us with four loads a thread, 153 us with one-wave
// workgroups and 165 us through the caches.  A fork's partly used pages (the tokens before the
// end only) go in small workgroups, of which those behind the end do nothing, and are loaded
// through the caches, several children reading one page: 192 such pages of 32 KiB in 32 pools in 24 us;
// nt loads 46 us for the whole call against 34.
// E is 16, or 1 where pages (a fork's heads) are no multiple of 16 bytes or do not begin at one: pages of 8,190 bytes
// take 470 us where those of 8,192 take 163.
template <int E, int TH, int U, int LD, int ST, int WITH>
__global__ __launch_bounds__(TH) void page_copy_kernel(Pools pools, PageShape g, PagePairs pairs, uint32_t blocks,
        Rider rider) {
    constexpr uint32_t kBlock = TH * 16 * U;
    if constexpr (WITH != kAlone) {
        if (blockIdx.x == blocks * g.runs) {
            const uint32_t block = blockIdx.z * gridDim.y + blockIdx.y, all = gridDim.y * gridDim.z;
            if constexpr (WITH == kWithFork)
                fork_rows(rider, block, all);
            else
                compact_apply(rider, block, all);
            return;
        }
    }
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
        const uint64_t begin = (uint64_t)block * kBlock;
        if (begin >= bytes)
            continue;
        const uint32_t left = (uint32_t)(bytes - begin < kBlock ? bytes - begin : kBlock);
        const uint64_t at = run * run_step + begin;
        const uint64_t src = src0 + a * g.src_stride + at, dst = dst0 + b * g.dst_stride + at;
        if constexpr (E == 16) {
            const __amdgpu_buffer_rsrc_t in = buffer_over(src, left), out = buffer_over(dst, left);
            u32x4 v[U];
#pragma unroll
            for (int u = 0; u < U; u++)
                v[u] = __builtin_amdgcn_raw_buffer_load_b128(in, threadIdx.x * 16, u * TH * 16, LD);
#pragma unroll
            for (int u = 0; u < U; u++)
                __builtin_amdgcn_raw_buffer_store_b128(v[u], out, threadIdx.x * 16, u * TH * 16, ST);
        } else {
            for (uint32_t k = threadIdx.x; k < left; k += TH)
                *(gu8 *)(dst + k) = *(const gu8 *)(src + k);
        }
    }
}

template <int E, int TH, int U, int LD, int ST, int WITH>
static hipError_t launch_copy(const Pools &pools, uint32_t npools, const PageShape &g, const PagePairs &pairs,
                              const Rider &rider, hipStream_t stream) {
    const uint64_t run = (uint64_t)g.page_tokens * g.token_bytes, block = TH * 16 * U;
    const uint32_t blocks = (uint32_t)((run + block - 1) / block);
    uint64_t z = pairs.n;
    if (pairs.n_dev != nullptr) {
        // The device knows the number: enough workgroups to fill it some times over, each for several
        // pairs (a workgroup for each that there could be took 216 us where this takes 178).
        const uint64_t each = (uint64_t)blocks * g.runs * npools, want = (8192 + each - 1) / each;
        z = z < want ? z : want;
    }
    z = z < 65535 ? z : 65535;
    const dim3 grid(blocks * g.runs + (WITH != kAlone), npools, (uint32_t)(z > 0 ? z : 1));
    return launch(page_copy_kernel<E, TH, U, LD, ST, WITH>, grid, TH, stream, nullptr, pools, g, pairs, blocks, rider);
}

// Whole pages, of `run` bytes, alone or with what rides along.  Where a page fills the 512 threads of a
// workgroup, one load each; smaller ones, whose threads would be idle, go in workgroups of one wave with two
// loads.  420 MB copied in 64 pools, us by the first and the second: pages of 16 KiB 146 and 155, 8 KiB
// 162 and 165, 4 KiB 210 and 168, 2 KiB 356 and 166; a compaction of pages of 16, 4 and 2 KiB 161 and 166, 270
// and 168, 434 and 188.  (64 threads with one load: 152 to 177 and 182 to 190; 128: 150 to 167, 172 to 197.)
template <int WITH>
static hipError_t launch_whole(const Pools &pools, uint32_t npools, const PageShape &g, const PagePairs &pairs,
                               const Rider &rider, bool aligned16, hipStream_t stream) {
    if (!aligned16)
        return launch_copy<1, 256, 4, 0, 0, WITH>(pools, npools, g, pairs, rider, stream);
    if ((uint64_t)g.page_tokens * g.token_bytes < 16 * 512)
        return launch_copy<16, 64, 2, 2, 19, WITH>(pools, npools, g, pairs, rider, stream);
    return launch_copy<16, 512, 1, 2, 19, WITH>(pools, npools, g, pairs, rider, stream);
}

hipError_t launch_page_copy(const Pools &pools, uint32_t npools, const PageShape &g, const PagePairs &pairs,
                            bool aligned16, hipStream_t stream) {
    return launch_whole<kAlone>(pools, npools, g, pairs, Rider(), aligned16, stream);
}

// ---- append --------------------------------------------------------------------

template <int E>
struct Piece;
template <>
struct Piece<16> {
    typedef u32x4 T;
};
template <>
struct Piece<4> {
    typedef uint32_t T;
};
template <>
struct Piece<1> {
    typedef uint8_t T;
};

// One thread moves E bytes of one token in kAppendPools pools (x: token and place, strided; y: pools), so
// that the way to the page (list, length, table, references: four loads, each waiting for the one before) is
// gone once for all of them and their loads are in flight together.  The bytes are only moved, so HBM
// bounds it: 4,096 tokens of 2 KiB in 64 pools in 193 us, 5.6 TB/s; with one pool a thread 273 us, with two
// 225, with eight 534; without nontemporal stores 284 with
// one.  The loads go through the caches: nontemporal ones cost 512 tokens 36 us where these take 24.
// A few tokens are a launch: 4 us.  E is what all addresses are multiples of: 2,048 tokens
// of 1,600 bytes in 16 pools take 18 us by 16 bytes and took 200 by single ones.
constexpr int kAppendPools = 4;
template <int E>
__global__ __launch_bounds__(256) void append_kernel(Pools pools, CacheState s, AppendArgs a, uint32_t parts,
        uint32_t npools) {
    typedef typename Piece<E>::T piece;
    typedef __attribute__((address_space(1))) piece gpiece;
    const uint64_t all = (uint64_t)a.n * parts;
    constexpr uint32_t U = kAppendPools;
    const uint32_t pool = blockIdx.y * U;
    for (uint64_t at = (uint64_t)blockIdx.x * 256 + threadIdx.x; at < all; at += (uint64_t)gridDim.x * 256) {
        const uint32_t i = at <= 0xffffffffu ? (uint32_t)at / parts : (uint32_t)(at / parts);
        const uint32_t off = (uint32_t)(at - (uint64_t)i * parts) * E;
        const int32_t q = a.seqs[i];
        if (q < 0)
            continue;
        const int32_t pos = a.positions[i];
        const uint64_t row = a.index != nullptr ? (uint64_t)(int64_t)a.index[i] : i;
        if ((uint32_t)q >= s.max_seqs || pos < 0 || pos >= length_of(s, q) || row >= a.nrows) {
            if (off == 0 && blockIdx.y == 0)
                raise(s, TB_CACHE_RANGE);
            continue;
        }
        const uint32_t j = (uint32_t)pos / s.page_tokens, in_page = (uint32_t)pos % s.page_tokens;
        const uint32_t page = (uint32_t)s.table[(uint64_t)q * s.max_pages + j];
        if (page >= s.num_pages || s.refs[page] > 1) {
            if (off == 0 && blockIdx.y == 0)
                raise(s, page >= s.num_pages ? TB_CACHE_RANGE : TB_CACHE_SHARED);
            continue;
        }
        const uint64_t src = a.rows + pool * a.pool_stride + row * a.row_stride + off;
        const uint64_t dst = page * a.page_stride + in_page * a.token_step + (off / a.head_bytes) * a.head_step
                + off % a.head_bytes;
        piece x[U];
#pragma unroll
        for (uint32_t u = 0; u < U; u++)
            if (pool + u < npools)
                x[u] = *(const gpiece *)(src + u * a.pool_stride);
#pragma unroll
        for (uint32_t u = 0; u < U; u++)
            if (pool + u < npools)
                __builtin_nontemporal_store(x[u], (gpiece *)(pools.dst[pool + u] + dst));
    }
}

hipError_t launch_append(const Pools &pools, uint32_t npools, const CacheState &s, const AppendArgs &a,
                         uint32_t piece, hipStream_t stream) {
    const uint32_t parts = a.heads * a.head_bytes / piece;
    const uint64_t blocks = ((uint64_t)a.n * parts + 255) / 256, most = 1u << 22;
    const dim3 grid((uint32_t)(blocks < most ? blocks : most), (npools + kAppendPools - 1) / kAppendPools, 1);
    return launch(piece == 16 ? append_kernel<16> : (piece == 4 ? append_kernel<4> : append_kernel<1>), grid, 256,
            stream, nullptr, pools, s, a, parts, npools);
}

// ---- fork ----------------------------------------------------------------------

// One workgroup plans the whole call: which entries count (the first of a child, by a minimum over
// its entries), who gets which new page (its rank among those that need one, by a sum over the list).  Chains
// of dependent loads bound it: 3 entries 4 us, 192 entries 5 us.  from[i], to[i]: the tail's page and its copy's; aux[i]: the length, or
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

// The children's rows and the references.
__device__ void fork_rows(const Rider &r, uint32_t block, uint32_t blocks) {
    const CacheState &s = r.s;
    for (uint32_t i = block; i < r.n; i += blocks) {
        const int32_t len = s.w.aux[i];
        if (len <= 0)
            continue;
        const uint32_t full = (uint32_t)len / s.page_tokens;
        const uint64_t to = (uint64_t)r.children[i] * s.max_pages, from = (uint64_t)r.parents[i] * s.max_pages;
        for (uint32_t j = threadIdx.x; j < full; j += blockDim.x) {
            const int32_t page = s.table[from + j];
            s.table[to + j] = page;
            if ((uint32_t)page < s.num_pages)
                atomicAdd(&s.refs[page], 1);
        }
        if (threadIdx.x == 0 && (uint32_t)len % s.page_tokens != 0) {
            const int32_t page = s.w.to[i];
            s.table[to + full] = page;
            if ((uint32_t)page < s.num_pages)
                s.refs[page] = 1;
        }
    }
}

hipError_t launch_fork_plan(const CacheState &s, const int32_t *parents, const int32_t *children, uint32_t n,
                            hipStream_t stream) {
    return launch(fork_plan_kernel, 1, 1024, stream, nullptr, s, parents, children, n);
}

hipError_t launch_fork_copy(const Pools &pools, uint32_t npools, const PageShape &g, const PagePairs &pairs,
                            bool aligned16, const CacheState &s, const int32_t *parents, const int32_t *children,
                            uint32_t n, bool rows, hipStream_t stream) {
    const Rider rider = {s, parents, children, rows ? n : 0};
    return aligned16 ? launch_copy<16, 64, 4, 0, 2, kWithFork>(pools, npools, g, pairs, rider, stream)
                     : launch_copy<1, 256, 4, 0, 0, kWithFork>(pools, npools, g, pairs, rider, stream);
}

// ---- resize --------------------------------------------------------------------

// The three steps of a resize.  With many table entries each is a launch of its own, spread over
// the chip; with few, one workgroup does all three.  A page's last reference is found by the atomic that takes
// it away; which pages those were is a set of bits, so that the stack's order does not depend on the order
// of the atomics.  511 rows of up to 1,000 pages, of which 171 go with 86,000 references: 12.5 us of release (3.8 to
// where a row's table is read, 5 of taking the references away, 3.7 of setting the bits; 128 to 1,024 threads a
// row, or four pages of a thread at once, change nothing), 7 of restack, 4.7 of grow.

// Release of entry i by BS threads, a workgroup or a wave, of which this is number t.  from[i]:
// pages the row had, -1 for an entry that is skipped; to[i]: pages it is to have; aux[i]: the page in which
// a growing row's present tokens end, -1 if they fill it.
// CLAIMED: an entry's row came earlier in the list if the row's claim says so, else if one of the earlier entries does.
template <int BS, bool CLAIMED>
__device__ __forceinline__ void release(const CacheState &s, const int32_t *seqs, const int32_t *lens, uint32_t i,
        uint32_t t) {
    const int32_t q = seqs[i], len = lens[i];
    const bool in_range = (uint32_t)q < s.max_seqs && len >= 0 && (uint32_t)len <= s.max_pages * s.page_tokens;
    bool again = false;
    if constexpr (CLAIMED) {
        again = in_range && s.w.claim[q] != (int32_t)i;
    } else {
        if (in_range)
            for (uint32_t k = t; k < i; k += BS)
                again |= seqs[k] == q;
        if constexpr (BS == 64)
            again = __any(again);
        else
            again = __syncthreads_or(again);
    }
    if (!in_range || again) {
        if (t == 0) {
            s.w.from[i] = -1;
            if (q >= 0)
                raise(s, in_range ? TB_CACHE_TWICE : TB_CACHE_RANGE);
        }
        return;
    }
    const int32_t before = length_of(s, q), had = pages_of(before, s.page_tokens), has = pages_of(len, s.page_tokens);
    if (t == 0) {
        s.w.from[i] = had;
        s.w.to[i] = has;
        const bool inside = len > before && (uint32_t)before % s.page_tokens != 0;
        s.w.aux[i] = inside ? s.table[(uint64_t)q * s.max_pages + had - 1] : -1;
    }
    for (int32_t j = has + (int32_t)t; j < had; j += BS) {
        const uint32_t page = (uint32_t)s.table[(uint64_t)q * s.max_pages + j];
        if (page < s.num_pages && atomicSub(&s.refs[page], 1) == 1)
            atomicOr(&s.w.bits[page >> 5], 1u << (page & 31));
    }
}

// One workgroup does a whole resize up to these limits: a wave takes an entry, 64 pages of its row at
// a time.  Against the three launches, us a call: 6 rows of 500 tokens 11.2 to 17.9, 16 rows of 8,000
// (500 pages) 14.4 to 16.4, 32 rows of 2,000 12.1 to 17.1; past the limits 32 rows of 8,000 19.9 to
// 17.1 and 64 rows of 2,000 17.5 both ways.
constexpr uint32_t kFewEntries = 32, kFewPages = 512, kFewWork = 8192;

// Words a thread of restack(): with many pages one, over as many workgroups as that makes (1.2 million
// pages, 28 us the whole resize; with two 29, with four 32), with few the one workgroup's four.
constexpr int kFewWords = 4, kManyWords = 1;

// Pushes the released pages of one chunk of 1,024 W words of their bits, the highest page
// first, on a stack that had `top` pages.  The chunks above are counted first; the one
// with the lowest pages then knows all of them, and deals the new pages.
template <int W>
__device__ __forceinline__ void restack(const CacheState &s, const int32_t *seqs, const int32_t *lens, uint32_t n,
                                        uint32_t chunk, uint32_t top, uint32_t *lds, uint64_t *wide) {
    constexpr uint32_t kStackWords = 1024 * W;
    const uint32_t t = threadIdx.x, words = (s.num_pages + 31) / 32;
    uint32_t total, above = 0;
#pragma unroll 4
    for (uint32_t k = (chunk + 1) * kStackWords + t; k < words; k += 1024)
        above += (uint32_t)__popc(fresh(&s.w.bits[k]));
    (void)block_sum<1024>(above, &total, lds);
    top += total;
    // thread t has the words W t' .. W t' + W - 1 of the chunk, t' counted from its end
    uint32_t word[W], count = 0;
    const uint32_t at0 = chunk * kStackWords + (1023 - t) * W;
#pragma unroll
    for (int k = 0; k < W; k++) {
        word[k] = at0 + k < words ? fresh(&s.w.bits[at0 + k]) : 0;
        count += (uint32_t)__popc(word[k]);
    }
    uint32_t at = top + block_sum<1024>(count, &total, lds);
#pragma unroll
    for (int k = W - 1; k >= 0; k--)
        while (word[k] != 0) {
            const int b = 31 - __clz((int)word[k]);
            word[k] &= ~(1u << b);
            if (at < s.num_pages)
                s.free_list[at] = (int32_t)((at0 + k) * 32 + b);
            at++;
        }
    if (chunk != 0)
        return;
    top = min(top + total, s.num_pages);
    uint64_t need_all = 0, asked;   // rows may ask for 2^31 pages each
    for (uint32_t i0 = 0; i0 < n; i0 += 1024) {
        const uint32_t i = i0 + t;
        uint64_t need = 0;
        if (i < n) {
            const int32_t had = s.w.from[i], has = s.w.to[i];
            const uint32_t page = (uint32_t)s.w.aux[i];   // of an entry that counts
            // The references are final by now: a row that would grow in a page of another row's, too, stays as it is.
            if (had >= 0 && page < s.num_pages && fresh(&s.refs[page]) > 1) {
                s.w.from[i] = -1;
                raise(s, TB_CACHE_SHARED);
            } else if (had >= 0 && has > had) {
                need = (uint32_t)(has - had);
            }
        }
        const uint64_t before = block_sum<1024>(need, &asked, wide);
        if (i < n)
            s.w.aux[i] = (int32_t)(top - 1 - (uint32_t)(need_all + before));   // used only if there are enough
        need_all += asked;
    }
    const bool enough = need_all <= top;
    for (uint32_t i = t; i < n; i += 1024) {
        if (s.w.from[i] < 0)
            continue;
        if (!enough && s.w.to[i] > s.w.from[i]) {
            s.w.from[i] = -1;
            continue;
        }
        s.lens[seqs[i]] = lens[i];
    }
    if (t == 0) {
        s.counts[0] = (int32_t)(enough ? top - (uint32_t)need_all : top);
        if (!enough)
            raise(s, TB_CACHE_SHORT);
    }
}

template <int BS>
__device__ __forceinline__ void grow(const CacheState &s, const int32_t *seqs, uint32_t i, uint32_t t) {
    const int32_t had = s.w.from[i];
    if (had < 0)
        return;
    const int32_t has = s.w.to[i], first = s.w.aux[i];
    for (int32_t j = had + (int32_t)t; j < has; j += BS) {
        const int32_t page = s.free_list[first - (j - had)];
        s.table[(uint64_t)seqs[i] * s.max_pages + j] = page;
        if ((uint32_t)page < s.num_pages)
            s.refs[page] = 1;
    }
}

__device__ __forceinline__ uint32_t stack_top(const CacheState &s) {
    const int32_t top = s.counts[0];
    return top < 0 ? 0 : min((uint32_t)top, s.num_pages);
}

// claim[q]: the first entry of row q, for the rows of a long list.
__global__ __launch_bounds__(256) void unclaim_kernel(CacheState s, const int32_t *seqs, uint32_t n) {
    for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256)
        if ((uint32_t)seqs[i] < s.max_seqs)
            s.w.claim[seqs[i]] = 0x7fffffff;
}

__global__ __launch_bounds__(256) void claim_kernel(CacheState s, const int32_t *seqs, uint32_t n) {
    for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256)
        if ((uint32_t)seqs[i] < s.max_seqs)
            atomicMin(&s.w.claim[seqs[i]], (int32_t)i);
}

template <bool CLAIMED>
__global__ __launch_bounds__(256) void release_kernel(CacheState s, const int32_t *seqs, const int32_t *lens,
        uint32_t n) {
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *s.w.top = stack_top(s);   // restack's last chunk writes the new one while others still start
    for (uint32_t i = blockIdx.x; i < n; i += gridDim.x)
        release<256, CLAIMED>(s, seqs, lens, i, threadIdx.x);
}

__global__ __launch_bounds__(1024) void restack_kernel(CacheState s, const int32_t *seqs, const int32_t *lens,
        uint32_t n) {
    __shared__ uint32_t lds[16];
    __shared__ uint64_t wide[16];
    restack<kManyWords>(s, seqs, lens, n, blockIdx.x, *s.w.top, lds, wide);
}

// The first `rows` workgroups.  The others clear the bits, which every chunk of restack has read by now.
__global__ __launch_bounds__(256) void grow_kernel(CacheState s, const int32_t *seqs, uint32_t n, uint32_t rows) {
    if (blockIdx.x < rows) {
        for (uint32_t i = blockIdx.x; i < n; i += rows)
            grow<256>(s, seqs, i, threadIdx.x);
        return;
    }
    const uint32_t words = (s.num_pages + 31) / 32;
    for (uint32_t k = (blockIdx.x - rows) * 256 + threadIdx.x; k < words; k += (gridDim.x - rows) * 256)
        if (s.w.bits[k] != 0)
            s.w.bits[k] = 0;
}

// A wave an entry.
__global__ __launch_bounds__(1024) void resize_few_kernel(CacheState s, const int32_t *seqs, const int32_t *lens,
        uint32_t n) {
    __shared__ uint32_t lds[16];
    __shared__ uint64_t wide[16];
    const uint32_t top = stack_top(s), lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (uint32_t i = wave; i < n; i += 16)
        release<64, false>(s, seqs, lens, i, lane);
    __syncthreads();
    restack<kFewWords>(s, seqs, lens, n, 0, top, lds, wide);
    __syncthreads();
    for (uint32_t i = wave; i < n; i += 16)
        grow<64>(s, seqs, i, lane);
    for (uint32_t k = threadIdx.x; k < (s.num_pages + 31) / 32; k += 1024)
        if (s.w.bits[k] != 0)
            s.w.bits[k] = 0;
}

// Workgroups of release and grow at most, each then for several entries: a grid holds 2^32 threads, n may be 2^30.
constexpr uint32_t kMostRows = 1u << 16;
// Up to so many entries each looks through those before it; past that, where this would grow with the square of the
// list, two launches more let every row claim its first entry.  Rows of up to 5 pages, us a call by the first and
// the second: 1,024 entries 16.7 and 22.4, 2,048 21.5 and 24.4, 4,096 33.2 and 34.1, 8,192 60 and 51, 16,384 127 and 86.
constexpr uint32_t kScanned = 4096;

hipError_t launch_resize(const CacheState &s, const int32_t *seqs, const int32_t *lens, uint32_t n,
                         hipStream_t stream) {
    const uint32_t words = (s.num_pages + 31) / 32, chunks = (words + 1024 * kManyWords - 1) / (1024 * kManyWords);
    if (words <= 1024 * kFewWords && n <= kFewEntries && s.max_pages <= kFewPages && (uint64_t)n * s.max_pages <= kFewWork)
        return launch(resize_few_kernel, 1, 1024, stream, nullptr, s, seqs, lens, n);
    const uint32_t rows = n < kMostRows ? n : kMostRows;
    LaunchSeq seq;
    hipError_t e = hipSuccess;
    if (n > kScanned) {
        const uint32_t grid = (uint32_t)(((uint64_t)n + 255) / 256 < 4096 ? (n + 255) / 256 : 4096);
        e = launch(unclaim_kernel, grid, 256, stream, nullptr, s, seqs, n);
        if (e == hipSuccess)
            e = launch(claim_kernel, grid, 256, stream, nullptr, s, seqs, n);
    }
    if (e == hipSuccess)
        e = launch(n > kScanned ? release_kernel<true> : release_kernel<false>, rows, 256, stream, nullptr, s, seqs,
                lens, n);
    if (e == hipSuccess)
        e = launch(restack_kernel, chunks, 1024, stream, nullptr, s, seqs, lens, n);
    seq.last();
    if (e == hipSuccess)
        e = launch(grow_kernel, rows + (words + 1023) / 1024, 256, stream, nullptr, s, seqs, n, rows);
    return e;
}

// ---- compact -------------------------------------------------------------------

__device__ __forceinline__ uint32_t border_of(const CacheState &s) {
    const int32_t top = s.counts[0];
    return top < 0 ? s.num_pages : ((uint32_t)top > s.num_pages ? 0 : s.num_pages - (uint32_t)top);
}

// This thread's four pages of a chunk, as bits: whether page 4 t + k is a hole (free, below the
// border) and whether it moves (used, at or above it).
__device__ __forceinline__ void look_at(const CacheState &s, uint32_t chunk, uint32_t live, uint32_t *holes,
        uint32_t *movers) {
    typedef int32_t i32x4a __attribute__((ext_vector_type(4), aligned(4)));
    const uint32_t p = chunk * kScanChunk + threadIdx.x * 4;
    int32_t r[4] = {0, 0, 0, 0};
    if (p + 4 <= s.num_pages) {
        const i32x4a x = *reinterpret_cast<const i32x4a *>(s.refs + p);
        r[0] = x.x, r[1] = x.y, r[2] = x.z, r[3] = x.w;
    } else {
        for (uint32_t k = 0; k < 4 && p + k < s.num_pages; k++)
            r[k] = s.refs[p + k];
    }
    *holes = *movers = 0;
#pragma unroll
    for (uint32_t k = 0; k < 4; k++) {
        *holes |= (uint32_t)(r[k] <= 0 && p + k < live) << k;
        *movers |= (uint32_t)(r[k] > 0 && p + k >= live) << k;
    }
}

// The two sums that rank holes and movers, by chunks: 16 KiB of references a workgroup, read by this kernel
// and again, from the L2, by the next.  131,072 pages 5 us each.
__global__ __launch_bounds__(1024) void compact_count_kernel(CacheState s) {
    __shared__ uint32_t lds[16];
    uint32_t holes, movers, total;
    look_at(s, blockIdx.x, border_of(s), &holes, &movers);
    // both counts are at most kScanChunk, 4096: one sum
    (void)block_sum<1024>((uint32_t)(__popc(holes) | __popc(movers) << 16), &total, lds);
    if (threadIdx.x == 0) {
        s.w.chunk[2 * blockIdx.x] = total & 0xffff;
        s.w.chunk[2 * blockIdx.x + 1] = total >> 16;
    }
}

// to[r]: the r-th hole; from[r]: the r-th mover; rank[p]: r of mover p.  One workgroup a
// chunk, after compact_count_kernel; or one for all of a few chunks, by itself.
__global__ __launch_bounds__(1024) void compact_rank_kernel(CacheState s, uint32_t chunks) {
    __shared__ uint32_t lds[16];
    const uint32_t live = border_of(s), mine = gridDim.x == 1 ? chunks : 1;
    uint32_t holes = 0, movers = 0, total;
    if (gridDim.x > 1) {
        for (uint32_t k = threadIdx.x; k < blockIdx.x; k += 1024) {
            holes += s.w.chunk[2 * k];
            movers += s.w.chunk[2 * k + 1];
        }
        (void)block_sum<1024>(holes, &total, lds);
        holes = total;
        (void)block_sum<1024>(movers, &total, lds);
        movers = total;
    }
    for (uint32_t c = blockIdx.x; c < blockIdx.x + mine; c++) {
        uint32_t h, m;
        look_at(s, c, live, &h, &m);
        const uint32_t before = block_sum<1024>((uint32_t)(__popc(h) | __popc(m) << 16), &total, lds);
        uint32_t at = holes + (before & 0xffff), page = c * kScanChunk + threadIdx.x * 4;
        for (uint32_t k = 0; k < 4; k++)
            if (h >> k & 1)
                s.w.to[at++] = (int32_t)(page + k);
        at = movers + (before >> 16);
        for (uint32_t k = 0; k < 4; k++)
            if (m >> k & 1) {
                s.w.rank[page + k] = (int32_t)at;
                s.w.from[at++] = (int32_t)(page + k);
            }
        holes += total & 0xffff;
        movers += total >> 16;
    }
    // pairs that exist on both sides (all of them, in a cache that is in order)
    if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0)
        *s.w.pairs = holes < movers ? holes : movers;
}

// Tables, references and the stack after the moves.
__device__ void compact_apply(const Rider &rider, uint32_t block, uint32_t blocks) {
    const CacheState &s = rider.s;
    if (rider.n == 0)
        return;
    const uint32_t live = border_of(s), pairs = *s.w.pairs;
    const uint32_t n = blocks * blockDim.x, at = block * blockDim.x + threadIdx.x;
    for (uint32_t q = block; q < s.max_seqs; q += blocks) {
        const uint32_t pages = (uint32_t)pages_of(length_of(s, (int32_t)q), s.page_tokens);
        int32_t *row = s.table + (uint64_t)q * s.max_pages;
        for (uint32_t j = threadIdx.x; j < pages; j += blockDim.x) {
            const uint32_t page = (uint32_t)row[j];
            if (page < live || page >= s.num_pages)
                continue;
            const uint32_t r = (uint32_t)s.w.rank[page];
            if (r < pairs && s.w.from[r] == (int32_t)page)
                row[j] = s.w.to[r];
        }
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
    if (chunks <= 4)   // a chunk takes a workgroup some 1.5 us, a launch more than 3
        return launch(compact_rank_kernel, 1, 1024, stream, nullptr, s, chunks);
    hipError_t e = launch(compact_count_kernel, chunks, 1024, stream, nullptr, s);
    if (e == hipSuccess)
        e = launch(compact_rank_kernel, chunks, 1024, stream, nullptr, s, chunks);
    return e;
}

hipError_t launch_compact_copy(const Pools &pools, uint32_t npools, const PageShape &g, const PagePairs &pairs,
                               bool aligned16, const CacheState &s, bool apply, hipStream_t stream) {
    const Rider rider = {s, nullptr, nullptr, apply ? 1u : 0u};
    return launch_whole<kWithCompact>(pools, npools, g, pairs, rider, aligned16, stream);
}

}  // namespace tbk
