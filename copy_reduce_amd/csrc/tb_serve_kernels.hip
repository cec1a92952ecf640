// tb_serve_kernels.hip -- gfx950 kernels of the verification of drafted tokens, and of tokens on
// their way into a cache held in 4 bits and out of a cache.
//
// As in tb_cache_kernels.hip every number from device memory is checked against its array before it is used as an
// index.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tb_cache_internal.h"
#include "tb_fp4.h"
#include "tb_launch.h"

namespace tbk {

// ---- tokens in 4 bits ------------------------------------------------------------

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef __attribute__((address_space(1))) u32x4_at2 gu32x4_at2;
typedef __attribute__((address_space(1))) uint32_t gu32;
typedef __attribute__((address_space(1))) uint8_t gu8;

// The place of a listed token in its pool's bytes, or a flag to raise; -1 for padding.
struct TokenPlace {
    int32_t flag;   // 0: there
    uint64_t at;
};
__device__ __forceinline__ TokenPlace place_of_token(const CacheState &s, int32_t q, int32_t pos, uint64_t page_stride,
        uint64_t token_step, bool to_write) {
    if ((uint32_t)q >= s.max_seqs)
        return {q < 0 ? -1 : (int32_t)TB_CACHE_RANGE, 0};
    const int32_t most = (int32_t)(s.max_pages * s.page_tokens), n = s.lens[q];
    if (pos < 0 || pos >= min(n, most))
        return {TB_CACHE_RANGE, 0};
    const uint32_t j = (uint32_t)pos / s.page_tokens, in_page = (uint32_t)pos % s.page_tokens;
    const uint32_t page = (uint32_t)s.table[(uint64_t)q * s.max_pages + j];
    if (page >= s.num_pages)
        return {TB_CACHE_RANGE, 0};
    if (to_write && s.refs[page] > 1)
        return {TB_CACHE_SHARED, 0};
    return {0, page * page_stride + in_page * token_step};
}

template <typename T>
struct Type16;
template <>
struct Type16<__bf16> {
    typedef __bf16 V2 __attribute__((ext_vector_type(2)));
    static constexpr uint32_t kInf = 0x7f80;
    static constexpr int kLow = -126 + 127, kHigh = 125 + 127;   // of the powers' bytes
    static __device__ __forceinline__ uint32_t bits32(uint32_t x) { return x << 16; }
    template <int I>
    static __device__ __forceinline__ uint32_t round(uint32_t to, uint32_t x, float power) {
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(to, __builtin_bit_cast(V2, x), power, I);
    }
};
template <>
struct Type16<_Float16> {
    typedef _Float16 V2 __attribute__((ext_vector_type(2)));
    static constexpr uint32_t kInf = 0x7c00;
    static constexpr int kLow = -23 + 127, kHigh = 13 + 127;
    static __device__ __forceinline__ uint32_t bits32(uint32_t x) {
        return __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)x));
    }
    template <int I>
    static __device__ __forceinline__ uint32_t round(uint32_t to, uint32_t x, float power) {
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(to, __builtin_bit_cast(V2, x), power, I);
    }
};

// The byte of a block's power, of its largest magnitude's 16 bits: with 2^E <= x < 2^(E + 1) it is E - 2 below
// 1.75 * 2^E and E - 1 from there on, where a quarter more in the significand carries.
template <typename T>
__device__ __forceinline__ uint32_t power_byte(uint32_t top) {
    if (top >= Type16<T>::kInf)
        return 255;
    const int e = (int)((Type16<T>::bits32(top) + 0x200000) >> 23) - 2;
    return (uint32_t)min(max(e, Type16<T>::kLow), Type16<T>::kHigh);
}

// A thread has 8 elements of one token in kFp4Pools pools, four threads a block of 32.  The conversion to 4 bits is the
// hardware's: to the nearest, of two the even code, larger ones to 6.
constexpr int kFp4Pools = 4;
template <typename T>
__global__ __launch_bounds__(256) void fp4_append_kernel(Pools pools, CacheState s, Fp4Args a, uint32_t parts,
        uint32_t npools) {
    constexpr uint32_t U = kFp4Pools;
    const uint64_t all = (uint64_t)a.n * parts;
    const uint32_t pool = blockIdx.y * U, of_head = a.dim / 8;
    const bool whole = 64 % of_head == 0;   // no head lies in two waves
    for (uint64_t at = (uint64_t)blockIdx.x * 256 + threadIdx.x; at < all; at += (uint64_t)gridDim.x * 256) {
        const uint32_t i = at <= 0xffffffffu ? (uint32_t)at / parts : (uint32_t)(at / parts);
        const uint32_t part = (uint32_t)(at - (uint64_t)i * parts), head = part / of_head, in_head = part % of_head;
        const int32_t q = a.seqs[i];
        if (q < 0)
            continue;
        const uint64_t row = a.index != nullptr ? (uint64_t)(int64_t)a.index[i] : i;
        TokenPlace to = place_of_token(s, q, a.positions[i], a.page_stride, a.token_step, true);
        if (row >= a.nrows)
            to.flag = TB_CACHE_RANGE;
        if (to.flag != 0) {
            if (part == 0 && blockIdx.y == 0)
                atomicOr(&s.counts[1], to.flag);
            continue;
        }
        const uint64_t src = a.rows + pool * a.pool_stride + row * a.row_stride + part * 16ull;
        const uint64_t dst = to.at + head * a.head_step;
        u32x4 x[U];
#pragma unroll
        for (uint32_t u = 0; u < U; u++)
            if (pool + u < npools)
                x[u] = *(const gu32x4_at2 *)(src + u * a.pool_stride);
#pragma unroll
        for (uint32_t u = 0; u < U; u++) {
            if (pool + u >= npools)
                break;
            u16x2 m = {0, 0};
#pragma unroll
            for (int e = 0; e < 4; e++)
                m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, x[u][e] & 0x7fff7fffu));
            uint32_t top = max((uint32_t)m.x, (uint32_t)m.y);
            top = max(top, (uint32_t)__shfl_xor((int)top, 1));
            top = max(top, (uint32_t)__shfl_xor((int)top, 2));
            const uint32_t byte = power_byte<T>(top);
            const float power = __uint_as_float(byte << 23);
            uint32_t code = Type16<T>::template round<0>(0, x[u][0], power);
            code = Type16<T>::template round<1>(code, x[u][1], power);
            code = Type16<T>::template round<2>(code, x[u][2], power);
            code = Type16<T>::template round<3>(code, x[u][3], power);
            const uint64_t there = pools.dst[pool + u] + dst;
            *(gu32 *)(there + in_head * 4) = byte == 255 ? 0 : code;
            const uint32_t block = in_head / 4, blocks = of_head / 4;
            if (whole) {   // a word of powers, from the first of its blocks' threads
                uint32_t word = byte;
#pragma unroll
                for (int k = 1; k < 4; k++) {
                    const uint32_t other = (uint32_t)__shfl_down((int)byte, 4 * k);
                    word |= block + k < blocks ? other << (8 * k) : 0;
                }
                if (in_head % 16 == 0)
                    *(gu32 *)(there + a.dim / 2 + block) = word;
            } else if (in_head % 4 == 0) {
                *(gu8 *)(there + a.dim / 2 + block) = (uint8_t)byte;
                if (block + 1 == blocks)
                    for (uint32_t k = blocks; k % 4 != 0; k++)
                        *(gu8 *)(there + a.dim / 2 + k) = 0;
            }
        }
    }
}

hipError_t launch_fp4_append(const Pools &pools, uint32_t npools, const CacheState &s, const Fp4Args &a,
                             uint32_t dtype, hipStream_t stream) {
    const uint32_t parts = a.heads * (a.dim / 8);
    const uint64_t blocks = ((uint64_t)a.n * parts + 255) / 256, most = 1u << 22;
    const dim3 grid((uint32_t)(blocks < most ? blocks : most), (npools + kFp4Pools - 1) / kFp4Pools, 1);
    return launch(dtype == TB_BF16 ? fp4_append_kernel<__bf16> : fp4_append_kernel<_Float16>, grid, 256, stream,
                  nullptr, pools, s, a, parts, npools);
}

template <typename T>
__global__ __launch_bounds__(256) void fp4_read_kernel(Pools pools, CacheState s, Fp4Args a, uint32_t parts,
        uint32_t npools) {
    constexpr uint32_t U = kFp4Pools;
    const uint64_t all = (uint64_t)a.n * parts;
    const uint32_t pool = blockIdx.y * U, of_head = a.dim / 8;
    for (uint64_t at = (uint64_t)blockIdx.x * 256 + threadIdx.x; at < all; at += (uint64_t)gridDim.x * 256) {
        const uint32_t i = at <= 0xffffffffu ? (uint32_t)at / parts : (uint32_t)(at / parts);
        const uint32_t part = (uint32_t)(at - (uint64_t)i * parts), head = part / of_head, in_head = part % of_head;
        const TokenPlace from = place_of_token(s, a.seqs[i], a.positions[i], a.page_stride, a.token_step, false);
        if (from.flag > 0 && part == 0 && blockIdx.y == 0)
            atomicOr(&s.counts[1], from.flag);
        const uint64_t src = from.at + head * a.head_step;
        const uint64_t dst = a.rows + pool * a.pool_stride + i * a.row_stride + part * 16ull;
        uint32_t code[U], byte[U];
#pragma unroll
        for (uint32_t u = 0; u < U; u++) {
            code[u] = byte[u] = 0;
            if (pool + u < npools && from.flag == 0) {
                code[u] = *(const gu32 *)(pools.dst[pool + u] + src + in_head * 4);
                byte[u] = *(const gu8 *)(pools.dst[pool + u] + src + a.dim / 2 + in_head / 4);
            }
        }
#pragma unroll
        for (uint32_t u = 0; u < U; u++)
            if (pool + u < npools)
                *(gu32x4_at2 *)(dst + u * a.pool_stride) = eight_of<T>(code[u], power_of(byte[u], 0));
    }
}

hipError_t launch_fp4_read(const Pools &pools, uint32_t npools, const CacheState &s, const Fp4Args &a,
                           uint32_t dtype, hipStream_t stream) {
    const uint32_t parts = a.heads * (a.dim / 8);
    const uint64_t blocks = ((uint64_t)a.n * parts + 255) / 256, most = 1u << 22;
    const dim3 grid((uint32_t)(blocks < most ? blocks : most), (npools + kFp4Pools - 1) / kFp4Pools, 1);
    return launch(dtype == TB_BF16 ? fp4_read_kernel<__bf16> : fp4_read_kernel<_Float16>, grid, 256, stream, nullptr,
                  pools, s, a, parts, npools);
}

// The bytes of tokens out of their pages: E bytes of one token in kFp4Pools pools a thread.
template <int E>
struct Bytes;
template <>
struct Bytes<16> {
    typedef u32x4 T;
};
template <>
struct Bytes<4> {
    typedef uint32_t T;
};
template <>
struct Bytes<1> {
    typedef uint8_t T;
};

template <int E>
__global__ __launch_bounds__(256) void read_kernel(Pools pools, CacheState s, AppendArgs a, uint32_t parts,
        uint32_t npools) {
    typedef typename Bytes<E>::T piece;
    typedef __attribute__((address_space(1))) piece gpiece;
    constexpr uint32_t U = kFp4Pools;
    const uint64_t all = (uint64_t)a.n * parts;
    const uint32_t pool = blockIdx.y * U;
    for (uint64_t at = (uint64_t)blockIdx.x * 256 + threadIdx.x; at < all; at += (uint64_t)gridDim.x * 256) {
        const uint32_t i = at <= 0xffffffffu ? (uint32_t)at / parts : (uint32_t)(at / parts);
        const uint32_t off = (uint32_t)(at - (uint64_t)i * parts) * E;
        const TokenPlace from = place_of_token(s, a.seqs[i], a.positions[i], a.page_stride, a.token_step, false);
        if (from.flag > 0 && off == 0 && blockIdx.y == 0)
            atomicOr(&s.counts[1], from.flag);
        const uint64_t src = from.at + (off / a.head_bytes) * a.head_step + off % a.head_bytes;
        const uint64_t dst = a.rows + pool * a.pool_stride + i * a.row_stride + off;
        piece x[U];
#pragma unroll
        for (uint32_t u = 0; u < U; u++) {
            x[u] = piece{};
            if (pool + u < npools && from.flag == 0)
                x[u] = *(const gpiece *)(pools.dst[pool + u] + src);
        }
#pragma unroll
        for (uint32_t u = 0; u < U; u++)
            if (pool + u < npools)
                *(gpiece *)(dst + u * a.pool_stride) = x[u];
    }
}

hipError_t launch_read(const Pools &pools, uint32_t npools, const CacheState &s, const AppendArgs &a, uint32_t piece,
                       hipStream_t stream) {
    const uint32_t parts = a.heads * a.head_bytes / piece;
    const uint64_t blocks = ((uint64_t)a.n * parts + 255) / 256, most = 1u << 22;
    const dim3 grid((uint32_t)(blocks < most ? blocks : most), (npools + kFp4Pools - 1) / kFp4Pools, 1);
    return launch(piece == 16 ? read_kernel<16> : (piece == 4 ? read_kernel<4> : read_kernel<1>), grid, 256, stream,
                  nullptr, pools, s, a, parts, npools);
}

// ---- verification ----------------------------------------------------------------
//
// Every test of a node needs three numbers only, p and q at its token and its random number, until one that was
// drawn is rejected: what is left then has a sum over the vocabulary.  Chains and chosen candidates need that sum once, at the
// end, for the next token; drawn siblings once for each that is rejected.  What is left after several
// rejections at one node is max(p - taken q, 0), taken the sum of the z's: where an earlier difference was cut
// at 0, so is the later one.
//
// The first kernel has a workgroup for each stretch of the vocabulary.  Each walks its sequence's tree by itself (one wave; the
// numbers of 64 nodes at once, so that a chain of any length up to that costs two latencies) up to the first sum, and
// sums its stretch.  The second, a workgroup a sequence, goes on from there, and draws the token: the stretch in which the sums
// pass, then the place in it.

struct VerifyArgs {
    const uint8_t *probs, *draft;
    uint64_t probs_stride[2], draft_stride[2];   // bytes
    const int32_t *tokens, *parents;
    const float *uniform;
    const int32_t *tree_nodes, *seqs, *lens;
    int32_t *count, *path, *token, *new_lens, *append_seqs, *append_positions, *append_index;
    uint32_t batch, nodes, vocab, max_seqs;
    uint32_t stretch, stretches;                 // elements, and how many of them the vocabulary is
    struct Walk *walks;                          // [batch] workspace
    double *sums;                                // [batch][stretches]
};

// Where a walk stands.
struct Walk {
    int32_t cur, last;     // the current node; the last one tested
    int32_t count;         // accepted ones
    int32_t waits;         // whether it stands at a rejection that needs its sum
    double z, taken;
};

constexpr uint32_t kMaxStretch = 8192, kMaxStretches = 2048;
// Elements of a stretch: enough workgroups to fill the chip, but none with less than 1,024 elements.
static uint32_t stretch_of(uint32_t batch, uint32_t vocab) {
    uint32_t n = kMaxStretch;
    while (n > 1024 && (uint64_t)batch * ((vocab + n - 1) / n) < 1024)
        n /= 2;
    return n;
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        x += __shfl_xor(x, d);
    return x;
}
__device__ __forceinline__ double lane_double(double x, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Nodes of sequence b.
__device__ __forceinline__ uint32_t nodes_of(const VerifyArgs &g, uint32_t b) {
    if (g.seqs != nullptr && (uint32_t)g.seqs[b] >= g.max_seqs)
        return 0;
    const int32_t n = g.tree_nodes != nullptr ? g.tree_nodes[b] : (int32_t)g.nodes;
    return (uint32_t)min(max(n, 0), (int32_t)g.nodes);
}
// What node t of sequence b proposes; false where it is passed over.
__device__ __forceinline__ bool proposal(const VerifyArgs &g, uint32_t b, uint32_t t, uint32_t n, int32_t *parent,
        int32_t *x) {
    *parent = *x = -1;
    if (t < 1 || t >= n)
        return false;
    const uint64_t at = (uint64_t)b * g.nodes + t;
    *parent = g.parents != nullptr ? g.parents[at] : (int32_t)t - 1;
    *x = g.tokens[at];
    return (uint32_t)*parent < t && (uint32_t)*x < g.vocab;
}

// Goes on with a walk, the same in all lanes of one whole wave: to its end, or (Q) to a rejection.  `write`: the path
// is written.
template <typename T, bool Q>
__device__ __forceinline__ Walk go_on(const VerifyArgs &g, uint32_t b, uint32_t n, Walk w, bool write) {
    const uint32_t lane = threadIdx.x & 63;
    const uint64_t row0 = reinterpret_cast<uint64_t>(g.probs) + b * g.probs_stride[0];
    const uint64_t draft0 = reinterpret_cast<uint64_t>(g.draft) + b * g.draft_stride[0];
    w.waits = 0;
    for (uint32_t g0 = (uint32_t)(w.last + 1) & ~63u; g0 < n && !w.waits; g0 += 64) {
        const uint32_t t = g0 + lane;
        int32_t parent, x;
        const bool there = proposal(g, b, t, n, &parent, &x);
        double u = 0, p = 0, q = 1;
        if (there) {
            u = g.uniform[(uint64_t)b * g.nodes + t];
            p = (double)(float)reinterpret_cast<const T *>(row0 + parent * g.probs_stride[1])[x];
            if (Q)
                q = (double)(float)reinterpret_cast<const T *>(draft0 + parent * g.draft_stride[1])[x];
        }
        if (!Q && g.parents != nullptr) {
            // a token that an earlier sibling had is gone
            bool again = false;
            for (uint32_t h0 = 0; h0 <= g0; h0 += 64) {
                int32_t parent2 = parent, x2 = x;
                bool there2 = there;
                if (h0 != g0)
                    there2 = proposal(g, b, h0 + lane, n, &parent2, &x2);
                parent2 = there2 ? parent2 : -1;
                const uint32_t end = min(64u, n - h0);
                for (uint32_t k = 0; k < end; k++)
                    again |= __builtin_amdgcn_readlane(parent2, k) == parent && __builtin_amdgcn_readlane(x2, k) == x
                            && h0 + k < t;
            }
            if (again)
                p = 0;
        }
        for (;;) {
            const uint64_t next = __ballot(there && parent == w.cur && (int32_t)t > w.last);
            if (next == 0)
                break;
            const int k = __builtin_ctzll(next);
            const double pk = lane_double(p, k), qk = lane_double(q, k), uk = lane_double(u, k);
            const double left = Q ? fmax(pk - w.taken * qk, 0.0) : pk;
            w.last = (int32_t)g0 + k;
            if (uk * qk * w.z < left) {
                w.cur = w.last;
                w.z = 1;
                w.taken = 0;
                if (write && lane == 0)
                    g.path[(uint64_t)b * g.nodes + w.count] = w.cur;
                w.count++;
            } else if (Q) {
                w.taken += w.z;
                w.waits = 1;
                break;
            } else {
                w.z -= pk;
            }
        }
    }
    return w;
}

// What is left at one place of the vocabulary.
template <typename T, bool Q>
struct Left {
    const T *p, *q;
    double taken;
    const uint32_t *gone;   // a bit for each place from `first` on; null: none is gone
    uint32_t first;

    __device__ __forceinline__ Left(const VerifyArgs &g, uint32_t b, const Walk &w, const uint32_t *gone_,
            uint32_t first_) : taken(w.taken), gone(gone_), first(first_) {
        p = reinterpret_cast<const T *>(g.probs + b * g.probs_stride[0] + w.cur * g.probs_stride[1]);
        q = reinterpret_cast<const T *>(g.draft + b * g.draft_stride[0] + w.cur * g.draft_stride[1]);
    }
    __device__ __forceinline__ double of(double p_, double q_, uint32_t x) const {
        if (Q)
            return fmax(p_ - taken * q_, 0.0);
        return gone != nullptr && (gone[(x - first) / 32] >> ((x - first) % 32) & 1) ? 0.0 : p_;
    }
    __device__ __forceinline__ double at(uint32_t x) const {
        return of((double)(float)p[x], Q ? (double)(float)q[x] : 0.0, x);
    }
    // The sum over this thread's part of [begin, end), of `threads`.
    __device__ __forceinline__ double sum(uint32_t begin, uint32_t end, uint32_t thread, uint32_t threads) const {
        constexpr uint32_t E = 16 / sizeof(T);
        typedef T Vec __attribute__((ext_vector_type(E), aligned(sizeof(T))));
        double s = 0;
        for (uint32_t x = begin + thread * E; x < end; x += threads * E) {
            if (x + E <= end) {
                const Vec pv = *reinterpret_cast<const Vec *>(p + x);
                Vec qv = pv;
                if (Q)
                    qv = *reinterpret_cast<const Vec *>(q + x);
#pragma unroll
                for (uint32_t e = 0; e < E; e++)
                    s += of((double)(float)pv[e], (double)(float)qv[e], x + e);
            } else {
                for (uint32_t e = x; e < end; e++)
                    s += at(e);
            }
        }
        return s;
    }
};

// Marks what the current node's children stood for, of [first, end), in gone[]; all threads, with a barrier.
__device__ __forceinline__ void mark_gone(const VerifyArgs &g, uint32_t b, uint32_t n, const Walk &w, uint32_t first,
        uint32_t end, uint32_t *gone) {
    for (uint32_t i = threadIdx.x; i < (end - first + 31) / 32; i += blockDim.x)
        gone[i] = 0;
    __syncthreads();
    for (uint32_t t = threadIdx.x; t < n; t += blockDim.x) {
        int32_t parent, x;
        if (proposal(g, b, t, n, &parent, &x) && parent == w.cur && (uint32_t)x >= first && (uint32_t)x < end)
            atomicOr(&gone[((uint32_t)x - first) / 32], 1u << (((uint32_t)x - first) % 32));
    }
    __syncthreads();
}

template <typename T, bool Q>
__global__ __launch_bounds__(256) void verify_walk_kernel(VerifyArgs g) {
    __shared__ Walk walk;
    __shared__ double parts[4];
    __shared__ uint32_t gone[kMaxStretch / 32];
    const uint32_t b = blockIdx.x / g.stretches, k = blockIdx.x % g.stretches, thread = threadIdx.x;
    const uint32_t n = nodes_of(g, b);
    if (n == 0)
        return;
    if (thread < 64) {
        const Walk to = go_on<T, Q>(g, b, n, Walk{0, 0, 1, 0, 1.0, 0.0}, k == 0);
        if (thread == 0) {
            walk = to;
            if (k == 0)
                g.path[(uint64_t)b * g.nodes] = 0;
        }
    }
    __syncthreads();
    const Walk w = walk;
    const uint32_t begin = k * g.stretch, end = min(begin + g.stretch, g.vocab);
    if (!Q)
        mark_gone(g, b, n, w, begin, end, gone);
    const double s = wave_sum(Left<T, Q>(g, b, w, gone, begin).sum(begin, end, thread, 256));
    if (thread % 64 == 0)
        parts[thread / 64] = s;
    __syncthreads();
    if (thread == 0) {
        g.sums[(uint64_t)b * g.stretches + k] = parts[0] + parts[1] + (parts[2] + parts[3]);
        if (k == 0)
            g.walks[b] = w;
    }
}

constexpr uint32_t kDraw = 1024;   // threads

// The sum of v over the workgroup, the same in all threads and the same whenever it is taken.
__device__ __forceinline__ double block_total(double v, double *lds) {
    v = wave_sum(v);
    __syncthreads();
    if (threadIdx.x % 64 == 0)
        lds[threadIdx.x / 64] = v;
    __syncthreads();
    double all = 0;
    for (uint32_t k = 0; k < kDraw / 64; k++)
        all += lds[k];
    return all;
}
// The sum of v over the threads up to and with this one.
__device__ __forceinline__ double block_upto(double v, double *lds) {
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double y = __shfl_up(v, d);
        if (lane >= (uint32_t)d)
            v += y;
    }
    __syncthreads();
    if (lane == 63)
        lds[wave] = v;
    __syncthreads();
    double before = 0;
    for (uint32_t k = 0; k < wave; k++)
        before += lds[k];
    return before + v;
}

template <typename T, bool Q>
__global__ __launch_bounds__(kDraw) void verify_draw_kernel(VerifyArgs g) {
    __shared__ Walk walk;
    __shared__ double sums[kMaxStretches], lds[kDraw / 64], before;
    __shared__ uint32_t gone[kMaxStretch / 32], found, spare;
    const uint32_t b = blockIdx.x, thread = threadIdx.x, n = nodes_of(g, b);
    const uint64_t row = (uint64_t)b * g.nodes;
    int32_t token = -1;
    if (thread == 0)
        walk = n == 0 ? Walk{0, 0, 0, 0, 1.0, 0.0} : g.walks[b];
    if (n != 0) {
        double s = 0;
        for (uint32_t k = thread; k < g.stretches; k += kDraw)
            s += sums[k] = g.sums[(uint64_t)b * g.stretches + k];
        double total = block_total(s, lds);
        // Takes the sums of what is left anew, a wave a stretch.
        const auto take_sums = [&](const Left<T, Q> &left) {
            for (uint32_t k = thread / 64; k < g.stretches; k += kDraw / 64) {
                const double x = wave_sum(
                        left.sum(k * g.stretch, min((k + 1) * g.stretch, g.vocab), thread % 64, 64));
                if (thread % 64 == 0)
                    sums[k] = x;
            }
            __syncthreads();
            double y = 0;
            for (uint32_t k = thread; k < g.stretches; k += kDraw)
                y += sums[k];
            total = block_total(y, lds);
        };
        if (Q)
            while (walk.waits) {
                Walk w = walk;
                const int32_t last = w.last;
                __syncthreads();
                if (thread < 64) {
                    w.z = total;
                    w = go_on<T, Q>(g, b, n, w, true);
                    if (thread == 0)
                        walk = w;
                }
                __syncthreads();
                if (walk.last == last)   // it had no sibling left
                    break;
                take_sums(Left<T, Q>(g, b, walk, nullptr, 0));
            }
        Walk w = walk;
        bool all = false;   // whether p itself is drawn from
        if (!(total > 0)) {
            w.taken = 0;
            all = true;
            take_sums(Left<T, Q>(g, b, w, nullptr, 0));
        }
        if (total > 0 && total < INFINITY) {
            const double target = (double)g.uniform[row] * total;
            // the first stretch whose sums pass the target, or (rounding) the last with anything in it
            if (thread == 0) {
                found = ~0u;
                spare = 0;
            }
            double passed = 0;
            for (uint32_t k0 = 0; k0 < g.stretches; k0 += kDraw) {
                const uint32_t k = k0 + thread;
                const double mine = k < g.stretches ? sums[k] : 0;
                const double upto = passed + block_upto(mine, lds);
                if (mine > 0 && upto > target)
                    atomicMin(&found, k);
                if (mine > 0)
                    atomicMax(&spare, k);
                passed += block_total(mine, lds);
            }
            __syncthreads();
            const uint32_t k = found != ~0u ? found : spare;
            __syncthreads();
            double s0 = 0;
            for (uint32_t j = thread; j < k; j += kDraw)
                s0 += sums[j];
            s0 = block_total(s0, lds);
            if (thread == 0) {
                before = s0;
                found = ~0u;
                spare = 0;
            }
            const uint32_t begin = k * g.stretch, end = min(begin + g.stretch, g.vocab);
            const bool any_gone = !Q && !all;
            if (any_gone)
                mark_gone(g, b, n, w, begin, end, gone);
            const Left<T, Q> left(g, b, w, any_gone ? gone : nullptr, begin);
            const uint32_t each = g.stretch / kDraw, x0 = begin + thread * each;
            double mine = 0;
            for (uint32_t x = x0; x < min(x0 + each, end); x++)
                mine += left.at(x);
            double upto = block_upto(mine, lds) + before;
            if (mine > 0) {
                // from here on by single places; this thread's end is the sum just taken
                double run = upto - mine;
                uint32_t last = x0;
                for (uint32_t x = x0; x < min(x0 + each, end); x++) {
                    const double v = left.at(x);
                    if (v > 0)
                        last = x;
                }
                atomicMax(&spare, last + 1);
                if (upto > target) {
                    uint32_t hit = last;
                    for (uint32_t x = x0; x < last; x++) {
                        const double v = left.at(x);
                        run += v;
                        if (v > 0 && run > target) {
                            hit = x;
                            break;
                        }
                    }
                    atomicMin(&found, hit);
                }
            }
            __syncthreads();
            token = (int32_t)(found != ~0u ? found : (spare != 0 ? spare - 1 : begin));
        }
    }
    __syncthreads();
    const int32_t count = walk.count;
    const int32_t q = g.seqs != nullptr ? g.seqs[b] : -1;
    const bool held = g.seqs != nullptr && (uint32_t)q < g.max_seqs;
    const int32_t had = held ? g.lens[q] : 0;
    if (thread == 0) {
        g.count[b] = count;
        g.token[b] = token;
        if (g.seqs != nullptr)
            g.new_lens[b] = had + count;
    }
    for (uint32_t i = thread; i < g.nodes; i += kDraw) {
        const bool real = (int32_t)i < count;
        // written by this kernel too: past the L1
        const int32_t node = real ? __hip_atomic_load(&g.path[row + i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : -1;
        if (!real)
            g.path[row + i] = -1;
        if (g.seqs != nullptr) {
            g.append_seqs[row + i] = real ? q : -1;
            g.append_positions[row + i] = real ? had + (int32_t)i : 0;
            g.append_index[row + i] = real ? (int32_t)(row + node) : 0;
        }
    }
}

static uint64_t round16(uint64_t n) { return (n + 15) / 16 * 16; }

uint64_t verify_workspace(uint32_t batch, uint32_t vocab) {
    const uint32_t stretch = stretch_of(batch, vocab);
    return round16(sizeof(Walk) * batch) + round16(8ull * batch * ((vocab + stretch - 1) / stretch));
}

template <typename T>
static hipError_t launch_verify_type(const VerifyArgs &g, bool drafted, hipStream_t stream) {
    LaunchSeq seq;
    const hipError_t e = launch(drafted ? verify_walk_kernel<T, true> : verify_walk_kernel<T, false>,
            g.batch * g.stretches, 256, stream, nullptr, g);
    if (e != hipSuccess)
        return e;
    seq.last();
    return launch(drafted ? verify_draw_kernel<T, true> : verify_draw_kernel<T, false>, g.batch, kDraw, stream,
            nullptr, g);
}

hipError_t launch_verify(const tb_verify &v, hipStream_t stream) {
    VerifyArgs g;
    const uint64_t size = v.dtype == TB_FP32 ? 4 : 2;
    g.probs = static_cast<const uint8_t *>(v.probs);
    g.draft = static_cast<const uint8_t *>(v.draft_probs);
    for (int k = 0; k < 2; k++) {
        g.probs_stride[k] = v.probs_stride[k] * size;
        g.draft_stride[k] = v.draft_stride[k] * size;
    }
    g.tokens = v.tokens;
    g.parents = v.parents;
    g.uniform = v.uniform;
    g.tree_nodes = v.tree_nodes;
    g.seqs = v.seqs;
    g.lens = v.lens;
    g.count = v.count;
    g.path = v.path;
    g.token = v.token;
    g.new_lens = v.new_lens;
    g.append_seqs = v.append_seqs;
    g.append_positions = v.append_positions;
    g.append_index = v.append_index;
    g.batch = v.batch;
    g.nodes = v.nodes;
    g.vocab = v.vocab;
    g.max_seqs = v.max_seqs;
    g.stretch = stretch_of(v.batch, v.vocab);
    g.stretches = (v.vocab + g.stretch - 1) / g.stretch;   // <= kMaxStretches
    uint8_t *ws = static_cast<uint8_t *>(v.workspace);
    g.walks = reinterpret_cast<Walk *>(ws);
    g.sums = reinterpret_cast<double *>(ws + round16(sizeof(Walk) * v.batch));
    switch (v.dtype) {
    case TB_BF16: return launch_verify_type<__bf16>(g, v.draft_probs != nullptr, stream);
    case TB_FP16: return launch_verify_type<_Float16>(g, v.draft_probs != nullptr, stream);
    default: return launch_verify_type<float>(g, v.draft_probs != nullptr, stream);
    }
}

}  // namespace tbk
