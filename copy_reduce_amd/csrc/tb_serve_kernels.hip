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
    const uint32_t j = (uint32_t)pos / s.page_tokens, in_page = (uint32_t)pos % s.page_tokens;
    const uint32_t page = (uint32_t)s.table[(uint64_t)q * s.max_pages + min(j, s.max_pages - 1)];   // beside the length
    if (pos < 0 || pos >= min(n, most))
        return {TB_CACHE_RANGE, 0};
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

// A workgroup has a few tokens of one pool: it finds their places, one a thread, and then goes over their elements, 8 a
// thread and four threads a block of 32, kAtOnce such pieces on their way at once and as many behind them.  The conversion to 4
// bits is the hardware's: to the nearest, of two the even code, larger ones to 6.
//
// Each of the 8 XCDs has an eighth of the work, pool by pool.  Heads of 68 bytes share lines with their neighbours, which so
// meet in one L2, in whatever order the tokens are listed.
//
// Bound by HBM in the large: 3,500 tokens of 64 pools, 8 heads of 128, in 109 us by token and 111 by head, back out in 81 (a
// copy's rate would be 89 either way); in random order 111 and 114, and 82; 131,072 tokens of 2 pools in 133, back out
// in 95 (104).  With a token's pools in one thread instead, which finds its place by itself: 106 and 115, 86; 107 and 122, 88
// and 113; 163, 100; 16,384 tokens of 8 pools, 4 heads of 256, which partly stay in the caches, 61 against 71 here, where
// instructions count.  Registers for 8 waves spill: 143 and 104 instead of 111 and 81.
constexpr uint32_t kXcds = 8, kAtOnce = 4, kTokens = 64, kPieces = 2048;
struct TokenWork {
    uint32_t heads, of_head, parts;    // of a token; pieces of a head and of a token
    uint32_t tokens, groups;           // of a workgroup; workgroups a pool
    uint32_t step_token, step_head, step_in;   // 256 pieces on
    uint64_t share;                    // (pool, group) pairs an XCD
    uint32_t npools;
};
static TokenWork token_work(const Fp4Args &a, uint32_t npools) {
    TokenWork w;
    w.heads = a.heads;
    w.of_head = a.dim / 8;
    w.parts = a.heads * w.of_head;
    w.tokens = 1;
    while (w.tokens < kTokens && w.tokens * 2 * (uint64_t)w.parts <= kPieces)
        w.tokens *= 2;
    while (w.tokens > 1 && w.tokens * (uint64_t)w.parts > 256 && ((uint64_t)a.n + w.tokens - 1) / w.tokens * npools < 1024)
        w.tokens /= 2;
    w.groups = (uint32_t)(((uint64_t)a.n + w.tokens - 1) / w.tokens);
    w.share = ((uint64_t)w.groups * npools + kXcds - 1) / kXcds;
    const uint32_t heads = 256 / w.of_head;
    w.step_token = heads / w.heads;
    w.step_head = heads % w.heads;
    w.step_in = 256 % w.of_head;
    w.npools = npools;
    return w;
}
static uint32_t token_grid(const TokenWork &w) {
    return kXcds * (uint32_t)(w.share < (1u << 19) ? w.share : 1u << 19);
}

// A thread's place among the pieces of its workgroup's tokens.
struct Piece {
    uint32_t token, head, in_head;

    __device__ __forceinline__ explicit Piece(const TokenWork &w) {
        const uint32_t h = threadIdx.x / w.of_head;
        in_head = threadIdx.x % w.of_head;
        token = h / w.heads;
        head = h % w.heads;
    }
    __device__ __forceinline__ void next(const TokenWork &w) {
        in_head += w.step_in;
        head += w.step_head;
        token += w.step_token;
        if (in_head >= w.of_head) {
            in_head -= w.of_head;
            head++;
        }
        if (head >= w.heads) {
            head -= w.heads;
            token++;
        }
    }
};

// f(pool, first token, tokens) for each share of this workgroup's; f has barriers.
template <typename F>
__device__ __forceinline__ void over_tokens(const TokenWork &w, uint32_t n, F f) {
    const uint64_t end = min((uint64_t)(blockIdx.x % kXcds + 1) * w.share, (uint64_t)w.groups * w.npools);
    for (uint64_t k = blockIdx.x % kXcds * w.share + blockIdx.x / kXcds; k < end; k += gridDim.x / kXcds) {
        const uint32_t pool = k <= 0xffffffffu ? (uint32_t)k / w.groups : (uint32_t)(k / w.groups);
        const uint32_t first = (uint32_t)(k - (uint64_t)pool * w.groups) * w.tokens;
        f(pool, first, min(w.tokens, n - first));
    }
}

constexpr uint64_t kNowhere = ~0ull;

// The lane's value of `x` C says, in its row of 16; 0 past the row's end.
template <int C>
__device__ __forceinline__ uint32_t of_lane(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, C, 0xf, 0xf, true);
}
constexpr int kPairs = 0xb1, kTwos = 0x4e, kAhead4 = 0x104;   // 1 0 3 2; 2 3 0 1; four lanes on

// WHOLE: no head lies in two waves, and a thread's place in a head is the same for all of its pieces.
template <typename T, bool WHOLE>
__global__ __launch_bounds__(256, 6) void fp4_append_kernel(Pools pools, CacheState s, Fp4Args a, TokenWork w) {
    __shared__ uint64_t rows[kTokens], places[kTokens];
    constexpr uint32_t U = kAtOnce;
    const uint32_t blocks = w.of_head / 4, mine = threadIdx.x % w.of_head;
    const uint32_t powers = ~0u >> (8 * max(4 - (int)(blocks - min(mine / 4, blocks)), 0));   // of a word
    over_tokens(w, a.n, [&](uint32_t pool, uint32_t first, uint32_t tokens) {
        if (threadIdx.x < tokens) {
            const uint32_t i = first + threadIdx.x;
            const int32_t q = a.seqs[i], position = a.positions[i];
            const uint64_t row = a.index != nullptr ? (uint64_t)(int64_t)a.index[i] : i;
            TokenPlace to = place_of_token(s, q, position, a.page_stride, a.token_step, true);
            if (q >= 0 && row >= a.nrows)
                to.flag = TB_CACHE_RANGE;
            if (to.flag > 0 && pool == 0)
                atomicOr(&s.counts[1], to.flag);
            rows[threadIdx.x] = a.rows + row * a.row_stride + pool * a.pool_stride;
            places[threadIdx.x] = to.flag == 0 ? pools.dst[pool] + to.at : kNowhere;
        }
        __syncthreads();
        const uint32_t pieces = tokens * w.parts;
        Piece ahead(w), here(w);
        const auto load = [&](uint32_t at, u32x4 *x) {
#pragma unroll
            for (uint32_t u = 0; u < U; u++) {
                if (at + u * 256 < pieces && places[ahead.token] != kNowhere)
                    x[u] = __builtin_nontemporal_load(
                            (const gu32x4_at2 *)(rows[ahead.token] + (ahead.head * w.of_head + (WHOLE ? mine : ahead.in_head)) * 16ull));
                ahead.next(w);
            }
        };
        u32x4 x[U], after[U];
        load(threadIdx.x, x);
        for (uint32_t at = threadIdx.x; at < pieces; at += U * 256) {
            load(at + U * 256, after);   // past the last: none
#pragma unroll
            for (uint32_t u = 0; u < U; u++) {
                const Piece piece = here;
                here.next(w);
                if (at + u * 256 >= pieces)
                    break;
                const uint64_t token = places[piece.token];
                if (token == kNowhere)
                    continue;
                const uint64_t place = token + piece.head * (uint32_t)a.head_step;
                u16x2 m = {0, 0};
#pragma unroll
                for (int e = 0; e < 4; e++)
                    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, x[u][e] & 0x7fff7fffu));
                uint32_t top = max((uint32_t)m.x, (uint32_t)m.y);
                top = max(top, of_lane<kPairs>(top));
                top = max(top, of_lane<kTwos>(top));
                const uint32_t byte = power_byte<T>(top);
                const float power = __uint_as_float(byte << 23);
                uint32_t code = Type16<T>::template round<0>(0, x[u][0], power);
                code = Type16<T>::template round<1>(code, x[u][1], power);
                code = Type16<T>::template round<2>(code, x[u][2], power);
                code = Type16<T>::template round<3>(code, x[u][3], power);
                const uint32_t in_head = WHOLE ? mine : piece.in_head, block = in_head / 4;
                *(gu32 *)(place + in_head * 4) = byte == 255 ? 0 : code;
                if (WHOLE) {   // a word of powers, from the first of its blocks' threads
                    const uint32_t word = byte | of_lane<kAhead4>(byte) << 8 | of_lane<kAhead4 + 4>(byte) << 16 |
                                          of_lane<kAhead4 + 8>(byte) << 24;
                    if (in_head % 16 == 0)
                        *(gu32 *)(place + a.dim / 2 + block) = word & powers;
                } else if (in_head % 4 == 0) {
                    *(gu8 *)(place + a.dim / 2 + block) = (uint8_t)byte;
                    if (block + 1 == blocks)
                        for (uint32_t k = blocks; k % 4 != 0; k++)
                            *(gu8 *)(place + a.dim / 2 + k) = 0;
                }
            }
#pragma unroll
            for (uint32_t u = 0; u < U; u++)
                x[u] = after[u];
        }
        __syncthreads();
    });
}

hipError_t launch_fp4_append(const Pools &pools, uint32_t npools, const CacheState &s, const Fp4Args &a,
                             uint32_t dtype, hipStream_t stream) {
    const TokenWork w = token_work(a, npools);
    const bool whole = 64 % w.of_head == 0;
    return launch(dtype == TB_BF16 ? (whole ? fp4_append_kernel<__bf16, true> : fp4_append_kernel<__bf16, false>)
                                   : (whole ? fp4_append_kernel<_Float16, true> : fp4_append_kernel<_Float16, false>),
                  token_grid(w), 256, stream, nullptr, pools, s, a, w);
}

template <typename T>
__global__ __launch_bounds__(256, 6) void fp4_read_kernel(Pools pools, CacheState s, Fp4Args a, TokenWork w) {
    __shared__ uint64_t places[kTokens];
    constexpr uint32_t U = kAtOnce;
    over_tokens(w, a.n, [&](uint32_t pool, uint32_t first, uint32_t tokens) {
        if (threadIdx.x < tokens) {
            const uint32_t i = first + threadIdx.x;
            const TokenPlace from = place_of_token(s, a.seqs[i], a.positions[i], a.page_stride, a.token_step, false);
            if (from.flag > 0 && pool == 0)
                atomicOr(&s.counts[1], from.flag);
            places[threadIdx.x] = from.flag == 0 ? pools.dst[pool] + from.at : kNowhere;
        }
        __syncthreads();
        const uint32_t pieces = tokens * w.parts;
        const uint64_t out = a.rows + pool * a.pool_stride + first * a.row_stride;
        Piece ahead(w), here(w);
        const auto load = [&](uint32_t at, uint32_t *code, uint32_t *byte) {
#pragma unroll
            for (uint32_t u = 0; u < U; u++) {
                code[u] = byte[u] = 0;
                const uint64_t token = at + u * 256 < pieces ? places[ahead.token] : kNowhere;
                if (token != kNowhere) {
                    const uint64_t place = token + ahead.head * (uint32_t)a.head_step;
                    code[u] = *(const gu32 *)(place + ahead.in_head * 4);
                    byte[u] = *(const gu8 *)(place + a.dim / 2 + ahead.in_head / 4);
                }
                ahead.next(w);
            }
        };
        uint32_t code[U], byte[U], code2[U], byte2[U];
        load(threadIdx.x, code, byte);
        for (uint32_t at = threadIdx.x; at < pieces; at += U * 256) {
            load(at + U * 256, code2, byte2);
#pragma unroll
            for (uint32_t u = 0; u < U; u++) {
                if (at + u * 256 < pieces)
                    __builtin_nontemporal_store(eight_of<T>(code[u], power_of(byte[u], 0)),
                            (gu32x4_at2 *)(out + here.token * a.row_stride + (here.head * w.of_head + here.in_head) * 16ull));
                here.next(w);
                code[u] = code2[u];
                byte[u] = byte2[u];
            }
        }
        __syncthreads();
    });
}

hipError_t launch_fp4_read(const Pools &pools, uint32_t npools, const CacheState &s, const Fp4Args &a,
                           uint32_t dtype, hipStream_t stream) {
    const TokenWork w = token_work(a, npools);
    return launch(dtype == TB_BF16 ? fp4_read_kernel<__bf16> : fp4_read_kernel<_Float16>, token_grid(w), 256, stream,
                  nullptr, pools, s, a, w);
}

// The bytes of tokens out of their pages: E bytes of one token in kReadPools pools a thread.  Bound by HBM: 3,500 tokens of 64
// pools, 8 heads of 256 bytes, in 160 to 170 us, 5.4 to 5.7 TB/s (140 at a copy's rate).
constexpr uint32_t kReadPools = 4;
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
    constexpr uint32_t U = kReadPools;
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
    const dim3 grid((uint32_t)(blocks < most ? blocks : most), (npools + kReadPools - 1) / kReadPools, 1);
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
// The first kernel, a wave a sequence, walks the tree up to the first sum: the numbers of 64 nodes at once, so that a
// chain of any length up to that costs two latencies.  The second has a wave for each stretch of the vocabulary, which sums
// it; the last workgroup of a sequence to end goes on with the walk, if it is not at its end, and draws the token: the stretch in which the
// sums pass, then the place in it.
//
// Bound by latencies: 64 chains of 8 over 131,072 in 32 bits, 67 MB, in 28 us, 5 of the walk and 24 of sums and draw (10 at a
// copy's rate); 3 such chains of 5 over 32,000 in 16.  8 trees of 13 drawn nodes over 50,001 in 36, where one workgroup
// goes over the rows once for each rejected sibling.

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
    uint32_t groups;                             // workgroups a sequence
    uint32_t *ended;                             // [batch] those that have ended
    double *sums;                                // [batch][stretches]
};

// Where a walk stands.
struct Walk {
    int32_t cur, last;     // the current node; the last one tested
    int32_t count;         // accepted ones
    int32_t waits;         // whether it stands at a rejection that needs its sum
    double z, taken;
};

constexpr uint32_t kDraw = 1024, kDrawWaves = kDraw / 64;   // threads and waves of a workgroup
constexpr uint32_t kMaxStretch = 8192, kMaxStretches = 4096;
// Elements of a stretch: small enough that a workgroup's waves all have one, where that takes no more workgroups, and that
// there are up to as many workgroups as CUs, which all run at once; but no more stretches than there is room for in LDS.
// Halved until there are at least as many workgroups as CUs, whatever their waves have, 16 bits: 255 chains over 32,000 tokens
// 34 us against 22, 256 of them 26 against 22, 130 over 131,072 tokens 44 against 35.
// Stretches of 1,024 at least instead of 512: 16 chains over 131,072 tokens 23.2 us against 19.5; workgroups of 512
// threads, two on a CU: 25.5, and 64 such chains 29.6 against 30.3.
constexpr uint32_t kDrawGroups = 256;
static uint32_t stretch_of(uint32_t batch, uint32_t vocab) {
    const auto groups = [&](uint32_t n) { return (vocab + n * kDrawWaves - 1) / (n * kDrawWaves); };
    uint32_t n = kMaxStretch;
    while (n > 512 && (vocab + n / 2 - 1) / (n / 2) <= kMaxStretches
            && (groups(n / 2) == groups(n) || (uint64_t)batch * groups(n / 2) <= kDrawGroups))
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
// 64 nodes of a sequence, one a lane: what each proposes and the numbers of its test.
struct Proposals {
    uint32_t first;      // of the 64; ~0: none yet
    bool there;          // not passed over
    int32_t parent, x;
    double u, p, q;
};

// What node t of sequence b proposes; false where it is passed over.  t < nodes of the call, n: of the sequence.
__device__ __forceinline__ bool proposal(const VerifyArgs &g, uint32_t b, uint32_t t, uint32_t n, int32_t *parent,
        int32_t *x) {
    const uint64_t at = (uint64_t)b * g.nodes + t;
    *parent = g.parents != nullptr ? g.parents[at] : (int32_t)t - 1;
    *x = g.tokens[at];
    return t >= 1 && t < n && (uint32_t)*parent < t && (uint32_t)*x < g.vocab;
}

template <typename T, bool Q>
__device__ __forceinline__ void look_at(const VerifyArgs &g, uint32_t b, uint32_t n, uint32_t first, Proposals *s) {
    const uint32_t lane = threadIdx.x & 63, t = first + lane;
    const uint8_t *const row0 = g.probs + b * g.probs_stride[0], *const draft0 = g.draft + b * g.draft_stride[0];
    s->first = first;
    s->there = false;
    s->parent = s->x = -1;
    s->u = s->p = 0;
    s->q = 1;
    if (t < g.nodes) {
        s->u = g.uniform[(uint64_t)b * g.nodes + t];
        s->there = proposal(g, b, t, n, &s->parent, &s->x);
    }
    if (s->there) {
        s->p = (double)(float)reinterpret_cast<const T *>(row0 + s->parent * g.probs_stride[1])[s->x];
        if (Q)
            s->q = (double)(float)reinterpret_cast<const T *>(draft0 + s->parent * g.draft_stride[1])[s->x];
    }
}

// Whether an earlier child of `cur` than the k-th of these nodes proposes the same.
__device__ __forceinline__ bool proposed_before(const VerifyArgs &g, uint32_t b, uint32_t n, const Proposals &s, int k,
        int32_t cur) {
    const uint32_t lane = threadIdx.x & 63;
    const int32_t x = __builtin_amdgcn_readlane(s.x, k);
    if (__ballot(s.there && s.parent == cur && (int)lane < k && s.x == x) != 0)
        return true;
    for (uint32_t first = (uint32_t)(cur + 1) & ~63u; first < s.first; first += 64) {
        int32_t parent = -1, other = -1;
        const bool there = proposal(g, b, first + lane, n, &parent, &other);
        if (__ballot(there && parent == cur && other == x) != 0)
            return true;
    }
    return false;
}

// Goes on with a walk, the same in all lanes of one whole wave: to its end, or (Q) to a rejection after which the current
// node has another child.  `write`: the path is written.
template <typename T, bool Q>
__device__ __forceinline__ Walk go_on(const VerifyArgs &g, uint32_t b, uint32_t n, Walk w, Proposals *s, bool write) {
    const uint32_t lane = threadIdx.x & 63;
    bool rejected = false;
    w.waits = 0;
    for (uint32_t first = (uint32_t)(w.last + 1) & ~63u; first < n; first += 64) {
        if (s->first != first)
            look_at<T, Q>(g, b, n, first, s);
        for (;;) {
            const uint64_t next = __ballot(s->there && s->parent == w.cur && (int32_t)(first + lane) > w.last);
            if (next == 0)
                break;
            if (Q && rejected) {   // its test needs the sum
                w.waits = 1;
                return w;
            }
            const int k = __builtin_ctzll(next);
            double p = lane_double(s->p, k);
            const double q = lane_double(s->q, k), u = lane_double(s->u, k);
            if (!Q && g.parents != nullptr && proposed_before(g, b, n, *s, k, w.cur))
                p = 0;   // that token is gone
            const double left = Q ? fmax(__builtin_fma(-w.taken, q, p), 0.0) : p;
            w.last = (int32_t)first + k;
            if (u * q * w.z < left) {
                w.cur = w.last;
                w.z = 1;
                w.taken = 0;
                if (write && lane == 0)
                    g.path[(uint64_t)b * g.nodes + w.count] = w.cur;
                w.count++;
            } else if (Q) {
                w.taken += w.z;
                rejected = true;
            } else {
                w.z -= p;
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
            return fmax(__builtin_fma(-taken, q_, p_), 0.0);
        return gone != nullptr && p_ > 0 && (gone[(x - first) / 32] >> ((x - first) % 32) & 1) ? 0.0 : p_;
    }
    __device__ __forceinline__ double at(uint32_t x) const {
        return of((double)(float)p[x], Q ? (double)(float)q[x] : 0.0, x);
    }
    // The sums of the stretches that lie in [begin, end), by one whole wave: done(k, sum) for each.  begin is a whole number of
    // stretches, or of runs of kRun elements, whose loads are on their way together.
    static constexpr uint32_t E = 16 / sizeof(T), kLoads = 8, kRun = kLoads * 64 * E;
    // ready() is called once, with the first loads on their way.
    template <typename Done, typename Ready>
    __device__ __forceinline__ void sums(uint32_t begin, uint32_t end, uint32_t stretch, Done done, Ready ready) const {
        typedef T Vec __attribute__((ext_vector_type(E), aligned(sizeof(T))));
        const uint32_t lane = threadIdx.x & 63;
        double s = 0;
#pragma unroll 1
        for (uint32_t x0 = begin; x0 < end; x0 += kRun) {
            Vec pv[kLoads], qv[kLoads];
#pragma unroll
            for (uint32_t i = 0; i < kLoads; i++) {
                const uint32_t x = x0 + (i * 64 + lane) * E;
                pv[i] = qv[i] = Vec{};
                if (x + E <= end) {
                    pv[i] = *reinterpret_cast<const Vec *>(p + x);
                    if (Q)
                        qv[i] = *reinterpret_cast<const Vec *>(q + x);
                } else if (x < end) {   // the end of the vocabulary
#pragma unroll
                    for (uint32_t e = 0; e < E - 1; e++)
                        if (x + e < end) {
                            pv[i][e] = p[x + e];
                            if (Q)
                                qv[i][e] = q[x + e];
                        }
                }
            }
            if (x0 == begin)
                ready();
#pragma unroll
            for (uint32_t i = 0; i < kLoads; i++) {
                const uint32_t x = x0 + i * 64 * E, next = x + 64 * E;
                if (x >= end)
                    break;
#pragma unroll
                for (uint32_t e = 0; e < E; e++)
                    s += of((double)(float)pv[i][e], Q ? (double)(float)qv[i][e] : 0.0, x + lane * E + e);
                if (next % stretch == 0 || next >= end) {
                    const double all = wave_sum(s);
                    done(x / stretch, all);
                    s = 0;
                }
            }
        }
    }
};

// What this thread's nodes propose, the first of them read before it is known what for.
struct Gone {
    const VerifyArgs &g;
    uint32_t b, n;
    bool there;
    int32_t parent, x;

    __device__ __forceinline__ Gone(const VerifyArgs &g_, uint32_t b_, uint32_t n_) : g(g_), b(b_), n(n_), there(false),
            parent(-1), x(-1) {
        if (n != 0 && threadIdx.x < g.nodes)
            there = proposal(g, b, threadIdx.x, n, &parent, &x);
    }
    __device__ __forceinline__ void one(bool there_, int32_t parent_, uint32_t x_, int32_t cur, uint32_t first,
            uint32_t end, uint32_t *bits) const {
        if (there_ && parent_ == cur && x_ >= first && x_ < end)
            atomicOr(&bits[(x_ - first) / 32], 1u << ((x_ - first) % 32));
    }
    // Marks what the children of `cur` propose, of [first, end), in bits[]; all threads, with barriers.
    __device__ __forceinline__ void mark(int32_t cur, uint32_t first, uint32_t end, uint32_t *bits) const {
        for (uint32_t i = threadIdx.x; i < (end - first + 31) / 32; i += kDraw)
            bits[i] = 0;
        __syncthreads();
        one(there, parent, (uint32_t)x, cur, first, end, bits);
        for (uint32_t t = threadIdx.x + kDraw; t < n; t += kDraw) {
            int32_t parent2 = -1, x2 = -1;
            const bool there2 = proposal(g, b, t, n, &parent2, &x2);
            one(there2, parent2, (uint32_t)x2, cur, first, end, bits);
        }
        __syncthreads();
    }
};

template <typename T, bool Q>
__global__ __launch_bounds__(64) void verify_walk_kernel(VerifyArgs g) {
    const uint32_t b = blockIdx.x;
    const uint64_t row = (uint64_t)b * g.nodes;
    Proposals s;
    const uint32_t n = nodes_of(g, b);
    look_at<T, Q>(g, b, n, 0, &s);
    Walk w = {0, 0, n == 0 ? 0 : 1, 0, 1.0, 0.0};
    w = go_on<T, Q>(g, b, n, w, &s, true);
    if (threadIdx.x == 0) {
        if (n != 0)
            g.path[row] = 0;
        g.walks[b] = w;
        g.ended[b] = 0;
    }
}

// Sums of x over the lanes up to and with this one.
__device__ __forceinline__ double wave_upto(double x) {
    const uint32_t lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double y = __shfl_up(x, d);
        if (lane >= (uint32_t)d)
            x += y;
    }
    return x;
}

// Values that other workgroups of this kernel wrote, or another wave of this one: past the L1.
template <typename N>
__device__ __forceinline__ N fresh(const N *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <typename T, bool Q>
__global__ __launch_bounds__(kDraw) void verify_draw_kernel(VerifyArgs g) {
    __shared__ Walk walk;
    __shared__ double sums[kMaxStretches], waves[kDrawWaves];
    __shared__ uint32_t gone[kMaxStretch * kDrawWaves / 32], found, spare, last_one;
    const uint32_t b = blockIdx.x / g.groups, thread = threadIdx.x, lane = thread & 63, wave = thread >> 6;
    const uint64_t row = (uint64_t)b * g.nodes;
    const double u = g.uniform[row];
    Walk w = g.walks[b];
    const uint32_t n = nodes_of(g, b);
    const int32_t seq = g.seqs != nullptr ? g.seqs[b] : -1;
    const Gone whose(g, b, Q ? 0 : n);
    int32_t token = -1, had = 0, node = -1, walked = 0;
    if (n != 0) {   // this wave's stretch
        const uint32_t first = blockIdx.x % g.groups * kDrawWaves, k = first + wave;
        const uint32_t begin = first * g.stretch, end = min(begin + kDrawWaves * g.stretch, g.vocab);
        const auto ready = [&] {
            if (!Q)
                whose.mark(w.cur, begin, end, gone);
        };
        if (k < g.stretches)
            Left<T, Q>(g, b, w, gone, begin).sums(
                    k * g.stretch, min((k + 1) * g.stretch, g.vocab), g.stretch, [&](uint32_t j, double x) {
                        if (lane == 0)
                            __hip_atomic_store(&g.sums[(uint64_t)b * g.stretches + j], x, __ATOMIC_RELAXED,
                                    __HIP_MEMORY_SCOPE_AGENT);
                    }, ready);
        else
            ready();
        // The sums bypass the L2, so that the wait makes them seen by all before this workgroup is counted.  A
        // release would do as well, and write the L2 back first.
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (thread == 0)
            last_one = __hip_atomic_fetch_add(&g.ended[b], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1;
        __syncthreads();
        if (last_one != g.groups)
            return;
        for (uint32_t i = thread; i < g.stretches; i += kDraw)
            sums[i] = fresh(&g.sums[(uint64_t)b * g.stretches + i]);
        had = g.seqs != nullptr ? g.lens[seq] : 0;
        node = (int32_t)thread < w.count ? g.path[row + thread] : -1;   // of the first kernel
        walked = w.count;
        __syncthreads();
        // The same in every wave, and no barrier.
        const auto total_of = [&] {
            double y = 0;
            for (uint32_t k = lane; k < g.stretches; k += 64)
                y += sums[k];
            return wave_sum(y);
        };
        // Takes the sums of what is left anew: by stretches, or by runs of several.
        const auto take_sums = [&](const Left<T, Q> &left) {
            const uint32_t step = max(g.stretch, Left<T, Q>::kRun);
            __syncthreads();
            for (uint32_t x = wave * step; x < g.vocab; x += kDrawWaves * step)
                left.sums(x, min(x + step, g.vocab), g.stretch, [&](uint32_t j, double y) {
                    if (lane == 0)
                        sums[j] = y;
                }, [] {});
            __syncthreads();
        };
        double total = total_of();
        if (Q) {
            Proposals s;
            s.first = ~0u;
            while (w.waits) {
                if (wave == 0) {
                    w.z = total;
                    w = go_on<T, Q>(g, b, n, w, &s, true);
                    if (lane == 0)
                        walk = w;
                }
                __syncthreads();
                w = walk;
                take_sums(Left<T, Q>(g, b, w, nullptr, 0));
                total = total_of();
            }
        }
        Walk from = w;
        bool all = false;   // whether p itself is drawn from
        if (!(total > 0)) {
            from.taken = 0;
            all = true;
            take_sums(Left<T, Q>(g, b, from, nullptr, 0));
            total = total_of();
        }
        if (total > 0 && total < INFINITY) {
            const double target = u * total;
            // the first stretch whose sums pass the target, or (rounding) the last with anything in it
            uint32_t stretch = 0;
            double passed = 0, before = 0;
            for (uint32_t k0 = 0; k0 < g.stretches; k0 += 64) {
                const double mine = k0 + lane < g.stretches ? sums[k0 + lane] : 0;
                const double upto = passed + wave_upto(mine);
                const uint64_t some = __ballot(mine > 0), over = __ballot(mine > 0 && upto > target);
                const uint64_t pick = over != 0 ? over & -over : some;
                if (pick != 0) {
                    const int k = 63 - __builtin_clzll(pick);
                    stretch = k0 + k;
                    before = lane_double(upto, k) - lane_double(mine, k);
                }
                if (over != 0)
                    break;
                passed = lane_double(upto, 63);
            }
            // the first place in it
            const uint32_t begin = stretch * g.stretch, end = min(begin + g.stretch, g.vocab);
            const bool any_gone = !Q && !all;
            if (thread == 0) {
                found = ~0u;
                spare = begin;
            }
            if (any_gone)
                whose.mark(w.cur, begin, end, gone);
            const Left<T, Q> left(g, b, from, any_gone ? gone : nullptr, begin);
            const uint32_t each = max(g.stretch / kDraw, 1u), x0 = begin + thread * each;
            constexpr uint32_t kEach = kMaxStretch / kDraw;
            double v[kEach], mine = 0;
#pragma unroll
            for (uint32_t e = 0; e < kEach; e++) {
                v[e] = e < each && x0 + e < end ? left.at(x0 + e) : 0;
                mine += v[e];
            }
            double upto = wave_upto(mine);
            if (lane == 63)
                waves[wave] = upto;
            __syncthreads();
            for (uint32_t k = 0; k < wave; k++)
                before += waves[k];
            upto += before;
            if (mine > 0) {
                uint32_t hit = ~0u, last = 0;
                double run = upto - mine;
#pragma unroll
                for (uint32_t e = 0; e < kEach; e++) {
                    run += v[e];
                    if (v[e] > 0)
                        last = x0 + e;
                    if (v[e] > 0 && run > target && hit == ~0u)
                        hit = x0 + e;
                }
                atomicMax(&spare, last);
                if (upto > target)   // the last place where the sum by single places falls short
                    atomicMin(&found, hit != ~0u ? hit : last);
            }
            __syncthreads();
            token = (int32_t)(found != ~0u ? found : spare);
        }
    } else if (blockIdx.x % g.groups != 0) {
        return;   // one workgroup writes that there is nothing
    } else if (g.seqs != nullptr && (uint32_t)seq < g.max_seqs) {
        had = g.lens[seq];
    }
    if (thread == 0) {
        g.count[b] = w.count;
        g.token[b] = token;
        if (g.seqs != nullptr)
            g.new_lens[b] = had + w.count;
    }
    if (Q)
        __syncthreads();   // of the path's last entries, which the first wave may have written
    for (uint32_t i = thread; i < g.nodes; i += kDraw) {
        const bool real = (int32_t)i < w.count;
        if (i >= kDraw || (int32_t)i >= walked)   // not had yet
            node = real ? fresh(&g.path[row + i]) : -1;
        if (!real)
            g.path[row + i] = -1;
        if (g.seqs != nullptr) {
            g.append_seqs[row + i] = real ? seq : -1;
            g.append_positions[row + i] = real ? had + (int32_t)i : 0;
            g.append_index[row + i] = real ? (int32_t)(row + node) : 0;
        }
    }
}

static uint64_t round16(uint64_t n) { return (n + 15) / 16 * 16; }

uint64_t verify_workspace(uint32_t batch, uint32_t vocab) {
    const uint32_t stretch = stretch_of(batch, vocab);
    return round16(sizeof(Walk) * batch) + round16(4ull * batch) + round16(8ull * batch * ((vocab + stretch - 1) / stretch));
}

template <typename T>
static hipError_t launch_verify_type(const VerifyArgs &g, bool drafted, hipStream_t stream) {
    LaunchSeq seq;
    const hipError_t e = launch(drafted ? verify_walk_kernel<T, true> : verify_walk_kernel<T, false>,
            g.batch, 64, stream, nullptr, g);
    if (e != hipSuccess)
        return e;
    seq.last();
    return launch(drafted ? verify_draw_kernel<T, true> : verify_draw_kernel<T, false>, g.batch * g.groups, kDraw,
            stream, nullptr, g);
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
    g.groups = (g.stretches + kDrawWaves - 1) / kDrawWaves;
    uint8_t *ws = static_cast<uint8_t *>(v.workspace);
    g.walks = reinterpret_cast<Walk *>(ws);
    g.ended = reinterpret_cast<uint32_t *>(ws + round16(sizeof(Walk) * v.batch));
    g.sums = reinterpret_cast<double *>(ws + round16(sizeof(Walk) * v.batch) + round16(4ull * v.batch));
    switch (v.dtype) {
    case TB_BF16: return launch_verify_type<__bf16>(g, v.draft_probs != nullptr, stream);
    case TB_FP16: return launch_verify_type<_Float16>(g, v.draft_probs != nullptr, stream);
    default: return launch_verify_type<float>(g, v.draft_probs != nullptr, stream);
    }
}

}  // namespace tbk
