// tb_attention_kernels.h -- gfx950 kernels of the attention of drafted tokens over the
// paged cache.  WIN: over a window of it; FP4: over one held in 4 bits.
//
// The M = nodes * (heads_q / heads) rows of one sequence that read one
// key/value head share each of its keys, so a key costs M multiply-adds a
// byte: up to some 200 rows the cache's bytes decide, beyond that the
// products.  With up to 16 rows every key and value goes from memory straight into
// the registers of the one wave that multiplies it; with more, the waves of a
// workgroup share them through LDS.
//
// A wave owns R = 16 NT rows and walks over tiles of 32 keys with a running
// maximum and sum.  Both products run on 16x16x32 matrix instructions and are
// taken transposed, rows along the columns:
//   S' = K Q'   a lane (n = lane % 16, g = lane / 16) then holds, of row n, the
//               scores of keys 4g .. 4g+3 and 16+4g .. 16+4g+3,
//   O' = V' P'  which are just the k-places that lane has to supply of P', so
//               that the probabilities never leave their lane.  V' wants, for
//               one element of the head, the values of those eight keys in one
//               register quad.  From registers: each lane loads D/16 neighbouring
//               elements of its eight keys and pairs them up by byte permutes (the
//               order in which elements meet the instruction's rows is free: place
//               n of instruction j is element n D/16 + j).  From LDS: two
//               transposing reads of four keys each, place n being element 16 j + n.
// The statistics of row n are in the lanes with that n, as is its column of O'.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "tb_cache_internal.h"
#include "tb_fp4.h"
#include "tb_launch.h"
#include "tb_serve.h"

namespace tbk {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x3 __attribute__((ext_vector_type(3)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(1))) u32x4 gu32x4;
typedef __attribute__((address_space(1))) f32x4 gf32x4;
typedef __attribute__((address_space(1))) void gvoid;
typedef __attribute__((address_space(3))) void svoid;

constexpr int kTile = 32;              // keys of a tile
constexpr uint32_t kListPages = 2048;  // page numbers of a chunk kept in LDS
// A row's maximum is let stand until a score exceeds it by this much (in powers of
// two): weights then stay below 2^8, or 2^15 with kLift, inside every type here, and after the
// first tiles the accumulators are hardly ever scaled again.
constexpr float kSlack = 8.f;

struct AttnArgs {
    const uint8_t *q, *k, *v;
    uint8_t *out;
    float *lse;
    uint64_t q_stride[3], k_stride[3], v_stride[3], out_stride[3];   // bytes
    const int32_t *seqs;
    const uint32_t *mask;              // 32 nodes a word
    const int32_t *tree_nodes;
    const uint8_t *k_cache, *v_cache;
    const int32_t *table, *lens;
    uint32_t batch, nodes, heads_q, heads, group, rows;   // rows: nodes * group
    uint32_t page_step, token_step, head_step;            // in pieces of 16 bytes (FP4: 4), see Keys
    uint32_t num_pages, page_tokens, max_seqs, max_pages;
    uint32_t div_mul, div_shift;       // token / page_tokens = token * div_mul >> div_shift
    uint32_t row_blocks;               // workgroups that share a head's rows
    uint32_t budget;                   // shares that a head's stream of keys is cut into; 0: one for each sequence
    float scale, scale2;               // |scale| log2 e; 1 for scale 0, see load_q
    int32_t sign;                      // of scale
    int32_t *split_base, *split_count; // [batch] workspace
    float *part_ml;                    // [slots][rows][2]
    float *part_o;                     // [slots][rows][D]
    uint32_t window, sinks;            // WIN only; window 0: the whole context
    const int32_t *depths;             // [batch][nodes], or null: a chain's
};

template <typename T>
struct Mfma;
template <>
struct Mfma<__bf16> {
    typedef bf16x8 V;
    static __device__ __forceinline__ f32x4 mul(V a, V b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    // Of two pairs: the sum of the products and c.  One of a pair.
    static __device__ __forceinline__ float dot(uint32_t a, uint32_t b, float c) {
        typedef __bf16 V2 __attribute__((ext_vector_type(2)));
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(V2, a), __builtin_bit_cast(V2, b), c, false);
    }
    static __device__ __forceinline__ float number(uint32_t two, int i) {
        return __uint_as_float(i == 0 ? two << 16 : two & 0xffff0000u);
    }
    static constexpr uint32_t kExp = 0x7f80;   // exponent bits, all set where a value is not finite
    // Weights are taken times 2^kLift, numerator and denominator alike.  fp16 begins to lose bits below 2^-14 and
    // everything below 2^-25, where many small weights can still count together: seven bits are to spare above.
    static constexpr float kLift = 0.f;
};
template <>
struct Mfma<_Float16> {
    typedef f16x8 V;
    static __device__ __forceinline__ f32x4 mul(V a, V b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ float dot(uint32_t a, uint32_t b, float c) {
        typedef _Float16 V2 __attribute__((ext_vector_type(2)));
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(V2, a), __builtin_bit_cast(V2, b), c, false);
    }
    static __device__ __forceinline__ float number(uint32_t two, int i) {
        typedef _Float16 V2 __attribute__((ext_vector_type(2)));
        return (float)__builtin_bit_cast(V2, two)[i];
    }
    static constexpr uint32_t kExp = 0x7c00;
    static constexpr float kLift = 7.f;
};

// Cache policy of the keys and values: nontemporal, each is read by one workgroup (or by few, at
// the same time).  Against plain loads: 64 sequences of up to 8,191 tokens 209 us against 216, trees of 64
// nodes over up to 16,383 tokens 215 against 220.
constexpr int kStream = 2;

// N dwords at 4-byte alignment or better, as 16-byte loads and one rest.
template <int N>
__device__ __forceinline__ void load_dwords(uint32_t *r, uint64_t at) {
    typedef __attribute__((address_space(1))) u32x2 gu32x2;
    typedef uint32_t u32x3a __attribute__((ext_vector_type(3), aligned(4)));
    typedef __attribute__((address_space(1))) u32x3a gu32x3;
    if constexpr (N >= 4) {
        const u32x4 x = __builtin_nontemporal_load((const gu32x4 *)at);
        r[0] = x.x, r[1] = x.y, r[2] = x.z, r[3] = x.w;
        if constexpr (N > 4)
            load_dwords<N - 4>(r + 4, at + 16);
    } else if constexpr (N == 3) {
        const u32x3a x = *(const gu32x3 *)at;
        r[0] = x.x, r[1] = x.y, r[2] = x.z;
    } else {
        static_assert(N == 2, "dwords");
        const u32x2 x = *(const gu32x2 *)at;
        r[0] = x.x, r[1] = x.y;
    }
}

// Logarithm of the sum of exponentials, of a row's maximum and its sum of lifted weights.
template <typename T>
__device__ __forceinline__ float lse_of(float m, float l, float scale) {
    return m * scale + logf(l * (1.f / (1 << (int)Mfma<T>::kLift)));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}
// Over the lanes with the same lane % 16.
__device__ __forceinline__ float lanes_max(float x) {
    u32x2 y = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(y.x), __uint_as_float(y.y));
    y = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(y.x), __uint_as_float(y.y));
}
__device__ __forceinline__ float lanes_sum(float x) {
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

__device__ __forceinline__ int32_t uniform(int32_t x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)x); }
__device__ __forceinline__ uint64_t uniform(uint64_t x) {
    return (uint64_t)uniform((uint32_t)(x >> 32)) << 32 | uniform((uint32_t)x);
}

// x again, as a value the compiler knows nothing about: what follows from it is
// computed where it is used and not kept in registers across the loop over parts.
__device__ __forceinline__ uint32_t anew(uint32_t x) {
    asm volatile("" : "+v"(x));
    return x;
}

// Context of sequence b of the batch, its row and its drafted nodes.
struct Sequence {
    int32_t row;   // -1: none
    uint32_t context, nodes;
    __device__ __forceinline__ uint32_t special() const { return nodes; }
};
// With a window, nodes of different depths see different ends of it.  The keys that some node may not see, the
// zone of up to nodes - 1 tokens where the windows begin, are taken together with the drafted nodes, for which there
// is a mask anyway; what is left, `context` tokens that every node sees, is the sinks and what follows the
// zone, in one row: token i of it is token i of the sequence below sink_end, and i + gap from there on.
struct WindowSequence : Sequence {
    uint32_t sink_end, gap, zone;
    __device__ __forceinline__ uint32_t length() const { return context + gap; }
    __device__ __forceinline__ uint32_t zone_begin() const { return sink_end + gap - zone; }
    __device__ __forceinline__ uint32_t zone_room() const { return (zone + kTile - 1) / kTile * kTile; }
    // Places for the zone, up to whole tiles, and the nodes.
    __device__ __forceinline__ uint32_t special() const { return zone_room() + nodes; }
};
__device__ __forceinline__ uint32_t zone_of(const Sequence &) { return 0; }
__device__ __forceinline__ uint32_t zone_of(const WindowSequence &s) { return s.zone; }
template <bool WIN>
struct SequenceOf {
    typedef Sequence T;
};
template <>
struct SequenceOf<true> {
    typedef WindowSequence T;
};

template <bool WIN>
__device__ __forceinline__ typename SequenceOf<WIN>::T sequence_of(const AttnArgs &g, uint32_t b) {
    typename SequenceOf<WIN>::T s = {};
    s.row = -1;
    const int32_t q = g.seqs[b];
    if ((uint32_t)q >= g.max_seqs)
        return s;
    s.row = q;
    const int32_t n = g.lens[q], most = (int32_t)(g.max_pages * g.page_tokens);
    s.context = (uint32_t)(n < 0 ? 0 : (n < most ? n : most));
    s.nodes = g.nodes;
    if (g.tree_nodes != nullptr) {
        const int32_t x = g.tree_nodes[b];
        s.nodes = x < 0 ? 0 : min((uint32_t)x, g.nodes);
    }
    if constexpr (WIN) {
        if (g.window != 0) {
            // the root's window begins at n + 1 - window, that of the greatest depth nodes - 1 tokens later
            const uint32_t all = s.context, first = all + 1 > g.window ? all + 1 - g.window : 0;
            s.sink_end = min(g.sinks, all);
            const uint32_t lo = max(first, s.sink_end);
            const uint32_t last = all + s.nodes > g.window ? all + s.nodes - g.window : 0;
            s.zone = last > lo ? min(last, all) - lo : 0;
            s.gap = lo + s.zone - s.sink_end;
            s.context = all - s.gap;
        }
    }
    return s;
}

// The batch's keys as one stream: each sequence's context and nodes, rounded up to kUnit
// keys, and some units more for what a sequence costs by itself, one after the other.  It is cut into equal shares,
// one for each of the workgroups that a head's rows have, so that they all end together
// however the lengths differ.  A share may cover parts of several sequences.
// Every workgroup finds its place by itself (a few loads and a sum over the
// batch): nothing is planned before the launch and the lengths stay on the device.
constexpr uint32_t kUnit = 128;
// What a sequence costs by itself, a dozen latencies, in units of its keys: of 4 bits they take a quarter of the time.
// 64 sequences of up to 8,191 tokens in 4 bits with one unit 73 us, with three 65.5, five 64.5, eight 65.5.
constexpr uint32_t own_units(bool fp4) { return fp4 ? 4 : 1; }
template <bool FP4, typename Seq>
__device__ __forceinline__ uint32_t weight_of(const Seq &s) {
    return ((s.context + s.special() + kUnit - 1) / kUnit + own_units(FP4)) * kUnit;
}

constexpr uint64_t kWhole = 1ull << 40;   // a share longer than any sequence
struct Place {
    uint64_t start;   // of sequence `batch` in the stream
    uint64_t share;
    uint32_t batch;   // the sequence in which the share begins; g.batch: no share
};

// `known`: LDS for a sequence a thread; filled where the batch has no more than that.
template <int WAVES, bool WIN, bool FP4>
__device__ __forceinline__ void find_place(const AttnArgs &g, uint32_t mine, Place *out, uint64_t *lds,
        typename SequenceOf<WIN>::T *known) {
    if (g.budget == 0) {   // one sequence, from its first key to its last
        if (threadIdx.x == 0)
            *out = {0, kWhole, mine};
        __syncthreads();
        return;
    }
    const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6;
    uint64_t total = 0, w = 0;
    for (uint32_t b0 = 0; b0 < g.batch; b0 += 64 * WAVES) {
        w = 0;
        if (b0 + t < g.batch) {
            const auto q = sequence_of<WIN>(g, b0 + t);
            known[t] = q;
            w = weight_of<FP4>(q);
        }
        total += w;
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        total += __shfl_xor(total, d);
    if (lane == 0)
        lds[wave] = total;
    if (t == 0)
        out->batch = g.batch;
    __syncthreads();
    total = 0;
    for (int k = 0; k < WAVES; k++)
        total += lds[k];
    const uint64_t share = units_of_share(total / kUnit, g.budget) * kUnit;
    const uint64_t begin = mine * share;
    uint64_t before = 0;
    for (uint32_t b0 = 0; b0 < g.batch; b0 += 64 * WAVES) {
        if (g.batch > 64 * WAVES)
            w = b0 + t < g.batch ? weight_of<FP4>(sequence_of<WIN>(g, b0 + t)) : 0;
        uint64_t x = w;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint64_t y = __shfl_up(x, d);
            if (lane >= (uint32_t)d)
                x += y;
        }
        __syncthreads();
        if (lane == 63)
            lds[wave] = x;
        __syncthreads();
        uint64_t start = before + x - w;
        for (uint32_t k = 0; k < WAVES; k++) {
            start += k < wave ? lds[k] : 0;
            before += lds[k];
        }
        if (begin >= start && begin < start + w) {
            out->batch = b0 + t;
            out->start = start;
            out->share = share;
        }
    }
    __syncthreads();
}

// What a workgroup does of one sequence: the part [c0, c1) of its context and, if
// `last`, its nodes.  Shares of one sequence are joined afterwards, from slot
// (workgroup + sequence), unless there is only one.
template <bool WIN, bool FP4>
struct Part {
    typedef typename SequenceOf<WIN>::T Seq;
    Seq seq;
    uint32_t b, c0, c1, slot, splits;
    uint64_t end;       // of the sequence in the stream
    bool first, last;

    // known: what find_place() left, for up to `room` sequences
    __device__ __forceinline__ Part(const AttnArgs &g, const Place &at, uint32_t mine, const Seq *known,
            uint32_t room) : b(at.batch) {
        const Seq s = g.batch <= room && at.share != kWhole ? known[b] : sequence_of<WIN>(g, b);
        seq.row = uniform(s.row);
        seq.context = uniform(s.context);
        seq.nodes = uniform(s.nodes);
        if constexpr (WIN) {
            seq.sink_end = uniform(s.sink_end);
            seq.gap = uniform(s.gap);
            seq.zone = uniform(s.zone);
        }
        end = at.start + weight_of<FP4>(seq);
        if (at.share == kWhole) {
            c0 = slot = 0;
            c1 = seq.context;
            splits = 1;
            first = last = true;
            end = ~0ull;   // no other sequence follows
            return;
        }
        const uint64_t begin = mine * at.share;
        const uint64_t lo = begin > at.start ? begin - at.start : 0;
        const uint64_t hi = min(begin + at.share, end) - at.start;
        c0 = (uint32_t)min(lo, (uint64_t)seq.context);
        c1 = (uint32_t)min(hi, (uint64_t)seq.context);
        last = at.start + hi == end;
        first = begin <= at.start;
        if (first && last) {
            splits = 1;
        } else {
            const uint64_t u = at.share / kUnit, a = at.start / kUnit, z = end / kUnit - 1;
            splits = uniform(z <= 0xffffffffu ? (uint32_t)z / (uint32_t)u - (uint32_t)a / (uint32_t)u + 1
                    : (uint32_t)(z / u - a / u + 1));
        }
        slot = mine + b;
    }
};

// Where the part's keys are.
template <int WAVES, bool WIN, bool FP4>
struct Keys {
    const AttnArgs &g;
    typename SequenceOf<WIN>::T seq;
    uint32_t b, head, count, p0;
    uint32_t p1;    // WIN: likewise of the tokens past the sinks, less the places that the sinks' pages take in the list
    bool listed;
    const int32_t *row_table;
    const uint32_t *list;
    static constexpr uint32_t kPiece = FP4 ? 4 : 16;

    // Places in a pool count pieces of 16 bytes (FP4: 4): 32 bits reach 64 GiB (16), and the address costs one
    // instruction.
    __device__ __forceinline__ Keys(const AttnArgs &g_, const Part<WIN, FP4> &part, uint32_t head_, uint32_t *lds)
        : g(g_), seq(part.seq), b(part.b), head(head_), count(part.seq.nodes), p1(0), list(lds) {
        row_table = g.table + (uint64_t)max(part.seq.row, 0) * g.max_pages;
        p0 = page_of(part.c0);
        if constexpr (WIN) {
            // two runs of pages: of the sinks, and of what follows the gap
            const uint32_t border = min(max(seq.sink_end, part.c0), part.c1);
            const uint32_t before = border > part.c0 ? page_of(border - 1) - p0 + 1 : 0;
            const uint32_t begin = page_of(border + seq.gap);
            const uint32_t pages = before + (part.c1 > border ? page_of(part.c1 - 1 + seq.gap) - begin + 1 : 0);
            p1 = begin - before;
            listed = pages <= kListPages;
            if (listed)
                for (uint32_t i = threadIdx.x; i < pages; i += 64 * WAVES)
                    lds[i] = checked(i < before ? p0 + i : p1 + i);
        } else {
            const uint32_t pages = part.c1 > part.c0 ? page_of(part.c1 - 1) - p0 + 1 : 0;
            listed = pages <= kListPages;
            if (listed)
                for (uint32_t i = threadIdx.x; i < pages; i += 64 * WAVES)
                    lds[i] = checked(p0 + i);
        }
    }
    // Place of the row's p-th page, a number out of range being that of page 0.
    __device__ __forceinline__ uint32_t checked(uint32_t p) const {
        const uint32_t page = (uint32_t)row_table[p];
        return (page < g.num_pages ? page : 0) * g.page_step;
    }
    __device__ __forceinline__ uint32_t page_of(uint32_t token) const {
        return (uint32_t)(((uint64_t)token * g.div_mul) >> g.div_shift);
    }
    // Place of a context token's head in its pool.
    __device__ __forceinline__ uint32_t place_of(uint32_t token) const {
        if constexpr (WIN) {
            const bool past = token >= seq.sink_end;
            const uint32_t real = token + (past ? seq.gap : 0), p = page_of(real), in_page = real - p * g.page_tokens;
            const uint32_t at = listed ? list[p - (past ? p1 : p0)] : checked(p);
            return at + in_page * g.token_step + head * g.head_step;
        } else {
            const uint32_t p = page_of(token), in_page = token - p * g.page_tokens;
            const uint32_t at = listed ? list[p - p0] : checked(p);
            return at + in_page * g.token_step + head * g.head_step;
        }
    }
    __device__ __forceinline__ uint64_t offset_of(uint32_t token) const { return (uint64_t)place_of(token) * kPiece; }
    // The same of the u-th token of the zone, whose pages are in no list.
    __device__ __forceinline__ uint64_t offset_in_zone(uint32_t u) const {
        const uint32_t real = seq.zone_begin() + u, p = page_of(real), in_page = real - p * g.page_tokens;
        return (uint64_t)(checked(p) + in_page * g.token_step + head * g.head_step) * kPiece;
    }
    __device__ __forceinline__ uint32_t depth_of(uint32_t node) const {
        if (g.depths == nullptr)
            return node;
        const int32_t d = g.depths[(uint64_t)b * g.nodes + node];
        return d < 0 ? 0 : min((uint32_t)d, count - 1);
    }
    // Bits of the nodes first .. first + 31 that row r sees; there is a node.
    __device__ __forceinline__ uint32_t seen(uint32_t r, uint32_t first) const {
        const uint32_t words = (g.nodes + 63) / 64 * 2, node = min(r, g.rows - 1) / g.group;
        uint32_t bits;
        if (g.mask != nullptr)
            bits = g.mask[((uint64_t)b * g.nodes + node) * words + first / 32];
        else
            bits = node < first ? 0u : (node >= first + 31 ? 0xffffffffu : (2u << (node - first)) - 1);
        bits = count < first + 32 ? bits & ((1u << (count - first)) - 1) : bits;
        if constexpr (WIN)
            if (g.window != 0 && g.window < count) {   // a window shorter than a path can be
                const uint32_t depth = depth_of(min(node, count - 1));
                for (uint32_t left = bits; left != 0; left &= left - 1) {
                    const uint32_t u = __builtin_ctz(left), d = depth_of(first + u);
                    if (depth >= d + g.window && seq.length() + d >= g.sinks)
                        bits &= ~(1u << u);
                }
            }
        return bits;
    }
    // Bits of the zone's tokens first .. first + 31 that row r sees.
    __device__ __forceinline__ uint32_t seen_in_zone(uint32_t r, uint32_t first) const {
        const uint32_t node = min(min(r, g.rows - 1) / g.group, count - 1);
        // what the row's window begins at, from the zone's begin
        const int64_t from = (int64_t)seq.length() + depth_of(node) + 1 - g.window - seq.zone_begin() - first;
        const uint32_t bits = from <= 0 ? 0xffffffffu : (from >= 32 ? 0 : 0xffffffffu << from);
        return seq.zone < first + 32 ? bits & ((1u << (seq.zone - first)) - 1) : bits;
    }
};

// A dword of two values, those that are not finite replaced by 0; *wild becomes nonzero then.
template <typename T>
__device__ __forceinline__ uint32_t tamed(uint32_t x, uint32_t *wild) {
    const bool lo = (x & Mfma<T>::kExp) == Mfma<T>::kExp, hi = (x >> 16 & Mfma<T>::kExp) == Mfma<T>::kExp;
    *wild |= (uint32_t)(lo || hi);
    return x & (lo ? 0xffff0000u : 0xffffffffu) & (hi ? 0x0000ffffu : 0xffffffffu);
}

// Key of the tile that is the i-th of lane group q4.
__device__ __forceinline__ uint32_t key_of(uint32_t q4, int i) { return (i < 4 ? 0 : 12) + 4 * q4 + i; }

// The rows of one wave, 16 NT of them from row0 on, and what has been summed up for them.
// RUNS: each lane group has a quarter of the head in one run; else, of every 32 elements a quarter.
template <typename T, int D, int NT, bool RUNS>
struct Rows {
    typedef typename Mfma<T>::V V8;
    static constexpr int KS = D / 32;   // steps of the first product
    static constexpr int DJ = D / 16;   // instructions of the second one
    static constexpr int GJ = DJ % 4 == 0 ? 4 : 2;   // of them, whose operands are had together
    static constexpr int kRegs = NT * DJ * 4;
    static constexpr int kMergeFloats = 64 * (kRegs + 2 * NT);   // of one wave, see join()
    V8 q[NT][KS];
    // Where in a head of 16 bits a lane group's 16 bytes of step s are: at lane_at(q4) + s * kStepBytes.
    static constexpr int kStepBytes = RUNS ? 16 : 64;
    static __device__ __forceinline__ uint32_t lane_at(uint32_t q4) { return q4 * (RUNS ? D / 2 : 16); }
    f32x4 o[NT][DJ];
    float m[NT], l[NT];                 // l: this lane's keys only, until join()
    float base[NT];                     // of the exponents: m scaled, less the lift; any while m is -inf

    // Row r is node r / group of query head head * group + r % group.
    __device__ __forceinline__ void open(const AttnArgs &g, uint32_t b, uint32_t head, uint32_t row0, uint32_t lane) {
        const uint32_t n = lane & 15, q4 = lane >> 4;
#pragma unroll
        for (int t = 0; t < NT; t++) {
            const uint32_t r = row0 + t * 16 + n, node = r / g.group, h = head * g.group + r % g.group;
            const uint64_t at = reinterpret_cast<uint64_t>(g.q) + b * g.q_stride[0] + node * g.q_stride[1] +
                                h * g.q_stride[2] + lane_at(q4);
#pragma unroll
            for (int s = 0; s < KS; s++) {
                u32x4 x = {0, 0, 0, 0};
                if (r < g.rows && g.sign != 0)
                    x = *(const gu32x4 *)(at + s * kStepBytes);
                if (g.sign < 0)   // a negative scale: the sign goes to q, exactly
                    x ^= 0x80008000u;
                q[t][s] = __builtin_bit_cast(V8, x);
            }
            m[t] = -INFINITY;
            l[t] = base[t] = 0.f;
#pragma unroll
            for (int j = 0; j < DJ; j++)
                o[t][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
        }
    }

    // Raises the maxima to what the lanes saw, and scales what has been summed up.
    __device__ __forceinline__ void raise_maxima(const AttnArgs &g, const float *tops) {
#pragma unroll
        for (int t = 0; t < NT; t++) {
            const float top = fmaxf(lanes_max(tops[t]), m[t]);
            const float to = top == -INFINITY ? 0.f : top * g.scale2;
            base[t] = to - Mfma<T>::kLift;
            // a row's first keys: m = -inf, the factor 0 meets sums that are 0
            const float fade = __builtin_amdgcn_exp2f(__builtin_fmaf(m[t], g.scale2, -to));
            m[t] = top;
            l[t] *= fade;
#pragma unroll
            for (int j = 0; j < DJ; j++)
                o[t][j] *= fade;
        }
    }

    // A tile is worked on in two halves, scores() and apply().  Where scores() says so, the
    // maxima have to be raised in between, which is rare.
    //
    // keys(k, x): x[2 e + z] becomes step k + e's operand for keys 16 z .. 16 z + 15, e and z 0 and 1;
    // keep(t, i): whether row t * 16 + n sees the lane's i-th key, asked only if `some` row may not see all (MASKED: always).
    template <bool MASKED, typename Keys2, typename Keep>
    __device__ __forceinline__ bool scores(const AttnArgs &g, bool some, Keys2 keys, Keep keep, f32x4 (&s)[NT][2],
            float (&tops)[NT]) {
#pragma unroll
        for (int t = 0; t < NT; t++)
            s[t][0] = s[t][1] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < KS; k += 2) {
            V8 x[4];
            keys(k, x);
#pragma unroll
            for (int e = 0; e < 2 && k + e < KS; e++)
#pragma unroll
                for (int z = 0; z < 2; z++)
#pragma unroll
                    for (int t = 0; t < NT; t++)
                        s[t][z] = Mfma<T>::mul(x[2 * e + z], q[t][k + e], s[t][z]);
        }
        // The results may be read 8 states after the last product.  The compiler counts them on the way through the branch below
        // and not on the way past it.  With NT 1 it left 2 to 6 there, and now and then what the registers had before came out;
        // with NT 2 it leaves enough only by the order of its reads.  So all results are tied to the wait: trees of 64
        // nodes take 1 % longer over 4 bits, those of 8 nodes 1 % less, a chain of 1,024 over a window of 256 3 % longer, the
        // others what they took.  MASKED has no branch (trees over windows 61.3 us against 61.9 with the wait there as well).
        if constexpr (MASKED)
            some = true;
        else if constexpr (NT == 1)
            asm volatile("s_nop 7" : "+v"(s[0][0]), "+v"(s[0][1]));
        else
            asm volatile("s_nop 7" : "+v"(s[0][0]), "+v"(s[0][1]), "+v"(s[1][0]), "+v"(s[1][1]));
        static_assert(NT <= 2, "the wait names each result");
        if (some) {
#pragma unroll
            for (int t = 0; t < NT; t++)
#pragma unroll
                for (int i = 0; i < 8; i++)
                    s[t][i / 4][i % 4] = keep(t, i) ? s[t][i / 4][i % 4] : -INFINITY;
        }
        bool above = false;
#pragma unroll
        for (int t = 0; t < NT; t++) {
            // a NaN among the scores stays one: the row is NaN then, whatever its maximum
            tops[t] = max3(max3(s[t][0][0], s[t][0][1], s[t][0][2]), max3(s[t][0][3], s[t][1][0], s[t][1][1]),
                           __builtin_elementwise_maximum(s[t][1][2], s[t][1][3]));
            above |= tops[t] * g.scale2 > __builtin_fmaf(m[t], g.scale2, kSlack);
        }
        return __any(above);
    }

    // values(j, x): x[0 .. GJ - 1] become the operands of the second product's instructions j on.
    template <typename Values>
    __device__ __forceinline__ void apply(const AttnArgs &g, const f32x4 (&s)[NT][2], Values values) {
        V8 p[NT];
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][i / 4][i % 4], g.scale2, -base[t]));
                l[t] += e;
                // rounded to the element type, which is what the matrix instruction takes; the sum keeps all bits
                p[t][i] = (T)e;
            }
#pragma unroll
        for (int j = 0; j < DJ; j += GJ) {
            V8 x[GJ];
            values(j, x);
#pragma unroll
            for (int e = 0; e < GJ; e++)
#pragma unroll
                for (int t = 0; t < NT; t++)
                    o[t][j + e] = Mfma<T>::mul(x[e], p[t], o[t][j + e]);
        }
    }

    // Adds the values that tamed() left out to the rows that see them; value(u, e): element e of the values of
    // key u; element(j, r): which element of the head o[t][j][r] is.
    template <typename Value, typename Element>
    __device__ __forceinline__ void add_wild(Value value, uint32_t first, uint32_t end, const uint32_t *bits,
            Element element) {
        for (uint32_t u = first; u < end; u++) {
#pragma unroll
            for (int j = 0; j < DJ; j++) {
                // rare: a few loads at a time, so that this does not decide the kernel's registers
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    const float x = value(u, element(j, r));
                    if (!(fabsf(x) < INFINITY)) {
#pragma unroll
                        for (int t = 0; t < NT; t++)
                            o[t][j][r] += bits[t] >> (u - first) & 1 ? x : 0.f;   // any weight of it gives the same
                    }
                }
            }
        }
    }

    // Joins the WK waves (wave = wk * WM + wm) that divided the keys of the same rows; the
    // result is in those with wk = 0.  lds: WM * WK / 2 * kMergeFloats floats.
    template <int WM, int WK>
    __device__ __forceinline__ void join(const AttnArgs &g, float *lds, uint32_t wave, uint32_t lane) {
        const uint32_t wm = wave % WM, wk = wave / WM;
#pragma unroll
        for (int t = 0; t < NT; t++)
            l[t] = lanes_sum(l[t]);
#pragma unroll
        for (int half = WK / 2; half > 0; half /= 2) {
            if (wk >= (uint32_t)half && wk < (uint32_t)(2 * half)) {
                float *at = lds + ((wk - half) * WM + wm) * kMergeFloats + lane;
#pragma unroll
                for (int t = 0; t < NT; t++) {
                    at[t * 128] = m[t];
                    at[t * 128 + 64] = l[t];
#pragma unroll
                    for (int j = 0; j < DJ; j++)
#pragma unroll
                        for (int r = 0; r < 4; r++)
                            at[64 * (2 * NT + (t * DJ + j) * 4 + r)] = o[t][j][r];
                }
            }
            __syncthreads();
            if (wk < (uint32_t)half) {
                const float *at = lds + (wk * WM + wm) * kMergeFloats + lane;
#pragma unroll
                for (int t = 0; t < NT; t++) {
                    const float m2 = at[t * 128], top = fmaxf(m[t], m2), base = top == -INFINITY ? 0.f : top * g.scale2;
                    const float f1 = __builtin_amdgcn_exp2f(__builtin_fmaf(m[t], g.scale2, -base));
                    const float f2 = __builtin_amdgcn_exp2f(__builtin_fmaf(m2, g.scale2, -base));
                    m[t] = top;
                    l[t] = l[t] * f1 + at[t * 128 + 64] * f2;
#pragma unroll
                    for (int j = 0; j < DJ; j++)
#pragma unroll
                        for (int r = 0; r < 4; r++)
                            o[t][j][r] = o[t][j][r] * f1 + at[64 * (2 * NT + (t * DJ + j) * 4 + r)] * f2;
                }
            }
            __syncthreads();
        }
    }

    // Writes the rows: the result where the sequence is one chunk, else the chunk's share.
    // Each lane holds, of row n, runs of RUN neighbouring elements: run i begins at element
    // begin(i), and its element e is value(t, i, e).
    template <int RUN, typename PartT, typename Begin, typename Value>
    __device__ __forceinline__ void close(const AttnArgs &g, const PartT &w, uint32_t head, uint32_t row0,
            uint32_t lane, Begin begin, Value value) {
        constexpr int kRuns = 4 * DJ / RUN;
        typedef T tv __attribute__((ext_vector_type(RUN)));
        const uint32_t n = lane & 15, q4 = lane >> 4;
#pragma unroll
        for (int t = 0; t < NT; t++) {
            const uint32_t r = row0 + t * 16 + n;
            if (r >= g.rows)
                continue;
            const uint32_t node = r / g.group, h = head * g.group + r % g.group;
            if (w.splits > 1) {
                const uint64_t at = ((uint64_t)w.slot * g.heads + head) * g.rows + r;
                if (q4 == 0) {
                    g.part_ml[2 * at] = m[t];
                    g.part_ml[2 * at + 1] = l[t];
                }
#pragma unroll
                for (int i = 0; i < kRuns; i++) {
                    gf32x4 *to = (gf32x4 *)(reinterpret_cast<uint64_t>(g.part_o) + (at * D + begin(i)) * 4);
#pragma unroll
                    for (int e = 0; e < RUN; e += 4)
                        to[e / 4] = (f32x4){value(t, i, e), value(t, i, e + 1), value(t, i, e + 2), value(t, i, e + 3)};
                }
                continue;
            }
            const bool empty = l[t] == 0.f || node >= w.seq.nodes;
            const float inv = empty ? 0.f : 1.f / l[t];
            const uint64_t to = reinterpret_cast<uint64_t>(g.out) + w.b * g.out_stride[0] +
                                node * g.out_stride[1] + h * g.out_stride[2];
#pragma unroll
            for (int i = 0; i < kRuns; i++) {
                tv x;
#pragma unroll
                for (int e = 0; e < RUN; e++)
                    x[e] = (T)(empty ? 0.f : value(t, i, e) * inv);
                typedef __attribute__((address_space(1))) tv gtv;
                *(gtv *)(to + begin(i) * 2) = x;
            }
            if (g.lse != nullptr && q4 == 0)
                g.lse[((uint64_t)w.b * g.nodes + node) * g.heads_q + h] =
                    empty ? -INFINITY : lse_of<T>(m[t], l[t], g.scale);
        }
    }
};

// The combine kernel's way into the slots.
template <typename PartT>
__device__ __forceinline__ void note_splits(const AttnArgs &g, const PartT &w, uint32_t head, uint32_t block) {
    if (g.budget != 0 && block == 0 && head == 0 && w.first && threadIdx.x == 0) {
        g.split_base[w.b] = (int32_t)w.slot;
        g.split_count[w.b] = (int32_t)w.splits;
    }
}

// ---- few rows ------------------------------------------------------------------
//
// Up to 16 rows: the cache's bytes decide.  Each of the four waves
// takes every fourth tile and reads its keys and values straight into the registers
// from which they are multiplied; the next tile's keys are on their way during the
// second product, its values during the first.
//
// 64 sequences of up to 8,191 tokens, 8 heads of 128, 4 rows a head: 1.09 GB of keys and values in 208 us,
// 5.2 TB/s, where a large copy reaches 6.5 TB/s; every request to memory is of 128 bytes and nothing is read
// twice.  Pages by token spread a head over slices of 256 bytes, and two heads of the eight take 175 us
// for theirs where the others take 139, on whichever XCD they run: memory channels, which pages by head
// (200 us) meet less.  Three waves a SIMD instead of two spill at D = 128 (372 us); more shares, and heads in
// another order, gain nothing.  A short part is its latencies one after the other, some 10 us: lengths,
// page numbers, first keys, the join of the waves.
constexpr int kWaves = 4;

// Where the context's keys and values of a wave's next tile wait in registers, and how they become operands.  16 bits:
// kr[z][s] is step s's operand for keys 16 z .. 16 z + 15, vr[i] this lane's D / 16 neighbouring elements of its i-th key.
template <typename T, int D, bool FP4>
struct Held {
    static constexpr int KS = D / 32, DJ = D / 16;
    uint32_t kr[2][KS][4], vr[8][DJ / 2];

    __device__ __forceinline__ void load_k(uint64_t at0, uint64_t at1, uint32_t q4) {
#pragma unroll
        for (int s = 0; s < KS; s++) {
            load_dwords<4>(kr[0][s], at0 + s * 64 + q4 * 16);
            load_dwords<4>(kr[1][s], at1 + s * 64 + q4 * 16);
        }
    }
    __device__ __forceinline__ void load_v(int i, uint64_t at, uint32_t n) {
        load_dwords<DJ / 2>(vr[i], at + n * (2 * DJ));
    }
    __device__ __forceinline__ void clear_v(int i, bool keep) {
#pragma unroll
        for (int j = 0; j < DJ / 2; j++)
            vr[i][j] = keep ? vr[i][j] : 0;
    }
    __device__ __forceinline__ u32x4 key(int z, int s, uint32_t) const {
        return (u32x4){kr[z][s][0], kr[z][s][1], kr[z][s][2], kr[z][s][3]};
    }
    __device__ __forceinline__ uint32_t value(int i, int j, uint32_t) const { return vr[i][j]; }   // elements 2j, 2j + 1
};
// 4 bits: the codes and the powers, 9 and 16 registers for 128 elements where 16 bits take 64.  They are converted where
// they are used.
template <typename T, int D>
struct Held<T, D, true> {
    static constexpr int DJ = D / 16, kWords = D / 32;   // of a key's quarter
    static constexpr int kPowers = (D / 32 + 3) / 4;      // words of powers
    uint32_t kr[2][kWords], kp[2][kPowers], vr[8][D == 256 ? 2 : 1], vp[8];

    __device__ __forceinline__ void load_k(uint64_t at0, uint64_t at1, uint32_t q4) {
        load_words<kWords>(kr[0], at0 + q4 * (D / 8));
        load_words<kWords>(kr[1], at1 + q4 * (D / 8));
        load_words<kPowers>(kp[0], at0 + D / 2);
        load_words<kPowers>(kp[1], at1 + D / 2);
    }
    // Powers: of 96 elements a lane's six may belong to two blocks; else it has one.
    __device__ __forceinline__ void load_v(int i, uint64_t at, uint32_t n) {
        typedef uint32_t u32u __attribute__((aligned(1)));
        typedef uint16_t u16u __attribute__((aligned(1)));
        typedef __attribute__((address_space(1))) u32u gu32u;
        typedef __attribute__((address_space(1))) u16u gu16u;
        typedef __attribute__((address_space(1))) uint8_t gu8;
        const uint64_t from = at + n * (DJ / 2);
        if constexpr (D == 256)
            load_words<2>(vr[i], from);
        else if constexpr (D == 64)
            vr[i][0] = *(const gu16u *)from;
        else
            vr[i][0] = *(const gu32u *)from;   // of 96: a byte more than is used, still of the head
        if constexpr (D == 96)
            load_words<1>(&vp[i], at + D / 2);
        else
            vp[i] = *(const gu8 *)(at + D / 2 + n * DJ / 32);
    }
    __device__ __forceinline__ void clear_v(int i, bool keep) {   // 0 times 2^-127
        vr[i][0] = keep ? vr[i][0] : 0;
        if constexpr (D == 256)
            vr[i][1] = keep ? vr[i][1] : 0;
        vp[i] = keep ? vp[i] : 0;
    }
    __device__ __forceinline__ u32x4 key(int z, int s, uint32_t q4) const {
        const uint32_t block = (q4 * (D / 4) + 8 * s) / 32;
        const uint32_t powers = kPowers == 2 && block >= 4 ? kp[z][kPowers - 1] : kp[z][0];
        return eight_of<T>(kr[z][s], power_of(powers, block % 4));
    }
    __device__ __forceinline__ uint32_t value(int i, int j, uint32_t n) const {
        const float power = power_of(vp[i], D == 96 ? (n * DJ + 2 * j) / 32 : 0);
        return two_at<T>(vr[i][D == 256 ? j / 4 : 0], j % 4, power);
    }
};

// The zone's keys and the drafted nodes one by one, every fourth a wave's: for the kernel over a cache in 4 bits, whose rows
// see few of either (up to 16 nodes, and 15 tokens of the zone), and whose registers the tiles' way (both operands in 16 bits,
// values that are not finite apart) would decide.
// A lane has, of row n, elements q4 D / 4 on of key and values alike.
template <typename T, int D, typename R, typename K, typename Seq>
__device__ __forceinline__ void single_keys(const AttnArgs &g, const K &keys, const Seq &seq, R &rows, uint64_t kb,
        uint64_t vb, uint32_t wk, uint32_t n, uint32_t q4) {
    constexpr int KS = D / 32, DJ = D / 16;
    // the lane's quarter of a head, in 16 bits or in the cache
    const auto quarter = [&](bool in_zone, uint64_t row, u32x4 *x) {
#pragma unroll
        for (int s = 0; s < KS; s++) {
            if (in_zone) {
                uint32_t code;
                load_words<1>(&code, row + q4 * (D / 8) + s * 4);
                const uint8_t p = *reinterpret_cast<const uint8_t *>(row + D / 2 + (q4 * (D / 4) + 8 * s) / 32);
                x[s] = eight_of<T>(code, power_of(p, 0));
            } else {
                x[s] = *(const gu32x4 *)(row + R::lane_at(q4) + s * R::kStepBytes);
            }
        }
    };
#pragma unroll 1
    for (uint32_t at = wk; at < seq.zone + keys.count; at += kWaves) {
        const bool in_zone = at < seq.zone;
        const uint32_t u = in_zone ? at : at - seq.zone;
        uint64_t key = kb + u * g.k_stride[1], values = vb + u * g.v_stride[1];
        if (in_zone) {
            const uint64_t offset = keys.offset_in_zone(u);
            key = reinterpret_cast<uint64_t>(g.k_cache) + offset;
            values = reinterpret_cast<uint64_t>(g.v_cache) + offset;
        }
        u32x4 k[KS], v[KS];
        quarter(in_zone, key, k);
        quarter(in_zone, values, v);
        const uint32_t bits = in_zone ? keys.seen_in_zone(n, u & ~31u) : keys.seen(n, u & ~31u);
        const bool sees = bits >> (u & 31) & 1;
        float score = 0;
#pragma unroll
        for (int s = 0; s < KS; s++) {
            const u32x4 q = __builtin_bit_cast(u32x4, rows.q[0][s]);
#pragma unroll
            for (int e = 0; e < 4; e++)
                score = Mfma<T>::dot(q[e], k[s][e], score);
        }
        score = lanes_sum(score);
        const float top = sees ? score : -INFINITY;
        if (__any(top * g.scale2 > __builtin_fmaf(rows.m[0], g.scale2, kSlack)))
            rows.raise_maxima(g, &top);
        const float weight = sees ? __builtin_amdgcn_exp2f(__builtin_fmaf(score, g.scale2, -rows.base[0])) : 0.f;
        rows.l[0] += q4 == 0 ? weight : 0.f;
#pragma unroll
        for (int e = 0; e < D / 4; e++) {   // not seen: 0 times 0
            const uint32_t two = sees ? v[e / 8][e % 8 / 2] : 0;
            rows.o[0][e % DJ][e / DJ] =
                __builtin_fmaf(weight, Mfma<T>::number(two, e % 2), rows.o[0][e % DJ][e / DJ]);
        }
    }
}

// Workgroups of the kernel for few rows that a CU holds, by the registers it is built with.  In 4 bits three of 128
// elements, or two of 256, fit with spills in the loop, and take 68 us against 67, and 168 against 136 (64 sequences of up
// to 8,191 tokens).
constexpr int few_resident(int head_dim) { return head_dim == 64 ? 3 : (head_dim <= 128 ? 2 : 1); }

template <typename T, int D, bool WIN, bool FP4>
__global__ __launch_bounds__(64 * kWaves, few_resident(D)) void tree_attention_kernel(AttnArgs g) {
    constexpr int NT = 1;
    typedef Rows<T, D, NT, FP4> R;
    typedef typename R::V8 V8;
    typedef typename SequenceOf<WIN>::T Seq;
    constexpr int KS = R::KS, DJ = R::DJ;
    __shared__ Place place;
    __shared__ Seq known[64 * kWaves];
    __shared__ uint64_t sums[kWaves];
    __shared__ uint32_t list[kListPages];
    __shared__ float merge[kWaves / 2 * R::kMergeFloats];
    __shared__ __attribute__((aligned(16))) uint32_t spots[kWaves][WIN || FP4 ? kTile : 4];   // of a wave's next tile

    const uint32_t wk = uniform(threadIdx.x >> 6);
    uint32_t mine = blockIdx.x / g.heads, head = blockIdx.x % g.heads;
    if constexpr (FP4) {
        // Pages by token: all heads of a share run on one XCD at about the same time, as their rows are neighbours of
        // less than a line each.  64 sequences of up to 8,191 tokens 124 us to 87; pages by head 67, this way 70.
        if (g.head_step < g.token_step) {
            head = blockIdx.x / 8 % g.heads;
            mine = blockIdx.x / 8 / g.heads * 8 + blockIdx.x % 8;
        }
        if (mine >= (g.budget != 0 ? g.budget : g.batch))
            return;
    }
    find_place<kWaves, WIN, FP4>(g, mine, &place, sums, known);
    Place at = {uniform(place.start), uniform(place.share), uniform(place.batch)};
#pragma unroll 1
    for (uint64_t end = at.share == kWhole ? kWhole : (mine + 1) * at.share; at.batch < g.batch && at.start < end;
            at.batch++) {
        const uint32_t thread = anew(threadIdx.x), lane = thread & 63, n = lane & 15, q4 = lane >> 4;
        const Part<WIN, FP4> w(g, at, mine, known, 64 * kWaves);
        at.start = w.end;
        note_splits(g, w, head, 0);
        R rows;
        if constexpr (FP4)   // on its way while the pages are read
            rows.open(g, w.b, head, 0, lane);
        const Keys<kWaves, WIN, FP4> keys(g, w, head, list);
        const uint32_t c0 = w.c0, c1 = w.c1;
        if constexpr (!FP4)
            rows.open(g, keys.b, head, 0, lane);
        __syncthreads();

        const uint64_t k_pool = reinterpret_cast<uint64_t>(g.k_cache), v_pool = reinterpret_cast<uint64_t>(g.v_cache);
        Held<T, D, FP4> held;
        // Tokens first .. first + 31, those past the chunk its last one.  Where finding a place counts, each lane finds
        // that of token first + lane % 32, and all have them from LDS: ten times some 15 instructions of a tile become once.
        constexpr bool kShare = WIN || FP4;
        const auto find = [&](uint32_t first) {
            if constexpr (kShare) {
                spots[wk][lane & 31] = keys.place_of(min(first + (lane & 31), c1 - 1));
                // the wave's own, in order: only the compiler has to be told
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            }
        };
        const auto load_ctx_k = [&](uint32_t first) {
            if constexpr (kShare)
                held.load_k(k_pool + (uint64_t)spots[wk][n] * keys.kPiece,
                        k_pool + (uint64_t)spots[wk][16 + n] * keys.kPiece, q4);
            else
                held.load_k(k_pool + keys.offset_of(min(first + n, c1 - 1)),
                        k_pool + keys.offset_of(min(first + 16 + n, c1 - 1)), q4);
        };
        const auto load_ctx_v = [&](uint32_t first) {
            if constexpr (kShare) {
                const u32x4 at0 = *reinterpret_cast<const u32x4 *>(&spots[wk][key_of(q4, 0)]),
                            at1 = *reinterpret_cast<const u32x4 *>(&spots[wk][key_of(q4, 4)]);
#pragma unroll
                for (int i = 0; i < 8; i++)
                    held.load_v(i, v_pool + (uint64_t)(i < 4 ? at0[i] : at1[i - 4]) * keys.kPiece, n);
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++)
                    held.load_v(i, v_pool + keys.offset_of(min(first + key_of(q4, i), c1 - 1)), n);
            }
        };
        // element j + e of the lane's D/16 elements of keys 2i and 2i + 1 side by side
        const auto pair_up = [&](int j, V8 *x, auto value) {
#pragma unroll
            for (int e = 0; e < R::GJ; e++) {
                u32x4 y;
#pragma unroll
                for (int i = 0; i < 4; i++)
                    y[i] = __builtin_amdgcn_perm(value(2 * i + 1, (j + e) / 2), value(2 * i, (j + e) / 2),
                                                 (j + e) % 2 == 0 ? 0x05040100u : 0x07060302u);
                x[e] = __builtin_bit_cast(V8, y);
            }
        };

        // the chunk of the context
        if (c0 + wk * kTile < c1) {
            find(c0 + wk * kTile);
            load_ctx_k(c0 + wk * kTile);
            load_ctx_v(c0 + wk * kTile);
        }
        if constexpr (FP4)   // while the first tiles are on their way
            if (w.last)
                single_keys<T, D, R>(g, keys, w.seq, rows,
                        reinterpret_cast<uint64_t>(g.k) + w.b * g.k_stride[0] + head * g.k_stride[2],
                        reinterpret_cast<uint64_t>(g.v) + w.b * g.v_stride[0] + head * g.v_stride[2], wk, n, q4);
        f32x4 score[NT][2];
        float tops[NT];
#pragma unroll 1
        for (uint32_t first = c0 + wk * kTile; first < c1; first += kWaves * kTile) {
            const uint32_t next = first + kWaves * kTile;
            const auto key = [&](int k, V8 *x) {
#pragma unroll
                for (int i = 0; i < 4 && k + i / 2 < KS; i++)
                    x[i] = __builtin_bit_cast(V8, held.key(i % 2, k + i / 2, q4));
            };
            const auto values = [&](int j, V8 *x) {
                pair_up(j, x, [&](int i, int p) { return held.value(i, p, n); });
            };
            const bool some = first + kTile > c1;
            const bool raise = rows.template scores<false>(g, some, key, [&](int, int i) { return key_of(q4, i) < c1 - first; },
                    score, tops);
            // Past the end the last key once more: with a branch here, or below, the compiler no longer knows how many loads
            // are on their way after the keys', and waits for the values as well before the first product.
            if (kShare || next < c1) {
                find(next);
                load_ctx_k(next);
            }
            if (some) {
                // values of keys past the end meet weights of 0 and have to be finite: 0
#pragma unroll
                for (int i = 0; i < 8; i++)
                    held.clear_v(i, key_of(q4, i) < c1 - first);
            }
            if (raise)
                rows.raise_maxima(g, tops);
            rows.apply(g, score, values);
            if (kShare || next < c1)
                load_ctx_v(next);
        }

        // the drafted nodes, and before them the zone, with the sequence's last chunk
        if constexpr (!FP4)
            if (w.last) {
                const uint64_t kb = reinterpret_cast<uint64_t>(g.k) + keys.b * g.k_stride[0] + head * g.k_stride[2];
                const uint64_t vb = reinterpret_cast<uint64_t>(g.v) + keys.b * g.v_stride[0] + head * g.v_stride[2];
                const uint32_t count = keys.count, special = w.seq.special(), room = special - count;
                for (uint32_t first = wk * kTile; first < special; first += kWaves * kTile) {
                    const bool in_zone = WIN && first < room;   // room is whole tiles
                    const uint32_t begin = in_zone ? first : first - room, end = in_zone ? zone_of(w.seq) : count;
                    // Of key u, and of its values.
                    const auto key_row = [&](uint32_t u) {
                        if constexpr (WIN)
                            if (in_zone)
                                return k_pool + keys.offset_in_zone(min(u, end - 1));
                        return kb + min(u, end - 1) * g.k_stride[1];
                    };
                    const auto value_row = [&](uint32_t u) {
                        if constexpr (WIN)
                            if (in_zone)
                                return v_pool + keys.offset_in_zone(min(u, end - 1));
                        return vb + min(u, end - 1) * g.v_stride[1];
                    };
                    held.load_k(key_row(begin + n), key_row(begin + 16 + n), q4);
                    // A value that is not finite would turn a weight of 0 into NaN: here it counts
                    // as 0, and the rows that do see it get it added afterwards.
                    uint32_t wild = 0;
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        const uint32_t u = begin + key_of(q4, i);
                        held.load_v(i, value_row(u), n);
#pragma unroll
                        for (int j = 0; j < DJ / 2; j++)
                            held.vr[i][j] = tamed<T>(u < end ? held.vr[i][j] : 0, &wild);
                    }
                    uint32_t bits[NT];
#pragma unroll
                    for (int t = 0; t < NT; t++) {
                        bits[t] = 0;
                        if constexpr (WIN)
                            if (in_zone)
                                bits[t] = keys.seen_in_zone(t * 16 + n, begin);
                        if (!in_zone)
                            bits[t] = keys.seen(t * 16 + n, begin);
                    }
                    const auto key16 = [&](int k, V8 *x) {
#pragma unroll
                        for (int i = 0; i < 4 && k + i / 2 < KS; i++)
                            x[i] = __builtin_bit_cast(V8, held.key(i % 2, k + i / 2, q4));
                    };
                    const auto values16 = [&](int j, V8 *x) {
                        pair_up(j, x, [&](int i, int p) { return held.value(i, p, n); });
                    };
                    if (rows.template scores<true>(g, true, key16, [&](int t, int i) { return (bits[t] >> key_of(q4, i) & 1) != 0; },
                            score, tops))
                        rows.raise_maxima(g, tops);
                    rows.apply(g, score, values16);
                    if (__any(wild))
                        rows.add_wild(
                            [&](uint32_t u, uint32_t e) { return (float)reinterpret_cast<const T *>(value_row(u))[e]; },
                            begin, min(begin + kTile, end), bits, [&](int j, int r) { return (4 * q4 + r) * DJ + j; });
                }
            }

        rows.template join<1, kWaves>(g, merge, wk, lane);
        if (wk == 0)
            rows.template close<2 * DJ % 8 == 0 ? 8 : 4>(
                g, w, head, 0, lane, [&](int i) { return 4 * q4 * DJ + i * (2 * DJ % 8 == 0 ? 8 : 4); },
                [&](int t, int i, int e) {
                    const int k = i * (2 * DJ % 8 == 0 ? 8 : 4) + e;
                    return rows.o[t][k % DJ][k / DJ];
                });
    }   // join() left the LDS free
}

// ---- many rows -----------------------------------------------------------------
//
// More rows than one wave can hold: eight waves share the keys and values of a
// workgroup's steps through LDS, WM of them with rows of their own, 8 / WM
// dividing the step's tiles.  A step of kStep keys comes from memory to one of two
// LDS buffers while the step before is worked on in the other.  Its pieces lie so that neither
// product's reads meet in the banks, see place_of_piece().
//
// 16 trees of 64 nodes over up to 16,383 tokens, 8 heads of 128, 256 rows a head: 0.59 GB and 147 GFLOP in
// 198 us, where either alone would take some 100 us.  A turn of the loop, 32 keys by the 256 rows, takes 2,340 cycles;
// 735 of them are waits for the other waves at the ends of steps, and each wave has 32 matrix instructions, some 100 of
// the vector unit and 16 exponentials.  Steps of 32 keys cost 2 % more, steps of 128 the same; the waves' priorities
// make no difference.  The same with 8 nodes, 32 rows a head: 126 us, and 173 with two
// rows' worth of registers in the kernel for few.
constexpr int kSharedWaves = 8;
constexpr int shared_nt(int head_dim) { return head_dim <= 128 ? 2 : 1; }
// Keys of a step: a tile at least for each wave that divides them, whole pieces for each thread.  In 4 bits, where a
// step ends with its unpacking, 128 where LDS has room: the trees 220 us against 227.
constexpr int shared_step(int head_dim, int wm, bool fp4) {
    return head_dim < 128 || wm == 2 || (fp4 && head_dim == 128) ? 128 : 64;
}

// Place of a piece in its key's row of D / 8. The first product reads one piece of sixteen keys at
// once (of keys 0 to 3 and 12 to 15 together with the neighbouring piece of 4 to 11), the second two
// neighbouring pieces of eight: with these places both meet every bank once, where plain rows would meet the
// same few.  No conflict is counted for 64, 128 and 256 elements; for 96, with rows of three quarters of the
// banks, half of the reads' cycles are.
template <int D>
__device__ __forceinline__ uint32_t place_of_piece(uint32_t key, uint32_t piece) {
    if constexpr (D >= 128)
        return piece ^ (key & 7) << 1;
    else if constexpr (D == 64)
        return piece ^ (key >> 1 & 3) << 1;
    else
        return (piece + (key >> 2 & 3)) % (D / 8);
}
// The piece at a place: the way back.
template <int D>
__device__ __forceinline__ uint32_t piece_at_place(uint32_t key, uint32_t place) {
    if constexpr (D == 96)
        return (place + D / 8 - (key >> 2 & 3)) % (D / 8);
    else
        return place_of_piece<D>(key, place);
}

template <typename T, int D, int WM, bool WIN, bool FP4>
__global__ __launch_bounds__(64 * kSharedWaves, 2) void tree_attention_shared_kernel(AttnArgs g) {
    constexpr int NT = shared_nt(D), kStep = shared_step(D, WM, FP4), WK = kSharedWaves / WM;
    constexpr int kThreads = 64 * kSharedWaves, kPieces = D / 8, kEach = kStep * kPieces / kThreads;
    static_assert(kStep * kPieces % kThreads == 0 && kStep % (WK * kTile) == 0, "step");
    typedef Rows<T, D, NT, false> R;
    typedef typename R::V8 V8;
    constexpr int kBuffer = kStep * D * 2;   // bytes of a step's keys, or values
    constexpr int kMerge = WK > 1 ? WM * WK / 2 * R::kMergeFloats * 4 : 0;
    // two buffers, keys before values
    __shared__ __attribute__((aligned(16))) uint8_t data[4 * kBuffer > kMerge ? 4 * kBuffer : kMerge];
    __shared__ Place place;
    __shared__ typename SequenceOf<WIN>::T known[kThreads];
    __shared__ uint64_t sums[kSharedWaves];
    __shared__ uint32_t list[kListPages];
    __shared__ uint32_t wild_step;           // the last step of nodes with values that are not finite, plus 1

    const uint32_t wave = uniform(threadIdx.x >> 6), wm = wave % WM, wk = wave / WM;
    // The row blocks of one head's share run on one XCD, one after the other: they read the same keys.
    uint32_t unit = blockIdx.x, block = 0;
    if (g.row_blocks > 1) {
        const uint32_t at = blockIdx.x >> 3;
        block = at % g.row_blocks;
        unit = at / g.row_blocks * 8 + (blockIdx.x & 7);
    }
    const uint32_t mine = unit / g.heads, head = unit % g.heads;
    if (mine >= (g.budget != 0 ? g.budget : g.batch))
        return;
    find_place<kSharedWaves, WIN, FP4>(g, mine, &place, sums, known);
    Place at = {uniform(place.start), uniform(place.share), uniform(place.batch)};
#pragma unroll 1
    for (uint64_t end = at.share == kWhole ? kWhole : (mine + 1) * at.share; at.batch < g.batch && at.start < end;
            at.batch++) {
        const uint32_t thread = anew(threadIdx.x), lane = thread & 63, n = lane & 15, q4 = lane >> 4;
        const Part<WIN, FP4> w(g, at, mine, known, kThreads);
        at.start = w.end;
        note_splits(g, w, head, block);
        const Keys<kSharedWaves, WIN, FP4> keys(g, w, head, list);
        const uint32_t c0 = w.c0, c1 = w.c1, count = w.seq.nodes, special = w.seq.special(), room = special - count;
        const uint32_t row0 = (block * WM + wm) * 16 * NT;
        R rows;
        rows.open(g, keys.b, head, row0, lane);
        if (threadIdx.x == 0)
            wild_step = 0;
        __syncthreads();

        const uint64_t k_pool = reinterpret_cast<uint64_t>(g.k_cache), v_pool = reinterpret_cast<uint64_t>(g.v_cache);
        // 16 bits: this thread's pieces of a step, place at % kPieces of key at / kPieces, at = i * kThreads + thread.
        // Each wave's loads go straight to LDS, 64 places in a row.
        const uint64_t pools_apart = v_pool - k_pool;
        // The key of each piece as its page in the list and its place in the page, carried from step to step
        // (not with a window, where the list has a gap).
        const uint32_t head_at = head * g.head_step, page_end = g.page_tokens * g.token_step;
        const uint32_t pages_on = keys.page_of(kStep), places_on = (kStep - pages_on * g.page_tokens) * g.token_step;
        uint32_t in_list[kEach], in_page[kEach];
        if constexpr (!WIN) {
#pragma unroll
            for (int i = 0; i < kEach; i++) {
                const uint32_t token = c0 + (i * kThreads + thread) / kPieces, p = keys.page_of(token);
                in_list[i] = p - keys.p0;
                in_page[i] = (token - p * g.page_tokens) * g.token_step;
            }
        }
        // 4 bits: this thread's blocks of a step, the keys' before the values', on their way through registers.
        constexpr int kBlocks = D / 32, kStepBlocks = kStep * kBlocks, kMine = (2 * kStepBlocks + kThreads - 1) / kThreads;
        uint32_t codes[FP4 ? kMine : 1][4], power[FP4 ? kMine : 1];
        // Called for the part's steps in turn.
        const auto fetch = [&](uint8_t *to, uint32_t first) {
            if constexpr (FP4) {
#pragma unroll
                for (int i = 0; i < kMine; i++) {
                    const uint32_t at = i * kThreads + thread, in_half = at % kStepBlocks;
                    if (2 * kStepBlocks % kThreads != 0 && at >= 2 * kStepBlocks)
                        break;
                    const uint64_t from = (at < kStepBlocks ? k_pool : v_pool) +
                            keys.offset_of(min(first + in_half / kBlocks, c1 - 1));
                    load_words<4>(codes[i], from + in_half % kBlocks * 16);
                    typedef __attribute__((address_space(1))) uint8_t gu8;
                    power[i] = *(const gu8 *)(from + D / 2 + in_half % kBlocks);
                }
                return;
            }
            uint32_t place[kEach];
            const bool whole = !WIN && keys.listed && first + kStep <= c1;
            if (whole) {
#pragma unroll
                for (int i = 0; i < kEach; i++) {
                    place[i] = list[in_list[i]] + in_page[i] + head_at;
                    const uint32_t next = in_page[i] + places_on;
                    const bool over = next >= page_end;
                    in_page[i] = over ? next - page_end : next;
                    in_list[i] += over ? pages_on + 1 : pages_on;
                }
            } else {
#pragma unroll
                for (int i = 0; i < kEach; i++)
                    place[i] = keys.place_of(min(first + (i * kThreads + thread) / kPieces, c1 - 1));
            }
#pragma unroll
            for (int i = 0; i < kEach; i++) {
                const uint32_t at = i * kThreads + thread, key = at / kPieces,
                        piece = piece_at_place<D>(key, at % kPieces);
                const uint64_t from = k_pool + (uint64_t)(place[i] + piece) * 16;
                uint8_t *const there = to + (i * kThreads + wave * 64) * 16;
                __builtin_amdgcn_global_load_lds((const gvoid *)from, (svoid *)there, 16, 0, kStream);
                __builtin_amdgcn_global_load_lds((const gvoid *)(from + pools_apart), (svoid *)(there + kBuffer), 16,
                        0, kStream);
            }
        };
        // 4 bits: what fetch() has on its way becomes elements of T in LDS.
        const auto unpack = [&](uint8_t *to) {
            if constexpr (FP4) {
#pragma unroll
                for (int i = 0; i < kMine; i++) {
                    const uint32_t at = i * kThreads + thread, in_half = at % kStepBlocks, key = in_half / kBlocks;
                    if (2 * kStepBlocks % kThreads != 0 && at >= 2 * kStepBlocks)
                        break;
                    uint8_t *const row = to + (at < kStepBlocks ? 0 : kBuffer) + key * kPieces * 16;
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        *reinterpret_cast<u32x4 *>(row + place_of_piece<D>(key, in_half % kBlocks * 4 + j) * 16) =
                            eight_of<T>(codes[i][j], power_of(power[i], 0));
                }
            }
        };
        // A step of the drafted nodes, likewise.
        const uint64_t kb = reinterpret_cast<uint64_t>(g.k) + keys.b * g.k_stride[0] + head * g.k_stride[2];
        const uint64_t vb = reinterpret_cast<uint64_t>(g.v) + keys.b * g.v_stride[0] + head * g.v_stride[2];
        const auto fetch_nodes = [&](uint8_t *to, uint32_t first) {
#pragma unroll
            for (int i = 0; i < kEach; i++) {
                const uint32_t at = i * kThreads + thread, key = at / kPieces,
                        piece = piece_at_place<D>(key, at % kPieces);
                // what is in the zone's places is put there later
                const uint32_t u = WIN ? (uint32_t)min(max((int)(first + key - room), 0), (int)count - 1)
                                       : min(first + key, count - 1);
                uint8_t *const there = to + (i * kThreads + wave * 64) * 16;
                __builtin_amdgcn_global_load_lds((const gvoid *)(kb + u * g.k_stride[1] + piece * 16), (svoid *)there,
                        16, 0, 0);
                __builtin_amdgcn_global_load_lds((const gvoid *)(vb + u * g.v_stride[1] + piece * 16),
                        (svoid *)(there + kBuffer), 16, 0, 0);
            }
        };
        // What follows the context's step before `next`: its next step, or the first of the nodes.
        const auto fetch_after = [&](uint8_t *to, uint32_t next) {
            if (next < c1)
                fetch(to, next);
            else if (w.last && special > 0)
                fetch_nodes(to, 0);
        };
        const auto buffer_at = [&](uint32_t buffer) { return data + buffer * 2 * kBuffer; };
        // Waits for the step's loads; values of keys past the end meet weights of 0 and have to be finite: 0.
        const auto arrived = [&](uint8_t *to, uint32_t left) {
            __builtin_amdgcn_s_waitcnt(0);
            __syncthreads();
            if (left < kStep) {
                for (uint32_t at = left * kPieces + thread; at < kStep * kPieces; at += kThreads)
                    *reinterpret_cast<u32x4 *>(to + kBuffer + at * 16) = (u32x4){0, 0, 0, 0};
                __syncthreads();
            }
        };

        // Where this lane reads in a tile.  The reads are in assembly, each group with its own wait: the compiler
        // does not see that they have nothing to do with the loads on their way to the other buffer, and
        // would wait for those as well.
        const uint32_t data_at = (uint32_t)(uintptr_t)(svoid *)data;
        uint32_t key_at[R::KS], value_at[R::DJ];
#pragma unroll
        for (int k = 0; k < R::KS; k++)
            key_at[k] = (n * kPieces + place_of_piece<D>(n, k * 4 + q4)) * 16;
#pragma unroll
        for (int j = 0; j < R::DJ; j++) {
            const uint32_t row = 4 * q4 + n / 4;
            value_at[j] = kBuffer + (row * kPieces + place_of_piece<D>(row, 2 * j + (n % 4) / 2)) * 16 + (n & 1) * 8;
        }
        uint32_t tile_at = 0;   // of the tile in LDS
        const auto key = [&](int k, V8 *x) {
            u32x4 y[4];
            if (k + 1 < R::KS)
                asm volatile("ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:%6\n\t"
                             "ds_read_b128 %2, %5\n\tds_read_b128 %3, %5 offset:%6\n\ts_waitcnt lgkmcnt(0)"
                             : "=&v"(y[0]), "=&v"(y[1]), "=&v"(y[2]), "=&v"(y[3])
                             : "v"(tile_at + key_at[k]), "v"(tile_at + key_at[k + 1 < R::KS ? k + 1 : k]), "n"(16 * D * 2)
                             : "memory");
            else
                asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %2 offset:%3\n\ts_waitcnt lgkmcnt(0)"
                             : "=&v"(y[0]), "=&v"(y[1])
                             : "v"(tile_at + key_at[k]), "n"(16 * D * 2)
                             : "memory");
#pragma unroll
            for (int i = 0; i < 4 && k + i / 2 < R::KS; i++)
                x[i] = __builtin_bit_cast(V8, y[i]);
        };
        // Elements 16 j .. 16 j + 15 of the lane group's eight keys, transposed on the way: two reads of four keys.
        const auto values = [&](int j, V8 *x) {
            u32x2 y[2 * R::GJ];
            if constexpr (R::GJ == 4)
                asm volatile("ds_read_b64_tr_b16 %0, %8\n\tds_read_b64_tr_b16 %1, %8 offset:%12\n\t"
                             "ds_read_b64_tr_b16 %2, %9\n\tds_read_b64_tr_b16 %3, %9 offset:%12\n\t"
                             "ds_read_b64_tr_b16 %4, %10\n\tds_read_b64_tr_b16 %5, %10 offset:%12\n\t"
                             "ds_read_b64_tr_b16 %6, %11\n\tds_read_b64_tr_b16 %7, %11 offset:%12\n\t"
                             "s_waitcnt lgkmcnt(0)"
                             : "=&v"(y[0]), "=&v"(y[1]), "=&v"(y[2]), "=&v"(y[3]), "=&v"(y[4]), "=&v"(y[5]), "=&v"(y[6]), "=&v"(y[7])
                             : "v"(tile_at + value_at[j]), "v"(tile_at + value_at[j + 1]), "v"(tile_at + value_at[j + R::GJ - 2]),
                               "v"(tile_at + value_at[j + R::GJ - 1]), "n"(16 * D * 2)
                             : "memory");
            else
                asm volatile("ds_read_b64_tr_b16 %0, %4\n\tds_read_b64_tr_b16 %1, %4 offset:%6\n\t"
                             "ds_read_b64_tr_b16 %2, %5\n\tds_read_b64_tr_b16 %3, %5 offset:%6\n\t"
                             "s_waitcnt lgkmcnt(0)"
                             : "=&v"(y[0]), "=&v"(y[1]), "=&v"(y[2]), "=&v"(y[3])
                             : "v"(tile_at + value_at[j]), "v"(tile_at + value_at[j + 1]), "n"(16 * D * 2)
                             : "memory");
#pragma unroll
            for (int e = 0; e < R::GJ; e++)
                x[e] = __builtin_bit_cast(V8, (u32x4){y[2 * e].x, y[2 * e].y, y[2 * e + 1].x, y[2 * e + 1].y});
        };
        f32x4 score[NT][2];
        float tops[NT];

        // The part of the context.  Every wave does kTurns tiles of each step, also of the last one, where keys past
        // the end are masked.  The scores of a tile are had at the end of the turn before its
        // own, so that the loop has one way out, at its end, for the end and for maxima that have
        // to be raised alike: with a branch or a break inside, the compiler moves all accumulators in
        // every turn.  (After the last tile the scores of it are had once more, for nothing.)
        constexpr uint32_t kTurns = kStep / kTile / WK, kTileBytes = kTile * D * 2;
        uint32_t buffer = 0;
        fetch_after(data, c0);
        if (c0 < c1) {
            unpack(data);
            arrived(data, c1 - c0);
            fetch_after(buffer_at(1), c0 + kStep);
            uint32_t first = c0, turn = 0;
            const auto look = [&] {
                tile_at = uniform(data_at + buffer * 2 * kBuffer + (turn * WK + wk) * kTileBytes);
                const uint32_t t0 = first + (turn * WK + wk) * kTile;
                return rows.template scores<false>(g, t0 + kTile > c1, key, [&](int, int i) { return t0 + key_of(q4, i) < c1; },
                        score, tops);
            };
            bool raise = look();
            bool more = true;
            do {
                if (raise)
                    rows.raise_maxima(g, tops);
                do {
                    rows.apply(g, score, values);
                    turn++;
                    if (turn == kTurns) {
                        more = first + kStep < c1;
                        if (more) {
                            turn = 0;
                            buffer ^= 1;
                            first += kStep;
                            unpack(buffer_at(buffer));   // which all waves are past
                            arrived(buffer_at(buffer), c1 - first);
                            fetch_after(buffer_at(buffer ^ 1), first + kStep);
                        } else {
                            turn = kTurns - 1;
                        }
                    }
                    raise = look();
                } while (more && !raise);
            } while (more);
            buffer ^= 1;
        }

        // the drafted nodes, and before them the zone, with the sequence's last part
#pragma unroll 1
        for (uint32_t first = 0; w.last && first < special; first += kStep, buffer ^= 1) {
            __builtin_amdgcn_s_waitcnt(0);
            __syncthreads();
            if (first + kStep < special)
                fetch_nodes(buffer_at(buffer ^ 1), first + kStep);
            // A value that is not finite would turn a weight of 0 into NaN: here it counts as 0, and
            // the rows that do see it get it added afterwards.  Nodes past the last count as 0 altogether.
            uint32_t wild = 0;
#pragma unroll 1
            for (uint32_t at = thread; at < kStep * kPieces; at += kThreads) {
                u32x4 *const place = reinterpret_cast<u32x4 *>(buffer_at(buffer) + kBuffer + at * 16);
                u32x4 x = {0, 0, 0, 0};
                const uint32_t u = first + at / kPieces;
                bool real = u < special;
                if constexpr (WIN) {
                    if (u < room) {   // the zone's keys, read here
                        real = u < w.seq.zone;
                        const uint64_t row = keys.offset_in_zone(min(u, w.seq.zone - 1));
                        const uint32_t piece = piece_at_place<D>(at / kPieces, at % kPieces);
                        u32x4 y[2];
#pragma unroll
                        for (int z = 0; z < 2; z++) {
                            const uint64_t from = (z == 0 ? k_pool : v_pool) + row;
                            if constexpr (FP4) {
                                uint32_t code;
                                load_words<1>(&code, from + piece * 4);
                                const uint8_t p = *reinterpret_cast<const uint8_t *>(from + D / 2 + piece / 4);
                                y[z] = eight_of<T>(code, power_of(p, 0));
                            } else {
                                y[z] = *(const gu32x4 *)(from + piece * 16);
                            }
                        }
                        *reinterpret_cast<u32x4 *>(buffer_at(buffer) + at * 16) = y[0];
                        x = y[1];
                    } else if (real) {
                        x = *place;
                    }
                } else if (real) {
                    x = *place;
                }
                for (int e = 0; e < 4; e++)
                    x[e] = tamed<T>(real ? x[e] : 0, &wild);
                *place = x;
            }
            if (wild)
                wild_step = first + 1;
            __syncthreads();
            const bool any_wild = wild_step == first + 1;
#pragma unroll 1
            for (uint32_t turn = 0; turn < kTurns; turn++) {
                const uint32_t tile = turn * WK + wk, t0 = first + tile * kTile;
                if (t0 >= special)
                    break;
                const bool in_zone = WIN && t0 < room;   // room is whole tiles
                const uint32_t begin = in_zone ? t0 : t0 - room;
                tile_at = uniform(data_at + buffer * 2 * kBuffer + tile * kTileBytes);
                uint32_t bits[NT];
#pragma unroll
                for (int t = 0; t < NT; t++) {
                    bits[t] = 0;
                    if constexpr (WIN)
                        if (in_zone)
                            bits[t] = keys.seen_in_zone(row0 + t * 16 + n, begin);
                    if (!in_zone)
                        bits[t] = keys.seen(row0 + t * 16 + n, begin);
                }
                if (rows.template scores<true>(g, true, key, [&](int t, int i) { return (bits[t] >> key_of(q4, i) & 1) != 0; },
                        score, tops))
                    rows.raise_maxima(g, tops);
                rows.apply(g, score, values);
                if (any_wild)
                    rows.add_wild(
                        [&](uint32_t u, uint32_t e) {
                            uint64_t row = vb + u * g.v_stride[1];
                            if constexpr (WIN)
                                if (in_zone) {
                                    row = v_pool + keys.offset_in_zone(u);
                                    if constexpr (FP4)
                                        return fp4_number<D>(row, e);
                                }
                            return (float)reinterpret_cast<const T *>(row)[e];
                        },
                        begin, min(begin + kTile, in_zone ? zone_of(w.seq) : count), bits,
                        [&](int j, int r) { return 16 * j + 4 * q4 + r; });
            }
        }
        __syncthreads();

        rows.template join<WM, WK>(g, reinterpret_cast<float *>(data), wave, lane);
        if (wk == 0)
            rows.template close<4>(g, w, head, row0, lane, [&](int i) { return 16 * i + 4 * q4; },
                                   [&](int t, int i, int e) { return rows.o[t][i][e]; });
        __syncthreads();   // before the next part fills the LDS
    }
}


// ---- host ----------------------------------------------------------------------

// Which kernel, how many of its waves hold rows of their own, and the rows of a workgroup.
struct Shape {
    bool shared;
    int wm;
    uint32_t rows;
};

// Launches the kernel for elements of type T, heads of `dim`: one translation unit has each (WIN, FP4).
template <bool WIN, bool FP4, typename T, int D>
static hipError_t launch_dim(const AttnArgs &g, Shape s, uint32_t grid, hipStream_t stream) {
    if (!s.shared)
        return launch(tree_attention_kernel<T, D, WIN, FP4>, grid, 64 * kWaves, stream, nullptr, g);
    if (s.wm == 8)
        return launch(tree_attention_shared_kernel<T, D, 8, WIN, FP4>, grid, 64 * kSharedWaves, stream, nullptr, g);
    if (s.wm == 4)
        return launch(tree_attention_shared_kernel<T, D, 4, WIN, FP4>, grid, 64 * kSharedWaves, stream, nullptr, g);
    if constexpr (D <= 128)
        return launch(tree_attention_shared_kernel<T, D, 2, WIN, FP4>, grid, 64 * kSharedWaves, stream, nullptr, g);
    return hipErrorInvalidValue;
}

template <bool WIN, bool FP4, typename T>
static hipError_t launch_type(const AttnArgs &g, uint32_t dim, Shape s, uint32_t grid, hipStream_t stream) {
    switch (dim) {
    case 64: return launch_dim<WIN, FP4, T, 64>(g, s, grid, stream);
    case 96: return launch_dim<WIN, FP4, T, 96>(g, s, grid, stream);
    case 128: return launch_dim<WIN, FP4, T, 128>(g, s, grid, stream);
    case 256: return launch_dim<WIN, FP4, T, 256>(g, s, grid, stream);
    default: return hipErrorInvalidValue;
    }
}

template <bool WIN, bool FP4>
static hipError_t launch_kernel(const AttnArgs &g, uint32_t dtype, uint32_t dim, Shape s, uint32_t grid,
        hipStream_t stream) {
    return dtype == TB_BF16 ? launch_type<WIN, FP4, __bf16>(g, dim, s, grid, stream)
                            : launch_type<WIN, FP4, _Float16>(g, dim, s, grid, stream);
}
hipError_t launch_window_attention(const AttnArgs &g, uint32_t dtype, uint32_t dim, Shape s, uint32_t grid,
        hipStream_t stream);   // a window of 16 bits
hipError_t launch_fp4_attention(const AttnArgs &g, uint32_t dtype, uint32_t dim, Shape s, uint32_t grid,
        hipStream_t stream);   // 4 bits, with a window or none

}  // namespace tbk
