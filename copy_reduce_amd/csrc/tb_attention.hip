// tb_attention.hip -- gfx950 kernels of the attention of drafted tokens over the
// paged cache.
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
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "tb_cache_internal.h"
#include "tb_launch.h"

namespace tbk {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x3 __attribute__((ext_vector_type(3)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
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
    uint32_t page_step, token_step, head_step;            // in pieces of 16 bytes, see Keys
    uint32_t num_pages, page_tokens, max_seqs, max_pages;
    uint32_t div_mul, div_shift;       // token / page_tokens = token * div_mul >> div_shift
    uint32_t row_blocks;               // workgroups that share a head's rows
    uint32_t budget;                   // shares that a head's stream of keys is cut into; 0: one for each sequence
    float scale, scale2;               // |scale| log2 e; 1 for scale 0, see load_q
    int32_t sign;                      // of scale
    int32_t *split_base, *split_count; // [batch] workspace
    float *part_ml;                    // [slots][rows][2]
    float *part_o;                     // [slots][rows][D]
};

template <typename T>
struct Mfma;
template <>
struct Mfma<__bf16> {
    typedef bf16x8 V;
    static __device__ __forceinline__ f32x4 mul(V a, V b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
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
};
__device__ __forceinline__ Sequence sequence_of(const AttnArgs &g, uint32_t b) {
    Sequence s = {-1, 0, 0};
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
    return s;
}

// The batch's keys as one stream: each sequence's context and nodes, rounded up to kUnit
// keys, and one unit more for what a sequence costs by itself, one after the other.  It is cut into equal shares,
// one for each of the workgroups that a head's rows have, so that they all end together
// however the lengths differ.  A share may cover parts of several sequences.
// Every workgroup finds its place by itself (a few loads and a sum over the
// batch): nothing is planned before the launch and the lengths stay on the device.
constexpr uint32_t kUnit = 128;
__device__ __forceinline__ uint32_t weight_of(const Sequence &s) {
    return ((s.context + s.nodes + kUnit - 1) / kUnit + 1) * kUnit;
}

constexpr uint64_t kWhole = 1ull << 40;   // a share longer than any sequence
struct Place {
    uint64_t start;   // of sequence `batch` in the stream
    uint64_t share;
    uint32_t batch;   // the sequence in which the share begins; g.batch: no share
};

// `known`: LDS for a sequence a thread; filled where the batch has no more than that.
template <int WAVES>
__device__ __forceinline__ void find_place(const AttnArgs &g, uint32_t mine, Place *out, uint64_t *lds,
        Sequence *known) {
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
            const Sequence q = sequence_of(g, b0 + t);
            known[t] = q;
            w = weight_of(q);
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
            w = b0 + t < g.batch ? weight_of(sequence_of(g, b0 + t)) : 0;
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
struct Part {
    Sequence seq;
    uint32_t b, c0, c1, slot, splits;
    uint64_t end;       // of the sequence in the stream
    bool first, last;

    // known: what find_place() left, for up to `room` sequences
    __device__ __forceinline__ Part(const AttnArgs &g, const Place &at, uint32_t mine, const Sequence *known,
            uint32_t room) : b(at.batch) {
        const Sequence s = g.batch <= room && at.share != kWhole ? known[b] : sequence_of(g, b);
        seq.row = uniform(s.row);
        seq.context = uniform(s.context);
        seq.nodes = uniform(s.nodes);
        end = at.start + weight_of(seq);
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
template <int WAVES>
struct Keys {
    const AttnArgs &g;
    uint32_t b, head, count, p0;
    bool listed;
    const int32_t *row_table;
    const uint32_t *list;

    // Places in a pool count pieces of 16 bytes: 32 bits reach 64 GiB, and the address costs one instruction.
    __device__ __forceinline__ Keys(const AttnArgs &g_, const Part &part, uint32_t head_, uint32_t *lds)
        : g(g_), b(part.b), head(head_), count(part.seq.nodes), list(lds) {
        row_table = g.table + (uint64_t)max(part.seq.row, 0) * g.max_pages;
        p0 = page_of(part.c0);
        const uint32_t pages = part.c1 > part.c0 ? page_of(part.c1 - 1) - p0 + 1 : 0;
        listed = pages <= kListPages;
        if (listed)
            for (uint32_t i = threadIdx.x; i < pages; i += 64 * WAVES) {
                const uint32_t p = (uint32_t)row_table[p0 + i];
                lds[i] = (p < g.num_pages ? p : 0) * g.page_step;
            }
    }
    __device__ __forceinline__ uint32_t page_of(uint32_t token) const {
        return (uint32_t)(((uint64_t)token * g.div_mul) >> g.div_shift);
    }
    // Place of a context token's head in its pool.
    __device__ __forceinline__ uint32_t place_of(uint32_t token) const {
        const uint32_t p = page_of(token), in_page = token - p * g.page_tokens;
        uint32_t at;
        if (listed) {
            at = list[p - p0];
        } else {
            const uint32_t page = (uint32_t)row_table[p];
            at = (page < g.num_pages ? page : 0) * g.page_step;
        }
        return at + in_page * g.token_step + head * g.head_step;
    }
    __device__ __forceinline__ uint64_t offset_of(uint32_t token) const { return (uint64_t)place_of(token) * 16; }
    // Bits of the nodes first .. first + 31 that row r sees.
    __device__ __forceinline__ uint32_t seen(uint32_t r, uint32_t first) const {
        const uint32_t words = (g.nodes + 63) / 64 * 2, node = min(r, g.rows - 1) / g.group;
        uint32_t bits;
        if (g.mask != nullptr)
            bits = g.mask[((uint64_t)b * g.nodes + node) * words + first / 32];
        else
            bits = node < first ? 0u : (node >= first + 31 ? 0xffffffffu : (2u << (node - first)) - 1);
        return count < first + 32 ? bits & ((1u << (count - first)) - 1) : bits;
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
template <typename T, int D, int NT>
struct Rows {
    typedef typename Mfma<T>::V V8;
    static constexpr int KS = D / 32;   // steps of the first product
    static constexpr int DJ = D / 16;   // instructions of the second one
    static constexpr int GJ = DJ % 4 == 0 ? 4 : 2;   // of them, whose operands are had together
    static constexpr int kRegs = NT * DJ * 4;
    static constexpr int kMergeFloats = 64 * (kRegs + 2 * NT);   // of one wave, see join()
    V8 q[NT][KS];
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
                                h * g.q_stride[2] + q4 * 16;
#pragma unroll
            for (int s = 0; s < KS; s++) {
                u32x4 x = {0, 0, 0, 0};
                if (r < g.rows && g.sign != 0)
                    x = *(const gu32x4 *)(at + s * 64);
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
    // keep(t, i): whether row t * 16 + n sees the lane's i-th key, asked only if `some` row may not see all.
    template <typename Keys2, typename Keep>
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

    // Adds the values that tamed() left out to the rows that see them; element(j, r): which
    // element of the head o[t][j][r] is.
    template <typename Element>
    __device__ __forceinline__ void add_wild(const AttnArgs &g, uint64_t values, uint32_t first, uint32_t end,
                                             const uint32_t *bits, Element element) {
        for (uint32_t u = first; u < end; u++) {
            const T *row = reinterpret_cast<const T *>(values + u * g.v_stride[1]);
#pragma unroll
            for (int j = 0; j < DJ; j++) {
                // rare: a few loads at a time, so that this does not decide the kernel's registers
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    const float x = (float)row[element(j, r)];
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
    template <int RUN, typename Begin, typename Value>
    __device__ __forceinline__ void close(const AttnArgs &g, const Part &w, uint32_t head, uint32_t row0,
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
__device__ __forceinline__ void note_splits(const AttnArgs &g, const Part &w, uint32_t head, uint32_t block) {
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

template <typename T, int D>
__global__ __launch_bounds__(64 * kWaves, D == 64 ? 3 : (D <= 128 ? 2 : 1)) void tree_attention_kernel(AttnArgs g) {
    constexpr int NT = 1;
    typedef Rows<T, D, NT> R;
    typedef typename R::V8 V8;
    constexpr int KS = R::KS, DJ = R::DJ;
    __shared__ Place place;
    __shared__ Sequence known[64 * kWaves];
    __shared__ uint64_t sums[kWaves];
    __shared__ uint32_t list[kListPages];
    __shared__ float merge[kWaves / 2 * R::kMergeFloats];

    const uint32_t wk = uniform(threadIdx.x >> 6), mine = blockIdx.x / g.heads, head = blockIdx.x % g.heads;
    find_place<kWaves>(g, mine, &place, sums, known);
    Place at = {uniform(place.start), uniform(place.share), uniform(place.batch)};
#pragma unroll 1
    for (uint64_t end = at.share == kWhole ? kWhole : (mine + 1) * at.share; at.batch < g.batch && at.start < end;
            at.batch++) {
        const uint32_t thread = anew(threadIdx.x), lane = thread & 63, n = lane & 15, q4 = lane >> 4;
        const Part w(g, at, mine, known, 64 * kWaves);
        at.start = w.end;
        note_splits(g, w, head, 0);
        const Keys<kWaves> keys(g, w, head, list);
        const uint32_t c0 = w.c0, c1 = w.c1;
        R rows;
        rows.open(g, keys.b, head, 0, lane);
        __syncthreads();

        uint32_t kr[2][KS][4], vr[8][DJ / 2];
        const auto load_k = [&](uint64_t at0, uint64_t at1) {
#pragma unroll
            for (int s = 0; s < KS; s++) {
                load_dwords<4>(kr[0][s], at0 + s * 64 + q4 * 16);
                load_dwords<4>(kr[1][s], at1 + s * 64 + q4 * 16);
            }
        };
        // tokens first .. first + 31, those past the chunk its last one
        const auto load_ctx_k = [&](uint32_t first) {
            const uint64_t base = reinterpret_cast<uint64_t>(g.k_cache);
            load_k(base + keys.offset_of(min(first + n, c1 - 1)), base + keys.offset_of(min(first + 16 + n, c1 - 1)));
        };
        const auto load_ctx_v = [&](uint32_t first) {
#pragma unroll
            for (int i = 0; i < 8; i++)
                load_dwords<DJ / 2>(vr[i], reinterpret_cast<uint64_t>(g.v_cache) + n * (2 * DJ) +
                                               keys.offset_of(min(first + key_of(q4, i), c1 - 1)));
        };
        const auto key = [&](int k, V8 *x) {
#pragma unroll
            for (int i = 0; i < 4 && k + i / 2 < KS; i++) {
                const uint32_t *r = kr[i % 2][k + i / 2];
                x[i] = __builtin_bit_cast(V8, (u32x4){r[0], r[1], r[2], r[3]});
            }
        };
        // element j + e of the lane's D/16 elements of keys 2i and 2i + 1 side by side
        const auto values = [&](int j, V8 *x) {
#pragma unroll
            for (int e = 0; e < R::GJ; e++) {
                u32x4 y;
#pragma unroll
                for (int i = 0; i < 4; i++)
                    y[i] = __builtin_amdgcn_perm(vr[2 * i + 1][(j + e) / 2], vr[2 * i][(j + e) / 2],
                                                 (j + e) % 2 == 0 ? 0x05040100u : 0x07060302u);
                x[e] = __builtin_bit_cast(V8, y);
            }
        };

        // the chunk of the context
        if (c1 > c0 + wk * kTile) {
            load_ctx_k(c0 + wk * kTile);
            load_ctx_v(c0 + wk * kTile);
        }
        f32x4 score[NT][2];
        float tops[NT];
#pragma unroll 1
        for (uint32_t first = c0 + wk * kTile; first < c1; first += kWaves * kTile) {
            const uint32_t next = first + kWaves * kTile;
            const bool some = first + kTile > c1;
            const bool raise = rows.scores(g, some, key, [&](int, int i) { return key_of(q4, i) < c1 - first; },
                    score, tops);
            if (next < c1)
                load_ctx_k(next);
            if (some) {
                // values of keys past the end meet weights of 0 and have to be finite: 0
#pragma unroll
                for (int i = 0; i < 8; i++)
#pragma unroll
                    for (int j = 0; j < DJ / 2; j++)
                        vr[i][j] = key_of(q4, i) < c1 - first ? vr[i][j] : 0;
            }
            if (raise)
                rows.raise_maxima(g, tops);
            rows.apply(g, score, values);
            if (next < c1)
                load_ctx_v(next);
        }

        // the drafted nodes, with the sequence's last chunk
        if (w.last) {
            const uint64_t kb = reinterpret_cast<uint64_t>(g.k) + keys.b * g.k_stride[0] + head * g.k_stride[2];
            const uint64_t vb = reinterpret_cast<uint64_t>(g.v) + keys.b * g.v_stride[0] + head * g.v_stride[2];
            const uint32_t count = keys.count;
            for (uint32_t first = wk * kTile; first < count; first += kWaves * kTile) {
                load_k(kb + min(first + n, count - 1) * g.k_stride[1],
                        kb + min(first + 16 + n, count - 1) * g.k_stride[1]);
                // A value that is not finite would turn a weight of 0 into NaN: here it counts
                // as 0, and the rows that do see it get it added afterwards.
                uint32_t wild = 0;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const uint32_t u = first + key_of(q4, i);
                    load_dwords<DJ / 2>(vr[i], vb + min(u, count - 1) * g.v_stride[1] + n * (2 * DJ));
#pragma unroll
                    for (int j = 0; j < DJ / 2; j++)
                        vr[i][j] = tamed<T>(u < count ? vr[i][j] : 0, &wild);
                }
                uint32_t bits[NT];
#pragma unroll
                for (int t = 0; t < NT; t++)
                    bits[t] = keys.seen(t * 16 + n, first);
                if (rows.scores(g, true, key, [&](int t, int i) { return (bits[t] >> key_of(q4, i) & 1) != 0; },
                        score, tops))
                    rows.raise_maxima(g, tops);
                rows.apply(g, score, values);
                if (__any(wild))
                    rows.add_wild(g, vb, first, min(first + kTile, count), bits,
                                  [&](int j, int r) { return (4 * q4 + r) * DJ + j; });
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
// Keys of a step: a tile at least for each wave that divides them, whole pieces for each thread.
constexpr int shared_step(int head_dim, int wm) { return head_dim < 128 || wm == 2 ? 128 : 64; }

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

template <typename T, int D, int WM>
__global__ __launch_bounds__(64 * kSharedWaves, 2) void tree_attention_shared_kernel(AttnArgs g) {
    constexpr int NT = shared_nt(D), kStep = shared_step(D, WM), WK = kSharedWaves / WM;
    constexpr int kThreads = 64 * kSharedWaves, kPieces = D / 8, kEach = kStep * kPieces / kThreads;
    static_assert(kStep * kPieces % kThreads == 0 && kStep % (WK * kTile) == 0, "step");
    typedef Rows<T, D, NT> R;
    typedef typename R::V8 V8;
    constexpr int kBuffer = kStep * D * 2;   // bytes of a step's keys, or values
    constexpr int kMerge = WK > 1 ? WM * WK / 2 * R::kMergeFloats * 4 : 0;
    // two buffers, keys before values
    __shared__ __attribute__((aligned(16))) uint8_t data[4 * kBuffer > kMerge ? 4 * kBuffer : kMerge];
    __shared__ Place place;
    __shared__ Sequence known[kThreads];
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
    find_place<kSharedWaves>(g, mine, &place, sums, known);
    Place at = {uniform(place.start), uniform(place.share), uniform(place.batch)};
#pragma unroll 1
    for (uint64_t end = at.share == kWhole ? kWhole : (mine + 1) * at.share; at.batch < g.batch && at.start < end;
            at.batch++) {
        const uint32_t thread = anew(threadIdx.x), lane = thread & 63, n = lane & 15, q4 = lane >> 4;
        const Part w(g, at, mine, known, kThreads);
        at.start = w.end;
        note_splits(g, w, head, block);
        const Keys<kSharedWaves> keys(g, w, head, list);
        const uint32_t c0 = w.c0, c1 = w.c1, count = w.seq.nodes;
        const uint32_t row0 = (block * WM + wm) * 16 * NT;
        R rows;
        rows.open(g, keys.b, head, row0, lane);
        if (threadIdx.x == 0)
            wild_step = 0;
        __syncthreads();

        // This thread's pieces of a step: place at % kPieces of key at / kPieces, at = i * kThreads + thread.
        // Each wave's loads go straight to LDS, 64 places in a row.
        const uint64_t pools_apart = reinterpret_cast<uint64_t>(g.v_cache) - reinterpret_cast<uint64_t>(g.k_cache);
        // The key of each piece as its page in the list and its place in the page, carried from step to step.
        const uint32_t head_at = head * g.head_step, page_end = g.page_tokens * g.token_step;
        const uint32_t pages_on = keys.page_of(kStep), places_on = (kStep - pages_on * g.page_tokens) * g.token_step;
        uint32_t in_list[kEach], in_page[kEach];
#pragma unroll
        for (int i = 0; i < kEach; i++) {
            const uint32_t token = c0 + (i * kThreads + thread) / kPieces, p = keys.page_of(token);
            in_list[i] = p - keys.p0;
            in_page[i] = (token - p * g.page_tokens) * g.token_step;
        }
        // Called for the part's steps in turn.
        const auto fetch = [&](uint8_t *to, uint32_t first) {
            uint32_t place[kEach];
            const bool whole = keys.listed && first + kStep <= c1;
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
                const uint64_t from = reinterpret_cast<uint64_t>(g.k_cache) + (uint64_t)(place[i] + piece) * 16;
                uint8_t *const there = to + (i * kThreads + wave * 64) * 16;
                __builtin_amdgcn_global_load_lds((const gvoid *)from, (svoid *)there, 16, 0, kStream);
                __builtin_amdgcn_global_load_lds((const gvoid *)(from + pools_apart), (svoid *)(there + kBuffer), 16,
                        0, kStream);
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
                const uint32_t u = min(first + key, count - 1);
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
            else if (w.last && count > 0)
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
            arrived(data, c1 - c0);
            fetch_after(buffer_at(1), c0 + kStep);
            uint32_t first = c0, turn = 0;
            const auto look = [&] {
                tile_at = uniform(data_at + buffer * 2 * kBuffer + (turn * WK + wk) * kTileBytes);
                const uint32_t t0 = first + (turn * WK + wk) * kTile;
                return rows.scores(g, t0 + kTile > c1, key, [&](int, int i) { return t0 + key_of(q4, i) < c1; },
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

        // the drafted nodes, with the sequence's last part
#pragma unroll 1
        for (uint32_t first = 0; w.last && first < count; first += kStep, buffer ^= 1) {
            __builtin_amdgcn_s_waitcnt(0);
            __syncthreads();
            if (first + kStep < count)
                fetch_nodes(buffer_at(buffer ^ 1), first + kStep);
            // A value that is not finite would turn a weight of 0 into NaN: here it counts as 0, and
            // the rows that do see it get it added afterwards.  Nodes past the last count as 0 altogether.
            uint32_t wild = 0;
#pragma unroll 1
            for (uint32_t at = thread; at < kStep * kPieces; at += kThreads) {
                u32x4 *const place = reinterpret_cast<u32x4 *>(buffer_at(buffer) + kBuffer + at * 16);
                u32x4 x = {0, 0, 0, 0};
                if (first + at / kPieces < count) {
                    x = *place;
                    for (int e = 0; e < 4; e++)
                        x[e] = tamed<T>(x[e], &wild);
                }
                *place = x;
            }
            if (wild)
                wild_step = first + 1;
            __syncthreads();
            const bool any_wild = wild_step == first + 1;
#pragma unroll 1
            for (uint32_t turn = 0; turn < kTurns; turn++) {
                const uint32_t tile = turn * WK + wk, t0 = first + tile * kTile;
                if (t0 >= count)
                    break;
                tile_at = uniform(data_at + buffer * 2 * kBuffer + tile * kTileBytes);
                uint32_t bits[NT];
#pragma unroll
                for (int t = 0; t < NT; t++)
                    bits[t] = keys.seen(row0 + t * 16 + n, t0);
                if (rows.scores(g, true, key, [&](int t, int i) { return (bits[t] >> key_of(q4, i) & 1) != 0; },
                        score, tops))
                    rows.raise_maxima(g, tops);
                rows.apply(g, score, values);
                if (any_wild)
                    rows.add_wild(g, vb, t0, min(t0 + kTile, count), bits,
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

constexpr uint32_t combine_lanes(int head_dim) { return head_dim <= 64 ? 16 : (head_dim <= 128 ? 32 : 64); }
// From so many rows on a wave has several, a row's lanes go through all of its shares, and the kernel takes fewer rounds
// of waves; below, its lanes divide the shares.  The whole call by the second and the first way: 32,768 rows, some three
// shares each, 202 us and 196; 16,384 rows 147 and 145; 8,192 rows 134 either way; 128 rows, 32 shares, 26 and 31.
constexpr uint32_t kCombineMany = 16384;

// Joins the shares of sequences that have several.  With m the largest of the shares' maxima,
// l = sum_s exp(m_s - m) l_s and o likewise.  The shares' rows are read once, mostly from the caches that
// they were written to a moment ago: 32,768 rows of 128 elements, some three shares each, 12 us.
// With many shares the latency of its loads counts, so a few are made at once: for one sequence of 16,383 tokens in
// 64 shares the whole call takes 30 us, and 35 with one at a time; eight at once cost the trees 4 us.
template <typename T, int D, bool MANY>
__global__ __launch_bounds__(256) void tree_combine_kernel(AttnArgs g) {
    // kLanes lanes have a row's elements, four each; the other lanes of a wave have other splits, or other rows
    constexpr uint32_t kLanes = combine_lanes(D), kGroups = MANY ? 1 : 64 / kLanes, kWidth = MANY ? kLanes : 64;
    const uint32_t lane = threadIdx.x % kWidth, at = blockIdx.x * (256 / kWidth) + threadIdx.x / kWidth;
    const uint32_t r = at % g.rows, head = at / g.rows % g.heads;
    const uint64_t b = at / g.rows / g.heads;
    if (b >= g.batch)
        return;
    const int32_t splits = g.split_count[b];
    if (splits <= 1)
        return;
    const uint64_t first = (uint64_t)g.split_base[b], step = (uint64_t)g.heads * g.rows;
    const uint64_t slot0 = first * step + (uint64_t)head * g.rows + r;
    const uint32_t part = lane / kLanes, at4 = lane % kLanes * 4;
    float m = -INFINITY, l = 0.f;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    for (int32_t s0 = 0; s0 < splits; s0 += kWidth) {   // lane s has split s0 + s's maximum and sum
        const bool there = s0 + (int32_t)lane < splits;
        float ms = -INFINITY, ls = 0.f;
        if (there) {
            const uint64_t k = slot0 + (uint64_t)(s0 + lane) * step;
            ms = g.part_ml[2 * k];
            ls = g.part_ml[2 * k + 1];
        }
        float top = fmaxf(ms, m);
#pragma unroll
        for (int d = kWidth / 2; d > 0; d >>= 1)
            top = fmaxf(top, __shfl_xor(top, d));
        const float base = top == -INFINITY ? 0.f : top * g.scale2;
        const float fade = __builtin_amdgcn_exp2f(__builtin_fmaf(m, g.scale2, -base));
        const float f = __builtin_amdgcn_exp2f(__builtin_fmaf(ms, g.scale2, -base));
        m = top;
        o *= fade;
        float sum = f * ls;
#pragma unroll
        for (int d = kWidth / 2; d > 0; d >>= 1)
            sum += __shfl_xor(sum, d);
        l = l * fade + sum;
        const int32_t n = min(splits - s0, (int32_t)kWidth);
        // The loads of four splits a group are on their way together; past the last, the last once more.
        constexpr int kLoads = 4;
        for (int32_t i = 0; i < n; i += kLoads * (int32_t)kGroups) {
            f32x4 x[kLoads];
#pragma unroll
            for (int u = 0; u < kLoads; u++) {
                const int32_t s = min(i + u * (int32_t)kGroups + (int32_t)part, n - 1);
                const uint64_t k = slot0 + (uint64_t)(s0 + s) * step;
                x[u] = *(const gf32x4 *)(reinterpret_cast<uint64_t>(g.part_o) + (k * D + min(at4, D - 4u)) * 4);
            }
#pragma unroll
            for (int u = 0; u < kLoads; u++) {   // every lane of the row in every turn: all supply their f
                const int32_t s = i + u * (int32_t)kGroups + (int32_t)part;
                const float fs = __shfl(f, min(s, (int32_t)kWidth - 1), kWidth);
                o += s < n ? x[u] * fs : (f32x4){0.f, 0.f, 0.f, 0.f};
            }
        }
    }
#pragma unroll
    for (uint32_t d = kLanes; d < kWidth; d <<= 1)
#pragma unroll
        for (int e = 0; e < 4; e++)
            o[e] += __shfl_xor(o[e], (int)d);
    const uint32_t node = r / g.group, h = head * g.group + r % g.group;
    int32_t nodes = (int32_t)g.nodes;
    if (g.tree_nodes != nullptr)
        nodes = g.tree_nodes[b];
    const bool empty = l == 0.f || (int32_t)node >= nodes;
    if (part == 0 && at4 < D) {
        typedef T t4 __attribute__((ext_vector_type(4)));
        t4 x;
        for (int e = 0; e < 4; e++)
            x[e] = (T)(empty ? 0.f : o[e] / l);
        *reinterpret_cast<t4 *>(g.out + b * g.out_stride[0] + node * g.out_stride[1] + h * g.out_stride[2]
                + lane * 8) = x;
    }
    if (g.lse != nullptr && lane == 0)
        g.lse[(b * g.nodes + node) * g.heads_q + h] = empty ? -INFINITY : lse_of<T>(m, l, g.scale);
}

// ---- host ----------------------------------------------------------------------

// Which kernel, how many of its waves hold rows of their own, and the rows of a workgroup.
struct Shape {
    bool shared;
    int wm;
    uint32_t rows;
};
static Shape shape_of(uint32_t rows, uint32_t head_dim) {
    if (rows <= 16)
        return {false, 1, 16};
    const uint32_t each = 16 * shared_nt((int)head_dim);
    int wm = head_dim <= 128 ? 2 : 4;
    while (wm < kSharedWaves && wm * each < rows)
        wm *= 2;
    return {true, wm, wm * each};
}

// Workgroups of the kernel that a CU holds, by the registers they are built with.
static uint32_t resident(const Shape &s, uint32_t head_dim) {
    if (s.shared)
        return 1;
    return head_dim == 64 ? 3 : (head_dim <= 128 ? 2 : 1);
}

// Up to this many tokens a sequence (by the table's room, the lengths are not known here) a workgroup
// takes a whole sequence; up to the second, where many rows' workgroups fill the chip that way.
// Measured with lengths spread evenly up to the bound, whole against shares: 4 sequences of 2 heads,
// one node of 4 rows, 500 tokens 16.7 us against 19.5, 1,000 tokens 19.6 against 18.0; 32 sequences of
// 8 heads, 64 rows, 2,000 tokens 53 us against 70, 4,000 tokens 89 against 92, 8,000 tokens 156 against 142.
constexpr uint64_t kShort = 768, kShortMany = 4096;

struct Plan {
    Shape shape;
    uint32_t rows, row_blocks, budget;
    uint64_t slots;
};
static Plan plan_of(const tb_tree_attn &a, uint32_t heads, int cu_count, uint64_t longest = ~0ull) {
    Plan p;
    p.rows = a.nodes * (a.heads_q / heads);
    p.shape = shape_of(p.rows, a.head_dim);
    p.row_blocks = (p.rows + p.shape.rows - 1) / p.shape.rows;
    // Shares a head's stream is cut into: as many as run at once, or, where heads and row
    // blocks leave CUs idle that way, the number up to four rounds that leaves the fewest.
    const uint64_t each = (uint64_t)heads * p.row_blocks, room = (uint64_t)cu_count * resident(p.shape, a.head_dim);
    const uint64_t most = 4 * room / each > 1 ? 4 * room / each : 1, least = room / each > 1 ? room / each : 1;
    uint64_t best = least;
    double best_use = 0;
    for (uint64_t n = least; n <= most && best_use < 0.96; n++) {
        const double use = (double)(n * each) / (double)((n * each + room - 1) / room * room);
        if (use > best_use + 0.04) {
            best = n;
            best_use = use;
        }
    }
    p.budget = (uint32_t)best;
    p.slots = (uint64_t)p.budget + a.batch;
    // Where the table has room for short contexts only, a workgroup takes a whole sequence, and
    // there is nothing to find and nothing to join.
    if (longest <= kShort || (p.shape.shared && longest <= kShortMany && a.batch * each >= room))
        p.budget = 0;
    return p;
}

static uint64_t round16(uint64_t n) { return (n + 15) / 16 * 16; }

uint64_t tree_attention_workspace(const tb_tree_attn &a, uint32_t heads, int cu_count) {
    const Plan p = plan_of(a, heads, cu_count);
    const uint64_t rows = p.slots * heads * p.rows;
    return round16(8ull * a.batch) + round16(8 * rows) + 4 * rows * a.head_dim;
}

template <typename T, int D>
static hipError_t launch_dim(const AttnArgs &g, Shape s, uint32_t grid, hipStream_t stream) {
    LaunchSeq seq;
    hipError_t e;
    if (g.budget == 0)
        seq.last();
    if (!s.shared) {
        e = launch(tree_attention_kernel<T, D>, grid, 64 * kWaves, stream, nullptr, g);
    } else if (s.wm == 8) {
        e = launch(tree_attention_shared_kernel<T, D, 8>, grid, 64 * kSharedWaves, stream, nullptr, g);
    } else if (s.wm == 4) {
        e = launch(tree_attention_shared_kernel<T, D, 4>, grid, 64 * kSharedWaves, stream, nullptr, g);
    } else {
        if constexpr (D <= 128)
            e = launch(tree_attention_shared_kernel<T, D, 2>, grid, 64 * kSharedWaves, stream, nullptr, g);
        else
            e = hipErrorInvalidValue;
    }
    if (e != hipSuccess || g.budget == 0)
        return e;
    seq.last();
    const uint32_t rows = g.batch * g.heads * g.rows;   // < 2^24
    constexpr uint32_t kMany = 256 / combine_lanes(D);
    if (D < 256 && rows >= kCombineMany)
        return launch(tree_combine_kernel<T, D, D < 256>, (rows + kMany - 1) / kMany, 256, stream, nullptr, g);
    return launch(tree_combine_kernel<T, D, false>, (rows + 3) / 4, 256, stream, nullptr, g);
}

template <typename T>
static hipError_t launch_type(const AttnArgs &g, uint32_t dim, Shape s, uint32_t grid, hipStream_t stream) {
    switch (dim) {
    case 64: return launch_dim<T, 64>(g, s, grid, stream);
    case 96: return launch_dim<T, 96>(g, s, grid, stream);
    case 128: return launch_dim<T, 128>(g, s, grid, stream);
    case 256: return launch_dim<T, 256>(g, s, grid, stream);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_tree_attention(const tb_tree_attn &a, const tb_cache &c, int cu_count, hipStream_t stream) {
    const Plan p = plan_of(a, c.heads, cu_count, (uint64_t)c.max_pages * c.page_tokens);
    AttnArgs g;
    g.q = static_cast<const uint8_t *>(a.q);
    g.k = static_cast<const uint8_t *>(a.k);
    g.v = static_cast<const uint8_t *>(a.v);
    g.out = static_cast<uint8_t *>(a.out);
    g.lse = a.lse;
    for (int k = 0; k < 3; k++) {
        g.q_stride[k] = 2 * a.q_stride[k];
        g.k_stride[k] = 2 * a.k_stride[k];
        g.v_stride[k] = 2 * a.v_stride[k];
        g.out_stride[k] = 2 * a.out_stride[k];
    }
    g.seqs = a.seqs;
    g.mask = reinterpret_cast<const uint32_t *>(a.mask);
    g.tree_nodes = a.tree_nodes;
    g.k_cache = static_cast<const uint8_t *>(c.pools[a.k_pool]);
    g.v_cache = static_cast<const uint8_t *>(c.pools[a.v_pool]);
    g.table = c.table;
    g.lens = c.lens;
    g.batch = a.batch;
    g.nodes = a.nodes;
    g.heads_q = a.heads_q;
    g.heads = c.heads;
    g.group = a.heads_q / c.heads;
    g.rows = p.rows;
    const bool token_major = c.layout == TB_CACHE_TOKEN_MAJOR;
    g.page_step = (uint32_t)(c.page_stride / 16);
    g.token_step = (token_major ? c.heads * c.head_bytes : c.head_bytes) / 16;
    g.head_step = (token_major ? c.head_bytes : c.page_tokens * c.head_bytes) / 16;
    g.num_pages = c.num_pages;
    g.page_tokens = c.page_tokens;
    g.max_seqs = c.max_seqs;
    g.max_pages = c.max_pages;
    // x / d for x < 2^31: with 2^(s-1) < d <= 2^s and f = ceil(2^(31+s) / d) < 2^32, x f / 2^(31+s)
    // exceeds x / d by less than x / 2^(31+s) <= 1 / d, too little to reach the next whole number
    uint32_t s = 0;
    while ((1u << s) < c.page_tokens)
        s++;
    g.div_shift = 31 + s;
    g.div_mul = (uint32_t)(((1ull << (31 + s)) + c.page_tokens - 1) / c.page_tokens);
    g.row_blocks = p.row_blocks;
    g.budget = p.budget;
    g.sign = a.scale > 0.f ? 1 : (a.scale < 0.f ? -1 : 0);
    // scale 0: q is taken as 0, and any positive scale will do
    g.scale = g.sign == 0 ? 1.f : fabsf(a.scale);
    g.scale2 = (float)((double)g.scale * 1.4426950408889634);
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    const uint64_t rows = p.slots * c.heads * p.rows;
    g.split_base = reinterpret_cast<int32_t *>(ws);
    g.split_count = g.split_base + a.batch;
    g.part_ml = reinterpret_cast<float *>(ws + round16(8ull * a.batch));
    g.part_o = reinterpret_cast<float *>(ws + round16(8ull * a.batch) + round16(8 * rows));
    const uint64_t units = (uint64_t)(p.budget != 0 ? p.budget : a.batch) * c.heads;
    const uint64_t grid = p.row_blocks > 1 ? (units + 7) / 8 * 8 * p.row_blocks : units;
    return a.dtype == TB_BF16 ? launch_type<__bf16>(g, a.head_dim, p.shape, (uint32_t)grid, stream)
                              : launch_type<_Float16>(g, a.head_dim, p.shape, (uint32_t)grid, stream);
}

}  // namespace tbk
