// tb_attention.hip -- gfx950 kernels of the attention of drafted tokens over the
// paged cache.
//
// The M = nodes * (heads_q / heads) rows of one sequence that read one
// key/value head share each of its keys, so a key costs M multiply-adds a
// byte: up to some 200 rows the cache's bytes decide, beyond that the
// products.  Either way every key and value goes from memory straight into the
// registers of the one wave (or, for many rows, the few waves) that multiplies it.
//
// A wave owns R = 16 NT rows and walks over tiles of 32 keys with a running
// maximum and sum.  Both products run on 16x16x32 matrix instructions and are
// taken transposed, rows along the columns:
//   S' = K Q'   a lane (n = lane % 16, g = lane / 16) then holds, of row n, the
//               scores of keys 4g .. 4g+3 and 16+4g .. 16+4g+3,
//   O' = V' P'  which are just the k-places that lane has to supply of P', so
//               that the probabilities never leave their lane.  V' wants, for
//               one element of the head, the values of those eight keys in one
//               register quad: each lane loads D/16 neighbouring elements of
//               its eight keys and pairs them up by byte permutes.  The order
//               in which elements meet the instruction's rows is free: place n
//               of instruction j is element n D/16 + j.
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

constexpr int kTile = 32;              // keys of a tile
constexpr uint32_t kListPages = 2048;  // page numbers of a chunk kept in LDS
constexpr uint32_t kMinChunk = 128;    // fewest tokens a workgroup is given
// A row's maximum is let stand until a score exceeds it by this much (in powers of
// two): weights then stay below 2^8, well inside every type here, and after the
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
    uint32_t page_stride, token_step, head_step;          // bytes
    uint32_t num_pages, page_tokens, max_seqs, max_pages;
    uint32_t div_mul, div_shift;       // token / page_tokens = token * div_mul >> div_shift
    uint32_t row_blocks;               // workgroups that share a head's rows
    uint32_t budget;                   // chunks that all sequences together are cut into, one more each
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
};
template <>
struct Mfma<_Float16> {
    typedef f16x8 V;
    static __device__ __forceinline__ f32x4 mul(V a, V b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static constexpr uint32_t kExp = 0x7c00;
};

// N dwords at 4-byte alignment or better, as 16-byte loads and one rest.
template <int N>
__device__ __forceinline__ void load_dwords(uint32_t *r, uint64_t at) {
    typedef __attribute__((address_space(1))) u32x2 gu32x2;
    typedef uint32_t u32x3a __attribute__((ext_vector_type(3), aligned(4)));
    typedef __attribute__((address_space(1))) u32x3a gu32x3;
    if constexpr (N >= 4) {
        const u32x4 x = *(const gu32x4 *)at;
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

// What a workgroup works on.
struct Work {
    int32_t batch;   // -1: nothing
    int32_t split;
    int32_t splits;
    int32_t slot;    // number of the split among all
    int32_t chunk;   // tokens of a split
    int32_t seq;
    int32_t context;
};

__device__ __forceinline__ int32_t context_of(const AttnArgs &g, uint32_t b, int32_t *seq) {
    const int32_t q = g.seqs[b];
    *seq = (uint32_t)q < g.max_seqs ? q : -1;
    if (*seq < 0)
        return 0;
    const int32_t n = g.lens[q], most = (int32_t)(g.max_pages * g.page_tokens);
    return n < 0 ? 0 : (n < most ? n : most);
}

// Cuts the contexts into chunks of equal length, as many as `budget` and one
// more a sequence at most, and finds chunk number `want`.  Every workgroup does
// the whole of it (a few loads and two sums), so nothing has to be planned
// before the launch and the lengths stay on the device.
template <int kWaves>
__device__ __forceinline__ void find_work(const AttnArgs &g, int32_t want, Work *out, uint64_t *lds) {
    const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6;
    int32_t seq = -1, ctx = 0;
    uint64_t total = 0;
    for (uint32_t b0 = 0; b0 < g.batch; b0 += 64 * kWaves) {
        ctx = b0 + t < g.batch ? context_of(g, b0 + t, &seq) : 0;
        total += (uint32_t)ctx;
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        total += __shfl_xor(total, d);
    if (lane == 0)
        lds[wave] = total;
    if (t == 0)
        out->batch = -1;
    __syncthreads();
    total = 0;
    for (int w = 0; w < kWaves; w++)
        total += lds[w];
    uint64_t chunk = (total + g.budget - 1) / g.budget;
    chunk = chunk < kMinChunk ? kMinChunk : (chunk + kMinChunk - 1) / kMinChunk * kMinChunk;
    uint32_t before = 0;
    for (uint32_t b0 = 0; b0 < g.batch; b0 += 64 * kWaves) {
        if (g.batch > 64 * kWaves)
            ctx = b0 + t < g.batch ? context_of(g, b0 + t, &seq) : 0;
        const uint32_t n = b0 + t >= g.batch ? 0 : (ctx == 0 ? 1 : (uint32_t)(((uint32_t)ctx + chunk - 1) / chunk));
        uint32_t x = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t y = __shfl_up(x, d);
            if (lane >= (uint32_t)d)
                x += y;
        }
        __syncthreads();
        if (lane == 63)
            lds[wave] = x;
        __syncthreads();
        uint32_t base = before + x - n;
        for (uint32_t w = 0; w < kWaves; w++) {
            base += w < wave ? (uint32_t)lds[w] : 0;
            before += (uint32_t)lds[w];
        }
        if ((uint32_t)want >= base && (uint32_t)want < base + n) {
            out->batch = (int32_t)(b0 + t);
            out->split = want - (int32_t)base;
            out->splits = (int32_t)n;
            out->slot = want;
            out->chunk = (int32_t)(chunk < 0x7fffffff ? chunk : 0x7fffffff);
            out->seq = seq;
            out->context = ctx;
        }
    }
    __syncthreads();
}

// Where a workgroup's keys are: its chunk [c0, c1) of the context, the drafted
// nodes if `last`, and the pages of the chunk.
template <int kWaves>
struct Keys {
    const AttnArgs &g;
    const Work w;
    uint32_t b, head, c0, c1, count, p0;
    bool last, listed;
    const int32_t *row_table;
    const uint32_t *list;

    __device__ __forceinline__ Keys(const AttnArgs &g_, const Work &w_, uint32_t head_, uint32_t *lds)
        : g(g_), w(w_), b((uint32_t)w_.batch), head(head_), list(lds) {
        int32_t nodes = w.seq < 0 ? 0 : (int32_t)g.nodes;
        if (w.seq >= 0 && g.tree_nodes != nullptr) {
            const int32_t x = g.tree_nodes[b];
            nodes = x < 0 ? 0 : (x < nodes ? x : nodes);
        }
        count = (uint32_t)nodes;
        c0 = (uint32_t)w.split * (uint32_t)w.chunk;
        c1 = min(c0 + (uint32_t)w.chunk, (uint32_t)w.context);
        last = w.split + 1 == w.splits;
        row_table = g.table + (uint64_t)(w.seq < 0 ? 0 : w.seq) * g.max_pages;
        p0 = page_of(c0);
        const uint32_t pages = c1 > c0 ? page_of(c1 - 1) - p0 + 1 : 0;
        listed = pages <= kListPages;
        if (listed)
            for (uint32_t i = threadIdx.x; i < pages; i += 64 * kWaves) {
                const uint32_t p = (uint32_t)row_table[p0 + i];
                lds[i] = p < g.num_pages ? p : 0;
            }
    }
    __device__ __forceinline__ uint32_t page_of(uint32_t token) const {
        return (uint32_t)(((uint64_t)token * g.div_mul) >> g.div_shift);
    }
    // Byte offset of a context token's head in its pool.
    __device__ __forceinline__ uint64_t offset_of(uint32_t token) const {
        const uint32_t p = page_of(token), in_page = token - p * g.page_tokens;
        uint32_t page;
        if (listed) {
            page = list[p - p0];
        } else {
            page = (uint32_t)row_table[p];
            page = page < g.num_pages ? page : 0;
        }
        return (uint64_t)page * g.page_stride + in_page * g.token_step + head * g.head_step;
    }
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
    static constexpr int kRegs = NT * DJ * 4;
    static constexpr int kMergeFloats = 64 * (kRegs + 2 * NT);   // of one wave, see join()
    V8 q[NT][KS];
    f32x4 o[NT][DJ];
    float m[NT], l[NT];                 // l: this lane's keys only, until close()

    // Row r is node r / group of query head head * group + r % group.
    __device__ __forceinline__ void open(const AttnArgs &g, uint32_t b, uint32_t head, uint32_t row0) {
        const uint32_t lane = threadIdx.x & 63, n = lane & 15, q4 = lane >> 4;
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
            l[t] = 0.f;
#pragma unroll
            for (int j = 0; j < DJ; j++)
                o[t][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
        }
    }

    // One tile of keys.  key(z, k): step k's operand for keys 16 z .. 16 z + 15; value(j):
    // instruction j's operand; keep(t, i): whether row t * 16 + n sees the lane's
    // i-th key, asked only if `some` row may not see all.  between() runs once
    // the keys are no longer needed.
    template <typename Key, typename Value, typename Keep, typename Between>
    __device__ __forceinline__ void tile(const AttnArgs &g, bool some, Key key, Value value, Keep keep, Between between) {
        f32x4 s[NT][2];
#pragma unroll
        for (int t = 0; t < NT; t++)
            s[t][0] = s[t][1] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < KS; k++)
#pragma unroll
            for (int z = 0; z < 2; z++) {
                const V8 x = key(z, k);
#pragma unroll
                for (int t = 0; t < NT; t++)
                    s[t][z] = Mfma<T>::mul(x, q[t][k], s[t][z]);
            }
        between();
        V8 p[NT];
#pragma unroll
        for (int t = 0; t < NT; t++) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; i++)
                x[i] = s[t][i / 4][i % 4];
            if (some) {
#pragma unroll
                for (int i = 0; i < 8; i++)
                    x[i] = keep(t, i) ? x[i] : -INFINITY;
            }
            float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
            if (__any(top * g.scale2 > __builtin_fmaf(m[t], g.scale2, kSlack))) {
                top = fmaxf(lanes_max(top), m[t]);
                const float base = top == -INFINITY ? 0.f : top * g.scale2;
                // a row's first keys: m = -inf, the factor 0 meets sums that are 0
                const float fade = __builtin_amdgcn_exp2f(__builtin_fmaf(m[t], g.scale2, -base));
                l[t] *= fade;
#pragma unroll
                for (int j = 0; j < DJ; j++)
                    o[t][j] *= fade;
                m[t] = top;
            }
            const float base = m[t] == -INFINITY ? 0.f : m[t] * g.scale2;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], g.scale2, -base));
                l[t] += e;
                // rounded to the element type, which is what the matrix instruction takes; the sum keeps all bits
                p[t][i] = (T)e;
            }
        }
#pragma unroll
        for (int j = 0; j < DJ; j++) {
            const V8 x = value(j);
#pragma unroll
            for (int t = 0; t < NT; t++)
                o[t][j] = Mfma<T>::mul(x, p[t], o[t][j]);
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
    __device__ __forceinline__ void join(const AttnArgs &g, float *lds) {
        const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave % WM, wk = wave / WM;
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
    __device__ __forceinline__ void close(const AttnArgs &g, const Work &w, uint32_t head, uint32_t row0, uint32_t count,
                                          Begin begin, Value value) {
        constexpr int kRuns = 4 * DJ / RUN;
        typedef T tv __attribute__((ext_vector_type(RUN)));
        const uint32_t lane = threadIdx.x & 63, n = lane & 15, q4 = lane >> 4;
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
            const bool empty = l[t] == 0.f || node >= count;
            const float inv = empty ? 0.f : 1.f / l[t];
            const uint64_t to = reinterpret_cast<uint64_t>(g.out) + (uint32_t)w.batch * g.out_stride[0] +
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
                g.lse[((uint64_t)(uint32_t)w.batch * g.nodes + node) * g.heads_q + h] =
                    empty ? -INFINITY : m[t] * g.scale + logf(l[t]);
        }
    }
};

// The combine kernel's way into the slots.
__device__ __forceinline__ void note_splits(const AttnArgs &g, const Work &w, uint32_t head, uint32_t block) {
    if (block == 0 && head == 0 && w.split == 0 && threadIdx.x == 0) {
        g.split_base[w.batch] = w.slot;
        g.split_count[w.batch] = w.splits;
    }
}

// ---- few rows ------------------------------------------------------------------
//
// Up to 32 rows (16 NT): the cache's bytes decide.  Each of the four waves
// takes every fourth tile and reads its keys and values straight into the registers
// from which they are multiplied; the next tile's keys are on their way during the
// second product, its values during the first.
constexpr int kWaves = 4;

template <typename T, int D, int NT>
__global__ __launch_bounds__(64 * kWaves, D <= 128 ? 2 : 1) void tree_attention_kernel(AttnArgs g) {
    typedef Rows<T, D, NT> R;
    typedef typename R::V8 V8;
    constexpr int KS = R::KS, DJ = R::DJ;
    __shared__ Work work;
    __shared__ uint64_t sums[kWaves];
    __shared__ uint32_t list[kListPages];
    __shared__ float merge[kWaves / 2 * R::kMergeFloats];

    const uint32_t lane = threadIdx.x & 63, wk = threadIdx.x >> 6, n = lane & 15, q4 = lane >> 4;
    const uint32_t head = blockIdx.x % g.heads;
    find_work<kWaves>(g, (int32_t)(blockIdx.x / g.heads), &work, sums);
    if (work.batch < 0)
        return;
    const Work w = work;
    note_splits(g, w, head, 0);
    const Keys<kWaves> keys(g, w, head, list);
    const uint32_t c0 = keys.c0, c1 = keys.c1;
    R rows;
    rows.open(g, keys.b, head, 0);
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
    const auto key = [&](int z, int k) {
        return __builtin_bit_cast(V8, (u32x4){kr[z][k][0], kr[z][k][1], kr[z][k][2], kr[z][k][3]});
    };
    // element j of the lane's D/16 elements of keys 2i and 2i + 1 side by side
    const auto value = [&](int j) {
        u32x4 x;
#pragma unroll
        for (int i = 0; i < 4; i++)
            x[i] = __builtin_amdgcn_perm(vr[2 * i + 1][j / 2], vr[2 * i][j / 2], j % 2 == 0 ? 0x05040100u : 0x07060302u);
        return __builtin_bit_cast(V8, x);
    };

    // the chunk of the context
    if (c1 > c0 + wk * kTile) {
        load_ctx_k(c0 + wk * kTile);
        load_ctx_v(c0 + wk * kTile);
    }
    for (uint32_t first = c0 + wk * kTile; first < c1; first += kWaves * kTile) {
        const uint32_t next = first + kWaves * kTile;
        const bool some = first + kTile > c1;
        if (some) {
            // values of keys past the end meet weights of 0 and have to be finite: 0
#pragma unroll
            for (int i = 0; i < 8; i++)
#pragma unroll
                for (int j = 0; j < DJ / 2; j++)
                    vr[i][j] = first + key_of(q4, i) < c1 ? vr[i][j] : 0;
        }
        rows.tile(g, some, key, value, [&](int, int i) { return first + key_of(q4, i) < c1; },
                  [&] {
                      if (next < c1)
                          load_ctx_k(next);
                  });
        if (next < c1)
            load_ctx_v(next);
    }

    // the drafted nodes, with the sequence's last chunk
    if (keys.last) {
        const uint64_t kb = reinterpret_cast<uint64_t>(g.k) + keys.b * g.k_stride[0] + head * g.k_stride[2];
        const uint64_t vb = reinterpret_cast<uint64_t>(g.v) + keys.b * g.v_stride[0] + head * g.v_stride[2];
        const uint32_t count = keys.count;
        for (uint32_t first = wk * kTile; first < count; first += kWaves * kTile) {
            load_k(kb + min(first + n, count - 1) * g.k_stride[1], kb + min(first + 16 + n, count - 1) * g.k_stride[1]);
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
            rows.tile(g, true, key, value, [&](int t, int i) { return (bits[t] >> key_of(q4, i) & 1) != 0; }, [] {});
            if (__any(wild))
                rows.add_wild(g, vb, first, min(first + kTile, count), bits,
                              [&](int j, int r) { return (4 * q4 + r) * DJ + j; });
        }
    }

    rows.template join<1, kWaves>(g, merge);
    if (wk == 0)
        rows.template close<2 * DJ % 8 == 0 ? 8 : 4>(
            g, w, head, 0, keys.count, [&](int i) { return 4 * q4 * DJ + i * (2 * DJ % 8 == 0 ? 8 : 4); },
            [&](int t, int i, int e) {
                const int k = i * (2 * DJ % 8 == 0 ? 8 : 4) + e;
                return rows.o[t][k % DJ][k / DJ];
            });
}

// ---- many rows -----------------------------------------------------------------
//
// More rows than one wave can hold: eight waves share the keys and values of a
// workgroup's steps through LDS, WM of them with rows of their own, 8 / WM
// dividing the step's tiles.  A step of kStep keys is copied from memory to
// registers while the one before is worked on, and from there to the other of
// two LDS buffers.  A key's 16-byte pieces are stored at places
// piece ^ (key % 16), so that neither product's reads, one a column of
// pieces and one a transposing read of four keys, meet in the banks.
constexpr int kSharedWaves = 8;
constexpr int shared_nt(int head_dim) { return head_dim <= 128 ? 2 : 1; }
constexpr int shared_step(int head_dim) { return head_dim <= 128 ? 128 : 64; }

template <typename T, int D, int WM>
__global__ __launch_bounds__(64 * kSharedWaves, 2) void tree_attention_shared_kernel(AttnArgs g) {
    constexpr int NT = shared_nt(D), kStep = shared_step(D), WK = kSharedWaves / WM;
    constexpr int kThreads = 64 * kSharedWaves, kPieces = D / 8, kEach = kStep * kPieces / kThreads;
    static_assert(kStep * kPieces % kThreads == 0 && kStep % (WK * kTile) == 0, "step");
    typedef Rows<T, D, NT> R;
    typedef typename R::V8 V8;
    constexpr int kBuffer = kStep * D * 2;   // bytes of a step's keys, or values
    constexpr int kSwizzle = kPieces >= 16 ? 15 : (kPieces == 8 ? 7 : 0);   // 12 pieces: their rows differ in banks by themselves
    union Lds {
        uint8_t data[2][2][kBuffer];         // [buffer][keys, values]
        float merge[WK > 1 ? WM * WK / 2 * R::kMergeFloats : 1];
    };
    __shared__ __attribute__((aligned(16))) Lds lds;
    __shared__ Work work;
    __shared__ uint64_t sums[kSharedWaves];
    __shared__ uint32_t list[kListPages];
    __shared__ uint32_t wild_step[2];        // by buffer: the last step with values that are not finite, plus 1

    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, q4 = lane >> 4;
    const uint32_t wm = wave % WM, wk = wave / WM;
    // The row blocks of one head's chunk run on one XCD, one after the other: they read the same keys.
    uint32_t unit = blockIdx.x, block = 0;
    if (g.row_blocks > 1) {
        const uint32_t at = blockIdx.x >> 3;
        block = at % g.row_blocks;
        unit = at / g.row_blocks * 8 + (blockIdx.x & 7);
    }
    const uint32_t head = unit % g.heads;
    find_work<kSharedWaves>(g, (int32_t)(unit / g.heads), &work, sums);
    if (work.batch < 0)
        return;
    const Work w = work;
    note_splits(g, w, head, block);
    const Keys<kSharedWaves> keys(g, w, head, list);
    const uint32_t c0 = keys.c0, c1 = keys.c1, count = keys.count;
    const uint32_t row0 = (block * WM + wm) * 16 * NT;
    R rows;
    rows.open(g, keys.b, head, row0);
    if (threadIdx.x < 2)
        wild_step[threadIdx.x] = 0;
    __syncthreads();

    const uint32_t steps_ctx = c1 > c0 ? (c1 - c0 + kStep - 1) / kStep : 0;
    const uint32_t steps = steps_ctx + (keys.last ? (count + kStep - 1) / kStep : 0);
    const uint64_t kb = reinterpret_cast<uint64_t>(g.k) + keys.b * g.k_stride[0] + head * g.k_stride[2];
    const uint64_t vb = reinterpret_cast<uint64_t>(g.v) + keys.b * g.v_stride[0] + head * g.v_stride[2];

    u32x4 sk[kEach], sv[kEach];
    const auto fetch = [&](uint32_t step) {
        const bool ctx = step < steps_ctx;
        const uint32_t first = ctx ? c0 + step * kStep : (step - steps_ctx) * kStep, end = ctx ? c1 : count;
#pragma unroll
        for (int i = 0; i < kEach; i++) {
            const uint32_t at = i * kThreads + threadIdx.x, key = at / kPieces, piece = at % kPieces;
            const uint32_t k = min(first + key, end - 1);
            uint64_t ka, va;
            if (ctx) {
                const uint64_t off = keys.offset_of(k) + piece * 16;
                ka = reinterpret_cast<uint64_t>(g.k_cache) + off;
                va = reinterpret_cast<uint64_t>(g.v_cache) + off;
            } else {
                ka = kb + k * g.k_stride[1] + piece * 16;
                va = vb + k * g.v_stride[1] + piece * 16;
            }
            sk[i] = *(const gu32x4 *)ka;
            sv[i] = *(const gu32x4 *)va;
        }
    };
    const auto put = [&](uint32_t step) {
        const bool ctx = step < steps_ctx;
        const uint32_t first = ctx ? c0 + step * kStep : (step - steps_ctx) * kStep, end = ctx ? c1 : count;
        uint32_t wild = 0;
#pragma unroll
        for (int i = 0; i < kEach; i++) {
            const uint32_t at = i * kThreads + threadIdx.x, key = at / kPieces, piece = at % kPieces;
            const uint32_t to = (key * kPieces + (piece ^ (key & kSwizzle))) * 16;
            // values of keys past the end, and (until add_wild) those that are not finite, count as 0
            u32x4 v = first + key < end ? sv[i] : (u32x4){0, 0, 0, 0};
            if (!ctx)
                for (int e = 0; e < 4; e++)
                    v[e] = tamed<T>(v[e], &wild);
            *reinterpret_cast<u32x4 *>(lds.data[step & 1][0] + to) = sk[i];
            *reinterpret_cast<u32x4 *>(lds.data[step & 1][1] + to) = v;
        }
        if (wild)
            wild_step[step & 1] = step + 1;
    };

    if (steps > 0) {
        fetch(0);
        put(0);
    }
    __syncthreads();
    for (uint32_t step = 0; step < steps; step++) {
        if (step + 1 < steps)
            fetch(step + 1);
        const bool ctx = step < steps_ctx;
        const uint32_t first = ctx ? c0 + step * kStep : (step - steps_ctx) * kStep, end = ctx ? c1 : count;
        const bool wild = wild_step[step & 1] == step + 1;
#pragma unroll 1
        for (uint32_t tile = wk; tile < kStep / kTile; tile += WK) {
            const uint32_t t0 = first + tile * kTile;
            if (t0 >= end)
                break;
            const uint8_t *kp = lds.data[step & 1][0] + tile * kTile * D * 2, *vp = lds.data[step & 1][1] + tile * kTile * D * 2;
            const auto key = [&](int z, int k) {
                const uint32_t row = z * 16 + n;
                return *reinterpret_cast<const V8 *>(kp + (row * kPieces + ((k * 4 + q4) ^ (row & kSwizzle))) * 16);
            };
            // elements 16 j .. 16 j + 15 of the lane group's eight keys, transposed on the way: two reads of four keys
            const auto value = [&](int j) {
                typedef short s16x4 __attribute__((ext_vector_type(4)));
                typedef __attribute__((address_space(3))) s16x4 ls16x4;
                s16x4 half[2];
#pragma unroll
                for (int z = 0; z < 2; z++) {
                    const uint32_t row = z * 16 + 4 * q4 + n / 4, piece = 2 * j + (n % 4) / 2;
                    half[z] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (ls16x4 *)(vp + (row * kPieces + (piece ^ (row & kSwizzle))) * 16 + (n & 1) * 8));
                }
                return __builtin_bit_cast(V8, __builtin_shufflevector(half[0], half[1], 0, 1, 2, 3, 4, 5, 6, 7));
            };
            if (ctx) {
                rows.tile(g, t0 + kTile > c1, key, value, [&](int, int i) { return t0 + key_of(q4, i) < c1; }, [] {});
            } else {
                uint32_t bits[NT];
#pragma unroll
                for (int t = 0; t < NT; t++)
                    bits[t] = keys.seen(row0 + t * 16 + n, t0);
                rows.tile(g, true, key, value, [&](int t, int i) { return (bits[t] >> key_of(q4, i) & 1) != 0; }, [] {});
                if (wild)
                    rows.add_wild(g, vb, t0, min(t0 + kTile, count), bits,
                                  [&](int j, int r) { return 16 * j + 4 * q4 + r; });
            }
        }
        if (step + 1 < steps)
            put(step + 1);
        __syncthreads();
    }

    rows.template join<WM, WK>(g, lds.merge);
    if (wk == 0)
        rows.template close<4>(g, w, head, row0, count, [&](int i) { return 16 * i + 4 * q4; },
                               [&](int t, int i, int e) { return rows.o[t][i][e]; });
}

// Joins the chunks of sequences that have several: one wave a row.
template <typename T, int D>
__global__ __launch_bounds__(256) void tree_combine_kernel(AttnArgs g) {
    const uint32_t lane = threadIdx.x & 63;
    const uint64_t at = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const uint32_t r = (uint32_t)(at % g.rows), head = (uint32_t)(at / g.rows % g.heads);
    const uint64_t b = at / g.rows / g.heads;
    if (b >= g.batch)
        return;
    const int32_t splits = g.split_count[b];
    if (splits <= 1)
        return;
    const uint64_t first = (uint64_t)g.split_base[b];
    float m = -INFINITY;
    for (int32_t s = lane; s < splits; s += 64)
        m = fmaxf(m, g.part_ml[2 * (((first + s) * g.heads + head) * g.rows + r)]);
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        m = fmaxf(m, __shfl_xor(m, d));
    const float base = m == -INFINITY ? 0.f : m * g.scale2;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    float l = 0.f;
    for (int32_t s = 0; s < splits; s++) {
        const uint64_t k = ((first + s) * g.heads + head) * g.rows + r;
        const float f = __builtin_amdgcn_exp2f(__builtin_fmaf(g.part_ml[2 * k], g.scale2, -base));
        l += f * g.part_ml[2 * k + 1];
        if (lane * 4 < D) {
            const f32x4 x = *(const gf32x4 *)(reinterpret_cast<uint64_t>(g.part_o) + (k * D + lane * 4) * 4);
            o += x * f;
        }
    }
    const uint32_t node = r / g.group, h = head * g.group + r % g.group;
    int32_t nodes = (int32_t)g.nodes;
    if (g.tree_nodes != nullptr)
        nodes = g.tree_nodes[b];
    const bool empty = l == 0.f || (int32_t)node >= nodes;
    if (lane * 4 < D) {
        typedef T t4 __attribute__((ext_vector_type(4)));
        t4 x;
        for (int e = 0; e < 4; e++)
            x[e] = (T)(empty ? 0.f : o[e] / l);
        *reinterpret_cast<t4 *>(g.out + b * g.out_stride[0] + node * g.out_stride[1] + h * g.out_stride[2] + lane * 8) = x;
    }
    if (g.lse != nullptr && lane == 0)
        g.lse[(b * g.nodes + node) * g.heads_q + h] = empty ? -INFINITY : m * g.scale + logf(l);
}

// ---- host ----------------------------------------------------------------------

// Which kernel, how many of its waves hold rows of their own, and the rows of a workgroup.
struct Shape {
    bool shared;
    int nt, wm;
    uint32_t rows;
};
static Shape shape_of(uint32_t rows, uint32_t head_dim) {
    if (rows <= 16 || (rows <= 32 && head_dim <= 128))
        return {false, rows <= 16 ? 1 : 2, 1, rows <= 16 ? 16u : 32u};
    const uint32_t each = 16 * shared_nt((int)head_dim);
    int wm = head_dim <= 128 ? 2 : 4;
    while (wm < kSharedWaves && wm * each < rows)
        wm *= 2;
    return {true, 0, wm, wm * each};
}

struct Plan {
    Shape shape;
    uint32_t rows, row_blocks, budget;
    uint64_t slots;
};
static Plan plan_of(const tb_tree_attn &a, uint32_t heads, int cu_count) {
    Plan p;
    p.rows = a.nodes * (a.heads_q / heads);
    p.shape = shape_of(p.rows, a.head_dim);
    p.row_blocks = (p.rows + p.shape.rows - 1) / p.shape.rows;
    const uint32_t target = (uint32_t)cu_count * (p.shape.shared ? 2 : (p.shape.nt == 1 ? 3 : 2));
    p.budget = target / (heads * p.row_blocks);
    if (p.budget < 1)
        p.budget = 1;
    p.slots = (uint64_t)p.budget + a.batch;
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
    if (!s.shared) {
        if (s.nt == 1)
            e = launch(tree_attention_kernel<T, D, 1>, grid, 64 * kWaves, stream, nullptr, g);
        else if constexpr (D <= 128)
            e = launch(tree_attention_kernel<T, D, 2>, grid, 64 * kWaves, stream, nullptr, g);
        else
            e = hipErrorInvalidValue;
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
    if (e != hipSuccess)
        return e;
    seq.last();
    const uint64_t rows = (uint64_t)g.batch * g.heads * g.rows;
    return launch(tree_combine_kernel<T, D>, (uint32_t)((rows + 3) / 4), 256, stream, nullptr, g);
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
    const Plan p = plan_of(a, c.heads, cu_count);
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
    g.page_stride = (uint32_t)c.page_stride;
    g.token_step = token_major ? c.heads * c.head_bytes : c.head_bytes;
    g.head_step = token_major ? c.head_bytes : c.page_tokens * c.head_bytes;
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
    const uint64_t units = p.slots * c.heads;
    const uint64_t grid = p.row_blocks > 1 ? (units + 7) / 8 * 8 * p.row_blocks : units;
    if (grid > (1u << 30))
        return hipErrorInvalidValue;
    return a.dtype == TB_BF16 ? launch_type<__bf16>(g, a.head_dim, p.shape, (uint32_t)grid, stream)
                              : launch_type<_Float16>(g, a.head_dim, p.shape, (uint32_t)grid, stream);
}

}  // namespace tbk
