// tb_attention.hip -- attention of drafted tokens over the paged cache: the kernels for the
// whole context in 16 bits, the one that joins the shares, and how a call is planned.
#include "tb_attention_kernels.h"

namespace tbk {

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
    return s.shared ? 1 : (uint32_t)few_resident((int)head_dim);
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

// With a window the table says nothing about how many keys a sequence shows, and what the lengths are is not known here.
//
// Many rows of few keys are divided instead of the keys, so that every workgroup has a whole sequence and nothing is joined.
// 16 trees of 64 nodes by rows and by shares, of up to 16,383 tokens and one of 16,000 among 15 of some 100: windows of 2,000
// 61.5 us and 83, 59 and 49; of 4,000 103 and 107, 98 and 37, where the gain is no longer worth it.
//
// Few rows are shared out as without a window.  64 sequences, windows of 4,096, by shares and by a workgroup a sequence
// and head: of up to 32,767 tokens 192 us and 186, in 4 bits 81 and 71; of up to 8,192 tokens 161 and 173, 54 and 50;
// 60 of up to 300 tokens and 4 of 32,000 42 and 143, 27 and 48.
constexpr uint64_t kShortWindow = 2048;
static Plan plan_of_window(const tb_tree_attn &a, uint32_t heads, int cu_count, uint64_t longest, uint64_t table) {
    Plan p = plan_of(a, heads, cu_count, longest <= kShortWindow ? longest : table);
    if (!p.shape.shared || p.budget == 0 || longest > kShortWindow)
        return p;
    for (int wm = p.shape.wm; wm >= (a.head_dim <= 128 ? 2 : 4); wm /= 2) {
        const uint32_t rows = wm * 16 * shared_nt((int)a.head_dim), blocks = (p.rows + rows - 1) / rows;
        if ((uint64_t)a.batch * heads * blocks >= (uint64_t)cu_count) {
            p.shape = {true, wm, rows};
            p.row_blocks = blocks;
            p.budget = 0;
            break;
        }
    }
    return p;
}

static uint64_t round16(uint64_t n) { return (n + 15) / 16 * 16; }

uint64_t tree_attention_workspace(const tb_tree_attn &a, uint32_t heads, int cu_count) {
    const Plan p = plan_of(a, heads, cu_count);
    const uint64_t rows = p.slots * heads * p.rows;
    return round16(8ull * a.batch) + round16(8 * rows) + 4 * rows * a.head_dim;
}

template <typename T, int D>
static hipError_t launch_combine(const AttnArgs &g, hipStream_t stream) {
    const uint32_t rows = g.batch * g.heads * g.rows;   // < 2^24
    constexpr uint32_t kMany = 256 / combine_lanes(D);
    if (D < 256 && rows >= kCombineMany)
        return launch(tree_combine_kernel<T, D, D < 256>, (rows + kMany - 1) / kMany, 256, stream, nullptr, g);
    return launch(tree_combine_kernel<T, D, false>, (rows + 3) / 4, 256, stream, nullptr, g);
}
template <typename T>
static hipError_t launch_combine(const AttnArgs &g, uint32_t dim, hipStream_t stream) {
    switch (dim) {
    case 64: return launch_combine<T, 64>(g, stream);
    case 96: return launch_combine<T, 96>(g, stream);
    case 128: return launch_combine<T, 128>(g, stream);
    case 256: return launch_combine<T, 256>(g, stream);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_tree_attention(const tb_tree_attn &a, const tb_attn_view &view, const tb_cache &c, int cu_count,
        hipStream_t stream) {
    // the longest context that a sequence can show
    const uint64_t table = (uint64_t)c.max_pages * c.page_tokens;
    uint64_t longest = table;
    if (view.window != 0 && (uint64_t)view.window + view.sinks < longest)
        longest = (uint64_t)view.window + view.sinks;
    const bool fp4 = view.fp4 != 0;
    const Plan p = view.window != 0 ? plan_of_window(a, c.heads, cu_count, longest, table)
                                    : plan_of(a, c.heads, cu_count, longest);
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
    const uint32_t piece = fp4 ? 4 : 16;
    g.page_step = (uint32_t)(c.page_stride / piece);
    g.token_step = (token_major ? c.heads * c.head_bytes : c.head_bytes) / piece;
    g.head_step = (token_major ? c.head_bytes : c.page_tokens * c.head_bytes) / piece;
    g.window = view.window;
    g.sinks = view.sinks;
    g.depths = view.depths;
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
    uint64_t grid = p.row_blocks > 1 ? (units + 7) / 8 * 8 * p.row_blocks : units;
    if (fp4 && !p.shape.shared)   // whole XCDs
        grid = (units / c.heads + 7) / 8 * 8 * c.heads;
    LaunchSeq seq;
    if (g.budget == 0)
        seq.last();
    const hipError_t e =
        fp4 ? launch_fp4_attention(g, a.dtype, a.head_dim, p.shape, (uint32_t)grid, stream)
        : view.window != 0 ? launch_window_attention(g, a.dtype, a.head_dim, p.shape, (uint32_t)grid, stream)
                           : launch_kernel<false, false>(g, a.dtype, a.head_dim, p.shape, (uint32_t)grid, stream);
    if (e != hipSuccess || g.budget == 0)
        return e;
    seq.last();
    return a.dtype == TB_BF16 ? launch_combine<__bf16>(g, a.head_dim, stream)
                              : launch_combine<_Float16>(g, a.head_dim, stream);
}

}  // namespace tbk
