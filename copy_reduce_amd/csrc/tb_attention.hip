// tb_attention.hip -- gfx950 kernel of the attention of drafted tokens over the
// paged cache.
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "tb_cache_internal.h"
#include "tb_launch.h"

namespace tbk {

struct AttnArgs {
    tb_tree_attn a;
    const uint8_t *k_cache, *v_cache;
    const int32_t *table, *lens;
    uint64_t page_stride, token_step, head_step;
    uint32_t num_pages, page_tokens, max_seqs, max_pages, heads;
};

__device__ __forceinline__ float to_float(__hip_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ void from_float(float v, __hip_bfloat16 *o) { *o = __float2bfloat16(v); }
__device__ __forceinline__ void from_float(float v, __half *o) { *o = __float2half(v); }

// One wave a row (sequence, node, query head): one key after the other with a
// running maximum and sum, each lane holding ceil(D / 64) of the elements.
template <typename T, int D>
__global__ __launch_bounds__(64) void tree_attention_kernel(AttnArgs g) {
    constexpr int R = (D + 63) / 64;
    const uint32_t lane = threadIdx.x, h = blockIdx.x, t = blockIdx.y, b = blockIdx.z;
    const uint32_t kvh = h / (g.a.heads_q / g.heads);
    const int32_t seq = g.a.seqs[b];
    const bool there = seq >= 0 && (uint32_t)seq < g.max_seqs;
    int32_t nodes = there ? (int32_t)g.a.nodes : 0, ctx = 0;
    if (there) {
        if (g.a.tree_nodes != nullptr)
            nodes = min(max(g.a.tree_nodes[b], 0), nodes);
        ctx = min(max(g.lens[seq], 0), (int32_t)(g.max_pages * g.page_tokens));
    }
    if ((int32_t)t >= nodes)
        ctx = 0, nodes = 0;
    const T *qp = (const T *)g.a.q + b * g.a.q_stride[0] + t * g.a.q_stride[1] + h * g.a.q_stride[2];
    float q[R], o[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
        q[r] = lane + 64 * r < D ? to_float(qp[lane + 64 * r]) : 0.f;
        o[r] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    const uint32_t words = (g.a.nodes + 63) / 64;
    for (int32_t j = 0; j < ctx + nodes; j++) {
        const T *kp, *vp;
        if (j < ctx) {
            uint32_t page = (uint32_t)g.table[(uint64_t)seq * g.max_pages + j / g.page_tokens];
            page = page < g.num_pages ? page : 0;
            const uint64_t at = page * g.page_stride + (j % g.page_tokens) * g.token_step + kvh * g.head_step;
            kp = (const T *)(g.k_cache + at);
            vp = (const T *)(g.v_cache + at);
        } else {
            const uint32_t u = j - ctx;
            const bool sees = g.a.mask == nullptr ? u <= t
                                                  : (g.a.mask[((uint64_t)b * g.a.nodes + t) * words + u / 64] >> (u % 64)) & 1;
            if (!sees)
                continue;
            kp = (const T *)g.a.k + b * g.a.k_stride[0] + u * g.a.k_stride[1] + kvh * g.a.k_stride[2];
            vp = (const T *)g.a.v + b * g.a.v_stride[0] + u * g.a.v_stride[1] + kvh * g.a.v_stride[2];
        }
        float x = 0.f;
#pragma unroll
        for (int r = 0; r < R; r++)
            if (lane + 64 * r < D)
                x += q[r] * to_float(kp[lane + 64 * r]);
#pragma unroll
        for (int d = 32; d > 0; d >>= 1)
            x += __shfl_xor(x, d);
        x *= g.a.scale;
        const float top = fmaxf(m, x), base = top == -INFINITY ? 0.f : top;
        const float keep = expf(m - base), p = expf(x - base);
        m = top;
        l = l * keep + p;
#pragma unroll
        for (int r = 0; r < R; r++)
            if (lane + 64 * r < D)
                o[r] = o[r] * keep + p * to_float(vp[lane + 64 * r]);
    }
    T *op = (T *)g.a.out + b * g.a.out_stride[0] + t * g.a.out_stride[1] + h * g.a.out_stride[2];
#pragma unroll
    for (int r = 0; r < R; r++)
        if (lane + 64 * r < D)
            from_float(l == 0.f ? 0.f : o[r] / l, &op[lane + 64 * r]);
    if (g.a.lse != nullptr && lane == 0)
        g.a.lse[((uint64_t)b * g.a.nodes + t) * g.a.heads_q + h] = l == 0.f ? -INFINITY : m + logf(l);
}

uint64_t tree_attention_workspace(const tb_tree_attn &, uint32_t, int) { return 16; }

hipError_t launch_tree_attention(const tb_tree_attn &a, const tb_cache &c, hipStream_t stream) {
    AttnArgs g;
    g.a = a;
    g.k_cache = static_cast<const uint8_t *>(c.pools[a.k_pool]);
    g.v_cache = static_cast<const uint8_t *>(c.pools[a.v_pool]);
    g.table = c.table;
    g.lens = c.lens;
    g.page_stride = c.page_stride;
    const bool token_major = c.layout == TB_CACHE_TOKEN_MAJOR;
    g.token_step = token_major ? (uint64_t)c.heads * c.head_bytes : c.head_bytes;
    g.head_step = token_major ? c.head_bytes : (uint64_t)c.page_tokens * c.head_bytes;
    g.num_pages = c.num_pages;
    g.page_tokens = c.page_tokens;
    g.max_seqs = c.max_seqs;
    g.max_pages = c.max_pages;
    g.heads = c.heads;
    const dim3 grid(a.heads_q, a.nodes, a.batch);
    const bool bf = a.dtype == TB_BF16;
    switch (a.head_dim) {
    case 64: return launch(bf ? tree_attention_kernel<__hip_bfloat16, 64> : tree_attention_kernel<__half, 64>, grid, 64, stream, nullptr, g);
    case 96: return launch(bf ? tree_attention_kernel<__hip_bfloat16, 96> : tree_attention_kernel<__half, 96>, grid, 64, stream, nullptr, g);
    case 128: return launch(bf ? tree_attention_kernel<__hip_bfloat16, 128> : tree_attention_kernel<__half, 128>, grid, 64, stream, nullptr, g);
    case 256: return launch(bf ? tree_attention_kernel<__hip_bfloat16, 256> : tree_attention_kernel<__half, 256>, grid, 64, stream, nullptr, g);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace tbk
