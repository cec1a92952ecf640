/*
 * serve_check.c -- the serving step's C ABI (include/tb_serve.h) used from plain
 * C11: device memory from the HIP runtime's C API, no Python, no torch.
 *
 * Calls every entry point of the header: a prompt is appended to a cache held in
 * 4 bits (numbers that it holds exactly) and read back, as elements and as bytes;
 * two drafted tokens attend to it through a window with a sink, with all keys
 * equal, so that each output is a mean of values; and the two are verified against
 * distributions that accept the first and reject the second.  Prints "serve ok" and
 * exits 0 on success.
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <hip/hip_runtime_api.h>

#include "tb.h"
#include "tb_serve.h"

#define CHECK(x)                                                              \
    do {                                                                      \
        if (!(x)) {                                                           \
            fprintf(stderr, "line %d: %s (%s)\n", __LINE__, #x, tb_last_hip_error()); \
            return 1;                                                         \
        }                                                                     \
    } while (0)

enum { PAGES = 12, PT = 4, HEADS = 2, DIM = 64, HB = TB_FP4_HEAD_BYTES(DIM), SEQS = 4, ROW = 6, N = 10, NODES = 3, HQ = 4, VOCAB = 5 };

static void *dev(size_t bytes, const void *from) {
    void *p = NULL;
    if (hipMalloc(&p, bytes ? bytes : 1) != hipSuccess)
        return NULL;
    if (from != NULL ? hipMemcpy(p, from, bytes, hipMemcpyHostToDevice) : hipMemset(p, 0, bytes))
        return NULL;
    return p;
}

/* bfloat16 of a number that it holds exactly, and the way back */
static uint16_t bf(float x) {
    uint32_t u;
    memcpy(&u, &x, 4);
    return (uint16_t)(u >> 16);
}
static float fb(uint16_t x) {
    const uint32_t u = (uint32_t)x << 16;
    float f;
    memcpy(&f, &u, 4);
    return f;
}

/* token i's value */
static const float value[N] = {0.5f, 1, 1.5f, 2, 3, 4, 6, 12, 24, 48};

int main(void) {
    static uint16_t rows[2][N][HEADS * DIM], back[2][N][HEADS * DIM], drafted[2][NODES][HEADS * DIM], q[NODES * HQ * DIM],
        got[NODES][HQ][DIM];
    static uint8_t raw[2][N][HEADS][HB];
    const size_t pool = (size_t)PAGES * PT * HEADS * HB;
    uint64_t bytes = 0;
    hipStream_t s;
    CHECK(HB == 36 && hipStreamCreate(&s) == hipSuccess);
    CHECK(tb_cache_scratch_bytes(PAGES, SEQS, &bytes) == TB_OK);
    const void *pools[2] = {dev(pool, NULL), dev(pool, NULL)};
    tb_cache c;
    memset(&c, 0, sizeof c);
    c.pools = pools;
    c.npools = 2;
    c.layout = TB_CACHE_HEAD_MAJOR;
    c.num_pages = PAGES;
    c.page_tokens = PT;
    c.heads = HEADS;
    c.head_bytes = HB;
    c.page_stride = PT * HEADS * HB;
    c.max_seqs = SEQS;
    c.max_pages = ROW;
    c.table = dev(SEQS * ROW * 4, NULL);
    c.lens = dev(SEQS * 4, NULL);
    c.refs = dev(PAGES * 4, NULL);
    c.free_list = dev(PAGES * 4, NULL);
    c.counts = dev(16, NULL);
    c.scratch = dev(bytes, NULL);
    CHECK(tb_cache_init(&c, s) == TB_OK);

    int32_t seq[N], pos[N], one = 1, ten = N;
    for (int i = 0; i < N; i++) {
        seq[i] = 1;
        pos[i] = i;
        for (int e = 0; e < HEADS * DIM; e++) {
            rows[0][i][e] = bf(1);
            rows[1][i][e] = bf(value[i]);
        }
    }
    int32_t *d_one = dev(4, &one), *d_ten = dev(4, &ten), *d_seq = dev(sizeof seq, seq), *d_pos = dev(sizeof pos, pos);
    CHECK(hipDeviceSynchronize() == hipSuccess);
    CHECK(tb_page_resize(&c, d_one, d_ten, 1, s) == TB_OK);
    CHECK(tb_fp4_append(&c, TB_BF16, DIM, dev(sizeof rows, rows), N, sizeof rows[0][0], sizeof rows[0], d_seq, d_pos, NULL, N, s) == TB_OK);
    void *d_back = dev(sizeof back, NULL), *d_raw = dev(sizeof raw, NULL);
    CHECK(hipDeviceSynchronize() == hipSuccess);
    CHECK(tb_fp4_read(&c, TB_BF16, DIM, 0, 2, d_back, sizeof back[0][0], sizeof back[0], d_seq, d_pos, N, s) == TB_OK);
    CHECK(tb_page_read(&c, 0, 2, d_raw, HEADS * HB, sizeof raw[0], d_seq, d_pos, N, s) == TB_OK);
    CHECK(hipStreamSynchronize(s) == hipSuccess);
    CHECK(hipMemcpy(back, d_back, sizeof back, hipMemcpyDeviceToHost) == hipSuccess);
    CHECK(hipMemcpy(raw, d_raw, sizeof raw, hipMemcpyDeviceToHost) == hipSuccess);
    CHECK(memcmp(back, rows, sizeof back) == 0);
    /* 1 is 4 times 2^-2: code 6, byte 125 */
    CHECK(raw[0][3][1][0] == 0x66 && raw[0][3][1][31] == 0x66 && raw[0][3][1][32] == 125 && raw[0][3][1][33] == 125);
    CHECK(raw[0][3][1][34] == 0 && raw[0][3][1][35] == 0);

    /* three nodes, a chain: the root of value 20 and two drafted ones; window 4, one sink: node t sees token 0, the
       last 3 - t tokens and the nodes up to itself */
    for (int i = 0; i < NODES; i++)
        for (int e = 0; e < HEADS * DIM; e++) {
            drafted[0][i][e] = bf(1);
            drafted[1][i][e] = bf(20.f * (float)(i + 1));
        }
    for (int e = 0; e < NODES * HQ * DIM; e++)
        q[e] = bf(1);
    tb_tree_attn a;
    memset(&a, 0, sizeof a);
    uint16_t *kv = dev(sizeof drafted, drafted);
    a.q = dev(sizeof q, q);
    a.k = kv;
    a.v = kv + NODES * HEADS * DIM;
    a.out = dev(sizeof q, NULL);
    a.q_stride[1] = a.out_stride[1] = HQ * DIM;
    a.q_stride[2] = a.out_stride[2] = DIM;
    a.k_stride[1] = a.v_stride[1] = HEADS * DIM;
    a.k_stride[2] = a.v_stride[2] = DIM;
    a.seqs = d_one;
    a.batch = 1;
    a.nodes = NODES;
    a.heads_q = HQ;
    a.head_dim = DIM;
    a.dtype = TB_BF16;
    a.v_pool = 1;
    a.scale = 1.f / 64;
    const tb_attn_view view = {4, 1, NULL, 1};
    CHECK(tb_view_attention_workspace(&a, &view, &c, &a.workspace_bytes) == TB_OK);
    a.workspace = dev(a.workspace_bytes, NULL);
    CHECK(hipDeviceSynchronize() == hipSuccess);
    CHECK(tb_view_attention(&a, &view, &c, s) == TB_OK);
    CHECK(hipStreamSynchronize(s) == hipSuccess);
    CHECK(hipMemcpy(got, a.out, sizeof got, hipMemcpyDeviceToHost) == hipSuccess);
    for (int t = 0; t < NODES; t++) {
        double sum = value[0];
        for (int i = N - 3 + t; i < N; i++)
            sum += value[i];
        for (int u = 0; u <= t; u++)
            sum += 20 * (u + 1);
        const double mean = sum / 5;
        for (int h = 0; h < HQ; h++)
            for (int e = 0; e < DIM; e++)
                CHECK(fabs(fb(got[t][h][e]) - mean) <= mean / 128);
    }

    /* token 2, drawn with 0.5 where the target has 0.4: accepted below 0.8; then token 4, drawn with 1 where the
       target has 0.25: rejected, and the next token comes from the other 0.75 */
    const float p[NODES][VOCAB] = {{0.3f, 0.3f, 0.4f, 0, 0}, {0, 0.5f, 0.25f, 0, 0.25f}, {1, 0, 0, 0, 0}};
    const float d[NODES][VOCAB] = {{0, 0.5f, 0.5f, 0, 0}, {0, 0, 0, 0, 1}, {1, 0, 0, 0, 0}};
    const float u[NODES] = {0.7f, 0.75f, 0.5f};
    const int32_t proposed[NODES] = {0, 2, 4};
    int32_t out[NODES], count, token, list[3][NODES], lens;
    tb_verify v;
    memset(&v, 0, sizeof v);
    v.probs = dev(sizeof p, p);
    v.draft_probs = dev(sizeof d, d);
    v.probs_stride[1] = v.draft_stride[1] = VOCAB;
    v.tokens = dev(sizeof proposed, proposed);
    v.uniform = dev(sizeof u, u);
    v.batch = 1;
    v.nodes = NODES;
    v.vocab = VOCAB;
    v.dtype = TB_FP32;
    v.count = dev(4, NULL);
    v.path = dev(sizeof out, NULL);
    v.token = dev(4, NULL);
    v.seqs = d_one;
    v.lens = c.lens;
    v.max_seqs = SEQS;
    v.new_lens = dev(4, NULL);
    v.append_seqs = dev(sizeof out, NULL);
    v.append_positions = dev(sizeof out, NULL);
    v.append_index = dev(sizeof out, NULL);
    CHECK(tb_verify_workspace(&v, &v.workspace_bytes) == TB_OK);
    v.workspace = dev(v.workspace_bytes, NULL);
    CHECK(hipDeviceSynchronize() == hipSuccess);
    CHECK(tb_verify_drafts(&v, s) == TB_OK);
    CHECK(hipStreamSynchronize(s) == hipSuccess);
    CHECK(hipMemcpy(out, v.path, sizeof out, hipMemcpyDeviceToHost) == hipSuccess);
    CHECK(hipMemcpy(&count, v.count, 4, hipMemcpyDeviceToHost) == hipSuccess);
    CHECK(hipMemcpy(&token, v.token, 4, hipMemcpyDeviceToHost) == hipSuccess);
    CHECK(hipMemcpy(&lens, v.new_lens, 4, hipMemcpyDeviceToHost) == hipSuccess);
    CHECK(hipMemcpy(list[0], v.append_seqs, sizeof out, hipMemcpyDeviceToHost) == hipSuccess);
    CHECK(hipMemcpy(list[1], v.append_positions, sizeof out, hipMemcpyDeviceToHost) == hipSuccess);
    CHECK(hipMemcpy(list[2], v.append_index, sizeof out, hipMemcpyDeviceToHost) == hipSuccess);
    CHECK(count == 2 && out[0] == 0 && out[1] == 1 && out[2] == -1 && token == 2 && lens == N + 2);
    CHECK(list[0][0] == 1 && list[0][1] == 1 && list[0][2] == -1 && list[1][0] == N && list[1][1] == N + 1);
    CHECK(list[2][0] == 0 && list[2][1] == 1 && list[2][2] == 0);
    CHECK(tb_verify_drafts(NULL, s) == TB_ERR_INVALID);
    printf("serve ok\n");
    return 0;
}
