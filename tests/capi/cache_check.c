/*
 * cache_check.c -- the paged cache's C ABI (include/tb_cache.h) used from plain
 * C11: device memory from the HIP runtime's C API, no Python, no torch.
 *
 * A consumer-side check of the boundary that calls every entry point of the
 * header once, in the order a serving step would: an empty cache, a prompt
 * appended, a fork, attention of two drafted tokens over both sequences (with
 * all keys equal, so that each output is the mean of the values and the
 * logarithm of the sum is known in closed form), pages copied to a second
 * cache, sequences freed and the rest compacted.  Prints "cache ok" and exits 0 on
 * success.
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <hip/hip_runtime_api.h>

#include "tb.h"
#include "tb_cache.h"

#define CHECK(x)                                                              \
    do {                                                                      \
        if (!(x)) {                                                           \
            fprintf(stderr, "line %d: %s (%s)\n", __LINE__, #x, tb_last_hip_error()); \
            return 1;                                                         \
        }                                                                     \
    } while (0)

enum { PAGES = 12, PT = 4, HEADS = 2, DIM = 64, SEQS = 4, ROW = 6, N = 10, NODES = 2, HQ = 4 };

static void *dev(size_t bytes, const void *from) {
    void *p = NULL;
    if (hipMalloc(&p, bytes ? bytes : 1) != hipSuccess)
        return NULL;
    if (from != NULL ? hipMemcpy(p, from, bytes, hipMemcpyHostToDevice) : hipMemset(p, 0, bytes))
        return NULL;
    return p;
}

/* bfloat16 of a number that it holds exactly */
static uint16_t bf(float x) {
    uint32_t u;
    memcpy(&u, &x, 4);
    return (uint16_t)(u >> 16);
}

int main(void) {
    static uint16_t rows[2][N][HEADS * DIM], drafted[2][NODES][HEADS * DIM], q[2 * NODES * HQ * DIM], got[2][NODES][HQ][DIM];
    static uint16_t page[PT][HEADS][DIM];
    static float lse[2][NODES][HQ];
    const size_t pool = (size_t)PAGES * PT * HEADS * DIM * 2;
    uint64_t bytes = 0;
    hipStream_t s;
    CHECK(hipStreamCreate(&s) == hipSuccess);
    CHECK(tb_cache_scratch_bytes(PAGES, SEQS, &bytes) == TB_OK);
    const void *pools[2] = {dev(pool, NULL), dev(pool, NULL)}, *other[2] = {dev(pool, NULL), dev(pool, NULL)};
    tb_cache c;
    memset(&c, 0, sizeof c);
    c.pools = pools;
    c.npools = 2;
    c.layout = TB_CACHE_TOKEN_MAJOR;
    c.num_pages = PAGES;
    c.page_tokens = PT;
    c.heads = HEADS;
    c.head_bytes = DIM * 2;
    c.page_stride = PT * HEADS * DIM * 2;
    c.max_seqs = SEQS;
    c.max_pages = ROW;
    c.table = dev(SEQS * ROW * 4, NULL);
    c.lens = dev(SEQS * 4, NULL);
    c.refs = dev(PAGES * 4, NULL);
    c.free_list = dev(PAGES * 4, NULL);
    c.counts = dev(16, NULL);
    c.scratch = dev(bytes, NULL);
    CHECK(tb_cache_init(&c, s) == TB_OK);

    /* a prompt of ten tokens: keys all one, the value of token i is i */
    int32_t seq[N], pos[N], list[SEQS], zero[SEQS] = {0};
    for (int i = 0; i < N; i++) {
        seq[i] = 1;
        pos[i] = i;
        for (int e = 0; e < HEADS * DIM; e++) {
            rows[0][i][e] = bf(1);
            rows[1][i][e] = bf((float)i);
        }
    }
    int32_t one = 1, ten = N, two = 2, first = 0, last = PAGES - 1;
    int32_t *d_one = dev(4, &one), *d_ten = dev(4, &ten), *d_two = dev(4, &two), *d_first = dev(4, &first), *d_last = dev(4, &last);
    CHECK(hipDeviceSynchronize() == hipSuccess);
    CHECK(tb_page_resize(&c, d_one, d_ten, 1, s) == TB_OK);
    CHECK(tb_page_append(&c, dev(sizeof rows, rows), N, HEADS * DIM * 2, sizeof rows[0], dev(sizeof seq, seq), dev(sizeof pos, pos), NULL,
                         N, s) == TB_OK);
    CHECK(tb_page_fork(&c, d_one, d_two, 1, s) == TB_OK);

    /* two drafted tokens a sequence: keys one, values 20 and 40; q = 1, scale 1/64: every score is 1 */
    for (int i = 0; i < NODES; i++)
        for (int e = 0; e < HEADS * DIM; e++) {
            drafted[0][i][e] = bf(1);
            drafted[1][i][e] = bf(20.f * (float)(i + 1));
        }
    for (int e = 0; e < 2 * NODES * HQ * DIM; e++)
        q[e] = bf(1);
    tb_tree_attn a;
    memset(&a, 0, sizeof a);
    uint16_t *kv = dev(sizeof drafted, drafted);
    list[0] = 1;
    list[1] = 2;
    a.q = dev(sizeof q, q);
    a.k = kv;
    a.v = kv + NODES * HEADS * DIM;
    a.out = dev(sizeof q, NULL);
    a.lse = dev(sizeof lse, NULL);
    a.q_stride[0] = a.out_stride[0] = NODES * HQ * DIM;
    a.q_stride[1] = a.out_stride[1] = HQ * DIM;
    a.q_stride[2] = a.out_stride[2] = DIM;
    a.k_stride[1] = a.v_stride[1] = HEADS * DIM; /* both sequences draft the same: stride 0 between them */
    a.k_stride[2] = a.v_stride[2] = DIM;
    a.seqs = dev(8, list);
    a.batch = 2;
    a.nodes = NODES;
    a.heads_q = HQ;
    a.head_dim = DIM;
    a.dtype = TB_BF16;
    a.v_pool = 1;
    a.scale = 1.f / 64;
    CHECK(tb_tree_attention_workspace(&a, &c, &a.workspace_bytes) == TB_OK);
    a.workspace = dev(a.workspace_bytes, NULL);
    CHECK(hipDeviceSynchronize() == hipSuccess);
    CHECK(tb_tree_attention(&a, &c, s) == TB_OK);
    CHECK(hipStreamSynchronize(s) == hipSuccess);
    CHECK(hipMemcpy(got, a.out, sizeof got, hipMemcpyDeviceToHost) == hipSuccess);
    CHECK(hipMemcpy(lse, a.lse, sizeof lse, hipMemcpyDeviceToHost) == hipSuccess);
    for (int b = 0; b < 2; b++)
        for (int t = 0; t < NODES; t++)
            for (int h = 0; h < HQ; h++) {
                const double n = N + t + 1, mean = (45.0 + 20 + 40 * t) / n;
                CHECK(fabs(lse[b][t][h] - (1 + log(n))) < 1e-5);
                for (int e = 0; e < DIM; e++) {
                    uint32_t u = (uint32_t)got[b][t][h][e] << 16;
                    float x;
                    memcpy(&x, &u, 4);
                    CHECK(fabs(x - mean) <= mean / 128);
                }
            }

    /* the prompt's first page to another cache's last one */
    tb_cache d = c;
    d.pools = other;
    int32_t table[SEQS * ROW], lens[SEQS], counts[4];
    CHECK(hipMemcpy(table, c.table, sizeof table, hipMemcpyDeviceToHost) == hipSuccess);
    CHECK(table[ROW] == 0 && table[2 * ROW] == 0 && table[ROW + 2] != table[2 * ROW + 2]);
    CHECK(tb_page_copy(&d, &c, d_last, d_first, 1, s) == TB_OK);
    CHECK(hipStreamSynchronize(s) == hipSuccess);
    CHECK(hipMemcpy(page, (const char *)other[1] + last * c.page_stride, sizeof page, hipMemcpyDeviceToHost) == hipSuccess);
    CHECK(page[3][1][DIM - 1] == bf(3));

    /* the prompt is freed: the fork keeps the shared pages and its own, which move together */
    CHECK(tb_page_resize(&c, d_one, dev(4, zero), 1, s) == TB_OK);
    CHECK(tb_page_compact(&c, s) == TB_OK);
    CHECK(hipStreamSynchronize(s) == hipSuccess);
    CHECK(hipMemcpy(table, c.table, sizeof table, hipMemcpyDeviceToHost) == hipSuccess);
    CHECK(hipMemcpy(lens, c.lens, sizeof lens, hipMemcpyDeviceToHost) == hipSuccess);
    CHECK(hipMemcpy(counts, c.counts, sizeof counts, hipMemcpyDeviceToHost) == hipSuccess);
    CHECK(lens[1] == 0 && lens[2] == N && counts[0] == PAGES - 3 && counts[1] == 0 && table[2 * ROW + 2] == 2);
    CHECK(hipMemcpy(page, (const char *)pools[1] + 2 * c.page_stride, sizeof page, hipMemcpyDeviceToHost) == hipSuccess);
    CHECK(page[0][0][0] == bf(8) && page[1][0][0] == bf(9));
    CHECK(tb_page_fork(&c, NULL, d_two, 1, s) == TB_ERR_INVALID);
    printf("cache ok\n");
    return 0;
}
