"""GPU tests of tb_tree_attention's probabilities at the ends of their range: one key far above all others, whose small
weights together decide the output, and weights as large as the kernels let them become.

All scores are known exactly (q is a unit vector, keys are multiples of it), so the definition is a sum of two terms.
Bounds as derived in test_gpu_tree_attention.py (u the half step of the element type, E = 2^-24), with
one term sharper: an fp16 weight is taken times 2^7, so a subnormal one is off by 2^-25 / 2^7 = 2^-32 of a sum of at
least 1."""
import math

import pytest
import torch

from gpu_util import note, require_gpu

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
V = 57344.0          # 7 x 2^13: exact in both types
DTYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def scored(scores, value, dim, dtype, room, nodes, batch):
    """Context tokens with these scores and values (one row, attended to by the whole batch) and a chain of
    nodes of score 0 and value V: what tree_attention returns, in 64 bits."""
    require_gpu()
    from copy_reduce_amd.torch_api import PagedCache, tree_attention
    n, pt = len(scores), 16
    pages = -(-n // pt)
    kv = torch.zeros(2, pages * pt, 1, dim, dtype=torch.float64)
    kv[0, :n, 0, 0] = scores
    kv[1, :n, 0] = value[:, None]
    assert torch.equal(kv.to(dtype).double(), kv)
    c = PagedCache(kv.to(dtype).view(2, pages, pt, 1, dim).cuda(), pt, 1, max(pages, -(-room // pt)))
    c.resize(ints([0]), ints([n]))
    c.table[0, :pages] = torch.arange(pages, dtype=torch.int32, device="cuda")
    q = torch.zeros(batch, nodes, 1, dim, dtype=dtype)
    q[..., 0] = 1
    k, v = torch.zeros_like(q), torch.full_like(q, V)
    out, lse = tree_attention(q.cuda(), k.cuda(), v.cuda(), c, 0, ints([0] * batch), scale=1.0)
    return out.double().cpu(), lse.double().cpu()


def check(got, scores, value, dim, dtype, nodes):
    out, lse = got
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    u, s = torch.finfo(dtype).eps / 2, float(scores.abs().max())
    w = (2 * dim + 8) * E * s + 8 * E
    for t in range(nodes):
        n = len(scores) + t + 1
        x = torch.cat([scores, torch.zeros(t + 1, dtype=torch.float64)])
        y = torch.cat([value, torch.full((t + 1,), V, dtype=torch.float64)])
        z = torch.logsumexp(x, 0)
        want = float((torch.exp(x - z) * y).sum())      # values are not negative: A of the bound is the output
        tol = want * (2 * u + 2 * w + 2 * (n + 64) * E)
        if dtype == torch.float16:
            tol += n * 2.0 ** -32 * V + 2.0 ** -25
        worst = float((out[:, t] - want).abs().max())
        assert worst <= tol, f"node {t}: off by {worst:.3g} of {want:.6g}, at most {tol:.3g}"
        assert float((lse[:, t] - z).abs().max()) <= w + (n + 64) * E + 4 * E * abs(float(z))


@DTYPES
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("nodes", [1, 20], ids=["few rows", "many rows"])
@pytest.mark.parametrize("room,batch", [(0, 2), (8192, 1000)], ids=["whole", "shares"])
@pytest.mark.parametrize("place", [0, 350, 699])
def test_small_weights_count_together(place, room, batch, nodes, dim, dtype):
    """700 keys 17.5 below one of value 0: weights of 2^-25.2, together a share of 1.7e-5 that is the whole output."""
    note(f"tree attention, a key far above 700, at {place}, dim {dim} {dtype} {nodes} nodes {batch} sequences")
    scores, value = torch.zeros(701, dtype=torch.float64), torch.full((701,), V, dtype=torch.float64)
    scores[place], value[place] = 17.5, 0
    check(scored(scores, value, dim, dtype, room, nodes, batch), scores, value, dim, dtype, nodes)


@DTYPES
@pytest.mark.parametrize("nodes", [1, 20], ids=["few rows", "many rows"])
def test_small_weights_over_a_long_context(nodes, dtype):
    """131,072 keys 18 below one of value 0: their share is 0.2 %."""
    note(f"tree attention, a key far above 131,072, {dtype} {nodes} nodes")
    n = 131073
    scores, value = torch.zeros(n, dtype=torch.float64), torch.full((n,), V, dtype=torch.float64)
    scores[0], value[0] = 18.0, 0
    check(scored(scores, value, 64, dtype, 0, nodes, 256), scores, value, 64, dtype, nodes)


@DTYPES
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("nodes", [1, 20], ids=["few rows", "many rows"])
@pytest.mark.parametrize("top", [5.5, 5.625, 11.0])
def test_large_weights_stay_finite(top, nodes, dim, dtype):
    """Scores that rise to just below, just above and far above what moves the running maximum (8 ln 2 = 5.545)."""
    note(f"tree attention, scores that rise by {top}, dim {dim} {dtype} {nodes} nodes")
    scores = torch.full((700,), top, dtype=torch.float64)
    scores[:256] = 0          # each wave's first keys
    value = torch.full((700,), V, dtype=torch.float64)
    value[1::2] = V / 2
    check(scored(scores, value, dim, dtype, 0, nodes, 2), scores, value, dim, dtype, nodes)
