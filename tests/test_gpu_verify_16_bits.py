"""GPU tests of tb_verify_drafts with trees whose probabilities are in 16 bits, as test_gpu_verify.py has them in 32: over
vocabularies on both sides of what a wave, a workgroup and a run of loads take, captured, and on two streams."""
import pytest
import torch

from gpu_util import note, require_gpu
from serve_model import verify
from test_gpu_verify import case, check, ints

pytestmark = pytest.mark.gpu
DTYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])


@DTYPES
@pytest.mark.parametrize("drafted", [True, False], ids=["drawn", "chosen"])
@pytest.mark.parametrize("t,kids", [(13, 3), (64, 4), (70, 0), (40, 39)])
@pytest.mark.parametrize("vocab", [50, 4097, 8200])
def test_trees(t, kids, vocab, drafted, dtype):
    note(f"verify trees of {t} with {kids} children, vocabulary {vocab}, {dtype}, drafted {drafted}")
    g = torch.Generator().manual_seed(t + vocab)
    probs, draft, parents, tokens, u = case(g, 4, t, vocab, kids, drafted, dtype)
    check(probs, tokens, u, parents, draft, nodes=[t, t - t // 3, 1, 0], what="ragged")
    check(probs, tokens, torch.full_like(u, 1 - 2.0 ** -24), parents, draft, what="hardly anything is accepted")


@DTYPES
@pytest.mark.parametrize("b,t,kids,vocab", [(2, 9, 4, 65537), (1, 7, 6, 131073), (260, 4, 3, 9001), (129, 4, 2, 16385)])
def test_large_vocabularies_and_many_sequences(b, t, kids, vocab, dtype):
    """Drawn siblings of which most are rejected: the rows are summed again for each."""
    note(f"verify {b} trees of {t}, vocabulary {vocab}, {dtype}")
    g = torch.Generator().manual_seed(vocab)
    probs, draft, parents, tokens, u = case(g, b, t, vocab, kids, True, dtype, apart=2.0)
    check(probs, tokens, u, parents, draft)
    check(probs, tokens, 1 - u / 8, parents, draft, what="most are rejected")
    check(probs, tokens, u, parents, None, what="taken as chosen")


@DTYPES
def test_unaligned_rows(dtype):
    note(f"verify with rows at odd places, {dtype}")
    g = torch.Generator().manual_seed(2)
    probs, draft, parents, tokens, u = case(g, 3, 6, 5001, 2, True, dtype)
    require_gpu()
    room = torch.zeros(6, 3, 2, 5009, dtype=dtype, device="cuda")
    ps, ds = room[:, :, 0, 3:5004].transpose(0, 1), room[:, :, 1, 7:5008].transpose(0, 1)
    ps.copy_(probs)
    ds.copy_(draft)
    check(ps, tokens, u, parents, ds)
    check(ps, tokens, u, parents, None)


@DTYPES
def test_a_captured_call_is_replayed(dtype):
    note(f"verify captured, {dtype}")
    require_gpu()
    from copy_reduce_amd.torch_api import verify_drafts
    g = torch.Generator().manual_seed(3)
    shape = (3, 8, 33000, 3, True, dtype)
    probs, draft, parents, tokens, u = case(g, *shape)
    held = [probs.cuda(), draft.cuda(), ints(parents), ints(tokens), u.cuda()]

    def call():
        return verify_drafts(held[0], held[3], held[4], parents=held[2], draft_probs=held[1])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = call()
    for turn in range(4):
        new = case(g, *shape)
        for a, n in zip(held, new):
            a.copy_(n)
        graph.replay()
        want = verify(new[0], new[3], new[4], new[2], new[1])
        for i, (count, path, token) in enumerate(want):
            assert (int(r.count[i]), r.path[i].tolist(), int(r.token[i])) == (count, path + [-1] * (8 - count), token), f"turn {turn}"
        eager = call()
        assert all(torch.equal(p, q) for p, q in zip(eager[:3], r[:3]))
        torch.cuda.synchronize()


@DTYPES
def test_two_streams_at_once(dtype):
    note(f"verify on two streams, {dtype}")
    require_gpu()
    from copy_reduce_amd.torch_api import verify_drafts
    g = torch.Generator().manual_seed(4)
    sets = [case(g, 5, 7, 60000, 3, True, dtype) for _ in range(2)]
    on = [[x[0].cuda(), ints(x[3]), x[4].cuda(), ints(x[2]), x[1].cuda()] for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[verify_drafts(*x, stream=s) for x, s in zip(on, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    for i, x in enumerate(sets):
        want = verify(x[0], x[3], x[4], x[2], x[1])
        for r in got:
            for j, (count, path, token) in enumerate(want):
                assert (int(r[i].count[j]), r[i].path[j].tolist(), int(r[i].token[j])) == (count, path + [-1] * (7 - count), token)
