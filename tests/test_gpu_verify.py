"""GPU tests of tb_verify_drafts against the walk as its header tells it, in 64 bits.  All outputs are whole numbers and have
to be equal: random numbers come from inputs, and none of them lies within the sums' rounding (some 1e-13) of a border, which
for the few thousand draws here has a chance of about 1e-6."""
import pytest
import torch

from gpu_util import note, require_gpu
from serve_model import verify

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.as_tensor(v, dtype=torch.int32).cuda()


def check(probs, tokens, uniform, parents=None, draft=None, nodes=None, what="", **kw):
    require_gpu()
    from copy_reduce_amd.torch_api import verify_drafts
    r = verify_drafts(probs.cuda() if not probs.is_cuda else probs, ints(tokens), uniform.cuda(), parents=None if parents is None else ints(parents),
                      draft_probs=None if draft is None else draft.cuda() if not draft.is_cuda else draft, nodes=None if nodes is None else ints(nodes), **kw)
    want = verify(probs.cpu(), tokens, uniform, parents, None if draft is None else draft.cpu(), nodes)
    t = probs.shape[1]
    for i, (count, path, token) in enumerate(want):
        got = int(r.count[i]), r.path[i].tolist(), int(r.token[i])
        assert got == (count, path + [-1] * (t - len(path)), token), f"{what}: sequence {i}: {got}, not {(count, path, token)}"
    return r


def case(g, b, t, vocab, kids, drafted, dtype=torch.float32, sharp=2.0, apart=0.7):
    x = sharp * torch.randn(b, t, vocab, generator=g)
    probs = torch.softmax(x, 2).to(dtype)
    draft = torch.softmax(x + apart * torch.randn(b, t, vocab, generator=g), 2).to(dtype)
    parents = torch.zeros(b, t, dtype=torch.int64)
    for i in range(1, t):
        parents[:, i] = (i - 1) // kids if kids else (torch.rand(b, generator=g) * i).long()
    tokens = torch.zeros(b, t, dtype=torch.int64)
    for i in range(b):
        used = {}
        for u in range(1, t):
            p = int(parents[i, u])
            if drafted:
                tokens[i, u] = torch.multinomial(draft[i, p].float(), 1, generator=g)
            else:
                k = used.get(p, 0)
                used[p] = k + 1
                tokens[i, u] = torch.topk(draft[i, p].float(), min(k + 1, vocab)).indices[-1]
    return probs, draft if drafted else None, parents, tokens, torch.rand(b, t, generator=g)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab", [1, 2, 3, 31, 1000, 1023, 1024, 1025, 4099, 32003])
@pytest.mark.parametrize("drafted", [True, False], ids=["drawn", "chosen"])
def test_chains(vocab, dtype, drafted):
    note(f"verify chains, vocabulary {vocab}, {dtype}, drafted {drafted}")
    g = torch.Generator().manual_seed(vocab)
    for b, t in ((1, 1), (5, 2), (3, 7)):
        probs, draft, _, tokens, u = case(g, b, t, vocab, 1, drafted, dtype)
        check(probs, tokens, u, None, draft, what=f"{b} of {t}")


@pytest.mark.parametrize("drafted", [True, False], ids=["drawn", "chosen"])
@pytest.mark.parametrize("t,kids", [(4, 3), (13, 3), (64, 4), (65, 0), (200, 5), (130, 0), (100, 99)])
@pytest.mark.parametrize("vocab", [50, 2500])
def test_trees(t, kids, vocab, drafted):
    note(f"verify trees of {t} with {kids} children, vocabulary {vocab}, drafted {drafted}")
    g = torch.Generator().manual_seed(t)
    b = 4
    probs, draft, parents, tokens, u = case(g, b, t, vocab, kids, drafted)
    check(probs, tokens, u, parents, draft, nodes=[t, t - t // 3, 1, 0], what="ragged")
    check(probs, tokens, torch.full_like(u, 1 - 2.0 ** -24), parents, draft, what="hardly anything is accepted")
    check(probs, tokens, torch.zeros_like(u), parents, draft, what="everything with a chance is accepted")


def test_many_sequences_and_a_large_vocabulary():
    note("verify 300 chains; one of 2^20 + 3 entries")
    g = torch.Generator().manual_seed(3)
    probs, draft, _, tokens, u = case(g, 300, 3, 2100, 1, True)
    check(probs, tokens, u, None, draft)
    probs, draft, _, tokens, u = case(g, 1, 2, 2 ** 20 + 3, 1, True)
    check(probs, tokens, u, None, draft)


def test_long_chains():
    """Longer than a wave's nodes; the draft agrees with the target, so that paths are long."""
    note("verify chains of 1,000 and 4,096")
    g = torch.Generator().manual_seed(4)
    for t in (1000, 4096):
        probs, draft, _, tokens, u = case(g, 2, t, 16, 1, True, apart=0.0)
        u[1, t // 2] = 0.5
        draft[1, t // 2 - 1] = 0
        draft[1, t // 2 - 1, int(tokens[1, t // 2])] = 1.0   # drawn where the target hardly goes
        r = check(probs, tokens, u, None, draft)
        assert int(r.count[0]) == t


def test_greedy_targets_are_one_hot():
    """Temperature 0: a distribution with one entry accepts that token alone, whatever the random number."""
    note("verify one-hot targets")
    g = torch.Generator().manual_seed(5)
    probs = torch.nn.functional.one_hot(torch.randint(0, 500, (6, 9), generator=g), 500).float()
    best = probs.argmax(2)
    tokens = torch.cat([torch.zeros(6, 1, dtype=torch.int64), best[:, :-1]], 1)
    for i in range(5):
        tokens[i, i + 1] = (tokens[i, i + 1] + 1) % 500
    u = torch.rand(6, 9, generator=g)
    r = check(probs, tokens, u)
    assert r.count.tolist() == [1, 2, 3, 4, 5, 9]
    assert r.token.tolist() == [int(best[i, i]) for i in range(5)] + [int(best[5, 8])]


def test_children_that_take_all_there_is():
    """Nothing is left: the next token is drawn from the node's own distribution, as for equal distributions too."""
    note("verify with nothing left")
    probs = torch.tensor([[[0.25, 0.75, 0, 0], [0, 0, 1, 0], [0, 1, 0, 0]]])
    u = torch.tensor([[0.5, 0.9, 0.9999]])
    parents = torch.tensor([[0, 0, 0]])
    check(probs, torch.tensor([[0, 0, 1]]), u, parents, None, what="chosen: the second has all that is left")
    check(probs, torch.tensor([[0, 3, 2]]), u, parents, None, what="chosen where there is nothing")
    check(probs, torch.tensor([[0, 0, 0]]), u, parents, None, what="the same token twice")
    check(probs, torch.tensor([[0, 3, 3]]), u, parents, probs.clone(), what="equal distributions, a token without a chance")
    lower = probs.clone()
    lower[0, 0] = torch.tensor([0.2, 0.7, 0, 0])
    check(lower, torch.tensor([[0, 3, 2]]), u, parents, probs, what="below the draft everywhere")
    zero = torch.zeros_like(probs)
    r = check(zero, torch.tensor([[0, 1, 2]]), u, parents, None, what="no distribution")
    assert r.token.tolist() == [-1]


def test_nodes_that_are_passed_over():
    note("verify with wrong parents and tokens")
    g = torch.Generator().manual_seed(7)
    probs, draft, parents, tokens, u = case(g, 3, 12, 40, 2, True)
    parents[0, 3], parents[0, 4], parents[1, 1], parents[2, 11] = 3, 7, -1, 2 ** 31 - 1
    tokens[0, 1], tokens[1, 2], tokens[2, 5] = 40, -1, -2 ** 31
    check(probs, tokens, u, parents, draft)
    check(probs, tokens, u, parents, None)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -1.0])
def test_bad_probabilities_stay_within_the_outputs(bad):
    note(f"verify with {bad} among the probabilities and the random numbers")
    require_gpu()
    from copy_reduce_amd.torch_api import verify_drafts
    g = torch.Generator().manual_seed(8)
    probs, draft, parents, tokens, u = case(g, 4, 6, 3000, 2, True)
    probs[0, 0, 5], probs[1] = bad, bad
    draft[2, 0, 7] = bad
    u[3, 0] = bad
    for d in (draft.cuda(), None):
        r = verify_drafts(probs.cuda(), ints(tokens), u.cuda(), parents=ints(parents), draft_probs=d)
        assert bool(((r.token >= -1) & (r.token < 3000)).all()) and bool(((r.count >= 1) & (r.count <= 6)).all())
        assert bool(((r.path >= -1) & (r.path < 6)).all())


def test_strides_and_a_workspace_used_again():
    note("verify with strided probabilities")
    from copy_reduce_amd.torch_api import verify_drafts_workspace
    g = torch.Generator().manual_seed(9)
    probs, draft, parents, tokens, u = case(g, 3, 5, 777, 2, True)
    room = torch.zeros(5, 3, 2, 790, device="cuda")
    ps, ds = room[:, :, 0, 3:780].transpose(0, 1), room[:, :, 1, 13:].transpose(0, 1)
    ps.copy_(probs)
    ds.copy_(draft)
    ws = verify_drafts_workspace(ps)
    ws.fill_(255)
    check(ps, tokens, u, parents, ds, workspace=ws)
    check(ps, tokens, u, parents, None, workspace=ws)
    same = probs[:1, :1].expand(3, 5, 777)   # one row for all: strides of 0
    check(same.cuda()[:1, :1].expand(3, 5, 777), tokens, u, parents, ds, workspace=ws)


def test_lists_for_the_cache():
    note("verify with a cache's lists")
    require_gpu()
    from copy_reduce_amd.torch_api import PagedCache
    g = torch.Generator().manual_seed(10)
    cache = PagedCache(torch.zeros(2, 50, 8, 1, 8, dtype=torch.bfloat16, device="cuda"), 8, 6, 10)
    cache.resize(ints([0, 1, 2, 3]), ints([5, 17, 30, 1]))
    probs, draft, parents, tokens, u = case(g, 5, 7, 300, 2, True)
    seqs = [2, -1, 0, 9, 3]
    r = check(probs, tokens, u, parents, draft, nodes=[7, 0, 0, 0, 7], cache=cache, seqs=ints(seqs))   # as out of range sequences count
    had = [30, 0, 5, 0, 1]
    for i in range(5):
        n = int(r.count[i])
        assert int(r.lens[i]) == had[i] + n
        at = slice(7 * i, 7 * i + 7)
        assert r.append_seqs[at].tolist() == [seqs[i]] * n + [-1] * (7 - n)
        assert r.append_positions[at].tolist() == [had[i] + k for k in range(n)] + [0] * (7 - n)
        assert r.append_index[at].tolist() == [7 * i + k for k in r.path[i, :n].tolist()] + [0] * (7 - n)
    full = check(probs[:2], tokens[:2], u[:2], parents[:2], draft[:2], nodes=[7, 0], cache=cache, seqs=ints([2, -1]))
    assert full.lens.tolist()[1] == 0


def test_the_tokens_are_distributed_as_the_target_s():
    """20,000 sequences of one chain: the next token after the root, drafted or drawn, has the target's distribution.  Each
    of 8 shares has a standard deviation of at most 0.5 / sqrt(20000) = 0.0036; five of them are allowed."""
    note("verify: distribution of what is emitted")
    g = torch.Generator().manual_seed(11)
    n, vocab = 20000, 8
    p = torch.softmax(torch.randn(3, vocab, generator=g), 1)
    q = torch.softmax(torch.randn(3, vocab, generator=g), 1)
    from copy_reduce_amd.torch_api import verify_drafts
    require_gpu()
    for kids in (1, 2):
        t = kids + 1
        rows = [0] + [1] * kids
        probs, draft = p[rows].expand(n, t, vocab).contiguous(), q[rows].expand(n, t, vocab).contiguous()
        tokens = torch.multinomial(q[0].expand(n, vocab), t, replacement=True, generator=g)
        r = verify_drafts(probs.cuda(), ints(tokens), torch.rand(n, t, generator=g).cuda(), parents=ints(torch.zeros(n, t)), draft_probs=draft.cuda())
        second = r.path[:, 1].cpu().long() if t > 1 else None
        first = torch.where(second > 0, tokens.gather(1, second.clamp(min=0)[:, None]).squeeze(1), r.token.cpu().long())
        share = torch.bincount(first, minlength=vocab) / n
        assert float((share - p[0]).abs().max()) < 5 * 0.0036


def test_two_graphs_share_a_workspace():
    """Replayed in turns over new inputs, with an eager call of the same workspace in between."""
    note("verify: two captured graphs with one workspace")
    require_gpu()
    from copy_reduce_amd.torch_api import verify_drafts, verify_drafts_workspace
    g = torch.Generator().manual_seed(12)
    shapes = [(3, 6, 70000, 2, True), (3, 9, 70000, 3, False)]
    held = []
    for b, t, vocab, kids, drafted in shapes:
        probs, draft, parents, tokens, u = case(g, b, t, vocab, kids, drafted)
        held.append([probs.cuda(), None if draft is None else draft.cuda(), ints(parents), ints(tokens), u.cuda()])
    ws = verify_drafts_workspace(held[0][0])

    def call(x):
        return verify_drafts(x[0], x[3], x[4], parents=x[2], draft_probs=x[1], workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for x in held:
            call(x)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for x in held:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call(x))
        graphs.append(graph)
    for turn in range(4):
        for i, (b, t, vocab, kids, drafted) in enumerate(shapes):
            new = case(g, b, t, vocab, kids, drafted)
            for a, n in zip(held[i], new[:1] + (new[1],) + tuple(z.to(torch.int32) for z in new[2:4]) + new[4:]):
                if a is not None:
                    a.copy_(n)
            graphs[i].replay()
            want = verify(new[0], new[3], new[4], new[2], new[1])
            for j, (count, path, token) in enumerate(want):
                assert (int(outs[i].count[j]), outs[i].path[j].tolist(), int(outs[i].token[j])) == (count, path + [-1] * (t - count), token), f"turn {turn}"
            eager = call(held[i])
            assert all(torch.equal(p, q) for p, q in zip(eager[:3], outs[i][:3]))


def test_two_streams_at_once():
    note("verify on two streams")
    require_gpu()
    from copy_reduce_amd.torch_api import verify_drafts
    g = torch.Generator().manual_seed(13)
    sets = [case(g, 5, 7, 60000, 2, True) for _ in range(2)]
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
