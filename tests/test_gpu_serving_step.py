"""GPU tests of the serving step as it is used: the attention of drafted tokens over a window of a cache held in 4 bits, their
verification, the accepted ones' growth and append, with nothing read back in between; captured and replayed, on other
streams, two at once; and the step from plain C (tests/capi/serve_check.c)."""
import os
import subprocess

import pytest
import torch

from gpu_util import note, require_gpu
from serve_model import decode, encode, verify, window_attention
from test_gpu_fp4_cache import make
from test_gpu_tree_attention import compare, ints

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
B, T, HQ, HK, D, VOCAB, WINDOW, SINKS = 3, 6, 4, 2, 64, 400, 40, 4


def draws(g):
    """One step's inputs: queries, the nodes' keys and values, distributions, proposals, random numbers."""
    q, k, v = [torch.randn(B, T, h, D, generator=g).to(torch.bfloat16) for h in (HQ, HK, HK)]
    x = 2 * torch.randn(B, T, VOCAB, generator=g)
    p, d = torch.softmax(x, 2), torch.softmax(x + 0.5 * torch.randn(B, T, VOCAB, generator=g), 2)
    parents = torch.tensor([0, 0, 0, 1, 1, 3]).repeat(B, 1)
    tokens = torch.stack([torch.multinomial(d[i, parents[i]], 1, generator=g).flatten() for i in range(B)])
    return q, k, v, p, d, tokens.to(torch.int32), torch.rand(B, T, generator=g)


class Step:
    """The step over buffers that stay where they are."""

    def __init__(self, cache, seqs):
        from copy_reduce_amd.torch_api import tree_attention_workspace, verify_drafts_workspace
        self.cache, self.seqs = cache, ints(seqs)
        self.x = [t.cuda() for t in draws(torch.Generator().manual_seed(0))]
        self.parents = ints([[0, 0, 0, 1, 1, 3]] * B)
        sees = torch.tensor([0b1, 0b11, 0b101, 0b1011, 0b10011, 0b101011], dtype=torch.int64)
        self.mask, self.depths = sees.view(1, T, 1).repeat(B, 1, 1).cuda(), ints([[0, 1, 1, 2, 2, 3]] * B)
        self.ws = tree_attention_workspace(self.x[0], cache), verify_drafts_workspace(self.x[3])

    def load(self, g):
        new = draws(g)
        for a, b in zip(self.x, new):
            a.copy_(b)
        return new

    def __call__(self, stream=None):
        from copy_reduce_amd.torch_api import tree_attention, verify_drafts
        q, k, v, p, d, tokens, u = self.x
        out, lse = tree_attention(q, k, v, self.cache, 0, self.seqs, mask=self.mask, depths=self.depths, window=WINDOW, sinks=SINKS, workspace=self.ws[0], stream=stream)
        r = verify_drafts(p, tokens, u, parents=self.parents, draft_probs=d, cache=self.cache, seqs=self.seqs, workspace=self.ws[1], stream=stream)
        self.cache.resize(self.seqs, r.lens, stream=stream)
        with torch.cuda.stream(stream) if stream is not None else torch.cuda.stream(torch.cuda.current_stream()):
            rows = torch.stack([k.reshape(B * T, HK, D), v.reshape(B * T, HK, D)])
        self.cache.append(rows, r.append_seqs, r.append_positions, r.append_index, stream=stream)
        return out, lse, r


def follow(m, new, seqs):
    """The same step on the model: (out, lse ...), what is accepted."""
    q, k, v, p, d, tokens, u = new
    parents = torch.tensor([[0, 0, 0, 1, 1, 3]] * B)
    mask = torch.tensor([0b1, 0b11, 0b101, 0b1011, 0b10011, 0b101011], dtype=torch.int64).view(1, T, 1).repeat(B, 1, 1)
    ref = window_attention(m, 0, q, k, v, seqs, mask, window=WINDOW, sinks=SINKS, depths=torch.tensor([[0, 1, 1, 2, 2, 3]] * B))
    found = verify(p, tokens, u, parents, d)
    had = [m.lens[s] for s in seqs]
    m.resize(seqs, [h + f[0] for h, f in zip(had, found)])
    for i, (count, path, _) in enumerate(found):
        for j, node in enumerate(path):
            page, off = m.table[seqs[i]][(had[i] + j) // m.pt], (had[i] + j) % m.pt
            for pool, x in enumerate((k, v)):
                m.by_token()[pool, page, off] = decode(encode(x[i, node]), D).to(torch.bfloat16)
    return ref, found


def same(m, cache, seqs):
    assert cache.flags() == 0 and cache.lens.tolist()[:len(m.lens)] == m.lens
    for s in seqs:
        n = m.lens[s]
        got = cache.read(ints([s] * n), ints(list(range(n)))).cpu()
        for pool in range(2):
            for h in range(HK):
                assert torch.equal(got[pool, :, h].double(), m.context(pool, s, h))


def agree(got, want, m, what):
    (out, lse, r), (ref, found) = got, want
    compare((out, lse), ref, 400, D, torch.bfloat16, what)
    for i, (count, path, token) in enumerate(found):
        assert (int(r.count[i]), r.path[i].tolist(), int(r.token[i])) == (count, path + [-1] * (T - count), token), what


def test_steps_in_a_row():
    note("serving steps one after the other")
    seqs = [2, 0, 3]
    c, m, g = make([50, 7, 30, 0], heads=HK, dim=D, pt=8, spare=60, room=300)
    step = Step(c, seqs)
    for i in range(12):
        new = step.load(g)
        agree(step(), follow(m, new, seqs), m, f"step {i}")
    same(m, c, range(4))


@pytest.mark.parametrize("room", [300, 8192], ids=["whole", "shares"])
def test_a_captured_step_is_replayed(room):
    """One graph of the whole step, replayed over changing inputs with eager work in between."""
    note(f"serving step captured, room {room}")
    seqs = [2, 0, 3]
    c, m, g = make([50, 7, 30, 0], heads=HK, dim=D, pt=8, spare=60, room=room)
    step = Step(c, seqs)
    held = c.state.clone(), [p.clone() for p in c.pools]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    c.state.copy_(held[0])
    for p, h in zip(c.pools, held[1]):
        p.copy_(h)
    for i in range(6):
        new = step.load(g)
        graph.replay()
        agree(got, follow(m, new, seqs), m, f"replay {i}")
        if i % 2 == 0:   # an eager step between replays
            new = step.load(g)
            agree(step(), follow(m, new, seqs), m, f"eager {i}")
        torch.cuda.synchronize()
    same(m, c, range(4))


def test_two_steps_at_once():
    """Two caches, two streams, neither the current one."""
    note("two serving steps on two streams")
    seqs = [2, 0, 3]
    both = [make([50, 7, 30, 0], heads=HK, dim=D, pt=8, spare=60, room=8192, seed=s) for s in (1, 2)]
    steps = [Step(c, seqs) for c, _, _ in both]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(4):
        new = [s.load(g) for s, (_, _, g) in zip(steps, both)]
        torch.cuda.synchronize()
        got = [s(stream=st) for s, st in zip(steps, streams)]
        torch.cuda.synchronize()
        for x, n, (_, m, _) in zip(got, new, both):
            agree(x, follow(m, n, seqs), m, f"step {i}")
    for c, m, _ in both:
        same(m, c, range(4))


def test_refusals_with_tensors_on_the_device():
    note("refusals of the serving step's calls")
    from copy_reduce_amd.torch_api import PagedCache, tree_attention, verify_drafts
    require_gpu()
    c, m, g = make([50, 7, 30, 0], heads=HK, dim=D, pt=8)
    step = Step(c, [2, 0, 3])
    q, k, v, p, d, tokens, u = step.x
    with pytest.raises(ValueError):
        tree_attention(q.half(), k.half(), v.half(), c, 0, step.seqs)
    with pytest.raises(ValueError):
        c.append(torch.zeros(2, 3, HK, D + 4, dtype=torch.bfloat16, device="cuda"), step.seqs, step.seqs)
    with pytest.raises(ValueError):
        c.append(torch.zeros(2, 3, HK, 36, dtype=torch.uint8, device="cuda"), step.seqs, step.seqs)
    with pytest.raises(ValueError):
        c.read(step.seqs, step.seqs, layer=1)
    with pytest.raises(ValueError):
        c.read(step.seqs, step.seqs, out=torch.zeros(2, 3, HK, D, device="cuda"))
    with pytest.raises(ValueError):
        c.copy_pages(step.seqs, step.seqs, src=PagedCache(torch.zeros(2, 9, 8, HK, 36, dtype=torch.uint8, device="cuda"), 8, 4, 4))
    for shape, dtype in (((2, 9, 8, HK, 35), torch.uint8), ((2, 9, 8, HK, 64), torch.bfloat16), ((2, 9, 8, HK, 16), torch.uint8)):
        with pytest.raises(ValueError):
            PagedCache(torch.zeros(shape, dtype=dtype, device="cuda"), 8, 4, 4, fp4=torch.bfloat16)
    with pytest.raises(ValueError):
        PagedCache(torch.zeros(2, 9, 8, HK, 36, dtype=torch.uint8, device="cuda"), 8, 4, 4, fp4=torch.float32)
    odd = torch.zeros(2 * 9 * 8 * HK * 36 + 2, dtype=torch.uint8, device="cuda")[2:].view(2, 9, 8, HK, 36)
    with pytest.raises(ValueError):
        PagedCache(odd, 8, 4, 4, fp4=torch.bfloat16)
    with pytest.raises(ValueError):
        verify_drafts(p, tokens, u, cache=c)
    with pytest.raises(ValueError):
        verify_drafts(p, tokens.cpu(), u)
    with pytest.raises(Exception):
        verify_drafts(p, tokens, u, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="gradient"):
        verify_drafts(p.clone().requires_grad_(), tokens, u)
    with pytest.raises(ValueError, match="gradient"):
        c.read(step.seqs, step.seqs, out=torch.zeros(2, 3, HK, D, dtype=torch.bfloat16, device="cuda").requires_grad_())


def test_c_program_uses_the_step():
    binary = os.path.join(ROOT, "tests", "capi", "serve_check")
    if not os.path.exists(binary):
        pytest.fail(f"{binary} is missing: build first (python -c 'import __graft_entry__ as g; g.build()')")
    note("C-ABI consumer of the serving step")
    r = subprocess.run([binary], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, f"rc={r.returncode}\n{r.stdout}\n{r.stderr}"
    assert "serve ok" in r.stdout
