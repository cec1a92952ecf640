"""GPU tests: tensors that carry a gradient or a tangent are refused, since no call of the cache has either."""
import pytest
import torch
from torch.autograd import forward_ad

from gpu_util import note
from test_gpu_cache import ints, make

pytestmark = pytest.mark.gpu


def case():
    from copy_reduce_amd.torch_api import tree_attention
    c, _ = make(pt=4, heads=2, dim=64)
    c.resize(ints([0]), ints([9]))
    for p in c.pools:      # make() fills the pools with any bits
        p.zero_()
    g = torch.Generator().manual_seed(1)
    q, k, v = [torch.randn(1, 2, h, 64, generator=g).to(torch.bfloat16).cuda() for h in (4, 2, 2)]
    return c, [q, k, v], lambda *x, **kw: tree_attention(*x, c, 0, ints([0]), **kw)


@pytest.mark.parametrize("which", [0, 1, 2])
def test_dual_tensors_are_refused(which):
    note(f"tree attention, a tangent of input {which}")
    c, x, call = case()
    want = call(*x)
    with forward_ad.dual_level():
        dual = list(x)
        dual[which] = forward_ad.make_dual(x[which], torch.ones_like(x[which]))
        with pytest.raises(ValueError, match="tangent"):
            call(*dual)
        got = call(*x)           # the same call of plain tensors inside the level
        primal = forward_ad.unpack_dual(dual[which]).primal
        dual[which] = primal
        again = call(*dual)
    for y in (got, again):
        assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])


@pytest.mark.parametrize("which", [0, 1])
def test_pools_that_carry_a_gradient_or_a_tangent_are_refused(which):
    note(f"tree attention, pool {which} wants a gradient")
    c, x, call = case()
    plain = c.pools[which]
    plain.requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        call(*x)
    with torch.no_grad():
        call(*x)
    plain.requires_grad_(False)
    with forward_ad.dual_level():
        c.pools[which] = forward_ad.make_dual(plain, torch.ones_like(plain))
        with pytest.raises(ValueError, match="tangent"):
            call(*x)
        c.pools[which] = plain


def test_outputs_that_carry_a_gradient_are_refused():
    note("tree attention, outputs that want a gradient")
    c, x, call = case()
    for kw in (dict(out=torch.empty_like(x[0])), dict(lse=torch.empty(1, 2, 4, device="cuda"))):
        for t in kw.values():
            t.requires_grad_()
        with pytest.raises(ValueError, match="gradient"):
            call(*x, **kw)


def test_appended_rows_that_carry_a_gradient_or_a_tangent_are_refused():
    note("paged cache, appended rows with a gradient")
    c, _, _ = case()
    rows = torch.ones(2, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    before = [p.clone() for p in c.pools]
    with pytest.raises(ValueError, match="gradient"):
        c.append(rows.clone().requires_grad_(), ints([0]), ints([8]))
    with forward_ad.dual_level():
        with pytest.raises(ValueError, match="tangent"):
            c.append(forward_ad.make_dual(rows, rows), ints([0]), ints([8]))
    assert all(torch.equal(a, b) for a, b in zip(before, c.pools))
    with torch.no_grad():
        c.append(rows.clone().requires_grad_(), ints([0]), ints([8]))
    assert bool((c.pools[0][int(c.table[0, 2]), 0] == 1).all()) and c.flags() == 0
