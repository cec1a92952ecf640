"""GPU tests of many drafted nodes over windows, as a windowed layer has them that takes in a prompt by chunks: chains and trees
of up to 4,096 nodes, longer than their windows, in 16 bits and over a cache in 4, against the definition in 64 bits.  The bounds
are those of test_gpu_tree_attention.py."""
import pytest
import torch

from gpu_util import note
from test_gpu_fp4_cache import make
from test_gpu_tree_attention import compare, inputs, ints, setup, tree_mask
from test_gpu_window_attention import depths_of
from wide_model import window_attention

pytestmark = pytest.mark.gpu


def check(c, m, q, k, v, seqs, window, sinks, mask=None, nodes=None, depths=None):
    from copy_reduce_amd.torch_api import tree_attention
    got = tree_attention(q.cuda(), k.cuda(), v.cuda(), c, 0, ints(seqs), mask=None if mask is None else mask.cuda(),
                         nodes=None if nodes is None else ints(nodes), window=window, sinks=sinks, depths=None if depths is None else depths.cuda())
    ref = window_attention(m, 0, q, k, v, seqs, mask, nodes, None, window, sinks, depths)
    compare(got, ref, max(m.lens) + q.shape[1], q.shape[3], q.dtype, f"window {window}, sinks {sinks}")


@pytest.mark.parametrize("fp4", [False, True], ids=["16 bits", "4 bits"])
@pytest.mark.parametrize("room", [0, 16384], ids=["whole", "shares"])
@pytest.mark.parametrize("t,group,dim,dtype,lens", [(1000, 2, 64, torch.bfloat16, [700, 0, 31]), (777, 1, 128, torch.float16, [1500, 1]),
                                                    (600, 3, 96, torch.bfloat16, [333]), (515, 2, 256, torch.float16, [40, 900])])
def test_chains(t, group, dim, dtype, lens, room, fp4):
    """A chain with depths by themselves, and with the same depths given."""
    note(f"chains of {t} over {lens}, dim {dim} {dtype}, room {room}, 4 bits {fp4}")
    c, m, g = (make if fp4 else setup)(lens, heads=1, dim=dim, pt=16, dtype=dtype, seed=t, room=room)
    b = len(lens)
    q, k, v = inputs(g, b, t, group, 1, dim, dtype)
    order = torch.randperm(b, generator=g).tolist()
    nodes = [t - 37 * i for i in range(b)]
    for window, sinks in ((1, 0), (33, 5), (300, 0), (300, 450), (t, 3)):
        check(c, m, q, k, v, order, window, sinks, None, nodes)
    check(c, m, q, k, v, order, 100, 7, None, nodes, torch.arange(t, dtype=torch.int32).repeat(b, 1))


@pytest.mark.parametrize("fp4", [False, True], ids=["16 bits", "4 bits"])
@pytest.mark.parametrize("t,window,sinks,n,dim", [(4096, 1024, 4, 2000, 64), (4096, 129, 2500, 2000, 64), (2048, 1024, 0, 1, 128), (4095, 4096, 0, 300, 64)])
def test_the_longest_chains(t, window, sinks, n, dim, fp4):
    note(f"a chain of {t} over {n}, window {window}, sinks {sinks}, 4 bits {fp4}")
    c, m, g = (make if fp4 else setup)([n], heads=1, dim=dim, pt=16, seed=n, room=16384)
    q, k, v = inputs(g, 1, t, 2, 1, dim, torch.bfloat16)
    check(c, m, q, k, v, [0], window, sinks)


@pytest.mark.parametrize("fp4", [False, True], ids=["16 bits", "4 bits"])
@pytest.mark.parametrize("window,sinks", [(2, 0), (5, 620), (40, 9)])
def test_large_trees(window, sinks, fp4):
    """Random trees, and one that is a chain of 400 nodes with leaves: deeper than the window."""
    note(f"trees of 700 nodes, window {window}, sinks {sinks}, 4 bits {fp4}")
    c, m, g = (make if fp4 else setup)([600, 250], heads=2, dim=64, pt=8, seed=sinks, room=4000)
    t = 700
    q, k, v = inputs(g, 2, t, 4, 2, 64, torch.bfloat16)
    mask = tree_mask(g, 2, t)
    for x in range(t):   # the second tree
        bit = 1 << (x % 64)
        mask[1, x] = 0 if x == 0 else mask[1, x - 1 if x < 400 else x - 300]
        mask[1, x, x // 64] |= bit - (1 << 64) if bit >> 63 else bit
    depths = depths_of(mask)
    check(c, m, q, k, v, [0, 1], window, sinks, mask, [t, t - 11], depths)
