"""GPU tests of windows over sequences of which few are long: the long ones' keys are shared out over the workgroups, however
wide the table is.  A call that shares keys writes the shares to its workspace, one that does not leaves
it as it was."""
import pytest
import torch

from gpu_util import note
from test_gpu_fp4_cache import make
from test_gpu_fp4_cache import run as run_fp4
from test_gpu_tree_attention import inputs, setup
from test_gpu_window_attention import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("room", [2000, 8192])
@pytest.mark.parametrize("fp4", [False, True], ids=["16 bits", "4 bits"])
def test_long_sequences_among_many_short_ones_are_shared_out(fp4, room):
    note(f"60 short and 4 long sequences, windows of 800, a table of {room}, 4 bits: {fp4}")
    from copy_reduce_amd.torch_api import tree_attention_workspace
    lens = [1200 if i % 16 == 5 else 1 + (i * 37) % 60 for i in range(64)]
    c, m, g = (make if fp4 else setup)(lens, heads=8, dim=128, pt=32, seed=room, room=room)
    q, k, v = inputs(g, 64, 1, 8, 8, 128, torch.bfloat16)
    ws = tree_attention_workspace(q.cuda(), c)
    ws.fill_(0xEE)
    order = torch.randperm(64, generator=g).tolist()
    if fp4:
        run_fp4(c, m, q, k, v, order, window=800, sinks=4, workspace=ws)
    else:
        run(c, m, q, k, v, order, 800, 4, workspace=ws)
    assert bool((ws != 0xEE).any())


@pytest.mark.parametrize("fp4", [False, True], ids=["16 bits", "4 bits"])
def test_a_long_sequence_among_short_ones_is_shared_out_for_many_rows(fp4):
    note(f"31 short sequences and a long one, 40 nodes, windows of 3,001, 4 bits: {fp4}")
    from copy_reduce_amd.torch_api import tree_attention_workspace
    lens = [1 + i for i in range(31)] + [3500]
    c, m, g = (make if fp4 else setup)(lens, heads=8, dim=64, pt=32, seed=1, room=16384)
    q, k, v = inputs(g, 32, 40, 8, 8, 64, torch.bfloat16)
    ws = tree_attention_workspace(q.cuda(), c)
    ws.fill_(0xEE)
    order = torch.randperm(32, generator=g).tolist()
    if fp4:
        run_fp4(c, m, q, k, v, order, window=3001, sinks=4, workspace=ws)
    else:
        run(c, m, q, k, v, order, 3001, 4, workspace=ws)
    assert bool((ws != 0xEE).any())
