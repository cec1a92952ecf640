"""CPU tests of refusals by the Python side of the paged cache, made before any call of the library, and of
what its import needs."""
import os
import subprocess
import sys

import pytest
import torch
from torch.autograd import forward_ad

import copy_reduce_amd as tb
from copy_reduce_amd.torch_api import tree_attention
from test_cache_host import _attn, _cache

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_needs_no_gpu_build_of_torch():
    """A torch without a GPU runtime lacks the functions that ask it for a device and its stream."""
    code = ("import torch\nfor n in ('_cuda_getDevice', '_cuda_getCurrentRawStream'):\n    delattr(torch._C, n)\n"
            "import copy_reduce_amd.torch_api as t\nprint(t.PagedCache.state_words(3, 2, 5))")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["22"]


class Cache:
    """What tree_attention looks at before it calls the library; the device has none of its kernels."""

    def __init__(self):
        self.dtype, self.device, self.head_dim, self.heads = torch.bfloat16, torch.device("cpu"), 64, 2
        self.pools = [torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16) for _ in range(2)]


def arguments():
    q, k, v = [torch.zeros(1, 2, h, 64, dtype=torch.bfloat16) for h in (4, 2, 2)]
    return Cache(), dict(q=q, k=k, v=v, layer=0, seqs=torch.zeros(1, dtype=torch.int32),
                         out=torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16), lse=torch.zeros(1, 2, 4))


@pytest.mark.parametrize("name", ["q", "k", "v", "out", "lse", 0, 1])
def test_a_gradient_is_refused(name):
    cache, args = arguments()
    t = cache.pools[name] if isinstance(name, int) else args[name]
    t.requires_grad_()
    with pytest.raises(ValueError, match="no gradient"):
        tree_attention(cache=cache, **args)


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("name", ["q", "k", "v", "out", "lse", 0, 1])
def test_a_tangent_is_refused(name, grad):
    cache, args = arguments()
    where = cache.pools if isinstance(name, int) else args
    with forward_ad.dual_level(), torch.set_grad_enabled(grad):
        where[name] = forward_ad.make_dual(where[name], torch.ones_like(where[name]))
        with pytest.raises(ValueError, match="no forward mode"):
            tree_attention(cache=cache, **args)


@pytest.mark.parametrize("stride,extent", [((1024, 256, 0), (3, 4, 4)), ((1024, 0, 64), (3, 4, 4)), ((0, 256, 64), (3, 4, 4)), ((1024, 256, 56), (3, 4, 4)),
                                           ((1024, 192, 64), (3, 4, 4)), ((960, 256, 64), (3, 4, 4)), ((256, 64, 64), (3, 4, 4)),
                                           ((64, 128, 512), (3, 4, 4)), ((0, 0, 64), (2, 1, 4)), ((64, 128, 64), (2, 2, 2))], ids=str)
def test_rows_of_out_that_overlap_are_refused(stride, extent):
    b, t, h = extent
    assert tb.lib.tb_tree_attention(_attn(out_stride=stride, batch=b, nodes=t, heads_q=h), _cache(), None) == tb.TB_ERR_INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not to be followed: needs a machine on which nothing is launched")
@pytest.mark.parametrize("stride,extent", [((1024, 256, 64), (3, 4, 4)), ((64, 192, 768), (3, 4, 4)), ((4096, 1024, 72), (3, 4, 4)), ((1 << 40, 256, 64), (3, 4, 4)),
                                           ((0, 256, 64), (1, 4, 4)), ((256, 0, 64), (3, 1, 4)), ((0, 0, 64), (1, 1, 4))], ids=str)
def test_rows_of_out_that_lie_apart_are_not_refused(stride, extent):
    b, t, h = extent
    assert tb.lib.tb_tree_attention(_attn(out_stride=stride, batch=b, nodes=t, heads_q=h), _cache(), None) == tb.TB_ERR_HIP
