"""CPU test that wide_model is serve_model's definition."""
import pytest
import torch

import serve_model
import wide_model
from cache_model import Model
from test_gpu_tree_attention import tree_mask
from test_gpu_window_attention import depths_of


@pytest.mark.parametrize("window,sinks", [(None, 0), (1, 0), (4, 3), (20, 0), (50, 40), (9, 100)])
@pytest.mark.parametrize("tree", [False, True])
def test_both_models_agree(window, sinks, tree):
    g = torch.Generator().manual_seed(sinks)
    kv = torch.randn(2, 20, 4, 2, 8, generator=g)
    m = Model(20, 4, 3, 10, kv, "token")
    m.stack = list(range(20))
    m.resize([0, 1, 2], [30, 0, 5])
    q, k, v = [torch.randn(4, 13, h, 8, generator=g) for h in (4, 2, 2)]
    mask = tree_mask(g, 4, 13) if tree else None
    depths = depths_of(mask) if tree else None
    args = (m, 0, q, k, v, [2, 0, 1, 7], mask, [13, 9, 13, 13], None, window, sinks, depths)
    for x, y in zip(serve_model.window_attention(*args), wide_model.window_attention(*args)):
        torch.testing.assert_close(x, y, rtol=1e-12, atol=1e-12)
