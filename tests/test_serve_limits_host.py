"""CPU tests of the sizes at which a serving step's calls (include/tb_serve.h) are refused, because a kernel's grid would pass
2^32 threads: before anything is launched."""
import pytest
import torch

import copy_reduce_amd as tb
from test_serve_host import INV, _python, _verify

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not to be followed: needs a machine on which nothing is launched")


@pytest.mark.parametrize("batch,vocab", [(1 << 16, 1 << 24), (1 << 16, (1 << 22) + 1), (1 << 15, (1 << 23) + 1), ((1 << 14) + 1, 1 << 24)])
def test_verification_of_more_entries_than_a_grid_has_room_for(batch, vocab):
    """With rows that are shared (strides of 0) so many take no memory."""
    assert tb.lib.tb_verify_drafts(_verify(batch=batch, vocab=vocab, nodes=1), None) == INV


def test_python_says_so():
    vocab = (1 << 22) + 1
    probs = torch.empty(vocab).as_strided((1 << 16, 1, vocab), (0, 0, 1))
    u = torch.zeros(1, 1).expand(1 << 16, 1)
    with pytest.raises(ValueError, match="all sequences together"):
        _python(probs=probs, tokens=u.int(), uniform=u)()


@no_gpu
@pytest.mark.parametrize("batch,vocab", [(1 << 16, 1 << 22), (1 << 14, 1 << 24), (1, 1 << 24)])
def test_as_many_as_fit_are_not(batch, vocab):
    assert tb.lib.tb_verify_drafts(_verify(batch=batch, vocab=vocab, nodes=1), None) == tb.TB_ERR_HIP
