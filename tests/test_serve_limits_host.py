"""CPU tests of the sizes at which a serving step's calls (include/tb_serve.h) are refused, because a kernel's grid would pass
2^32 threads: before anything is launched."""
import pytest
import torch

import copy_reduce_amd as tb
from copy_reduce_amd import _tb_serve
from test_cache_host import _attn, _cache
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


def _many(batch, heads, nodes=1, **kw):
    """Sequences of `heads` key heads of 64 elements in 4 bits, a query head each."""
    cache = _cache(heads=heads, page_tokens=1, head_bytes=36, page_stride=heads * 36)
    attn = _attn(batch=batch, nodes=nodes, heads_q=heads, head_dim=64, workspace_bytes=1 << 62, **kw)
    for s in (attn.q_stride, attn.k_stride, attn.v_stride, attn.out_stride):
        s[0], s[1], s[2] = nodes * heads * 64, heads * 64, 64
    return tb.lib.tb_view_attention(attn, _tb_serve.tb_attn_view(fp4=1), cache, None)


@pytest.mark.parametrize("batch,heads,nodes", [(16377, 1024, 1), (16383, 1024, 1)])
def test_attention_over_4_bits_counts_the_batch_in_eights(batch, heads, nodes):
    assert batch * nodes * heads < 1 << 24
    assert _many(batch, heads, nodes) == INV


@no_gpu
@pytest.mark.parametrize("batch,heads,nodes", [(16376, 1024, 1), (1023, 1024, 16), (7, 1024, 2047), (1, 1024, 4096)])
def test_attention_over_4_bits_below_that_is_not_refused(batch, heads, nodes):
    assert _many(batch, heads, nodes) == tb.TB_ERR_HIP
