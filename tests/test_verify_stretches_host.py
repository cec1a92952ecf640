"""CPU test of how tb_verify_drafts cuts a vocabulary up, read off the size of its workspace, which has a sum for each
stretch: a workgroup's 16 waves sum one each, and up to 256 workgroups run at once."""
import ctypes

import pytest

import copy_reduce_amd as tb
from copy_reduce_amd import _tb_serve


def stretches(batch, vocab):
    n = ctypes.c_uint64()
    assert tb.lib.tb_verify_workspace(_tb_serve.tb_verify(batch=batch, vocab=vocab), ctypes.byref(n)) == tb.TB_OK
    walks, ended = 32 * batch, -(-4 * batch // 16) * 16   # a place in the walk and a count for each sequence
    return (n.value - walks - ended) // (8 * batch)


@pytest.mark.parametrize("batch", [256, 300, 1000])
@pytest.mark.parametrize("vocab,least", [(4000, 8), (32000, 16), (50257, 13), (65536, 16), (131072, 16)])
def test_the_waves_of_a_workgroup_have_work(batch, vocab, least):
    """As many as the next smaller stretch still leaves in one workgroup."""
    assert least <= stretches(batch, vocab) <= 16


@pytest.mark.parametrize("batch", [2, 3, 20, 65, 100, 129, 130, 200, 255, 256])
@pytest.mark.parametrize("vocab", [513, 32000, 50257, 100003, 131072])
def test_the_workgroups_run_at_once(batch, vocab):
    assert batch * -(-stretches(batch, vocab) // 16) <= 256


@pytest.mark.parametrize("batch,vocab,groups", [(3, 32000, 4), (16, 131072, 16), (64, 131072, 4), (2, 1 << 20, 128)])
def test_and_few_sequences_are_summed_by_many(batch, vocab, groups):
    assert -(-stretches(batch, vocab) // 16) == groups
