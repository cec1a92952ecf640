"""CPU tests of the serving step's boundary (include/tb_serve.h): exports, the C structures as the binding lays them
out, and the refusals of the library and of the Python side, all before anything is launched."""
import ctypes
import os
import re
import subprocess

import pytest
import torch
from torch.autograd import forward_ad

import copy_reduce_amd as tb
from copy_reduce_amd import _tb_cache, _tb_serve
from copy_reduce_amd.torch_api import PagedCache, fp4_head_bytes, tree_attention, verify_drafts
from test_cache_host import BAD_POOLS, BAD_STATE, _attn, _cache

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, OK = tb.TB_ERR_INVALID, tb.TB_OK


def test_header_symbols_exported():
    text = open(os.path.join(ROOT, "include", "tb_serve.h")).read()
    declared = sorted(set(re.findall(r"^int (tb_\w+)\s*\(", text, re.M)))
    assert sorted(_tb_serve.EXPORTS) == declared
    for name in declared:
        assert hasattr(tb.lib, name)


def test_c_consumer_calls_every_entry_point():
    consumer = open(os.path.join(ROOT, "tests", "capi", "serve_check.c")).read()
    assert [d for d in _tb_serve.EXPORTS if d + "(" not in consumer] == []


def test_header_is_plain_c_and_the_binding_has_its_layout(tmp_path):
    names = ("tb_verify", "tb_attn_view")
    fields = {s: [f[0] for f in getattr(_tb_serve, s)._fields_] for s in names}
    lines = [f'printf("{s} %zu\\n", sizeof({s}));' for s in fields]
    lines += [f'printf("{s}.{f} %zu\\n", offsetof({s}, {f}));' for s, fs in fields.items() for f in fs]
    lines += [f'printf("bytes{d} %d\\n", TB_FP4_HEAD_BYTES({d}));' for d in (32, 64, 96, 128, 160, 256)]
    lines += ['printf("fp32 %d\\nblock %d\\nvocab %u\\n", TB_FP32, TB_FP4_BLOCK, TB_VERIFY_MAX_VOCAB);']
    src, exe = tmp_path / "use.c", tmp_path / "use"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"tb_serve.h\"\nint main(void){" + "".join(lines) + "return 0;}\n")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True).stdout.splitlines())
    for s, fs in fields.items():
        cls = getattr(_tb_serve, s)
        assert int(got[s]) == ctypes.sizeof(cls)
        for f in fs:
            assert int(got[f"{s}.{f}"]) == getattr(cls, f).offset
    for d in (32, 64, 96, 128, 160, 256):
        assert int(got[f"bytes{d}"]) == fp4_head_bytes(d) == tb.TB_FP4_HEAD_BYTES(d)
    assert (int(got["fp32"]), int(got["block"]), int(got["vocab"])) == (_tb_serve.TB_FP32, tb.TB_FP4_BLOCK, tb.TB_VERIFY_MAX_VOCAB)


def test_packed_arguments_have_the_structures_layout():
    for pack, cls in ((_tb_serve.pack_verify, _tb_serve.tb_verify), (_tb_serve.pack_view, _tb_serve.tb_attn_view)):
        n = sum(2 if name.endswith("_stride") else 1 for name, _ in cls._fields_)
        raw = pack(*range(1, n + 1))
        assert len(raw) == ctypes.sizeof(cls)
        flat = []
        for name, _ in cls._fields_:
            x = getattr(cls.from_buffer_copy(raw), name)
            flat += list(x) if name.endswith("_stride") else [x]
        assert flat == [*range(1, n + 1)]


def _verify(**kw):
    v = _tb_serve.tb_verify(probs=0x10000, draft_probs=0x20000, tokens=0x1000, parents=0x2000, uniform=0x3000, tree_nodes=0x4000, batch=3, nodes=4, vocab=100, dtype=2,
                            count=0x5000, path=0x6000, token=0x7000, seqs=0x8000, lens=0x9000, max_seqs=8, new_lens=0xa000, append_seqs=0xb000, append_positions=0xc000,
                            append_index=0xd000, workspace=0xe000, workspace_bytes=1 << 40)
    for k, x in kw.items():
        setattr(v, k, x)
    return v


BAD_VERIFY = [dict(probs=None), dict(probs=0x10002), dict(draft_probs=0x20002), dict(tokens=None), dict(tokens=0x1002), dict(parents=0x2001), dict(uniform=None),
              dict(uniform=0x3002), dict(tree_nodes=0x4002), dict(batch=(1 << 16) + 1), dict(nodes=0), dict(nodes=(1 << 12) + 1), dict(vocab=0), dict(vocab=(1 << 24) + 1),
              dict(dtype=3), dict(count=None), dict(path=None), dict(token=None), dict(path=0x6002), dict(seqs=0x8002), dict(lens=None), dict(new_lens=None),
              dict(append_seqs=None), dict(append_positions=None), dict(append_index=None), dict(append_index=0xd001), dict(workspace=None), dict(workspace=0xe008),
              dict(workspace_bytes=7), dict(probs_stride=((1 << 40) + 1, 0)), dict(draft_stride=(0, (1 << 40) + 1)), dict(dtype=0, probs=0x10001)]


@pytest.mark.parametrize("bad", BAD_VERIFY, ids=str)
def test_bad_verification_is_refused(bad):
    if "probs_stride" in bad or "draft_stride" in bad:
        bad = {k: (ctypes.c_uint64 * 2)(*x) for k, x in bad.items()}
    assert tb.lib.tb_verify_drafts(_verify(**bad), None) == INV


def test_verification_of_nothing_and_its_workspace():
    assert tb.lib.tb_verify_drafts(None, None) == INV
    assert tb.lib.tb_verify_drafts(_verify(batch=0), None) == OK
    n = ctypes.c_uint64(7)
    assert tb.lib.tb_verify_workspace(_verify(), None) == INV
    assert tb.lib.tb_verify_workspace(None, ctypes.byref(n)) == INV
    assert tb.lib.tb_verify_workspace(_verify(vocab=0), ctypes.byref(n)) == INV
    assert tb.lib.tb_verify_workspace(_verify(batch=0), ctypes.byref(n)) == OK and n.value == 0
    for b, v in ((1, 1), (1, 1 << 24), (1 << 16, 1 << 24), (64, 131072)):
        assert tb.lib.tb_verify_workspace(_verify(batch=b, vocab=v), ctypes.byref(n)) == OK
        assert n.value >= 32 * b + 8 * b * max(1, v // 8192) and n.value % 16 == 0


FP4 = dict(head_bytes=36, page_stride=16 * 2 * 36)


def _fp4_calls(c, dtype=0, dim=64, rows=0x7000, stride=256, pool=1024, lists=0x8000, n=1, first=0, npools=2):
    lib = tb.lib
    return [lib.tb_fp4_append(c, dtype, dim, rows, 4, stride, pool, lists, lists, None, n, None),
            lib.tb_fp4_read(c, dtype, dim, first, npools, rows, stride, pool, lists, lists, n, None)]


@pytest.mark.parametrize("bad", BAD_POOLS + BAD_STATE, ids=str)
def test_bad_cache_is_refused_everywhere(bad):
    assert _fp4_calls(_cache(**{**FP4, **bad})) == [INV, INV]
    assert tb.lib.tb_page_read(_cache(**bad), 0, 2, 0x7000, 256, 1024, 0x8000, 0x8000, 1, None) == INV
    assert tb.lib.tb_view_attention(_attn(), _tb_serve.tb_attn_view(fp4=1), _cache(**{**FP4, **bad}), None) == INV
    assert tb.lib.tb_view_attention(_attn(), _tb_serve.tb_attn_view(window=5), _cache(**bad), None) == INV


@pytest.mark.parametrize("bad", [dict(dtype=2), dict(dim=0), dict(dim=63), dict(dim=96), dict(rows=None), dict(rows=0x7001), dict(stride=255), dict(pool=1023), dict(lists=None),
                                 dict(lists=0x8002), dict(n=(1 << 30) + 1)], ids=str)
def test_bad_4_bit_arguments_are_refused(bad):
    assert _fp4_calls(_cache(**FP4), **bad) == [INV, INV]


def test_pools_in_4_bits_lie_at_multiples_of_4_bytes():
    odd = _cache(**FP4)
    odd._keep[1] = 0x20002
    assert _fp4_calls(odd) == [INV, INV]
    assert _fp4_calls(_cache(head_bytes=36, page_stride=16 * 2 * 36 + 2)) == [INV, INV]
    assert tb.lib.tb_view_attention(_attn(), _tb_serve.tb_attn_view(fp4=1), odd, None) == INV


def test_reads_refuse_overlapping_rows_and_pools_that_are_not_there():
    lib, c = tb.lib, _cache()
    for first, npools in ((3, 0), (0, 3), (2, 1), (1, 2), (1 << 31, 1 << 31)):
        assert lib.tb_page_read(c, first, npools, 0x7000, 256, 1024, 0x8000, 0x8000, 1, None) == INV
        assert _fp4_calls(_cache(**FP4), first=first, npools=npools)[1] == INV
    for row, pool in ((255, 1024), (256, 255), (256, 1023), (256, 256), (512, 128), (0, 1024)):
        assert lib.tb_page_read(c, 0, 2, 0x7000, row, pool, 0x8000, 0x8000, 4, None) == INV
    assert lib.tb_page_read(c, 0, 2, None, 256, 1024, 0x8000, 0x8000, 4, None) == INV
    for nothing in ((0, 2, 0), (0, 0, 4), (2, 0, 4)):
        assert lib.tb_page_read(c, nothing[0], nothing[1], None, 0, 0, None, None, nothing[2], None) == OK
    assert _fp4_calls(_cache(**FP4), rows=None, lists=None, n=0) == [OK, OK]


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not to be followed: needs a machine on which nothing is launched")
def test_rows_that_lie_apart_are_not_refused():
    for row, pool, n, npools in ((256, 1024, 4, 2), (512, 256, 4, 2), (0, 256, 1, 2), (256, 0, 4, 1), (0, 0, 1, 1)):
        assert tb.lib.tb_page_read(_cache(), 0, npools, 0x7000, row, pool, 0x8000, 0x8000, n, None) == tb.TB_ERR_HIP


def test_bad_views_are_refused():
    lib, view = tb.lib, _tb_serve.tb_attn_view
    assert lib.tb_view_attention(_attn(), None, _cache(), None) == INV
    assert lib.tb_view_attention(_attn(), view(fp4=2), _cache(), None) == INV
    assert lib.tb_view_attention(_attn(), view(window=4, depths=0x8002), _cache(), None) == INV
    assert lib.tb_view_attention(_attn(mask=0x8000), view(window=4), _cache(), None) == INV    # a tree's depths
    assert lib.tb_view_attention(_attn(), view(fp4=1), _cache(), None) == INV                   # a cache in 16 bits
    assert lib.tb_view_attention(_attn(), view(), _cache(**FP4), None) == INV                   # and the other way
    assert lib.tb_tree_attention(_attn(), _cache(**FP4), None) == INV
    large = _cache(head_bytes=36, page_stride=1 << 30, num_pages=17)
    assert lib.tb_view_attention(_attn(), view(fp4=1), large, None) == INV
    n = ctypes.c_uint64()
    assert lib.tb_view_attention_workspace(_attn(), None, _cache(), ctypes.byref(n)) == INV
    assert lib.tb_view_attention_workspace(_attn(), view(fp4=2), _cache(), ctypes.byref(n)) == INV
    assert lib.tb_view_attention_workspace(_attn(), view(), _cache(), None) == INV
    for nothing in (dict(batch=0), dict(nodes=0)):
        assert lib.tb_view_attention(_attn(**nothing), view(window=3), _cache(), None) == OK
        assert lib.tb_view_attention_workspace(_attn(**nothing), view(), _cache(), ctypes.byref(n)) == OK and n.value == 0


class Cache:
    """What tree_attention looks at before it calls the library; the device has none of its kernels."""

    def __init__(self):
        self.dtype, self.device, self.head_dim, self.heads = torch.bfloat16, torch.device("cpu"), 64, 2
        self.pools = [torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16) for _ in range(2)]


@pytest.mark.parametrize("bad", [dict(window=0), dict(window=-1), dict(window=1 << 32), dict(sinks=-1, window=3), dict(sinks=1 << 32, window=3), dict(sinks=2),
                                 dict(window=3, depths=torch.zeros(1, 2)), dict(window=3, depths=torch.zeros(2, 1, dtype=torch.int32)),
                                 dict(window=3, mask=torch.zeros(1, 2, 1, dtype=torch.int64))], ids=str)
def test_python_refuses_bad_windows(bad):
    q, k, v = [torch.zeros(1, 2, h, 64, dtype=torch.bfloat16) for h in (4, 2, 2)]
    with pytest.raises(ValueError, match="window|sinks|depths"):
        tree_attention(q, k, v, Cache(), 0, torch.zeros(1, dtype=torch.int32), **bad)


def test_python_refuses_bad_pools_and_heads():
    for dim in (0, 16, 33, -32):
        with pytest.raises(ValueError):
            fp4_head_bytes(dim)
    with pytest.raises(ValueError):
        PagedCache(torch.zeros(2, 8, 16, 2, 36, dtype=torch.uint8), 16, 4, 6, fp4=torch.bfloat16)   # on the host
    with pytest.raises(ValueError):
        verify_drafts(torch.zeros(1, 2, 5), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, 2))


class Probs(torch.Tensor):
    """A host tensor that says it is on a GPU, to reach the refusals behind that check."""
    is_cuda = property(lambda self: True)


def _python(**kw):
    args = dict(probs=torch.zeros(2, 3, 5), tokens=torch.zeros(2, 3, dtype=torch.int32), uniform=torch.zeros(2, 3))
    args.update(kw)
    args["probs"] = args["probs"].as_subclass(Probs)
    return lambda: verify_drafts(**args)


@pytest.mark.parametrize("bad", [dict(probs=torch.zeros(2, 3, 5, dtype=torch.float64)), dict(probs=torch.zeros(2, 5)), dict(probs=torch.zeros(2, 5, 3).transpose(1, 2)),
                                 dict(probs=torch.zeros(2, 0, 5)), dict(probs=torch.zeros(2, 3, 0)), dict(draft_probs=torch.zeros(2, 3, 4)),
                                 dict(draft_probs=torch.zeros(2, 3, 5, dtype=torch.float16)), dict(draft_probs=torch.zeros(2, 5, 3).transpose(1, 2)),
                                 dict(tokens=torch.zeros(2, 3)), dict(tokens=torch.zeros(2, 3, dtype=torch.int64)), dict(tokens=torch.zeros(3, 2, dtype=torch.int32)),
                                 dict(tokens=torch.zeros(3, 2, dtype=torch.int32).T), dict(uniform=torch.zeros(2, 3, dtype=torch.float64)), dict(uniform=torch.zeros(2, 2)),
                                 dict(parents=torch.zeros(2, 3)), dict(nodes=torch.zeros(2)), dict(nodes=torch.zeros(3, dtype=torch.int32)),
                                 dict(seqs=torch.zeros(2, dtype=torch.int32))], ids=lambda d: next(iter(d)))
def test_python_refuses_bad_verification(bad):
    with pytest.raises(ValueError):
        _python(**bad)()


@pytest.mark.parametrize("name", ["draft_probs", "uniform"])
def test_verification_refuses_gradients_and_tangents(name):
    x = torch.zeros(2, 3, 5) if name == "draft_probs" else torch.zeros(2, 3)
    with pytest.raises(ValueError, match="no gradient"):
        _python(**{name: x.clone().requires_grad_()})()
    with forward_ad.dual_level(), pytest.raises(ValueError, match="no forward mode"):
        _python(**{name: forward_ad.make_dual(x, torch.ones_like(x))})()
