"""CPU tests of the paged cache's boundary (include/tb_cache.h): exports, the
C structures as the binding lays them out, and the argument checks, which
reject before any HIP call."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import copy_reduce_amd as tb
from copy_reduce_amd import _tb_cache
from copy_reduce_amd.torch_api import PagedCache, tree_attention

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_header_symbols_exported():
    text = open(os.path.join(ROOT, "include", "tb_cache.h")).read()
    declared = sorted(set(re.findall(r"^int (tb_\w+)\s*\(", text, re.M)))
    assert sorted(_tb_cache.EXPORTS) == declared
    for name in declared:
        assert hasattr(tb.lib, name)


def test_header_is_plain_c_and_the_binding_has_its_layout(tmp_path):
    fields = {"tb_cache": [f[0] for f in _tb_cache.tb_cache._fields_],
              "tb_tree_attn": [f[0] for f in _tb_cache.tb_tree_attn._fields_]}
    lines = [f'printf("{s} %zu\\n", sizeof({s}));' for s in fields]
    lines += [f'printf("{s}.{f} %zu\\n", offsetof({s}, {f}));' for s, fs in fields.items() for f in fs]
    src, exe = tmp_path / "use.c", tmp_path / "use"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"tb.h\"\n#include \"tb_cache.h\"\n"
                   "int main(void){" + "".join(lines) + "return 0;}\n")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    str(exe)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True).stdout.splitlines())
    for s, fs in fields.items():
        cls = getattr(_tb_cache, s)
        assert int(got[s]) == ctypes.sizeof(cls)
        for f in fs:
            assert int(got[f"{s}.{f}"]) == getattr(cls, f).offset


def test_packed_arguments_have_the_structure_s_layout():
    values = range(1, 31)                             # one for each field, the strides three each
    a = _tb_cache.tb_tree_attn.from_buffer_copy(_tb_cache.pack_tree_attn(*values))
    flat = []
    for name, _ in _tb_cache.tb_tree_attn._fields_:
        x = getattr(a, name)
        flat += list(x) if name.endswith("_stride") else [x]
    assert len(flat) == 5 + 12 + 3 + 7 + 1 + 2
    assert flat == [*range(1, len(flat) + 1)]


def test_c_consumer_calls_every_entry_point():
    consumer = open(os.path.join(ROOT, "tests", "capi", "cache_check.c")).read()
    assert [d for d in _tb_cache.EXPORTS if d + "(" not in consumer] == []


def test_constants_match_the_header():
    text = open(os.path.join(ROOT, "include", "tb_cache.h")).read()
    for name in ("TB_CACHE_TOKEN_MAJOR", "TB_CACHE_HEAD_MAJOR", "TB_CACHE_SHORT", "TB_CACHE_RANGE", "TB_CACHE_BUSY",
                 "TB_CACHE_TWICE", "TB_CACHE_SHARED", "TB_BF16", "TB_FP16"):
        assert int(re.search(rf"\b{name} = (\d+)", text).group(1)) == getattr(_tb_cache, name)
    assert int(re.search(r"#define TB_MAX_POOLS (\d+)", text).group(1)) == _tb_cache.TB_MAX_POOLS


def test_scratch_bytes():
    a, b = _tb_cache.tb_cache_scratch_bytes(1, 1), _tb_cache.tb_cache_scratch_bytes(1 << 20, 512)
    assert 0 < a < b and b >= 3 * 4 * (1 << 20) and a % 16 == 0
    n = ctypes.c_uint64()
    assert tb.lib.tb_cache_scratch_bytes(0, 1, ctypes.byref(n)) == tb.TB_ERR_INVALID
    assert tb.lib.tb_cache_scratch_bytes(1, 0, ctypes.byref(n)) == tb.TB_ERR_INVALID
    assert tb.lib.tb_cache_scratch_bytes((1 << 30) + 1, 1, ctypes.byref(n)) == tb.TB_ERR_INVALID
    assert tb.lib.tb_cache_scratch_bytes(1, 1, None) == tb.TB_ERR_INVALID


def _cache(**kw):
    """A cache of addresses that are never followed: every call below is refused."""
    c = _tb_cache.tb_cache()
    c._keep = (ctypes.c_void_p * 2)(0x10000, 0x20000)
    c.pools = ctypes.addressof(c._keep)
    c.npools, c.layout, c.num_pages, c.page_tokens, c.heads, c.head_bytes = 2, 0, 8, 16, 2, 128
    c.page_stride, c.max_seqs, c.max_pages = 16 * 2 * 128, 4, 6
    c.table, c.lens, c.refs, c.free_list, c.counts, c.scratch = 0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_POOLS = [dict(npools=257), dict(layout=2), dict(num_pages=0), dict(num_pages=(1 << 30) + 1), dict(page_tokens=0),
             dict(page_tokens=(1 << 16) + 1), dict(heads=0), dict(head_bytes=0), dict(pools=None), dict(heads=(1 << 16) + 1, head_bytes=1, page_tokens=1, page_stride=1 << 17),
             dict(head_bytes=1 << 26, page_stride=1 << 33),
             dict(page_stride=16 * 2 * 128 - 1), dict(page_stride=1 << 62)]
BAD_STATE = [dict(max_seqs=0), dict(max_pages=0), dict(max_pages=1 << 27), dict(table=None), dict(lens=None),
             dict(refs=None), dict(free_list=None), dict(counts=None), dict(scratch=None), dict(scratch=0x6004),
             dict(table=0x1002), dict(lens=0x2001)]


@pytest.mark.parametrize("bad", BAD_POOLS + BAD_STATE, ids=str)
def test_bad_cache_is_refused_everywhere(bad):
    lib, c, p = tb.lib, _cache(**bad), 0x7000
    inv = tb.TB_ERR_INVALID
    assert lib.tb_page_fork(c, p, p, 1, None) == inv
    assert lib.tb_page_compact(c, None) == inv
    assert lib.tb_page_append(c, p, 4, 256, 1024, p, p, None, 1, None) == inv
    if bad in BAD_STATE:
        assert lib.tb_cache_init(c, None) == inv
        assert lib.tb_page_resize(c, p, p, 1, None) == inv
    else:
        assert lib.tb_page_copy(c, c, p, p, 1, None) == inv
    assert lib.tb_tree_attention(_attn(), c, None) == inv


def test_null_pool_is_refused():
    c = _cache()
    c._keep[1] = None
    assert tb.lib.tb_page_copy(c, c, 0x7000, 0x7000, 1, None) == tb.TB_ERR_INVALID


def test_lists_and_counts():
    lib, c, p, inv, ok = tb.lib, _cache(), 0x7000, tb.TB_ERR_INVALID, tb.TB_OK
    assert lib.tb_page_fork(c, None, p, 1, None) == inv
    assert lib.tb_page_fork(c, p, 0x7002, 1, None) == inv
    assert lib.tb_page_fork(c, p, p, 5, None) == inv            # more entries than rows
    assert lib.tb_page_resize(c, p, None, 1, None) == inv
    assert lib.tb_page_resize(c, p, p, 5, None) == inv
    assert lib.tb_page_copy(c, c, p, None, 1, None) == inv
    assert lib.tb_page_copy(c, _cache(heads=1, head_bytes=256), p, p, 1, None) == inv
    assert lib.tb_page_copy(c, _cache(layout=1), p, p, 1, None) == inv
    assert lib.tb_page_copy(c, _cache(npools=1), p, p, 1, None) == inv
    assert lib.tb_page_append(c, None, 4, 256, 1024, p, p, None, 1, None) == inv
    assert lib.tb_page_append(c, p, 0, 256, 1024, p, p, None, 1, None) == inv
    assert lib.tb_page_append(c, p, 4, 255, 1024, p, p, None, 1, None) == inv   # rows overlap
    assert lib.tb_page_append(c, p, 4, 256, 1024, p, p, 0x7001, 1, None) == inv
    for null in (lib.tb_page_fork(None, p, p, 1, None), lib.tb_page_resize(None, p, p, 1, None),
                 lib.tb_page_compact(None, None), lib.tb_cache_init(None, None), lib.tb_page_copy(c, None, p, p, 1, None)):
        assert null == inv
    # nothing to do needs no device
    assert lib.tb_page_fork(c, None, None, 0, None) == ok
    assert lib.tb_page_resize(c, None, None, 0, None) == ok
    assert lib.tb_page_copy(c, c, None, None, 0, None) == ok
    assert lib.tb_page_append(c, None, 0, 0, 0, None, None, None, 0, None) == ok


def _attn(**kw):
    a = _tb_cache.tb_tree_attn()
    a.q, a.k, a.v, a.out, a.lse, a.seqs, a.workspace = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x7000, 0x60000
    a.q_stride, a.out_stride = (1024, 256, 64), (1024, 256, 64)
    a.k_stride, a.v_stride = (512, 128, 64), (512, 128, 64)
    a.batch, a.nodes, a.heads_q, a.head_dim, a.dtype, a.k_pool, a.v_pool, a.scale = 3, 4, 4, 64, 0, 0, 1, 0.125
    a.workspace_bytes = 1 << 40
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad", [dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(seqs=None), dict(q=0x10008),
                                 dict(k=0x20002), dict(out=0x40004), dict(lse=0x50002), dict(mask=0x8004),
                                 dict(tree_nodes=0x8002), dict(heads_q=3), dict(heads_q=0), dict(heads_q=1026),
                                 dict(head_dim=80), dict(head_dim=128), dict(dtype=2), dict(k_pool=2), dict(v_pool=7),
                                 dict(batch=(1 << 16) + 1), dict(nodes=(1 << 12) + 1), dict(q_stride=(1024, 260, 64)),
                                 dict(v_stride=(1 << 41, 128, 64)), dict(workspace=None), dict(workspace=0x60008),
                                 dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=-1e31),
                                 dict(batch=1 << 16, nodes=1 << 6), dict(batch=1 << 12, nodes=1 << 12)],
                         ids=str)
def test_bad_attention_is_refused(bad):
    assert tb.lib.tb_tree_attention(_attn(**bad), _cache(), None) == tb.TB_ERR_INVALID


def test_attention_refuses_other_caches_and_takes_nothing_to_do():
    inv = tb.TB_ERR_INVALID
    assert tb.lib.tb_tree_attention(_attn(), _cache(head_bytes=64, page_stride=1 << 16), None) == inv
    assert tb.lib.tb_tree_attention(_attn(), _cache(page_stride=16 * 2 * 128 + 8), None) == inv
    assert tb.lib.tb_tree_attention(None, _cache(), None) == inv
    assert tb.lib.tb_tree_attention(_attn(), None, None) == inv
    assert tb.lib.tb_tree_attention(_attn(batch=0), _cache(), None) == tb.TB_OK
    assert tb.lib.tb_tree_attention(_attn(nodes=0), _cache(), None) == tb.TB_OK
    n = ctypes.c_uint64()
    assert tb.lib.tb_tree_attention_workspace(_attn(head_dim=1), _cache(), ctypes.byref(n)) == inv
    assert tb.lib.tb_tree_attention_workspace(_attn(), _cache(), None) == inv
    assert tb.lib.tb_tree_attention_workspace(_attn(batch=1 << 16, nodes=1 << 6), _cache(), ctypes.byref(n)) == inv
    for nothing in (dict(batch=0), dict(nodes=0)):
        n.value = 7
        assert tb.lib.tb_tree_attention_workspace(_attn(**nothing), _cache(), ctypes.byref(n)) == tb.TB_OK
        assert n.value == 0


def test_python_refuses_host_tensors():
    with pytest.raises(ValueError):
        PagedCache(torch.zeros(2, 8, 16, 2, 64, dtype=torch.bfloat16), 16, 4, 6)
    with pytest.raises(ValueError):
        PagedCache([], 16, 4, 6)
    with pytest.raises(ValueError):
        PagedCache(torch.zeros(2, 8, 16, 2, 64), 16, 4, 6, layout="other")

    class Stub:
        dtype, device = torch.bfloat16, torch.device("cpu")
    with pytest.raises(ValueError):
        tree_attention(torch.zeros(1, 1, 2, 64), None, None, Stub(), 0, None)
