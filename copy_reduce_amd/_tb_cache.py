"""ctypes binding of the paged cache's entry points of libtb.so
(include/tb_cache.h): argument marshalling only, with the C calls' names.
"""
import ctypes
import struct

from ._tb import TBError, TB_OK, lib

TB_MAX_POOLS = 256
TB_CACHE_TOKEN_MAJOR, TB_CACHE_HEAD_MAJOR = 0, 1
TB_CACHE_SHORT, TB_CACHE_RANGE, TB_CACHE_BUSY, TB_CACHE_TWICE, TB_CACHE_SHARED = 1, 2, 4, 8, 16
TB_BF16, TB_FP16 = 0, 1

# Every symbol include/tb_cache.h declares.
EXPORTS = (
    "tb_cache_scratch_bytes", "tb_cache_init", "tb_page_copy", "tb_page_append", "tb_page_fork",
    "tb_page_resize", "tb_page_compact", "tb_tree_attention_workspace", "tb_tree_attention",
)

_u64, _u32, _f32, _vp = ctypes.c_uint64, ctypes.c_uint32, ctypes.c_float, ctypes.c_void_p


class tb_cache(ctypes.Structure):
    _fields_ = [("pools", _vp), ("npools", _u32), ("layout", _u32), ("num_pages", _u32), ("page_tokens", _u32),
                ("heads", _u32), ("head_bytes", _u32), ("page_stride", _u64), ("max_seqs", _u32),
                ("max_pages", _u32), ("table", _vp), ("lens", _vp), ("refs", _vp), ("free_list", _vp),
                ("counts", _vp), ("scratch", _vp)]


class tb_tree_attn(ctypes.Structure):
    _fields_ = [("q", _vp), ("k", _vp), ("v", _vp), ("out", _vp), ("lse", _vp),
                ("q_stride", _u64 * 3), ("k_stride", _u64 * 3), ("v_stride", _u64 * 3), ("out_stride", _u64 * 3),
                ("seqs", _vp), ("mask", _vp), ("tree_nodes", _vp), ("batch", _u32), ("nodes", _u32),
                ("heads_q", _u32), ("head_dim", _u32), ("dtype", _u32), ("k_pool", _u32), ("v_pool", _u32),
                ("scale", _f32), ("workspace", _vp), ("workspace_bytes", _u64)]


_cache_p, _attn_p, _u64_p = ctypes.POINTER(tb_cache), ctypes.POINTER(tb_tree_attn), ctypes.POINTER(_u64)
_SIGS = {
    "tb_cache_scratch_bytes": [_u32, _u32, _u64_p],
    "tb_cache_init": [_cache_p, _vp],
    "tb_page_copy": [_cache_p, _cache_p, _vp, _vp, _u32, _vp],
    "tb_page_append": [_cache_p, _vp, _u64, _u64, _u64, _vp, _vp, _vp, _u32, _vp],
    "tb_page_fork": [_cache_p, _vp, _vp, _u32, _vp],
    "tb_page_resize": [_cache_p, _vp, _vp, _u32, _vp],
    "tb_page_compact": [_cache_p, _vp],
    "tb_tree_attention_workspace": [_attn_p, _cache_p, _u64_p],
    "tb_tree_attention": [_attn_p, _cache_p, _vp],
}
for _name, _args in _SIGS.items():
    _f = getattr(lib, _name)
    _f.restype = ctypes.c_int
    _f.argtypes = _args

# tb_tree_attn as bytes, one value a field in order: a call's arguments in a quarter of the time that
# filling the ctypes structure takes.
pack_tree_attn = struct.Struct("=5Q12Q3Q7If2Q").pack
_attention_packed = lib["tb_tree_attention"]
_attention_packed.restype = ctypes.c_int
_attention_packed.argtypes = [ctypes.c_char_p, _cache_p, _vp]


def _check(fn, status):
    if status != TB_OK:
        raise TBError(fn, status)


def tb_cache_scratch_bytes(num_pages: int, max_seqs: int) -> int:
    n = _u64()
    _check("tb_cache_scratch_bytes", lib.tb_cache_scratch_bytes(num_pages, max_seqs, ctypes.byref(n)))
    return n.value


def tb_cache_init(cache: tb_cache, stream: int) -> None:
    _check("tb_cache_init", lib.tb_cache_init(cache, stream))


def tb_page_copy(dst: tb_cache, src: tb_cache, dst_pages_ptr: int, src_pages_ptr: int, n: int, stream: int) -> None:
    _check("tb_page_copy", lib.tb_page_copy(dst, src, dst_pages_ptr, src_pages_ptr, n, stream))


def tb_page_append(cache: tb_cache, rows_ptr: int, nrows: int, row_stride: int, pool_stride: int, seqs_ptr: int,
                   positions_ptr: int, index_ptr: int, n: int, stream: int) -> None:
    """index_ptr 0: row i for entry i."""
    _check("tb_page_append", lib.tb_page_append(cache, rows_ptr, nrows, row_stride, pool_stride, seqs_ptr,
                                                positions_ptr, index_ptr or None, n, stream))


def tb_page_fork(cache: tb_cache, parents_ptr: int, children_ptr: int, n: int, stream: int) -> None:
    _check("tb_page_fork", lib.tb_page_fork(cache, parents_ptr, children_ptr, n, stream))


def tb_page_resize(cache: tb_cache, seqs_ptr: int, lens_ptr: int, n: int, stream: int) -> None:
    _check("tb_page_resize", lib.tb_page_resize(cache, seqs_ptr, lens_ptr, n, stream))


def tb_page_compact(cache: tb_cache, stream: int) -> None:
    _check("tb_page_compact", lib.tb_page_compact(cache, stream))


def tb_tree_attention_workspace(attn: tb_tree_attn, cache: tb_cache) -> int:
    n = _u64()
    _check("tb_tree_attention_workspace", lib.tb_tree_attention_workspace(attn, cache, ctypes.byref(n)))
    return n.value


def tb_tree_attention(attn, cache: tb_cache, stream: int) -> None:
    """attn: a tb_tree_attn, or the bytes of one from pack_tree_attn."""
    call = _attention_packed if isinstance(attn, bytes) else lib.tb_tree_attention
    _check("tb_tree_attention", call(attn, cache, stream))
