"""ctypes binding of the serving step's entry points of libtb.so
(include/tb_serve.h): argument marshalling only, with the C calls' names.
"""
import ctypes
import struct

from ._tb import lib
from ._tb_cache import _check, tb_cache, tb_tree_attn

TB_FP32 = 2   # beside TB_BF16 and TB_FP16
TB_VERIFY_MAX_VOCAB = 1 << 24
TB_VERIFY_MAX_ENTRIES = 1 << 38
TB_FP4_BLOCK = 32

# Every symbol include/tb_serve.h declares.
EXPORTS = (
    "tb_verify_drafts", "tb_verify_workspace", "tb_fp4_append", "tb_page_read", "tb_fp4_read",
    "tb_view_attention_workspace", "tb_view_attention",
)

_u64, _u32, _vp = ctypes.c_uint64, ctypes.c_uint32, ctypes.c_void_p


def TB_FP4_HEAD_BYTES(head_dim: int) -> int:
    return head_dim // 2 + (head_dim // TB_FP4_BLOCK + 3) // 4 * 4


class tb_verify(ctypes.Structure):
    _fields_ = [("probs", _vp), ("draft_probs", _vp), ("probs_stride", _u64 * 2), ("draft_stride", _u64 * 2),
                ("tokens", _vp), ("parents", _vp), ("uniform", _vp), ("tree_nodes", _vp), ("batch", _u32),
                ("nodes", _u32), ("vocab", _u32), ("dtype", _u32), ("count", _vp), ("path", _vp), ("token", _vp),
                ("seqs", _vp), ("lens", _vp), ("max_seqs", _u32), ("new_lens", _vp), ("append_seqs", _vp),
                ("append_positions", _vp), ("append_index", _vp), ("workspace", _vp), ("workspace_bytes", _u64)]


class tb_attn_view(ctypes.Structure):
    _fields_ = [("window", _u32), ("sinks", _u32), ("depths", _vp), ("fp4", _u32)]


_cache_p, _attn_p, _view_p = ctypes.POINTER(tb_cache), ctypes.POINTER(tb_tree_attn), ctypes.POINTER(tb_attn_view)
_verify_p, _u64_p = ctypes.POINTER(tb_verify), ctypes.POINTER(_u64)
_SIGS = {
    "tb_verify_drafts": [_verify_p, _vp],
    "tb_verify_workspace": [_verify_p, _u64_p],
    "tb_fp4_append": [_cache_p, _u32, _u32, _vp, _u64, _u64, _u64, _vp, _vp, _vp, _u32, _vp],
    "tb_page_read": [_cache_p, _u32, _u32, _vp, _u64, _u64, _vp, _vp, _u32, _vp],
    "tb_fp4_read": [_cache_p, _u32, _u32, _u32, _u32, _vp, _u64, _u64, _vp, _vp, _u32, _vp],
    "tb_view_attention_workspace": [_attn_p, _view_p, _cache_p, _u64_p],
    "tb_view_attention": [_attn_p, _view_p, _cache_p, _vp],
}
for _name, _args in _SIGS.items():
    _f = getattr(lib, _name)
    _f.restype = ctypes.c_int
    _f.argtypes = _args

# tb_verify and tb_attn_view as bytes, one value a field in order (filling the ctypes structures takes longer).
pack_verify = struct.Struct("=2Q4Q4Q4I3Q2QI4x4Q2Q").pack
pack_view = struct.Struct("=2IQI4x").pack
_verify_packed = lib["tb_verify_drafts"]
_verify_packed.restype = ctypes.c_int
_verify_packed.argtypes = [ctypes.c_char_p, _vp]
_attention_packed = lib["tb_view_attention"]
_attention_packed.restype = ctypes.c_int
_attention_packed.argtypes = [ctypes.c_char_p, ctypes.c_char_p, _cache_p, _vp]


def tb_verify_workspace(verify: tb_verify) -> int:
    n = _u64()
    _check("tb_verify_workspace", lib.tb_verify_workspace(verify, ctypes.byref(n)))
    return n.value


def tb_verify_drafts(verify, stream: int) -> None:
    """verify: a tb_verify, or the bytes of one from pack_verify."""
    call = _verify_packed if isinstance(verify, bytes) else lib.tb_verify_drafts
    _check("tb_verify_drafts", call(verify, stream))


def tb_fp4_append(cache: tb_cache, dtype: int, head_dim: int, rows_ptr: int, nrows: int, row_stride: int,
                  pool_stride: int, seqs_ptr: int, positions_ptr: int, index_ptr: int, n: int, stream: int) -> None:
    """index_ptr 0: row i for entry i."""
    _check("tb_fp4_append", lib.tb_fp4_append(cache, dtype, head_dim, rows_ptr, nrows, row_stride, pool_stride,
                                              seqs_ptr, positions_ptr, index_ptr or None, n, stream))


def tb_page_read(cache: tb_cache, first_pool: int, npools: int, out_ptr: int, row_stride: int, pool_stride: int,
                 seqs_ptr: int, positions_ptr: int, n: int, stream: int) -> None:
    _check("tb_page_read", lib.tb_page_read(cache, first_pool, npools, out_ptr, row_stride, pool_stride, seqs_ptr,
                                            positions_ptr, n, stream))


def tb_fp4_read(cache: tb_cache, dtype: int, head_dim: int, first_pool: int, npools: int, out_ptr: int,
                row_stride: int, pool_stride: int, seqs_ptr: int, positions_ptr: int, n: int, stream: int) -> None:
    _check("tb_fp4_read", lib.tb_fp4_read(cache, dtype, head_dim, first_pool, npools, out_ptr, row_stride,
                                          pool_stride, seqs_ptr, positions_ptr, n, stream))


def tb_view_attention_workspace(attn: tb_tree_attn, view: tb_attn_view, cache: tb_cache) -> int:
    n = _u64()
    _check("tb_view_attention_workspace", lib.tb_view_attention_workspace(attn, view, cache, ctypes.byref(n)))
    return n.value


def tb_view_attention(attn, view, cache: tb_cache, stream: int) -> None:
    """attn and view: a tb_tree_attn and a tb_attn_view, or the bytes of both from pack_tree_attn and pack_view."""
    call = _attention_packed if isinstance(attn, bytes) else lib.tb_view_attention
    _check("tb_view_attention", call(attn, view, cache, stream))
