"""Torch conveniences over the C ABI: torch supplies device memory, pinned
host memory and streams; every step of the path runs in libtb.

    RotatedSources   K slices per source (PR #365 rotation), prepared with
                     tb_prep_reference + tb_prep_sources
    reduce_copy      tb_reduce_copy on tensors / raw device addresses
    make_desc        (src_off, dst_off, bytes) offsets -> device tb_copy_desc array
    batched_copy     tb_batched_copy on a device descriptor tensor
    DescRing         tb_ring_* (descriptor-slot ring) over host descriptor arrays
    PagedCache       a paged key/value cache: tb_page_* over tensors
    tree_attention   tb_tree_attention of drafted tokens over a PagedCache, or over
                     a window of it (tb_view_attention)
    verify_drafts    tb_verify_drafts: which of the drafted tokens hold, and the next one
"""
import ctypes
import math
from contextlib import nullcontext
from typing import List, NamedTuple, Optional, Sequence, Tuple, Union

import numpy as np
import torch
from torch.autograd import forward_ad

from . import _tb, _tb_cache, _tb_serve


def stream_handle(stream: Optional[torch.cuda.Stream] = None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def _addr(x) -> int:
    return int(x.data_ptr()) if isinstance(x, torch.Tensor) else int(x)


def host_reference(nfloats: int, buffer_idx: int, fill=None, pin: bool = True) -> torch.Tensor:
    """PrepareReference of one source into a (pinned) host float32 tensor."""
    t = torch.empty(nfloats, dtype=torch.float32, pin_memory=pin and torch.cuda.is_available())
    if nfloats:
        _tb.tb_prep_reference(t.data_ptr(), nfloats, buffer_idx, fill)
    return t


class RotatedSources:
    """nsrc sources of nfloats floats, each replicated into K slices."""

    def __init__(self, nsrc: int, nfloats: int, rotate_bytes: int, fill=None,
                 device: Optional[torch.device] = None, host_refs: Optional[Sequence[torch.Tensor]] = None,
                 stream: Optional[torch.cuda.Stream] = None):
        self.nsrc = nsrc
        self.nfloats = nfloats
        self.num_bytes = nfloats * 4
        self.k = _tb.tb_num_slices(self.num_bytes, rotate_bytes)
        self.stride = _tb.tb_slice_stride(self.num_bytes)
        dev = device or torch.device("cuda", torch.cuda.current_device())
        self.buffers: List[torch.Tensor] = [
            torch.empty(max(1, self.k * self.stride), dtype=torch.uint8, device=dev) for _ in range(nsrc)]
        sh = stream_handle(stream)
        self.host_refs = list(host_refs) if host_refs is not None else [
            host_reference(nfloats, b, fill) for b in range(nsrc)]
        for b in range(nsrc):
            _tb.tb_prep_sources(self.buffers[b].data_ptr(), self.stride, self.k,
                                self.host_refs[b].data_ptr(), nfloats, sh)

    @property
    def bases(self) -> List[int]:
        return [int(b.data_ptr()) for b in self.buffers]

    def pointers(self, iteration: int) -> List[int]:
        """Device addresses of the slices iteration `iteration` reads (untimed host arithmetic)."""
        return _tb.tb_rotate_sources(self.bases, self.stride, self.k, iteration)

    def slice_view(self, b: int, s: int) -> torch.Tensor:
        """Source b, slice s, as a float32 tensor view."""
        off = s * self.stride
        return self.buffers[b][off:off + self.num_bytes].view(torch.float32)


def reduce_copy(dst, srcs, nfloats: Optional[int] = None, stream: Optional[torch.cuda.Stream] = None,
                memset_byte: int = 0) -> None:
    """dst = srcs[0] + ... (fixed order) via tb_reduce_copy; tensors or device addresses."""
    if isinstance(dst, torch.Tensor):
        if dst.dtype != torch.float32 or not dst.is_cuda or not dst.is_contiguous():
            raise ValueError("dst must be a contiguous float32 CUDA tensor")
        if nfloats is None:
            nfloats = dst.numel()
        elif nfloats > dst.numel():
            raise ValueError("nfloats exceeds dst")
    elif nfloats is None:
        raise ValueError("nfloats is required with raw addresses")
    for s in srcs:
        if isinstance(s, torch.Tensor) and (s.dtype != torch.float32 or not s.is_cuda or not s.is_contiguous()
                                            or s.numel() < nfloats):
            raise ValueError("sources must be contiguous float32 CUDA tensors of at least nfloats elements")
    _tb.tb_reduce_copy(_addr(dst), [_addr(s) for s in srcs], nfloats, stream_handle(stream), memset_byte)


def make_desc(offsets: np.ndarray, src_base: int, dst_base: int, device=None) -> torch.Tensor:
    """Device int64 tensor (n, 3) of tb_copy_desc records from (src_off, dst_off, bytes) offsets."""
    o = np.ascontiguousarray(offsets, dtype=np.uint64).reshape(-1, 3)
    d = o.copy()
    d[:, 0] += np.uint64(src_base)
    d[:, 1] += np.uint64(dst_base)
    dev = device or torch.device("cuda", torch.cuda.current_device())
    return torch.from_numpy(d.view(np.int64)).to(dev)


def batched_copy(desc: torch.Tensor, ncopies: Optional[int] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> None:
    """tb_batched_copy over a device (n, 3) int64 descriptor tensor."""
    if (desc.dtype != torch.int64 or not desc.is_cuda or not desc.is_contiguous() or desc.dim() != 2
            or desc.shape[1] != 3):
        raise ValueError("desc must be a contiguous int64 CUDA tensor of shape (n, 3)")
    n = desc.shape[0] if ncopies is None else ncopies
    if not 0 <= n <= desc.shape[0]:
        raise ValueError("ncopies must be between 0 and the number of descriptors in desc")
    _tb.tb_batched_copy(desc.data_ptr(), n, stream_handle(stream))


class DescRing:
    """Descriptor-slot ring on the current device: submit host (n, 3) uint64
    descriptor arrays (absolute src, dst, bytes) and poll their tickets.
    direct: the kernel reads the pinned slots itself (faster in every measured
    case); otherwise each slot is first copied to device memory."""

    def __init__(self, nslots: int = 32, slot_descs: int = 8192, direct: bool = True,
                 stream: Optional[torch.cuda.Stream] = None):
        self.handle = _tb.tb_ring_create(nslots, slot_descs, _tb.TB_RING_DIRECT if direct else _tb.TB_RING_STAGED,
                                         stream_handle(stream))

    def submit(self, desc: np.ndarray) -> int:
        d = np.ascontiguousarray(desc, dtype=np.uint64).reshape(-1, 3)
        return _tb.tb_ring_submit(self.handle, d.ctypes.data, d.shape[0])

    def poll(self, ticket: int) -> bool:
        return _tb.tb_ring_poll(self.handle, ticket)

    def wait(self, ticket: int) -> None:
        _tb.tb_ring_wait(self.handle, ticket)

    def close(self) -> None:
        if self.handle:
            h, self.handle = self.handle, 0
            _tb.tb_ring_destroy(h)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


_NO_CONTEXT = nullcontext()


def _list_arg(t: torch.Tensor, n: Optional[int], device: torch.device, what: str) -> int:
    """Address of an int32 index list on the cache's device."""
    if (not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.device != device or t.dim() != 1
            or not t.is_contiguous() or (n is not None and t.shape[0] != n)):
        raise ValueError(f"{what} must be a contiguous one-dimensional int32 tensor on {device}"
                         + ("" if n is None else f" of {n} entries"))
    return t.data_ptr()


def _no_gradient(what: str, *tensors: Optional[torch.Tensor]) -> None:
    """Refuses tensors whose gradient, or tangent in forward mode, the call would drop."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise ValueError(f"{what} has no gradient: call it under torch.no_grad(), or detach its tensors")
    # outside of a level no tensor has a tangent; where torch does not tell the level, each one is asked
    if getattr(forward_ad, "_current_level", 0) >= 0:
        for t in tensors:
            if t is not None and forward_ad.unpack_dual(t).tangent is not None:
                raise ValueError(f"{what} has no forward mode: its tensors must carry no tangent")


_ATTN_TYPES = {torch.bfloat16: _tb_cache.TB_BF16, torch.float16: _tb_cache.TB_FP16}


def fp4_head_bytes(head_dim: int) -> int:
    """Bytes of a head of head_dim elements in a cache held in 4 bits: half a byte an element, one for each 32 of
    them, rounded up to a multiple of 4."""
    if head_dim < 32 or head_dim % 32 != 0:
        raise ValueError("a head held in 4 bits has a multiple of 32 elements")
    return _tb_serve.TB_FP4_HEAD_BYTES(head_dim)


class PagedCache:
    """A paged key/value cache over tensors (include/tb_cache.h).

    pools        a tensor [npools, num_pages, ...] or a sequence of tensors
                 [num_pages, ...]: keys of layer l in pool 2 l, values in 2 l + 1.
                 A page is [page_tokens, heads, head_dim] (layout "token") or
                 [heads, page_tokens, head_dim] (layout "head"), contiguous.
    max_seqs     rows of the table, each of max_pages pages
    state        an int32 tensor of state_words() words with a state to go on
                 from; by default a new one, empty
    fp4          torch.bfloat16 or torch.float16: the pools are uint8, head_dim
                 being fp4_head_bytes() of the elements, and hold elements of that
                 type in 4 bits (include/tb_serve.h): append() rounds, read() and
                 tree_attention() give back what is held.  All else is alike.

    table, lens, refs, free_list and counts are views of `state`, on the device:
    copying `state` keeps the whole bookkeeping.  Index lists are contiguous
    int32 tensors on the cache's device; a negative entry is padding.  Every
    call only enqueues on the current stream of the cache's device, or on `stream`;
    the caller orders calls on one cache (a new one's state is written on the current stream).  What a listed entry asked for and
    could not have shows in counts[1] (TB_CACHE_* bits, see flags())."""

    def __init__(self, pools: Union[torch.Tensor, Sequence[torch.Tensor]], page_tokens: int, max_seqs: int,
                 max_pages: int, layout: str = "token", state: Optional[torch.Tensor] = None,
                 fp4: Optional[torch.dtype] = None):
        if layout not in ("token", "head"):
            raise ValueError("layout must be 'token' or 'head'")
        pools = list(pools)   # of a tensor: its pools
        if not 1 <= len(pools) <= _tb_cache.TB_MAX_POOLS:
            raise ValueError(f"a cache has 1 to {_tb_cache.TB_MAX_POOLS} pools")
        p0 = pools[0]
        for p in pools:
            if (not p.is_cuda or p.device != p0.device or p.dtype != p0.dtype or p.shape != p0.shape
                    or p.stride() != p0.stride()):
                raise ValueError("pools must be CUDA tensors of one device, type, shape and stride")
        _no_gradient("a paged cache", *pools)
        if p0.dim() != 4 or p0.shape[1 if layout == "token" else 2] != page_tokens or not p0[:1].is_contiguous():
            raise ValueError("a pool is [num_pages, page_tokens, heads, head_dim] (layout 'token') or "
                             "[num_pages, heads, page_tokens, head_dim] (layout 'head'), pages contiguous")
        self.pools, self.layout, self.page_tokens = pools, layout, page_tokens
        self.num_pages, self.head_dim = p0.shape[0], p0.shape[3]
        if fp4 is not None:
            dim = p0.shape[3] // 17 * 32   # 17 bytes for 32 elements, and up to 3
            if (fp4 not in _ATTN_TYPES or p0.dtype != torch.uint8 or dim == 0
                    or _tb_serve.TB_FP4_HEAD_BYTES(dim) != p0.shape[3]):
                raise ValueError("a cache held in 4 bits has uint8 pools with fp4_head_bytes(head_dim) bytes a head, "
                                 "and fp4 is bfloat16 or float16")
            if any(p.data_ptr() % 4 or (p.shape[0] > 1 and p.stride(0) % 4) for p in pools):
                raise ValueError("pools held in 4 bits begin, and their pages lie, at multiples of 4 bytes")
        self.heads = p0.shape[2 if layout == "token" else 1]
        self.max_seqs, self.max_pages = max_seqs, max_pages
        self.device, self.dtype = p0.device, p0.dtype
        page = page_tokens * self.heads * self.head_dim
        head_bytes = self.head_dim * p0.element_size()
        self.fp4 = fp4
        if fp4 is not None:
            self.head_dim, self.dtype = dim, fp4
        words = self.state_words(self.num_pages, max_seqs, max_pages)
        fresh = state is None
        if fresh:
            state = torch.empty(words, dtype=torch.int32, device=self.device)
            state[:max_seqs * max_pages] = 0
        elif (state.dtype != torch.int32 or state.device != self.device or state.dim() != 1
              or not state.is_contiguous() or state.shape[0] != words):
            raise ValueError(f"state must be a contiguous int32 tensor of {words} words on {self.device}")
        self.state = state
        cuts = [max_seqs * max_pages, max_seqs, self.num_pages, self.num_pages, 4]
        table, self.lens, self.refs, self.free_list, self.counts = torch.split(state, cuts)
        self.table = table.view(max_seqs, max_pages)
        self._scratch = torch.zeros(_tb_cache.tb_cache_scratch_bytes(self.num_pages, max_seqs), dtype=torch.uint8,
                                    device=self.device)
        self._pool_ptrs = (ctypes.c_void_p * len(pools))(*[p.data_ptr() for p in pools])
        c = _tb_cache.tb_cache()
        c.pools = ctypes.addressof(self._pool_ptrs)
        c.npools, c.num_pages, c.page_tokens, c.heads = len(pools), self.num_pages, page_tokens, self.heads
        c.layout = _tb_cache.TB_CACHE_TOKEN_MAJOR if layout == "token" else _tb_cache.TB_CACHE_HEAD_MAJOR
        size = p0.element_size()
        c.head_bytes = head_bytes
        c.page_stride = (p0.stride(0) if self.num_pages > 1 else page) * size
        c.max_seqs, c.max_pages = max_seqs, max_pages
        c.table, c.lens, c.refs = self.table.data_ptr(), self.lens.data_ptr(), self.refs.data_ptr()
        c.free_list, c.counts = self.free_list.data_ptr(), self.counts.data_ptr()
        c.scratch = self._scratch.data_ptr()
        self._c = c
        if fresh:
            with self._there():
                _tb_cache.tb_cache_init(c, self._stream(None))

    @staticmethod
    def state_words(num_pages: int, max_seqs: int, max_pages: int) -> int:
        return max_seqs * max_pages + max_seqs + 2 * num_pages + 4

    def _there(self):
        """The cache's device as the current one, for the length of a call."""
        return _NO_CONTEXT if torch._C._cuda_getDevice() == self.device.index else torch.cuda.device(self.device)

    def _stream(self, stream: Optional[torch.cuda.Stream]) -> int:
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self.device.index)   # without building a Stream object
        if stream.device != self.device:
            raise ValueError(f"the stream must be one of {self.device}")
        return int(stream.cuda_stream)

    def flags(self, clear: bool = False) -> int:
        """The TB_CACHE_* bits raised so far (waits for the device)."""
        bits = int(self.counts[1])
        if clear:
            self.counts[1] = 0
        return bits

    def copy_pages(self, dst_pages: torch.Tensor, src_pages: torch.Tensor, src: Optional["PagedCache"] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> None:
        """Copy src's pages src_pages (of this cache by default) to dst_pages, in every pool."""
        src = self if src is None else src
        if src.device != self.device or src.dtype != self.dtype or src.fp4 != self.fp4:
            raise ValueError("both caches must be of one device and type")
        d = _list_arg(dst_pages, None, self.device, "dst_pages")
        s = _list_arg(src_pages, len(dst_pages), self.device, "src_pages")
        with self._there():
            _tb_cache.tb_page_copy(self._c, src._c, d, s, len(dst_pages), self._stream(stream))

    def append(self, rows: torch.Tensor, seqs: torch.Tensor, positions: torch.Tensor,
               index: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> None:
        """Write rows[:, index[i]] ([npools, n, heads, head_dim]) to position positions[i] of sequence seqs[i].
        A cache held in 4 bits takes rows of its type and rounds them: each 32 elements of a head to a common power
        of two times 0, 0.5, 1, 1.5, 2, 3, 4 or 6, either sign.  A position listed twice holds a mixture there."""
        shape, stride = rows.shape, rows.stride()
        if (rows.dtype != self.dtype or rows.device != self.device or len(shape) != 4 or shape[0] != len(self.pools)
                or shape[2] != self.heads or shape[3] != self.head_dim or stride[3] != 1
                or (self.heads > 1 and stride[2] != self.head_dim)):
            raise ValueError("rows must be [npools, n, heads, head_dim] of the cache's type and device, "
                             "each token contiguous")
        _no_gradient("append", rows)
        n = len(seqs)
        q, p = _list_arg(seqs, None, self.device, "seqs"), _list_arg(positions, n, self.device, "positions")
        x = 0 if index is None else _list_arg(index, n, self.device, "index")
        if index is None and shape[1] < n:
            raise ValueError("rows must hold a row for each entry")
        size = rows.element_size()
        step = stride[1] if shape[1] > 1 else self.heads * self.head_dim
        with self._there():
            if self.fp4 is None:
                _tb_cache.tb_page_append(self._c, rows.data_ptr(), shape[1], step * size, stride[0] * size, q, p, x,
                                         n, self._stream(stream))
            else:
                _tb_serve.tb_fp4_append(self._c, _ATTN_TYPES[self.fp4], self.head_dim, rows.data_ptr(), shape[1],
                                        step * size, stride[0] * size, q, p, x, n, self._stream(stream))

    def read(self, seqs: torch.Tensor, positions: torch.Tensor, layer: Optional[int] = None,
             out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """What position positions[i] of sequence seqs[i] holds: [npools, n, heads, head_dim], or with `layer` the two
        pools of that layer.  append()'s way back; a cache held in 4 bits gives the numbers that it holds.
        A negative sequence reads as zeros, and so does what is out of range, with TB_CACHE_RANGE."""
        q = _list_arg(seqs, None, self.device, "seqs")
        n = seqs.shape[0]
        p = _list_arg(positions, n, self.device, "positions")
        if layer is None:
            first, count = 0, len(self.pools)
        elif 0 <= layer < len(self.pools) // 2:
            first, count = 2 * layer, 2
        else:
            raise ValueError("the cache has no such layer")
        shape = (count, n, self.heads, self.head_dim)
        if out is not None:
            st = out.stride()
            if (out.dtype != self.dtype or out.device != self.device or out.shape != shape or st[3] != 1
                    or (self.heads > 1 and st[2] != self.head_dim)):
                raise ValueError(f"out must be {self.dtype} of shape {shape} on {self.device}, each token contiguous")
            _no_gradient("read", out)
        with self._there(), _NO_CONTEXT if stream is None else torch.cuda.stream(stream):
            if out is None:   # it belongs to the stream that the call runs on
                out = torch.empty(shape, dtype=self.dtype, device=self.device)
            size = out.element_size()
            row = self.heads * self.head_dim
            step = (out.stride(1) if n > 1 else row) * size
            apart = (out.stride(0) if count > 1 else n * row) * size
            if self.fp4 is None:
                _tb_serve.tb_page_read(self._c, first, count, out.data_ptr(), step, apart, q, p, n, self._stream(stream))
            else:
                _tb_serve.tb_fp4_read(self._c, _ATTN_TYPES[self.fp4], self.head_dim, first, count, out.data_ptr(),
                                      step, apart, q, p, n, self._stream(stream))
        return out

    def fork(self, parents: torch.Tensor, children: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> None:
        """Make the empty sequences `children` copies of `parents`, sharing their full pages."""
        p = _list_arg(parents, None, self.device, "parents")
        c = _list_arg(children, len(parents), self.device, "children")
        with self._there():
            _tb_cache.tb_page_fork(self._c, p, c, len(parents), self._stream(stream))

    def resize(self, seqs: torch.Tensor, lens: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> None:
        """Give the sequences `seqs` the lengths `lens`, 0 freeing one: releases pages, then takes new ones.

        A sequence that was cut back into a page which another one shares cannot grow in it: it is skipped, with
        TB_CACHE_SHARED.  Fork it to an empty row, whose last page is its own, and go on with that one."""
        q = _list_arg(seqs, None, self.device, "seqs")
        n = _list_arg(lens, len(seqs), self.device, "lens")
        with self._there():
            _tb_cache.tb_page_resize(self._c, q, n, len(seqs), self._stream(stream))

    def free(self, seqs: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> None:
        """Free whole sequences."""
        with torch.cuda.stream(stream) if stream is not None else _NO_CONTEXT:
            zero = torch.zeros_like(seqs)
        self.resize(seqs, zero, stream)

    def compact(self, stream: Optional[torch.cuda.Stream] = None) -> None:
        """Move the pages in use to the lowest numbers."""
        with self._there():
            _tb_cache.tb_page_compact(self._c, self._stream(stream))


def tree_attention_workspace(q: torch.Tensor, cache: PagedCache) -> torch.Tensor:
    """Workspace for tree_attention calls with queries of q's shape over `cache`, whatever the lengths.
    One serves any number of calls that follow each other; calls that can overlap need one each."""
    a = _tb_cache.tb_tree_attn()
    a.batch, a.nodes, a.heads_q, a.head_dim = q.shape
    with cache._there():
        if cache.fp4 is None:
            n = _tb_cache.tb_tree_attention_workspace(a, cache._c)
        else:
            n = _tb_serve.tb_view_attention_workspace(a, _tb_serve.tb_attn_view(fp4=1), cache._c)
    return torch.empty(n, dtype=torch.uint8, device=cache.device)


def tree_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cache: PagedCache, layer: int,
                   seqs: torch.Tensor, mask: Optional[torch.Tensor] = None, nodes: Optional[torch.Tensor] = None,
                   scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None, window: Optional[int] = None, sinks: int = 0,
                   depths: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of drafted tokens over the cache's context of `layer` and over each other.

    q [batch, nodes, heads_q, head_dim]; k, v [batch, nodes, heads, head_dim] of the drafted tokens, which are
    not in the cache.  seqs [batch]: the sequences' rows in the cache.  mask int64 [batch, nodes, ceil(nodes /
    64)]: bit u % 64 of word u / 64 lets a node see node u (default: node t sees u <= t, so that one node is
    ordinary decoding).  nodes int32 [batch]: how many of the nodes are real (default: all).  scale: 1 /
    sqrt(head_dim) by default.  Returns (out, lse): out as q, lse float32 [batch, nodes, heads_q], the natural
    logarithm of the sum of exponentials; a row that sees nothing is 0 and -inf.

    window: a node sees what lies less than `window` positions before its own (1: itself only), and the first `sinks`
    tokens of the sequence; its position is the sequence's length plus its depth.  depths int32 [batch, nodes]: of
    each node in its tree (default: node t's is t, which a chain's are; a mask with a window needs them, without a
    window they have no effect).
    The cache may be held in 4 bits (fp4), of q's type.

    For serving: there is no gradient and no forward mode, and tensors that carry either are refused."""
    dtype, dev = q.dtype, cache.device
    kind = _ATTN_TYPES.get(dtype)
    if kind is None or cache.dtype != dtype:
        raise ValueError("q and the cache must be both bfloat16 or both float16")
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q must be [batch, nodes, heads_q, head_dim]")
    b, t, hq, d = shape
    if d != cache.head_dim:
        raise ValueError("q's head_dim must be the cache's")
    if not 0 <= layer < len(cache.pools) // 2:
        raise ValueError("the cache has no such layer")
    kv_shape = (b, t, cache.heads, d)
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    if q.device != dev or qs[3] != 1:
        raise ValueError(f"q must be on {dev}, head_dim contiguous")
    for x, st in ((k, ks), (v, vs)):
        if x.dtype != dtype or x.device != dev or x.shape != kv_shape or st[3] != 1:
            raise ValueError(f"k and v must be {dtype} of shape {kv_shape} on {dev}, head_dim contiguous")
    _no_gradient("tree_attention", q, k, v, cache.pools[2 * layer], cache.pools[2 * layer + 1], out, lse)
    sq = _list_arg(seqs, b, dev, "seqs")
    if mask is not None and (mask.dtype != torch.int64 or mask.device != dev or mask.shape != (b, t, (t + 63) // 64)
                             or not mask.is_contiguous()):
        raise ValueError(f"mask must be a contiguous int64 tensor of shape {(b, t, (t + 63) // 64)} on {dev}")
    tn = 0 if nodes is None else _list_arg(nodes, b, dev, "nodes")
    if out is not None and (out.dtype != dtype or out.device != dev or out.shape != shape or out.stride(3) != 1):
        raise ValueError("out must have q's type, shape and device, head_dim contiguous")
    if lse is not None and (lse.dtype != torch.float32 or lse.device != dev or lse.shape != (b, t, hq)
                            or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 tensor [batch, nodes, heads_q]")
    if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous tensor on the cache's device")
    if window is not None and not 1 <= window < 1 << 32:
        raise ValueError("window must be at least 1")
    if not 0 <= sinks < 1 << 32:
        raise ValueError("sinks must not be negative")
    if window is None and sinks:
        raise ValueError("sinks go with a window")
    if depths is not None and (depths.dtype != torch.int32 or depths.device != dev or depths.shape != (b, t)
                               or not depths.is_contiguous()):
        raise ValueError(f"depths must be a contiguous int32 tensor of shape {(b, t)} on {dev}")
    if window is not None and mask is not None and depths is None:
        raise ValueError("a mask with a window needs the nodes' depths")
    # what is allocated here belongs to the stream that the call runs on
    with cache._there(), _NO_CONTEXT if stream is None else torch.cuda.stream(stream):
        sh = cache._stream(stream)
        if out is None:
            out = q.new_empty(shape)
        if lse is None:
            lse = q.new_empty((b, t, hq), dtype=torch.float32)
        if workspace is None:
            workspace = tree_attention_workspace(q, cache)
        a = _tb_cache.pack_tree_attn(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), *qs[:3], *ks[:3], *vs[:3],
            *out.stride()[:3], sq, 0 if mask is None else mask.data_ptr(), tn, b, t, hq, d, kind, 2 * layer,
            2 * layer + 1, 1 / math.sqrt(d) if scale is None else scale, workspace.data_ptr(), workspace.nbytes)
        if window is None and cache.fp4 is None:
            _tb_cache.tb_tree_attention(a, cache._c, sh)
        else:
            view = _tb_serve.pack_view(window or 0, sinks, 0 if depths is None else depths.data_ptr(),
                                       0 if cache.fp4 is None else 1)
            _tb_serve.tb_view_attention(a, view, cache._c, sh)
    return out, lse


_PROB_TYPES = {torch.float32: _tb_serve.TB_FP32, **_ATTN_TYPES}


class Verified(NamedTuple):
    """What verify_drafts returns, all int32 on the device."""
    count: torch.Tensor                                # [batch]: accepted nodes, the root among them
    path: torch.Tensor                                 # [batch, nodes]: their numbers, then -1
    token: torch.Tensor                                # [batch]: the next token, -1 where there is none
    lens: Optional[torch.Tensor] = None                # with a cache: [batch], for resize()
    append_seqs: Optional[torch.Tensor] = None         # and [batch * nodes] each, for append() of
    append_positions: Optional[torch.Tensor] = None    # rows of which b * nodes + t is node t of
    append_index: Optional[torch.Tensor] = None        # sequence b


def verify_drafts_workspace(probs: torch.Tensor) -> torch.Tensor:
    """Workspace for verify_drafts calls with probabilities of this shape.  One serves any number of calls that
    follow each other; calls that can overlap need one each."""
    v = _tb_serve.tb_verify(batch=probs.shape[0], vocab=probs.shape[2])
    return torch.empty(_tb_serve.tb_verify_workspace(v), dtype=torch.uint8, device=probs.device)


def verify_drafts(probs: torch.Tensor, tokens: torch.Tensor, uniform: torch.Tensor,
                  parents: Optional[torch.Tensor] = None, draft_probs: Optional[torch.Tensor] = None,
                  nodes: Optional[torch.Tensor] = None, cache: Optional[PagedCache] = None,
                  seqs: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> Verified:
    """Which of the drafted tokens hold, so that they and the next one are distributed as the target's (the rule is
    tb_verify_drafts' in include/tb_serve.h).

    probs [batch, nodes, vocab]: the target's distribution of what follows each node; node 0 is the root, the last
    token that holds already.  tokens int32 [batch, nodes]: what the nodes propose.  uniform float32 [batch, nodes]:
    random numbers in [0, 1), a node's for its test, the root's for the next token.  parents int32 [batch, nodes], each
    below its node (default: chains).  draft_probs as probs: row t is what node t's children were drawn from,
    independently of each other; None: they were chosen, not drawn.  nodes int32 [batch]: how many are real.
    Probabilities are float32, bfloat16 or float16, any strides, the vocabulary contiguous.

    With cache and seqs int32 [batch], their rows in it, the result has the lengths and lists with which
    cache.resize(seqs, r.lens) and cache.append(rows, r.append_seqs, r.append_positions, r.append_index) take the
    accepted nodes into it."""
    dev, kind = probs.device, _PROB_TYPES.get(probs.dtype)
    if kind is None or probs.dim() != 3 or not probs.is_cuda or (probs.shape[2] > 1 and probs.stride(2) != 1):
        raise ValueError("probs must be a float32, bfloat16 or float16 CUDA tensor [batch, nodes, vocab], "
                         "the vocabulary contiguous")
    b, t, vocab = probs.shape
    if not (1 <= t <= 4096 and b <= 65536 and 1 <= vocab <= _tb_serve.TB_VERIFY_MAX_VOCAB
            and b * vocab <= _tb_serve.TB_VERIFY_MAX_ENTRIES):
        raise ValueError("probs must have 1 to 4096 nodes, up to 65536 sequences and 2^24 entries of the vocabulary, "
                         "2^38 of all sequences together")
    if draft_probs is not None and (draft_probs.dtype != probs.dtype or draft_probs.device != dev
                                    or draft_probs.shape != probs.shape
                                    or (vocab > 1 and draft_probs.stride(2) != 1)):
        raise ValueError("draft_probs must have probs' type, shape and device, the vocabulary contiguous")
    _no_gradient("verify_drafts", probs, draft_probs, uniform)
    for x, dtype, what in ((tokens, torch.int32, "tokens"), (uniform, torch.float32, "uniform"),
                           (parents, torch.int32, "parents")):
        if x is not None and (x.dtype != dtype or x.device != dev or x.shape != (b, t) or not x.is_contiguous()):
            raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {(b, t)} on {dev}")
    tn = 0 if nodes is None else _list_arg(nodes, b, dev, "nodes")
    if (cache is None) != (seqs is None):
        raise ValueError("cache and seqs go together")
    if cache is not None and cache.device != dev:
        raise ValueError("probs must be on the cache's device")
    sq = 0 if seqs is None else _list_arg(seqs, b, dev, "seqs")
    if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    if stream is not None and stream.device != dev:
        raise ValueError(f"the stream must be one of {dev}")
    there = _NO_CONTEXT if torch._C._cuda_getDevice() == dev.index else torch.cuda.device(dev)
    with there, _NO_CONTEXT if stream is None else torch.cuda.stream(stream):
        sh = torch._C._cuda_getCurrentRawStream(dev.index)
        if workspace is None:
            workspace = verify_drafts_workspace(probs)
        # one allocation, cut up
        sizes = [b, b * t, b] + ([] if cache is None else [b, b * t, b * t, b * t])
        whole = torch.empty(sum(sizes), dtype=torch.int32, device=dev)
        parts = whole.split_with_sizes(sizes)
        ptrs = [0] * 7
        at = whole.data_ptr()
        for i, size in enumerate(sizes):
            ptrs[i] = at
            at += 4 * size
        ps, ds = probs.stride(), (0, 0) if draft_probs is None else draft_probs.stride()
        v = _tb_serve.pack_verify(
            probs.data_ptr(), 0 if draft_probs is None else draft_probs.data_ptr(), ps[0], ps[1], ds[0], ds[1],
            tokens.data_ptr(), 0 if parents is None else parents.data_ptr(), uniform.data_ptr(), tn, b, t, vocab, kind,
            *ptrs[:3], sq, 0 if cache is None else cache.lens.data_ptr(), 0 if cache is None else cache.max_seqs,
            *ptrs[3:], workspace.data_ptr(), workspace.nbytes)
        _tb_serve.tb_verify_drafts(v, sh)
    return Verified(parts[0], parts[1].view(b, t), *parts[2:])
