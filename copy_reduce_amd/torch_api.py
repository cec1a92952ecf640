"""Torch conveniences over the C ABI: torch supplies device memory, pinned
host memory and streams; every step of the path runs in libtb.

    RotatedSources   K slices per source (PR #365 rotation), prepared with
                     tb_prep_reference + tb_prep_sources
    reduce_copy      tb_reduce_copy on tensors / raw device addresses
    make_desc        (src_off, dst_off, bytes) offsets -> device tb_copy_desc array
    batched_copy     tb_batched_copy on a device descriptor tensor
    DescRing         tb_ring_* (descriptor-slot ring) over host descriptor arrays
    PagedCache       a paged key/value cache: tb_page_* over tensors
    tree_attention   tb_tree_attention of drafted tokens over a PagedCache
"""
import ctypes
import math
from contextlib import nullcontext
from typing import List, Optional, Sequence, Tuple, Union

import numpy as np
import torch
from torch.autograd import forward_ad

from . import _tb, _tb_cache


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
            or not t.is_contiguous() or (n is not None and len(t) != n)):
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


class PagedCache:
    """A paged key/value cache over tensors (include/tb_cache.h).

    pools        a tensor [npools, num_pages, ...] or a sequence of tensors
                 [num_pages, ...]: keys of layer l in pool 2 l, values in 2 l + 1.
                 A page is [page_tokens, heads, head_dim] (layout "token") or
                 [heads, page_tokens, head_dim] (layout "head"), contiguous.
    max_seqs     rows of the table, each of max_pages pages
    state        an int32 tensor of state_words() words with a state to go on
                 from; by default a new one, empty

    table, lens, refs, free_list and counts are views of `state`, on the device:
    copying `state` keeps the whole bookkeeping.  Index lists are contiguous
    int32 tensors on the cache's device; a negative entry is padding.  Every
    call only enqueues on the current stream of the cache's device, or on `stream`;
    the caller orders calls on one cache (a new one's state is written on the current stream).  What a listed entry asked for and
    could not have shows in counts[1] (TB_CACHE_* bits, see flags())."""

    def __init__(self, pools: Union[torch.Tensor, Sequence[torch.Tensor]], page_tokens: int, max_seqs: int,
                 max_pages: int, layout: str = "token", state: Optional[torch.Tensor] = None):
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
        self.heads = p0.shape[2 if layout == "token" else 1]
        self.max_seqs, self.max_pages = max_seqs, max_pages
        self.device, self.dtype = p0.device, p0.dtype
        page = page_tokens * self.heads * self.head_dim
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
        c.head_bytes = self.head_dim * size
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
        if src.device != self.device or src.dtype != self.dtype:
            raise ValueError("both caches must be of one device and type")
        d = _list_arg(dst_pages, None, self.device, "dst_pages")
        s = _list_arg(src_pages, len(dst_pages), self.device, "src_pages")
        with self._there():
            _tb_cache.tb_page_copy(self._c, src._c, d, s, len(dst_pages), self._stream(stream))

    def append(self, rows: torch.Tensor, seqs: torch.Tensor, positions: torch.Tensor,
               index: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> None:
        """Write rows[:, index[i]] ([npools, n, heads, head_dim]) to position positions[i] of sequence seqs[i]."""
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
            _tb_cache.tb_page_append(self._c, rows.data_ptr(), shape[1], step * size, stride[0] * size, q, p, x, n,
                                     self._stream(stream))

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


_ATTN_TYPES = {torch.bfloat16: _tb_cache.TB_BF16, torch.float16: _tb_cache.TB_FP16}


def tree_attention_workspace(q: torch.Tensor, cache: PagedCache) -> torch.Tensor:
    """Workspace for tree_attention calls with queries of q's shape over `cache`, whatever the lengths.
    One serves any number of calls that follow each other; calls that can overlap need one each."""
    a = _tb_cache.tb_tree_attn()
    a.batch, a.nodes, a.heads_q, a.head_dim = q.shape
    with cache._there():
        n = _tb_cache.tb_tree_attention_workspace(a, cache._c)
    return torch.empty(n, dtype=torch.uint8, device=cache.device)


def tree_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cache: PagedCache, layer: int,
                   seqs: torch.Tensor, mask: Optional[torch.Tensor] = None, nodes: Optional[torch.Tensor] = None,
                   scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of drafted tokens over the cache's context of `layer` and over each other.

    q [batch, nodes, heads_q, head_dim]; k, v [batch, nodes, heads, head_dim] of the drafted tokens, which are
    not in the cache.  seqs [batch]: the sequences' rows in the cache.  mask int64 [batch, nodes, ceil(nodes /
    64)]: bit u % 64 of word u / 64 lets a node see node u (default: node t sees u <= t, so that one node is
    ordinary decoding).  nodes int32 [batch]: how many of the nodes are real (default: all).  scale: 1 /
    sqrt(head_dim) by default.  Returns (out, lse): out as q, lse float32 [batch, nodes, heads_q], the natural
    logarithm of the sum of exponentials; a row that sees nothing is 0 and -inf.  For serving:
    there is no gradient and no forward mode, and tensors that carry either are refused."""
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
        _tb_cache.tb_tree_attention(a, cache._c, sh)
    return out, lse
