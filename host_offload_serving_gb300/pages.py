"""Pages of the resident tier: who holds which, handed out and taken back on the device.

``PagePool`` keeps the block table that ``HiSparse.resolve_resident`` reads
(``tables`` int32 [R][max_blocks], -1 = not resident), the count of entries that
name each page, and the pages' bytes in every layer, through ``hisparse_pages_*``.
Calls launch on the current stream (or ``stream``) and return at once.
"""
import torch

from . import hisparse as H
from .cache8 import _i32, _need, _reach
from .runtime import _stream


class PagePool:
    """``store`` uint8 [layers][pages][page_tokens * row_bytes] (any page and
    layer strides that are multiples of 16 bytes).  ``tables`` and ``refs``
    (int32 [pages]) are given by the caller or made here: an empty pool over ``requests``
    requests of ``max_blocks`` blocks."""

    def __init__(self, store, tables=None, refs=None, *, block_tokens, requests=0, max_blocks=0,
                 status=None):
        _need(store.dtype is torch.uint8 and store.dim() == 3 and store.stride(2) == 1
              and store.shape[2] % block_tokens == 0,
              "PagePool: store is uint8 [layers][pages][block_tokens * row_bytes]")
        _need(store.is_cuda, "PagePool: store is on a CUDA device")
        pages = store.shape[1]
        if tables is None:
            tables = torch.full((requests, max_blocks), -1, dtype=torch.int32, device=store.device)
        if refs is None:
            refs = torch.zeros(pages, dtype=torch.int32, device=store.device)
        _need(tables.dim() == 2, "PagePool: tables is [R][max_blocks]")
        self.store, self.tables, self.refs, self.block_tokens = store, tables, refs, block_tokens
        words = H.hisparse_pages_work_ints(pages, tables.shape[0])
        _need(words > 0, "PagePool: at least one page and one request, at most 8192 requests")
        self.work = torch.empty(words, dtype=torch.int32, device=store.device)
        self.status = status
        self.c = H.PagePool(pages, tables.shape[0], tables.shape[1], block_tokens, store.shape[0],
                            store.shape[2] // block_tokens, store.data_ptr(), store.stride(0),
                            store.stride(1), _i32(tables, "PagePool: tables"),
                            _i32(refs, "PagePool: refs", pages), self.work.data_ptr(),
                            _i32(status, "PagePool: status"))

    def grow(self, reqs, blocks, stream=None):
        """Pages for blocks 0 .. blocks[i]-1 of request reqs[i] (int32, device)."""
        n = reqs.numel()
        d_reqs, d_blocks = _i32(reqs, "grow: reqs"), _i32(blocks, "grow: blocks", n)
        _reach("grow", self.store, self.tables, self.refs, self.status, reqs, blocks)
        H.check(H.hisparse_pages_grow(self.c, d_reqs, d_blocks, n, _stream(stream)), "hisparse_pages_grow")

    def fork(self, src, dst, tokens, stream=None):
        """Request dst[i] becomes a copy of the first tokens[i] positions of src[i]."""
        n = src.numel()
        lists = _i32(src, "fork: src"), _i32(dst, "fork: dst", n), _i32(tokens, "fork: tokens", n)
        _reach("fork", self.store, self.tables, self.refs, self.status, src, dst, tokens)
        H.check(H.hisparse_pages_fork(self.c, *lists, n, _stream(stream)), "hisparse_pages_fork")

    def free(self, reqs, stream=None):
        """Release every page of the listed requests."""
        d_reqs = _i32(reqs, "free: reqs")
        _reach("free", self.store, self.tables, self.refs, self.status, reqs)
        H.check(H.hisparse_pages_free(self.c, d_reqs, reqs.numel(), _stream(stream)), "hisparse_pages_free")

    def compact(self, stream=None):
        """Move the pages in use to the front of the store."""
        _reach("compact", self.store, self.tables, self.refs, self.status)
        H.check(H.hisparse_pages_compact(self.c, _stream(stream)), "hisparse_pages_compact")
