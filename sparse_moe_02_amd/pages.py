"""The paged cache's bookkeeping on device tensors (argument marshalling for ``include/pages.h``;
every step runs in the HIP kernels).

Calls are enqueued on torch's current stream of the pool's device and never wait for it, except
``PagePool.check``.
"""

from __future__ import annotations

import torch

from . import binding as B
from ._device import N, on, stream


class PagePool:
    """Which pages of a cache each sequence holds: ``table`` int32 [max_seqs][max_pages] and
    ``lens`` int32 [max_seqs], as ``rope_append`` and ``paged_attn`` take them, and ``refs`` int32
    [n_pages].  A new pool is empty.

    The calls change the pool in place, or leave it as it is and write the result to ``out``, a
    pool made by ``like()``.  Errors that only the device can see leave the pool unchanged and are
    found by ``check`` on the pool that took the result.  One pool's calls share its workspace:
    they belong on one stream at a time."""

    def __init__(self, n_pages: int, page_size: int, max_seqs: int, max_pages: int, device="cuda:0"):
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError("a pool lives on a GPU")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.n_pages, self.page_size, self.max_seqs, self.max_pages = n_pages, page_size, max_seqs, max_pages
        size = B.moe_pages_workspace(B.moe_pages(None, None, None, max_seqs, max_pages, n_pages, page_size), max_seqs)

        def zeros(*shape):
            return torch.zeros(shape, dtype=torch.int32, device=self.device)

        self.table, self.lens, self.refs = zeros(max_seqs, max_pages), zeros(max_seqs), zeros(n_pages)
        self.error = zeros(1)
        self.ws = torch.empty(size, dtype=torch.uint8, device=self.device)
        # the arrays are the pool's for its life: fill them, do not replace them
        self._index, self._error = self.device.index, self.error.data_ptr()
        self._ws, self._ws_bytes = self.ws.data_ptr(), size
        self._c = B.moe_pages(self.table.data_ptr(), self.lens.data_ptr(), self.refs.data_ptr(), max_seqs, max_pages,
                              n_pages, page_size)

    def like(self) -> "PagePool":
        """An empty pool of the same sizes, to take a call's result."""
        return PagePool(self.n_pages, self.page_size, self.max_seqs, self.max_pages, self.device)

    def _out(self, out):
        if out is None:
            return self
        if not isinstance(out, PagePool) or out.device != self.device:
            raise ValueError("out: a PagePool on the same device required")
        return out

    def _tail(self, out):
        return out._error, self._ws, self._ws_bytes, stream(self._index)

    def grow(self, seqs: torch.Tensor, tokens: torch.Tensor, out: "PagePool | None" = None) -> "PagePool":
        """Sequences seqs (int32, distinct) grow by tokens (int32) each."""
        out, n = self._out(out), seqs.shape[0]
        s = N.address("seqs", seqs, N.INT32, self._index, n)
        t = N.address("tokens", tokens, N.INT32, self._index, n)
        with on(self._index):
            B.moe_pages_grow(self._c, out._c, n, s, t, *self._tail(out))
        return out

    def fork(self, src: torch.Tensor, dst: torch.Tensor, cache: torch.Tensor,
             out: "PagePool | None" = None) -> "PagePool":
        """Empty sequences dst (int32, distinct) become copies of src (int32): full pages are
        shared, a last page that is not full is copied.  cache: [n_planes][n_pages][...]."""
        out, n = self._out(out), src.shape[0]
        s = N.address("src", src, N.INT32, self._index, n)
        d = N.address("dst", dst, N.INT32, self._index, n)
        m = N.memory(cache, self.n_pages, self._index)
        with on(self._index):
            B.moe_pages_fork(self._c, out._c, m, n, s, d, *self._tail(out))
        return out

    def free(self, seqs: torch.Tensor, out: "PagePool | None" = None) -> "PagePool":
        """Sequences seqs (int32, distinct) end."""
        out, n = self._out(out), seqs.shape[0]
        s = N.address("seqs", seqs, N.INT32, self._index, n)
        with on(self._index):
            B.moe_pages_free(self._c, out._c, n, s, *self._tail(out))
        return out

    def compact(self, cache: torch.Tensor, out: "PagePool | None" = None) -> "PagePool":
        """The pages in use move to the lowest numbers.  cache: [n_planes][n_pages][...]."""
        out = self._out(out)
        m = N.memory(cache, self.n_pages, self._index)
        with on(self._index):
            B.moe_pages_compact(self._c, out._c, m, *self._tail(out))
        return out

    def check(self) -> int:
        """moe_pages_check: 0 (MOE_OK), or the first error of the calls whose result this pool took
        (MOE_ERR_SHAPE, MOE_ERR_ALLOC) since ``clear_error``; waits for the stream."""
        with on(self._index):
            return B.moe_pages_check(self._error, stream(self._index))

    def clear_error(self) -> None:
        self.error.zero_()


def copy_pages(cache: torch.Tensor, src: torch.Tensor, dst: torch.Tensor) -> None:
    """Page src[i] is copied to page dst[i] in every plane of cache [n_planes][n_pages][...] (see
    ``moe_pages_copy``)."""
    index, n = cache.get_device(), src.shape[0]
    if index < 0:
        raise ValueError("cache: a GPU tensor required")
    s, d = N.address("src", src, N.INT32, index, n), N.address("dst", dst, N.INT32, index, n)
    m = N.memory(cache, cache.shape[1], index)
    with on(index):
        B.moe_pages_copy(m, cache.shape[1], n, s, d, stream(index))
