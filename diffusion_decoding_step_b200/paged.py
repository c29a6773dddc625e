"""Paged key/value cache held in torch tensors, driven through the C ABI.

PyTorch only allocates memory and provides the stream; the arithmetic runs in
libdllm.so (``dllm_paged_append``, ``dllm_paged_attn``,
``dllm_shared_prefix_attn``; include/dllm.h states what they compute).
"""
from __future__ import annotations

import ctypes as C
from typing import Optional

import torch

from . import abi

_TYPES = {torch.bfloat16: abi.DLLM_KV_BF16, torch.float16: abi.DLLM_KV_F16}

# the current stream of a device index, and the current device: the public calls
# (current_stream, current_device) take 2.2 and 0.2 us of a call's 11
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _ints(t: torch.Tensor, what: str, shape: tuple, index: int) -> int:
    """Address of a contiguous int32 tensor of the given shape on GPU `index`."""
    if t.dtype is torch.int32 and t.shape == shape and t.get_device() == index \
            and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{what}: a contiguous int32 tensor of shape {list(shape)} on cuda:{index} is "
                     f"needed, got {t.dtype} {list(t.shape)} on {t.device}")


class PagedKV:
    """Pages of keys and values, and the workspace of the attention over them.

    ``k_pages`` / ``v_pages``: bf16 or fp16 [n_pages][Hkv][page_size][D] on one GPU, with
    equal strides and contiguous D elements; other orders (slots before heads, keys and
    values of a page side by side) are views.  ``max_rows`` bounds the rows of an attention
    call, ``max_groups`` the prefix groups (0: ``shared_prefix_attn`` is not used).

    Calls run on the current stream of the pages' device and return without waiting.  The
    attention calls share one workspace: a PagedKV serves one of them at a time, and graphs or
    streams that may overlap each take a PagedKV of their own over the same pages.
    """

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, n_q_heads: int,
                 max_rows: int, max_groups: int = 0):
        if k_pages.dim() != 4 or k_pages.shape != v_pages.shape \
                or k_pages.stride() != v_pages.stride() or k_pages.dtype != v_pages.dtype \
                or k_pages.device != v_pages.device:
            raise ValueError("k_pages and v_pages: two [n_pages][Hkv][page_size][D] tensors of one "
                             "type, device and strides are needed")
        if k_pages.dtype not in _TYPES:
            raise ValueError(f"pages of {k_pages.dtype}: bfloat16 or float16 is needed")
        if not k_pages.is_cuda:
            raise ValueError("the pages have to be on a GPU")
        if k_pages.stride(3) != 1:
            raise ValueError("the D elements of a head have to be contiguous")
        self.k_pages, self.v_pages = k_pages, v_pages
        self.device, self.dtype = k_pages.device, k_pages.dtype
        self._index = k_pages.get_device()
        n_pages, self.n_kv_heads, self.page_size, self.head_dim = k_pages.shape
        self.n_q_heads, self.max_rows, self.max_groups = n_q_heads, max_rows, max_groups
        lib = abi.lib()
        self._append, self._attn = lib.dllm_paged_append, lib.dllm_paged_attn
        self._shared, self._status = lib.dllm_shared_prefix_attn, lib.dllm_device_status
        self._kv = abi.dllm_kv_pages(k_pages.data_ptr(), v_pages.data_ptr(), k_pages.stride(0),
                                     k_pages.stride(1), k_pages.stride(2), n_pages,
                                     self.page_size, self.n_kv_heads, self.head_dim,
                                     _TYPES[self.dtype])
        self._kv_p = C.byref(self._kv)
        n = C.c_size_t(0)
        abi.check(abi.dllm_paged_workspace_size(self._kv_p, n_q_heads, max_rows, C.byref(n)),
                  "paged_workspace_size")
        self.ws_bytes = int(n.value)
        with torch.cuda.device(self.device):
            self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
            self._ws_p = self.ws.data_ptr()
            abi.check(abi.dllm_paged_workspace_init(self._ws_p, self.ws_bytes,
                                                    _raw_stream(self._index)),
                      "paged_workspace_init")

    # ------------------------------------------------------------------ arguments
    def _call(self, what: str, fn, *args) -> None:
        if _current_device() == self._index:
            status = fn(*args, _raw_stream(self._index))
        else:
            with torch.cuda.device(self.device):
                status = fn(*args, _raw_stream(self._index))
        if status != abi.DLLM_OK:
            abi.check(status, what)

    def _rows(self, t: torch.Tensor, what: str, n_rows: int, heads: int):
        if t.dtype is self.dtype and t.shape == (n_rows, heads, self.head_dim) \
                and t.get_device() == self._index:
            row, head, one = t.stride()
            if one == 1:
                return C.byref(abi.dllm_rows(t.data_ptr(), row, head))
        raise ValueError(f"{what}: a {self.dtype} tensor [{n_rows}][{heads}][{self.head_dim}] on "
                         f"{self.device} with contiguous heads is needed, got {t.dtype} "
                         f"{list(t.shape)}, strides {t.stride()}, on {t.device}")

    def _batch(self, n_rows: int, row_start: torch.Tensor, page_table: torch.Tensor):
        n = row_start.numel() - 1
        width = page_table.shape[-1]
        return n, C.byref(abi.dllm_paged_batch(
            n, n_rows, width, width, _ints(row_start, "row_start", (n + 1,), self._index),
            _ints(page_table, "page_table", (n, width), self._index)))

    # ------------------------------------------------------------------ calls
    def append(self, k: torch.Tensor, v: torch.Tensor, row_start: torch.Tensor,
               page_table: torch.Tensor, pos: torch.Tensor, q: Optional[torch.Tensor] = None,
               q_out: Optional[torch.Tensor] = None, rope_theta: float = 0.0,
               rope_shift: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
        """Append rows k, v [rows][Hkv][D] to the cache, k rotated; returns q [rows][Hq][D]
        rotated (into q_out, which may be q), or None without q.

        Rows [row_start[s], row_start[s+1]) go to positions pos[s].. of sequence s, rotated by
        position + rope_shift[s]; page_table [n_seqs][pages] lists each sequence's pages."""
        rows, index = k.shape[0], self._index
        n, bt = self._batch(rows, row_start, page_table)
        heads, qp, qo = 0, None, None
        if q is not None:
            if q_out is None:
                q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
            heads = self.n_q_heads
            qp = self._rows(q, "q", rows, heads)
            qo = self._rows(q_out, "q_out", rows, heads)
        elif q_out is not None:
            raise ValueError("q_out without q")
        self._call("paged_append", self._append, self._kv_p, bt, heads, qp,
                   self._rows(k, "k", rows, self.n_kv_heads),
                   self._rows(v, "v", rows, self.n_kv_heads), qo, _ints(pos, "pos", (n,), index),
                   None if rope_shift is None else _ints(rope_shift, "rope_shift", (n,), index),
                   rope_theta, self._ws_p)
        return q_out

    def _attn_args(self, q, row_start, page_table, segs, row_limit, out, lse):
        rows = q.shape[0]
        if rows > self.max_rows:
            raise ValueError(f"{rows} rows: this PagedKV was made for {self.max_rows}")
        n, bt = self._batch(rows, row_start, page_table)
        if out is None:
            out = torch.empty(rows, self.n_q_heads, self.head_dim, dtype=self.dtype,
                              device=self.device)
        lp = None
        if lse is not None:
            if lse.dtype is not torch.float32 or lse.shape != (rows, self.n_q_heads) \
                    or lse.get_device() != self._index or not lse.is_contiguous():
                raise ValueError(f"lse: a contiguous float32 tensor [{rows}][{self.n_q_heads}] on "
                                 f"{self.device} is needed")
            lp = lse.data_ptr()
        return out, bt, (_ints(segs, "segs", (n, 2, 2), self._index),
                         None if row_limit is None
                         else _ints(row_limit, "row_limit", (rows,), self._index)), \
            (self._rows(q, "q", rows, self.n_q_heads), self._rows(out, "out", rows, self.n_q_heads),
             lp, self._ws_p, self.ws_bytes)

    def attn(self, q: torch.Tensor, row_start: torch.Tensor, page_table: torch.Tensor,
             segs: torch.Tensor, row_limit: Optional[torch.Tensor] = None, scale: float = 0.0,
             out: Optional[torch.Tensor] = None,
             lse: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Attention of rows q [rows][Hq][D] over the cache, into out (returned); lse, if given,
        receives each row's log-sum-exp.

        segs int32 [n_seqs][2][2]: (start, length) of the positions a sequence's rows see;
        row_limit int32 [rows]: a row sees only positions below it.  Rows of no sequence are
        left as they were (undefined in a fresh out)."""
        out, bt, keys, rest = self._attn_args(q, row_start, page_table, segs, row_limit, out, lse)
        self._call("paged_attn", self._attn, self._kv_p, bt, self.n_q_heads, *keys, scale, *rest)
        return out

    def shared_prefix_attn(self, q: torch.Tensor, row_start: torch.Tensor,
                           page_table: torch.Tensor, segs: torch.Tensor,
                           group_start: torch.Tensor, prefix_table: torch.Tensor,
                           prefix_len: torch.Tensor, row_limit: Optional[torch.Tensor] = None,
                           scale: float = 0.0, out: Optional[torch.Tensor] = None,
                           lse: Optional[torch.Tensor] = None) -> torch.Tensor:
        """attn() for sequences that share prefixes: sequences [group_start[g],
        group_start[g+1]) also see the prefix_len[g] positions of the pages in
        prefix_table[g]."""
        out, bt, keys, rest = self._attn_args(q, row_start, page_table, segs, row_limit, out, lse)
        n, index = group_start.numel() - 1, self._index
        if n < 1 or n > self.max_groups:
            raise ValueError(f"{n} prefix groups: this PagedKV was made for 1 to {self.max_groups}")
        width = prefix_table.shape[-1]
        g = abi.dllm_prefix_groups(n, width, width,
                                   _ints(group_start, "group_start", (n + 1,), index),
                                   _ints(prefix_table, "prefix_table", (n, width), index),
                                   _ints(prefix_len, "prefix_len", (n,), index))
        self._call("shared_prefix_attn", self._shared, self._kv_p, bt, C.byref(g), self.n_q_heads,
                   *keys, scale, *rest)
        return out

    def device_status(self) -> int:
        """The workspace's status word (waits for the current stream)."""
        code = C.c_int32(0)
        self._call("device_status", self._status, self._ws_p, C.byref(code))
        return int(code.value)
