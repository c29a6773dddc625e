"""Paged key/value cache held in torch tensors, driven through the C ABI.

PyTorch only allocates memory and provides the stream; the arithmetic runs in
libdllm.so (``dllm_paged_append``, ``dllm_paged_attn``,
``dllm_shared_prefix_attn``; include/dllm.h states what they compute).  The
tensors are checked and passed on by the compiled module ``_paged_torch``.
"""
from __future__ import annotations

import ctypes as C
from typing import Optional

import torch

from . import abi

_TYPES = {torch.bfloat16: abi.DLLM_KV_BF16, torch.float16: abi.DLLM_KV_F16}


def _binding():
    """The compiled binding; fails loudly if it has not been built."""
    try:
        from . import _paged_torch
    except ImportError as e:
        raise abi.DllmError(f"torch binding not built or not loadable ({e}); run "
                            "diffusion_decoding_step_b200/build.py") from e
    return _paged_torch


class PagedKV:
    """Pages of keys and values, and the workspace of the attention over them.

    ``k_pages`` / ``v_pages``: bf16 or fp16 [n_pages][Hkv][page_size][D] on one GPU, with
    equal strides and contiguous D elements; other orders (slots before heads, keys and
    values of a page side by side) are views.  ``max_rows`` bounds the rows of an attention
    call and sizes the workspace; ``max_groups`` bounds the prefix groups (0: no
    ``shared_prefix_attn``; the default is the most that a call takes).

    The cache only serves, there is no backward: tensors that require a gradient are refused
    while gradients are recorded (``torch.no_grad()``).

    Calls run on the current stream of the pages' device and return without waiting; a call
    without rows checks its arguments and does nothing.  The
    attention calls share one workspace: a PagedKV serves one of them at a time, and graphs or
    streams that may overlap each take a PagedKV of their own over the same pages.  Keep the
    object until its calls have run: the workspace's memory goes with it.
    """

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, n_q_heads: int,
                 max_rows: int, max_groups: int = 1024):
        if k_pages.dim() != 4 or k_pages.shape != v_pages.shape \
                or k_pages.stride() != v_pages.stride() or k_pages.dtype != v_pages.dtype \
                or k_pages.device != v_pages.device:
            raise ValueError("k_pages and v_pages: two [n_pages][Hkv][page_size][D] tensors of one "
                             "type, device and strides are needed")
        if k_pages.dtype not in _TYPES:
            raise ValueError(f"pages of {k_pages.dtype}: bfloat16 or float16 is needed")
        if not k_pages.is_cuda:
            raise ValueError("the pages have to be on a GPU")
        if k_pages.requires_grad or v_pages.requires_grad:
            raise ValueError("the pages are written in place: they cannot require a gradient")
        if k_pages.stride(3) != 1:
            raise ValueError("the D elements of a head have to be contiguous")
        for name, x in (("n_q_heads", n_q_heads), ("max_rows", max_rows), ("max_groups", max_groups)):
            if not 0 <= x < 2 ** 31:
                raise ValueError(f"{name}: {x} does not fit")
        self.k_pages, self.v_pages = k_pages, v_pages
        self.device, self.dtype = k_pages.device, k_pages.dtype
        n_pages, self.n_kv_heads, self.page_size, self.head_dim = k_pages.shape
        self.n_q_heads, self.max_rows, self.max_groups = n_q_heads, max_rows, max_groups
        binding, lib = _binding(), abi.lib()
        kv = abi.dllm_kv_pages(k_pages.data_ptr(), v_pages.data_ptr(), k_pages.stride(0),
                               k_pages.stride(1), k_pages.stride(2), n_pages, self.page_size,
                               self.n_kv_heads, self.head_dim, _TYPES[self.dtype])
        n = C.c_size_t(0)
        abi.check(abi.dllm_paged_workspace_size(C.byref(kv), n_q_heads, max_rows, C.byref(n)),
                  "paged_workspace_size")
        with torch.cuda.device(self.device):
            self.ws = torch.empty(int(n.value), dtype=torch.uint8, device=self.device)
            stream = torch.cuda.current_stream(self.device).cuda_stream
            abi.check(abi.dllm_paged_workspace_init(self.ws.data_ptr(), n.value, stream),
                      "paged_workspace_init")
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()  # calls may come on any stream
        fns = (C.cast(f, C.c_void_p).value for f in (lib.dllm_paged_append, lib.dllm_paged_attn,
                                                     lib.dllm_shared_prefix_attn))
        self._append, self._attn = binding.append, binding.attn
        self._h = binding.create(C.addressof(kv), n_q_heads, max_rows, max_groups,
                                 self.device.index, int(self.dtype is torch.float16),
                                 self.ws.data_ptr(), n.value, *fns, k_pages, v_pages)

    # ------------------------------------------------------------------ calls
    def append(self, k: torch.Tensor, v: torch.Tensor, row_start: torch.Tensor,
               page_table: torch.Tensor, pos: torch.Tensor, q: Optional[torch.Tensor] = None,
               q_out: Optional[torch.Tensor] = None, rope_theta: float = 0.0,
               rope_shift: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
        """Append rows k, v [rows][Hkv][D] to the cache, k rotated; returns q [rows][Hq][D]
        rotated (into q_out, which may be q), or None without q.

        Rows [row_start[s], row_start[s+1]) go to positions pos[s].. of sequence s, rotated by
        position + rope_shift[s]; page_table [n_seqs][pages] lists each sequence's pages.
        rope_theta (0: no rotation) is taken in fp32, as the model configuration holds it."""
        if q is not None:
            if q_out is None:
                q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        elif q_out is not None:
            raise ValueError("q_out without q")
        status = self._append(self._h, k, v, row_start, page_table, pos, q, q_out, rope_theta,
                              rope_shift)
        if status:
            abi.check(status, "paged_append")
        return q_out

    def _out(self, q):
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q: a tensor [rows][Hq][D] is needed")
        return torch.empty(q.shape[0], self.n_q_heads, self.head_dim, dtype=self.dtype,
                           device=self.device)

    def attn(self, q: torch.Tensor, row_start: torch.Tensor, page_table: torch.Tensor,
             segs: torch.Tensor, row_limit: Optional[torch.Tensor] = None, scale: float = 0.0,
             out: Optional[torch.Tensor] = None,
             lse: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Attention of rows q [rows][Hq][D] over the cache, into out (returned); lse, if given,
        receives each row's log-sum-exp.

        segs int32 [n_seqs][2][2]: (start, length) of the positions a sequence's rows see;
        row_limit int32 [rows]: a row sees only positions below it.  scale 0: 1 / sqrt(D).  Rows
        of no sequence are left as they were (undefined in a fresh out)."""
        if out is None:
            out = self._out(q)
        status = self._attn(self._h, q, row_start, page_table, segs, row_limit, scale, out, lse,
                            None, None, None)
        if status:
            abi.check(status, "paged_attn")
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
        if group_start is None:
            raise ValueError("group_start: a tensor is needed (attn() takes no groups)")
        if out is None:
            out = self._out(q)
        status = self._attn(self._h, q, row_start, page_table, segs, row_limit, scale, out, lse,
                            group_start, prefix_table, prefix_len)
        if status:
            abi.check(status, "shared_prefix_attn")
        return out

    def device_status(self) -> int:
        """The workspace's status word (waits for the current stream): 0, or the DLLM_DEVICE_*
        bits of all calls so far.  No call reads it: after DLLM_DEVICE_TIMEOUT outputs are
        undefined, after DLLM_DEVICE_INDEX bad pages and positions were left out."""
        code = C.c_int32(0)
        with torch.cuda.device(self.device):
            stream = torch.cuda.current_stream(self.device).cuda_stream
            abi.check(abi.dllm_device_status(self.ws.data_ptr(), C.byref(code), stream),
                      "device_status")
        return int(code.value)
