"""A paged KV cache for a batch of sequences, over qw_paged_append and qw_paged_attention.

``PagedKV`` holds one layer's pages and the batch's lengths and tables as torch CUDA tensors and
queues the two calls on torch's current stream. PyTorch is used for device memory and streams
only; every computation is a libqw.so kernel.
"""
from __future__ import annotations

import ctypes as C

from . import _binding as B

# Filled at the first use: torch's element types, and the raw handle of its current stream
# (torch.cuda.current_stream builds an object around it, which takes longer than the launch).
_FORMATS: dict = {}
_raw_stream = None


def _torch():
    global _raw_stream
    import torch
    if not _FORMATS:
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda index: torch.cuda.current_stream(index).cuda_stream)
        _FORMATS.update({torch.float32: 0, torch.bfloat16: 1})  # QW_KV_* and QW_ACT_* alike
    return torch


def _format(t, what: str) -> int:
    f = _FORMATS.get(t.dtype)
    if f is None:
        raise ValueError(f"{what}: float32 or bfloat16 wanted, got {t.dtype}")
    return f


class Workspace:
    """Scratch of PagedKV.attend, one for all caches whose calls follow one another (the layers of
    a model): pass the first cache's ``workspace`` to the others."""

    def __init__(self, device):
        self.device, self.bytes, self.ptr = device, 0, None
        self._kept = []
        self.streams = set()  # raw handles of the streams that the present buffer is known to be used on

    def use(self, raw: int) -> None:
        """The current stream (raw handle ``raw``) works on the scratch: once dropped, its memory is not
        given out again before that stream has done so."""
        self._kept[-1].record_stream(_torch().cuda.current_stream(self.device))
        self.streams.add(raw)

    def grow(self, need: int) -> None:
        torch = _torch()
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("the attention workspace is too small and cannot be made inside a graph "
                               "capture: call reserve(n_tokens, n_q_heads) before it")
        # smaller ones are kept, as a captured graph may hold their address; each is at least twice
        # the one before, so that they stay below the largest together
        size = max(need, 2 * self.bytes)
        self._kept.append(torch.zeros(size, dtype=torch.uint8, device=self.device))
        torch.cuda.current_stream(self.device).synchronize()  # zero for calls on any stream
        self.bytes, self.ptr = size, self._kept[-1].data_ptr()
        self.streams.clear()


class PagedKV:
    """One layer's pages and the batch that uses them (fields as in qw_paged_kv).

    k_pages, v_pages: [n_pages, n_kv_heads, page_size, head_dim], float32 or bfloat16;
    page_table: int32 [n_seqs, max_pages]; kv_len: int32 [n_seqs], keys of each sequence with the
    call's new tokens; q_start: int32 [n_seqs + 1], first token row of each sequence;
    prefix_pages: int32 pages of ``prefix_len`` keys that all sequences share, or None.
    workspace: another PagedKV's ``workspace``, to share its scratch.
    wait_limit_us: bound of a device-side wait of ``attend`` (0: one second).
    All are contiguous tensors on one CUDA device. They are borrowed, not copied: write new lengths
    or page ids into them between calls (or into a captured graph's inputs before a replay). Calls queue
    on the current stream; a PagedKV may be dropped while they run, but not while a captured graph that
    holds its calls may still be replayed (the graph knows its scratch by address only).
    """

    def __init__(self, k_pages, v_pages, page_table, kv_len, q_start, prefix_pages=None,
                 prefix_len: int = 0, workspace: "Workspace" = None, wait_limit_us: int = 0):
        torch = _torch()
        if not 0 <= wait_limit_us < 1 << 32:
            raise ValueError("wait_limit_us: 0 (one second) or microseconds below 2^32")
        if k_pages.dim() != 4 or k_pages.shape != v_pages.shape or k_pages.dtype != v_pages.dtype:
            raise ValueError("k_pages and v_pages: two [n_pages, n_kv_heads, page_size, head_dim] "
                             "tensors of one type")
        n_seqs = page_table.shape[0] if page_table.dim() == 2 else 0
        if n_seqs < 1 or kv_len.shape != (n_seqs,) or q_start.shape != (n_seqs + 1,):
            raise ValueError("page_table [n_seqs, max_pages], kv_len [n_seqs] and q_start [n_seqs + 1] "
                             "do not agree")
        ints = [page_table, kv_len, q_start] + ([prefix_pages] if prefix_pages is not None else [])
        if any(t.dtype != torch.int32 for t in ints):
            raise ValueError("page_table, kv_len, q_start and prefix_pages are int32")
        self.device = k_pages.device
        for t in [k_pages, v_pages] + ints:
            if not t.is_cuda or t.device != self.device or not t.is_contiguous():
                raise ValueError("every tensor of the cache is contiguous and on one CUDA device")
        page = k_pages.shape[2]
        if prefix_len < 0 or (prefix_len > 0 and (prefix_pages is None or
                                                  prefix_pages.numel() * page < prefix_len)):
            raise ValueError("prefix_pages do not hold prefix_len keys")
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        torch.cuda.current_stream(self.device).synchronize()  # zero for calls on any stream
        self._streams = set()  # those that status is known to be used on
        self._keep = (k_pages, v_pages, page_table, kv_len, q_start, prefix_pages)
        self.workspace = workspace if workspace is not None else Workspace(self.device)
        if self.workspace.device != self.device:
            raise ValueError("the workspace is on another device")
        self._lib = B.lib()
        self.head_dim = k_pages.shape[3]
        self.n_kv_heads = k_pages.shape[1]
        self.c = B.qw_paged_kv(
            struct_size=C.sizeof(B.qw_paged_kv), kv_format=_format(k_pages, "pages"),
            n_pages=k_pages.shape[0], page_size=page, n_kv_heads=k_pages.shape[1],
            head_dim=k_pages.shape[3], n_seqs=n_seqs, max_pages=page_table.shape[1],
            prefix_len=prefix_len, wait_limit_us=wait_limit_us, k_pages=k_pages.data_ptr(), v_pages=v_pages.data_ptr(),
            page_table=page_table.data_ptr(), kv_len=kv_len.data_ptr(),
            q_start=q_start.data_ptr(), status=self.status.data_ptr(),
            prefix_pages=prefix_pages.data_ptr() if prefix_len > 0 else None)
        self._cref = C.byref(self.c)
        self._index = self.device.index
        self._current = torch.cuda.current_device
        self._int32, self._gains = torch.int32, (torch.bfloat16, torch.int16)

    def _rows(self, t, what: str, width: int, rows: int) -> int:
        """Row stride of an activation matrix [rows, width] or [rows, heads, head_dim] whose rows
        are adjacent elements."""
        shape, inner = t.shape, t.stride()
        if len(shape) == 3:  # heads back to back
            ok = inner[2] == 1 and shape[1] * shape[2] == width and (inner[1] == shape[2] or shape[1] == 1)
        else:
            ok = len(shape) == 2 and inner[1] == 1 and shape[1] == width
        if not ok or shape[0] != rows or t.get_device() != self._index:
            raise ValueError(f"{what}: {rows} rows of {width} adjacent elements on {self.device} wanted, got "
                             f"{tuple(shape)} with strides {inner} on {t.device}")
        return inner[0] if rows > 1 else width

    def _out(self, out, like, n_q_heads: int, rows: int):
        if out is None:
            return _torch().zeros(rows, n_q_heads, self.head_dim, dtype=like.dtype, device=self.device)
        width = n_q_heads * self.head_dim
        if out.dtype is not like.dtype or self._rows(out, "out", width, rows) != width:
            raise ValueError("out: contiguous rows of the input's type wanted")
        return out

    def _stream(self):
        if self._current() != self._index:
            raise ValueError("the cache's device is not the current one")
        raw = _raw_stream(self._index)
        if raw not in self._streams:
            self.status.record_stream(_torch().cuda.current_stream(self.device))
            self._streams.add(raw)
        return raw

    def append(self, qkv, n_q_heads: int, q_norm=None, k_norm=None, eps: float = 1e-6,
               rope_theta: float = 1e6, positions=None, sections=None, out=None):
        """Norm, rotate and append the tokens' raw projections; returns the rotated queries.

        qkv: [n_tokens, (n_q_heads + 2 n_kv_heads) * head_dim] (rows may be strided); q_norm, k_norm:
        bfloat16 (or int16 bits) [head_dim]; positions: int32 [n_tokens], or [n_tokens, 3] with
        sections = (pairs of axis 0, 1, 2), or None for each token's place in the cache; rope_theta >= 1.
        ``out`` must not overlap qkv.
        """
        n = qkv.shape[0]
        fmt = _format(qkv, "qkv")
        ld = self._rows(qkv, "qkv", (n_q_heads + 2 * self.n_kv_heads) * self.head_dim, n)
        out = self._out(out, qkv, n_q_heads, n)
        for t in (q_norm, k_norm):
            if t is not None and (t.dtype not in self._gains or t.dim() != 1 or t.numel() != self.head_dim or
                                  t.stride(0) != 1 or t.get_device() != self._index):
                raise ValueError("q_norm and k_norm: bfloat16 (or its int16 bits) [head_dim] on the cache's "
                                 "device")
        if positions is not None:
            want = (n, 3) if sections is not None else (n,)
            if positions.dtype is not self._int32 or positions.shape != want or \
                    not positions.is_contiguous() or positions.get_device() != self._index:
                raise ValueError(f"positions: contiguous int32 {want} wanted")
        sec = (C.c_int32 * 3)(*sections) if sections is not None else None
        rc = self._lib.qw_paged_append(
            self._cref, qkv.data_ptr(), fmt, ld, n, n_q_heads,
            q_norm.data_ptr() if q_norm is not None else None,
            k_norm.data_ptr() if k_norm is not None else None, eps, rope_theta,
            positions.data_ptr() if positions is not None else None, sec, out.data_ptr(),
            self._stream())
        if rc:
            B.check("qw_paged_append", rc)
        return out

    def attend(self, q, max_new: int = 1, out=None):
        """Attention of the tokens' rotated queries [n_tokens, n_q_heads, head_dim] over their
        sequences' keys (and the shared prefix). max_new: the most new tokens of one sequence, a hint that
        chooses the kernels. ``out`` must not overlap q.
        Calls that share a workspace (those of one PagedKV, captured ones too) must not overlap on the
        GPU, and it has to exist before a capture: call once before, or ``reserve``."""
        shape, hd = q.shape, self.head_dim
        # (a head's size is not taken from the product: 8 heads of 64 are not 4 of 128)
        if not (len(shape) == 3 and shape[2] == hd or len(shape) == 2 and shape[1] % hd == 0):
            raise ValueError(f"q: [n_tokens, n_q_heads, {hd}] (or [n_tokens, n_q_heads * {hd}]) wanted, got "
                             f"{tuple(shape)}")
        n = shape[0]
        heads = shape[1] if len(shape) == 3 else shape[1] // hd
        fmt = _format(q, "q")
        ld = self._rows(q, "q", heads * self.head_dim, n)
        out = self._out(out, q, heads, n)
        need = self._lib.qw_paged_attention_workspace_bytes(n, heads, self.head_dim,
                                                            self.c.prefix_len)
        ws = self.workspace
        if ws.bytes < need:
            ws.grow(need)
        raw = self._stream()
        if raw not in ws.streams:
            ws.use(raw)
        rc = self._lib.qw_paged_attention(self._cref, q.data_ptr(), fmt, ld, n, heads, max_new,
                                          out.data_ptr(), ws.ptr, ws.bytes, raw)
        if rc:
            B.check("qw_paged_attention", rc)
        return out

    def reserve(self, n_tokens: int, n_q_heads: int) -> None:
        """Workspace for attention calls of up to n_tokens rows (as the first such call would)."""
        need = self._lib.qw_paged_attention_workspace_bytes(n_tokens, n_q_heads, self.head_dim,
                                                            self.c.prefix_len)
        if self.workspace.bytes < need:
            self.workspace.grow(need)

    def check(self) -> None:
        """Raises if a call so far met a bad page id or length or gave up a wait (synchronises)."""
        bits = int(self.status.item())
        if bits:
            names = [n for n in ("TIMEOUT", "BAD_PAGE", "BAD_LENGTH")
                     if bits & getattr(B, "QW_PAGED_" + n)]
            raise RuntimeError("paged cache: " + ", ".join(names))
