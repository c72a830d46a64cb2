"""Tokens of a batch's logits, over qw_sample_batch.

PyTorch is used for device memory and streams only; the computation is a libqw.so kernel.
"""
from __future__ import annotations

import ctypes as C

from . import _binding as B
from .paged import _format, _i32, _raw, _torch


def sample_batch(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, out=None, probs=None):
    """One token per row of ``logits`` [n_rows, vocab] (float32 or bfloat16; rows may be strided).

    Of a row's logits, largest first (ties: lowest id), weighted exp((l - max) / temperature), are kept
    the ``top_k`` first (0: all), of these the fewest that reach ``top_p`` of their sum, and only those of
    at least ``min_p`` times the largest weight; the token is the first whose running sum exceeds ``u`` times
    the kept sum. ``u``: float32 [n_rows] in [0, 1). temperature <= 0 or top_k == 1 is greedy.
    Each setting is one number, or a tensor [n_rows] on the logits' device (float32; top_k int32), whose
    values a replayed graph reads anew. A row with a NaN, +inf, nothing above -inf or settings out of range
    gets -1.

    Returns int32 [n_rows], or ``out``. ``probs``: float32 [n_rows], gets the probability with which each
    token was drawn. Queues on the current stream.
    """
    torch = _torch()
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits: [n_rows, vocab] of adjacent elements wanted")
    n, vocab = logits.shape
    index = logits.get_device()
    fmt = _format(logits, "logits")
    p = B.qw_sample_params(struct_size=C.sizeof(B.qw_sample_params))

    def column(t, what, dtype=torch.float32):
        if t.dtype is not dtype or t.shape != (n,) or t.get_device() != index or not t.is_contiguous():
            raise ValueError(f"{what}: contiguous {dtype} [{n}] on {logits.device} wanted")
        return t.data_ptr()

    for value, name, dtype in ((temperature, "temperature", torch.float32), (top_k, "top_k", torch.int32),
                               (top_p, "top_p", torch.float32), (min_p, "min_p", torch.float32)):
        if torch.is_tensor(value):
            setattr(p, name + "s", column(value, name, dtype))
            if name == "top_p":
                p.top_p = 1.0
        else:
            setattr(p, name, _i32(value) if name == "top_k" else value)
    u_ptr = column(u, "u")
    if out is None:
        out = torch.empty(n, dtype=torch.int32, device=logits.device)
    ld = logits.stride(0) if n > 1 else vocab
    stream = _raw(index)
    rc = B.lib().qw_sample_batch(C.byref(p), logits.data_ptr(), fmt, ld, n, vocab, u_ptr,
                                 column(out, "out", torch.int32), column(probs, "probs") if probs is not None
                                 else None, stream)
    if rc:
        B.check("qw_sample_batch", rc)
    return out
