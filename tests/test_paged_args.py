"""Refusals of the paged-cache calls: all of them return from the host checks, before any launch."""
import ctypes as C
import os
from types import SimpleNamespace

import pytest

from sequence_decode_step_gb300 import _binding as B


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        from sequence_decode_step_gb300 import build_lib
        build_lib.build()
    return B.lib()


def cache(**kw):
    f = dict(struct_size=C.sizeof(B.qw_paged_kv), kv_format=B.QW_KV_BF16, n_pages=4, page_size=16,
             n_kv_heads=2, head_dim=64, n_seqs=2, max_pages=2, prefix_len=0, k_pages=16, v_pages=16,
             page_table=16, kv_len=16, q_start=16, prefix_pages=None, status=None)
    f.update(kw)
    return B.qw_paged_kv(**f)


def append(L, c, qkv=16, act=0, ld=8 * 64, n=2, nq=4, qn=None, kn=None, eps=1e-6, theta=1e6, pos=None,
           sec=None, out=16):
    sec = (C.c_int32 * 3)(*sec) if sec else None
    return L.qw_paged_append(C.byref(c) if c else None, qkv, act, ld, n, nq, qn, kn, eps, theta, pos,
                             sec, out, None)


def attend(L, c, q=16, act=0, ldq=4 * 64, n=2, nq=4, max_new=1, out=16, ws=16, nbytes=1 << 40):
    return L.qw_paged_attention(C.byref(c) if c else None, q, act, ldq, n, nq, max_new, out, ws, nbytes,
                                None)


def test_layout(L):
    assert L.qw_sizeof_paged_kv() == C.sizeof(B.qw_paged_kv) == 96
    assert B.qw_paged_kv.k_pages.offset == 40 and B.qw_paged_kv.status.offset == 88


BAD_CACHE = [dict(kv_format=2), dict(head_dim=96), dict(n_kv_heads=0), dict(n_pages=0), dict(n_seqs=0),
             dict(max_pages=0), dict(page_size=8), dict(page_size=48), dict(page_size=512),
             dict(n_pages=1 << 26), dict(prefix_len=-1), dict(prefix_len=5), dict(k_pages=None),
             dict(page_table=None), dict(kv_len=None), dict(q_start=None), dict(v_pages=24)]


@pytest.mark.parametrize("bad", BAD_CACHE)
def test_bad_caches(L, bad):
    assert append(L, cache(**bad)) == B.QW_ERR_ARG
    assert B.last_error()
    assert attend(L, cache(**bad)) == B.QW_ERR_ARG
    assert B.last_error()


@pytest.mark.parametrize("bad", [dict(max_pages=1 << 27), dict(max_pages=(1 << 27) - 31),
                                 dict(max_pages=1 << 26, prefix_len=(1 << 30) - 511, prefix_pages=16)])
def test_places_beyond_32_bits(L, bad):
    assert append(L, cache(**bad)) == B.QW_ERR_ARG and "2^31" in B.last_error()
    assert attend(L, cache(**bad)) == B.QW_ERR_ARG and "2^31" in B.last_error()


def test_short_struct(L):
    c = cache(struct_size=C.sizeof(B.qw_paged_kv) - 8)
    assert append(L, c) == B.QW_ERR_ABI and attend(L, c) == B.QW_ERR_ABI
    assert "struct_size" in B.last_error()
    assert append(L, None) == B.QW_ERR_ARG and attend(L, None) == B.QW_ERR_ARG


@pytest.mark.parametrize("bad", [dict(act=2), dict(n=-1), dict(nq=0), dict(qkv=None), dict(out=None),
                                 dict(qn=16), dict(kn=16), dict(qn=16, kn=18), dict(ld=8 * 64 - 1), dict(ld=8 * 64 + 1),
                                 dict(qkv=24), dict(out=8), dict(theta=0.0), dict(theta=float("inf")),
                                 dict(theta=float("nan")), dict(eps=-1.0), dict(sec=(8, 8, 16)),
                                 dict(sec=(8, 8, 8), pos=16), dict(sec=(-8, 20, 20), pos=16)])
def test_bad_append(L, bad):
    assert append(L, cache(), **bad) == B.QW_ERR_ARG
    assert "qw_paged_append" in B.last_error()


@pytest.mark.parametrize("bad", [dict(act=2), dict(n=-1), dict(nq=0), dict(nq=3), dict(nq=18),
                                 dict(max_new=0), dict(q=None), dict(out=None), dict(ws=None),
                                 dict(ldq=4 * 64 - 4), dict(ldq=4 * 64 + 2), dict(q=8), dict(ws=8),
                                 dict(nbytes=1000)])
def test_bad_attention(L, bad):
    assert attend(L, cache(), **bad) == B.QW_ERR_ARG
    assert "qw_paged_attention" in B.last_error()


def test_an_empty_call_does_nothing(L):
    assert append(L, cache(), n=0, qkv=None, out=None) == B.QW_OK
    assert attend(L, cache(), n=0, q=None, out=None, ws=None, nbytes=0) == B.QW_OK


def test_workspace_sizes(L):
    f = L.qw_paged_attention_workspace_bytes
    assert f(-1, 4, 64, 0) == f(4, 0, 64, 0) == f(4, 4, 96, 0) == f(4, 4, 64, -1) == 0
    assert 0 < f(0, 4, 64, 0) <= f(64, 16, 128, 0)
    # a prefix adds a record of hd + 2 floats per token and query head
    assert f(64, 16, 128, 1) >= f(64, 16, 128, 0) + 64 * 16 * 130 * 4


def test_launches_of_a_call_share_no_scratch(L):
    # the launch over a prefix and the one over own keys may overlap: each has slots and records of its
    # own, and only the words per CTA at the front (below 64 KB) are laid out once
    f = L.qw_paged_attention_workspace_bytes
    for n in (1, 2, 3, 14, 64):
        assert f(n, 16, 128, 1) >= 2 * f(n, 16, 128, 0) - (64 << 10)


def test_wait_limit_takes_the_reserved_word(L):
    assert B.qw_paged_kv.wait_limit_us.offset == 36 and C.sizeof(B.qw_paged_kv) == 96
    from sequence_decode_step_gb300 import PagedKV
    for bad in (-1, 1 << 32):         # (the word would take -1 for no wait at all)
        with pytest.raises(ValueError, match="wait_limit_us"):
            PagedKV(None, None, None, None, None, wait_limit_us=bad)
    c = cache(wait_limit_us=B.QW_PAGED_WAIT_NONE)
    assert attend(L, c, n=0, q=None, out=None, ws=None, nbytes=0) == B.QW_OK


def test_scratch_is_recorded_on_every_stream_that_uses_it(monkeypatch):
    from sequence_decode_step_gb300 import paged
    recorded = []

    class Buffer:
        def __init__(self, size):
            self.size = size

        def data_ptr(self):
            return 16 * self.size

        def record_stream(self, stream):
            recorded.append((self.size, stream.name))

    stream = SimpleNamespace(name="a", synchronize=lambda: None)
    torch = SimpleNamespace(uint8=None, zeros=lambda size, dtype, device: Buffer(size), cuda=SimpleNamespace(
        is_current_stream_capturing=lambda: False, current_stream=lambda device: stream))
    monkeypatch.setattr(paged, "_torch", lambda: torch)
    w = paged.Workspace("cuda:0")
    w.grow(100)
    w.use(7)
    stream.name = "b"
    assert 7 in w.streams and 9 not in w.streams
    w.use(9)
    assert recorded == [(100, "a"), (100, "b")]
    w.grow(300)                     # a new buffer: no stream is known to use it
    assert not w.streams and w.bytes == 300
    w.use(9)
    assert recorded[2:] == [(300, "b")]


@pytest.mark.parametrize("theta", [0.999, 0.01, 1e-12, 1e-38])
def test_frequencies_that_grow_along_the_head_are_refused(L, theta):
    assert append(L, cache(), theta=theta) == B.QW_ERR_ARG and "rope_theta" in B.last_error()
