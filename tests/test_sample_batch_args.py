"""Refusals of qw_sample_batch, all from its host checks, and the reference of its tests on hand cases."""
import ctypes as C
import os

import numpy as np
import pytest

from sample_ref import pick
from sequence_decode_step_gb300 import _binding as B


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        from sequence_decode_step_gb300 import build_lib
        build_lib.build()
    return B.lib()


def params(**kw):
    f = dict(struct_size=C.sizeof(B.qw_sample_params), temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    f.update(kw)
    return B.qw_sample_params(**f)


def call(L, p, logits=16, act=0, ld=100, n=2, vocab=100, u=16, tokens=16, probs=None):
    return L.qw_sample_batch(C.byref(p) if p else None, logits, act, ld, n, vocab, u, tokens, probs, None)


def test_layout(L):
    assert L.qw_sizeof_sample_params() == C.sizeof(B.qw_sample_params) == 56
    assert B.qw_sample_params.temperatures.offset == 24


@pytest.mark.parametrize("bad", [dict(act=2), dict(n=-1), dict(vocab=0), dict(vocab=(1 << 20) + 1, ld=1 << 21),
                                 dict(ld=99), dict(logits=None), dict(u=None), dict(tokens=None), dict(logits=18),
                                 dict(logits=17, act=1), dict(n=1 << 30)])
def test_bad_arguments(L, bad):
    assert call(L, params(), **bad) == B.QW_ERR_ARG and B.last_error()


@pytest.mark.parametrize("bad", [dict(temperature=float("nan")), dict(temperature=float("inf")), dict(top_p=0.0),
                                 dict(top_p=float("nan")), dict(min_p=-0.1), dict(min_p=1.1),
                                 dict(min_p=float("nan"))])
def test_bad_settings(L, bad):
    assert call(L, params(**bad)) == B.QW_ERR_ARG and B.last_error()


@pytest.mark.parametrize("bad", [dict(top_p=0.0), dict(min_p=1.1), dict(min_p=float("nan"))])
@pytest.mark.parametrize("greedy", [dict(temperature=0.0), dict(top_k=1)])
def test_bad_settings_of_a_greedy_call(L, bad, greedy):
    assert call(L, params(**bad, **greedy)) == B.QW_ERR_ARG and B.last_error()


def test_struct_size_and_no_rows(L):
    assert call(L, params(struct_size=52)) == B.QW_ERR_ABI
    assert call(L, None) == B.QW_ERR_ARG
    assert call(L, params(), n=0, logits=None, u=None, tokens=None) == B.QW_OK


def test_reference_by_hand():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.3], np.float32))     # order 1, 3, 2, 0
    assert [pick(x, u=u)[0] for u in (0.0, 0.39, 0.41, 0.69, 0.71, 0.89, 0.91)] == [1, 1, 3, 3, 2, 2, 0]
    assert pick(x, top_k=2, u=0.6)[0] == 3 and abs(pick(x, top_k=2, u=0.6)[1] - 3 / 7) < 1e-6
    assert pick(x, top_p=0.65, u=0.99)[0] == 3                  # 0.4 + 0.3 reach it
    assert pick(x, top_k=2, top_p=0.5, u=0.99)[0] == 1          # 4/7 of the two
    assert pick(x, min_p=0.6, u=0.99)[0] == 3 and pick(x, min_p=0.6, top_k=1, u=0.99)[0] == 1
    assert pick(x, temperature=0.0, u=0.9)[0] == 1
    assert pick(np.zeros(4, np.float32), u=0.5)[0] == 2         # a running sum has to exceed u's
    assert pick(np.array([0.0, np.nan], np.float32))[0] == -1
    assert pick(np.array([-np.inf, -np.inf], np.float32))[0] == -1
