"""Sampling without a GPU: the plain form's own properties, and what the call refuses."""
import ctypes as C

import numpy as np
import pytest
import torch

import rag_non_prefix_gb300 as cb
from rag_non_prefix_gb300 import build as cbbuild
from tests import sample_ref as ref


@pytest.fixture(scope="module")
def lib():
    cbbuild.build()
    return cb.load_library()


def test_the_plain_form_draws_by_probability():
    x = np.log(np.array([1.0, 4.0, 2.0, 3.0]))
    got = [ref.token(x, (i + 0.5) / 1000) for i in range(1000)]
    assert [got.count(i) for i in range(4)] == [100, 400, 200, 300]
    assert got == sorted(got, key=[1, 3, 2, 0].index)  # along falling logits
    assert {ref.token(x, u / 100, k=2) for u in range(100)} == {1, 3}
    assert {ref.token(x, u / 100, p=0.41) for u in range(100)} == {1, 3}
    assert {ref.token(x, u / 100, p=0.39) for u in range(100)} == {1}
    assert {ref.token(x, u / 100, m=0.4) for u in range(100)} == {1, 3, 2}
    assert ref.token(x, 0.99, t=0) == 1 and ref.token(x, 0.99, p=0) == 1 and ref.token(x, 0.99, m=7) == 1
    assert ref.token(np.full(3, -np.inf), 0.5) == -1 and ref.token(np.array([np.nan, -5.0]), 0.5) == 1


def test_bad_arguments_are_refused(lib):
    call = lambda logits=256, ld=100, dt=0, rows=2, vocab=100, params=None, u=256, out=256: lib.cb_sample(logits, ld, dt, rows, vocab, params, u, out, None)  # noqa: E731
    assert [call(logits=None), call(u=None), call(out=None)] == [1] * 3
    assert [call(logits=258), call(u=257), call(out=258), call(logits=257, dt=1)] == [1] * 4
    assert [call(rows=-1), call(vocab=0), call(vocab=(1 << 18) + 1, ld=1 << 20), call(ld=99), call(rows=(1 << 24) + 1)] == [2] * 5
    assert call(dt=3) == 3 and call(rows=0, logits=None, u=None, out=None) == 0
    for field in range(4):
        p = [None] * 4
        p[field] = 258
        assert call(params=C.byref(cb.Sampling(*p))) == 1
    assert lib.cb_decode_step_sample(None, None, 1, None, None, 256, None, None) == 1
    assert [call(u=256, out=257), call(u=None, params=C.byref(cb.Sampling(256, 256, 256, 256)))] == [1, 1]


def test_the_binding_refuses_before_the_library(lib):
    x = torch.zeros(2, 5)
    for bad, name in ((x.half(), "CB_ERR_DTYPE"), (x[0], "CB_ERR_SHAPE"), (x, "CB_ERR_INVALID_ARG")):
        with pytest.raises(cb.CacheBlendError) as e:
            cb.cb_sample(bad, torch.zeros(2))
        assert e.value.name == name
