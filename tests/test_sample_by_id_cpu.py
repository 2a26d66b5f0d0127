"""Sampling by rising id without a GPU: the plain form's properties, and what is handed over."""
import ctypes as C

import numpy as np

import rag_non_prefix_gb300 as cb
from tests import sample_by_id_ref as ref
from tests import sample_ref


def test_the_plain_form_draws_by_probability_along_ids():
    x = np.log(np.array([1.0, 4.0, 2.0, 3.0]))
    got = [ref.token(x, (i + 0.5) / 1000) for i in range(1000)]
    assert [got.count(i) for i in range(4)] == [100, 400, 200, 300] and got == sorted(got)
    for f in (dict(k=2), dict(p=0.41), dict(p=0.39), dict(m=0.4), dict(m=7), dict(p=0), dict(t=0)):
        # the same tokens as along falling logits, as often
        a, b = [ref.token(x, (i + 0.5) / 700, **f) for i in range(700)], [sample_ref.token(x, (i + 0.5) / 700, **f) for i in range(700)]
        assert sorted(a) == sorted(b) and a == sorted(a)
    assert ref.token(np.full(3, -np.inf), 0.5) == -1 and ref.token(np.array([np.nan, -5.0]), 0.5) == 1


def test_the_order_is_handed_over_behind_the_filters():
    for by_id in (False, True):
        s = cb.Sampling.from_buffer_copy(cb._filters(3, 0, None, None, None, None, by_id))
        assert s.by_id == by_id and not (s.temperature or s.top_k or s.top_p or s.min_p)
    assert C.sizeof(cb.Sampling) == len(cb._filters(3, 0, None, None, None, None, True))
