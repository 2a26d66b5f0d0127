"""Sampling with a top_p of 0 or below: the first token, at the greedy way's time."""
import pytest
import torch

import rag_non_prefix_gb300 as cb
from tests._gpu import built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    built()


@pytest.mark.parametrize("by_id", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [3, 2000, 64000, 262144])
def test_top_p_of_zero_is_greedy(vocab, dtype, by_id):
    rows = 12
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x = (2 * torch.randn(rows, vocab, generator=g, device="cuda")).to(dtype)
    x[1, vocab // 2:] = x[1].max()  # many largest: the first of them
    x[2, 1] = float("inf")
    x[3] = -float("inf")
    want = torch.where(torch.arange(rows, device="cuda") == 3, -1, x.argmax(1)).int()
    want[1] = int((x[1] == x[1].max()).nonzero()[0])
    u = torch.rand(rows, generator=g, device="cuda")
    row = lambda v, d=torch.float32: torch.full((rows,), v, dtype=d, device="cuda")  # noqa: E731
    for p in (0.0, -0.0, -1.0, -float("inf")):
        for more in ({}, dict(temperature=row(1.3)), dict(top_k=row(40, torch.int32)), dict(top_k=row(1500, torch.int32)), dict(min_p=row(0.1))):
            assert torch.equal(cb.cb_sample(x, u, top_p=row(p), by_id=by_id, **more), want)
