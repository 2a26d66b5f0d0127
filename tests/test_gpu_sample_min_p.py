"""Tokens whose weight lies next to min_p, many and small."""
import math

import numpy as np
import pytest
import torch

import rag_non_prefix_gb300 as cb
from tests._gpu import built

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -44  # of a weight


@pytest.fixture(scope="module", autouse=True)
def _build():
    built()


def small(dtype, units):
    """A logit near log(units 2^-44) whose weight is not near a whole number of units, below and above it a min_p in the same unit."""
    x = torch.tensor(math.log(units * UNIT), dtype=dtype)
    for _ in range(1000):
        w = math.exp(float(x)) / UNIT
        if 0.3 < w % 1 < 0.7:
            return float(x), float(np.float32((w - 0.25) * UNIT)), float(np.float32((w + 0.25) * UNIT))
        x = torch.nextafter(x, torch.tensor(-100.0, dtype=dtype))
    raise AssertionError


@pytest.mark.parametrize("by_id", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab,k,units", [(401, 0, 20000), (5000, 500, 20000), (5000, 3000, 5000), (262144, 0, 1000), (30000, 0, 2000)])
def test_small_weights_next_to_min_p(vocab, k, units, dtype, by_id):
    """The crowd is kept where its weight is above min_p, by however little, and left out where it is below: the last number drawn tells."""
    x0, below, above = small(dtype, units)
    assert below < math.exp(x0) < above and above - below < UNIT
    n = min(vocab, k or vocab) - 1
    crowd = n * math.exp(x0)  # its mass, the likeliest token's being 1
    assert crowd > 2.0 ** -22
    u = np.float32(1 - min(2.0 ** -23, crowd / 2)) if crowd < 2.0 ** -20 else np.float32(1 - crowd / 2)
    assert (1 + crowd) * float(u) > 1 + crowd / 8
    logits = torch.full((4, vocab), x0, dtype=dtype, device="cuda")
    logits[:, 0] = 0
    row = lambda v, d=torch.float32: torch.tensor(v, dtype=d, device="cuda")  # noqa: E731
    got = cb.cb_sample(logits, row([u] * 4), min_p=row([below, above, 0.0, 1.0]), top_k=row([k] * 4, torch.int32) if k else None, by_id=by_id).tolist()
    assert got[0] == got[2] > 0 and got[1] == got[3] == 0


def test_min_p_at_every_temperature():
    """The last kept of 4000 tokens at equal steps, by the definition in 64 bits."""
    steps = 4000
    x = torch.arange(steps, device="cuda").float().mul(-1 / 256)[None].contiguous()
    for t in (1e-3, 0.07, 1.0, 1.3, 77.0, 1e6):
        for m in (1.0, 0.999, 0.5, 0.1, 1e-3, 1e-6):
            w = np.exp(x[0].double().cpu().numpy() / float(np.float32(t)))
            near = np.abs(w / float(np.float32(m)) - 1).min()
            keep = int(np.count_nonzero(w >= float(np.float32(m))))
            if m < 1 and near < 2.0 ** -40:
                continue
            total = float(w[:keep].sum())
            if w[keep - 1] / total < 2.0 ** -20:
                continue  # (no number below 1 draws the last one)
            one = lambda v: torch.tensor([v], dtype=torch.float32, device="cuda")  # noqa: E731
            for by_id in (False, True):
                assert int(cb.cb_sample(x, one(1 - 2.0 ** -24), temperature=one(t), min_p=one(m), by_id=by_id)) == keep - 1, (t, m)
