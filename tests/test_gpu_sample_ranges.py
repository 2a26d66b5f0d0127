"""Rows whose targets lie at the far end of the near masses, where their fp32 sums decide least."""
import numpy as np
import pytest
import torch

import rag_non_prefix_gb300 as cb
from tests._gpu import built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    built()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab,rows", [(32003, 4), (64000, 160), (65533, 20)])
def test_targets_at_the_end_of_the_mass(vocab, rows, dtype):
    """top_p and the number drawn a few steps below 1, an odd row and a pitch: nothing but the row's own tokens is drawn."""
    g = torch.Generator(device="cuda").manual_seed(vocab + rows)
    x = torch.full((rows, vocab + 5), 50.0, device="cuda", dtype=dtype)  # what lies between the rows is likelier than all of them
    spread = torch.logspace(-1, 1, rows, device="cuda")[:, None]
    x[:, 1:vocab + 1] = (spread * torch.randn(rows, vocab, generator=g, device="cuda")).clamp(max=40).to(dtype)
    logits = x[:, 1:vocab + 1]
    below = 1 - 2.0 ** -24 * torch.arange(1, rows + 1, device="cuda").fmod(7).add(1)
    for by_id in (False, True):
        for p in (None, below, below.flip(0)):
            u = below.float()
            got = cb.cb_sample(logits, u, top_p=None if p is None else p.float(), by_id=by_id).cpu()
            assert int(got.min()) >= 0 and int(got.max()) < vocab
            some = range(0, rows, max(1, rows // 16))
            near = logits[list(some)].double().cpu().numpy()
            for i, row in zip(some, near):
                assert int(got[i]) in _within(by_id, row, float(u[i]), 1.0 if p is None else float(p[i].float()))


def _within(by_id, x, u, p):
    """Tokens that the plain form draws with borders off by as much as the masses: 2^-28, and vocab units of 2^-44."""
    room = 2.0 ** -28 + x.size * 2.0 ** -44
    order = np.argsort(-x, kind="stable")
    weight = np.exp(x - x.max())
    mass = np.cumsum(weight[order])
    out = set()
    for b in (-room, room):
        n = x.size if p >= 1 else min(x.size, 1 + int(np.searchsorted(mass, (p + b) * mass[-1], side="left")))
        walk = np.sort(order[:n]) if by_id else order[:n]
        run = np.cumsum(weight[walk])
        lo, hi = (min(n - 1, int(np.searchsorted(run, (u + a) * run[-1], side="right"))) for a in (-room, room))
        out |= set(walk[lo:hi + 1].tolist())
    return out
