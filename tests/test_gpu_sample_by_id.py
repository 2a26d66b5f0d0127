"""Sampling whose draw walks the kept tokens by rising id, against the plain 64-bit form."""
import numpy as np
import pytest
import torch

import harness as hz
import harness.device as hd
import oracle.cacheblend as orc
import rag_non_prefix_gb300 as cb
from tests import sample_by_id_ref as ref
from tests._gpu import GpuWorkload, built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    built()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def row(x, dtype=torch.float32):
    return None if x is None else torch.tensor(x, dtype=dtype, device="cuda")


def check(logits, u, t=None, k=None, p=None, m=None):
    """Draws a token of every row (the filters: lists of a value per row, or None) and compares."""
    got = cb.cb_sample(logits, row(u), row(t), row(k, torch.int32), row(p), row(m), by_id=True).tolist()
    x = logits.double().cpu().numpy()
    f32 = lambda v, i, off: off if v is None else float(np.float32(v[i]))  # noqa: E731
    for i, tok in enumerate(got):
        want = ref.tokens(x[i], f32(u, i, 0.0), f32(t, i, 1.0), 0 if k is None else k[i], f32(p, i, 1.0), f32(m, i, 0.0))
        assert tok in want, (i, tok, want)
    return got


def likely(g, rows, vocab, dtype):
    """Logits as a model gives them: a broad crowd and a few likely tokens."""
    x = 2.0 * torch.randn(rows, vocab, generator=g, device="cuda")
    for _ in range(12):
        x.scatter_(1, torch.randint(0, vocab, (rows, 1), generator=g, device="cuda"), 4 + 5 * torch.rand(rows, 1, generator=g, device="cuda"))
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("filters", ["", "k", "p", "m", "kp", "km", "pm", "kpm"])
@pytest.mark.parametrize("vocab", [1, 2, 33, 1000, 4097, 32000, 128256, 262144])
def test_sample_matches_the_plain_form(vocab, filters, dtype):
    rows = 5
    rng = np.random.default_rng(vocab)
    x = likely(gen(vocab + len(filters)), rows, vocab, dtype)
    u = [0.0, 0.999999] + list(rng.random(rows - 2))
    check(x, u, [0.7, 1.0, 1.3, 0.2, 3.0], [1, 2, 50, 1000, 3000] if "k" in filters else None,
          [0.9, 0.5, 0.99, 0.999, 0.05] if "p" in filters else None, [0.05, 0.5, 0.001, 1e-5, 0.3] if "m" in filters else None)


@pytest.mark.parametrize("rows", [1, 70, 200, 400])
@pytest.mark.parametrize("vocab", [515, 20001])
def test_batches(rows, vocab):
    rng = np.random.default_rng(rows)
    x = likely(gen(rows), rows, vocab, torch.float32)
    f = [rng.choice([0.0, 0.5, 1.0, 2.0], rows).tolist(), rng.choice([0, 1, 40, 500], rows).tolist(),
         rng.choice([1.0, 0.9, 0.3], rows).tolist(), rng.choice([0.0, 0.02, 0.4], rows).tolist()]
    check(x, rng.random(rows).tolist(), *f)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [7, 3000, 64000])
def test_equal_logits(vocab, dtype):
    """Every token alike, two values, few values: the filters keep the lower ids."""
    flat = torch.full((1, vocab), 3.25, device="cuda")
    two = flat.clone()
    two[0, ::3] = 2.5
    few = torch.randint(0, 5, (1, vocab), generator=gen(1), device="cuda") * 0.5
    x = torch.cat([flat, two, few, -flat, few - 2]).to(dtype)
    for u in (0.0, 0.37, 0.9999):
        us = [u] * 5
        check(x, us)
        check(x, us, k=[5, vocab // 2 + 1, 2000, vocab - 1, vocab])
        check(x, us, p=[0.5, 0.9, 0.01, 0.77, 0.5])
        check(x, us, k=[2500, 1500, 40, vocab - 1, 3], p=[0.5, 0.9, 0.8, 0.77, 0.5], m=[0.0, 0.4, 0.1, 0.2, 0.9])
        check(x, us, t=[100.0, 1e-4, 1e6, 5.0, 30.0], p=[0.5, 0.9, 0.8, 0.77, 0.5])


def test_masked_rows():
    """-infinity, NaN and the type's lowest value in masked places, +infinity, nothing left, one token left."""
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    base = likely(gen(2), 12, 5000, torch.float32)
    for i, bad in enumerate((-inf, nan, low)):
        base[i, 100:] = bad
        base[3 + i, :] = bad
        base[6 + i, :] = bad
        base[6 + i, 4321] = -7.0
    base[9, 17] = base[9, 4000] = inf
    base[10, ::2] = -inf
    base[11, 1:] = -0.0
    base[11, 0] = 0.0
    for dtype in (torch.float32, torch.bfloat16):
        x = base.to(dtype)
        for u in (0.0, 0.6, 0.99999):
            us = [u] * 12
            got = check(x, us)
            assert got[3] == got[4] == -1 and got[6] == got[7] == got[8] == 4321 and got[9] == (17 if u < 0.5 else 4000)
            check(x, us, k=[200] * 12)
            check(x, us, k=[3000] * 12, p=[0.9] * 12)
            check(x, us, k=[40] * 12, p=[0.9] * 12, m=[0.1] * 12)
            check(x, us, t=[0.0] * 12)
            check(x, us, p=[0.8] * 12, t=[0.5] * 12)


def test_edges_of_the_filters():
    x = likely(gen(3), 8, 2000, torch.float32)
    us = [0.0, 0.2, 0.4, 0.6, 0.8, 0.9, 0.99, 0.99999]
    check(x, us, p=[0.0, -1.0, 1.0, 2.0, 1e-30, 0.999999, 0.5, 0.5])
    check(x, us, m=[1.0, 2.0, -1.0, 1e-30, 0.999, 0.0, 0.5, 0.5])
    check(x, us, k=[0, -5, 1, 2, 1024, 1025, 1999, 2000])
    check(x, us, t=[0.0, -1.0, 1e-30, 1e-3, 1e30, 50.0, float("inf"), 1.0])
    assert check(x, us, t=[float("nan")] * 8) == x.argmax(1).tolist()
    # random numbers outside [0, 1): the ends of what is kept
    three = x.topk(3).indices.sort(1).values
    k = row([3] * 8, torch.int32)
    for u, at in ((-1.0, 0), (float("nan"), 0), (1.5, 2)):
        assert cb.cb_sample(x, row([u] * 8), top_k=k, by_id=True).tolist() == three[:, at].tolist()


def test_close_tokens_are_told_apart():
    """65536 neighbours in fp32 within one range of the first cut, in no order."""
    n = 65536
    x = (torch.full((n,), 5.0, device="cuda").view(torch.int32) - torch.randperm(n, generator=gen(4), device="cuda").to(torch.int32)).view(torch.float32)
    x = x.repeat(4, 1)
    check(x, [0.1, 0.5, 0.9, 0.99], p=[0.9, 0.5, 1.0, 0.2])
    check(x, [0.1, 0.5, 0.9, 0.99], k=[10, 1024, 30000, 5000], p=[0.9, 0.5, 1.0, 0.2])


def test_rows_with_a_pitch_and_odd_addresses():
    wide = likely(gen(5), 6, 3001, torch.bfloat16)
    for start, vocab in ((0, 3001), (1, 3000), (7, 1001), (3, 2)):
        x = wide[:, start:start + vocab]
        check(x, [0.1, 0.3, 0.5, 0.7, 0.9, 0.99])
        check(x, [0.1, 0.3, 0.5, 0.7, 0.9, 0.99], p=[0.9] * 6)
        check(x[::2], [0.1, 0.5, 0.9], k=[7] * 3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [65520, 65533, 65536])
def test_the_ends_of_the_largest_rows_a_cta_takes(vocab, dtype):
    """Rows that start off a 16-byte boundary and whose likely tokens are their first and last."""
    rows, g = 200, gen(vocab)
    x = torch.randn(rows, vocab + 1, generator=g, device="cuda").to(dtype)[:, 1:]
    x[:, -2:] = x[:, :2] = 20.0
    for filters in ({}, dict(top_k=row([4] * rows, torch.int32)), dict(top_p=row([0.9] * rows)), dict(top_k=row([1000] * rows, torch.int32)),
                    dict(min_p=row([0.5] * rows))):
        for u, at in ((0.0, 0), (0.3, 1), (0.6, vocab - 2), (0.999, vocab - 1)):
            got = cb.cb_sample(x, row([u] * rows), by_id=True, **filters)
            assert set(got.tolist()) == {at}, (filters, u)


def test_a_graph_draws_anew_and_both_orders_share_a_stream():
    rows = 64
    x = likely(gen(6), rows, 32000, torch.float32)
    u = torch.rand(rows, generator=gen(7), device="cuda")
    p = row([0.9] * rows)
    falling = cb.cb_sample(x, u, top_p=p)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = cb.cb_sample(x, u, top_p=p, by_id=True)
        b = cb.cb_sample(x, u, top_p=p)
    for seed in (7, 8):
        u.copy_(torch.rand(rows, generator=gen(seed), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, cb.cb_sample(x, u, top_p=p, by_id=True)) and torch.equal(b, cb.cb_sample(x, u, top_p=p))
        assert seed != 7 or torch.equal(b, falling)
    assert not torch.equal(a, b)
    check(x, u.tolist(), p=[0.9] * rows)


def test_decode_step_draws_by_id():
    spec = hz.workload("tiny")
    g = GpuWorkload(spec, extra_positions=8)
    cfg = spec.cfg
    req = spec.requests[0]
    r = g.eng.make_request([s.chunk for s in req if s.chunk >= 0], hd.ids_tensor(req[-1].ids), decode_room=4)
    g.eng.blend_prefill([r], orc.ratio_schedule(cfg.n_layers, spec.ratio, spec.schedule))
    tok = r["first_token"].clone()
    hid = torch.zeros((1, cfg.d_model), dtype=torch.float32, device="cuda")
    lm = g.W["lm_head"].double()
    for u in (0.05, 0.5, 0.95):
        got = g.eng.decode_step([r], tok, n_past=[r["n_tokens"]], out_hidden=hid,
                                sampling={"uniform": row([u]), "temperature": row([1.5]), "top_k": row([40], torch.int32), "by_id": True})
        h = hid[0].double()
        logits = (lm @ (h / torch.sqrt((h * h).mean() + cfg.rms_eps))).cpu().numpy()
        # (fp32 logits: the number may be off the borders by what their error moves the masses)
        assert int(got) in {ref.token(logits, u + d, t=1.5, k=40) for d in (-1e-3, 0, 1e-3)}
    g.eng.get_status()
