"""Sampling against the plain 64-bit form."""
import numpy as np
import pytest
import torch

import harness as hz
import harness.device as hd
import oracle.cacheblend as orc
import rag_non_prefix_gb300 as cb
from tests import sample_ref as ref
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
    got = cb.cb_sample(logits, row(u), row(t), row(k, torch.int32), row(p), row(m)).tolist()
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


VOCABS = [1, 2, 31, 33, 1000, 4097, 32000, 64000, 128256, 262144]
FILTERS = ["", "k", "p", "m", "kp", "km", "pm", "kpm"]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("filters", FILTERS)
@pytest.mark.parametrize("vocab", VOCABS)
def test_sample_matches_the_plain_form(vocab, filters, dtype):
    rows = 5
    g = gen(vocab + len(filters))
    rng = np.random.default_rng(vocab)
    x = likely(g, rows, vocab, dtype)
    u = [0.0, 0.999999] + list(rng.random(rows - 2))
    check(x, u, [0.7, 1.0, 1.3, 0.2, 3.0], [1, 2, 50, 1000, 3000] if "k" in filters else None,
          [0.9, 0.5, 0.99, 0.999, 0.05] if "p" in filters else None, [0.05, 0.5, 0.001, 1e-5, 0.3] if "m" in filters else None)


@pytest.mark.parametrize("rows", [1, 3, 70, 200, 400])
@pytest.mark.parametrize("vocab", [515, 20001])
def test_batches(rows, vocab):
    """Rows that share an SM or spread over several, none of them aligned."""
    rng = np.random.default_rng(rows)
    x = likely(gen(rows), rows, vocab, torch.float32)
    f = [rng.choice([0.0, 0.5, 1.0, 2.0], rows).tolist(), rng.choice([0, 1, 40, 500], rows).tolist(),
         rng.choice([1.0, 0.9, 0.3], rows).tolist(), rng.choice([0.0, 0.02, 0.4], rows).tolist()]
    check(x, rng.random(rows).tolist(), *f)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [7, 3000, 64000])
def test_equal_logits(vocab, dtype):
    """Every token alike, two values, few values: rank goes by index."""
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
        base[i, 100:] = bad                 # 100 tokens left
        base[3 + i, :] = bad                # none (the lowest value: all alike)
        base[6 + i, :] = bad
        base[6 + i, 4321] = -7.0            # one
    base[9, 17] = base[9, 4000] = inf       # two of +infinity
    base[10, ::2] = -inf
    base[11, 1:] = -0.0
    base[11, 0] = 0.0                       # 0 and -0 are equal
    for dtype in (torch.float32, torch.bfloat16):
        x = base.to(dtype)
        for u in (0.0, 0.6, 0.99999):
            us = [u] * 12
            got = check(x, us)
            assert got[3] == got[4] == -1 and got[6] == got[7] == got[8] == 4321 and got[9] in (17, 4000)
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
    # random numbers outside [0, 1): the ends
    first, last = x.argmax(1).tolist(), check(x, [1 - 2.0 ** -24] * 8, k=[3] * 8)
    assert cb.cb_sample(x, row([-1.0] * 8), top_k=row([3] * 8, torch.int32)).tolist() == first
    assert cb.cb_sample(x, row([1.5] * 8), top_k=row([3] * 8, torch.int32)).tolist() == last
    assert cb.cb_sample(x, row([float("nan")] * 8), top_k=row([3] * 8, torch.int32)).tolist() == first


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
        check(x, [0.1, 0.3, 0.5, 0.7, 0.9, 0.99], p=[0.9] * 6)
        check(x[::2], [0.1, 0.5, 0.9], k=[7] * 3)
    guard = torch.full((8,), 77, dtype=torch.int32, device="cuda")
    cb.cb_sample(wide, row([0.5] * 6), out=guard[1:7])
    assert guard[0] == 77 and guard[7] == 77


def test_results_repeat_on_streams_and_in_graphs():
    rows = 64
    x = likely(gen(6), rows, 32000, torch.float32)
    u = torch.rand(rows, generator=gen(7), device="cuda")
    p, k = row([0.9] * rows), row([60] * rows, torch.int32)
    want = [cb.cb_sample(x, u, top_p=p), cb.cb_sample(x, u, top_k=k, top_p=p)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[cb.cb_sample(x, u, top_p=p, stream=s), cb.cb_sample(x, u, top_k=k, top_p=p, stream=s)] for _ in range(10) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cb.cb_sample(x, u, top_p=p)
    u.copy_(torch.rand(rows, generator=gen(8), device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, cb.cb_sample(x, u, top_p=p))


def test_empty_batch_and_refusals():
    assert cb.cb_sample(torch.zeros(0, 10, device="cuda"), torch.zeros(0, device="cuda")).shape == (0,)
    x, u = torch.zeros(2, 10, device="cuda"), torch.zeros(2, device="cuda")
    bad = [lambda: cb.cb_sample(x.half(), u), lambda: cb.cb_sample(x, u[:1]), lambda: cb.cb_sample(x, u.double()), lambda: cb.cb_sample(x, u.cpu()),
           lambda: cb.cb_sample(x, None), lambda: cb.cb_sample(x.t(), u), lambda: cb.cb_sample(x, u, top_k=u),
           lambda: cb.cb_sample(x, u, temperature=u[:1]), lambda: cb.cb_sample(x, u, out=u), lambda: cb.cb_sample(x[:1].expand(2, 10), u),
           lambda: cb.cb_sample(torch.zeros(1, (1 << 18) + 1, device="cuda"), u[:1])]
    for call in bad:
        with pytest.raises(cb.CacheBlendError):
            call()


def test_decode_step_draws_from_the_logits():
    """The engine's decode step with sampling: greedy filters give the greedy step's tokens, and a drawn token is
    the one that the plain form draws from the step's own logits."""
    spec = hz.workload("tiny")
    g = GpuWorkload(spec, extra_positions=8)
    cfg = spec.cfg
    req = spec.requests[0]

    def blended():
        r = g.eng.make_request([s.chunk for s in req if s.chunk >= 0], hd.ids_tensor(req[-1].ids), decode_room=4)
        g.eng.blend_prefill([r], orc.ratio_schedule(cfg.n_layers, spec.ratio, spec.schedule))
        return r

    a, b = blended(), blended()
    tok = a["first_token"].clone()
    want = g.eng.decode_step([a], tok)
    for sampling in ({"uniform": row([0.7]), "temperature": row([0.0])}, {"uniform": row([0.9]), "top_k": row([1], torch.int32)},
                     {"uniform": row([0.0])}):
        assert torch.equal(g.eng.decode_step([b], tok, n_past=[b["n_tokens"]], sampling=sampling), want)
    hid = torch.zeros((1, cfg.d_model), dtype=torch.float32, device="cuda")
    lm = g.W["lm_head"].double()
    for u in (0.05, 0.5, 0.95):
        got = g.eng.decode_step([b], tok, n_past=[b["n_tokens"]], out_hidden=hid,
                                sampling={"uniform": row([u]), "temperature": row([1.5]), "top_k": row([40], torch.int32), "top_p": row([0.9])})
        h = hid[0].double()
        logits = (lm @ (h / torch.sqrt((h * h).mean() + cfg.rms_eps))).cpu().numpy()
        # (fp32 logits: the number may be off the borders by what their error moves the masses)
        near = {ref.token(logits, u + d, 1.5, 40, 0.9 + e) for d in (-1e-3, 0, 1e-3) for e in (-1e-3, 0, 1e-3)}
        assert int(got) in near
    with pytest.raises(cb.CacheBlendError):
        g.eng.decode_step([b], tok, n_past=[b["n_tokens"]], sampling={"temperature": row([1.0])})
    with pytest.raises(cb.CacheBlendError):
        g.eng.decode_step([b], tok, n_past=[b["n_tokens"]], sampling={"uniform": row([0.5]), "topk": None})
    g.eng.get_status()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [65520, 65533, 65536])
def test_the_last_tokens_of_the_largest_rows_a_cta_takes(vocab, dtype):
    """Rows that start off a 16-byte boundary and whose likely tokens are their last."""
    rows, g = 200, gen(vocab)
    wide = torch.randn(rows, vocab + 1, generator=g, device="cuda").to(dtype)
    x = wide[:, 1:]
    x[:, -4:] = 20.0
    got = cb.cb_sample(x, torch.rand(rows, generator=g, device="cuda"), top_k=row([4] * rows, torch.int32))
    assert set(got.tolist()) == set(range(vocab - 4, vocab))
    for filters in (dict(top_k=row([4] * rows, torch.int32)), dict(top_p=row([0.9] * rows)), dict(top_k=row([1000] * rows, torch.int32))):
        got = cb.cb_sample(x, row([0.999] * rows), **filters)
        assert set(got.tolist()) == {vocab - 1}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [300, 32000, 128256])
def test_rows_masked_by_the_lowest_value(vocab, dtype):
    """Fewer tokens than top-k keeps, the others at the type's lowest value, at -infinity, or far below."""
    g, rng = gen(vocab), np.random.default_rng(vocab)
    x = likely(g, 8, vocab, dtype)
    some = torch.rand(8, vocab, generator=g, device="cuda") < 20 / vocab
    some[:, vocab - 1] = True
    low = [torch.finfo(dtype).min, -float("inf"), -1e4, -60.0] * 2
    x = torch.where(some, x, torch.tensor(low, dtype=dtype, device="cuda")[:, None])
    u, t = list(rng.random(8)), [0.7, 1.0, 2.0, 1.5, 1e-3, 1e3, 20.0, 0.1]
    check(x, u, t, [50] * 8)
    check(x, u, t, [200] * 8, [0.9, 0.5, 0.99, 1.0] * 2, [0.0, 0.1, 0.0, 0.01] * 2)
    check(x, u, t, p=[0.9, 0.5, 0.99, 1.0] * 2)
    check(torch.full_like(x, torch.finfo(dtype).min), u, t, [50] * 8)
