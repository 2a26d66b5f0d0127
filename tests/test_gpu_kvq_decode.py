"""Decoding as a user runs it: a prompt enters a 4-bit cache, then every step writes the new rows, attends, and
draws the next tokens; against the plain 64-bit forms on the same tokens."""
import pytest
import torch

import rag_non_prefix_gb300 as cb
from tests import kvq_ref as ref
from tests import sample_ref
from tests._gpu import built

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_on_a_4_bit_cache(dtype):
    built()
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    d, heads, hkv, dh, vocab, page, theta, steps = 256, 4, 2, 64, 1024, 16, 10000.0, 5
    lens = [40, 7, 29]
    n = len(lens)
    embed, lm = rand(vocab, d).to(dtype), (rand(vocab, heads * dh) * 2).to(dtype)
    wq, wk, wv = ((rand(w * dh, d) / 16).to(dtype) for w in (heads, hkv, hkv))
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    per = -(-(max(lens) + steps) // page)
    pool, table = cb.kvq_pool(n * per, page, hkv, dh), torch.randperm(n * per, generator=g, device="cuda").view(n, per).to(torch.int32)
    scratch, scale = cb.kvq_scratch(), dh ** -0.5

    def project(x, w, width):
        out = torch.empty(x.shape[0], width * dh, device="cuda")
        return cb.cb_gemm(x, w, out).view(-1, width, dh).to(dtype)

    def turned(x, at):  # rotary positions: one call of the re-rotation for each row's own
        out = torch.empty_like(x)
        for i, p in enumerate(at):
            cb.cb_rope_rerotate(x[i:i + 1], out[i:i + 1], None, None, p, theta)
        return out

    tokens = [torch.randint(0, vocab, (m,), generator=g, device="cuda") for m in lens]
    for i, ids in enumerate(tokens):
        x = embed[ids]
        cb.cb_kvq_write(pool, table, turned(project(x, wk, hkv), range(len(ids))), project(x, wv, hkv), ints(range(len(ids))), ints([i] * len(ids)))
    last = torch.stack([t[-1] for t in tokens])
    u = torch.rand(steps, n, generator=g, device="cuda")
    t, k, p = torch.full((n,), 0.8, device="cuda"), ints([50] * n), torch.full((n,), 0.95, device="cuda")
    for step in range(steps):
        at = [m + step for m in lens]
        x = embed[last]
        q, kn, vn = turned(project(x, wq, heads), at), turned(project(x, wk, hkv), at), project(x, wv, hkv)
        cb.cb_kvq_write(pool, table, kn, vn, ints(at))
        out = cb.cb_kvq_attention(q, ints(at), pool, table, scratch=scratch)
        logits = cb.cb_gemm(out.view(n, -1), lm, torch.empty(n, vocab, device="cuda"))
        last = cb.cb_sample(logits, u[step], t, k, p).long()

        # the new rows are held as the form holds them, the output is that of the rows held, the token that of the logits
        kr, vr = cb.cb_kvq_read(pool, table, ints(at), dtype=torch.float32)
        assert torch.equal(kr.double().cpu(), ref.values(kn)) and torch.equal(vr.double().cpu(), ref.values(vn))
        want, mass, room = ref.attention(q[:, None], ints(at), pool, table, scale)
        eps = torch.finfo(dtype).eps / 2
        room = room + mass * (eps if dtype is torch.bfloat16 else 0) + eps * want.abs() * 1.01
        assert torch.all((out.double().cpu() - want[:, 0]).abs() <= room[:, 0])
        for i in range(n):
            assert int(last[i]) in sample_ref.tokens(logits[i].double().cpu().numpy(), float(u[step, i]), float(t[i]), 50, float(p[i]))
    cb.cb_gemm_get_status()
