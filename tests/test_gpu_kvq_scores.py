"""Attention over the 4-bit cache where scores leave float32's range downwards."""
import pytest
import torch

import rag_non_prefix_gb300 as cb
from tests import kvq_ref as ref
from tests._gpu import built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    built()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("n", [40, 700, 3200])
@pytest.mark.parametrize("heads", [1, 12])
def test_scores_of_minus_infinity_weigh_nothing(n, dh, heads, dtype):
    """The first keys' products with the query are below -1e39: the others share the weight evenly."""
    out = n // 2
    pool, table = cb.kvq_pool(-(-n // 16), 16, 1, dh), torch.arange(-(-n // 16), dtype=torch.int32, device="cuda")[None].contiguous()
    g = torch.Generator(device="cuda").manual_seed(n + dh)
    k, v = torch.zeros(n, 1, dh, device="cuda"), torch.randn(n, 1, dh, generator=g, device="cuda")
    k[:out, 0, 0] = -1e20
    cb.cb_kvq_write(pool, table, k, v, ints(range(n)), ints([0] * n))
    q = torch.zeros(1, 2, heads, dh, device="cuda").to(dtype)
    q[..., 0] = 1e20
    got = cb.cb_kvq_attention(q, ints([[n - 1, n - 3]]), pool, table)[0].double().cpu()
    codes, scale, zero = ref.unpack(pool)[1]
    rows = ref.sequence(table.cpu(), 0, n, ref.decode((codes, scale, zero)))[:, 0]
    size = ref.sequence(table.cpu(), 0, n, (47 + zero.abs()) * scale)[:, 0].repeat_interleave(32, 1)
    for i, m in enumerate((n, n - 2)):
        want = rows[out:m].mean(0)
        # weights of 1: a step of the sums for 16 keys of a warp (64 of a CTA), the merges and the quotient, and the output's rounding
        room = (m / 64 + 32) * 2.0 ** -23 * size[out:m].mean(0) * 2 + want.abs() * torch.finfo(dtype).eps / 2
        assert torch.all((got[i] - want).abs() <= room)
    cb.cb_gemm_get_status()
