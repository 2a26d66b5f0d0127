"""The 4-bit cache at the ends of float32's range."""
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


@pytest.mark.parametrize("delta", [0, 5])
@pytest.mark.parametrize("dh", [64, 128])
def test_groups_of_the_largest_numbers(dh, delta):
    """Finite groups whose zero times scale passes float32's range: values that do not are read as they are."""
    most = torch.finfo(torch.float32).max
    ramp = torch.linspace(0, 1, 32, dtype=torch.float64)
    rows = [torch.full((32,), -most), torch.full((32,), most), -most + 4e37 * ramp, most - 4e37 * ramp, -most + 3.3e38 * ramp,
            most - 3.3e38 * ramp, -3.39e38 + 1e36 * ramp, -most * ramp, most * ramp]
    two = torch.full((32,), -3e38, dtype=torch.float64)
    two[3] = -most
    x = torch.stack([r.double() for r in rows + [two, -two]]).clamp(-most, most).float()
    per = dh // 32
    x = torch.cat([x, x[: -len(x) % per]]).view(-1, 1, dh)
    n = x.shape[0]
    pool, table = cb.kvq_pool(1, 16, 1, dh), ints([[0]])
    cb.cb_kvq_write(pool, table, x.cuda(), x.flip(0).contiguous().cuda(), ints(range(n)), ints([0] * n))
    want_k, want_v = ref.values(x), ref.values(x.flip(0))
    kp, vp = (ref.decode(p)[0, 0, :n].unsqueeze(1) for p in ref.unpack(pool))
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)
    for dtype in (torch.float32, torch.bfloat16):
        k, v = cb.cb_kvq_read(pool, table, ints(range(n)), ints([0] * n), delta_pos=delta, dtype=dtype)
        # (a value within half a step of the largest number may itself lie beyond it: an infinity)
        assert torch.equal(v.cpu(), want_v.float().to(dtype))
        if delta == 0:
            assert torch.equal(k.cpu(), want_k.float().to(dtype))
    assert torch.isfinite(want_v.float()).sum() > want_v.numel() // 2
    cb.cb_gemm_get_status()
