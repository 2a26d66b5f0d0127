"""Outputs that the 4-bit cache's calls and the sampler allocate belong to the stream that the call runs on."""
import pytest
import torch

import rag_non_prefix_gb300 as cb
from tests._gpu import built

pytestmark = pytest.mark.gpu

INPUT = {}


@pytest.fixture(scope="module", autouse=True)
def inputs():
    built()
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = 8192
    k = torch.randn(rows, 8, 128, generator=g, device="cuda").bfloat16()
    INPUT.update(pool=cb.kvq_pool(rows // 64, 64, 8, 128), table=torch.arange(rows // 64, dtype=torch.int32, device="cuda")[None],
                 pos=torch.arange(rows, dtype=torch.int32, device="cuda"), seq=torch.zeros(rows, dtype=torch.int32, device="cuda"),
                 q=torch.randn(1, 4096, 8, 128, generator=g, device="cuda").bfloat16(), q_pos=torch.arange(4096, dtype=torch.int32, device="cuda")[None] % 40,
                 logits=torch.randn(3 << 20, 4, generator=g, device="cuda"), uniform=torch.rand(3 << 20, generator=g, device="cuda"))
    cb.cb_kvq_write(INPUT["pool"], INPUT["table"], k, k, INPUT["pos"], INPUT["seq"])
    torch.cuda.synchronize()
    yield
    INPUT.clear()


def read(stream):
    return cb.cb_kvq_read(INPUT["pool"], INPUT["table"], INPUT["pos"], INPUT["seq"], stream=stream)[0]


def attention(stream):
    q = INPUT["q"].float() if stream is None else INPUT["q32"]
    INPUT["q32"] = q
    return cb.cb_kvq_attention(q, INPUT["q_pos"], INPUT["pool"], INPUT["table"], stream=stream)


def sample(stream):
    return cb.cb_sample(INPUT["logits"], INPUT["uniform"], stream=stream)


@pytest.mark.parametrize("call", [read, attention, sample])
def test_outputs_are_not_taken_from_a_busy_stream(call):
    out = call(None)
    torch.cuda.synchronize()
    want = out.clone()
    storage = out.untyped_storage().nbytes()
    assert storage >= 10 << 20  # (a block of its own in torch's allocator)
    side = torch.cuda.Stream()
    del out
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = torch.empty(storage, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(200_000_000)  # some 100 ms
    old.fill_(0x33)
    del old
    got = call(side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
