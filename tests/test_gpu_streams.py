"""Outputs that a call allocates itself belong to the stream that the call runs on."""
import pytest
import torch

import rag_non_prefix_gb300 as cb
from tests._gpu import built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    built()


def rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def quantize_rows(stream):
    return cb.cb_quantize(INPUT["x"], stream=stream)[0]


def quantize_blocks(stream):
    return cb.cb_quantize(INPUT["x"], 128, stream=stream)[0]


def norm(stream):
    return cb.cb_add_rmsnorm_quantize(INPUT["x"], INPUT["res"], stream=stream)[0]


def scales_of_few_rows(stream):
    """(a group-major matrix of 12 MiB: one row of scales per 128 of 16 channels)"""
    return cb.cb_quantize(INPUT["tall"], stream=stream)[1]


def deviation(stream):
    k = INPUT["kv"]
    return cb.cb_kv_deviation(k, k, INPUT["kv2"], INPUT["kv2"], None, stream=stream)


def attention(stream):
    a = INPUT["q"]
    return cb.cb_attention(a, INPUT["pos"], INPUT["k"], INPUT["k"], stream=stream)


def encode(stream):
    return cb.cb_kv_encode(INPUT["chunk"], INPUT["chunk"], 8, stream=stream)


def decode(stream):
    return cb.cb_kv_decode(INPUT["blob"], INPUT["chunk"].shape, 8, 0, 1e4, torch.bfloat16, stream=stream)[0]


INPUT = {}
CALLS = [quantize_rows, quantize_blocks, norm, scales_of_few_rows, deviation, attention, encode, decode]


@pytest.fixture(scope="module", autouse=True)
def inputs(_build):
    rows = 3 << 20
    INPUT.update(x=rand(1, 4096, 4096).bfloat16(), res=rand(2, 4096, 4096), tall=rand(3, rows, 16).bfloat16(),
                 kv=rand(4, rows, 32), kv2=rand(5, rows, 32), q=rand(6, 4096, 16, 128).bfloat16(),
                 pos=torch.arange(4096, dtype=torch.int32, device="cuda"), k=rand(7, 4096, 4, 128).bfloat16(),
                 chunk=rand(8, 8, 2048, 4, 128).bfloat16())
    INPUT["blob"] = cb.cb_kv_encode(INPUT["chunk"], INPUT["chunk"], 8)
    torch.cuda.synchronize()
    yield
    INPUT.clear()


def plain(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("call", CALLS)
def test_outputs_are_not_taken_from_a_busy_stream(call):
    """The current stream still has to write to a block that it has given back: the output of a call
    on another stream, which does not wait for that, may not lie there."""
    out = call(None)
    torch.cuda.synchronize()
    want = plain(out).clone()
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
    assert torch.equal(plain(got), want)


@pytest.mark.parametrize("call", CALLS)
def test_dropped_outputs_are_not_given_to_another_stream(call):
    """The result of a call on a busy stream is dropped at once: its block may not go to the current stream."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    out = call(side)
    storage = out.untyped_storage().nbytes()
    del out
    mine = torch.full((storage,), 0x33, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert bool((mine == 0x33).all())


def test_a_raw_handle_is_a_stream_too():
    side = torch.cuda.Stream()
    want = plain(quantize_rows(None)).clone()
    torch.cuda.synchronize()
    for handle in (side.cuda_stream, 0):
        got = quantize_rows(handle)
        torch.cuda.synchronize()
        assert torch.equal(plain(got), want)
