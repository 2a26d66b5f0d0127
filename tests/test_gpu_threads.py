"""Calls of a thread that has not used the device yet, next to one that has."""
import threading

import pytest
import torch

import rag_non_prefix_gb300 as cb
from tests._gpu import built

pytestmark = pytest.mark.gpu


def rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def in_a_new_thread(call):
    """What ``call`` raised there, or None."""
    failed = []

    def run():
        try:
            call()
        except cb.CacheBlendError as e:
            failed.append(e)

    thread = threading.Thread(target=run)
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    return failed[0] if failed else None


@pytest.mark.parametrize("tiles", [1, 2])
def test_attention_as_a_threads_first_call(tiles):
    built()
    q, k, v = rand(1, 300, 8, 128), rand(2, 300, 2, 128), rand(3, 300, 2, 128)
    pos = torch.arange(300, dtype=torch.int32, device="cuda")
    cb.cb_attention_set_tiles(tiles)
    try:
        want, out = cb.cb_attention(q, pos, k, v), torch.zeros_like(q)
        torch.cuda.synchronize()
        stream = torch.cuda.Stream()
        assert in_a_new_thread(lambda: cb.cb_attention(q, pos, k, v, out, stream)) is None
    finally:
        cb.cb_attention_set_tiles(0)
    assert torch.equal(out, want)


@pytest.mark.parametrize("m", [40, 535])
def test_bf16_product_as_a_threads_first_call(m):
    built()
    a, b = rand(4, m, 512), rand(5, 768, 512)
    want, out = torch.empty(m, 768, device="cuda"), torch.zeros(m, 768, device="cuda")
    cb.cb_gemm(a, b, want)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    assert in_a_new_thread(lambda: cb.cb_gemm(a, b, out, stream=stream)) is None
    assert torch.equal(out, want)
