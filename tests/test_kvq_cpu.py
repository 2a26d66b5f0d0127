"""The 4-bit cache without a GPU: its layout, its arithmetic's bounds, and what the calls refuse."""
import ctypes as C
import math
import random

import pytest
import torch

import rag_non_prefix_gb300 as cb
from rag_non_prefix_gb300 import build as cbbuild
from tests import kvq_ref as ref


@pytest.fixture(scope="module")
def lib():
    cbbuild.build()
    return cb.load_library()


@pytest.mark.parametrize("dh", [64, 128])
def test_every_byte_of_a_block_has_one_meaning(dh):
    seen = {}
    for r in range(16):
        key, val, ks, vs = ref.offsets(dh, r)
        for c, at in enumerate(key):
            assert seen.setdefault((*at, "n"), ("k", r, c)) == ("k", r, c)
        for c, at in enumerate(val):
            assert seen.setdefault((*at, "n"), ("v", r, c)) == ("v", r, c)
        for name, start in (("ks", ks), ("vs", vs)):
            for b in range(dh // 8):
                for nib in (0, 1):
                    assert seen.setdefault((start + b, nib, "n"), (name, r, b, nib)) == (name, r, b, nib)
    assert len(seen) == 2 * 20 * dh


def test_bounds_of_the_form():
    """Every number is held within half a step, zeros are multiples of 1/4 of at most 64, scales are bf16."""
    rng = random.Random(3)
    for _ in range(300):
        mid, span = rng.choice([0, 0, 1, -40, 1e6]), 10.0 ** rng.uniform(-6, 6)
        g = torch.tensor([mid + span * rng.uniform(-1, 1) for _ in range(32)]).float().tolist()
        s, z = ref.params(min(g), max(g))
        assert torch.tensor(s).bfloat16().item() == s and abs(z) <= 64 and 4 * z == int(4 * z)
        assert torch.tensor(z).bfloat16().item() == z
        for x in g:
            assert abs(s * (ref.code(x, s, z) + z) - x) <= s / 2


def test_a_group_of_one_number():
    for x in (0.0, 1.0, -3.1416, 1e-30, -1e-45, 3e38):
        x = torch.tensor(x).float().item()
        s, z = ref.params(x, x)
        assert abs(s * (ref.code(x, s, z) + z) - x) <= max(abs(x) * 2.0 ** -7, 2.0 ** -120)


def cache(**kw):
    base = dict(pool=256, n_pages=4, page_tokens=16, n_kv_heads=2, head_dim=64, table=256, ld_table=2, max_pages=2, n_seqs=2)
    base.update(kw)
    return C.byref(cb.KvqCache(*[base[k] for k in ("pool", "n_pages", "page_tokens", "n_kv_heads", "head_dim", "table",
                                                     "ld_table", "max_pages", "n_seqs")]))


BAD_CACHES = [(dict(head_dim=96), 2), (dict(page_tokens=8), 2), (dict(page_tokens=24), 2), (dict(page_tokens=0), 2),
              (dict(n_kv_heads=0), 2), (dict(n_kv_heads=2000), 2), (dict(n_pages=-1), 2), (dict(max_pages=-1), 2),
              (dict(ld_table=1), 2), (dict(n_seqs=-1), 2), (dict(n_seqs=1 << 21), 2), (dict(pool=None), 1),
              (dict(pool=264), 1), (dict(table=None), 1), (dict(table=258), 1),
              (dict(page_tokens=1 << 20, max_pages=1 << 11, ld_table=1 << 11), 2)]


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_bad_caches_are_refused(lib, change, status):
    c = cache(**change)
    assert lib.cb_kvq_write(c, 256, 128, 256, 128, 1, None, 256, 1, None) == status
    assert lib.cb_kvq_read(c, None, 256, 1, 0, 1e4, 1, 256, 128, 256, 128, None) == status
    assert lib.cb_kvq_attention(c, 256, 256, 256, 1, 4, 0.1, 1, 256, 256, 256, 1 << 30, None) == status


def test_bad_arguments_are_refused(lib):
    c = cache()
    write = lambda k=256, ldk=128, v=256, ldv=128, dt=1, pos=256, rows=1: lib.cb_kvq_write(c, k, ldk, v, ldv, dt, None, pos, rows, None)  # noqa: E731
    assert [write(k=None), write(v=None), write(pos=None)] == [1, 1, 1]
    assert [write(k=264), write(v=264), write(ldk=127), write(ldv=120), write(ldk=132), write(rows=-1), write(rows=(1 << 30) + 1)] == [2] * 7
    assert write(dt=7) == 3 and write(rows=0, k=None, v=None, pos=None) == 0
    read = lambda k=256, ldk=128, pos=256, rows=1, theta=1e4, dt=1: lib.cb_kvq_read(c, None, pos, rows, 3, theta, dt, k, ldk, 256, 128, None)  # noqa: E731
    assert [read(k=None), read(pos=None)] == [1, 1] and read(dt=7) == 3 and read(rows=0, k=None) == 0
    assert [read(k=264), read(ldk=64), read(theta=0.0), read(theta=math.nan), read(rows=-1)] == [2] * 5
    att = lambda q=256, ldq=256, pos=256, t=1, h=4, dt=1, out=256, ldo=256, sc=256, size=1 << 30: lib.cb_kvq_attention(c, q, ldq, pos, t, h, 0.1, dt, out, ldo, sc, size, None)  # noqa: E731
    assert [att(q=None), att(pos=None), att(out=None)] == [1] * 3 and att(dt=5) == 3
    assert [att(h=3), att(h=0), att(t=-1), att(ldq=128), att(ldo=252), att(q=258), att(t=1 << 28)] == [2] * 7
    need = lib.cb_kvq_scratch_size()
    assert [att(sc=None), att(sc=264), att(size=need - 1)] == [5] * 3 and att(t=0, q=None) == 0


def test_page_bytes(lib):
    assert lib.cb_kvq_page_bytes(64, 8, 128) == 64 * 8 * 160
    assert lib.cb_kvq_page_bytes(16, 1, 64) == 1280
    assert [lib.cb_kvq_page_bytes(*a) for a in ((8, 8, 128), (16, 0, 128), (16, 8, 96), (-16, 8, 128))] == [0] * 4


def test_the_binding_refuses_before_the_library(lib):
    pool, table = cb.kvq_pool(2, 16, 2, 64, device="cpu"), torch.zeros(1, 2, dtype=torch.int32)
    assert pool.shape == (2, 2, 1, 1280)
    k, pos = torch.zeros(1, 2, 64), torch.zeros(1, dtype=torch.int32)
    for bad, name in (((pool.int(), table), "CB_ERR_DTYPE"), ((pool, table.long()), "CB_ERR_DTYPE"),
                      ((pool[0], table), "CB_ERR_SHAPE"), ((pool, table[0]), "CB_ERR_SHAPE"),
                      ((pool, table), "CB_ERR_INVALID_ARG")):  # (the last: not on a GPU)
        with pytest.raises(cb.CacheBlendError) as e:
            cb.cb_kvq_write(*bad, k, k, pos)
        assert e.value.name == name
    with pytest.raises(cb.CacheBlendError):
        cb.kvq_pool(2, 24, 2, 64, device="cpu")


def test_sizes_beyond_64_bits_and_misaligned_indices_are_refused(lib):
    """n_seqs * n_tok * n_heads that only wraps to a small number; int32 arrays off a multiple of 4 bytes."""
    many = cache(n_seqs=1 << 20)
    assert lib.cb_kvq_attention(many, 256, 1 << 20, 256, 1 << 30, 1 << 14, 0.1, 1, 256, 1 << 20, 256, 1 << 30, None) == 2
    c = cache()
    assert lib.cb_kvq_write(c, 256, 128, 256, 128, 1, None, 258, 1, None) == 1
    assert lib.cb_kvq_write(c, 256, 128, 256, 128, 1, 257, 256, 1, None) == 1
    assert lib.cb_kvq_read(c, None, 258, 1, 0, 1e4, 1, 256, 128, 256, 128, None) == 1
    assert lib.cb_kvq_read(c, 257, 256, 1, 0, 1e4, 1, 256, 128, 256, 128, None) == 1
    assert lib.cb_kvq_attention(c, 256, 256, 258, 1, 4, 0.1, 1, 256, 256, 256, 1 << 30, None) == 1
