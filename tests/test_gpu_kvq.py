"""A KV cache in 4 bits: written, read back and attended to, against the plain 64-bit form."""
import math

import pytest
import torch

import rag_non_prefix_gb300 as cb
from tests import kvq_ref as ref
from tests._gpu import built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    built()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(seed, n_seqs, tokens, page, hkv, dh, spare=1):
    """(pool, table): every sequence with pages for ``tokens`` positions, in no order, some pages unused."""
    g = gen(seed)
    per = -(-tokens // page)
    order = torch.randperm(n_seqs * per + spare, generator=g, device="cuda")[:n_seqs * per]
    return cb.kvq_pool(n_seqs * per + spare, page, hkv, dh), order.view(n_seqs, per).to(torch.int32).contiguous()


def held(pool, table, seq, pos):
    """Rows the pool holds, by the plain unpacking: (k, v) [rows, heads, D] in 64 bits."""
    parts = [ref.decode(p) for p in ref.unpack(pool)]
    page = pool.shape[2] * 16
    t = table.cpu()
    return [torch.stack([p[int(t[s, x // page]), :, x % page] for s, x in zip(seq, pos)]) for p in parts]


# rows that fill blocks, that start and end inside them, that are scattered, one row
ROWS = {"whole": lambda n: [(s, p) for s in range(n) for p in range(48)],
        "ragged": lambda n: [(s, p) for s in range(n) for p in range(5 + s, 39)],
        "scattered": lambda n: [(s, (37 * i + 11 * s) % 48) for s in range(n) for i in range(0, 13)],
        "backwards": lambda n: [(n - 1 - s, 47 - p) for s in range(n) for p in range(48)],
        "one": lambda n: [(n - 1, 17)]}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("page", [16, 48])
def test_written_rows_hold_the_exact_form(dtype, dh, rows, page):
    n, hkv = 2, 3
    pool, table = make(1, n, 48, page, hkv, dh)
    pool.fill_(0xA5)
    where = ROWS[rows](n)
    seq, pos = zip(*where)
    g = gen(2)
    k, v = (rand(g, len(where), hkv, dh) * 3).to(dtype), rand(g, len(where), hkv, dh).to(dtype)
    k[..., 5] *= 30
    k[0, 0], v[0, 1] = 0, 1.5  # all alike
    v[-1, 2, :32] += 200
    before = pool.clone()
    cb.cb_kvq_write(pool, table, k, v, ints(pos), ints(seq))
    torch.cuda.synchronize()
    for got, want in zip(held(pool, table, seq, pos), (ref.values(k), ref.values(v))):
        assert torch.equal(got, want)
    # nothing else moved: the same bytes put back give the pool as it was
    mask = torch.zeros_like(pool, dtype=torch.bool)
    for s, p in where:
        key, val, ks, vs = ref.offsets(dh, p % 16)
        at = sorted({b for b, _ in key} | {b for b, _ in val}) + list(range(ks, ks + dh // 8)) + list(range(vs, vs + dh // 8))
        mask[int(table[s, p // page]), :, p % page // 16, torch.tensor(at)] = True
    assert torch.equal(torch.where(mask, before, pool), before)
    # read back: exact in fp32, one rounding in bf16
    kr, vr = cb.cb_kvq_read(pool, table, ints(pos), ints(seq), dtype=torch.float32)
    assert torch.equal(kr.double().cpu(), ref.values(k)) and torch.equal(vr.double().cpu(), ref.values(v))
    kb, vb = cb.cb_kvq_read(pool, table, ints(pos), ints(seq))
    assert torch.equal(kb, kr.bfloat16()) and torch.equal(vb, vr.bfloat16())
    cb.cb_gemm_get_status()


@pytest.mark.parametrize("dh", [64, 128])
def test_groups_at_the_edges_of_the_form(dh):
    """Constant, tiny, huge, one-sided and non-finite groups, ties between two codes, both zeros."""
    f = torch.float32
    rows = []
    base = torch.linspace(-1, 1, 32)
    for scale in (1e-44, 1e-38, 1e-30, 1.0, 1e30, 1e38):
        rows.append(base * scale)
    for mid in (0.0, -0.0, 1.0, -1.0, 1e-40, 3.3e38, -3.3e38, 100.3):
        rows.append(torch.full((32,), mid))
        rows.append(torch.full((32,), mid) * (1 + 0.001 * base))
    rows += [base + 5, base - 5, base + 50, base.abs() * 7, -base.abs() * 7]
    # exact ties: scale 1 (d = 14.75), zero -7.5: numbers at halves
    tie = torch.arange(32).float() * 0.5 - 7.5
    tie[0], tie[31] = -7.375, 7.375
    rows += [tie, tie * 2.0 ** -60, tie + 1]
    for bad in (float("inf"), -float("inf"), float("nan")):
        r = base.clone()
        r[7] = bad
        rows.append(r)
    r = base * 1e38
    r[0], r[1] = -3e38, 3e38  # the spread passes fp32's range
    rows.append(r)
    x = torch.stack(rows).to(f)
    per = dh // 32
    x = torch.cat([x, x[: -len(x) % per]]).view(-1, 1, dh)
    n = x.shape[0]
    pool, table = make(3, 1, n, 16, 1, dh)
    k = x.cuda()
    cb.cb_kvq_write(pool, table, k, k.flip(0).contiguous(), ints(range(n)), ints([0] * n))
    got = held(pool, table, [0] * n, range(n))
    for a, b in zip(got, (ref.values(x), ref.values(x.flip(0)))):
        assert torch.equal(a.nan_to_num(nan=12345.0), b.nan_to_num(nan=12345.0))


def test_random_numbers_of_every_kind_have_the_nearest_code():
    """bf16 numbers: many lie exactly between two codes."""
    g = gen(4)
    x = (rand(g, 96, 1, 128) * torch.exp(rand(g, 96, 1, 1))).bfloat16()
    pool, table = make(5, 1, 96, 32, 1, 128)
    cb.cb_kvq_write(pool, table, x, x * 8, ints(range(96)), ints([0] * 96))
    k, v = held(pool, table, [0] * 96, range(96))
    assert torch.equal(k, ref.values(x)) and torch.equal(v, ref.values(x * 8))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("delta,theta", [(1, 1e4), (517, 5e6), (100003, 1e4), (-517, 5e6)])
def test_keys_are_read_at_new_positions(dtype, delta, theta):
    n, hkv, dh = 40, 2, 128
    pool, table = make(6, 1, n, 16, hkv, dh)
    g = gen(7)
    cb.cb_kvq_write(pool, table, rand(g, n, hkv, dh), rand(g, n, hkv, dh), ints(range(n)), ints([0] * n))
    k, v = held(pool, table, [0] * n, range(n))
    kr, vr = cb.cb_kvq_read(pool, table, ints(range(n)), ints([0] * n), delta_pos=delta, theta=theta, dtype=dtype)
    a = delta * theta ** (-torch.arange(64, dtype=torch.float64) / 64)
    x, y = k[..., :64], k[..., 64:]
    want = torch.cat([x * a.cos() - y * a.sin(), x * a.sin() + y * a.cos()], -1)
    # cos and sin rounded to fp32, a product and a fused one: 3 roundings of 2^-24 of |x| + |y|; the output's rounding
    room = 3 * 2.0 ** -24 * (x.abs() + y.abs()).repeat(1, 1, 2) + torch.finfo(dtype).eps / 2 * want.abs() * 1.001
    assert torch.all((kr.double().cpu() - want).abs() <= room)
    assert torch.equal(vr, v.to(dtype).cuda())


def check_attention(q, q_pos, pool, table, scale=None, **kw):
    got = cb.cb_kvq_attention(q, q_pos, pool, table, scale=scale, **kw)
    shape = q.shape
    q4 = q if q.dim() == 4 else q[:, None]
    want, mass, room = ref.attention(q4, q_pos, pool, table, q4.shape[-1] ** -0.5 if scale is None else scale)
    eps = torch.finfo(q.dtype).eps / 2
    # fp32 arithmetic, the weights' rounding to bf16 (fp32 outputs: none) and the output's rounding
    room = room + mass * (eps if q.dtype is torch.bfloat16 else 0) + eps * want.abs() * 1.01 + 1e-30
    err = (got.double().cpu().view(want.shape) - want).abs()
    assert got.shape == shape and torch.all(err <= room), (err / room).max()
    return got


ATT = [  # sequences, tokens, kv heads, group, channels, page, lengths
    (1, 1, 1, 1, 128, 16, [1]), (1, 1, 2, 4, 128, 16, [16]), (1, 1, 2, 7, 128, 64, [17]), (2, 1, 2, 8, 64, 16, [63, 1]),
    (3, 1, 2, 4, 64, 48, [64, 65, 200]), (2, 1, 1, 16, 128, 64, [300, 5]), (2, 1, 2, 3, 128, 16, [129, 128]),
    (2, 3, 2, 4, 128, 16, [70, 3]), (1, 5, 2, 2, 64, 32, [90]), (2, 4, 1, 8, 128, 64, [257, 31]), (1, 17, 2, 5, 128, 16, [100]),
    (1, 1, 1, 40, 64, 16, [77]), (1, 1, 1, 2, 128, 64, [2000]), (40, 1, 2, 2, 64, 16, list(range(1, 121, 3)))]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", ATT, ids=lambda c: "-".join(map(str, c[:6])))
def test_attention_over_the_cache(case, dtype):
    n, t, hkv, grp, dh, page, lens = case
    top = max(lens)
    pool, table = make(8, n, top, page, hkv, dh)
    pool.fill_(0xFF)  # (unwritten positions hold NaN scales)
    g = gen(9)
    for i, m in enumerate(lens):
        k = rand(g, m, hkv, dh)
        k[..., 3] *= 8
        cb.cb_kvq_write(pool, table, k, rand(g, m, hkv, dh) + 0.3, ints(range(m)), ints([i] * m))
    q = (rand(g, n, t, hkv * grp, dh) * 1.5).to(dtype)
    # tokens end at the sequence's end; some see less than the one before, some nothing
    pos = torch.tensor([[m - t + i for i in range(t)] for m in lens]).clamp(min=-1)
    if t > 2:
        pos[0, 1] = 0
        pos[-1, 0] = -1
    q_pos = pos.to(torch.int32).cuda()
    if t == 1:
        check_attention(q[:, 0].contiguous(), q_pos.view(-1), pool, table)
    got = check_attention(q, q_pos, pool, table)
    again = cb.cb_kvq_attention(q, q_pos, pool, table)
    assert torch.equal(got, again)
    assert torch.all(got[(q_pos < 0).nonzero(as_tuple=True)] == 0)
    cb.cb_gemm_get_status()


def test_many_sequences_and_long_ones():
    """More tiles than are kept in shared memory, of one to some hundred keys; a sequence whose parts are many."""
    lens = [1 + (37 * i) % 90 for i in range(300)]
    pool, table, g = filled(30, lens, 16, 1, 64)
    q = rand(g, 300, 2, 64).bfloat16()
    check_attention(q, ints([m - 1 for m in lens]), pool, table)
    pool, table, g = filled(32, [30000], 256, 1, 128)
    for dtype in (torch.bfloat16, torch.float32):
        check_attention(rand(g, 1, 3, 2, 128).to(dtype), ints([[29999, 20000, 29998]]), pool, table)


def test_pages_beyond_32_bits():
    """A pool of 2.5 GB: pages at its end, written, read and attended to."""
    pool = torch.zeros(31000, 8, 4, 2560, dtype=torch.uint8, device="cuda")
    assert pool.numel() > 2 ** 31
    table = ints([[30999, 5, 30998], [3, 30500, 26300]])
    g = gen(34)
    k, v = rand(g, 300, 8, 128).bfloat16(), rand(g, 300, 8, 128).bfloat16()
    pos, seq = [p for p in range(150)] * 2, [0] * 150 + [1] * 150
    cb.cb_kvq_write(pool, table, k, v, ints(pos), ints(seq))
    near = [30999, 5, 30998, 3, 30500, 26300]
    few, small = pool[near].contiguous(), ints([[0, 1, 2], [3, 4, 5]])
    kr, vr = cb.cb_kvq_read(pool, table, ints(pos), ints(seq), dtype=torch.float32)
    for got, want in zip((kr, vr), cb.cb_kvq_read(few, small, ints(pos), ints(seq), dtype=torch.float32)):
        assert torch.equal(got, want)
    assert torch.equal(kr[:40].double().cpu(), ref.values(k[:40]))
    q = rand(g, 2, 16, 128).bfloat16()
    assert torch.equal(cb.cb_kvq_attention(q, ints([149, 149]), pool, table), cb.cb_kvq_attention(q, ints([149, 149]), few, small))


def test_padded_queries_of_nan():
    """A padding row's query may hold anything: its output is zero, and no other row sees it."""
    pool, table, g = filled(36, [50, 20], 16, 1, 128)
    q = rand(g, 2, 3, 4, 128).bfloat16()
    q[0, 1] = float("nan")
    q[1, 0] = float("inf")
    got = cb.cb_kvq_attention(q, ints([[48, -1, 49], [-1, 18, 19]]), pool, table)
    assert torch.all(got[0, 1] == 0) and torch.all(got[1, 0] == 0) and not torch.any(got.isnan())
    clean = q.clone()
    clean[0, 1], clean[1, 0] = 0, 0
    assert torch.equal(got, cb.cb_kvq_attention(clean, ints([[48, -1, 49], [-1, 18, 19]]), pool, table))


def test_pages_shared_by_two_sequences():
    """A common beginning in one set of pages, each sequence going on in its own."""
    g = gen(38)
    pool = cb.kvq_pool(6, 16, 2, 64)
    table = ints([[4, 0, 1], [4, 0, 5]])
    k, v = rand(g, 32, 2, 64), rand(g, 32, 2, 64)
    cb.cb_kvq_write(pool, table, k, v, ints(range(32)), ints([1] * 32))
    own = rand(g, 2, 2, 64)
    cb.cb_kvq_write(pool, table, own, own, ints([32, 32]))  # (row i of sequence i)
    check_attention(rand(g, 2, 4, 64).bfloat16(), ints([32, 32]), pool, table)


def test_the_first_calls_of_a_process_may_be_captured(tmp_path):
    """No call needs one before it: all three are captured first, replayed, and give what eager calls give."""
    code = """
import torch, rag_non_prefix_gb300 as cb
pool, table = cb.kvq_pool(4, 16, 1, 64), torch.tensor([[2, 0], [3, 1]], dtype=torch.int32, device="cuda")
k, q = torch.randn(2, 1, 64, device="cuda"), torch.randn(2, 2, 64, device="cuda")
pos, x, u = torch.tensor([0, 0], dtype=torch.int32, device="cuda"), torch.randn(2, 500, device="cuda"), torch.rand(2, device="cuda")
scratch, out = cb.kvq_scratch(), torch.empty_like(q)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    cb.cb_kvq_write(pool, table, k, k, pos)
    cb.cb_kvq_attention(q, pos, pool, table, out=out, scratch=scratch)
    kr, vr = cb.cb_kvq_read(pool, table, pos, dtype=torch.float32)
    tok = cb.cb_sample(x, u)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(tok, cb.cb_sample(x, u)) and torch.equal(out, cb.cb_kvq_attention(q, pos, pool, table))
assert torch.equal(vr, cb.cb_kvq_read(pool, table, pos, dtype=torch.float32)[1]) and (vr - k).abs().max() < 0.5
print("fine")
"""
    import subprocess
    import sys

    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=200)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def filled(seed, lens, page, hkv, dh, spare=1):
    pool, table = make(seed, len(lens), max(lens), page, hkv, dh, spare)
    g = gen(seed + 1)
    for i, m in enumerate(lens):
        cb.cb_kvq_write(pool, table, rand(g, m, hkv, dh), rand(g, m, hkv, dh), ints(range(m)), ints([i] * m))
    return pool, table, g


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_peaked_and_flat_scores(dtype):
    """One key that takes all the weight, late and early in the sequence, and keys that all weigh the same."""
    pool, table, g = filled(10, [700], 64, 1, 128)
    q = torch.zeros(1, 4, 128, device="cuda").to(dtype)
    k = cb.cb_kvq_read(pool, table, ints([3, 690]), ints([0, 0]), dtype=torch.float32)[0][:, 0]
    q[0, 0], q[0, 1], q[0, 2] = (k[0] * 20).to(dtype), (k[1] * 20).to(dtype), (-k[1] * 20).to(dtype)
    check_attention(q, ints([699]), pool, table)
    check_attention(q, ints([699]), pool, table, scale=0.0)


def test_strided_queries_and_outputs():
    pool, table, g = filled(12, [90, 50], 16, 2, 64)
    both = rand(g, 2, 3, 3 * 8 * 64).bfloat16()  # rows of q, k and v of a fused projection
    q = both[..., :8 * 64].unflatten(-1, (8, 64))
    out = torch.full((2, 3, 2 * 8 * 64), 7.0, device="cuda").bfloat16()
    q_pos = ints([[87, 88, 89], [47, 48, 49]])
    got = check_attention(q, q_pos, pool, table, out=out[..., 8 * 64:].unflatten(-1, (8, 64)))
    assert torch.equal(got, cb.cb_kvq_attention(q.contiguous(), q_pos, pool, table))
    assert torch.all(out[..., :8 * 64] == 7.0)
    # rows of k and v with a pitch, a page table with one
    wide = torch.zeros(2, table.shape[1] + 5, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    kv = both.view(6, 3 * 8 * 64)[:, 8 * 64:].unflatten(-1, (8, 128))
    k, v = kv[:, :2, :64], kv[:, :2, :64]
    with pytest.raises(cb.CacheBlendError):
        cb.cb_kvq_write(pool, wide[:, :table.shape[1]], k, v, ints(range(6)), ints([0] * 6))  # heads 128 apart
    k = both.view(6, 3 * 8 * 64)[:, 512:640].unflatten(-1, (2, 64))
    cb.cb_kvq_write(pool, wide[:, :table.shape[1]], k, k, ints(range(6)), ints([0] * 6))
    assert torch.equal(held(pool, table, [0] * 6, range(6))[0], ref.values(k))


def test_padding_rows_and_bad_indices():
    """Rows of negative position or sequence are left out; what lies outside the tables is reported."""
    pool, table, g = filled(14, [40, 40], 16, 1, 64)
    before = pool.clone()
    k = rand(g, 4, 1, 64)
    cb.cb_kvq_write(pool, table, k, k, ints([-1, 3, -7, 2]), ints([0, -1, 1, -5]))
    assert torch.equal(pool, before)
    out = torch.full((4, 1, 64), 9.0, device="cuda")
    kr, vr = cb.cb_kvq_read(pool, table, ints([-1, 3, 5, 2]), ints([0, -1, 1, -5]), k_out=out, v_out=out.clone())
    assert torch.all(kr[[0, 1, 3]] == 0) and torch.all(vr[[0, 1, 3]] == 0) and torch.any(kr[2] != 0)
    cb.cb_gemm_get_status()
    for pos, seq in (([48], [0]), ([2 ** 31 - 1], [0]), ([0], [2]), ([0], [2 ** 31 - 1])):
        cb.cb_kvq_write(pool, table, k[:1], k[:1], ints(pos), ints(seq))
        with pytest.raises(cb.CacheBlendError) as e:
            cb.cb_gemm_get_status()
        assert e.value.name == "CB_ERR_DEVICE"
        kr, _ = cb.cb_kvq_read(pool, table, ints(pos), ints(seq))
        assert torch.all(kr == 0)
        with pytest.raises(cb.CacheBlendError):
            cb.cb_gemm_get_status()
    assert torch.equal(pool, before)
    # a page that does not exist: its keys are left out
    q = rand(g, 2, 2, 64)
    want = cb.cb_kvq_attention(q, ints([15, 15]), pool, table)
    for bad in (-1, pool.shape[0], 2 ** 31 - 1):
        t2 = table.clone()
        t2[:, 1:] = bad
        cb.cb_kvq_write(pool, t2, k[:1], k[:1], ints([20]), ints([0]))
        with pytest.raises(cb.CacheBlendError):
            cb.cb_gemm_get_status()
        got = cb.cb_kvq_attention(q, ints([39, 39]), pool, t2)
        with pytest.raises(cb.CacheBlendError):
            cb.cb_gemm_get_status()
        assert (got - want).abs().max() < 1e-5
    assert torch.equal(pool, before)
    # a position beyond the table: seen as far as the table goes
    got = cb.cb_kvq_attention(q, ints([1000, 2 ** 31 - 1]), pool, table)
    assert torch.equal(got, cb.cb_kvq_attention(q, ints([47, 47]), pool, table))
    with pytest.raises(cb.CacheBlendError):
        cb.cb_gemm_get_status()


def test_nan_keys_and_values_reach_only_who_sees_them():
    pool, table, g = filled(16, [64], 16, 1, 128)
    k = rand(g, 1, 1, 128)
    k[0, 0, 40] = float("nan")
    cb.cb_kvq_write(pool, table, k, k, ints([37]), ints([0]))
    q = rand(g, 1, 3, 2, 128).bfloat16()
    got = cb.cb_kvq_attention(q, ints([[36, 37, 5]]), pool, table)
    assert torch.all(got[0, 1].isnan()) and not torch.any(got[0, 0].isnan()) and not torch.any(got[0, 2].isnan())
    # a NaN value alone: its group's channels
    ok = rand(g, 1, 1, 128)
    cb.cb_kvq_write(pool, table, ok, k, ints([37]), ints([0]))
    for dtype in (torch.bfloat16, torch.float32):
        for last in (37, 63):
            got = cb.cb_kvq_attention(q.to(dtype), ints([[36, last, 5]]), pool, table)
            assert torch.all(got[0, 1, :, 32:64].isnan()) and not torch.any(got[0, 1, :, :32].isnan())
            assert not torch.any(got[0, 1, :, 64:].isnan()) and not torch.any(got[0, 0].isnan())


def test_empty_calls():
    pool, table = make(18, 2, 32, 16, 1, 64)
    none = torch.zeros(0, 1, 64, device="cuda")
    cb.cb_kvq_write(pool, table, none, none, ints([]).view(0))
    k, v = cb.cb_kvq_read(pool, table, ints([]).view(0))
    assert k.shape == (0, 1, 64)
    assert cb.cb_kvq_attention(torch.zeros(0, 2, 64, device="cuda"), ints([]).view(0), pool, table[:0]).shape == (0, 2, 64)
    out = cb.cb_kvq_attention(torch.ones(2, 2, 64, device="cuda"), ints([5, 5]), pool, table[:, :0])
    assert torch.all(out == 0)  # no pages: nothing to see, and a report
    with pytest.raises(cb.CacheBlendError):
        cb.cb_gemm_get_status()


def test_streams_graphs_and_scratch():
    """Two streams with a scratch each; a captured write and attention, replayed after the inputs changed."""
    pool, table, g = filled(20, [300, 900, 20], 64, 2, 128)
    q = rand(g, 3, 8, 128).bfloat16()
    q_pos = ints([299, 899, 19])
    want = cb.cb_kvq_attention(q, q_pos, pool, table)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    scratch = [cb.kvq_scratch() for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, b in zip(streams, scratch):
            outs.append(cb.cb_kvq_attention(q, q_pos, pool, table, scratch=b, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    assert all(int(b[:3200].sum()) == 0 for b in scratch)

    k = rand(g, 3, 2, 128).bfloat16()
    out = torch.empty_like(q)
    step = lambda: (cb.cb_kvq_write(pool, table, k, k, q_pos), cb.cb_kvq_attention(q, q_pos, pool, table, out=out, scratch=scratch[0]))  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        k.copy_(rand(gen(seed), 3, 2, 128))
        q_pos.copy_(ints([299 - seed, 899 - 70 * seed, 19 - seed]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, check_attention(q, q_pos, pool, table))
    # a default scratch inside a capture is the graph's own
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out2 = cb.cb_kvq_attention(q, q_pos, pool, table)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out2, out)


def test_refusals_of_the_binding():
    pool, table = make(22, 2, 32, 16, 2, 64)
    q = torch.zeros(2, 4, 64, device="cuda")
    pos = ints([1, 1])
    bad = [lambda: cb.cb_kvq_attention(q.half(), pos, pool, table), lambda: cb.cb_kvq_attention(q[:1], pos, pool, table),
           lambda: cb.cb_kvq_attention(q, pos.long(), pool, table), lambda: cb.cb_kvq_attention(q, pos[:1], pool, table),
           lambda: cb.cb_kvq_attention(q[:, :3], pos, pool, table), lambda: cb.cb_kvq_attention(q[..., :32], pos, pool, table),
           lambda: cb.cb_kvq_attention(q.cpu(), pos, pool, table), lambda: cb.cb_kvq_attention(q, pos.cpu(), pool, table),
           lambda: cb.cb_kvq_attention(q, pos, pool, table, scratch=cb.kvq_scratch()[:64]),
           lambda: cb.cb_kvq_attention(q, pos, pool, table, out=q.bfloat16()),
           lambda: cb.cb_kvq_attention(q, pos, pool.transpose(0, 1), table),
           lambda: cb.cb_kvq_write(pool, table, q[:, :2], q[:, :2].bfloat16(), pos),
           lambda: cb.cb_kvq_write(pool, table, q, q, pos), lambda: cb.cb_kvq_write(pool, table.t(), q[:, :2], q[:, :2], pos),
           lambda: cb.cb_kvq_read(pool, table, pos, dtype=torch.float16), lambda: cb.cb_kvq_read(pool, table, pos, pos[:1]),
           lambda: cb.cb_kvq_read(pool, table, pos[:, None])]
    for call in bad:
        with pytest.raises(cb.CacheBlendError):
            call()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dh", [64, 128])
def test_nan_in_keys_of_no_weight(dtype, dh):
    """A NaN that a row sees reaches it, however little its key weighs, from whichever CTA's part of the sequence."""
    pool, table, g = filled(40, [3200], 64, 1, dh)
    k, v, q = torch.zeros(3200, 1, dh, device="cuda"), rand(g, 3200, 1, dh), torch.zeros(1, 2, 3, dh, device="cuda").to(dtype)
    q[..., 0] = 40.0
    v[700, 0, 40] = float("nan")
    k[:1000, 0, 0] = -64.0  # (a weight of exp(-40 * 64 / 8) or less)
    cb.cb_kvq_write(pool, table, k, v, ints(range(3200)), ints([0] * 3200))
    got = cb.cb_kvq_attention(q, ints([[3199, 699]]), pool, table)
    assert torch.all(got[0, 0, :, 32:64].isnan()) and not torch.any(got[0, 1].isnan())
    assert not torch.any(got[0, 0, :, :32].isnan()) and not torch.any(got[0, 0, :, 64:].isnan())
    # whole parts without a score that is a number
    k[:1000, 0, 0] = float("nan")
    cb.cb_kvq_write(pool, table, k, rand(g, 3200, 1, dh), ints(range(3200)), ints([0] * 3200))
    assert torch.all(cb.cb_kvq_attention(q, ints([[3199, 699]]), pool, table).isnan())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_sequence_of_almost_2_31_keys(dtype):
    """The longest sequence there is, 2^31 - 16 positions: one page at all of them but the last 8176."""
    page, n = 8176, 262657
    assert page * n == 2 ** 31 - 16
    pool, table = cb.kvq_pool(2, page, 1, 64), torch.zeros(1, n, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    k, v = torch.zeros(page, 1, 64, device="cuda"), torch.ones(page, 1, 64, device="cuda")
    cb.cb_kvq_write(pool, table, k, v, ints(range(page)), ints([0] * page))
    cb.cb_kvq_write(pool, table, k + 1, -v, ints(range(page * (n - 1), page * n)), ints([0] * page))
    q = torch.zeros(1, 3, 1, 64, device="cuda").to(dtype)
    q[..., 0] = 12.5  # a key of the last page weighs exp(12.5): 8176 of them about as much as all others
    seen = [page * n, page * n - 4000, page * (n - 1)]
    got = cb.cb_kvq_attention(q, ints([[x - 1 for x in seen]]), pool, table, scale=1.0)[0, :, 0].double().cpu()
    for row, x in zip(got, seen):
        a, b = min(x, page * (n - 1)), max(0, x - page * (n - 1)) * math.exp(12.5)
        want = (a - b) / (a + b)
        # weights of 1 and values of +-1 add up exactly within a CTA; at most 800 parts are added in fp32, each step off by
        # 2^-24 of the sum (2^-14.3), and scores and exponentials are good to 2^-16
        assert torch.all((row - want).abs() <= 2.0 ** -13 + abs(want) * torch.finfo(dtype).eps / 2)
    cb.cb_gemm_get_status()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [9, 3000])
def test_reads_into_strided_outputs(dtype, n):
    """Outputs at every 16-byte offset and pitch; what lies between their rows stays."""
    hkv, dh, vec = 3, 64, 16 // dtype.itemsize
    pool, table, _ = filled(50, [n], 64, hkv, dh)
    at = (ints(range(n)), ints([0] * n))
    want = cb.cb_kvq_read(pool, table, *at, dtype=dtype)
    for start, pad in ((0, vec), (vec, 0), (vec, 3 * vec), (2 * vec, 2 * vec)):
        bufs = [torch.full((n * (hkv * dh + pad) + 4 * vec,), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
        outs = [b[start:start + n * (hkv * dh + pad)].view(n, -1)[:, :hkv * dh].view(n, hkv, dh) for b in bufs]
        cb.cb_kvq_read(pool, table, *at, k_out=outs[0], v_out=outs[1])
        for b, o, w in zip(bufs, outs, want):
            assert torch.equal(o, w)
            o.fill_(7.0)
            assert torch.all(b == 7.0)
    mixed = torch.empty(n * hkv * dh + vec, dtype=dtype, device="cuda")[vec:].view(n, hkv, dh)
    got = cb.cb_kvq_read(pool, table, *at, k_out=mixed, dtype=dtype)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
