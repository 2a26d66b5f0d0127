"""More cases of the 8-bit operators on the GPU: reuse of the products' rings, ranges, offsets, plans,
against the definition in 64 bits with the bounds of tests/fp8_ref.py."""
import ctypes as C
import subprocess

import pytest
import torch

import rag_non_prefix_gb300 as cb
from tests import fp8_ref as ref
from tests._gpu import built
from tests.test_gpu_fp8 import ADD, BF16, DT, F32, HALF, SWIGLU, check_gemm, check_norm, gemm, operands, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    built()


@pytest.fixture
def set_plan():
    yield cb.cb_gemm_scaled_set_plan
    cb.cb_gemm_scaled_set_plan(0, 0)


# ---------------------------------------------------------------------------------- rings
@pytest.mark.parametrize("epi", [F32, SWIGLU])
@pytest.mark.parametrize("plan", [(16, 1), (16, 3), (32, 2), (48, 1), (64, 1), (80, 3), (96, 1), (128, 1), (128, 2), (256, 1)])
def test_every_group_meets_its_own_factors(set_plan, plan, epi):
    """Sums of many more groups than a ring has stages, whose scales differ by orders of magnitude from
    one group to the next: a list of factors written over before it was read would show."""
    m, width, k = 130, 640, 7296
    o, whole, _ = operands(m, width, k, epi, seed=5)
    o["sa"].mul_(torch.tensor([1.0, 2.0 ** 12, 2.0 ** -12], device="cuda").repeat(19)[:, None])
    o["sb"].mul_(torch.tensor([1.0, 0.25, 4.0], device="cuda").repeat_interleave(19)[None, :])
    if epi == SWIGLU:  # gates of about unit size: the products' own bound holds for them as it stands
        o["sa"].mul_(2.0 ** -9)
        o["sb2"].mul_(torch.tensor([4.0, 1.0, 0.25], device="cuda").repeat(19)[None, :])
    set_plan(*plan)
    gemm(o, epi)
    check_gemm(o["a"], o["sa"], o["b"], o["sb"], epi, o["c"], None, o["b2"], o["sb2"], o["c_scales"])
    first = o["c"].view(torch.uint8).clone()
    for _ in range(20):
        o["c"].view(torch.uint8).zero_()
        gemm(o, epi)
        assert torch.equal(first, o["c"].view(torch.uint8))
    cb.cb_gemm_get_status()


# ---------------------------------------------------------------------------------- the tuning hook
TURNER = """
#include <pthread.h>
typedef int (*set_plan)(int, int);
static set_plan set;
static volatile int on;
static pthread_t thread;
static void *turn(void *unused) {
  while (on) set(1, 0), set(0, 0);
  return unused;
}
void turner_start(set_plan f) { set = f, on = 1; pthread_create(&thread, 0, turn, 0); }
void turner_stop(void) { on = 0; pthread_join(thread, 0); }
"""


def test_plan_changed_by_another_thread_in_the_middle_of_calls(set_plan, tmp_path):
    """A call reads the hook once: it has a plan whatever another thread sets meanwhile."""
    (tmp_path / "turner.c").write_text(TURNER)
    subprocess.run(["gcc", "-O2", "-shared", "-fPIC", "-pthread", str(tmp_path / "turner.c"), "-o",
                    str(tmp_path / "turner.so")], check=True)
    turner = C.CDLL(str(tmp_path / "turner.so"))
    few, _, _ = operands(40, 512, 640, F32, seed=8)
    two, _, _ = operands(531, 7190, 4112, ADD, seed=9)  # (two parts, but for the hook)
    turner.turner_start(C.cast(cb.load_library().cb_gemm_scaled_set_plan, C.c_void_p))
    try:
        for _ in range(200):
            gemm(few, F32)
            gemm(two, ADD)
    finally:
        turner.turner_stop()
    set_plan(0, 0)
    check_gemm(few["a"], few["sa"], few["b"], few["sb"], F32, few["c"])
    check_gemm(two["a"], two["sa"], two["b"], two["sb"], ADD, two["c"], two["addend"])


# ---------------------------------------------------------------------------------- ranges
@pytest.mark.parametrize("rt", [None, "f32", "bf16"])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d", [(3, 16), (9, 256), (40, 512), (1030, 1008), (7, 4096), (1031, 4112), (330, 8208), (2, 32768)])
def test_norm_of_rows_whose_squares_leave_fp32(rows, d, xt, rt):
    """Rows of any size that the type has: their squares' sum is infinite, subnormal or zero in fp32."""
    x = rand(d, rows, d)
    size = torch.tensor([1e20, 1.0, 1e37, 1e-3, 3e18, 1e30, 1e-30], device="cuda")[torch.arange(rows, device="cuda") % 7]
    x = (x * size[:, None]).to(DT[xt])
    res = None if rt is None else (rand(d + 1, rows, d) * size[:, None]).to(DT[rt])
    weight = (1 + 0.1 * rand(7, d)).to(DT[xt]) if rows % 2 else None
    out = None if rt is None else torch.empty_like(res)
    codes, scales, _ = cb.cb_add_rmsnorm_quantize(x, res, weight, 1e-5, out)
    check_norm(x, res, weight, 1e-5, codes, scales, out)


@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-36, 1e-20])
@pytest.mark.parametrize("rt", [None, "f32", "bf16"])
@pytest.mark.parametrize("rows,d", [(8, 256), (41, 512), (7, 4096), (1031, 4112), (3, 16384)])
def test_norm_of_tiny_rows_with_little_or_no_eps(rows, d, rt, eps):
    x = rand(d, rows, d)
    size = torch.tensor([1e-25, 1.0, 1e-20, 1e-30, 1e20, 3e-19, 1e-36], device="cuda")[torch.arange(rows, device="cuda") % 7]
    x = x * size[:, None]
    res = None if rt is None else (rand(d + 1, rows, d) * size[:, None]).to(DT[rt])
    out = None if rt is None else torch.empty_like(res)
    codes, scales, _ = cb.cb_add_rmsnorm_quantize(x, res, None, eps, out)
    # (eps is an fp32 argument: 1e-44 is 7 of its smallest steps 2^-149, that is 9.8e-45)
    check_norm(x, res, None, float(torch.tensor(eps, dtype=torch.float32)), codes, scales, None)
    if out is not None:
        # the sum's rounding to its type is relative only above 2^-126: bf16 numbers below are 2^-133 apart,
        # fp32 ones 2^-149, and a rounding is off by half of that
        h = x.double() + res.double()
        assert torch.all((out.double() - h).abs() <= h.abs() * (HALF[out.dtype] + 2.0 ** -24) + 2.0 ** (-134 if rt == "bf16" else -150))


@pytest.mark.parametrize("d", [256, 512, 4096, 16384])
def test_norm_of_infinite_rows_and_infinite_eps(d):
    """What is not finite stays so: 1 / inf gives zeros beside an infinity, and 0 * inf a NaN in its group."""
    x = rand(d, 5, d)
    x[1] *= 1e30
    x[1, 17] = float("inf")
    x[2, 3] = float("nan")
    x[3] = 0
    codes, scales, _ = cb.cb_add_rmsnorm_quantize(x)
    v = ref.values(codes, scales, 1)
    assert torch.isnan(v[1, :128]).all() and torch.equal(v[1, 128:], torch.zeros_like(v[1, 128:]))
    assert torch.isnan(v[2]).all() and torch.equal(v[3], torch.zeros_like(v[3]))
    check_norm(x[4:], None, None, 1e-5, codes[4:], scales[:, 4:], None)
    codes, scales, _ = cb.cb_add_rmsnorm_quantize(x[4:] * 1e25, eps=float("inf"))
    assert torch.equal(codes.float(), torch.zeros(1, d, device="cuda"))


@pytest.mark.parametrize("plan", [(16, 1), (64, 2), (128, 1), (256, 1)])
def test_swiglu_of_gates_whose_exponential_overflows(set_plan, plan):
    """Gates of -87 to -103: exp(-gate) is beyond 2^126 or infinite in fp32, SiLU around -1e-36 to -1e-43
    is not zero, and up features of 1e36 and more make numbers of ordinary size of it."""
    m, width, k = 130, 272, 128
    o, _, _ = operands(m, width, k, SWIGLU)
    one = torch.zeros(1, k, device="cuda")
    one[0, 0] = 1.0
    o["a"].copy_(one.expand(m, k))
    o["sa"][0] = torch.linspace(0.5, 1.0, m, device="cuda")
    o["b"].copy_(-one.expand(width, k))
    o["sb"][:, 0] = torch.tensor([87.8, 100.0, 103.0], device="cuda")
    o["b2"].copy_(one.expand(width, k) * torch.linspace(-2, 2, width, device="cuda")[:, None])
    o["sb2"][:, 0] = 1e38
    set_plan(*plan)
    gemm(o, SWIGLU)
    gate, up = ref.product(o["a"], o["sa"], o["b"], o["sb"])[0], ref.product(o["a"], o["sa"], o["b2"], o["sb2"])[0]
    y = ref.silu64(gate) * up
    # one product of a group each, which the scales' product and its multiplication round (2 * 2^-24): a
    # gate off by 2^-23 |gate| moves SiLU by (1 + |gate|) 2^-23; the exponential is off by 2 + 1.2 |gate|
    # units of 2^-23 or, among the subnormal numbers, by their step 2^-149; its sum with one, the quotient, up
    # and two products round within 5 units, product and quotient among subnormal numbers by a step each
    rel = (8 + 2.2 * gate.abs()) * 2.0 ** -23
    err = y.abs() * rel + (gate.abs() * 2.0 ** -149 + 2.0 ** -148) * up.abs()
    ref.check_quantised(o["c"], o["c_scales"], y, 1, err=err)
    assert float(y.abs().max()) > 0.1


# ---------------------------------------------------------------------------------- plans
def described(m, width, k, epi):
    text = cb.cb_gemm_scaled_describe(m, 2 * width if epi == SWIGLU else width, k, epi)
    return [dict(f.split("=") for f in part.split()) for part in text.split("; ")]


@pytest.mark.parametrize("epi,m,width,k", [
    (F32, 531, 7190, 4112), (ADD, 531, 7190, 4112), (BF16, 531, 7190, 4112), (SWIGLU, 531, 4128, 4112),
    (F32, 1101, 8219, 8208), (ADD, 1101, 8219, 8208), (BF16, 1101, 8219, 8208), (SWIGLU, 1101, 4112, 8208)])
def test_the_products_in_two_parts_are_launched_in_two(epi, m, width, k):
    """These shapes (whose results other tests check) do split, 531 tokens by tokens, 1101 by features."""
    parts = described(m, width, k, epi)
    assert len(parts) == 2
    tokens, features = ([int(p[n]) for p in parts] for n in ("tokens", "features"))
    if m == 531:
        assert sum(tokens) == m and tokens[0] % 256 == 0 and features == [width, width]
    else:
        assert sum(features) == width and features[0] % 128 == 0 and tokens == [m, m]
    assert parts[0]["token_tile"] == "256"


def test_plans_as_described(set_plan):
    assert cb.cb_gemm_scaled_describe(0, 128, 128) == "empty"
    assert cb.cb_gemm_scaled_describe(3, 4096, 4096) == "handful"
    assert "handful" not in cb.cb_gemm_scaled_describe(3, 8192, 4096, SWIGLU)
    set_plan(48, 2)
    (part,) = described(531, 7190, 4112, F32)
    assert (part["tokens"], part["features"], part["token_tile"], part["split"]) == ("531", "7190", "48", "2")


# ---------------------------------------------------------------------------------- far offsets
def far(rows, cols, dtype, pitch):
    """[rows, cols] whose last rows lie more than 2^31 elements in."""
    assert (rows - 1) * pitch > 2 ** 31
    return torch.empty(rows, pitch, dtype=dtype, device="cuda")[:, :cols]


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("plan,m", [((64, 1), 66), ((16, 3), 66), ((256, 1), 66), ((1, 0), 16), ((1, 0), 7)])
@pytest.mark.parametrize("epi", [F32, ADD, BF16, SWIGLU])
def test_product_with_every_matrix_past_31_bits(set_plan, plan, m, epi):
    if epi == SWIGLU and plan == (1, 0):
        plan = (16, 1)  # (that kernel has no such form)
    width, k = 2176, 2176  # 17 groups
    o, _, _ = operands(m, width, k, epi, seed=3)
    set_plan(*plan)
    gemm(o, epi)
    want, want_scales = o["c"].clone(), None if epi != SWIGLU else o["c_scales"].clone()
    pitch = 1 << 25 if m == 66 else 1 << 28 if m == 16 else 1 << 29
    moved = dict(o)
    for name, p in (("b", 1 << 20), ("b2", 1 << 20), ("sa", 1 << 27), ("sb", 1 << 27), ("sb2", 1 << 27), ("c_scales", 1 << 27),
                    ("a", pitch), ("c", pitch), ("addend", pitch)):
        if o[name] is None:
            continue
        rows = o[name].shape[0]
        moved[name] = far(*o[name].shape, o[name].dtype, max(p, -(-2 ** 31 // (rows - 1)) // 64 * 64 + 64))
        moved[name].copy_(o[name])
        if name not in ("a", "c", "addend"):  # (these three stay; the others are tried one by one)
            gemm(moved, epi)
            assert same(moved["c"], want)
            if epi == SWIGLU:
                assert same(moved["c_scales"], want_scales)
            moved[name] = o[name]
            torch.cuda.empty_cache()
    moved["c"].fill_(7.0)
    gemm(moved, epi)
    assert same(moved["c"], want)
    del moved
    torch.cuda.empty_cache()


@pytest.mark.parametrize("xt,rt", [("bf16", "f32"), ("f32", "bf16"), ("bf16", None)])
@pytest.mark.parametrize("d", [256, 512, 1024, 2176])
def test_norm_with_every_matrix_past_31_bits(d, xt, rt):
    rows, pitch = 66, 1 << 25
    x = rand(1, rows, d).to(DT[xt])
    res = None if rt is None else rand(2, rows, d).to(DT[rt])
    out = None if rt is None else torch.empty_like(res)
    codes, scales, _ = cb.cb_add_rmsnorm_quantize(x, res, None, 1e-5, out)
    fx, fcodes = far(rows, d, x.dtype, pitch), far(rows, d, codes.dtype, pitch)
    fx.copy_(x)
    fres, fout = (None, None) if rt is None else (far(rows, d, res.dtype, pitch), far(rows, d, res.dtype, pitch))
    if res is not None:
        fres.copy_(res)
    groups = d // 128
    fscales = far(groups, rows, torch.float32, -(-2 ** 31 // (groups - 1)) // 64 * 64 + 64)
    cb.cb_add_rmsnorm_quantize(fx, fres, None, 1e-5, fout, fcodes, fscales)
    assert same(fcodes, codes) and same(fscales, scales) and (out is None or same(fout, out))
    del fx, fres, fout, fcodes, fscales
    torch.cuda.empty_cache()


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_with_every_matrix_past_31_bits(dtype, block):
    rows, cols, pitch = 66 if block == 1 else 2177, 2176, 1 << 25 if block == 1 else 1 << 20
    x = rand(1, rows, cols).to(DT[dtype])
    codes, scales = cb.cb_quantize(x, block)
    fx, fcodes = far(rows, cols, x.dtype, pitch), far(rows, cols, codes.dtype, pitch)
    fx.copy_(x)
    fscales = far(*scales.shape, torch.float32, -(-2 ** 31 // (scales.shape[0] - 1)) // 64 * 64 + 64)
    cb.cb_quantize(fx, block, fcodes, fscales)
    assert same(fcodes, codes) and same(fscales, scales)
    del fx, fcodes, fscales
    torch.cuda.empty_cache()
