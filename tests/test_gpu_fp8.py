"""The 8-bit operators on the GPU against their definition in 64 bits: quantiser, residual RMS norm,
block-scaled product and the three together.  Tolerances count roundings (tests/fp8_ref.py)."""
import threading

import pytest
import torch

import rag_non_prefix_gb300 as cb
from tests import fp8_ref as ref
from tests._gpu import built

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step, relative
F32, ADD, SWIGLU, BF16 = cb.CB_FP8_STORE_F32, cb.CB_FP8_ADD_F32, cb.CB_FP8_SWIGLU_FP8, cb.CB_FP8_STORE_BF16


@pytest.fixture(scope="module", autouse=True)
def _build():
    built()


def rand(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def pitched(rows, cols, dtype, extra):
    """An uninitialised [rows, cols] matrix inside one of ``extra`` more columns and two more rows, all
    bytes set to 0x5a; ``whole`` is that matrix."""
    whole = torch.empty(rows + 2, cols + extra, dtype=dtype, device="cuda")
    whole.view(torch.uint8).fill_(0x5A)
    return whole, whole[:rows, :cols]


def untouched(whole, rows, cols):
    """Whether everything outside [rows, cols] still has its bytes."""
    w = whole.view(torch.uint8)
    size = whole.element_size()
    return bool((w[rows:] == 0x5A).all()) and bool((w[:, cols * size:] == 0x5A).all())


def coded(seed, rows, cols, block, scale=1.0):
    x = rand(seed, rows, cols) * scale
    x[:, ::97] *= 20.0
    return cb.cb_quantize(x, block)


# ---------------------------------------------------------------------------------- quantiser
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 128), (3, 144), (127, 256), (128, 272), (130, 1040), (37, 4096),
                                       (1031, 7168)])
def test_quantize_matches_definition(rows, cols, dtype, block):
    x = rand(rows + cols, rows, cols).to(DT[dtype])
    x[:, ::61] *= 30.0
    whole, codes = pitched(rows, cols, E4M3, 16)
    groups, blocks = -(-cols // 128), -(-rows // block)
    if block == 1:
        sw, scales = pitched(groups, rows, torch.float32, 4 + -rows % 4)
    else:
        sw, scales = pitched(blocks, groups, torch.float32, 3)
    got = cb.cb_quantize(x, block, codes, scales)
    assert got[0] is codes and got[1] is scales
    ref.check_quantised(codes, scales, x.double(), block)
    assert untouched(whole, rows, cols) and untouched(sw, scales.shape[0], scales.shape[1])


@pytest.mark.parametrize("block", [1, 128])
def test_quantize_zeros_tiny_huge_and_not_finite(block):
    x = rand(5, 256, 1280)
    x[:, :128] = 0
    x[:, 128:256] *= 1e-38          # below the smallest magnitude that a scale stands for
    x[:, 256:384] *= 1e37           # largest magnitudes around 4e37
    x[0, 512] = float("inf")
    x[130, 640] = float("nan")
    x[0, 768:896] = -0.0
    x[0, 900] = 3e38
    codes, scales = cb.cb_quantize(x, block)
    v = ref.values(codes, scales, block)
    # an infinity or a NaN takes its whole group along, and no other
    hit = torch.zeros_like(v, dtype=torch.bool)
    hit[:1 if block == 1 else 128, 512:640] = True
    hit[130:131 if block == 1 else 256, 640:768] = True
    if block == 128:
        hit[128:256, 640:768] = True
    assert torch.equal(torch.isnan(v), hit)
    fine = ~torch.isnan(v)
    x64, v64 = torch.where(fine, x.double(), 0.0), torch.where(fine, v, 0.0)
    c64 = torch.where(fine, codes.double(), 0.0)
    s = torch.where(torch.isfinite(scales), scales, torch.ones_like(scales))
    ref.check_quantised(c64, torch.where(torch.isfinite(scales), scales, (ref.group_amax(x64, block) / 448).float().t()
                                         if block == 1 else (ref.group_amax(x64, block) / 448).float()), x64, block)
    assert torch.equal(v64[:, :128], torch.zeros_like(v64[:, :128])) and bool((s > 0).all())


def test_quantize_reads_a_pitch_and_a_view():
    big = rand(3, 70, 640)
    x = big[3:60, 128:416]
    codes, scales = cb.cb_quantize(x)
    ref.check_quantised(codes, scales, x.double(), 1)
    dense = cb.cb_quantize(x.contiguous())
    assert torch.equal(codes.view(torch.uint8), dense[0].view(torch.uint8)) and torch.equal(scales, dense[1])


# ---------------------------------------------------------------------------------- norm
# fp32 error of the normalised row: a thread's 32 squares and the tree of 10 additions round 43 times
# (positive terms: relative 43 * 2^-24, halved by the square root), mean, eps, root, quotient, the two
# products and h's own addition once each: below 32 * 2^-24 = 2^-19.
NORM_REL = 2.0 ** -19


def check_norm(x, res, weight, eps, codes, scales, res_out):
    h = x.double() + (0 if res is None else res.double())
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.double()
    ref.check_quantised(codes, scales, y, 1, rel=NORM_REL + 2.0 ** -21)
    if res_out is not None:
        # one rounding to fp32 and one to the residual's type
        assert torch.all((res_out.double() - h).abs() <= h.abs() * (HALF[res_out.dtype] + 2.0 ** -24))


@pytest.mark.parametrize("xt,rt", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", None),
                                   ("f32", None)])
@pytest.mark.parametrize("rows,d", [(1, 16), (1, 4096), (5, 272), (33, 4112), (3, 7168), (130, 1040), (2, 32768),
                                    (2, 8208)])
def test_norm_matches_definition(rows, d, xt, rt):
    x = rand(rows + d, rows, d).to(DT[xt])
    res = None if rt is None else (rand(d, rows, d) * 4).to(DT[rt])
    weight = (1 + 0.1 * rand(7, d)).to(DT[xt]) if (rows + d) % 2 else None
    whole, codes = pitched(rows, d, E4M3, 32)
    sw, scales = pitched(-(-d // 128), rows, torch.float32, 4 + -rows % 4)
    rw, out = (None, None) if rt is None else (None, torch.empty_like(res))
    cb.cb_add_rmsnorm_quantize(x, res, weight, 1e-5, out, codes, scales)
    check_norm(x, res, weight, 1e-5, codes, scales, out)
    assert untouched(whole, rows, d) and untouched(sw, scales.shape[0], rows)


@pytest.mark.parametrize("xt,rt", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("bf16", None), ("f32", None)])
@pytest.mark.parametrize("rows,d", [(9, 128), (613, 256), (1023, 400), (1030, 720), (1029, 1008), (1031, 4112), (700, 8192),
                                    (330, 8208)])
def test_norm_of_many_rows(rows, d, xt, rt):
    """Rows of a warp, of a CTA with one, two and four pieces a thread; rows behind the last one stay."""
    test_norm_matches_definition(rows, d, xt, rt)


def test_norm_in_place_and_without_keeping_the_sum():
    x, res = rand(1, 37, 4096).bfloat16(), rand(2, 37, 4096)
    a = cb.cb_add_rmsnorm_quantize(x, res)
    assert a[2] is None
    h = res.clone()
    b = cb.cb_add_rmsnorm_quantize(x, h, residual_out=h)
    assert b[2] is h and torch.equal(h, res + x.float())
    assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])


def test_norm_of_zero_rows_and_pitched_residual():
    big = rand(9, 20, 1024)
    res, out = big[:9, 256:784], torch.zeros(20, 1024, device="cuda")[:9, :528]
    x = torch.zeros(9, 528, device="cuda")
    x[4] = -res[4]  # the sum of this row is zero
    codes, scales, _ = cb.cb_add_rmsnorm_quantize(x, res, residual_out=out)
    check_norm(x, res, None, 1e-5, codes, scales, out)
    assert torch.equal(codes[4].float(), torch.zeros(528, device="cuda"))
    codes, scales, _ = cb.cb_add_rmsnorm_quantize(x, eps=0.0)  # 0 / 0 in the rows of zeros
    assert torch.isnan(ref.values(codes, scales, 1)[[0, 1, 2, 3, 5, 6, 7, 8]]).all()


# ---------------------------------------------------------------------------------- product
def check_gemm(a, sa, b, sb, epi, c, addend=None, b2=None, sb2=None, c_scales=None):
    k = a.shape[1]
    acc, terms = ref.product(a, sa, b, sb)
    err = ref.product_error(terms, k)
    if epi == SWIGLU:
        up, uterms = ref.product(a, sa, b2, sb2)
        uerr = ref.product_error(uterms, k)
        y = ref.silu64(acc) * up
        # |silu'| < 1.1; the exponential is off by 2 + 1.2 |gate| units of 2^-23 and underflows below
        # -87, where SiLU itself is below 1e-35; quotient and product round once each
        err = 1.1 * err * (up.abs() + uerr) + ref.silu64(acc).abs() * uerr + 1e-35 * up.abs() + \
            y.abs() * (5 + 1.2 * acc.abs().clamp(max=90)) * 2.0 ** -23
        ref.check_quantised(c, c_scales, y, 1, err=err)
        return
    want = acc if addend is None else acc + addend.double()
    err = err + want.abs() * ((2.0 ** -8 + 2.0 ** -24) if epi == BF16 else 2.0 ** -24)
    bad = (c.double() - want).abs() > err
    assert not bool(bad.any()), (int(bad.sum()), torch.nonzero(bad)[:4].tolist(), float((c.double() - want).abs().max()))


def operands(m, width, k, epi, seed=0, extra=0):
    a, sa = coded(seed + 1, m, k, 1)
    b, sb = coded(seed + 2, width, k, 128, 0.02)
    b2, sb2 = coded(seed + 3, width, k, 128, 0.02) if epi == SWIGLU else (None, None)
    dtype = E4M3 if epi == SWIGLU else torch.bfloat16 if epi == BF16 else torch.float32
    per16 = 16 // torch.empty(0, dtype=dtype).element_size()
    pad = -width % per16 + extra * per16
    whole, c = pitched(m, width, dtype, pad)
    addend = None
    if epi == ADD:
        addend = torch.zeros(m, width + pad, device="cuda")[:, :width]
        addend.copy_(rand(seed + 4, m, width) * 4)
    csw, cs = pitched(-(-width // 128), m, torch.float32, 4 + -m % 4) if epi == SWIGLU else (None, None)
    return dict(a=a, sa=sa, b=b, sb=sb, b2=b2, sb2=sb2, c=c, addend=addend, c_scales=cs), whole, csw


def gemm(o, epi, stream=None):
    cb.cb_gemm_scaled(o["a"], o["sa"], o["b"], o["sb"], o["c"], epi, B2=o["b2"], B2_scales=o["sb2"], addend=o["addend"],
                      C_scales=o["c_scales"], stream=stream)


SIZES = [(1, 16, 16), (1, 128, 128), (2, 4096, 4096), (3, 272, 144), (7, 1040, 512), (15, 256, 4112), (16, 512, 1024),
         (17, 144, 2064), (31, 384, 640), (33, 768, 272), (63, 128, 14336), (64, 2048, 256), (65, 1664, 1152),
         (100, 4096, 128), (127, 400, 384), (129, 256, 896), (192, 1408, 512), (257, 528, 1040), (300, 1024, 2048),
         (535, 1792, 768), (1000, 272, 256), (1357, 768, 528)]


@pytest.mark.parametrize("epi", [F32, ADD, SWIGLU, BF16])
@pytest.mark.parametrize("m,width,k", SIZES)
def test_gemm_matches_definition(m, width, k, epi):
    o, whole, csw = operands(m, width, k, epi, seed=m + k, extra=1)
    gemm(o, epi)
    check_gemm(o["a"], o["sa"], o["b"], o["sb"], epi, o["c"], o["addend"], o["b2"], o["sb2"], o["c_scales"])
    assert untouched(whole, m, width)
    if epi == SWIGLU:
        assert untouched(csw, -(-width // 128), m)
    cb.cb_gemm_get_status()


@pytest.mark.parametrize("epi", [F32, ADD, BF16])
@pytest.mark.parametrize("m,width", [(1, 1), (5, 3), (40, 131), (300, 129), (300, 257)])
def test_gemm_of_any_number_of_features(m, width, epi):
    o, whole, _ = operands(m, width, 272, epi, seed=width)
    gemm(o, epi)
    check_gemm(o["a"], o["sa"], o["b"], o["sb"], epi, o["c"], o["addend"])
    assert untouched(whole, m, width)


PLANS = [(1, 0), (16, 1), (16, 2), (16, 3), (16, 4), (32, 1), (32, 3), (32, 4), (48, 1), (48, 4), (64, 1), (64, 2), (80, 1), (80, 4), (96, 2), (128, 1),
         (128, 2), (128, 3), (128, 4), (256, 1)]


@pytest.fixture(params=PLANS)
def plan(request):
    cb.cb_gemm_scaled_set_plan(*request.param)
    yield request.param
    cb.cb_gemm_scaled_set_plan(0, 0)


@pytest.mark.parametrize("epi", [F32, ADD, SWIGLU, BF16])
@pytest.mark.parametrize("m,width,k", [(1, 144, 16), (8, 2064, 1296), (15, 272, 4224), (70, 400, 144), (300, 528, 1168),
                                       (261, 5008, 656)])
def test_every_plan_matches_definition(plan, m, width, k, epi):
    """Each tiling, with few and many tiles per CTA, odd tails and fewer groups than pairs."""
    o, whole, csw = operands(m, width, k, epi, seed=m, extra=1)
    gemm(o, epi)
    check_gemm(o["a"], o["sa"], o["b"], o["sb"], epi, o["c"], o["addend"], o["b2"], o["sb2"], o["c_scales"])
    assert untouched(whole, m, width)
    if epi == SWIGLU:
        assert untouched(csw, -(-width // 128), m)
    first = o["c"].clone()
    gemm(o, epi)
    assert torch.equal(first.view(torch.uint8), o["c"].view(torch.uint8))
    if epi == ADD:
        o["c"].copy_(o["addend"])
        o["addend"] = o["c"]
        gemm(o, ADD)
        assert torch.equal(first, o["c"])
    cb.cb_gemm_get_status()


@pytest.mark.parametrize("epi,m,width,k", [
    (F32, 531, 7190, 4112), (ADD, 531, 7190, 4112), (BF16, 531, 7190, 4112), (SWIGLU, 531, 4128, 4112),
    (F32, 1101, 8219, 8208), (ADD, 1101, 8219, 8208), (BF16, 1101, 8219, 8208), (SWIGLU, 1101, 4112, 8208)])
def test_products_computed_in_two_parts(epi, m, width, k):
    """A last round of few tiles: its tokens (531) or its features (1101) become a product of their own."""
    o, whole, csw = operands(m, width, k, epi, seed=m, extra=1)
    gemm(o, epi)
    check_gemm(o["a"], o["sa"], o["b"], o["sb"], epi, o["c"], o["addend"], o["b2"], o["sb2"], o["c_scales"])
    assert untouched(whole, m, width)
    if epi == SWIGLU:
        assert untouched(csw, -(-width // 128), m)
    first = o["c"].clone()
    if epi == ADD:
        o["c"].copy_(o["addend"])
        o["addend"] = o["c"]
    gemm(o, epi)
    assert torch.equal(first.view(torch.uint8), o["c"].view(torch.uint8))
    cb.cb_gemm_get_status()


@pytest.mark.parametrize("epi", [F32, ADD, BF16])
def test_every_plan_with_ragged_rows(plan, epi):
    for m in (41, 11):
        o, whole, _ = operands(m, 301, 272, epi, seed=3)
        gemm(o, epi)
        check_gemm(o["a"], o["sa"], o["b"], o["sb"], epi, o["c"], o["addend"])
        assert untouched(whole, m, 301)


@pytest.mark.parametrize("m", [9, 40])
@pytest.mark.parametrize("layout", ["gate first", "up first", "own pitches"])
def test_every_plan_with_gate_and_up_anywhere(plan, layout, m):
    """Gate and up rows in either order in memory, and in matrices of different pitches."""
    o, _, _ = operands(m, 272, 400, SWIGLU, seed=4)
    room = torch.zeros(2, 272, 512, dtype=torch.uint8, device="cuda").view(E4M3)
    gate, up = (room[0], room[1]) if layout == "gate first" else (room[1], room[0])
    if layout == "own pitches":
        up = torch.zeros(272, 416, dtype=torch.uint8, device="cuda").view(E4M3)
    gate[:, :400].copy_(o["b"]), up[:, :400].copy_(o["b2"])
    o["b"], o["b2"] = gate[:, :400], up[:, :400]
    gemm(o, SWIGLU)
    check_gemm(o["a"], o["sa"], o["b"], o["sb"], SWIGLU, o["c"], None, o["b2"], o["sb2"], o["c_scales"])


@pytest.mark.parametrize("m,width,k", [(4, 512, 4096), (90, 640, 1040), (600, 512, 528)])
def test_gemm_adds_in_place_and_repeats(m, width, k):
    o, _, _ = operands(m, width, k, ADD)
    gemm(o, ADD)
    first = o["c"].clone()
    gemm(o, ADD)
    assert torch.equal(first, o["c"])
    o["c"].copy_(o["addend"])
    o["addend"] = o["c"]
    gemm(o, ADD)
    assert torch.equal(first, o["c"])


@pytest.mark.parametrize("m,width,k", [(5, 256, 512), (150, 384, 272), (700, 512, 384)])
def test_gemm_of_views_with_pitches(m, width, k):
    o, _, _ = operands(m, width, k, F32)
    gemm(o, F32)
    wide = {n: torch.zeros(o[n].shape[0] + 3, k + 48, dtype=torch.uint8, device="cuda").fill_(0x7F).view(E4M3) for n in "ab"}
    for n in "ab":  # what surrounds the matrix is NaN
        wide[n][: o[n].shape[0], 16:16 + k].copy_(o[n])
    sa = torch.full((o["sa"].shape[0], (m + 3) // 4 * 4 + 8), float("nan"), device="cuda")
    sa[:, 4:4 + m] = o["sa"]
    sb = torch.full((o["sb"].shape[0], o["sb"].shape[1] + 3), float("nan"), device="cuda")
    sb[:, 1:-2] = o["sb"]
    c = torch.empty(m, width, device="cuda")
    cb.cb_gemm_scaled(wide["a"][:m, 16:16 + k], sa[:, 4:4 + m], wide["b"][:width, 16:16 + k], sb[:, 1:-2], c, F32)
    assert torch.equal(c, o["c"])


@pytest.mark.parametrize("m,width,k", [(3, 256, 512), (150, 384, 512), (700, 512, 384)])
def test_gemm_keeps_nan_to_its_row_and_feature(m, width, k):
    o, _, _ = operands(m, width, k, F32)
    gemm(o, F32)
    clean = o["c"].clone()
    o["a"].view(torch.uint8)[m - 1, 130] = 0x7F   # NaN code
    o["b"].view(torch.uint8)[width - 2, 5] = 0xFF
    o["sa"][0, 0] = float("inf")                  # an infinite scale: NaN or infinite rows
    gemm(o, F32)
    hit = torch.zeros(m, width, dtype=torch.bool, device="cuda")
    hit[m - 1], hit[:, width - 2], hit[0] = True, True, True
    assert torch.equal(torch.isfinite(o["c"]), ~hit)
    assert torch.equal(o["c"][~hit], clean[~hit])


@pytest.mark.parametrize("m,width,k", [(6, 256, 512), (150, 384, 512), (520, 512, 384)])
def test_swiglu_of_extreme_gates(m, width, k):
    """Gates far out on both sides (SiLU underflows to 0 or is the gate), groups of zeros and a NaN."""
    o, _, _ = operands(m, width, k, SWIGLU)
    o["sa"][:, 1] *= 1e4
    o["a"].view(torch.uint8)[2] = 0
    gemm(o, SWIGLU)
    check_gemm(o["a"], o["sa"], o["b"], o["sb"], SWIGLU, o["c"], None, o["b2"], o["sb2"], o["c_scales"])
    assert torch.equal(o["c"][2].float(), torch.zeros(width, device="cuda"))
    o["b2"].view(torch.uint8)[129, 3] = 0x7F
    gemm(o, SWIGLU)
    v = ref.values(o["c"], o["c_scales"], 1)
    assert torch.isnan(v[:, 128:256]).all() and not torch.isnan(v[:, :128]).any()


def test_nothing_to_do_for_no_rows():
    codes, scales = cb.cb_quantize(torch.empty(0, 128, device="cuda"))
    assert codes.shape == (0, 128)
    assert cb.cb_add_rmsnorm_quantize(torch.empty(0, 128, device="cuda"))[0].shape == (0, 128)
    b, sb = coded(1, 128, 128, 128)
    c = torch.empty(0, 128, device="cuda")
    cb.cb_gemm_scaled(codes, scales, b, sb, c, F32)


def test_offsets_past_31_bits():
    """Codes, outputs and weights whose last rows lie more than 2^31 elements in."""
    pitch = 1 << 25
    whole = torch.zeros(66, pitch, dtype=torch.uint8, device="cuda").view(E4M3)  # 2.2 GB
    x = rand(3, 66, 256)
    a, sa = cb.cb_quantize(x, 1, whole[:, :256])
    assert torch.equal(a.view(torch.uint8), cb.cb_quantize(x)[0].view(torch.uint8))
    b, sb = cb.cb_quantize(x, 128, whole[:, 512:768])
    c = torch.empty(66, 66, device="cuda")[:, :66]
    out = torch.empty(66, 68, device="cuda")[:, :66]
    cb.cb_gemm_scaled(a, sa, b, sb, out, F32)
    check_gemm(a, sa, b, sb, F32, out)
    del whole, c


# ---------------------------------------------------------------------------------- together
def mlp(s, stream=None):
    cb.cb_add_rmsnorm_quantize(s["x"], s["h"], None, 1e-5, s["h"], s["codes"], s["scales"], stream=stream)
    cb.cb_gemm_scaled(s["codes"], s["scales"], *s["gate"], s["mid"], SWIGLU, B2=s["up"][0], B2_scales=s["up"][1],
                      C_scales=s["mid_scales"], stream=stream)
    cb.cb_gemm_scaled(s["mid"], s["mid_scales"], *s["down"], s["h"], ADD, addend=s["h"], stream=stream)


def mlp_state(m, d, ffn):
    return dict(x=rand(1, m, d).bfloat16(), h=rand(2, m, d) * 4, gate=coded(3, ffn, d, 128, 0.02),
                up=coded(4, ffn, d, 128, 0.02), down=coded(5, d, ffn, 128, 0.02),
                codes=torch.empty(m, d, dtype=E4M3, device="cuda"), scales=cb.row_scales(m, d),
                mid=torch.empty(m, ffn, dtype=E4M3, device="cuda"), mid_scales=cb.row_scales(m, ffn))


@pytest.mark.parametrize("m,d,ffn", [(1, 512, 1024), (24, 1024, 2816), (140, 512, 1424), (600, 768, 1280)])
def test_mlp_block_matches_definition_step_by_step(m, d, ffn):
    s = mlp_state(m, d, ffn)
    h0 = s["h"].clone()
    mlp(s)
    h1 = h0 + s["x"].float()
    check_norm(s["x"], h0, None, 1e-5, s["codes"], s["scales"], None)
    check_gemm(s["codes"], s["scales"], *s["gate"], SWIGLU, s["mid"], None, *s["up"], s["mid_scales"])
    check_gemm(s["mid"], s["mid_scales"], *s["down"], ADD, s["h"], h1)


@pytest.mark.parametrize("m", [3, 140, 600])
def test_mlp_block_captured_and_on_a_side_stream(m):
    s = mlp_state(m, 512, 1424)
    h0 = s["h"].clone()
    mlp(s)
    torch.cuda.synchronize()
    want = s["h"].clone()
    side = torch.cuda.Stream()
    s["h"].copy_(h0)
    torch.cuda.synchronize()
    mlp(s, stream=side)
    side.synchronize()
    assert torch.equal(s["h"], want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mlp(s)
    for _ in range(3):
        s["h"].copy_(h0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s["h"], want)


def test_two_products_at_once():
    """Calls on two streams share nothing."""
    o1, _, _ = operands(300, 1024, 2048, F32, seed=1)
    o2, _, _ = operands(20, 1024, 4096, F32, seed=2)
    gemm(o1, F32), gemm(o2, F32)
    torch.cuda.synchronize()
    want = o1["c"].clone(), o2["c"].clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        o1["c"].zero_(), o2["c"].zero_()
        torch.cuda.synchronize()
        gemm(o1, F32, s1), gemm(o2, F32, s2)
        torch.cuda.synchronize()
        assert torch.equal(o1["c"], want[0]) and torch.equal(o2["c"], want[1])


@pytest.mark.parametrize("m,width", [(300, 1024), (20, 1024), (600, 2048), (5, 512)])
def test_product_as_a_threads_first_call(m, width):
    """A thread that has not used the device yet, next to one that has."""
    o, _, _ = operands(m, width, 1040, F32, seed=6)
    gemm(o, F32)
    want = o["c"].clone()
    o["c"].zero_()
    torch.cuda.synchronize()
    stream, failed = torch.cuda.Stream(), []

    def call():
        try:
            gemm(o, F32, stream)
        except cb.CacheBlendError as e:
            failed.append(e)

    thread = threading.Thread(target=call)
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert not failed and torch.equal(o["c"], want)


def test_binding_refuses_what_does_not_fit():
    x, res = rand(1, 6, 256), rand(2, 6, 256)
    codes, scales = cb.cb_quantize(x)
    b, sb = coded(3, 128, 256, 128)
    c = torch.empty(6, 128, device="cuda")
    bad = [lambda: cb.cb_quantize(x, codes=codes[:, :128]), lambda: cb.cb_quantize(x, scales=scales.t()),
           lambda: cb.cb_quantize(x.t()), lambda: cb.cb_quantize(x[:, :200]), lambda: cb.cb_quantize(x, 128, scales=sb[:, :1]),
           lambda: cb.cb_quantize(x, codes=codes.view(torch.uint8)), lambda: cb.cb_quantize(x[:, 1:129]),
           lambda: cb.cb_add_rmsnorm_quantize(x, res[:5]), lambda: cb.cb_add_rmsnorm_quantize(x, residual_out=res),
           lambda: cb.cb_add_rmsnorm_quantize(x, res, residual_out=res.bfloat16()),
           lambda: cb.cb_add_rmsnorm_quantize(x, weight=res[0, :128]), lambda: cb.cb_add_rmsnorm_quantize(x, weight=res[0].bfloat16()),
           lambda: cb.cb_gemm_scaled(codes, scales, b[:, :128], sb, c), lambda: cb.cb_gemm_scaled(codes, scales, b, sb[:, :1], c),
           lambda: cb.cb_gemm_scaled(codes, scales[:, :5], b, sb, c), lambda: cb.cb_gemm_scaled(codes, scales, b, sb, c[:, :64]),
           lambda: cb.cb_gemm_scaled(codes, scales, b, sb, c.bfloat16()), lambda: cb.cb_gemm_scaled(codes, scales, b, sb, c, BF16),
           lambda: cb.cb_gemm_scaled(codes, scales, b, sb, c, ADD), lambda: cb.cb_gemm_scaled(codes, scales, b, sb, c, SWIGLU),
           lambda: cb.cb_gemm_scaled(codes, scales, b, sb, c, 7),
           lambda: cb.cb_gemm_scaled(codes, scales, b, sb, c, ADD, addend=rand(1, 6, 256)[:, :128])]
    for call in bad:
        with pytest.raises(cb.CacheBlendError):
            call()
    torch.cuda.synchronize()


@pytest.mark.parametrize("block", [1, 128])
def test_quantize_many_millions_of_rows(block):
    """More row blocks than a grid's second axis counts: like the quantised first and last rows alone."""
    rows = 65536 * 128 + 3 * 128 + 5
    x = rand(9, rows, 16).bfloat16()
    codes, scales = cb.cb_quantize(x, block)
    for lo, hi in [(0, 512), (65534 * 128, rows)]:
        c, s = cb.cb_quantize(x[lo:hi], block)
        assert torch.equal(c.view(torch.uint8), codes[lo:hi].view(torch.uint8))
        assert torch.equal(s, scales[:, lo:hi] if block == 1 else scales[lo // 128:-(-hi // 128)])


def test_binding_refuses_another_device(monkeypatch):
    x = torch.zeros(4, 128, device="cuda")
    codes, scales = cb.cb_quantize(x)
    monkeypatch.setattr(cb, "_get_device", lambda: torch.cuda.current_device() + 1)
    for call in (lambda: cb.cb_quantize(x), lambda: cb.cb_add_rmsnorm_quantize(x),
                 lambda: cb.cb_gemm_scaled(codes, scales, codes, scales, x)):
        with pytest.raises(cb.CacheBlendError, match="another device"):
            call()
