"""Refusals of the 8-bit entry points (checked before anything is enqueued; no GPU needed)."""
import ctypes as C

import pytest
import torch

import rag_non_prefix_gb300 as cb
from rag_non_prefix_gb300 import build as cbbuild

OK, ARG, SHAPE, DTYPE = 0, 1, 2, 3
P = C.c_void_p(1 << 20)  # never dereferenced: every call below is refused, or has no rows
ODD = C.c_void_p((1 << 20) + 4)


@pytest.fixture(scope="module")
def lib():
    cbbuild.build()
    return cb.load_library()


def quantize(lib, x=P, ldx=256, rows=8, cols=256, dtype=1, block=1, codes=P, ldc=256, scales=P, lds=8):
    return lib.cb_quantize(x, ldx, rows, cols, dtype, block, codes, ldc, scales, lds, None)


@pytest.mark.parametrize("want,bad", [
    (SHAPE, dict(rows=-1)), (SHAPE, dict(cols=0)), (SHAPE, dict(cols=250)), (DTYPE, dict(dtype=2)),
    (ARG, dict(block=64)), (ARG, dict(x=None)), (ARG, dict(codes=None)), (ARG, dict(scales=None)),
    (SHAPE, dict(ldx=248)), (SHAPE, dict(ldx=260)), (SHAPE, dict(x=ODD)), (SHAPE, dict(codes=ODD)),
    (SHAPE, dict(ldc=240)), (SHAPE, dict(ldc=264)), (SHAPE, dict(scales=ODD)), (SHAPE, dict(lds=4)), (SHAPE, dict(lds=10)),
    (SHAPE, dict(block=128, lds=1)),
    (SHAPE, dict(rows=2 ** 30 + 4, lds=2 ** 30 + 4)), (SHAPE, dict(cols=2 ** 22 + 16, ldx=2 ** 23, ldc=2 ** 23)), (OK, dict(rows=0, x=None, codes=None))])
def test_quantize_refuses(lib, want, bad):
    assert quantize(lib, **bad) == want
    if want:
        assert lib.cb_last_error(None)


def norm(lib, x=P, ldx=256, xdt=1, res=P, res_out=P, ldr=256, rdt=0, w=None, rows=8, d=256, eps=1e-5, codes=P, ldc=256,
         scales=P, lds=8):
    return lib.cb_add_rmsnorm_quantize(x, ldx, xdt, res, res_out, ldr, rdt, w, rows, d, eps, codes, ldc, scales, lds, None)


@pytest.mark.parametrize("want,bad", [
    (SHAPE, dict(rows=-2)), (SHAPE, dict(d=0)), (SHAPE, dict(d=200)), (SHAPE, dict(d=32784, ldx=32784)),
    (DTYPE, dict(xdt=5)), (DTYPE, dict(rdt=-1)), (ARG, dict(eps=-1.0)), (ARG, dict(eps=float("nan"))),
    (ARG, dict(res=None)), (ARG, dict(x=None)), (ARG, dict(codes=None)), (ARG, dict(scales=None)), (SHAPE, dict(x=ODD)),
    (SHAPE, dict(ldx=100)), (SHAPE, dict(ldr=255)), (SHAPE, dict(ldr=258)), (SHAPE, dict(res=ODD)), (SHAPE, dict(res_out=ODD)),
    (SHAPE, dict(w=ODD)), (SHAPE, dict(ldc=128)), (SHAPE, dict(lds=7)), (SHAPE, dict(rows=2 ** 31 - 1, lds=2 ** 31)), (OK, dict(rows=0, x=None))])
def test_norm_refuses(lib, want, bad):
    assert norm(lib, **bad) == want


def mat(codes=P, ld=256, scales=P, lds=8):
    return cb.Fp8Mat(codes, ld, scales, lds)


def gemm(lib, a=None, b=None, b2=None, addend=P, c=P, ldc=512, cs=P, lds=8, m=8, n=512, k=256, epi=0, null=()):
    args = [None if i in null else C.byref(x if x is not None else mat()) for i, x in enumerate((a, b, b2))]
    return lib.cb_gemm_scaled(*args, addend, c, ldc, cs, lds, m, n, k, epi, None)


@pytest.mark.parametrize("want,bad", [
    (ARG, dict(epi=4)), (ARG, dict(epi=-1)), (SHAPE, dict(m=-1)), (SHAPE, dict(n=0)), (SHAPE, dict(k=0)), (SHAPE, dict(k=100)),
    (SHAPE, dict(n=48, epi=2)), (ARG, dict(null=(0,))), (ARG, dict(null=(1,))), (ARG, dict(null=(2,), epi=2)),
    (ARG, dict(c=None)), (ARG, dict(addend=None, epi=1)), (ARG, dict(cs=None, epi=2)), (ARG, dict(a=mat(codes=None))),
    (ARG, dict(b=mat(scales=None))), (SHAPE, dict(a=mat(ld=240))), (SHAPE, dict(a=mat(ld=264))), (SHAPE, dict(a=mat(codes=ODD))),
    (SHAPE, dict(a=mat(scales=ODD))), (SHAPE, dict(a=mat(lds=4))), (SHAPE, dict(a=mat(lds=9))), (SHAPE, dict(b=mat(lds=1))),
    (SHAPE, dict(b=mat(codes=ODD))), (SHAPE, dict(b2=mat(ld=16), epi=2)), (SHAPE, dict(c=ODD)), (SHAPE, dict(ldc=508)),
    (SHAPE, dict(ldc=514)), (SHAPE, dict(ldc=516, epi=3)), (SHAPE, dict(ldc=264, epi=2)), (SHAPE, dict(addend=ODD, epi=1)),
    (SHAPE, dict(cs=ODD, epi=2)), (SHAPE, dict(lds=6, epi=2)),
    (SHAPE, dict(m=2 ** 30 + 1, a=mat(lds=2 ** 31))), (SHAPE, dict(n=2 ** 30 + 32, ldc=2 ** 31)),
    (SHAPE, dict(k=2 ** 22 + 16, a=mat(ld=2 ** 23), b=mat(ld=2 ** 23, lds=2 ** 16))), (OK, dict(m=0, c=None))])
def test_gemm_refuses(lib, want, bad):
    assert gemm(lib, **bad) == want


def test_fp8_mat_layout_matches_c_compiler(tmp_path):
    import os
    import subprocess

    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "cacheblend.h"\nint main(void){printf("%zu %zu %zu %zu",'
                   "sizeof(cb_fp8_mat), offsetof(cb_fp8_mat, ld), offsetof(cb_fp8_mat, scales),"
                   " offsetof(cb_fp8_mat, ld_scales));return 0;}\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "layout")], check=True)
    got = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout.split()
    m = cb.Fp8Mat
    assert got == [str(v) for v in (C.sizeof(m), m.ld.offset, m.scales.offset, m.ld_scales.offset)]


def test_binding_refuses_what_is_no_cuda_matrix(lib):
    x = torch.zeros(4, 128)
    with pytest.raises(cb.CacheBlendError, match="CUDA matrix"):
        cb.cb_quantize(x)
    with pytest.raises(cb.CacheBlendError, match="unsupported dtype"):
        cb.cb_quantize(x.half())
    with pytest.raises(cb.CacheBlendError, match="must be a matrix"):
        cb.cb_quantize(x[0])
    with pytest.raises(cb.CacheBlendError):
        cb.cb_add_rmsnorm_quantize(x)
    c = torch.zeros(4, 128, dtype=torch.float8_e4m3fn)
    with pytest.raises(cb.CacheBlendError):
        cb.cb_gemm_scaled(c, x, c, x, x)


def test_plan_hook_refuses_what_has_no_kernel(lib):
    for bad in [(1, 1), (8, 1), (16, 0), (16, 5), (40, 1), (64, 8), (192, 1), (256, 2), (512, 1), (-16, 1), (0, 1), (128, -1)]:
        assert lib.cb_gemm_scaled_set_plan(*bad) == ARG
    for ok in [(1, 0), (16, 1), (16, 4), (48, 1), (64, 2), (80, 4), (96, 2), (128, 1), (128, 4), (256, 1), (0, 0)]:
        assert lib.cb_gemm_scaled_set_plan(*ok) == OK
