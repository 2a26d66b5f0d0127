"""Host logic of the 8-bit entry points (no GPU needed)."""
import pytest

import rag_non_prefix_gb300 as cb
from rag_non_prefix_gb300 import build as cbbuild


@pytest.fixture(scope="module", autouse=True)
def _build():
    cbbuild.build()


def test_plan_description_refuses_and_needs_no_gpu():
    for bad in [(4, 128, 100), (4, 0, 128), (-1, 128, 128), (4, 48, 128, cb.CB_FP8_SWIGLU_FP8), (4, 128, 128, 4),
                (2 ** 30 + 1, 128, 128), (4, 128, 2 ** 22 + 16)]:
        with pytest.raises(cb.CacheBlendError):
            cb.cb_gemm_scaled_describe(*bad)
    assert cb.load_library().cb_gemm_scaled_describe(4, 128, 128, 0, None, 0) == 1
    assert cb.cb_gemm_scaled_describe(0, 128, 128) == "empty"
    assert cb.cb_gemm_scaled_describe(4, 4096, 4096) == "handful"
    text = cb.cb_gemm_scaled_describe(531, 7190, 4112)
    assert text == "none" or text.startswith("tokens=")
