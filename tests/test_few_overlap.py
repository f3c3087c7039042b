"""The 4-bit conversions refuse buffers that lie in each other, before any launch."""

import ctypes

import pytest

import sparse_mixture_experts_22_b200 as M
from sparse_mixture_experts_22_b200 import binding as B
from sparse_mixture_experts_22_b200 import build as build_mod


@pytest.fixture(scope="module", autouse=True)
def built():
    build_mod.build()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("name", ["moe_q4_quantize", "moe_q4_dequantize"])
def test_results_that_overlap(name, which, group):
    """The two things that one call writes: the second inside the first, and each end
    by 16 bytes."""
    cfg = M.make_config(4, 256, 128, 4, 2, n_shared=1, h_shared=384)
    n, hid = (4, 128) if which == 0 else (1, 384)
    packed = (2 * n * hid * 256 * 2, n * hid * 256 * 2)
    codes = M.moe_q4_size(cfg, which, group)
    first, second = codes if name == "moe_q4_quantize" else packed
    at = 1 << 32
    for other in (at, at + first - 16, at - second + 16):
        ptrs = [1 << 30, 1 << 31, at, other]
        rc = getattr(B.load(), name)(ctypes.byref(cfg), which, group,
                                     *(ctypes.c_void_p(p) for p in ptrs), None)
        msg = B.load().moe_last_error().decode()
        assert rc == 1 and "overlap" in msg, (other - at, rc, msg)
