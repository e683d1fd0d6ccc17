"""The layer operators' largest sizes: refused on the host before an index of
32 bits could wrap."""
import ctypes

import pytest

from lossless_diffusion_speculative_b200 import binding as ob
from lossless_diffusion_speculative_b200 import build

P = ctypes.c_void_p(4096)         # a well aligned address that no refused call may touch


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ob.lib()


def test_quantize_refuses_rows_past_32_bit_columns(lib):
    for dtype in (ob.BF16, ob.F16, ob.F32):
        for H in ((1 << 30) + 1, (1 << 31) - 1024, (1 << 31) - 1):
            assert lib.orthrus_quantize_fp8(dtype, P, H, 1, H, P, P, None) == ob.ERR_UNSUPPORTED


def test_product_refuses_sizes_past_32_bits(lib):
    f = lib.orthrus_fp8_matmul
    for M, N, K in ((4, 64, (1 << 30) + 16), (4, 64, (1 << 31) - 16), (300, 600, (1 << 31) - 128)):
        assert f(P, P, P, P, M, N, K, ob.BF16, P, None, None) == ob.ERR_UNSUPPORTED
