"""GPU checks of the layer operators where a result is decided by the last bits.

8-bit scales   bitwise equal to the fp32 product of the group's largest value and
               the nearest value to 1 / 448: no tolerance.
"""
import pytest
import torch

from lossless_diffusion_speculative_b200 import binding as ob
from test_gpu_layer_ops import TYPES, gen, randn

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- 8-bit values
def plain_scales(x):
    """Scales of [T, H], one per row and 128 columns."""
    T, H = x.shape
    n = -(-H // 128)
    blk = torch.nn.functional.pad(x.float(), (0, n * 128 - H)).view(T, n, 128)
    part = torch.full((), 1 / 448, dtype=torch.float32, device="cuda")
    return torch.mul(blk.abs().amax(-1), part).clamp_min(2.0 ** -126)


def quantized(x):
    T, H = x.shape
    q, sc = torch.empty(T, H, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(T, -(-H // 128), device="cuda")
    ob.orthrus_quantize_fp8(x, q, sc)
    return q, sc


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,H", [(1, 1), (32, 4096), (700, 1000), (900, 1422), (300, 1001), (5, 128)])
def test_quantize_scales_are_the_rounded_products(dtype, T, H):
    g = gen(T + H)
    x = (randn(g, T, H) * torch.exp(0.7 * randn(g, H))).to(TYPES[dtype])
    assert torch.equal(quantized(x)[1], plain_scales(x))


@pytest.mark.parametrize("e", [-149, -130, -118, -100, -80, -72, -40, 0, 60, 126])
def test_quantize_scales_over_the_exponent_range(e):
    """Groups whose largest value lies around 2^e: subnormal numbers, scales at
    and near their floor, and up to the type's largest values."""
    g = gen(e + 200)
    x = torch.ldexp(randn(g, 300, 384).clamp(-3.9, 3.9).double(), torch.tensor(e, device="cuda")).clamp(-3.4e38, 3.4e38).float()
    assert torch.equal(quantized(x)[1], plain_scales(x))
