"""GPU checks of the layer operators where a result is decided by the last bits.

8-bit scales   bitwise equal to the fp32 product of the group's largest value and
               the nearest value to 1 / 448: no tolerance.
8-bit values   bitwise equal to the fp32 division by the scale, rounded once to
               e4m3: no tolerance.
Attention of mixed shapes: the bound that test_gpu_layer_ops.py derives.
"""
import math

import pytest
import torch

from lossless_diffusion_speculative_b200 import binding as ob
from test_gpu_layer_ops import (TYPES, check_product, close, fp8_operands, gen, guard, half_step, paged_cache, paged_ref, randn,
                                run_paged, tiny)

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


@pytest.mark.parametrize("e", [-149, -130, -118, -100, -80, -72, -40, 0, 60, 87, 89, 126])
def test_quantize_scales_over_the_exponent_range(e):
    """Groups whose largest value lies around 2^e: subnormal numbers, scales at
    and near their floor, and up to the type's largest values."""
    g = gen(e + 200)
    x = torch.ldexp(randn(g, 300, 384).clamp(-3.9, 3.9).double(), torch.tensor(e, device="cuda")).clamp(-3.4e38, 3.4e38).float()
    assert torch.equal(quantized(x)[1], plain_scales(x))


def plain_values(x, scale):
    T, H = x.shape
    q = x.float() / scale.repeat_interleave(128, 1)[:, :H]
    return q.clamp(-448, 448).to(torch.float8_e4m3fn)


def check_values(q, want):
    """The same bits (but for the sign of a zero)."""
    differ = (q.view(torch.uint8) != want.view(torch.uint8)) & ~((q.float() == 0) & (want.float() == 0))
    assert not differ.any(), f"{int(differ.sum())} of {differ.numel()} values differ"


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,H", [(1, 1), (32, 4096), (700, 1000), (900, 1422), (300, 1001), (5, 128)])
def test_quantize_values_are_the_rounded_quotients(dtype, T, H):
    g = gen(T + H)
    x = (randn(g, T, H) * torch.exp(0.7 * randn(g, H))).to(TYPES[dtype])
    q, sc = quantized(x)
    check_values(q, plain_values(x, sc))


@pytest.mark.parametrize("width", [384, 383, 382])
@pytest.mark.parametrize("e", [-149, -130, -118, -100, -80, -72, -40, 0, 60, 87, 89, 126])
def test_quantize_values_over_the_exponent_range(e, width):
    g = gen(e + 200)
    x = torch.ldexp(randn(g, 300, width).clamp(-3.9, 3.9).double(), torch.tensor(e, device="cuda")).clamp(-3.4e38, 3.4e38).float()
    q, sc = quantized(x)
    check_values(q, plain_values(x, sc))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,H", [(3000, 4096), (2200, 5000), (1500, 8200), (6000, 1536), (45000, 1024)])
@pytest.mark.parametrize("e", [0, -14])
def test_quantize_values_of_many_rows(dtype, T, H, e):
    """Rows enough for four chunks a lane (and, at 1536 columns, two), with groups
    of zeros, and a NaN and an infinity in groups of their own."""
    g = gen(T + H)
    x = torch.ldexp(randn(g, T, H), torch.tensor(e, device="cuda")).to(TYPES[dtype])
    x[T // 2, :256] = 0
    x[T - 1, H - 1], x[T - 2, 3] = math.nan, math.inf
    q, sc = quantized(x)
    plain = x.float()
    plain[T - 1, H - 1] = 0                                # (a NaN does not enter the maximum)
    assert torch.equal(sc, plain_scales(plain))
    assert q[T - 1, H - 1].float().isnan() and q[T - 2, 3].float().isnan() and int(q.float().isnan().sum()) == 2
    assert (q[T - 2, 4:128].float() == 0).all()
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[T - 2] = False
    plain[T - 2, 3] = 0
    q[T - 1, H - 1] = 0
    check_values(q[keep], plain_values(plain, sc)[keep])


def borders(seed, groups, e):
    """[groups, 128]: values on and up to two steps beside the borders between
    neighbouring e4m3 values (of each significand, below 2^-6 as well), times
    scales of any significand."""
    g = gen(seed)
    amax = torch.ldexp(1 + torch.rand(groups, generator=g, device="cuda", dtype=torch.float64), torch.tensor(e, device="cuda")).float()
    s = plain_scales(amax[:, None])
    odd = torch.arange(8, device="cuda")
    m = torch.cat([(17 + 2 * odd) / 16, (1 + 2 * odd) * 2.0 ** -10, (17 + 2 * odd) * 4.0])
    y = (m.double() * s.double()).float()
    out, lo, hi = [y], y, y
    for _ in range(2):
        lo, hi = torch.nextafter(lo, torch.full_like(lo, -math.inf)), torch.nextafter(hi, torch.full_like(hi, math.inf))
        out += [lo, hi]
    return torch.cat([*out, -y[:, :7], amax[:, None]], 1).contiguous()


@pytest.mark.parametrize("e", [-125, -110, -70, -1, 0, 87, 88, 100, 126])
def test_quantize_values_at_every_border(e):
    x = borders(e + 200, 40000, e)
    q, sc = quantized(x)
    check_values(q, plain_values(x, sc))


def test_norm_values_are_the_rounded_quotients():
    """Rows whose norm is exact (entries of magnitude 1, eps 0), with weights on
    the borders."""
    for width in (128, 2048):
        for seed in range(40):
            w = borders(seed, width // 128, -1).flatten()
            g = gen(seed)
            x = torch.where(torch.rand(9, width, generator=g, device="cuda") < 0.5, -1.0, 1.0)
            q, sc = torch.empty(9, width, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(9, width // 128, device="cuda")
            ob.orthrus_rmsnorm(x, w, 0.0, out_fp8=q, out_scale=sc)
            assert torch.equal(sc, plain_scales(x * w))
            check_values(q, plain_values(x * w, sc))


# ------------------------------------------------------------------- attention
def test_paged_attn_shapes_share_a_workspace():
    """Calls of different shapes and types through one workspace of the largest
    size, small ones before large ones and back: segments over many blocks, so
    that a counter that is not zero at its call shows as rows not written."""
    g = gen(61)
    shapes = [  # dtype, Hq, Hkv, D, page, lengths
        ("bf16", 8, 8, 128, 32, [20000]),
        ("bf16", 32, 8, 128, 16, [3000 + 37 * i for i in range(32)]),
        ("f16", 16, 2, 64, 8, [9000, 1, 0, 777]),
        ("bf16", 4, 1, 256, 64, [30000, 5]),
        ("bf16", 40, 2, 128, 16, [500 * i for i in range(20)]),
        ("f16", 6, 2, 64, 16, [i % 50 for i in range(700)]),
        ("bf16", 24, 8, 64, 128, [40000, 20000, 3])]
    calls = []
    for dtype, Hq, Hkv, D, page, lens in shapes:
        dt = TYPES[dtype]
        kp, vp, table = paged_cache(g, lens, page, Hkv, D, dt)
        q = randn(g, len(lens), Hq, D).to(dt)
        calls.append((q, kp, vp, table, lens, *paged_ref(q, kp, vp, table, lens)))
    size = max(ob.orthrus_paged_attn_workspace_size(q.shape[0], q.shape[1], kp.shape[1], q.shape[2]) for q, kp, *_ in calls)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for i in [0, 1, 0, 2, 1, 3, 4, 5, 0, 6, 5, 2, 4, 3, 1, 6]:
        q, kp, vp, table, lens, want, tol = calls[i]
        out = torch.full_like(q, math.nan)
        ob.orthrus_paged_attn(q, kp, vp, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), out, ws)
        close(out, want, tol, f"shape {i}")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_paged_attn_weights_keep_24_bits(dtype, D):
    """Two keys of weight 1 whose values cancel a third key's share p to about
    2^-18 of it (bf16; fp16 2^-24): what is left shows p's own bits.  Tolerance, in
    2^-24 p: exp2 to 2^-22 twice (4 + 4), its argument's rounding (at most 8 after
    fp16's offset of 7, and 2.9 for the factor log2 e, times ln 2: 7.5), eight fp32
    additions of at most p (8, truncated)."""
    dt = TYPES[dtype]
    k = torch.arange(64, 192, device="cuda") * -2.0 ** -7                         # -0.5 .. -1.5
    B = k.numel()
    p = k.double().exp()
    a1 = p.to(dt)
    a2 = (p - a1.double()).to(dt)
    kp, vp = (torch.zeros(B, 1, 4, D, dtype=dt, device="cuda") for _ in range(2))
    kp[:, 0, 2, 0] = k.to(dt)
    vp[:, 0, 0], vp[:, 0, 1], vp[:, 0, 2] = -a1[:, None], -a2[:, None], 1
    q = torch.zeros(B, 2, D, dtype=dt, device="cuda")
    q[..., 0] = 1
    out, st = run_paged(q, kp, vp, torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1), [3] * B, scale=1.0)
    want = (p - a1.double() - a2.double()) / (2 + p)
    tol = half_step(dt) * want.abs() + 24 * 2.0 ** -24 * p / (2 + p) + tiny(dt)
    close(out, want[:, None, None].expand_as(out), tol[:, None, None], "weights")
    assert st == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,lens", [(64, [40]), (128, [9, 5000]), (256, [300, 20000])])
def test_paged_attn_infinite_values(dtype, D, lens):
    """A visible key with weight and an infinite value: infinity in that place of
    the output, nothing elsewhere; both signs meet in a NaN."""
    dt, page, Hq = TYPES[dtype], 16, 4
    g = gen(D)
    P = sum(-(-n // page) for n in lens)
    table = torch.full((len(lens), -(-max(lens) // page)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        c = -(-n // page)
        table[b, :c] = torch.arange(at, at + c, dtype=torch.int32)
        at += c
    kp, vp = randn(g, P, 1, page, D).to(dt) / 8, randn(g, P, 1, page, D).to(dt)
    for b, n in enumerate(lens):
        for d, j, v in ((3, n // 2, math.inf), (5, n - 1, -math.inf), (7, 0, math.inf), (7, n - 1, -math.inf)):
            vp[int(table[b, j // page]), 0, j % page, d] = v
    q = randn(g, len(lens), Hq, D).to(dt)
    out, st = run_paged(q, kp, vp, table.cuda(), lens)
    assert (out[..., 3] == math.inf).all() and (out[..., 5] == -math.inf).all() and out[..., 7].isnan().all()
    rest = [d for d in range(D) if d not in (3, 5, 7)]
    assert out[..., rest].isfinite().all() and st == 0


# -------------------------------------------------------------------- rotation
@pytest.mark.parametrize("rot,D", [(64, 64), (128, 128), (10, 20), (6, 33)])
@pytest.mark.parametrize("layout", [ob.ROPE_HALF, ob.ROPE_INTERLEAVED])
def test_rope_sines_and_cosines_to_the_last_bits(rot, D, layout):
    """Pairs (1, 0) in fp32 come back as (cos, sin): within two steps for the
    function and half a step for the angle's last bits, at any position."""
    pos = torch.arange(0, 1 << 20, 97, dtype=torch.int32, device="cuda")
    turns = ob.orthrus_rope_table(rot, 1e4)[0].cuda()
    h = rot // 2
    ia = torch.arange(h, device="cuda") * (2 if layout == ob.ROPE_INTERLEAVED else 1)
    ib = ia + (1 if layout == ob.ROPE_INTERLEAVED else h)
    x = torch.zeros(pos.numel(), 1, D, device="cuda")
    x[..., ia] = 1
    out = torch.empty_like(x)
    ob.orthrus_rope(x, None, pos, turns, out, layout=layout)
    t = pos.double()[:, None] * turns
    ang = 2 * math.pi * (t - t.round())
    for at, want in ((ia, ang.cos()), (ib, ang.sin())):
        # (a step of fp32 is at most 2^-23 of the value; the angle's second order, 64 bits)
        close(out[:, 0, at], want, 2.5 * 2.0 ** -23 * want.abs() + 1e-13, "turn")


# --------------------------------------------------------------------- product
@pytest.mark.parametrize("M,N,K", [(256, 4608, 400), (129, 4609, 400), (256, 5120, 400), (512, 2304, 400), (513, 1536, 400),
                                   (1024, 1152, 144), (1025, 1152, 144), (1025, 700, 272),
                                   (9472, 128, 144), (9473, 128, 144)])
@pytest.mark.parametrize("out", list(TYPES))
def test_fp8_matmul_where_its_forms_meet(M, N, K, out):
    """Sizes on both sides of the change from the row form to the pairs."""
    g = gen(M + N + K)
    a, sa, w, sw = fp8_operands(g, M, N, K)
    o, ok = guard(M, N, dtype=TYPES[out])
    ob.orthrus_fp8_matmul(a, sa, w, sw, o)
    check_product(o, a, sa, w, sw)
    assert ok()


# ------------------------------------------------------- sums, streams, layers
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,H", [(300, 32767), (2, 32766), (301, 16384), (301, 9999), (40000, 3), (5, 32768)])
def test_rmsnorm_sums_of_the_widest_rows(dtype, T, H):
    """x + residual: one fp32 addition (exact for 16-bit values but for the last
    bits, 2^-24), rounded once."""
    dt, g = TYPES[dtype], gen(T + H)
    x, w, r = randn(g, T, H).to(dt), (1 + 0.3 * randn(g, H)).to(dt), randn(g, T, H).to(dt)
    out = torch.empty_like(x)
    so, ok = guard(T, H, dtype=dt)
    ob.orthrus_rmsnorm(x, w, 1e-5, out=out, residual=r, sum_out=so)
    s = x.double() + r.double()
    close(so, s, (half_step(dt) + 2.0 ** -23) * s.abs() + tiny(dt), "sum")
    assert ok()


def test_operators_of_two_streams_at_once():
    """A norm to 8 bits, a product of each form, a rotation and attention on each of
    two streams, interleaved: bitwise what they give alone."""
    g = gen(89)
    turns = ob.orthrus_rope_table(128, 1e6)[0].cuda()
    jobs = []
    for T, M, N in ((700, 600, 1536), (33, 20, 3000)):
        K, B, Hq, Hkv, D = 512, 5, 8, 2, 128
        a, sa, w, sw = fp8_operands(g, M, N, K)
        x, wn, r = randn(g, T, 1536).bfloat16(), randn(g, 1536).bfloat16(), randn(g, T, 1536).bfloat16()
        q, pos = randn(g, T, Hq, D).bfloat16(), torch.arange(T, dtype=torch.int32, device="cuda")
        lens = [3000, 17, 0, 400, 9001]
        kp, vp, table = paged_cache(g, lens, 16, Hkv, D, torch.bfloat16)
        aq, ctx = randn(g, B, Hq, D).bfloat16(), torch.tensor(lens, dtype=torch.int32, device="cuda")
        ws = torch.zeros(ob.orthrus_paged_attn_workspace_size(B, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
        outs = [torch.empty_like(x), torch.empty_like(x, dtype=torch.float8_e4m3fn), torch.empty(T, 12, device="cuda"),
                torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty_like(q), torch.empty_like(aq)]

        def run(stream, a=a, sa=sa, w=w, sw=sw, x=x, wn=wn, r=r, q=q, pos=pos, kp=kp, vp=vp, table=table, aq=aq, ctx=ctx,
                ws=ws, outs=outs):
            so, q8, s8, o, qo, ao = outs
            ob.orthrus_rmsnorm(x, wn, 1e-6, residual=r, sum_out=so, out_fp8=q8, out_scale=s8, stream=stream)
            ob.orthrus_fp8_matmul(a, sa, w, sw, o, stream=stream)
            ob.orthrus_rope(q, None, pos, turns, qo, stream=stream)
            ob.orthrus_paged_attn(aq, kp, vp, table, ctx, ao, ws, stream=stream)

        run(None)
        torch.cuda.synchronize()
        jobs.append((run, outs, [t.clone() for t in outs]))
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    for run, outs, _ in jobs:
        for t in outs:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(30):
        for (run, _, _), side in zip(jobs, sides):
            run(side)
    torch.cuda.synchronize()
    for _, outs, want in jobs:
        assert all(torch.equal(t.view(torch.uint8), w.view(torch.uint8)) for t, w in zip(outs, want))
