"""GPU parity of the layer operators against plain 64-bit evaluations.

Tolerances, per output value (h = half a step of the output type, relative):
  RMS norm   h|y| + 2^-18 |y|: the sum of squares is at most ~80 fp32 additions
             deep (2^-17.6 relative, halved by the root), a few roundings more.
  8-bit      scale: 2^-17 relative (the norm's error twice over); value: half an
             e4m3 step of the quotient (2^-4 relative, 2^-10 below the smallest
             normal number) plus 2^-17 of it.
  product    h|y| + (128 + blocks + 8) 2^-23 sum |sa sw a w|: fp32 sums of 128
             exact products in any order, then one per block.
  rotation   h|y| + 2^-19 m (|a| + |b|): the angle's fp32 fraction (2^-24 of half
             a turn: 2^-22.3 radians), sine and cosine to 2 ulp, the norm's 2^-18
             where there is one.
  attention  h|y| + (2^-15 + 2 d + (n / 64 + 64) 2^-23) sum_j p_j |v_j|: two 16-bit
             terms per weight (2^-17), exp2 to 2^-22, d = (D + 8) 2^-23 scale
             max_j sum |q k| the scores' error, fp32 additions n / 64 strips deep.
"""
import math
import os
import subprocess
import sys

import pytest
import torch

from lossless_diffusion_speculative_b200 import binding as ob

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def half_step(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    """Half the spacing of the type's subnormal numbers."""
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def close(got, want, tol, what):
    got, want = got.double(), want.double()
    assert got.shape == want.shape
    bad = torch.isnan(got) != torch.isnan(want)
    assert not bad.any(), f"{what}: {int(bad.sum())} NaNs differ"
    err = (got - want).abs()
    over = ~torch.isnan(want) & ~(err <= tol) & ~(got == want)
    assert not over.any(), f"{what}: {int(over.sum())} of {over.numel()} over, worst {float((err - tol)[over].max()):.3e}"


def guard(*shape, dtype, rows=2):
    """A buffer with `rows` canary rows behind the last one, and the check that they are untouched."""
    full = torch.full((shape[0] + rows, *shape[1:]), 77.0, device="cuda").to(dtype)
    return full[:shape[0]], lambda: bool((full[shape[0]:].float() == full[-1].float().flatten()[0]).all())


# ----------------------------------------------------------------------- norm
def norm_ref(x, r, w, eps):
    s = x.double() + (0 if r is None else r.double())
    return s, s / (s.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()


def check_fp8(q, scale, y, what):
    T, H = y.shape
    n = (H + 127) // 128
    amax = torch.stack([y[:, i * 128:(i + 1) * 128].abs().amax(1) for i in range(n)], 1)
    want = (amax / 448).clamp_min(2.0 ** -126)
    close(scale, want, 2.0 ** -17 * want, what + " scale")
    quot = y / scale.double().repeat_interleave(128, 1)[:, :H]
    tol = torch.maximum(2.0 ** -4 * quot.abs(), torch.full_like(quot, 2.0 ** -10)) + 2.0 ** -17 * quot.abs()
    close(q.float(), quot.clamp(-448, 448), tol, what + " value")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,H", [(1, 1), (1, 64), (3, 128), (5, 1000), (2, 4099), (300, 2048), (700, 520), (7, 12288),
                                 (301, 8200), (1, 32768)])
@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm(dtype, T, H, residual):
    dt, g = TYPES[dtype], gen(T * 31 + H)
    x, w = (3 * randn(g, T, H)).to(dt), (1 + 0.3 * randn(g, H)).to(dt)
    r = randn(g, T, H).to(dt) if residual else None
    out, ok1 = guard(T, H, dtype=dt)
    q, ok2 = guard(T, H, dtype=torch.float8_e4m3fn)
    sc, ok3 = guard(T, (H + 127) // 128, dtype=torch.float32)
    so, ok4 = guard(T, H, dtype=dt)
    ob.orthrus_rmsnorm(x, w, 1e-5, out=out, residual=r, sum_out=so if residual else None, out_fp8=q, out_scale=sc)
    s, y = norm_ref(x, r, w, 1e-5)
    close(out, y, (half_step(dt) + 2.0 ** -18) * y.abs() + tiny(dt), "norm")
    check_fp8(q, sc, y, "norm")
    if residual:
        close(so, s, (half_step(dt) + 2.0 ** -23) * s.abs() + tiny(dt), "sum")
    assert ok1() and ok2() and ok3() and ok4()


def test_rmsnorm_strided_rows_misaligned_and_in_place():
    g = gen(3)
    wide = randn(g, 40, 3 * 256).bfloat16()
    w = randn(g, 256).bfloat16()
    for x in (wide[:, 256:512], wide[:, 3:259], wide[::2, :256]):
        out = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda")
        ob.orthrus_rmsnorm(x, w, 1e-6, out=out)
        _, y = norm_ref(x, None, w, 1e-6)
        close(out, y, (2.0 ** -8 + 2.0 ** -18) * y.abs() + tiny(torch.bfloat16), "strided")
    x, r = randn(g, 40, 256).bfloat16(), randn(g, 40, 256).bfloat16()
    s, y = norm_ref(x, r, w, 1e-6)
    ob.orthrus_rmsnorm(x, w, 1e-6, out=x, residual=r, sum_out=r)            # both inputs overwritten
    close(r, s, 2.0 ** -8 * s.abs() + 2.0 ** -23 * s.abs(), "sum in place")
    close(x, y, (2.0 ** -8 + 2.0 ** -18) * y.abs() + tiny(torch.bfloat16), "norm in place")


def test_rmsnorm_zero_rows_and_non_finite_values():
    g = gen(4)
    x = randn(g, 4, 300)
    x[0] = 0
    x[1, 5] = math.nan
    x[2, 200] = math.inf
    w = torch.ones(300, device="cuda")
    out, q = torch.empty_like(x), torch.empty(4, 300, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(4, 3, device="cuda")
    ob.orthrus_rmsnorm(x, w, 1e-6, out=out, out_fp8=q, out_scale=sc)
    assert (out[0] == 0).all() and (q[0].float() == 0).all() and (sc[0] == 2.0 ** -126).all()
    assert out[1].isnan().all() and q[1].float().isnan().all()
    assert out[2, 200].isnan() and (out[2, :200] == 0).all()                # inf * 0; finite / inf
    assert out[3].isfinite().all() and q[3].float().isfinite().all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,H", [(1, 1), (32, 4096), (5, 1001), (1000, 640), (3, 40000), (400, 136)])
def test_quantize(dtype, T, H):
    dt, g = TYPES[dtype], gen(T + H)
    x = (randn(g, T, H) * torch.exp(2 * randn(g, H))).to(dt)
    x[0, :min(H, 128)] = 0
    q, ok1 = guard(T, H, dtype=torch.float8_e4m3fn)
    sc, ok2 = guard(T, (H + 127) // 128, dtype=torch.float32)
    ob.orthrus_quantize_fp8(x, q, sc)
    check_fp8(q, sc, x.double(), "quantize")
    assert ok1() and ok2()


def test_quantize_strided_nan_and_saturation():
    g = gen(9)
    wide = randn(g, 6, 512)
    x = wide[:, 100:356]
    x[1, 3] = math.nan
    x[2, 7] = math.inf
    x[3] = 1e-42                                                            # subnormal: the scale's floor
    q, sc = torch.empty(6, 256, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(6, 2, device="cuda")
    ob.orthrus_quantize_fp8(x, q, sc)
    f = q.float()
    assert f[1, 3].isnan() and int(f.isnan().sum()) == 2 and f[2, 7].isnan()
    assert (f[2, :7] == 0).all() and sc[2, 0] == math.inf
    assert (sc[3] == 2.0 ** -126).all() and f[3].isfinite().all()
    keep = torch.tensor([0, 4, 5], device="cuda")
    check_fp8(q[keep], sc[keep], x[keep].double(), "strided")


# -------------------------------------------------------------------- product
def fp8_operands(g, M, N, K):
    def q(rows, cols):
        return (randn(g, rows, cols) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    nk = (K + 127) // 128
    sa = torch.exp(randn(g, M, nk)) / 100
    sw = torch.exp(randn(g, (N + 127) // 128, nk)) / 100
    return q(M, K), sa, q(N, K), sw


def product_ref(a, sa, w, sw):
    N, K = w.shape
    A = a.double() * sa.double().repeat_interleave(128, 1)[:, :K]
    W = w.double() * sw.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return A @ W.t(), A.abs() @ W.abs().t()


def check_product(out, a, sa, w, sw, what="product"):
    want, mag = product_ref(a, sa, w, sw)
    n = 128 + sa.shape[1] + 8
    close(out, want, half_step(out.dtype) * want.abs() + n * 2.0 ** -23 * mag + tiny(out.dtype), what)


@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (1, 128, 128), (4, 1000, 272), (5, 1, 4096), (16, 300, 1040),
                                   (17, 6144, 512), (32, 6144, 4096), (33, 257, 640), (64, 512, 2560), (77, 130, 144),
                                   (128, 1024, 1024), (129, 384, 128), (200, 500, 4096), (300, 2049, 912),
                                   (1000, 1536, 256), (257, 7, 48)])
@pytest.mark.parametrize("out", list(TYPES))
def test_fp8_matmul(M, N, K, out):
    g = gen(M + 3 * N + 7 * K)
    a, sa, w, sw = fp8_operands(g, M, N, K)
    o, ok = guard(M, N, dtype=TYPES[out])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ob.orthrus_fp8_matmul(a, sa, w, sw, o, status=st)
    check_product(o, a, sa, w, sw)
    assert ok() and int(st) == 0


def test_fp8_matmul_persistent_sizes_and_repeats():
    """Many tiles per SM on both forms, bitwise the same twice, and with an
    output that is only element-aligned."""
    for M, N, K in ((3, 40000, 256), (700, 20000, 384)):
        g = gen(M)
        a, sa, w, sw = fp8_operands(g, M, N, K)
        store = torch.empty(M * N + 1, dtype=torch.bfloat16, device="cuda")
        o1, o2 = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), store[1:].view(M, N)
        ob.orthrus_fp8_matmul(a, sa, w, sw, o1)
        ob.orthrus_fp8_matmul(a, sa, w, sw, o2)
        check_product(o1, a, sa, w, sw)
        assert torch.equal(o1, o2)


def test_fp8_matmul_nan_stays_in_its_row_and_column():
    g = gen(5)
    for M in (9, 150):
        a, sa, w, sw = fp8_operands(g, M, 260, 256)
        a[3, 17] = math.nan
        sw[2, 1] = math.inf
        o = torch.empty(M, 260, device="cuda")
        ob.orthrus_fp8_matmul(a, sa, w, sw, o)
        assert o[3].isnan().all()
        rest = torch.cat((o[:3], o[4:]))
        assert rest[:, :256].isfinite().all() and not rest[:, 256:].isfinite().any()


# -------------------------------------------------------------------- rotation
def rope_ref(x, pos, turns, rot, layout, mag, w=None, eps=1e-6):
    """x [T,H,D], pos [T] -> (rotated in 64 bits, magnitude of the terms)."""
    y = x.double()
    if w is not None:
        y = y / (y.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    h = rot // 2
    ia = torch.arange(h, device="cuda") * (2 if layout == ob.ROPE_INTERLEAVED else 1)
    ib = ia + (1 if layout == ob.ROPE_INTERLEAVED else h)
    t = pos.double()[:, None] * turns
    ang = 2 * math.pi * (t - t.round())
    c, s = (mag * ang.cos())[:, None], (mag * ang.sin())[:, None]
    a, b = y[..., ia], y[..., ib]
    out, size = y.clone(), y.abs()
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = mag * (a.abs() + b.abs())
    return out, size


def check_rope(got, x, pos, turns, rot, layout, mag, w, what):
    want, size = rope_ref(x, pos, turns, rot, layout, mag, w)
    dt = got.dtype
    close(got, want, half_step(dt) * want.abs() + (2.0 ** -19 + (2.0 ** -18 if w is not None else 0)) * size + tiny(dt), what)


ROPE = [  # T, Hq, Hkv, D, rot
    (1, 32, 8, 128, 128), (5, 4, 4, 64, 64), (3, 5, 1, 256, 128), (70, 8, 2, 128, 32), (2, 3, 3, 96, 48),
    (900, 2, 1, 64, 16), (7, 4, 2, 20, 10), (3, 2, 1, 33, 6), (4, 2, 2, 16, 16), (2, 2, 1, 256, 256), (3, 2, 1, 2, 2)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("layout", [ob.ROPE_HALF, ob.ROPE_INTERLEAVED])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot", ROPE)
@pytest.mark.parametrize("norm", [False, True])
def test_rope(dtype, layout, T, Hq, Hkv, D, rot, norm):
    dt, g = TYPES[dtype], gen(T + D + rot)
    packed = randn(g, T, Hq + 2 * Hkv, D).to(dt)
    q, k = packed[:, :Hq], packed[:, Hq:Hq + Hkv]
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda").int()
    pos[0] = 0
    turns, mag = ob.orthrus_rope_table(rot, 1e6, ob.ROPE_YARN, factor=4.0, orig_len=32768.0)
    turns = turns.cuda()
    qn, kn = ((1 + 0.2 * randn(g, D)).to(dt) if norm else None for _ in range(2))
    qo, ok1 = guard(T, Hq, D, dtype=dt)
    ko, ok2 = guard(T, Hkv, D, dtype=dt)
    ob.orthrus_rope(q, k, pos, turns, qo, ko, layout=layout, magnitude=mag, q_norm=qn, k_norm=kn)
    check_rope(qo, q, pos, turns, rot, layout, mag, qn, "q")
    check_rope(ko, k, pos, turns, rot, layout, mag, kn, "k")
    before = packed.clone()
    ob.orthrus_rope(q, k, pos, turns, q, k, layout=layout, magnitude=mag, q_norm=qn, k_norm=kn)   # in place
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(packed[:, Hq + Hkv:], before[:, Hq + Hkv:])
    assert ok1() and ok2()


def test_rope_without_keys_one_norm_and_head_major_tensors():
    g = gen(8)
    turns, _ = ob.orthrus_rope_table(64, 1e4)
    turns = turns.cuda()
    q = randn(g, 6, 50, 64).bfloat16().transpose(0, 1)                       # [T, H, D] stored head-major
    k = randn(g, 50, 3, 64).bfloat16()
    pos = torch.arange(100, 150, device="cuda", dtype=torch.int32)
    qo, ko = torch.empty(6, 50, 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1), torch.empty_like(k)
    ob.orthrus_rope(q, None, pos, turns, qo)
    check_rope(qo, q, pos, turns, 64, ob.ROPE_HALF, 1.0, None, "q alone")
    kn = randn(g, 64).bfloat16()
    ob.orthrus_rope(q, k, pos, turns, qo, ko, k_norm=kn)
    check_rope(qo, q, pos, turns, 64, ob.ROPE_HALF, 1.0, None, "q, keys normed")
    check_rope(ko, k, pos, turns, 64, ob.ROPE_HALF, 1.0, kn, "k normed")


def paged_cache(g, lens, page, Hkv, D, dt, spare=2):
    need = [-(-n // page) for n in lens]
    P = sum(need) + spare
    order = torch.randperm(P, generator=g, device="cuda").tolist()
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    k, v = (randn(g, P, Hkv, page, D).to(dt) for _ in range(2))
    return k, v, table.cuda()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("B,K,Hq,Hkv,D,rot,page,ctx", [
    (3, 1, 8, 2, 128, 128, 16, [0, 15, 16]), (2, 5, 4, 4, 64, 32, 3, [1, 40]), (1, 32, 32, 8, 128, 128, 64, [100]),
    (4, 2, 2, 1, 20, 10, 7, [0, 6, 13, 50]), (200, 3, 2, 2, 64, 64, 8, list(range(200)))])
def test_rope_append(dtype, B, K, Hq, Hkv, D, rot, page, ctx):
    dt, g = TYPES[dtype], gen(B + K + D)
    packed = randn(g, B, K, Hq + 2 * Hkv, D).to(dt)
    q, k, v = packed[:, :, :Hq], packed[:, :, Hq:Hq + Hkv], packed[:, :, Hq + Hkv:]
    turns, mag = ob.orthrus_rope_table(rot, 1e6, ob.ROPE_LINEAR, factor=2.0)
    turns = turns.cuda()
    kn = (1 + 0.2 * randn(g, D)).to(dt)
    kp, vp, table = paged_cache(g, [c + K for c in ctx], page, Hkv, D, dt)
    k0, v0 = kp.clone(), vp.clone()
    qo = torch.empty(B, K, Hq, D, dtype=dt, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    ob.orthrus_rope_append(q, k, v, turns, qo, kp, vp, table, c, magnitude=mag, k_norm=kn, status=st)
    pos = (c[:, None] + torch.arange(K, device="cuda")).flatten()
    check_rope(qo.view(B * K, Hq, D), q.reshape(B * K, Hq, D), pos, turns, rot, 0, mag, None, "q")
    page_of = table.gather(1, (pos.view(B, K) // page).long()).flatten().long()
    row = (pos % page).long()
    check_rope(kp[page_of, :, row], k.reshape(B * K, Hkv, D), pos, turns, rot, 0, mag, kn, "k rows")
    assert torch.equal(vp[page_of, :, row], v.reshape(B * K, Hkv, D))
    written = torch.zeros(kp.shape[0], page, dtype=torch.bool, device="cuda")
    written[page_of, row] = True
    rest = (~written)[:, None].expand(-1, Hkv, -1)
    assert torch.equal(kp[rest], k0[rest]) and torch.equal(vp[rest], v0[rest]) and int(st) == 0
    # the same keys put into their rows first, then turned in place
    k0[page_of, :, row] = k.reshape(B * K, Hkv, D)
    ob.orthrus_rope_append(None, None, None, turns, None, k0, None, table, c, magnitude=mag, k_norm=kn, K=K, status=st)
    assert torch.equal(k0, kp) and int(st) == 0


def test_rope_append_contiguous_cache_after_qkv_project():
    """The block's projection into the contiguous cache, then its rotation
    there: page_size = S_max, block_table[b] = b."""
    B, K, Hq, Hkv, D, hid, S = 2, 8, 8, 2, 128, 256, 96
    g = gen(21)
    bf = torch.bfloat16
    x = randn(g, B, K, hid).to(bf)
    ws = [(randn(g, n * D, hid) / 16).to(bf) for n in (Hq, Hkv, Hkv)]
    kc, vc = torch.zeros(B, Hkv, S, D, dtype=bf, device="cuda"), torch.zeros(B, Hkv, S, D, dtype=bf, device="cuda")
    ctx = torch.tensor([5, 88], dtype=torch.int32, device="cuda")
    q = torch.empty(B, K, Hq, D, dtype=bf, device="cuda")
    work = torch.zeros(ob.orthrus_qkv_workspace_size(B, K, hid, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    ob.orthrus_qkv_project(x, *ws, ctx, q, kc, vc, work)
    raw_q, raw_k, raw_v = q.clone(), kc.clone(), vc.clone()
    turns = ob.orthrus_rope_table(D, 1e6)[0].cuda()
    table = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1)
    ob.orthrus_rope_append(q, None, None, turns, q, kc, None, table, ctx)
    for b in range(B):
        c = int(ctx[b])
        pos = torch.arange(c, c + K, device="cuda")
        check_rope(q[b], raw_q[b], pos, turns, D, 0, 1.0, None, "q")
        check_rope(kc[b, :, c:c + K].transpose(0, 1), raw_k[b, :, c:c + K].transpose(0, 1), pos, turns, D, 0, 1.0, None, "k")
        raw_k[b, :, c:c + K] = kc[b, :, c:c + K]
    assert torch.equal(kc, raw_k) and torch.equal(vc, raw_v)


@pytest.mark.parametrize("D", [128, 20])
def test_rope_append_reports_and_skips_what_has_no_row(D):
    B, K, Hkv, page = 4, 2, 2, 4
    g = gen(6)
    k, v, q = (randn(g, B, K, Hkv, D) for _ in range(3))
    kp, vp = randn(g, 6, Hkv, page, D), randn(g, 6, Hkv, page, D)
    table = torch.tensor([[0, 1], [2, 3], [4, 99], [-1, 5]], dtype=torch.int32, device="cuda")
    k0, v0 = kp.clone(), vp.clone()
    turns = ob.orthrus_rope_table(D - D % 4, 1e4)[0].cuda()
    qo = torch.full_like(q, math.nan)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ob.orthrus_rope_append(q, k, v, turns, qo, kp, vp, table,
                           torch.tensor([7, -1, 1, 4], dtype=torch.int32, device="cuda"), status=st)
    assert int(st) == ob.STATUS_CAPACITY                                     # sequences 0 and 1; 2 and 3 are fine
    assert torch.equal(vp[4, :, 1:3], v[2].transpose(0, 1)) and torch.equal(vp[5, :, 0:2], v[3].transpose(0, 1))
    same = torch.tensor([0, 1, 2, 3], device="cuda")
    assert torch.equal(kp[same], k0[same]) and torch.equal(vp[same], v0[same]) and qo.isfinite().all()
    st.zero_()
    kp.copy_(k0), vp.copy_(v0)
    ob.orthrus_rope_append(q, k, v, turns, qo, kp, vp, table,
                           torch.tensor([0, 0, 3, 3], dtype=torch.int32, device="cuda"), status=st)
    assert int(st) == ob.STATUS_PAGE                                         # entries 99 and -1
    assert torch.equal(vp[4, :, 3], v[2, 0]) and torch.equal(vp[5, :, 0], v[3, 1])
    assert torch.equal(vp[4, :, :3], v0[4, :, :3]) and torch.equal(vp[5, :, 1:], v0[5, :, 1:])


# ------------------------------------------------------------------- attention
def paged_ref(q, kp, vp, table, lens, scale=None, drop=()):
    """Outputs and tolerance of single-token attention, in 64 bits."""
    B, Hq, D = q.shape
    Hkv, page = kp.shape[1:3]
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    tol = torch.full_like(out, tiny(q.dtype))
    for b, n in enumerate(lens):
        keys = [j for j in range(n) if (b, j // page) not in drop]
        if not keys:
            continue
        if len(keys) == n:
            at = table[b, :-(-n // page)].long()
            k, v = (t[at].transpose(0, 1).flatten(1, 2)[:, :n].double() for t in (kp, vp))
        else:
            j = torch.tensor(keys, device="cuda")
            k, v = (t[table[b, j // page].long(), :, j % page].transpose(0, 1).double() for t in (kp, vp))
        qq = q[b].double().view(Hkv, G, D)
        p = torch.softmax(torch.einsum("hgd,hnd->hgn", qq, k) * scale, -1)
        d = (D + 8) * 2.0 ** -23 * scale * torch.einsum("hgd,hnd->hgn", qq.abs(), k.abs()).amax(-1, keepdim=True)
        o = (p @ v).flatten(0, 1)
        mag = ((2.0 ** -15 + 2 * d + (n / 64 + 64) * 2.0 ** -23) * (p @ v.abs())).flatten(0, 1)
        out[b] = o
        tol[b] += half_step(q.dtype) * o.abs() + mag
    return out, tol


def run_paged(q, kp, vp, table, lens, ws=None, n_new=0, scale=0.0):
    B, Hq, D = q.shape
    out, ok = guard(B, Hq, D, dtype=q.dtype)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    if ws is None:
        ws = torch.zeros(ob.orthrus_paged_attn_workspace_size(B, Hq, kp.shape[1], D), dtype=torch.uint8, device="cuda")
    c = torch.tensor([n - n_new for n in lens], dtype=torch.int32, device="cuda")
    ob.orthrus_paged_attn(q, kp, vp, table, c, out, ws, n_new=n_new, scale=scale, status=st)
    segments = B * kp.shape[1] * (-(-(Hq // kp.shape[1]) // 16))
    assert int(ws[:4 * segments].count_nonzero()) == 0 and ok()              # the counters
    return out, int(st)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (16, 8, 128), (8, 8, 64), (5, 1, 64), (16, 1, 128), (40, 2, 128),
                                      (4, 2, 256), (48, 1, 256), (3, 3, 128)])
@pytest.mark.parametrize("page,lens", [
    (16, [300]), (1, [1, 70]), (64, [0, 1, 16, 17, 63, 64, 65, 1000]), (24, [2500, 3, 0, 777]), (7, [5000])])
def test_paged_attn(dtype, Hq, Hkv, D, page, lens):
    dt, g = TYPES[dtype], gen(Hq + D + page)
    kp, vp, table = paged_cache(g, lens, page, Hkv, D, dt)
    q = randn(g, len(lens), Hq, D).to(dt)
    out, st = run_paged(q, kp, vp, table, lens)
    want, tol = paged_ref(q, kp, vp, table, lens)
    close(out, want, tol, "paged")
    assert st == 0


def test_paged_attn_many_sequences_one_workspace_and_poisoned_rows():
    """Ragged batches of two shapes' calls through one workspace; every row that
    no position names holds NaN or infinity."""
    g = gen(12)
    B, Hq, Hkv, D, page = 300, 8, 2, 128, 16
    ws = torch.zeros(ob.orthrus_paged_attn_workspace_size(B, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    for top in (40, 900, 3):
        lens = torch.randint(0, top, (B,), generator=g, device="cuda").tolist()
        kp, vp, table = paged_cache(g, lens, page, Hkv, D, torch.bfloat16)
        seen = torch.zeros(kp.shape[0], page, dtype=torch.bool, device="cuda")
        for b, n in enumerate(lens):
            for e in range(-(-n // page)):
                seen[int(table[b, e]), :min(page, n - e * page)] = True
        hide = (~seen)[:, None].expand(-1, Hkv, -1)
        kp[hide], vp[hide] = math.nan, math.inf
        q = randn(g, B, Hq, D).bfloat16()
        out, st = run_paged(q, kp, vp, table, lens, ws=ws)
        kp[hide], vp[hide] = 0, 0
        want, tol = paged_ref(q, kp, vp, table, lens)
        close(out, want, tol, f"ragged {top}")
        again, _ = run_paged(q, kp, vp, table, lens, ws=ws)
        assert st == 0 and torch.equal(out, again)


def test_paged_attn_long_and_peaked():
    """A long sequence with one dominant key far in, large scores, a caller's
    scale, and n_new; the maximum then moves by much inside the stream."""
    g = gen(13)
    Hq, Hkv, D, page, n = 8, 2, 128, 32, 40001
    kp, vp, table = paged_cache(g, [n], page, Hkv, D, torch.bfloat16)
    q = randn(g, 1, Hq, D).bfloat16()
    j = 33333
    kp[int(table[0, j // page]), :, j % page] = (3 * q[0].view(Hkv, Hq // Hkv, D)[:, 0])
    for scale in (0.05, 1.0):
        out, st = run_paged(q, kp, vp, table, [n], n_new=1, scale=scale)
        want, tol = paged_ref(q, kp, vp, table, [n], scale=scale)
        close(out, want, tol, f"scale {scale}")
        assert st == 0


def test_paged_attn_masked_by_lowest_values():
    """Keys that score the type's lowest finite value, or -inf, beside ordinary
    ones: they get no weight; a row whose every score is -inf gives zeros."""
    g = gen(14)
    kp, vp, table = paged_cache(g, [130, 70], 16, 1, 64, torch.bfloat16)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    lens = [130, 70]
    for b, n in enumerate(lens):
        for j in range(n):
            pg, r = int(table[b, j // 16]), j % 16
            kp[pg, 0, r, 0] = (torch.finfo(torch.bfloat16).min if j % 3 else 0.5) if b == 0 else -math.inf
    out, st = run_paged(q, kp, vp, table, lens, scale=1.0)
    want, tol = paged_ref(q[:1], kp, vp, table[:1], lens[:1], scale=1.0)
    # (the scores' error bound is taken over the keys that get weight)
    ref_tol = half_step(torch.bfloat16) * want.abs() + 2.0 ** -13 * 8
    close(out[:1], want, ref_tol, "lowest values")
    assert (out[1] == 0).all() and st == 0


def test_paged_attn_reports_bad_lengths_and_pages():
    g = gen(15)
    lens = [40, 33, 20, 48]
    kp, vp, table = paged_cache(g, lens, 16, 2, 64, torch.float16)
    q = randn(g, 4, 4, 64).half()
    bad = table.clone()
    bad[1, 1], bad[3, 0], bad[2, 2] = 10_000, -5, 1 << 30                    # (2, 2) is past its length
    out, st = run_paged(q, kp, vp, bad, lens)
    want, tol = paged_ref(q, kp, vp, table, lens, drop={(1, 1), (3, 0)})
    close(out, want, tol, "dropped pages")
    assert st == ob.STATUS_PAGE
    out, st = run_paged(q, kp, vp, table, [40, -1, 20, 49])
    want, tol = paged_ref(q, kp, vp, table, [40, 0, 20, 0])
    close(out, want, tol, "bad lengths")
    assert st == ob.STATUS_CAPACITY and (out[1] == 0).all() and (out[3] == 0).all()
    with pytest.raises(ob.OrthrusError):
        ob.orthrus_paged_attn(q, kp, vp, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                              torch.empty_like(q), torch.zeros(64, dtype=torch.uint8, device="cuda"))


def test_paged_attn_pool_past_32_bit_offsets():
    """Pages whose element offsets pass 2^32."""
    Hkv, page, D = 8, 64, 128
    P = (1 << 32) // (Hkv * page * D) + 8
    kp = torch.empty(P, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    g = gen(16)
    table = torch.tensor([[P - 1, 0, P - 2]], dtype=torch.int32, device="cuda")
    for i in (P - 1, 0, P - 2):
        kp[i], vp[i] = randn(g, Hkv, page, D).bfloat16(), randn(g, Hkv, page, D).bfloat16()
    q = randn(g, 1, 16, D).bfloat16()
    out, _ = run_paged(q, kp, vp, table, [150])
    want, tol = paged_ref(q, kp, vp, table, [150])
    close(out, want, tol, "far pages")
    turns = ob.orthrus_rope_table(D, 1e4)[0].cuda()
    v = randn(g, 1, 1, Hkv, D).bfloat16()
    ob.orthrus_rope_append(None, v, v, turns, None, kp, vp, table, torch.tensor([150], dtype=torch.int32, device="cuda"))
    assert torch.equal(vp[P - 2, :, 150 - 128], v[0, 0])
    del kp, vp
    torch.cuda.empty_cache()


# ------------------------------------------------------------- a layer of them
class Layer:
    """norm -> 8-bit projection -> rotation and append -> paged attention -> 8-bit
    output projection -> norm with the residual: one new token per sequence."""

    def __init__(self, seed, B=3, hidden=512, Hq=8, Hkv=2, D=128, page=16, top=200):
        g = gen(seed)
        self.B, self.Hq, self.Hkv, self.D, self.hidden = B, Hq, Hkv, D, hidden
        bf = torch.bfloat16
        self.lens = [top, 0, 37][:B]
        self.x = randn(g, B, hidden).to(bf)
        self.w1, self.w2 = ((1 + 0.1 * randn(g, hidden)).to(bf) for _ in range(2))
        self.qn, self.kn = ((1 + 0.1 * randn(g, D)).to(bf) for _ in range(2))
        F = (Hq + 2 * Hkv) * D
        _, _, self.wqkv, self.sqkv = fp8_operands(g, 1, F, hidden)
        _, _, self.wo, self.so = fp8_operands(g, 1, hidden, Hq * D)
        self.sqkv, self.so = self.sqkv * 2e-2, self.so * 2e-2
        self.kp, self.vp, self.table = paged_cache(g, [n + 1 for n in self.lens], page, Hkv, D, bf)
        self.ctx = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.turns = ob.orthrus_rope_table(D, 1e6)[0].cuda()
        e8, f32 = torch.float8_e4m3fn, torch.float32
        new = lambda *s, dtype=bf: torch.empty(*s, dtype=dtype, device="cuda")
        self.q8, self.s8 = new(B, hidden, dtype=e8), new(B, hidden // 128, dtype=f32)
        self.qkv, self.q = new(B, F), new(B, 1, Hq, D)
        self.att, self.a8, self.as8 = new(B, Hq, D), new(B, Hq * D, dtype=e8), new(B, Hq * D // 128, dtype=f32)
        self.o, self.sum, self.y = new(B, hidden), new(B, hidden), new(B, hidden)
        self.ws = torch.zeros(ob.orthrus_paged_attn_workspace_size(B, Hq, Hkv, D), dtype=torch.uint8, device="cuda")

    def run(self):
        B, Hq, Hkv, D = self.B, self.Hq, self.Hkv, self.D
        ob.orthrus_rmsnorm(self.x, self.w1, 1e-6, out_fp8=self.q8, out_scale=self.s8)
        ob.orthrus_fp8_matmul(self.q8, self.s8, self.wqkv, self.sqkv, self.qkv)
        h = self.qkv.view(B, 1, Hq + 2 * Hkv, D)
        ob.orthrus_rope_append(h[:, :, :Hq], h[:, :, Hq:Hq + Hkv], h[:, :, Hq + Hkv:], self.turns, self.q, self.kp,
                               self.vp, self.table, self.ctx, q_norm=self.qn, k_norm=self.kn)
        ob.orthrus_paged_attn(self.q.view(B, Hq, D), self.kp, self.vp, self.table, self.ctx, self.att, self.ws, n_new=1)
        ob.orthrus_quantize_fp8(self.att.view(B, Hq * D), self.a8, self.as8)
        ob.orthrus_fp8_matmul(self.a8, self.as8, self.wo, self.so, self.o)
        ob.orthrus_rmsnorm(self.o, self.w2, 1e-6, out=self.y, residual=self.x, sum_out=self.sum)

    def check(self):
        """Every stage against its definition on the stage before's own output."""
        B, Hq, Hkv, D = self.B, self.Hq, self.Hkv, self.D
        _, y = norm_ref(self.x, None, self.w1, 1e-6)
        check_fp8(self.q8, self.s8, y, "layer norm")
        check_product(self.qkv, self.q8, self.s8, self.wqkv, self.sqkv, "layer qkv")
        h = self.qkv.view(B, Hq + 2 * Hkv, D)
        check_rope(self.q.view(B, Hq, D), h[:, :Hq], self.ctx, self.turns, D, 0, 1.0, self.qn, "layer q")
        want, tol = paged_ref(self.q.view(B, Hq, D), self.kp, self.vp, self.table, [n + 1 for n in self.lens])
        close(self.att, want, tol, "layer attention")
        check_fp8(self.a8, self.as8, self.att.view(B, Hq * D).double(), "layer quantise")
        check_product(self.o, self.a8, self.as8, self.wo, self.so, "layer output")
        s, y = norm_ref(self.o, self.x, self.w2, 1e-6)
        close(self.sum, s, (2.0 ** -8 + 2.0 ** -23) * s.abs(), "layer sum")
        close(self.y, y, (2.0 ** -8 + 2.0 ** -18) * y.abs() + tiny(torch.bfloat16), "layer norm 2")

    def outputs(self):
        return [t.clone() for t in (self.qkv, self.q, self.kp, self.vp, self.att, self.o, self.sum, self.y)]


def test_layer_of_operators():
    l = Layer(31)
    l.run()
    l.check()


def test_layer_captured_replayed_and_on_other_streams():
    """Two layers captured into two graphs, replayed after their inputs changed,
    alternately; two more run on two streams at once."""
    layers = [Layer(41), Layer(42, Hq=4, Hkv=4, top=500)]
    side = torch.cuda.Stream()
    graphs = []
    for l in layers:
        l.run()
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            l.run()
        graphs.append(gr)
    for l in layers:
        l.x.mul_(0.5).add_(0.25)
        l.ctx.copy_(torch.tensor([max(0, n - 1) for n in l.lens], dtype=torch.int32))
        l.lens = [max(0, n - 1) for n in l.lens]
    for _ in range(3):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    for l in layers:
        l.check()
    want = [l.outputs() for l in layers]
    main = torch.cuda.current_stream()
    side.wait_stream(main)
    for _ in range(20):
        layers[0].run()
        with torch.cuda.stream(side):
            layers[1].run()
    main.wait_stream(side)
    torch.cuda.synchronize()
    for l, w in zip(layers, want):
        assert all(torch.equal(a, b) for a, b in zip(l.outputs(), w))


@pytest.mark.parametrize("M,N,K", [(300, 2050, 256), (700, 2052, 384), (260, 4095, 128), (40, 1002, 640), (9, 1001, 512),
                                   (100, 50, 4096), (2, 20, 8192), (513, 1024, 144)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_fp8_matmul_row_alignments_and_splits(M, N, K, out):
    """Outputs whose rows allow stores of 16 bytes, of pairs or of single values,
    and shapes whose K is split over a cluster."""
    g = gen(M + N + K)
    a, sa, w, sw = fp8_operands(g, M, N, K)
    for shift in (0, 1, 2):
        store = torch.full((M * N + 8,), 77.0, dtype=TYPES[out], device="cuda")
        o = store[shift:shift + M * N].view(M, N)
        ob.orthrus_fp8_matmul(a, sa, w, sw, o)
        check_product(o, a, sa, w, sw, f"shift {shift}")
        assert (store[:shift] == 77).all() and (store[shift + M * N:] == 77).all()


@pytest.mark.parametrize("M,N,K", [(129, 257, 128), (300, 259, 64), (515, 385, 128), (200, 263, 128), (200, 510, 256),
                                   (1030, 1291, 64)])
@pytest.mark.parametrize("out", list(TYPES))
def test_fp8_matmul_short_runs_at_every_alignment(M, N, K, out):
    """Last tiles of a few columns, at each of the eight places of a row's start
    within 16 bytes."""
    g = gen(M + N + K)
    a, sa, w, sw = fp8_operands(g, M, N, K)
    for shift in range(8):
        store = torch.full((M * N + 8,), 77.0, dtype=TYPES[out], device="cuda")
        o = store[shift:shift + M * N].view(M, N)
        ob.orthrus_fp8_matmul(a, sa, w, sw, o)
        check_product(o, a, sa, w, sw, f"shift {shift}")
        assert (store[:shift] == 77).all() and (store[shift + M * N:] == 77).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,H", [(4, 70), (600, 1422), (33, 9002), (1, 130)])
def test_rmsnorm_and_quantize_even_widths(dtype, T, H):
    """Rows aligned for pairs only."""
    dt, g = TYPES[dtype], gen(T + H)
    x, w, r = randn(g, T, H).to(dt), (1 + 0.3 * randn(g, H)).to(dt), randn(g, T, H).to(dt)
    out, so = torch.empty_like(x), torch.empty_like(x)
    q, ok = guard(T, H, dtype=torch.float8_e4m3fn)
    sc = torch.empty(T, (H + 127) // 128, device="cuda")
    ob.orthrus_rmsnorm(x, w, 1e-5, out=out, residual=r, sum_out=so, out_fp8=q, out_scale=sc)
    s, y = norm_ref(x, r, w, 1e-5)
    close(so, s, (half_step(dt) + 2.0 ** -23) * s.abs() + tiny(dt), "sum")
    close(out, y, (half_step(dt) + 2.0 ** -18) * y.abs() + tiny(dt), "norm")
    check_fp8(q, sc, y, "norm")
    ob.orthrus_quantize_fp8(x, q, sc)
    check_fp8(q, sc, x.double(), "quantize")
    assert ok()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("B,n", [(1, 700), (1, 60001), (296, 60001)])
@pytest.mark.parametrize("top", [8.0, 12.5, 14.0])
def test_paged_attn_small_weights_beside_dominant_keys(dtype, B, n, top):
    """A few keys of weight 1 whose values are 0 among the first, the others of
    weight e^-top each with values of 1: the output is the small weights' share.
    The largest batch gives a block whole sequences, so that one running maximum
    covers them."""
    dt = TYPES[dtype]
    page, D = 64, 64
    P = -(-n // page)
    kp, vp = torch.zeros(P, 1, page, D, device="cuda", dtype=dt), torch.ones(P, 1, page, D, device="cuda", dtype=dt)
    table = torch.arange(P, dtype=torch.int32, device="cuda").view(1, P).repeat(B, 1)
    kp[:2, :, ::16, 0] = top
    vp[:2, :, ::16] = 0
    q = torch.zeros(B, 6, D, device="cuda", dtype=dt)
    q[:, :, 0] = 1
    out, st = run_paged(q, kp, vp, table, [n] * B, scale=1.0)
    want, tol = paged_ref(q[:1], kp, vp, table, [n], scale=1.0)
    close(out, want.expand(B, -1, -1), tol.expand(B, -1, -1), "shares")
    assert st == 0


@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (5, 1, 128), (12, 1, 64), (16, 1, 256), (9, 1, 128), (24, 1, 64)])
def test_paged_attn_joins_of_many_blocks(Hq, Hkv, D):
    """One and two sequences of one KV head, long enough that every block of the
    grid holds a part, and lengths around a block's share."""
    g = gen(Hq + D)
    for lens in ([20000], [30011, 9000], [64, 64, 64], [193, 193]):
        kp, vp, table = paged_cache(g, lens, 32, Hkv, D, torch.bfloat16)
        q = randn(g, len(lens), Hq, D).bfloat16()
        out, st = run_paged(q, kp, vp, table, lens)
        want, tol = paged_ref(q, kp, vp, table, lens)
        close(out, want, tol, f"{lens}")
        assert st == 0


def test_paged_attn_on_the_contiguous_cache_matches_the_block_attention():
    """page_size = S_max, block_table[b] = b: the same keys and values through
    orthrus_attn with a block of one token (AR view)."""
    g = gen(77)
    B, Hq, Hkv, D, S = 3, 32, 8, 128, 520
    kc, vc = randn(g, B, Hkv, S, D).bfloat16() / 11, randn(g, B, Hkv, S, D).bfloat16() / 11
    q = randn(g, B, 1, Hq, D).bfloat16()
    ctx = torch.tensor([500, 0, 77], dtype=torch.int32, device="cuda")
    ref = torch.empty(B, 1, Hq, D, device="cuda")
    ws = torch.zeros(ob.orthrus_attn_workspace_size(B, Hq, Hkv, D, 1), dtype=torch.uint8, device="cuda")
    ob.orthrus_attn(ob.AR, q, kc, vc, ctx, ref, ws)
    table = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1)
    out, st = run_paged(q.view(B, Hq, D), kc, vc, table, [501, 1, 78], n_new=1)
    # half a step of bf16, and the block attention's own bound (2e-3 of the output's rms)
    close(out, ref.view(B, Hq, D), 2.0 ** -8 * ref.view(B, Hq, D).double().abs() + 2e-3 * float(ref.pow(2).mean().sqrt()), "views")
    assert st == 0


def test_calls_on_two_streams_at_once():
    """Products of both forms, norms and rotations enqueued on two streams together."""
    g = gen(88)
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    jobs = []
    for M, N, K in ((600, 1536, 512), (20, 3000, 1024)):
        a, sa, w, sw = fp8_operands(g, M, N, K)
        outs = [torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        ob.orthrus_fp8_matmul(a, sa, w, sw, outs[0])
        jobs.append((a, sa, w, sw, outs))
    torch.cuda.synchronize()
    for _ in range(30):
        for job, st in zip(jobs, sides):
            a, sa, w, sw, outs = job
            ob.orthrus_fp8_matmul(a, sa, w, sw, outs[1], stream=st)
    torch.cuda.synchronize()
    for *_, outs in jobs:
        assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,H", [(300, 32767), (2, 32766), (700, 16384), (301, 9999), (40000, 3)])
def test_rmsnorm_widest_rows(dtype, T, H):
    """Rows of a whole block's warps on each path, and many of the narrowest."""
    dt, g = TYPES[dtype], gen(T + H)
    x, w, r = randn(g, T, H).to(dt), (1 + 0.3 * randn(g, H)).to(dt), randn(g, T, H).to(dt)
    out, ok1 = guard(T, H, dtype=dt)
    q, ok2 = guard(T, H, dtype=torch.float8_e4m3fn)
    sc, so = torch.empty(T, (H + 127) // 128, device="cuda"), torch.empty_like(x)
    ob.orthrus_rmsnorm(x, w, 1e-5, out=out, residual=r, sum_out=so, out_fp8=q, out_scale=sc)
    s, y = norm_ref(x, r, w, 1e-5)
    close(out, y, (half_step(dt) + 2.0 ** -18) * y.abs() + tiny(dt), "norm")
    check_fp8(q, sc, y, "norm")
    assert ok1() and ok2()


@pytest.mark.parametrize("M,N,K", [(70001, 17, 64), (9000, 1, 48), (1, 1, 16), (128, 3, 12288), (129, 1, 12288)])
@pytest.mark.parametrize("out", ["f16", "f32"])
def test_fp8_matmul_tall_and_thin(M, N, K, out):
    g = gen(M + N + K)
    a, sa, w, sw = fp8_operands(g, M, N, K)
    o, ok = guard(M, N, dtype=TYPES[out])
    ob.orthrus_fp8_matmul(a, sa, w, sw, o)
    check_product(o, a, sa, w, sw)
    assert ok()


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 2, 1), (256, 17, 1), (128, 6, 2)])
def test_paged_attn_largest_batch(D, Hq, Hkv):
    """As many sequences as one call takes, most of them short and some empty, over
    pages that several of them share."""
    g = gen(D)
    B, page, P = 4096, 8, 64
    lens = torch.randint(0, 30, (B,), generator=g, device="cuda")
    lens[17], lens[4000] = 500, 0
    table = torch.randint(0, P, (B, 63), generator=g, device="cuda").int()
    kp, vp = (randn(g, P, Hkv, page, D).bfloat16() for _ in range(2))
    q = randn(g, B, Hq, D).bfloat16()
    out, st = run_paged(q, kp, vp, table, lens.tolist())
    some = [0, 1, 16, 17, 18, 2047, 2048, 3999, 4000, 4001, 4095] + torch.randint(0, B, (60,), generator=g, device="cuda").tolist()
    want, tol = paged_ref(q[some], kp, vp, table[some], lens[some].tolist())
    close(out[some], want, tol, "largest batch")
    assert st == 0 and not out[lens == 0].any()


FIRST = """
import sys, torch
from lossless_diffusion_speculative_b200 import binding as ob
sys.path.insert(0, sys.argv[1])
import test_gpu_layer_ops as t
l = t.Layer(51)
M, N, K = 300, 520, 256
a, sa, w, sw = t.fp8_operands(t.gen(1), M, N, K)
o = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    l.run()
    ob.orthrus_fp8_matmul(a, sa, w, sw, o)
for _ in range(2):
    g.replay()
torch.cuda.synchronize()
l.check()
t.check_product(o, a, sa, w, sw)
print("captured first")
"""


def test_first_calls_of_a_process_inside_a_capture():
    """No call needs one outside a capture before it."""
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", FIRST, here], cwd=os.path.dirname(here), capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]
