"""Host side of the layer operators (RMS norm, 8-bit quantisation and matrix
product, rotary positions, paged attention): argument checks of the entry
points, before any device call; the frequency table against its formulas; the
binding's refusals."""
import ctypes
import math

import pytest
import torch

from lossless_diffusion_speculative_b200 import binding as ob
from lossless_diffusion_speculative_b200 import build

BF, F32, F16 = ob.BF16, ob.F32, ob.F16


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ob.lib()


def vp(a):
    return ctypes.c_void_p(a)


P = vp(4096)          # a well aligned address that no refused call may touch


def test_rmsnorm_refusals(lib):
    f = lib.orthrus_rmsnorm
    good = [BF, P, 64, None, P, 2, 64, 1e-6, None, P, None, None, None]

    def rc(**kw):
        names = ["dtype", "x", "xs", "res", "w", "T", "H", "eps", "sum", "out", "q", "qs", "st"]
        a = list(good)
        for k, v in kw.items():
            a[names.index(k)] = v
        return f(*a)

    assert rc(x=None) == rc(w=None) == rc(out=None) == ob.ERR_ARG
    assert rc(dtype=7) == rc(T=0) == rc(T=-1) == rc(H=0) == ob.ERR_ARG
    assert rc(eps=-1.0) == rc(eps=math.inf) == rc(eps=math.nan) == ob.ERR_ARG
    assert rc(res=P) == rc(sum=P) == ob.ERR_ARG                 # residual and sum_out go together
    assert rc(res=vp(8192), sum=P, out=P) == ob.ERR_ARG         # two outputs in one place
    assert rc(q=P) == rc(qs=P) == ob.ERR_ARG                    # values and scales go together
    assert rc(xs=63) == ob.ERR_ARG                              # rows overlap
    assert rc(xs=128, out=P, x=P) == ob.ERR_ARG                 # in place through another stride
    assert rc(H=ob_max_norm() + 1, xs=ob_max_norm() + 1) == ob.ERR_UNSUPPORTED
    assert rc(x=vp(4097)) == rc(w=vp(4097)) == rc(out=vp(4097)) == ob.ERR_ALIGN
    assert rc(q=P, qs=vp(4098)) == ob.ERR_ALIGN


def ob_max_norm():
    return 32768


def test_quantize_refusals(lib):
    f = lib.orthrus_quantize_fp8
    assert f(BF, None, 64, 2, 64, P, P, None) == ob.ERR_ARG
    assert f(BF, P, 64, 2, 64, None, P, None) == ob.ERR_ARG
    assert f(BF, P, 64, 2, 64, P, None, None) == ob.ERR_ARG
    assert f(9, P, 64, 2, 64, P, P, None) == ob.ERR_ARG
    assert f(BF, P, 63, 2, 64, P, P, None) == ob.ERR_ARG
    assert f(BF, P, 64, 0, 64, P, P, None) == f(BF, P, 64, 2, 0, P, P, None) == ob.ERR_ARG
    assert f(F32, vp(4098), 64, 2, 64, P, P, None) == ob.ERR_ALIGN
    assert f(BF, P, 64, 2, 64, P, vp(4097), None) == ob.ERR_ALIGN


def test_fp8_matmul_refusals(lib):
    f = lib.orthrus_fp8_matmul
    for i in (0, 1, 2, 3, 8):
        a = [P, P, P, P, 4, 64, 64, BF, P, None, None]
        a[i] = None
        assert f(*a) == ob.ERR_ARG, i
    for M, N, K in ((0, 64, 64), (4, 0, 64), (4, 64, 0), (-1, 64, 64)):
        assert f(P, P, P, P, M, N, K, BF, P, None, None) == ob.ERR_ARG
    assert f(P, P, P, P, 4, 64, 64, 5, P, None, None) == ob.ERR_ARG
    assert f(P, P, P, P, 4, 64, 72, BF, P, None, None) == ob.ERR_UNSUPPORTED
    assert f(P, P, P, P, (1 << 30) + 1, 64, 64, BF, P, None, None) == ob.ERR_UNSUPPORTED
    assert f(vp(4104), P, P, P, 4, 64, 64, BF, P, None, None) == ob.ERR_ALIGN
    assert f(P, P, vp(4104), P, 4, 64, 64, BF, P, None, None) == ob.ERR_ALIGN
    assert f(P, vp(4098), P, P, 4, 64, 64, BF, P, None, None) == ob.ERR_ALIGN
    assert f(P, P, P, P, 4, 64, 64, F32, vp(4098), None, None) == ob.ERR_ALIGN


def test_rope_refusals(lib):
    f = lib.orthrus_rope

    def rc(**kw):
        names = ["dtype", "layout", "q", "qo", "k", "ko", "strides", "pos", "turns", "mag", "T", "Hq", "Hkv", "D",
                 "rot", "qn", "kn", "eps", "st"]
        a = [BF, 0, P, P, P, P, None, P, P, 1.0, 4, 8, 2, 64, 64, None, None, 1e-6, None]
        for k, v in kw.items():
            a[names.index(k)] = v
        return f(*a)

    assert rc(q=None) == rc(qo=None) == rc(pos=None) == rc(turns=None) == ob.ERR_ARG
    assert rc(k=None) == rc(ko=None) == rc(k=None, ko=None) == rc(Hkv=0) == ob.ERR_ARG
    assert rc(dtype=9) == rc(layout=2) == rc(T=0) == rc(Hq=0) == rc(D=0) == rc(rot=0) == rc(rot=66) == ob.ERR_ARG
    assert rc(mag=math.nan) == rc(eps=-1.0) == ob.ERR_ARG
    assert rc(rot=31) == rc(D=300) == ob.ERR_UNSUPPORTED
    assert rc(turns=vp(4100)) == ob.ERR_ALIGN
    other = (ctypes.c_int64 * 8)(512, 64, 1024, 64, 128, 64, 128, 64)
    assert rc(strides=ctypes.cast(other, ctypes.c_void_p)) == ob.ERR_ARG      # in place, through other strides


def test_rope_append_refusals(lib):
    f = lib.orthrus_rope_append

    def rc(**kw):
        names = ["dtype", "layout", "q", "qo", "k", "v", "strides", "turns", "mag", "B", "K", "Hq", "Hkv", "D", "rot",
                 "qn", "kn", "eps", "kp", "vpg", "P", "page", "table", "max", "ctx", "status", "st"]
        a = [BF, 0, P, P, P, P, None, P, 1.0, 2, 1, 8, 2, 64, 64, None, None, 1e-6, P, P, 4, 16, P, 2, P, None, None]
        for k, v in kw.items():
            a[names.index(k)] = v
        return f(*a)

    assert rc(q=None) == rc(qo=None) == rc(k=None) == rc(v=None) == rc(kp=None) == rc(vpg=None) == ob.ERR_ARG
    assert rc(table=None) == rc(ctx=None) == rc(turns=None) == ob.ERR_ARG
    assert rc(B=0) == rc(K=0) == rc(Hkv=0) == rc(P=0) == rc(page=0) == rc(max=0) == ob.ERR_ARG
    assert rc(max=1 << 20, page=1 << 12) == ob.ERR_UNSUPPORTED
    assert rc(rot=7) == ob.ERR_UNSUPPORTED


def test_paged_attn_refusals(lib):
    f = lib.orthrus_paged_attn

    def rc(**kw):
        names = ["dtype", "q", "kp", "vpg", "table", "ctx", "new", "B", "Hq", "Hkv", "D", "P", "page", "max", "scale",
                 "out", "ws", "bytes", "status", "st"]
        a = [BF, P, P, P, P, P, 0, 2, 8, 2, 128, 4, 16, 2, 0.0, P, P, 1 << 30, None, None]
        for k, v in kw.items():
            a[names.index(k)] = v
        return f(*a)

    for n in ("q", "kp", "vpg", "table", "ctx", "out"):
        assert rc(**{n: None}) == ob.ERR_ARG
    assert rc(new=-1) == rc(B=0) == rc(Hq=7) == rc(P=0) == rc(page=0) == rc(max=0) == rc(dtype=8) == ob.ERR_ARG
    assert rc(scale=math.nan) == rc(scale=math.inf) == ob.ERR_ARG
    assert rc(dtype=F32) == rc(D=96) == rc(B=5000) == rc(max=1 << 20, page=1 << 12) == ob.ERR_UNSUPPORTED
    for n in ("q", "kp", "vpg", "out", "ws"):
        assert rc(**{n: vp(4104)}) == ob.ERR_ALIGN
    assert ob.orthrus_paged_attn_workspace_size(2, 7, 2, 128) == 0
    assert ob.orthrus_paged_attn_workspace_size(2, 8, 2, 96) == 0


def test_rope_table_plain_linear_ntk():
    for rot, theta in ((64, 1e4), (128, 1e6), (10, 500.0)):
        plain, mag = ob.orthrus_rope_table(rot, theta)
        want = [theta ** (-2 * i / rot) / (2 * math.pi) for i in range(rot // 2)]
        assert mag == 1.0 and torch.allclose(plain, torch.tensor(want, dtype=torch.float64), rtol=1e-14, atol=0)
        lin, mag = ob.orthrus_rope_table(rot, theta, ob.ROPE_LINEAR, factor=8.0)
        assert mag == 1.0 and torch.allclose(lin, plain / 8, rtol=1e-14, atol=0)
        ntk, mag = ob.orthrus_rope_table(rot, theta, ob.ROPE_NTK, factor=8.0)
        # the fastest pair is kept, the slowest stretched by the whole factor
        assert mag == 1.0 and math.isclose(float(ntk[0]), float(plain[0]), rel_tol=1e-14)
        assert math.isclose(float(ntk[-1]), float(plain[-1]) / 8, rel_tol=1e-12)


def test_rope_table_yarn_bands():
    rot, theta, factor, old = 128, 1e6, 4.0, 32768.0
    plain, _ = ob.orthrus_rope_table(rot, theta)
    t, mag = ob.orthrus_rope_table(rot, theta, ob.ROPE_YARN, factor=factor, orig_len=old)
    assert math.isclose(mag, 0.1 * math.log(4.0) + 1, rel_tol=1e-6)
    turns_in_old = plain * old
    kept, slowed = turns_in_old > 40, turns_in_old < 0.8          # clear of the (rounded) band edges
    assert kept.any() and slowed.any()
    assert torch.equal(t[kept], plain[kept])
    assert torch.allclose(t[slowed], plain[slowed] / factor, rtol=1e-14, atol=0)
    ratio = t / plain
    assert (ratio[1:] <= ratio[:-1] + 1e-15).all() and (ratio >= 1 / factor - 1e-12).all()
    one, mag = ob.orthrus_rope_table(rot, theta, ob.ROPE_YARN, factor=1.0, orig_len=old)
    assert mag == 1.0 and torch.allclose(one, plain, rtol=1e-14, atol=0)


def test_rope_table_refusals():
    for kw in (dict(rot_dim=7, theta=1e4), dict(rot_dim=0, theta=1e4), dict(rot_dim=8, theta=1.0),
               dict(rot_dim=8, theta=1e4, kind=9), dict(rot_dim=8, theta=1e4, kind=ob.ROPE_LINEAR, factor=0.5),
               dict(rot_dim=2, theta=1e4, kind=ob.ROPE_NTK, factor=2.0),
               dict(rot_dim=8, theta=1e4, kind=ob.ROPE_YARN, factor=2.0, orig_len=0.0),
               dict(rot_dim=8, theta=1e4, kind=ob.ROPE_YARN, factor=2.0, orig_len=64.0, beta_fast=1.0, beta_slow=2.0)):
        with pytest.raises(ob.OrthrusError):
            ob.orthrus_rope_table(**kw)


def test_binding_refuses_wrong_shapes_types_and_host_tensors():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                                # host tensors
        ob.orthrus_rmsnorm(x, w, 1e-6, out=torch.empty_like(x))
    with pytest.raises(ValueError):
        ob.orthrus_rmsnorm(x, w.float(), 1e-6, out=torch.empty_like(x))
    with pytest.raises(ValueError):
        ob.orthrus_rmsnorm(x.t(), w, 1e-6, out=torch.empty_like(x))
    with pytest.raises(ValueError):                                # an 8-bit product takes 8-bit operands
        ob.orthrus_fp8_matmul(x, torch.zeros(4, 1), x, torch.zeros(1, 1), torch.empty(4, 4))
    with pytest.raises(ValueError):
        ob.orthrus_quantize_fp8(x, torch.empty(4, 64, dtype=torch.uint8), torch.empty(4, 1))
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    pages = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    table, ctx = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):                                # int64 lengths
        ob.orthrus_paged_attn(q, pages, pages, table, ctx.long(), q, torch.zeros(16))
    with pytest.raises(ValueError):                                # pages of another type
        ob.orthrus_paged_attn(q, pages.half(), pages.half(), table, ctx, q, torch.zeros(16))
    turns = torch.zeros(64, dtype=torch.float64)
    with pytest.raises(ValueError):                                # k without k_out
        ob.orthrus_rope(q, q, ctx, turns, q)
    with pytest.raises(ValueError):                                # in-place keys need K
        ob.orthrus_rope_append(None, None, None, turns, None, pages, None, table, ctx)
