"""Measured cases of the layer operators around the decode step's attention:
RMS norm with the residual's addition, quantisation to 8 bits, the 8-bit
matrix product, rotary positions, and single-token attention over paged caches.

`run` computes a case in its plain form (elementary torch operations in 32 bits,
rounded once at the end) or, where `own` is true, through the library's entry
points.  `exact` gives the same outputs from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

BLOCK = 128                      # values that share one scale
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -126          # smallest scale: a block of zeros keeps a finite reciprocal
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF, INTERLEAVED = 0, 1
DEV = "cuda"


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token entering a layer of the 1.7B-shaped model: pure latency
        dict(name="norm_token", op="norm", T=1, H=2048, dtype="bf16", residual=False, fp8=False),
        # a long prompt between two layers of the 8B-shaped model, feeding the 8-bit projections
        dict(name="norm_prompt_fp8", op="norm", T=16384, H=4096, dtype="bf16", residual=True, fp8=True),
        # the attention output of one decode block, on its way to the output projection
        dict(name="quantize_block", op="quant", T=32, H=4096, dtype="bf16"),
        # a prompt's gated activations before the down projection
        dict(name="quantize_prompt", op="quant", T=8192, H=12288, dtype="bf16"),
        # the QKV projection of one 32-token block (8B shape), weights in 8 bits
        dict(name="matmul_block_qkv", op="matmul", M=32, N=6144, K=4096, out="bf16"),
        # the LM head of four single-token sequences: fp32 logits for consensus or sampling
        dict(name="matmul_token_head", op="matmul", M=4, N=151936, K=4096, out="f32"),
        # a prompt's up projection: bound by the tensor cores
        dict(name="matmul_prompt", op="matmul", M=8192, N=12288, K=4096, out="bf16"),
        # the new tokens of 16 sequences: rotation, key norm and cache rows of one layer
        dict(name="rope_append_tokens", op="append", B=16, K=1, Hq=32, Hkv=8, D=128, rot=128, layout=HALF,
             dtype="bf16", norm=True, scaled=True, page=16, ctx=8192),
        # a prompt's queries and keys, out of the packed projection, positions far out
        dict(name="rope_prompt", op="rope", T=16384, Hq=32, Hkv=8, D=128, rot=128, layout=HALF, dtype="bf16",
             norm=False, scaled=True, far=131072),
        # one sequence, short context: latency
        dict(name="paged_token", op="paged", B=1, Hkv=8, G=2, D=128, page=16, len=300, dtype="bf16"),
        # sixteen ragged sequences of the 4B-shaped model's batch
        dict(name="paged_ragged", op="paged", B=16, Hkv=8, G=4, D=128, page=64, len=16384, dtype="bf16"),
        # long contexts: the stream of keys and values is everything
        dict(name="paged_long", op="paged", B=8, Hkv=8, G=4, D=128, page=32, len=65536, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "quant", "matmul", "append", "rope", "paged"])
    if op in ("norm", "quant"):
        H = _log(rng, 64, 12288)
        if rng.random() < 0.7:
            H = max(64, H // 64 * 64)
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        T = _log(rng, 1, max(1, min(16384, (1 << 26) // H // (2 if dtype == "f32" else 1))))
        c = dict(op=op, T=T, H=H, dtype=dtype)
        if op == "norm":
            c.update(residual=rng.random() < 0.6, fp8=rng.random() < 0.5)
        return c
    if op == "matmul":
        K = 16 * _log(rng, 4, 768)
        if rng.random() < 0.6:
            K = max(128, K // 128 * 128)
        N = _log(rng, 16, min(151936, 151936 * 4096 // K))
        M = _log(rng, 1, max(1, min(8192, (1 << 38) // (N * K), (1 << 27) // N)))
        return dict(op=op, M=M, N=N, K=K, out=rng.choice(["bf16", "bf16", "f16", "f32"]))
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 5, 8, 16])
    if op == "paged":
        page = rng.choice([1, 8, 16, 16, 24, 32, 64, 128, 256])
        B = _log(rng, 1, 128)
        top = (1 << 29) // (B * Hkv * D)            # keys and values held at once
        return dict(op=op, B=B, Hkv=Hkv, G=G, D=D, page=page, len=_log(rng, 1, min(65536, top)),
                    dtype=rng.choice(["bf16", "bf16", "f16"]))
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    rot = rng.choice([D, D, D // 2, D // 4])
    c = dict(op=op, Hq=Hkv * G, Hkv=Hkv, D=D, rot=rot, layout=rng.choice([HALF, INTERLEAVED]), dtype=dtype,
             norm=rng.random() < 0.5, scaled=rng.random() < 0.5)
    if op == "rope":
        c.update(T=_log(rng, 1, max(1, min(16384, (1 << 25) // ((Hkv * G + 2 * Hkv) * D)))), far=_log(rng, 128, 1 << 20))
    else:
        c.update(B=_log(rng, 1, 64), K=rng.choice([1, 1, 5, 32]), page=rng.choice([8, 16, 24, 64]))
        c.update(ctx=_log(rng, 1, max(1, min(8192, (1 << 26) // (c["B"] * Hkv * D)))))
    return c


# -------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _cdiv(a, b):
    return -(-a // b)


def _lengths(c):
    """The sequences' lengths: a property of the case, not of the seed."""
    r = random.Random(c["B"] * 1000003 + c["len"])
    n = [c["len"]] + [r.randint(max(1, c["len"] // 8), c["len"]) for _ in range(c["B"] - 1)]
    if c["B"] >= 3:
        n[1] = 1                                    # a sequence that has just begun
    if c["B"] >= 8:
        n[2] = 0                                    # an idle slot of the batch
    return n


def _contexts(c):
    r = random.Random(c["B"] * 1000003 + c["ctx"])
    return [c["ctx"]] + [r.randint(0, c["ctx"]) for _ in range(c["B"] - 1)]


def _turns(rot, scaled):
    """Turns per position of each rotated pair, and the factor on the rotated
    values: plain, or stretched fourfold with smooth bands between kept and
    interpolated frequencies (YaRN, arXiv 2309.00071, section 3.2)."""
    theta, factor, old = 1e6, 4.0, 32768.0
    half = rot // 2
    inv = [theta ** (-2.0 * i / rot) for i in range(half)]
    mag = 1.0
    if scaled:
        def place(turns):
            return rot * math.log(old / (turns * 2 * math.pi)) / (2 * math.log(theta))
        low, high = max(math.floor(place(32.0)), 0), min(math.ceil(place(1.0)), rot - 1)
        if high == low:
            high = low + 0.001
        ramp = [min(1.0, max(0.0, (i - low) / (high - low))) for i in range(half)]
        inv = [f / factor * r + f * (1 - r) for f, r in zip(inv, ramp)]
        mag = 0.1 * math.log(factor) + 1.0
    return torch.tensor([f / (2 * math.pi) for f in inv], dtype=torch.float64, device=DEV), mag


def _pages(g, lens, page, Hkv, D, dt):
    """A shuffled pool of pages [pages, Hkv, page, D] and the sequences' tables;
    entries that no sequence uses are -1."""
    need = [_cdiv(n, page) for n in lens]
    total = sum(need) + 2
    order = torch.randperm(total, generator=g, device=DEV).tolist()
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    k, v = (torch.empty((total, Hkv, page, D), dtype=dt, device=DEV) for _ in range(2))
    for t in (k, v):
        t.normal_(generator=g)
    return k, v, table.to(DEV)


def _to_e4m3(x, rows):
    """8-bit values and fp32 scales of [T, H], one scale per `rows` x 128 block."""
    T, H = x.shape
    pad = torch.zeros((_cdiv(T, rows) * rows, _cdiv(H, BLOCK) * BLOCK), device=DEV)
    pad[:T, :H] = x
    blk = pad.view(-1, rows, pad.shape[1] // BLOCK, BLOCK)
    scale = (blk.abs().amax((1, 3)) / E4M3_MAX).clamp_min(MIN_SCALE)
    q = (blk / scale[:, None, :, None]).view_as(pad)[:T, :H].contiguous()
    return q.to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    c, g, op = case, _gen(seed), case["op"]
    s = dict(case=c)
    if op in ("norm", "quant"):
        dt, T, H = TYPES[c["dtype"]], c["T"], c["H"]
        loud = torch.exp(0.7 * _randn(g, H))        # a few channels much larger than the rest
        s["x"] = (_randn(g, T, H) * loud).to(dt)
        if op == "norm":
            s["weight"] = (1 + 0.2 * _randn(g, H)).to(dt)
            if c["residual"]:
                s["residual"] = (_randn(g, T, H) * loud).to(dt)
                s["sum"] = torch.empty_like(s["x"])
        if op == "quant" or c["fp8"]:
            s["q"] = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=DEV)
            s["scale"] = torch.empty((T, _cdiv(H, BLOCK)), device=DEV)
        else:
            s["out"] = torch.empty_like(s["x"])
    elif op == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        s["a"], s["a_scale"] = _to_e4m3(_randn(g, M, K) * torch.exp(0.7 * _randn(g, K)), 1)
        s["w"], s["w_scale"] = _to_e4m3(_randn(g, N, K) / math.sqrt(K), BLOCK)
        s["out"] = torch.empty((M, N), dtype=TYPES[c["out"]], device=DEV)
    elif op in ("rope", "append"):
        dt, Hq, Hkv, D = TYPES[c["dtype"]], c["Hq"], c["Hkv"], c["D"]
        lead = (c["T"],) if op == "rope" else (c["B"], c["K"])
        qkv = _randn(g, *lead, Hq + 2 * Hkv, D).to(dt)         # the packed projection
        s["qx"], s["kx"], s["vx"] = qkv[..., :Hq, :], qkv[..., Hq:Hq + Hkv, :], qkv[..., Hq + Hkv:, :]
        s["turns"], s["mag"] = _turns(c["rot"], c["scaled"])
        s["qn"], s["kn"] = ((1 + 0.2 * _randn(g, D)).to(dt) if c["norm"] else None for _ in range(2))
        s["q_out"] = torch.empty((*lead, Hq, D), dtype=dt, device=DEV)
        if op == "rope":
            s["k_out"] = torch.empty((*lead, Hkv, D), dtype=dt, device=DEV)
            start = int(torch.randint(0, max(1, c["far"] - c["T"]), (1,), generator=g, device=DEV))
            s["pos"] = torch.arange(start, start + c["T"], dtype=torch.int32, device=DEV)
        else:
            ctx = _contexts(c)
            s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
            s["kp"], s["vp"], s["table"] = _pages(g, [n + c["K"] for n in ctx], c["page"], Hkv, D, dt)
    else:
        dt, Hkv, G, D = TYPES[c["dtype"]], c["Hkv"], c["G"], c["D"]
        lens = _lengths(c)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["kp"], s["vp"], s["table"] = _pages(g, lens, c["page"], Hkv, D, dt)
        s["qx"] = _randn(g, c["B"], Hkv * G, D).to(dt)
        s["out"] = torch.empty_like(s["qx"])
    return s


# ---------------------------------------------------------- the plain forms
def _plain_quantize(y):
    T, H = y.shape
    n = _cdiv(H, BLOCK)
    blk = torch.nn.functional.pad(y, (0, n * BLOCK - H)).view(T, n, BLOCK)
    scale = (blk.abs().amax(-1) / E4M3_MAX).clamp_min(MIN_SCALE)
    q = (blk / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).view(T, n * BLOCK)[:, :H]
    return q.to(torch.float8_e4m3fn), scale


def _plain_norm(s):
    x = s["x"].float()
    out = {}
    if "residual" in s:
        x = x + s["residual"].float()
        out["sum"] = x.to(s["x"].dtype)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    if "q" in s:
        out["q"], out["scale"] = _plain_quantize(y)
    else:
        out["out"] = y.to(s["x"].dtype)
    return out


def _spread(scale, rows, shape):
    return scale.repeat_interleave(rows, 0)[:shape[0]].repeat_interleave(BLOCK, 1)[:, :shape[1]]


def _plain_matmul(s):
    a = s["a"].float() * _spread(s["a_scale"], 1, s["a"].shape)
    w = s["w"].float() * _spread(s["w_scale"], BLOCK, s["w"].shape)
    return (a @ w.t()).to(s["out"].dtype)


def _plain_rotate(x, pos, s, weight):
    """x [..., H, D] at positions pos [...]: the head's norm, then the rotation."""
    c = s["case"]
    r, y = c["rot"], x.float()
    if weight is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * weight.float()
    angle = (pos.double()[..., None] * s["turns"]) * (2 * math.pi)
    cos, sin = ((f(angle) * s["mag"]).float()[..., None, :] for f in (torch.cos, torch.sin))
    a, b = (y[..., :r // 2], y[..., r // 2:r]) if c["layout"] == HALF else (y[..., 0:r:2], y[..., 1:r:2])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat((u, v), -1) if c["layout"] == HALF else torch.stack((u, v), -1).flatten(-2)
    return torch.cat((turned, y[..., r:]), -1).to(x.dtype)


def _plain_append(s):
    c = s["case"]
    pos = s["ctx"][:, None] + torch.arange(c["K"], dtype=torch.int32, device=DEV)
    q = _plain_rotate(s["qx"], pos, s, s["qn"])
    k = _plain_rotate(s["kx"], pos, s, s["kn"])
    page = s["table"].gather(1, (pos // c["page"]).long()).long()
    row = (pos % c["page"]).long()
    s["kp"][page, :, row] = k
    s["vp"][page, :, row] = s["vx"]
    return {"q": q, "k_pages": s["kp"], "v_pages": s["vp"]}


def _plain_paged(s):
    c = s["case"]
    B, Hkv, G, D, page = c["B"], c["Hkv"], c["G"], c["D"], c["page"]
    at = s["table"].clamp_min(0).long()
    n = at.shape[1] * page
    k = s["kp"][at].transpose(1, 2).reshape(B, Hkv, n, D).float()
    score = (s["qx"].float().view(B, Hkv, G, D) @ k.transpose(-1, -2)) / math.sqrt(D)
    del k
    seen = torch.arange(n, device=DEV) < s["lens"][:, None]
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min(-1e30)
    p = torch.exp(score - top)
    v = s["vp"][at].transpose(1, 2).reshape(B, Hkv, n, D).float()
    o = (p @ v) / p.sum(-1, keepdim=True).clamp_min(1e-30)      # a sequence of length zero gives zeros
    return o.reshape(B, Hkv * G, D).to(s["qx"].dtype)


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        return _own(s, c, op)
    if op == "norm":
        return _plain_norm(s)
    if op == "quant":
        q, scale = _plain_quantize(s["x"].float())
        return {"q": q, "scale": scale}
    if op == "matmul":
        return _plain_matmul(s)
    if op == "rope":
        return {"q": _plain_rotate(s["qx"], s["pos"], s, s["qn"]), "k": _plain_rotate(s["kx"], s["pos"], s, s["kn"])}
    if op == "append":
        return _plain_append(s)
    return _plain_paged(s)


# ------------------------------------------------------ the framework's calls
def _own(s, c, op):
    import lossless_diffusion_speculative_b200 as lib
    if op == "norm":
        lib.orthrus_rmsnorm(s["x"], s["weight"], EPS, out=s.get("out"), residual=s.get("residual"),
                            sum_out=s.get("sum"), out_fp8=s.get("q"), out_scale=s.get("scale"))
        return {k: s[k] for k in ("sum", "q", "scale", "out") if k in s}
    if op == "quant":
        lib.orthrus_quantize_fp8(s["x"], s["q"], s["scale"])
        return {"q": s["q"], "scale": s["scale"]}
    if op == "matmul":
        lib.orthrus_fp8_matmul(s["a"], s["a_scale"], s["w"], s["w_scale"], s["out"])
        return s["out"]
    if op == "rope":
        lib.orthrus_rope(s["qx"], s["kx"], s["pos"], s["turns"], s["q_out"], s["k_out"], layout=c["layout"],
                         magnitude=s["mag"], q_norm=s["qn"], k_norm=s["kn"], eps=EPS)
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "append":
        lib.orthrus_rope_append(s["qx"], s["kx"], s["vx"], s["turns"], s["q_out"], s["kp"], s["vp"], s["table"],
                                s["ctx"], layout=c["layout"], magnitude=s["mag"], q_norm=s["qn"], k_norm=s["kn"],
                                eps=EPS)
        return {"q": s["q_out"], "k_pages": s["kp"], "v_pages": s["vp"]}
    if "workspace" not in s:                        # kept by the program, as for the other attention calls
        size = lib.orthrus_paged_attn_workspace_size(c["B"], c["Hkv"] * c["G"], c["Hkv"], c["D"])
        s["workspace"] = torch.zeros(size, dtype=torch.uint8, device=DEV)
    lib.orthrus_paged_attn(s["qx"], s["kp"], s["vp"], s["table"], s["lens"], s["out"], s["workspace"])
    return s["out"]


# ---------------------------------------------------------------------- work
def work(case):
    c, op = case, case["op"]
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if op in ("norm", "quant"):
        T, H, e = c["T"], c["H"], size[c["dtype"]]
        fp8 = op == "quant" or c["fp8"]
        b = T * H * e + (T * (H + 4 * _cdiv(H, BLOCK)) if fp8 else T * H * e)
        if op == "norm":
            b += H * e + (2 * T * H * e if c["residual"] else 0)
        return {"bytes": b, "flops": (6 if op == "norm" else 3) * T * H}
    if op == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        b = M * K + N * K + 4 * _cdiv(K, BLOCK) * (M + _cdiv(N, BLOCK)) + M * N * size[c["out"]]
        return {"bytes": b, "flops": 2 * M * N * K}
    if op in ("rope", "append"):
        e, T = size[c["dtype"]], c["T"] if op == "rope" else c["B"] * c["K"]
        heads = c["Hq"] + c["Hkv"]
        b = 2 * T * heads * c["D"] * e + (2 * T * c["Hkv"] * c["D"] * e if op == "append" else 0) + 4 * T
        return {"bytes": b, "flops": T * heads * (3 * c["rot"] + (4 * c["D"] if c["norm"] else 0))}
    n = sum(_lengths(c))
    return {"bytes": 4 * n * c["Hkv"] * c["D"] + 4 * c["B"] * c["Hkv"] * c["G"] * c["D"],
            "flops": 4 * n * c["Hkv"] * c["G"] * c["D"]}


# --------------------------------------------------------------------- exact
def _exact_scales(y):
    """[T, ceil(H / 128)] scales and the unrounded quotients."""
    T, H = y.shape
    scale = torch.stack([y[:, i:i + BLOCK].abs().max(1).values for i in range(0, H, BLOCK)], 1) / E4M3_MAX
    scale = torch.maximum(scale, torch.full_like(scale, MIN_SCALE))
    return y / scale[:, torch.arange(H, device=DEV) // BLOCK], scale


def _exact_turned(x, pos, s, weight):
    c = s["case"]
    x = x.double()
    if weight is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / c["D"] + EPS).sqrt() * weight.double()
    y = x.clone()
    for i in range(c["rot"] // 2):
        j, l = (i, i + c["rot"] // 2) if c["layout"] == HALF else (2 * i, 2 * i + 1)
        part = pos.double() * s["turns"][i]
        z = torch.polar(torch.full_like(part, s["mag"]), 2 * math.pi * (part - part.floor()))[..., None]
        w = torch.complex(x[..., j], x[..., l]) * z
        y[..., j], y[..., l] = w.real, w.imag
    return y


def exact(case, seed):
    c, op, s = case, case["op"], prepare(case, seed)
    if op in ("norm", "quant"):
        out, y = {}, s["x"].double()
        if op == "norm":
            if c["residual"]:
                y = y + s["residual"].double()
                out["sum"] = y
            y = y / (y.pow(2).sum(1, keepdim=True) / c["H"] + EPS).sqrt() * s["weight"].double()
        if op == "norm" and not c["fp8"]:
            out["out"] = y
        else:
            out["q"], out["scale"] = _exact_scales(y)
        return out
    if op == "matmul":
        out = torch.zeros((c["M"], c["N"]), dtype=torch.float64, device=DEV)
        for n in range(0, c["N"], 16384):           # in parts: the 64-bit weights are eight times as large
            cols = torch.arange(n, min(n + 16384, c["N"]), device=DEV)
            kb = torch.arange(c["K"], device=DEV) // BLOCK
            w = s["w"][n:n + 16384].double() * s["w_scale"].double()[cols // BLOCK][:, kb]
            out[:, n:n + 16384] = (s["a"].double() * s["a_scale"].double()[:, kb]) @ w.t()
        return out
    if op == "rope":
        return {"q": _exact_turned(s["qx"], s["pos"], s, s["qn"]), "k": _exact_turned(s["kx"], s["pos"], s, s["kn"])}
    if op == "append":
        kp, vp = s["kp"].double(), s["vp"].double()
        pos = torch.stack([s["ctx"] + i for i in range(c["K"])], 1)
        k = _exact_turned(s["kx"], pos, s, s["kn"])
        table = s["table"].tolist()
        for b, n in enumerate(s["ctx"].tolist()):
            for i in range(c["K"]):
                page, row = table[b][(n + i) // c["page"]], (n + i) % c["page"]
                kp[page, :, row], vp[page, :, row] = k[b, i], s["vx"][b, i].double()
        return {"q": _exact_turned(s["qx"], pos, s, s["qn"]), "k_pages": kp, "v_pages": vp}
    out = torch.zeros(s["qx"].shape, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"].tolist()):
        if n:
            at = s["table"][b, :_cdiv(n, c["page"])].long()
            k, v = (t[at].transpose(0, 1).flatten(1, 2)[:, :n].double() for t in (s["kp"], s["vp"]))
            q = s["qx"][b].double().view(c["Hkv"], c["G"], c["D"])
            out[b] = (torch.softmax(torch.einsum("hgd,hnd->hgn", q, k) / math.sqrt(c["D"]), -1) @ v).flatten(0, 1)
    return out
