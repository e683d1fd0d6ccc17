"""Thin ctypes binding of liborthrus.so (argument marshalling only).

Every function here has the name of the C entry point it wraps and does nothing
but read shapes and device pointers off torch tensors and forward them; all
arithmetic runs in the library's CUDA kernels.  There is no CPU fallback: if the
library is missing or the device cannot run it, the call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Sequence

import torch

from .build import LIB

DIFF, AR = 0, 1
BF16, F32, F16 = 0, 1, 2
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_PLAIN, ROPE_LINEAR, ROPE_NTK, ROPE_YARN = 0, 1, 2, 3

ERR_ARG, ERR_UNSUPPORTED, ERR_ALIGN, ERR_WORKSPACE, ERR_LAUNCH, ERR_DEVICE = -1, -2, -3, -4, -5, -6
STATUS_CAPACITY, STATUS_ACCEPT, STATUS_TIMEOUT, STATUS_PAGE = 0x1, 0x2, 0x4, 0x8

EXPORTED = ("orthrus_attn_workspace_size", "orthrus_attn", "orthrus_attn_path",
            "orthrus_consensus_workspace_size", "orthrus_consensus",
            "orthrus_kv_commit", "orthrus_write_block", "orthrus_error_string",
            "orthrus_version", "orthrus_lm_head_workspace_size",
            "orthrus_lm_head_consensus", "orthrus_rejection_workspace_size",
            "orthrus_rejection_verify", "orthrus_qkv_workspace_size", "orthrus_qkv_project",
            "orthrus_prefill_workspace_size",
            "orthrus_prefill_attn", "orthrus_rmsnorm", "orthrus_quantize_fp8", "orthrus_fp8_matmul",
            "orthrus_rope_table", "orthrus_rope", "orthrus_rope_append",
            "orthrus_paged_attn_workspace_size", "orthrus_paged_attn")


class OrthrusError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} failed: {msg} (code {code})")
        self.code = code


_lib = None


def lib():
    """Load liborthrus.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB):
            raise RuntimeError(
                f"liborthrus.so not found at {LIB}; build it with "
                "`python -m lossless_diffusion_speculative_b200.build`")
        L = ctypes.CDLL(LIB)
        vp, sz, i32, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
        L.orthrus_attn_workspace_size.restype = sz
        L.orthrus_attn_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
        L.orthrus_attn.restype = i32
        L.orthrus_attn.argtypes = [i32, i32, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32,
                                   f32, vp, vp, sz, vp, vp]
        L.orthrus_consensus_workspace_size.restype = sz
        L.orthrus_consensus_workspace_size.argtypes = [i32, i32, i32]
        L.orthrus_consensus.restype = i32
        L.orthrus_consensus.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp, vp, sz, vp, vp]
        L.orthrus_kv_commit.restype = i32
        L.orthrus_kv_commit.argtypes = [i32, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                        i32, vp, vp]
        L.orthrus_write_block.restype = i32
        L.orthrus_write_block.argtypes = [i32, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                          i32, vp, vp]
        L.orthrus_attn_path.restype = i32
        L.orthrus_attn_path.argtypes = [i32, i32, i32, i32, i32, i32]
        L.orthrus_lm_head_workspace_size.restype = sz
        L.orthrus_lm_head_workspace_size.argtypes = [i32, i32]
        L.orthrus_lm_head_consensus.restype = i32
        L.orthrus_lm_head_consensus.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, sz,
                                                vp, vp]
        L.orthrus_rejection_workspace_size.restype = sz
        L.orthrus_rejection_workspace_size.argtypes = [i32, i32, i32]
        L.orthrus_rejection_verify.restype = i32
        L.orthrus_rejection_verify.argtypes = [vp, vp, vp, vp, vp, f32, i32, i32, i32, vp, vp, vp, sz,
                                               vp, vp]
        L.orthrus_qkv_workspace_size.restype = sz
        L.orthrus_qkv_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
        L.orthrus_qkv_project.restype = i32
        L.orthrus_qkv_project.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, vp, vp,
                                          vp, vp, sz, vp, vp]
        L.orthrus_prefill_workspace_size.restype = sz
        L.orthrus_prefill_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
        L.orthrus_prefill_attn.restype = i32
        L.orthrus_prefill_attn.argtypes = [i32, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, vp, vp, sz,
                                           vp, vp]
        i64, f64 = ctypes.c_int64, ctypes.c_double
        L.orthrus_rmsnorm.restype = i32
        L.orthrus_rmsnorm.argtypes = [i32, vp, i64, vp, vp, i32, i32, f32, vp, vp, vp, vp, vp]
        L.orthrus_quantize_fp8.restype = i32
        L.orthrus_quantize_fp8.argtypes = [i32, vp, i64, i32, i32, vp, vp, vp]
        L.orthrus_fp8_matmul.restype = i32
        L.orthrus_fp8_matmul.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp]
        L.orthrus_rope_table.restype = i32
        L.orthrus_rope_table.argtypes = [i32, i32, f64, f64, f64, f64, f64, vp, vp]
        L.orthrus_rope.restype = i32
        L.orthrus_rope.argtypes = [i32, i32, vp, vp, vp, vp, vp, vp, vp, f32, i32, i32, i32, i32, i32, vp, vp, f32,
                                   vp]
        L.orthrus_rope_append.restype = i32
        L.orthrus_rope_append.argtypes = [i32, i32, vp, vp, vp, vp, vp, vp, f32, i32, i32, i32, i32, i32, i32, vp, vp,
                                          f32, vp, vp, i32, i32, vp, i32, vp, vp, vp]
        L.orthrus_paged_attn_workspace_size.restype = sz
        L.orthrus_paged_attn_workspace_size.argtypes = [i32, i32, i32, i32]
        L.orthrus_paged_attn.restype = i32
        L.orthrus_paged_attn.argtypes = [i32, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, f32, vp, vp,
                                         sz, vp, vp]
        L.orthrus_error_string.restype = ctypes.c_char_p
        L.orthrus_error_string.argtypes = [i32]
        L.orthrus_version.restype = i32
        L.orthrus_version.argtypes = []
        _lib = L
    return _lib


def _check(fn: str, rc: int) -> None:
    if rc != 0:
        raise OrthrusError(fn, rc, lib().orthrus_error_string(rc).decode())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("liborthrus takes device tensors")
    if not t.is_contiguous():
        raise ValueError("liborthrus takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return BF16
    if dt == torch.float32:
        return F32
    raise ValueError(f"unsupported dtype {dt}")


def orthrus_version() -> int:
    return int(lib().orthrus_version())


def orthrus_attn_workspace_size(B: int, Hq: int, Hkv: int, D: int, K: int,
                                dtype: torch.dtype = torch.bfloat16) -> int:
    return int(lib().orthrus_attn_workspace_size(B, Hq, Hkv, D, K, _dtype_code(dtype)))


def orthrus_attn(view: int, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 ctx_lens: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor,
                 status: Optional[torch.Tensor] = None, scale: float = 0.0,
                 stream=None) -> None:
    """q [B,K,Hq,D], caches [B,Hkv,S_max,D] (bf16 or fp32), ctx_lens [B] int32,
    out [B,K,Hq,D] fp32, workspace uint8 of orthrus_attn_workspace_size bytes."""
    B, K, Hq, D = q.shape
    _, Hkv, S_max, _ = k_cache.shape
    assert ctx_lens.dtype == torch.int32 and out.dtype == torch.float32
    rc = lib().orthrus_attn(int(view), _dtype_code(q.dtype), _ptr(q), _ptr(k_cache),
                            _ptr(v_cache), _ptr(ctx_lens), B, Hq, Hkv, D, S_max, K,
                            float(scale), _ptr(out), _ptr(workspace),
                            workspace.numel() * workspace.element_size(), _ptr(status),
                            _stream(stream))
    _check("orthrus_attn", rc)


def orthrus_consensus_workspace_size(B: int, K: int, V: int) -> int:
    return int(lib().orthrus_consensus_workspace_size(B, K, V))


def orthrus_consensus(logits: torch.Tensor, proposed: torch.Tensor, accepted_len: torch.Tensor,
                      next_token: torch.Tensor, workspace: torch.Tensor,
                      argmax_out: Optional[torch.Tensor] = None,
                      status: Optional[torch.Tensor] = None, stream=None) -> None:
    """logits [B,K,V] fp32, proposed [B,K] int32 -> accepted_len [B], next_token [B]."""
    B, K, V = logits.shape
    assert logits.dtype == torch.float32 and proposed.dtype == torch.int32
    rc = lib().orthrus_consensus(_ptr(logits), _ptr(proposed), B, K, V, _ptr(accepted_len),
                                 _ptr(next_token), _ptr(argmax_out), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(),
                                 _ptr(status), _stream(stream))
    _check("orthrus_consensus", rc)


def _ptr_array(ts):
    """(void*, keep-alive) for a host array of device pointers, or (None, None)."""
    if ts is None:
        return None, None
    a = (ctypes.c_void_p * len(ts))(*[t.data_ptr() for t in ts])
    return ctypes.cast(a, ctypes.c_void_p), a


def orthrus_attn_path(B: int, Hq: int, Hkv: int, D: int, K: int,
                      dtype: torch.dtype = torch.bfloat16) -> int:
    """1 = tensor-core path, 0 = CUDA-core path (negative: error code)."""
    return int(lib().orthrus_attn_path(B, Hq, Hkv, D, K, _dtype_code(dtype)))


def orthrus_write_block(ctx_lens: torch.Tensor, k_caches: Sequence[torch.Tensor],
                        v_caches: Sequence[torch.Tensor], k_blks: Sequence[torch.Tensor],
                        v_blks: Sequence[torch.Tensor], status: Optional[torch.Tensor] = None,
                        stream=None) -> None:
    """Copy each layer's block K/V [B,K,Hkv,D] into cache rows [ctx, ctx+K)."""
    B, Hkv, S_max, D = k_caches[0].shape
    K = k_blks[0].shape[1]
    packs = [_ptr_array(x) for x in (k_caches, v_caches, k_blks, v_blks)]
    rc = lib().orthrus_write_block(len(k_caches), *[p[0] for p in packs], _ptr(ctx_lens), B, Hkv,
                                   D, S_max, K, _dtype_code(k_caches[0].dtype), _ptr(status),
                                   _stream(stream))
    _check("orthrus_write_block", rc)


def orthrus_kv_commit(ctx_lens: torch.Tensor, accepted_len: torch.Tensor, *, K: int, Hkv: int,
                      D: int, S_max: int, dtype: torch.dtype = torch.bfloat16,
                      num_layers: int = 1,
                      k_caches: Optional[Sequence[torch.Tensor]] = None,
                      v_caches: Optional[Sequence[torch.Tensor]] = None,
                      k_blks: Optional[Sequence[torch.Tensor]] = None,
                      v_blks: Optional[Sequence[torch.Tensor]] = None,
                      status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Commit min(a+1, K) block slots (copying from staging when k_blks is given)
    and advance ctx_lens once."""
    B = ctx_lens.shape[0]
    packs = [_ptr_array(x) for x in (k_caches, v_caches, k_blks, v_blks)]
    if k_blks is not None:
        num_layers = len(k_blks)
    rc = lib().orthrus_kv_commit(num_layers, *[p[0] for p in packs],
                                 _ptr(ctx_lens), _ptr(accepted_len), B, Hkv, D, S_max, K,
                                 _dtype_code(dtype), _ptr(status), _stream(stream))
    _check("orthrus_kv_commit", rc)


def orthrus_lm_head_workspace_size(B: int, K: int) -> int:
    return int(lib().orthrus_lm_head_workspace_size(B, K))


def orthrus_lm_head_consensus(hidden: torch.Tensor, lm_head: torch.Tensor, proposed: torch.Tensor,
                              accepted_len: torch.Tensor, next_token: torch.Tensor,
                              workspace: torch.Tensor, argmax_out: Optional[torch.Tensor] = None,
                              status: Optional[torch.Tensor] = None, stream=None) -> None:
    """hidden [B,K,Hd] bf16, lm_head [V,Hd] bf16, proposed [B,K] int32 ->
    accepted_len [B], next_token [B] (the logits are never materialised)."""
    B, K, Hd = hidden.shape
    V = lm_head.shape[0]
    assert hidden.dtype == torch.bfloat16 and lm_head.dtype == torch.bfloat16
    assert proposed.dtype == torch.int32 and lm_head.shape[1] == Hd
    rc = lib().orthrus_lm_head_consensus(_ptr(hidden), _ptr(lm_head), _ptr(proposed), B, K, V, Hd,
                                         _ptr(accepted_len), _ptr(next_token), _ptr(argmax_out),
                                         _ptr(workspace), workspace.numel() * workspace.element_size(),
                                         _ptr(status), _stream(stream))
    _check("orthrus_lm_head_consensus", rc)


def orthrus_rejection_workspace_size(B: int, K: int, V: int) -> int:
    return int(lib().orthrus_rejection_workspace_size(B, K, V))


def orthrus_rejection_verify(ar_logits: torch.Tensor, draft_logits: torch.Tensor,
                             proposed: torch.Tensor, u_accept: torch.Tensor, u_resample: torch.Tensor,
                             temperature: float, accepted_len: torch.Tensor, next_token: torch.Tensor,
                             workspace: torch.Tensor, status: Optional[torch.Tensor] = None,
                             stream=None) -> None:
    """Logits [B,K,V] fp32 of both views, proposals [B,K] int32, uniform draws
    u_accept [B,K] and u_resample [B] fp32 -> accepted_len [B], next_token [B]."""
    B, K, V = ar_logits.shape
    assert ar_logits.dtype == torch.float32 and draft_logits.dtype == torch.float32
    assert draft_logits.shape == ar_logits.shape and proposed.dtype == torch.int32
    assert u_accept.dtype == torch.float32 and u_resample.dtype == torch.float32
    rc = lib().orthrus_rejection_verify(_ptr(ar_logits), _ptr(draft_logits), _ptr(proposed),
                                        _ptr(u_accept), _ptr(u_resample), float(temperature), B, K, V,
                                        _ptr(accepted_len), _ptr(next_token), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), _ptr(status),
                                        _stream(stream))
    _check("orthrus_rejection_verify", rc)


def orthrus_qkv_workspace_size(B: int, K: int, hidden: int, Hq: int, Hkv: int, D: int) -> int:
    return int(lib().orthrus_qkv_workspace_size(B, K, hidden, Hq, Hkv, D))


def orthrus_qkv_project(x: torch.Tensor, w_q: torch.Tensor, w_k: torch.Tensor, w_v: torch.Tensor,
                        ctx_lens: torch.Tensor, q_out: torch.Tensor, k_cache: torch.Tensor,
                        v_cache: torch.Tensor, workspace: torch.Tensor,
                        status: Optional[torch.Tensor] = None, stream=None) -> None:
    """x [B,K,hidden] bf16, weights [features, hidden] bf16 -> q_out [B,K,Hq,D]
    and cache rows [ctx, ctx+K) of k_cache / v_cache [B,Hkv,S_max,D] (bf16)."""
    B, K, hidden = x.shape
    _, Hkv, S_max, D = k_cache.shape
    Hq = q_out.shape[2]
    for t in (x, w_q, w_k, w_v, q_out, k_cache, v_cache):
        assert t.dtype == torch.bfloat16
    assert ctx_lens.dtype == torch.int32 and w_q.shape == (Hq * D, hidden)
    assert w_k.shape == (Hkv * D, hidden) and w_v.shape == (Hkv * D, hidden)
    rc = lib().orthrus_qkv_project(_ptr(x), _ptr(w_q), _ptr(w_k), _ptr(w_v), _ptr(ctx_lens), B, K,
                                   hidden, Hq, Hkv, D, S_max, _ptr(q_out), _ptr(k_cache),
                                   _ptr(v_cache), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _ptr(status),
                                   _stream(stream))
    _check("orthrus_qkv_project", rc)


def orthrus_prefill_workspace_size(B: int, S: int, Hq: int, Hkv: int, D: int,
                                   dtype: torch.dtype = torch.bfloat16) -> int:
    return int(lib().orthrus_prefill_workspace_size(B, S, Hq, Hkv, D, _dtype_code(dtype)))


def orthrus_prefill_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                         out: torch.Tensor, workspace: torch.Tensor, status: Optional[torch.Tensor] = None,
                         scale: float = 0.0, stream=None) -> None:
    """Causal attention over the prompt: q [B,S,Hq,D], caches [B,Hkv,S_max,D]
    (rows [0, S) = the prompt) -> out [B,S,Hq,D] fp32."""
    B, S, Hq, D = q.shape
    _, Hkv, S_max, _ = k_cache.shape
    assert out.dtype == torch.float32 and out.shape == q.shape
    rc = lib().orthrus_prefill_attn(_dtype_code(q.dtype), _ptr(q), _ptr(k_cache), _ptr(v_cache), B, S, Hq,
                                    Hkv, D, S_max, float(scale), _ptr(out), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _ptr(status),
                                    _stream(stream))
    _check("orthrus_prefill_attn", rc)


# ---------------------------------------------------------------- layer operators
# (These calls are short on the GPU, so their argument checks are kept to what a
# few attribute reads per tensor cost.)
_CODES = {torch.bfloat16: BF16, torch.float32: F32, torch.float16: F16}
_E4M3, _FP32 = torch.float8_e4m3fn, torch.float32
# (torch's own short forms of these two look-ups; a torch built without CUDA has
# neither, and the package is imported there too)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _code(dt: torch.dtype) -> int:
    code = _CODES.get(dt)
    if code is None:
        raise ValueError(f"unsupported dtype {dt}")
    return code


def _fail(t: torch.Tensor, dtype, shape, dev):
    if t.get_device() < 0:
        raise ValueError("liborthrus takes device tensors")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"expected {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"tensors on devices {dev} and {t.get_device()}")
    raise ValueError("liborthrus takes contiguous tensors here")


def _dense(t: torch.Tensor, dtype, shape, dev: int):
    """Address of a contiguous tensor of this type and shape on device `dev`
    (a None type or shape is not checked)."""
    if ((dtype is not None and t.dtype is not dtype) or (shape is not None and t.shape != shape)
            or t.get_device() != dev or dev < 0 or not t.is_contiguous()):
        _fail(t, dtype, shape, dev)
    return t.data_ptr()


def _strided(t: torch.Tensor, dtype, shape, dev: int):
    """The same for a tensor whose strides are passed along."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or dev < 0:
        _fail(t, dtype, shape, dev)
    return t.data_ptr()


def _elsewhere(dev: int, fn, args) -> int:
    """The call with the tensors' device current (it is not)."""
    with torch.cuda.device(dev):
        return fn(*args)


def _on(stream, dev: int) -> int:
    """The raw stream a call goes to: by default the tensors' device's current one."""
    if stream is None:
        return _raw_stream(dev) if dev >= 0 else 0
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _rows(x: torch.Tensor):
    """(shape, row stride) of a [T, H] tensor whose rows are contiguous."""
    shape, st = x.shape, x.stride()
    if len(shape) != 2:
        raise ValueError(f"expected [rows, width], got {tuple(shape)}")
    if st[1] != 1 and shape[1] > 1:
        raise ValueError("rows have to be contiguous")
    return shape, (st[0] if shape[0] > 1 else shape[1])


def orthrus_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float, out: Optional[torch.Tensor] = None,
                    residual: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
                    out_fp8: Optional[torch.Tensor] = None, out_scale: Optional[torch.Tensor] = None,
                    stream=None) -> None:
    """x [T,H] (rows may be strided; bf16, fp16 or fp32), weight [H] -> out [T,H]
    and / or out_fp8 [T,H] e4m3 with out_scale [T,ceil(H/128)] fp32; with a
    residual [T,H], x + residual is normed and written to sum_out."""
    shape, stride = _rows(x)
    T, H = shape
    dt, dev = x.dtype, x.get_device()
    args = (_code(dt), x.data_ptr(), stride, None if residual is None else _dense(residual, dt, shape, dev),
            _dense(weight, dt, (H,), dev), T, H, eps, None if sum_out is None else _dense(sum_out, dt, shape, dev),
            None if out is None else _dense(out, dt, shape, dev),
            None if out_fp8 is None else _dense(out_fp8, _E4M3, shape, dev),
            None if out_scale is None else _dense(out_scale, _FP32, (T, (H + 127) // 128), dev), _on(stream, dev))
    fn = (_lib or lib()).orthrus_rmsnorm
    rc = fn(*args) if _current_device() == dev else _elsewhere(dev, fn, args)
    if rc:
        _check("orthrus_rmsnorm", rc)


def orthrus_quantize_fp8(x: torch.Tensor, out_fp8: torch.Tensor, out_scale: torch.Tensor, stream=None) -> None:
    """x [T,H] (rows may be strided) -> out_fp8 [T,H] e4m3 and out_scale
    [T,ceil(H/128)] fp32, one scale per row and 128 columns."""
    shape, stride = _rows(x)
    T, H = shape
    dev = x.get_device()
    args = (_code(x.dtype), x.data_ptr(), stride, T, H, _dense(out_fp8, _E4M3, shape, dev),
            _dense(out_scale, _FP32, (T, (H + 127) // 128), dev), _on(stream, dev))
    fn = (_lib or lib()).orthrus_quantize_fp8
    rc = fn(*args) if _current_device() == dev else _elsewhere(dev, fn, args)
    if rc:
        _check("orthrus_quantize_fp8", rc)


def orthrus_fp8_matmul(a: torch.Tensor, a_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                       out: torch.Tensor, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """a [M,K] and w [N,K] e4m3 with scales a_scale [M,ceil(K/128)] and w_scale
    [ceil(N/128),ceil(K/128)] fp32 -> out [M,N] (bf16, fp16 or fp32) = a w^T."""
    M, K = a.shape
    N = w.shape[0]
    nk = (K + 127) // 128
    dev = a.get_device()
    args = (_dense(a, _E4M3, None, dev), _dense(a_scale, _FP32, (M, nk), dev), _dense(w, _E4M3, (N, K), dev),
            _dense(w_scale, _FP32, ((N + 127) // 128, nk), dev), M, N, K, _code(out.dtype),
            _dense(out, None, (M, N), dev), None if status is None else _dense(status, torch.int32, None, dev),
            _on(stream, dev))
    fn = (_lib or lib()).orthrus_fp8_matmul
    rc = fn(*args) if _current_device() == dev else _elsewhere(dev, fn, args)
    if rc:
        _check("orthrus_fp8_matmul", rc)


def orthrus_rope_table(rot_dim: int, theta: float, kind: int = ROPE_PLAIN, factor: float = 1.0,
                       orig_len: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(turns, magnitude): turns per position of the rot_dim / 2 pairs as a CPU
    float64 tensor (upload it once), and the factor on the rotated values."""
    turns = torch.empty(max(rot_dim // 2, 1), dtype=torch.float64)
    mag = ctypes.c_float()
    rc = lib().orthrus_rope_table(kind, rot_dim, theta, factor, orig_len, beta_fast, beta_slow, turns.data_ptr(),
                                  ctypes.addressof(mag))
    _check("orthrus_rope_table", rc)
    return turns, mag.value


@functools.lru_cache(maxsize=256)
def _stride_array(*strides):
    """HOST array of eight strides (read during the call only)."""
    return (ctypes.c_int64 * 8)(*strides)


def _token_strides(t: torch.Tensor):
    """(token stride, head stride) of [T, H, D] or [B, K, H, D]: tokens evenly
    spaced, a head's elements contiguous."""
    s, n = t.stride(), t.shape
    if s[-1] != 1 and n[-1] > 1:
        raise ValueError("a head's elements have to be contiguous")
    if len(s) == 3:
        return s[0], s[1]
    if n[1] == 1:
        return s[0], s[2]
    if n[0] > 1 and s[0] != n[1] * s[1]:
        raise ValueError("tokens have to be evenly spaced over sequences and block slots")
    return s[1], s[2]


def orthrus_rope(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, turns: torch.Tensor,
                 q_out: torch.Tensor, k_out: Optional[torch.Tensor] = None, layout: int = ROPE_HALF,
                 magnitude: float = 1.0, q_norm: Optional[torch.Tensor] = None,
                 k_norm: Optional[torch.Tensor] = None, eps: float = 1e-6, stream=None) -> None:
    """q [T,Hq,D], k [T,Hkv,D] or None (tokens and heads may be strided) at
    positions [T] int32 -> q_out, k_out (may be q and k themselves).  turns
    [rot/2] float64 on the device and magnitude: from orthrus_rope_table."""
    T, Hq, D = q.shape
    dt, dev = q.dtype, q.get_device()
    pq, pqo = _strided(q, dt, q.shape, dev), _strided(q_out, dt, q.shape, dev)
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out go together")
    if k is not None:
        Hkv = k.shape[1]
        pk, pko = _strided(k, dt, (T, Hkv, D), dev), _strided(k_out, dt, (T, Hkv, D), dev)
        st = _stride_array(*_token_strides(q), *_token_strides(q_out), *_token_strides(k), *_token_strides(k_out))
    else:
        Hkv, pk, pko = 0, None, None
        st = _stride_array(*_token_strides(q), *_token_strides(q_out), 0, 0, 0, 0)
    args = (_code(dt), layout, pq, pqo, pk, pko, st, _dense(positions, torch.int32, (T,), dev),
            _dense(turns, torch.float64, None, dev), magnitude, T, Hq, Hkv, D, 2 * turns.numel(),
            None if q_norm is None else _dense(q_norm, dt, (D,), dev),
            None if k_norm is None else _dense(k_norm, dt, (D,), dev), eps, _on(stream, dev))
    fn = (_lib or lib()).orthrus_rope
    rc = fn(*args) if _current_device() == dev else _elsewhere(dev, fn, args)
    if rc:
        _check("orthrus_rope", rc)


def orthrus_rope_append(q: Optional[torch.Tensor], k: Optional[torch.Tensor], v: Optional[torch.Tensor],
                        turns: torch.Tensor, q_out: Optional[torch.Tensor], k_pages: torch.Tensor,
                        v_pages: Optional[torch.Tensor], block_table: torch.Tensor, ctx_lens: torch.Tensor,
                        layout: int = ROPE_HALF, magnitude: float = 1.0, q_norm: Optional[torch.Tensor] = None,
                        k_norm: Optional[torch.Tensor] = None, eps: float = 1e-6,
                        K: Optional[int] = None, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q [B,K,Hq,D], k and v [B,K,Hkv,D] (tokens and heads may be strided) at
    positions ctx_lens[b] + i -> q_out, and rows of k_pages / v_pages
    [num_pages,Hkv,page_size,D] through block_table [B,max_pages].  With k and v
    None the keys already in those rows are rotated in place (give K where q is
    None too)."""
    P, Hkv, page, D = k_pages.shape
    B, max_pages = block_table.shape
    dt, dev = k_pages.dtype, k_pages.get_device()
    if (q is None) != (q_out is None) or (k is None) != (v is None):
        raise ValueError("q and q_out, and k and v, go together")
    if q is not None:
        K, Hq = q.shape[1], q.shape[2]
        pq, pqo = _strided(q, dt, (B, K, Hq, D), dev), _strided(q_out, dt, (B, K, Hq, D), dev)
        st = _token_strides(q) + _token_strides(q_out)
    else:
        Hq, pq, pqo, st = 0, None, None, (0, 0, 0, 0)
        if k is not None:
            K = k.shape[1]
    if K is None:
        raise ValueError("the number of tokens per sequence is not known: give K")
    if k is not None:
        if v_pages is None:
            raise ValueError("v needs v_pages")
        pk, pv = _strided(k, dt, (B, K, Hkv, D), dev), _strided(v, dt, (B, K, Hkv, D), dev)
        st = _stride_array(*st, *_token_strides(k), *_token_strides(v))
    else:
        pk, pv = None, None
        st = _stride_array(*st, 0, 0, 0, 0)
    args = (_code(dt), layout, pq, pqo, pk, pv, st, _dense(turns, torch.float64, None, dev), magnitude, B, K, Hq, Hkv, D,
            2 * turns.numel(), None if q_norm is None else _dense(q_norm, dt, (D,), dev),
            None if k_norm is None else _dense(k_norm, dt, (D,), dev), eps, _dense(k_pages, dt, None, dev),
            None if v_pages is None else _dense(v_pages, dt, k_pages.shape, dev), P, page,
            _dense(block_table, torch.int32, None, dev), max_pages, _dense(ctx_lens, torch.int32, (B,), dev),
            None if status is None else _dense(status, torch.int32, None, dev), _on(stream, dev))
    fn = (_lib or lib()).orthrus_rope_append
    rc = fn(*args) if _current_device() == dev else _elsewhere(dev, fn, args)
    if rc:
        _check("orthrus_rope_append", rc)


def orthrus_paged_attn_workspace_size(B: int, Hq: int, Hkv: int, D: int) -> int:
    return int(lib().orthrus_paged_attn_workspace_size(B, Hq, Hkv, D))


def orthrus_paged_attn(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
                       ctx_lens: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor, n_new: int = 0,
                       scale: float = 0.0, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q [B,Hq,D], pages [num_pages,Hkv,page_size,D] (bf16 or fp16), block_table
    [B,max_pages] int32, ctx_lens [B] int32 -> out [B,Hq,D]: attention of one
    token per sequence over keys [0, ctx_lens[b] + n_new)."""
    B, Hq, D = q.shape
    P, Hkv, page, Dk = k_pages.shape
    max_pages = block_table.shape[1]
    if Dk != D:
        raise ValueError(f"head size {D} of q and {Dk} of the pages")
    dt, dev = q.dtype, q.get_device()
    args = (_code(dt), _dense(q, dt, None, dev), _dense(k_pages, dt, None, dev), _dense(v_pages, dt, k_pages.shape, dev),
            _dense(block_table, torch.int32, (B, max_pages), dev), _dense(ctx_lens, torch.int32, (B,), dev), n_new, B, Hq,
            Hkv, D, P, page, max_pages, scale, _dense(out, dt, q.shape, dev), _dense(workspace, None, None, dev),
            workspace.nbytes, None if status is None else _dense(status, torch.int32, None, dev), _on(stream, dev))
    fn = (_lib or lib()).orthrus_paged_attn
    rc = fn(*args) if _current_device() == dev else _elsewhere(dev, fn, args)
    if rc:
        _check("orthrus_paged_attn", rc)
