"""PyTorch-facing API over the C ABI: tensors in, tensors out.

PyTorch only provides device memory, the current stream and autograd; every
step of the computation runs in the library's CUDA kernels. Nothing here
computes attention, and nothing falls back to another implementation: an
unsupported call raises (FFPA docs, "Backends Overview" page, "Automatic SDPA
fallback": unsupported dtype and similar raise NotImplementedError /
ValueError, no silent fallback).

Layouts (FFPA docs, "CuTe-DSL Backend" page): dense q [B, Hq, Nq, D],
k/v [B, Hkv, Nkv, D]; packed varlen q [Tq, Hq, D], k/v [Tk, Hkv, D] with
int32 cu_seqlens; LSE is fp32 [B, Hq, Nq] (dense) or [Hq, Tq] (varlen).

Dense tensors are passed as strided views (ffpa_view) with no copy whenever
the head dim is the innermost, unit-stride dimension and the other strides are
multiples of 8 elements: contiguous [B, H, N, D] tensors, ``x.transpose(1, 2)``
of a [B, N, H, D] projection output, slices of a fused QKV buffer. Any other
layout is copied to a contiguous tensor first. Dense outputs default to the
layout of the matching input (``torch.empty_like``). Varlen inputs are made
contiguous.
"""
from __future__ import annotations

import functools
import math

import torch

from . import _ffi

_DTYPES = {torch.bfloat16: _ffi.BF16, torch.float16: _ffi.FP16}


def _dt(x: torch.Tensor) -> int:
    if x.dtype not in _DTYPES:
        raise NotImplementedError(f"dtype {x.dtype}: only torch.bfloat16 and torch.float16 are supported")
    return _DTYPES[x.dtype]


def _prep(*xs):
    out = []
    for x in xs:
        if not x.is_cuda:
            raise ValueError("tensors must be on a CUDA device")
        out.append(x.contiguous())
    dt = out[0].dtype
    for x in out[1:]:
        if x.dtype != dt:
            raise ValueError(f"mixed dtypes {dt} and {x.dtype}")
    return out


def _viewable(x: torch.Tensor) -> bool:
    """True when the dense 4-D tensor can be handed to the kernels as an ffpa_view."""
    if x.dim() != 4 or x.stride(-1) != 1 or x.data_ptr() % 16 != 0:
        return False
    for size, stride in zip(x.shape[:3], x.stride()[:3]):
        if stride < 0 or stride % 8 != 0 or (size > 1 and stride == 0):
            return False
    return True


def _dense(*xs):
    """Dense inputs: checked, and copied only when no view of them fits the ABI."""
    out = []
    for x in xs:
        if not x.is_cuda:
            raise ValueError("tensors must be on a CUDA device")
        out.append(x if _viewable(x) else x.contiguous())
    dt = out[0].dtype
    for x in out[1:]:
        if x.dtype != dt:
            raise ValueError(f"mixed dtypes {dt} and {x.dtype}")
    return out


def _out_like(x: torch.Tensor) -> torch.Tensor:
    y = torch.empty_like(x)
    return y if _viewable(y) else torch.empty(x.shape, dtype=x.dtype, device=x.device)


def _view(x: torch.Tensor) -> _ffi.View:
    if not _viewable(x):
        raise ValueError(f"output of shape {tuple(x.shape)} and strides {x.stride()} is not an ffpa_view "
                         "(head dim innermost with unit stride, other strides multiples of 8 elements)")
    return _ffi.View(x.data_ptr(), x.stride(0), x.stride(1), x.stride(2))


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _scale(scale, D):
    return float(1.0 / math.sqrt(D)) if scale is None else float(scale)


# ----------------------------------------------------------------- dense
def fwd(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None):
    """Dense forward through ffpa_fwd_strided (views, no copy). Returns (o, lse)."""
    if q.dim() != 4 or k.dim() != 4 or v.shape != k.shape:
        raise ValueError("expected q [B,Hq,Nq,D], k and v [B,Hkv,Nkv,D]")
    q, k, v = _dense(q, k, v)
    B, Hq, Nq, D = q.shape
    Bk, Hkv, Nkv, Dk = k.shape
    if Bk != B or Dk != D:
        raise ValueError("q and k/v disagree on B or D")
    o = _out_like(q) if out is None else out
    l = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device) if lse is None else lse
    if not l.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [B, Hq, Nq] tensor")
    st = _ffi.ffpa_fwd_strided(_dt(q), _view(q), _view(k), _view(v), _view(o), l.data_ptr(),
                               B, Hq, Hkv, Nq, Nkv, D, int(bool(causal)), _scale(scale, D), _stream())
    _ffi.raise_for(st, "ffpa_fwd_strided")
    return o, l


DECODE_ROWS = 16    # query rows of one kv head's group per decode CTA
DECODE_MAX_NQ = 8   # attention() sends Nq below this to the decode path


def decode_supported(q, k) -> bool:
    """True when ffpa_decode_fwd takes this problem (D % 64 == 0, grid within limits)."""
    B, Hq, Nq, D = q.shape
    Hkv = k.shape[1]
    if Hkv <= 0 or Hq % Hkv != 0 or D % 64 != 0:
        return False
    return B * Hkv * -(-(Hq // Hkv) * Nq // DECODE_ROWS) <= 65535 * 65535


def decode_fwd(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None, workspace=None):
    """Decode / short-query forward through ffpa_decode_fwd (split over the keys).
    Same result as fwd(); raises NotImplementedError outside decode_supported()."""
    if q.dim() != 4 or k.dim() != 4 or v.shape != k.shape:
        raise ValueError("expected q [B,Hq,Nq,D], k and v [B,Hkv,Nkv,D]")
    q, k, v = _dense(q, k, v)
    B, Hq, Nq, D = q.shape
    _, Hkv, Nkv, _ = k.shape
    o = _out_like(q) if out is None else out
    l = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device) if lse is None else lse
    ws_bytes = int(_ffi.ffpa_decode_workspace_bytes(_dt(q), B, Hq, Hkv, Nq, Nkv, D))
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=q.device)
    st = _ffi.ffpa_decode_fwd(_dt(q), _view(q), _view(k), _view(v), _view(o), l.data_ptr(), workspace.data_ptr(),
                              workspace.numel() * workspace.element_size(), B, Hq, Hkv, Nq, Nkv, D,
                              int(bool(causal)), _scale(scale, D), _stream())
    _ffi.raise_for(st, "ffpa_decode_fwd")
    return o, l


def fp8_supported(D: int) -> bool:
    """Head dims of the FP8 forward: every multiple of 32 in [64, 1024]."""
    return D % 32 == 0 and 64 <= D <= 1024


def fp8_workspace(q, k):
    """Device scratch for fwd_fp8 (uint8, 256-byte aligned by the allocator)."""
    B, Hq, Nq, D = q.shape
    _, Hkv, Nkv, _ = k.shape
    n = int(_ffi.ffpa_fp8_workspace_bytes(B, Hq, Hkv, Nq, Nkv, D))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)


def _fp8_args(q, k, v):
    if q.dim() != 4 or k.dim() != 4 or v.shape != k.shape:
        raise ValueError("expected q [B,Hq,Nq,D], k and v [B,Hkv,Nkv,D]")
    return _dense(q, k, v)


def fp8_quantize(q, k, v, workspace=None):
    """Runs only the e4m3 quantization; returns (workspace, {name: view}) with
    q8, k8 (uint8 codes), v8t ([B, Hkv, D, ldv] codes of V^T) and the fp32 scales sq, sk, sv.
    The code views cover the D real columns; the workspace pads each code row
    to Dp = D rounded up to 128 with zero codes (q8_padded, k8_padded, v8t_padded)."""
    q, k, v = _fp8_args(q, k, v)
    B, Hq, Nq, D = q.shape
    _, Hkv, Nkv, _ = k.shape
    ws = fp8_workspace(q, k) if workspace is None else workspace
    st = _ffi.ffpa_fp8_quantize(_dt(q), _view(q), _view(k), _view(v), ws.data_ptr(), ws.numel(),
                                B, Hq, Hkv, Nq, Nkv, D, _stream())
    _ffi.raise_for(st, "ffpa_fp8_quantize")
    off = _ffi.ffpa_fp8_workspace_layout(B, Hq, Hkv, Nq, Nkv, D)
    ldv = off[6]

    def region(i, n, shape, dtype=torch.uint8):
        t = ws[off[i]:off[i] + n * (4 if dtype == torch.float32 else 1)]
        return t.view(dtype).view(shape)

    Dp = (D + 127) // 128 * 128
    views = {
        "q8_padded": region(0, B * Hq * Nq * Dp, (B, Hq, Nq, Dp)),
        "k8_padded": region(1, B * Hkv * Nkv * Dp, (B, Hkv, Nkv, Dp)),
        "v8t_padded": region(2, B * Hkv * Dp * ldv, (B, Hkv, Dp, ldv)),
        "sq": region(3, B * Hq, (B, Hq), torch.float32),
        "sk": region(4, B * Hkv, (B, Hkv), torch.float32),
        "sv": region(5, B * Hkv, (B, Hkv), torch.float32),
    }
    views["q8"] = views["q8_padded"][..., :D]
    views["k8"] = views["k8_padded"][..., :D]
    views["v8t"] = views["v8t_padded"][:, :, :D]
    return ws, views


def fwd_fp8(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None, workspace=None):
    """FP8 (e4m3) forward through ffpa_fwd_fp8: bf16/fp16 in, O in the input
    dtype and fp32 LSE out; D a multiple of 32 in [64, 1024]. Returns (o, lse)."""
    q, k, v = _fp8_args(q, k, v)
    B, Hq, Nq, D = q.shape
    _, Hkv, Nkv, _ = k.shape
    o = _out_like(q) if out is None else out
    l = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device) if lse is None else lse
    ws = fp8_workspace(q, k) if workspace is None else workspace
    st = _ffi.ffpa_fwd_fp8(_dt(q), _view(q), _view(k), _view(v), _view(o), l.data_ptr(), ws.data_ptr(), ws.numel(),
                           B, Hq, Hkv, Nq, Nkv, D, int(bool(causal)), _scale(scale, D), _stream())
    _ffi.raise_for(st, "ffpa_fwd_fp8")
    return o, l


def fwd_fp8_quantized(workspace, shape_q, shape_k, dtype, causal: bool = False, scale: float | None = None,
                      out=None, lse=None):
    """The FP8 attention alone, on a workspace that fp8_quantize filled for q of
    shape_q and k/v of shape_k (inputs quantized once, attended many times)."""
    B, Hq, Nq, D = shape_q
    _, Hkv, Nkv, _ = shape_k
    o = torch.empty(shape_q, dtype=dtype, device=workspace.device) if out is None else out
    l = torch.empty((B, Hq, Nq), dtype=torch.float32, device=workspace.device) if lse is None else lse
    st = _ffi.ffpa_fwd_fp8_quantized(_dt(o), _view(o), l.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                     B, Hq, Hkv, Nq, Nkv, D, int(bool(causal)), _scale(scale, D), _stream())
    _ffi.raise_for(st, "ffpa_fwd_fp8_quantized")
    return o, l


# Default cap of the backward workspace bwd() and varlen_bwd() allocate: the
# stored P^T / dS^T tiles of every head when they fit in it (8.6 GB at
# B1 H32 N8192 D512), else of as many kv groups per chunk as fit. A fixed
# size, so that the path a call takes never depends on what else is allocated.
BWD_WORKSPACE_BUDGET = 16 << 30


def bwd_workspace_bytes(q, k, causal: bool | None = None, budget: int | None = None) -> int:
    """Backward workspace bytes: the row statistics only (causal None); with
    room for the stored dS and P tiles of every head where that path applies
    (budget None: ffpa_bwd_workspace_bytes_ds); or the largest useful size
    within `budget` bytes (ffpa_bwd_workspace_bytes_budget: the tiles of every
    head, else of a chunk of kv groups, else the row statistics)."""
    B, Hq, Nq, D = q.shape
    _, Hkv, Nkv, _ = k.shape
    if causal is None:
        return int(_ffi.ffpa_bwd_workspace_bytes(_dt(q), B, Hq, Hkv, Nq, Nkv, D))
    if budget is None:
        return int(_ffi.ffpa_bwd_workspace_bytes_ds(_dt(q), B, Hq, Hkv, Nq, Nkv, D, int(bool(causal))))
    return int(_ffi.ffpa_bwd_workspace_bytes_budget(_dt(q), B, Hq, Hkv, Nq, Nkv, D, int(bool(causal)),
                                                     int(budget)))


def bwd_workspace(q, k, causal: bool, budget: int = BWD_WORKSPACE_BUDGET):
    """A backward workspace of the largest useful size within `budget` bytes."""
    n = bwd_workspace_bytes(q, k, causal, budget)
    return torch.empty(max(n, 1), dtype=torch.uint8, device=q.device)


def bwd(q, k, v, o, lse, dout, causal: bool = False, scale: float | None = None, workspace=None,
        dq=None, dk=None, dv=None, stages: int = 15):
    """Dense backward through ffpa_bwd_strided (views, no copy), or ffpa_bwd_stages
    for a subset of its launches (bit 0 preprocess, bit 1 dV, bit 2 dQ, bit 3 dK,
    bit 4 dQ from the dS a dK stage stored, bit 5 dV storing P / dK reading it;
    contiguous tensors). Without a workspace, one of at most
    BWD_WORKSPACE_BUDGET bytes is allocated (bwd_workspace): the stored-tile
    path for every head, or in chunks of kv groups, where it applies. Returns
    (dq, dk, dv)."""
    q, k, v, o, dout = _dense(q, k, v, o, dout)
    lse = lse.contiguous()
    B, Hq, Nq, D = q.shape
    _, Hkv, Nkv, _ = k.shape
    if workspace is None:
        workspace = bwd_workspace(q, k, causal)
    dq = _out_like(q) if dq is None else dq
    dk = _out_like(k) if dk is None else dk
    dv = _out_like(v) if dv is None else dv
    tail = (workspace.data_ptr(), workspace.numel() * workspace.element_size(),
            B, Hq, Hkv, Nq, Nkv, D, int(bool(causal)), _scale(scale, D))
    if stages == 15:
        st = _ffi.ffpa_bwd_strided(_dt(q), _view(q), _view(k), _view(v), _view(o), lse.data_ptr(), _view(dout),
                                   _view(dq), _view(dk), _view(dv), *tail, _stream())
        _ffi.raise_for(st, "ffpa_bwd_strided")
    else:
        ts = [x.contiguous() for x in (q, k, v, o, dout)]
        for name, x in (("dq", dq), ("dk", dk), ("dv", dv)):
            if not x.is_contiguous():
                raise ValueError(f"{name} must be contiguous when stages != 15")
        st = _ffi.ffpa_bwd_stages(_dt(q), *(x.data_ptr() for x in ts[:4]), lse.data_ptr(), ts[4].data_ptr(),
                                  dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), *tail, int(stages), _stream())
        _ffi.raise_for(st, "ffpa_bwd_stages")
    return dq, dk, dv


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, causal, scale):
        # short queries (Nq < 8, decode) take the split-KV path; the backward
        # is the same either way (O and LSE have the same meaning)
        if q.dim() == 4 and 0 < q.shape[2] < DECODE_MAX_NQ and decode_supported(q, k):
            o, lse = decode_fwd(q, k, v, causal, scale)
        else:
            o, lse = fwd(q, k, v, causal, scale)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.causal, ctx.scale = causal, scale
        return o, lse

    @staticmethod
    def backward(ctx, do, dlse):
        q, k, v, o, lse = ctx.saved_tensors
        dq, dk, dv = bwd(q, k, v, o, lse, do, ctx.causal, ctx.scale)
        return dq, dk, dv, None, None


def attention(q, k, v, causal: bool = False, scale: float | None = None, return_lse: bool = False):
    """O = softmax(scale * Q K^T [bottom-right causal]) V, differentiable w.r.t. q, k, v.

    The gradient of the returned LSE is not propagated (it is an auxiliary output).
    """
    o, lse = _Attention.apply(q, k, v, bool(causal), scale)
    return (o, lse) if return_lse else o


# ----------------------------------------------------------------- varlen
def _cu(cu, device):
    if cu is None:
        return None
    if cu.dtype != torch.int32:
        raise ValueError("cu_seqlens must be int32")
    return cu.to(device).contiguous()


def varlen_fwd(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, causal=False, scale=None):
    """Packed forward through ffpa_varlen_fwd. Returns (o [Tq,Hq,D], lse [Hq,Tq])."""
    q, k, v = _prep(q, k, v)
    Tq, Hq, D = q.shape
    Tk, Hkv, _ = k.shape
    cq, ck = _cu(cu_seqlens_q, q.device), _cu(cu_seqlens_k, q.device)
    batch = cq.numel() - 1
    o = torch.empty_like(q)
    lse = torch.empty((Hq, Tq), dtype=torch.float32, device=q.device)
    st = _ffi.ffpa_varlen_fwd(_dt(q), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                              cq.data_ptr(), ck.data_ptr(), batch, Tq, Tk, int(max_seqlen_q), int(max_seqlen_k),
                              Hq, Hkv, D, int(bool(causal)), _scale(scale, D), _stream())
    _ffi.raise_for(st, "ffpa_varlen_fwd")
    return o, lse


def varlen_fp8_workspace(q, k, cu_seqlens_q, max_seqlen_q, max_seqlen_k):
    """Device scratch for varlen_fwd_fp8 (uint8, 256-byte aligned by the allocator)."""
    Tq, Hq, D = q.shape
    Tk, Hkv, _ = k.shape
    batch = cu_seqlens_q.numel() - 1
    n = int(_ffi.ffpa_varlen_fp8_workspace_bytes(batch, Tq, Tk, int(max_seqlen_q), int(max_seqlen_k), Hq, Hkv, D))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)


def varlen_fwd_fp8(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, causal=False, scale=None,
                   workspace=None):
    """Packed FP8 (e4m3) forward through ffpa_varlen_fwd_fp8: each sequence quantized
    per head as fwd_fp8 quantizes a batch entry. Returns (o [Tq,Hq,D], lse [Hq,Tq])."""
    q, k, v = _prep(q, k, v)
    Tq, Hq, D = q.shape
    Tk, Hkv, _ = k.shape
    cq, ck = _cu(cu_seqlens_q, q.device), _cu(cu_seqlens_k, q.device)
    batch = cq.numel() - 1
    o = torch.empty_like(q)
    lse = torch.empty((Hq, Tq), dtype=torch.float32, device=q.device)
    ws = varlen_fp8_workspace(q, k, cq, max_seqlen_q, max_seqlen_k) if workspace is None else workspace
    st = _ffi.ffpa_varlen_fwd_fp8(_dt(q), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                  cq.data_ptr(), ck.data_ptr(), batch, Tq, Tk, int(max_seqlen_q), int(max_seqlen_k),
                                  Hq, Hkv, D, int(bool(causal)), _scale(scale, D), ws.data_ptr(), ws.numel(),
                                  _stream())
    _ffi.raise_for(st, "ffpa_varlen_fwd_fp8")
    return o, lse


def varlen_workspace_bytes(q, k, cu_seqlens_q, max_seqlen_q, max_seqlen_k, causal: bool,
                           budget: int = BWD_WORKSPACE_BUDGET) -> int:
    """Largest useful packed-backward workspace within `budget` bytes
    (ffpa_varlen_bwd_workspace_bytes_budget)."""
    Tq, Hq, D = q.shape
    Tk, Hkv, _ = k.shape
    batch = cu_seqlens_q.numel() - 1
    return int(_ffi.ffpa_varlen_bwd_workspace_bytes_budget(_dt(q), batch, Tq, Tk, int(max_seqlen_q),
                                                            int(max_seqlen_k), Hq, Hkv, D, int(bool(causal)),
                                                            int(budget)))


def varlen_bwd(q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, causal=False,
               scale=None, workspace=None):
    """Packed backward through ffpa_varlen_bwd. Without a workspace, one of at
    most BWD_WORKSPACE_BUDGET bytes is allocated (the stored-tile path for
    every head, or in chunks of kv groups, where it applies). Returns
    (dq, dk, dv)."""
    q, k, v, o, dout = _prep(q, k, v, o, dout)
    lse = lse.contiguous()
    Tq, Hq, D = q.shape
    Tk, Hkv, _ = k.shape
    cq, ck = _cu(cu_seqlens_q, q.device), _cu(cu_seqlens_k, q.device)
    batch = cq.numel() - 1
    sizes = (_dt(q), batch, Tq, Tk, int(max_seqlen_q), int(max_seqlen_k), Hq, Hkv, D)
    if workspace is None:
        n = int(_ffi.ffpa_varlen_bwd_workspace_bytes_budget(*sizes, int(bool(causal)), BWD_WORKSPACE_BUDGET))
        workspace = torch.empty(max(n, 1), dtype=torch.uint8, device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    st = _ffi.ffpa_varlen_bwd(_dt(q), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                              dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), cq.data_ptr(),
                              ck.data_ptr(), batch, Tq, Tk, int(max_seqlen_q), int(max_seqlen_k), Hq, Hkv, D,
                              int(bool(causal)), _scale(scale, D), workspace.data_ptr(),
                              workspace.numel() * workspace.element_size(), _stream())
    _ffi.raise_for(st, "ffpa_varlen_bwd")
    return dq, dk, dv


class _VarlenAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cq, ck, mq, mk, causal, scale):
        o, lse = varlen_fwd(q, k, v, cq, ck, mq, mk, causal, scale)
        ctx.save_for_backward(q, k, v, o, lse, cq, ck)
        ctx.args = (mq, mk, causal, scale)
        return o, lse

    @staticmethod
    def backward(ctx, do, dlse):
        q, k, v, o, lse, cq, ck = ctx.saved_tensors
        mq, mk, causal, scale = ctx.args
        dq, dk, dv = varlen_bwd(q, k, v, o, lse, do, cq, ck, mq, mk, causal, scale)
        return dq, dk, dv, None, None, None, None, None, None


def varlen_attention(q, k, v, cu_seqlens_q, cu_seqlens_k=None, max_seqlen_q=None, max_seqlen_k=None,
                     causal: bool = False, scale: float | None = None, return_lse: bool = False):
    """Packed-THD attention (FFPA docs, "CuTe-DSL Backend" page, "Varlen (packed THD) API").

    cu_seqlens_k=None means cu_seqlens_k = cu_seqlens_q. When max_seqlen_* is
    None it is read from cu_seqlens (one device-to-host copy).
    """
    if cu_seqlens_k is None:
        cu_seqlens_k = cu_seqlens_q
    if max_seqlen_q is None:
        max_seqlen_q = int((cu_seqlens_q[1:] - cu_seqlens_q[:-1]).max().item()) if cu_seqlens_q.numel() > 1 else 0
    if max_seqlen_k is None:
        max_seqlen_k = int((cu_seqlens_k[1:] - cu_seqlens_k[:-1]).max().item()) if cu_seqlens_k.numel() > 1 else 0
    cq, ck = _cu(cu_seqlens_q, q.device), _cu(cu_seqlens_k, q.device)
    o, lse = _VarlenAttention.apply(q, k, v, cq, ck, int(max_seqlen_q), int(max_seqlen_k), bool(causal), scale)
    return (o, lse) if return_lse else o


# ----------------------------------------------------------------- 4-bit K/V cache
KV4_TILE = 576  # bytes of a cache tile: 16 tokens x 64 head dims, 512 of codes and 64 of scales


def kv4_cache(num_pages: int, page_size: int, Hkv: int, D: int, device="cuda") -> torch.Tensor:
    """A zeroed paged 4-bit K/V cache (ffpa_kv4_cache in include/ffpa.h): uint8
    [num_pages, 2 (K, V), Hkv, page_size / 16, D / 64, 576]. page_size is a multiple
    of 16 (tokens per page), D a multiple of 64 in [64, 1024]."""
    if page_size <= 0 or page_size % 16 != 0:
        raise ValueError(f"page_size {page_size} must be a positive multiple of 16")
    if D % 64 != 0 or not 64 <= D <= 1024:
        raise NotImplementedError(f"head dim {D}: the 4-bit cache takes multiples of 64 in [64, 1024]")
    return torch.zeros((num_pages, 2, Hkv, page_size // 16, D // 64, KV4_TILE), dtype=torch.uint8, device=device)


# The 4-bit cache's calls run once per layer and token on tensors of a few
# kilobytes, where the host's part is what a call costs: each property of a
# tensor is read once, and the device is entered only when it is not current.
def _kv4(cache, block_table, B: int):
    """The ffpa_kv4_cache of a cache tensor and a block table [B, max_blocks], with Hkv, D and the device."""
    shape, dev = cache.shape, cache.device
    if cache.dtype is not torch.uint8 or len(shape) != 6 or shape[1] != 2 or shape[5] != KV4_TILE:
        raise ValueError(f"expected a cache of kv4_cache(), got {cache.dtype} {tuple(shape)}")
    if dev.type != "cuda" or not cache.is_contiguous():
        raise ValueError("the cache must be a contiguous tensor on a CUDA device")
    rows, stride = block_table.shape, block_table.stride()
    if block_table.dtype is not torch.int32 or len(rows) != 2 or rows[0] != B:
        raise ValueError(f"expected an int32 block_table [{B}, max_blocks], got {block_table.dtype} {tuple(rows)}")
    if block_table.device != dev:
        raise ValueError("block_table and cache are on different devices")
    blocks = rows[1]
    if blocks > 1 and stride[1] != 1 or B > 1 and stride[0] < blocks:
        raise ValueError(f"block_table's rows must be contiguous, got strides {stride}")
    c = _ffi.Kv4Cache(cache.data_ptr(), shape[0], 16 * shape[3], block_table.data_ptr(), blocks,
                      stride[0] if B > 1 else blocks)
    return c, shape[2], 64 * shape[4], dev


def _lengths(x, n: int, name: str, device) -> int | None:
    """The address of an optional int32 [n] tensor of lengths on `device`."""
    if x is None:
        return None
    if x.dtype is not torch.int32 or x.shape != (n,) or not x.is_contiguous() or x.device != device:
        raise ValueError(f"{name} must be a contiguous int32 [{n}] tensor on {device}, got {x.dtype} "
                         f"{tuple(x.shape)} on {x.device}")
    return x.data_ptr()


def _kv4_pair(k, v, dims: int, Hkv: int, D: int, device):
    """The shape of a k, v pair that fits a cache."""
    shape = k.shape
    if len(shape) != dims or v.shape != shape or shape[1] != Hkv or shape[-1] != D:
        raise ValueError(f"k {tuple(shape)} and v {tuple(v.shape)} do not match a cache of Hkv={Hkv}, D={D}")
    if k.device != device or v.device != device:
        raise ValueError("k, v and the cache must be on one device")
    if k.dtype != v.dtype:
        raise ValueError(f"mixed dtypes {k.dtype} and {v.dtype}")
    return shape


def _view_or_none(x):
    """The ffpa_view of a dense 4-D tensor, or None where it has none (as _viewable)."""
    (B, H, N, _), (sb, sh, sn, sd), p = x.shape, x.stride(), x.data_ptr()
    if sd != 1 or p & 15 or (sb | sh | sn) & 7 or sb < 0 or sh < 0 or sn < 0:
        return None
    if B > 1 and sb == 0 or H > 1 and sh == 0 or N > 1 and sn == 0:
        return None
    return _ffi.View(p, sb, sh, sn)


def _in_view(x):
    """(tensor, its ffpa_view) of an input, copied only where no view of it fits."""
    w = _view_or_none(x)
    if w is None:
        x = x.clone(memory_format=torch.contiguous_format)  # what is contiguous may begin off 16 bytes
        w = _view(x)
    return x, w


def _in_packed(x):
    """A packed input, copied only where it is not contiguous from 16 bytes on."""
    return x if x.is_contiguous() and not x.data_ptr() & 15 else x.clone(memory_format=torch.contiguous_format)


def _out_view(x):
    w = _view_or_none(x)
    return _view(x) if w is None else w  # _view() says what is wrong


def _elsewhere(device) -> bool:
    """True when `device` is not the current one, and a call has to enter it."""
    return device.index != torch.cuda.current_device()


# Not a public name of torch, but a tenth of torch.cuda.current_stream's time (0.1 us against 1.1; a token written and
# read back 22.5 against 26.3): that one takes its place in a torch without it.
_raw_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(device) -> int:
    """The current stream of a device."""
    if _raw_stream_of is None:
        return torch.cuda.current_stream(device.index).cuda_stream
    return _raw_stream_of(device.index)


def kv4_write(cache, block_table, k, v, start=None, count=None) -> None:
    """Quantises new tokens into the cache through ffpa_kv4_write (views, no copy):
    row i of sequence b becomes cached token start[b] + i, for i < count[b].

    k, v: [B, Hkv, N, D]; block_table: int32 [B, max_blocks]; start, count: int32 [B]
    on the device (None: 0 and N)."""
    B = k.shape[0]
    c, Hkv, D, dev = _kv4(cache, block_table, B)
    N = _kv4_pair(k, v, 4, Hkv, D, dev)[2]
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return kv4_write(cache, block_table, k, v, start, count)
    (k, wk), (v, wv) = _in_view(k), _in_view(v)
    st = _ffi.load().ffpa_kv4_write(_dt(k), wk, wv, c, _lengths(start, B, "start", dev),
                                    _lengths(count, B, "count", dev), B, Hkv, N, D, _raw_stream(dev))
    if st:
        _ffi.raise_for(st, "ffpa_kv4_write")


def varlen_kv4_write(cache, block_table, k, v, cu_seqlens, max_seqlen: int, start=None) -> None:
    """As kv4_write, for a packed batch: k, v [T, Hkv, D], sequence b's tokens the rows
    [cu_seqlens[b], cu_seqlens[b + 1]) (int32 on the device), at most max_seqlen of them."""
    B = cu_seqlens.numel() - 1
    c, Hkv, D, dev = _kv4(cache, block_table, B)
    T = _kv4_pair(k, v, 3, Hkv, D, dev)[0]
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return varlen_kv4_write(cache, block_table, k, v, cu_seqlens, max_seqlen, start)
    k, v = _in_packed(k), _in_packed(v)
    st = _ffi.load().ffpa_varlen_kv4_write(_dt(k), k.data_ptr(), v.data_ptr(), c,
                                           _lengths(cu_seqlens, B + 1, "cu_seqlens", dev),
                                           _lengths(start, B, "start", dev), B, T, int(max_seqlen), Hkv, D,
                                           _raw_stream(dev))
    if st:
        _ffi.raise_for(st, "ffpa_varlen_kv4_write")


def kv4_read(cache, block_table, count, max_count: int | None = None, dtype=torch.bfloat16, start=None, k_out=None,
             v_out=None):
    """Reads cached tokens back through ffpa_kv4_read: token start[b] + i of sequence b to
    row i, for i < count[b] (int32 [B] on the device). Returns (k, v) [B, Hkv, N, D].

    With k_out and v_out given, N is theirs and rows at and past count[b] keep what they
    hold; else N is max_count and those rows are zero."""
    B = block_table.shape[0]
    c, Hkv, D, dev = _kv4(cache, block_table, B)
    if (k_out is None) != (v_out is None) or (k_out is None) == (max_count is None):
        raise ValueError("give either k_out and v_out or max_count")
    if count is None:
        raise ValueError("count is required")
    if k_out is None:
        k_out, v_out = (torch.zeros((B, Hkv, max_count, D), dtype=dtype, device=dev) for _ in range(2))
    shape = _kv4_pair(k_out, v_out, 4, Hkv, D, dev)
    if shape[0] != B:
        raise ValueError(f"k_out has {shape[0]} sequences, block_table {B}")
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return kv4_read(cache, block_table, count, start=start, k_out=k_out, v_out=v_out)
    st = _ffi.load().ffpa_kv4_read(_dt(k_out), c, _out_view(k_out), _out_view(v_out),
                                   _lengths(start, B, "start", dev), _lengths(count, B, "count", dev), B, Hkv,
                                   shape[2], D, _raw_stream(dev))
    if st:
        _ffi.raise_for(st, "ffpa_kv4_read")
    return k_out, v_out


def varlen_kv4_read(cache, block_table, cu_seqlens, max_seqlen: int, total: int | None = None, dtype=torch.bfloat16,
                    start=None, k_out=None, v_out=None):
    """As kv4_read, into packed tensors [T, Hkv, D] (what varlen_fwd takes as keys and
    values): sequence b's tokens to the rows [cu_seqlens[b], cu_seqlens[b + 1]). T is
    `total` or that of k_out and v_out."""
    B = cu_seqlens.numel() - 1
    c, Hkv, D, dev = _kv4(cache, block_table, B)
    if (k_out is None) != (v_out is None) or (k_out is None) == (total is None):
        raise ValueError("give either k_out and v_out or total")
    if k_out is None:
        k_out, v_out = (torch.zeros((total, Hkv, D), dtype=dtype, device=dev) for _ in range(2))
    T = _kv4_pair(k_out, v_out, 3, Hkv, D, dev)[0]
    if not k_out.is_contiguous() or not v_out.is_contiguous():
        raise ValueError("k_out and v_out must be contiguous")
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return varlen_kv4_read(cache, block_table, cu_seqlens, max_seqlen, start=start, k_out=k_out, v_out=v_out)
    st = _ffi.load().ffpa_varlen_kv4_read(_dt(k_out), c, k_out.data_ptr(), v_out.data_ptr(),
                                          _lengths(cu_seqlens, B + 1, "cu_seqlens", dev),
                                          _lengths(start, B, "start", dev), B, T, int(max_seqlen), Hkv, D,
                                          _raw_stream(dev))
    if st:
        _ffi.raise_for(st, "ffpa_varlen_kv4_read")
    return k_out, v_out


@functools.lru_cache(maxsize=256)
def _kv4_workspace_bytes(device: int, dt: int, B: int, Hq: int, Hkv: int, Nq: int, D: int) -> int:
    """ffpa_decode_kv4_workspace_bytes, which depends on its arguments and the device's SMs alone."""
    with torch.cuda.device(device):
        return max(256, int(_ffi.load().ffpa_decode_kv4_workspace_bytes(dt, B, Hq, Hkv, Nq, D)))


def decode_kv4_workspace(q, cache) -> torch.Tensor:
    """Device scratch for decode_fwd_kv4 (uint8, 256-byte aligned by the allocator), for one call at a time."""
    B, Hq, Nq, D = q.shape
    n = _kv4_workspace_bytes(q.device.index, _dt(q), B, Hq, cache.shape[2], Nq, D)
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def decode_fwd_kv4(q, cache, block_table, seq_lens, causal: bool = False, scale: float | None = None, out=None,
                   lse=None, workspace=None):
    """Decode / short-query forward over the 4-bit cache through ffpa_decode_fwd_kv4: the
    keys and values of sequence b are its first seq_lens[b] cached tokens (int32 [B] on
    the device); causal is bottom-right per sequence. q [B, Hq, Nq, D]; returns (o, lse).

    A long chunk of queries goes through varlen_kv4_read and varlen_fwd instead."""
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("expected q [B,Hq,Nq,D]")
    B, Hq, Nq, D = shape
    c, Hkv, Dc, dev = _kv4(cache, block_table, B)
    if D != Dc:
        raise ValueError(f"q has head dim {D}, the cache {Dc}")
    if q.device != dev:
        raise ValueError("q and the cache are on different devices")
    if seq_lens is None:
        raise ValueError("seq_lens is required")
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return decode_fwd_kv4(q, cache, block_table, seq_lens, causal, scale, out, lse, workspace)
    q, wq = _in_view(q)
    dt = _dt(q)
    if out is None:
        out = torch.empty_like(q)
        wo = _view_or_none(out)
        if wo is None:
            out = torch.empty(shape, dtype=q.dtype, device=dev)
            wo = _view(out)
    elif out.shape != shape or out.dtype != q.dtype or out.device != dev:
        raise ValueError("out must have q's shape, dtype and device")
    else:
        wo = _out_view(out)
    if lse is None:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=dev)
    elif not lse.is_contiguous() or lse.dtype != torch.float32 or lse.shape != shape[:3] or lse.device != dev:
        raise ValueError("lse must be a contiguous fp32 [B, Hq, Nq] tensor")
    if workspace is None:
        n = _kv4_workspace_bytes(dev.index, dt, B, Hq, Hkv, Nq, D)
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on q's device")
    else:
        n = workspace.numel() * workspace.element_size()
    st = _ffi.load().ffpa_decode_fwd_kv4(dt, wq, c, _lengths(seq_lens, B, "seq_lens", dev), wo, lse.data_ptr(),
                                         workspace.data_ptr(), n, B, Hq, Hkv, Nq, D, int(bool(causal)),
                                         _scale(scale, D), _raw_stream(dev))
    if st:
        _ffi.raise_for(st, "ffpa_decode_fwd_kv4")
    return out, lse


def get_status() -> None:
    """Synchronises the current stream and raises if a kernel reported a device time-out, a packed
    sequence that breaks the varlen contract, or one whose lengths or pages lie outside its 4-bit cache."""
    _ffi.raise_for(_ffi.ffpa_get_status(_stream()), "device status")
