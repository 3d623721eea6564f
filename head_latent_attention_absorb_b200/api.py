"""Python binding of libmla_b200.so with the C names.  Argument marshalling only: torch owns
the device memory and the stream; every step of the computation runs in the library's kernels.

All tensors are CUDA tensors.  Strides are read from the tensors, so a packed
[B, n_max, d_c + d_r] cache can be passed as two views (``cache[..., :d_c]``, ``cache[..., d_c:]``).
"""

from __future__ import annotations

import ctypes
import functools
import struct
from typing import Optional, Sequence

import torch

from . import _capi
from ._capi import MLADims, check, lib

_DT = {torch.bfloat16: _capi.MLA_BF16, torch.float32: _capi.MLA_F32}


def dims_of(n_h: int, d_c: int, d_r: int, d_h: int, d_v: int) -> MLADims:
    return MLADims(n_h, d_c, d_r, d_h, d_v)


def _dtc(dtype: torch.dtype) -> int:
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}")
    return _DT[dtype]


def _dt(t: torch.Tensor) -> int:
    return _dtc(t.dtype)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream if hasattr(s, "cuda_stream") else s


def _rows(t: torch.Tensor, name: str):
    if t.stride(-1) != 1:
        raise ValueError(f"{name}: last axis must be contiguous")


def _headrows(t: torch.Tensor, name: str) -> int:
    """Row stride of a [B, n_h, width] tensor whose (b, h) rows are evenly strided."""
    _rows(t, name)
    if t.dim() != 3 or t.stride(0) != t.shape[1] * t.stride(1):
        raise ValueError(f"{name}: expected [B, n_h, width] with row (b, h) at (b*n_h + h)*stride")
    return t.stride(1)


def _dims(x: Sequence[int]) -> MLADims:
    return x if isinstance(x, MLADims) else MLADims(*x)


# ---- The cache operators (4-bit cache, attention weights, eviction) are called once or more for every decoded
# token, where a few microseconds on the host count.  Their checks take the common case first.
def _fast_dims(x: Sequence[int]) -> MLADims:
    if isinstance(x, MLADims):
        return x
    d = _DIMS.get(x) if type(x) is tuple else None
    if d is None:
        d = MLADims(*x)
        if len(_DIMS) < 256:
            _DIMS[tuple(x)] = d
    return d


_PLANES = _capi.MLARows * _capi.MAX_PLANES
# fills an array of planes in one call: base, strides, row bytes and the struct's padding
_PACK_PLANES = [struct.Struct("@" + "Pqqi4x" * n).pack_into for n in range(_capi.MAX_PLANES + 1)]
_DIMS: dict = {}
_FN: dict = {}


def _fn(name: str):
    f = _FN.get(name)
    if f is None:
        f = _FN[name] = getattr(lib(), name)
    return f


def _i32(t: torch.Tensor, shape: tuple, name: str):
    if t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 {list(shape)} tensor")


def _shape(t: torch.Tensor, shape: tuple, dtype: torch.dtype, name: str) -> tuple:
    """Checks a tensor with contiguous rows; its strides."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        _rows(t, name)
    return st


def _on_device(*tensors) -> int:
    """Index of the one CUDA device that all the tensors (None: absent) live on."""
    dev = None
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d != dev:
                if d < 0:
                    raise ValueError("expected a CUDA tensor")
                if dev is not None:
                    raise ValueError(f"tensors on two devices: cuda:{dev} and cuda:{d}")
                dev = d
    return dev


class _Entered:
    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_HERE = _Entered()
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: torch.cuda.current_stream(d).cuda_stream)


def _launch_on(stream, device: int):
    """(context, handle) of a call: inside the context the tensors' device is current, and so is the
    stream, so that what the call allocates belongs to the stream that uses it."""
    cur = _raw_stream(device)
    handle = cur if stream is None else getattr(stream, "cuda_stream", stream)
    if handle == cur and device == torch.cuda.current_device():
        return _HERE, cur
    if stream is None:
        stream = torch.cuda.current_stream(device)
    elif not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(stream, device=torch.device("cuda", device))
    return torch.cuda.stream(stream), handle


def _flag(dev_err: Optional[torch.Tensor]):
    if dev_err is not None and (dev_err.dtype is not torch.int32 or dev_err.numel() < 1):
        raise TypeError("dev_err must be an int32 tensor")


def _empty(like: torch.Tensor, shape: tuple) -> torch.Tensor:
    """A contiguous tensor of like's type and device (torch.empty_strided takes half of torch.empty's time)."""
    strides, n = [], 1
    for w in reversed(shape):
        strides.append(n)
        n *= w
    strides.reverse()
    return torch.empty_strided(shape, strides, dtype=like.dtype, device=like.device)


def _at(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _fp4_planes(d: MLADims, c4: torch.Tensor, kv_scale: torch.Tensor, k_r: Optional[torch.Tensor],
                dtype: Optional[torch.dtype]):
    """Shapes of a 4-bit cache; returns (B, n_max, batch and row strides of c4, of kv_scale, of k_r)."""
    shape = c4.shape
    if len(shape) != 3:
        raise ValueError("c4 must be [B, n_max, d_c / 2]")
    B, n_max, d_c = shape[0], shape[1], d.d_c
    a = _shape(c4, (B, n_max, d_c // 2), torch.uint8, "c4")
    b = _shape(kv_scale, (B, n_max, d_c // 16), torch.uint8, "kv_scale")
    if k_r is None:
        return B, n_max, a[0], a[1], b[0], b[1], 0, 0
    c = _shape(k_r, (B, n_max, d.d_r), dtype, "k_r")
    return B, n_max, a[0], a[1], b[0], b[1], c[0], c[1]


def _token_stride(q: torch.Tensor, name: str) -> int:
    """Stride of the evenly strided rows (b, t, h) of a [B, n_h, w] or [B, T, n_h, w] tensor."""
    if q.is_contiguous():
        return q.shape[-1]
    if q.dim() == 4:
        try:
            q = q.view(-1, q.shape[2], q.shape[3])
        except RuntimeError:
            raise ValueError(f"{name}: the tokens of consecutive sequences must be evenly strided") from None
    return _headrows(q, name)


def _queries(d: MLADims, q_tilde: torch.Tensor, q_pe: torch.Tensor, B: int, lengths: torch.Tensor):
    """Query tensors [B, n_h, .] or [B, T, n_h, .]; returns (T, row stride of q_tilde, of q_pe)."""
    shape = q_tilde.shape
    if len(shape) not in (3, 4):
        raise ValueError("q_tilde must be [B, n_h, d_c] or [B, T, n_h, d_c]")
    lead, dtype = tuple(shape[:-2]), q_tilde.dtype
    _shape(q_tilde, (*lead, d.n_h, d.d_c), dtype, "q_tilde")
    _shape(q_pe, (*lead, d.n_h, d.d_r), dtype, "q_pe")
    if lead[0] != B:
        raise ValueError(f"q_tilde holds {lead[0]} sequences, the cache {B}")
    _i32(lengths, (B,), "lengths")
    return 1 if len(lead) == 1 else lead[1], _token_stride(q_tilde, "q_tilde"), _token_stride(q_pe, "q_pe")


def mla_absorb_q(dims, q_nope: torch.Tensor, w_kv_b: torch.Tensor, q_tilde: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """q~[b,h,:] = (W^UK_h)^T q_nope[b,h,:].  q_nope [B, n_h, d_h] (rows may be strided)."""
    d = _dims(dims)
    B = q_nope.shape[0]
    ldq = _headrows(q_nope, "q_nope")
    if q_tilde is None:
        q_tilde = torch.empty((B, d.n_h, d.d_c), dtype=q_nope.dtype, device=q_nope.device)
    check(lib().mla_absorb_q(d, _dt(q_nope), B, _ptr(q_nope), ldq, _ptr(w_kv_b), _ptr(q_tilde),
                             _stream(stream)), "mla_absorb_q")
    return q_tilde


def mla_decode_workspace_size(dims, dtype: torch.dtype, B: int, n_max: int, topk: int = 0) -> int:
    return int(lib().mla_decode_workspace_size(_dims(dims), _dtc(dtype), B, n_max, topk))


def mla_decode_num_launches(dims, dtype: torch.dtype, B: int, n_max: int, topk: int = 0) -> int:
    return int(lib().mla_decode_num_launches(_dims(dims), _dtc(dtype), B, n_max, topk))


def mla_decode_absorb(dims, q_tilde: torch.Tensor, q_pe: torch.Tensor, c_kv: torch.Tensor, k_r: torch.Tensor,
                      lengths: torch.Tensor, scale: float, topk_idx: Optional[torch.Tensor] = None,
                      ctx: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """Latent-space attention of one query token per sequence.  c_kv [B, n_max, d_c] and
    k_r [B, n_max, d_r] may be strided views; lengths int32 [B]; topk_idx int32 [B, k] or None."""
    d = _dims(dims)
    B, n_max = c_kv.shape[0], c_kv.shape[1]
    ldqt, ldqp = _headrows(q_tilde, "q_tilde"), _headrows(q_pe, "q_pe")
    _rows(c_kv, "c_kv")
    _rows(k_r, "k_r")
    if lengths.dtype != torch.int32 or (topk_idx is not None and topk_idx.dtype != torch.int32):
        raise TypeError("lengths and topk_idx must be int32")
    if topk_idx is not None and not topk_idx.is_contiguous():
        raise ValueError("topk_idx must be contiguous")
    topk = 0 if topk_idx is None else topk_idx.shape[1]
    if ctx is None:
        ctx = torch.empty((B, d.n_h, d.d_c), dtype=q_tilde.dtype, device=q_tilde.device)
    if workspace is None:
        nbytes = mla_decode_workspace_size(d, q_tilde.dtype, B, n_max, topk)
        workspace = torch.empty((max(nbytes, 16),), dtype=torch.uint8, device=q_tilde.device)
    check(lib().mla_decode_absorb(
        d, _dt(q_tilde), B,
        _ptr(q_tilde), ldqt, _ptr(q_pe), ldqp,
        _ptr(c_kv), c_kv.stride(0), c_kv.stride(1), _ptr(k_r), k_r.stride(0), k_r.stride(1),
        n_max, _ptr(lengths), _ptr(topk_idx), topk, float(scale),
        _ptr(ctx), _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(dev_err), _stream(stream)), "mla_decode_absorb")
    return ctx


def mla_decode_absorb_fp8kv(dims, q_tilde: torch.Tensor, q_pe: torch.Tensor, c8: torch.Tensor,
                            kv_scale: torch.Tensor, k_r: torch.Tensor, lengths: torch.Tensor, scale: float,
                            ctx: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """The absorbed decode over an FP8 latent cache: c8 [B, n_max, d_c] uint8 E4M3 codes, kv_scale
    [B, n_max, d_c / 128] float32 (one scale per 128 latent features of a row), k_r [B, n_max, d_r]
    bf16; all three may be strided views (e.g. of one packed 656-byte row)."""
    d = _dims(dims)
    B, n_max = c8.shape[0], c8.shape[1]
    ldqt, ldqp = _headrows(q_tilde, "q_tilde"), _headrows(q_pe, "q_pe")
    for t, n in ((c8, "c8"), (kv_scale, "kv_scale"), (k_r, "k_r")):
        _rows(t, n)
    if c8.dtype != torch.uint8 or kv_scale.dtype != torch.float32:
        raise TypeError("c8 must be uint8 and kv_scale float32")
    if lengths.dtype != torch.int32:
        raise TypeError("lengths must be int32")
    if ctx is None:
        ctx = torch.empty((B, d.n_h, d.d_c), dtype=q_tilde.dtype, device=q_tilde.device)
    if workspace is None:
        nbytes = mla_decode_workspace_size(d, q_tilde.dtype, B, n_max, 0)
        workspace = torch.empty((max(nbytes, 16),), dtype=torch.uint8, device=q_tilde.device)
    check(lib().mla_decode_absorb_fp8kv(
        d, B, _ptr(q_tilde), ldqt, _ptr(q_pe), ldqp,
        _ptr(c8), c8.stride(0), c8.stride(1), _ptr(kv_scale), kv_scale.stride(0), kv_scale.stride(1),
        _ptr(k_r), k_r.stride(0), k_r.stride(1), n_max, _ptr(lengths), float(scale),
        _ptr(ctx), _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(dev_err), _stream(stream)), "mla_decode_absorb_fp8kv")
    return ctx


def mla_decode_absorb_multi(dims, q_tilde: torch.Tensor, q_pe: torch.Tensor, c_kv: torch.Tensor,
                            k_r: torch.Tensor, lengths: torch.Tensor, scale: float,
                            ctx: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """T new tokens per sequence: q_tilde [B, T, n_h, d_c] and q_pe [B, T, n_h, d_r] (the last T cached
    rows of each sequence are those tokens); returns ctx [B, T, n_h, d_c].  c_kv / k_r / lengths as in
    mla_decode_absorb."""
    d = _dims(dims)
    B, T = q_tilde.shape[0], q_tilde.shape[1]
    n_max = c_kv.shape[1]
    qt = q_tilde.reshape(B * T, d.n_h, -1)
    qp = q_pe.reshape(B * T, d.n_h, -1)
    ldqt, ldqp = _headrows(qt, "q_tilde"), _headrows(qp, "q_pe")
    _rows(c_kv, "c_kv")
    _rows(k_r, "k_r")
    if lengths.dtype != torch.int32:
        raise TypeError("lengths must be int32")
    if ctx is None:
        ctx = torch.empty((B, T, d.n_h, d.d_c), dtype=q_tilde.dtype, device=q_tilde.device)
    if workspace is None:
        nbytes = mla_decode_workspace_size(d, q_tilde.dtype, B * T, n_max, 0)
        workspace = torch.empty((max(nbytes, 16),), dtype=torch.uint8, device=q_tilde.device)
    check(lib().mla_decode_absorb_multi(
        d, _dt(q_tilde), B, T, _ptr(qt), ldqt, _ptr(qp), ldqp,
        _ptr(c_kv), c_kv.stride(0), c_kv.stride(1), _ptr(k_r), k_r.stride(0), k_r.stride(1),
        n_max, _ptr(lengths), float(scale), _ptr(ctx), _ptr(lse), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(dev_err), _stream(stream)), "mla_decode_absorb_multi")
    return ctx


def mla_decode_absorb_multi_topk(dims, q_tilde: torch.Tensor, q_pe: torch.Tensor, c_kv: torch.Tensor,
                                 k_r: torch.Tensor, lengths: torch.Tensor, topk_idx: torch.Tensor, scale: float,
                                 ctx: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                                 workspace: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None,
                                 stream=None) -> torch.Tensor:
    """mla_decode_absorb_multi with a top-k set per new token: topk_idx int32 [B, T, k] (token s of
    sequence b attends its set's rows t <= lengths[b] - T + s); returns ctx [B, T, n_h, d_c]."""
    d = _dims(dims)
    B, T = q_tilde.shape[0], q_tilde.shape[1]
    n_max = c_kv.shape[1]
    qt = q_tilde.reshape(B * T, d.n_h, -1)
    qp = q_pe.reshape(B * T, d.n_h, -1)
    ldqt, ldqp = _headrows(qt, "q_tilde"), _headrows(qp, "q_pe")
    _rows(c_kv, "c_kv")
    _rows(k_r, "k_r")
    if lengths.dtype != torch.int32:
        raise TypeError("lengths must be int32")
    if topk_idx.dtype != torch.int32 or not topk_idx.is_contiguous() or tuple(topk_idx.shape[:2]) != (B, T):
        raise TypeError("topk_idx must be a contiguous int32 [B, T, k] tensor")
    k = topk_idx.shape[2]
    if ctx is None:
        ctx = torch.empty((B, T, d.n_h, d.d_c), dtype=q_tilde.dtype, device=q_tilde.device)
    if workspace is None:
        nbytes = mla_decode_workspace_size(d, q_tilde.dtype, B * T, n_max, k)
        workspace = torch.empty((max(nbytes, 16),), dtype=torch.uint8, device=q_tilde.device)
    check(lib().mla_decode_absorb_multi_topk(
        d, _dt(q_tilde), B, T, _ptr(qt), ldqt, _ptr(qp), ldqp,
        _ptr(c_kv), c_kv.stride(0), c_kv.stride(1), _ptr(k_r), k_r.stride(0), k_r.stride(1),
        n_max, _ptr(lengths), _ptr(topk_idx), k, float(scale), _ptr(ctx), _ptr(lse), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(dev_err), _stream(stream)), "mla_decode_absorb_multi_topk")
    return ctx


def mla_decode_absorb_static(dims, q_tilde: torch.Tensor, q_pe: torch.Tensor, c_kv: torch.Tensor,
                             k_r: torch.Tensor, lengths: torch.Tensor, scale: float,
                             ctx: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                             dev_err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """bf16 dense decode with the library's built-in scratch (for callers that cannot allocate a
    workspace).  `ctx` (and `lse`) are allocated here only when not given."""
    d = _dims(dims)
    B, n_max = c_kv.shape[0], c_kv.shape[1]
    ldqt, ldqp = _headrows(q_tilde, "q_tilde"), _headrows(q_pe, "q_pe")
    _rows(c_kv, "c_kv")
    _rows(k_r, "k_r")
    if lengths.dtype != torch.int32:
        raise TypeError("lengths must be int32")
    if ctx is None:
        ctx = torch.empty((B, d.n_h, d.d_c), dtype=q_tilde.dtype, device=q_tilde.device)
    check(lib().mla_decode_absorb_static(
        d, _dt(q_tilde), B, _ptr(q_tilde), ldqt, _ptr(q_pe), ldqp,
        _ptr(c_kv), c_kv.stride(0), c_kv.stride(1), _ptr(k_r), k_r.stride(0), k_r.stride(1),
        n_max, _ptr(lengths), float(scale), _ptr(ctx), _ptr(lse), _ptr(dev_err), _stream(stream)),
        "mla_decode_absorb_static")
    return ctx


def mla_out_up(dims, ctx: torch.Tensor, w_kv_b: torch.Tensor, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """o[b,h,:] = W^UV_h ctx[b,h,:].  ctx [B, n_h, d_c] contiguous."""
    d = _dims(dims)
    B = ctx.shape[0]
    if not ctx.is_contiguous():
        raise ValueError("ctx must be contiguous")
    if out is None:
        out = torch.empty((B, d.n_h, d.d_v), dtype=ctx.dtype, device=ctx.device)
    check(lib().mla_out_up(d, _dt(ctx), B, _ptr(ctx), _ptr(w_kv_b), _ptr(out), _stream(stream)), "mla_out_up")
    return out


def mla_absorb_q_fp8(dims, q_nope: torch.Tensor, w_fp8: torch.Tensor, w_scale: torch.Tensor,
                     q_tilde: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """mla_absorb_q with an e4m3 wkv_b (w_fp8, torch.float8_e4m3fn) and its fp32 128 x 128 block
    scales (w_scale [rows / 128, d_c / 128])."""
    d = _dims(dims)
    B = q_nope.shape[0]
    ldq = _headrows(q_nope, "q_nope")
    if w_fp8.dtype != torch.float8_e4m3fn or w_scale.dtype != torch.float32 or not w_scale.is_contiguous():
        raise TypeError("w_fp8 must be float8_e4m3fn and w_scale contiguous float32")
    if q_tilde is None:
        q_tilde = torch.empty((B, d.n_h, d.d_c), dtype=torch.bfloat16, device=q_nope.device)
    check(lib().mla_absorb_q_fp8(d, B, _ptr(q_nope), ldq, _ptr(w_fp8), _ptr(w_scale), _ptr(q_tilde), _ptr(dev_err),
                                 _stream(stream)), "mla_absorb_q_fp8")
    return q_tilde


def mla_out_up_fp8(dims, ctx: torch.Tensor, w_fp8: torch.Tensor, w_scale: torch.Tensor,
                   out: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """mla_out_up with an e4m3 wkv_b and its fp32 128 x 128 block scales."""
    d = _dims(dims)
    B = ctx.shape[0]
    if not ctx.is_contiguous():
        raise ValueError("ctx must be contiguous")
    if w_fp8.dtype != torch.float8_e4m3fn or w_scale.dtype != torch.float32 or not w_scale.is_contiguous():
        raise TypeError("w_fp8 must be float8_e4m3fn and w_scale contiguous float32")
    if out is None:
        out = torch.empty((B, d.n_h, d.d_v), dtype=torch.bfloat16, device=ctx.device)
    check(lib().mla_out_up_fp8(d, B, _ptr(ctx), _ptr(w_fp8), _ptr(w_scale), _ptr(out), _ptr(dev_err),
                               _stream(stream)), "mla_out_up_fp8")
    return out


def mla_prefill_workspace_size(dims, dtype: torch.dtype, B: int, S: int) -> int:
    return int(lib().mla_prefill_workspace_size(_dims(dims), _dtc(dtype), B, S))


def mla_prefill_naive(dims, q: torch.Tensor, c_kv: torch.Tensor, k_r: torch.Tensor, w_kv_b: torch.Tensor,
                      scale: float, causal: bool = True, out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Naive-path prefill.  q [B, S, n_h, d_h + d_r] contiguous; c_kv [B, S, d_c] and k_r [B, S, d_r]
    with contiguous rows and (b, s) rows evenly strided."""
    d = _dims(dims)
    B, S = c_kv.shape[0], c_kv.shape[1]
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    for t, n in ((c_kv, "c_kv"), (k_r, "k_r")):
        _rows(t, n)
        if t.stride(0) != S * t.stride(1):
            raise ValueError(f"{n}: rows of consecutive sequences must be evenly strided")
    if out is None:
        out = torch.empty((B, S, d.n_h, d.d_v), dtype=q.dtype, device=q.device)
    if workspace is None:
        nbytes = mla_prefill_workspace_size(d, q.dtype, B, S)
        workspace = torch.empty((max(nbytes, 16),), dtype=torch.uint8, device=q.device)
    check(lib().mla_prefill_naive(d, _dt(q), B, S, _ptr(q), _ptr(c_kv), c_kv.stride(1), _ptr(k_r), k_r.stride(1),
                                  _ptr(w_kv_b), float(scale), 1 if causal else 0, _ptr(out), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(stream)),
          "mla_prefill_naive")
    return out


def mla_cache_append(dims, kv_a: torch.Tensor, positions: torch.Tensor, c_kv: torch.Tensor, k_r: torch.Tensor,
                     gain: Optional[torch.Tensor] = None, eps: float = 1e-6, rope_base: float = 10000.0,
                     dev_err: Optional[torch.Tensor] = None, stream=None,
                     rows: Optional[torch.Tensor] = None) -> None:
    """Write each sequence's new token into the caches in place: RMSNorm(kv_a[b, :d_c]) * gain into
    c_kv[b, positions[b]] and the rotary key kv_a[b, d_c:] rotated by positions[b] into
    k_r[b, positions[b]].  kv_a [B, d_c + d_r] (rows may be strided); positions int32 [B];
    c_kv [B, n_max, d_c] and k_r [B, n_max, d_r] may be views of one packed cache; gain fp32 [d_c].
    rows int32 [B] gives the cache rows apart from the positions (a cache whose rows were evicted)."""
    d = _dims(dims)
    B, n_max = c_kv.shape[0], c_kv.shape[1]
    _rows(kv_a, "kv_a")
    _rows(c_kv, "c_kv")
    _rows(k_r, "k_r")
    if kv_a.dim() != 2 or kv_a.shape[0] != B:
        raise ValueError("kv_a must be [B, d_c + d_r]")
    if positions.dtype != torch.int32 or not positions.is_contiguous():
        raise TypeError("positions must be a contiguous int32 tensor")
    if gain is not None and (gain.dtype != torch.float32 or not gain.is_contiguous()):
        raise TypeError("gain must be a contiguous float32 tensor")
    if rows is None:
        check(lib().mla_cache_append(d, _dt(kv_a), B, _ptr(kv_a), kv_a.stride(0), _ptr(gain), float(eps),
                                     float(rope_base), _ptr(positions), n_max,
                                     _ptr(c_kv), c_kv.stride(0), c_kv.stride(1), _ptr(k_r), k_r.stride(0),
                                     k_r.stride(1), _ptr(dev_err), _stream(stream)), "mla_cache_append")
        return
    dtype = kv_a.dtype
    if kv_a.shape[1] < d.d_c + d.d_r:
        raise ValueError("kv_a must be [B, d_c + d_r]")
    c = _shape(c_kv, (B, n_max, d.d_c), dtype, "c_kv")
    k = _shape(k_r, (B, n_max, d.d_r), dtype, "k_r")
    _i32(positions, (B,), "positions")
    _i32(rows, (B,), "rows")
    if gain is not None:
        _shape(gain, (d.d_c,), torch.float32, "gain")
    _flag(dev_err)
    on, st = _launch_on(stream, _on_device(kv_a, positions, rows, c_kv, k_r, gain, dev_err))
    with on:
        check(_fn("mla_cache_append_at")(
            d, _dtc(dtype), B, kv_a.data_ptr(), kv_a.stride(0), _at(gain), eps, rope_base, positions.data_ptr(),
            rows.data_ptr(), n_max, c_kv.data_ptr(), c[0], c[1], k_r.data_ptr(), k[0], k[1], _at(dev_err), st),
            "mla_cache_append_at")


def mla_check_topk(topk_idx: torch.Tensor, n_max: int, lengths: Optional[torch.Tensor] = None,
                   dev_err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Validate a top-k index array on the device: every index of row b inside [0, lengths[b])
    (n_max when lengths is None) and listed once.  Sets MLA_ERR_INDEX / MLA_ERR_LENGTH in `dev_err`
    (allocated zeroed here when not given), which is returned; read it with mla_get_device_error."""
    if topk_idx.dtype != torch.int32 or not topk_idx.is_contiguous() or topk_idx.dim() != 2:
        raise TypeError("topk_idx must be a contiguous int32 [B, topk] tensor")
    if lengths is not None and (lengths.dtype != torch.int32 or not lengths.is_contiguous()):
        raise TypeError("lengths must be a contiguous int32 tensor")
    if dev_err is None:
        dev_err = torch.zeros(1, dtype=torch.int32, device=topk_idx.device)
    check(lib().mla_check_topk(topk_idx.shape[0], _ptr(topk_idx), topk_idx.shape[1], _ptr(lengths), int(n_max),
                               _ptr(dev_err), _stream(stream)), "mla_check_topk")
    return dev_err


def mla_prefill_sparse(dims, q: torch.Tensor, c_kv: torch.Tensor, k_r: torch.Tensor, w_kv_b: torch.Tensor,
                       scale: float, topk_idx: torch.Tensor, out: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """Sparse prefill: as mla_prefill_naive (causal), each query row attending only the positions
    its row of topk_idx (int32 [B, S, k]) selects."""
    d = _dims(dims)
    B, S = c_kv.shape[0], c_kv.shape[1]
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    for t, n in ((c_kv, "c_kv"), (k_r, "k_r")):
        _rows(t, n)
        if t.stride(0) != S * t.stride(1):
            raise ValueError(f"{n}: rows of consecutive sequences must be evenly strided")
    if topk_idx.dtype != torch.int32 or not topk_idx.is_contiguous() or tuple(topk_idx.shape[:2]) != (B, S):
        raise TypeError("topk_idx must be a contiguous int32 [B, S, k] tensor")
    if out is None:
        out = torch.empty((B, S, d.n_h, d.d_v), dtype=q.dtype, device=q.device)
    if workspace is None:
        nbytes = int(lib().mla_prefill_sparse_workspace_size(d, _dt(q), B, S))
        workspace = torch.empty((max(nbytes, 16),), dtype=torch.uint8, device=q.device)
    check(lib().mla_prefill_sparse(d, _dt(q), B, S, _ptr(q), _ptr(c_kv), c_kv.stride(1), _ptr(k_r), k_r.stride(1),
                                   _ptr(w_kv_b), float(scale), _ptr(topk_idx), topk_idx.shape[2], _ptr(out),
                                   _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(dev_err),
                                   _stream(stream)), "mla_prefill_sparse")
    return out


def mla_cache_append_fp4(dims, kv_a: torch.Tensor, positions: torch.Tensor, c4: torch.Tensor, kv_scale: torch.Tensor,
                         k_r: torch.Tensor, rows: Optional[torch.Tensor] = None,
                         counts: Optional[torch.Tensor] = None, gain: Optional[torch.Tensor] = None,
                         eps: float = 1e-6, rope_base: float = 10000.0, latent_scale: float = 1.0,
                         dev_err: Optional[torch.Tensor] = None, stream=None) -> None:
    """Write new tokens into a 4-bit latent cache in place: E2M1 codes of RMSNorm(latent) * gain with an
    E4M3 scale per 16 features, and the rotary key.  kv_a [B, d_c + d_r] or [B, T, d_c + d_r];
    positions int32 [B], the position of each sequence's first token; rows int32 [B], its cache row
    (None: the position); counts int32 [B], tokens of each sequence (None: all T).  c4 uint8
    [B, n_max, d_c / 2], kv_scale uint8 [B, n_max, d_c / 16] and k_r [B, n_max, d_r] may be views of one
    packed row.  latent_scale: a power of two, the same for every call on the cache."""
    d = _fast_dims(dims)
    dtype = kv_a.dtype
    B, n_max, c4b, c4r, scb, scr, krb, krr = _fp4_planes(d, c4, kv_scale, k_r, dtype)
    width = d.d_c + d.d_r
    if kv_a.dim() == 3:
        T = kv_a.shape[1]
        lda = _shape(kv_a, (B, T, width), dtype, "kv_a")
        lda_b, lda = lda[0], lda[1] if T > 1 else width
    elif kv_a.dim() == 2:
        T = 1
        lda_b, lda = _shape(kv_a, (B, width), dtype, "kv_a")[0], width
    else:
        raise ValueError("kv_a must be [B, d_c + d_r] or [B, T, d_c + d_r]")
    index = (B,)
    _i32(positions, index, "positions")
    if rows is not None:
        _i32(rows, index, "rows")
    if counts is not None:
        _i32(counts, index, "counts")
    if gain is not None:
        _shape(gain, (d.d_c,), torch.float32, "gain")
    _flag(dev_err)
    dev = _on_device(kv_a, positions, c4, kv_scale, k_r, rows, counts, gain, dev_err)
    on, st = _launch_on(stream, dev)
    with on:
        check(_fn("mla_cache_append_fp4")(
            d, _dtc(dtype), B, T, kv_a.data_ptr(), lda_b, lda, _at(gain), eps, rope_base, latent_scale,
            positions.data_ptr(), _at(rows), _at(counts), n_max, c4.data_ptr(), c4b, c4r, kv_scale.data_ptr(), scb, scr,
            k_r.data_ptr(), krb, krr, _at(dev_err), st), "mla_cache_append_fp4")


def mla_cache_read_fp4(dims, c4: torch.Tensor, kv_scale: torch.Tensor, n: int, first: Optional[torch.Tensor] = None,
                       counts: Optional[torch.Tensor] = None, latent_scale: float = 1.0,
                       dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                       dev_err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The values of n latent rows per sequence of a 4-bit cache, from row first[b] on (int32 [B]; None: 0):
    out [B, n, d_c], zeros from counts[b] on (int32 [B]; None: n)."""
    d = _fast_dims(dims)
    B, n_max, c4b, c4r, scb, scr, _, _ = _fp4_planes(d, c4, kv_scale, None, None)
    shape = (B, n, d.d_c)
    if out is not None:
        dtype = out.dtype
        strides = _shape(out, shape, dtype, "out")
    code = _dtc(dtype)
    if first is not None:
        _i32(first, (B,), "first")
    if counts is not None:
        _i32(counts, (B,), "counts")
    _flag(dev_err)
    dev = _on_device(c4, kv_scale, out, first, counts, dev_err)
    on, st = _launch_on(stream, dev)
    with on:
        if out is None:
            out = torch.empty_strided(shape, (n * d.d_c, d.d_c, 1), dtype=dtype, device=c4.device)
            strides = (n * d.d_c, d.d_c, 1)
        check(_fn("mla_cache_read_fp4")(
            d, code, B, n, _at(first), _at(counts), n_max, c4.data_ptr(), c4b, c4r, kv_scale.data_ptr(), scb, scr,
            latent_scale, out.data_ptr(), strides[0], strides[1] if n > 1 else d.d_c, _at(dev_err), st),
            "mla_cache_read_fp4")
    return out


def mla_decode_fp4kv_workspace_size(dims, dtype: torch.dtype, B: int, T: int, n_max: int) -> int:
    """Bytes of workspace on the current device; 0 for arguments that the call would reject."""
    return int(lib().mla_decode_fp4kv_workspace_size(_dims(dims), _dtc(dtype), B, T, n_max))


@functools.lru_cache(maxsize=1024)
def _fp4kv_workspace(device: int, n_h: int, d_c: int, d_r: int, dtype: torch.dtype, B: int, T: int, n_max: int) -> int:
    return mla_decode_fp4kv_workspace_size((n_h, d_c, d_r, 1, 1), dtype, B, T, n_max)


def mla_decode_absorb_fp4kv(dims, q_tilde: torch.Tensor, q_pe: torch.Tensor, c4: torch.Tensor, kv_scale: torch.Tensor,
                            k_r: torch.Tensor, lengths: torch.Tensor, scale: float, latent_scale: float = 1.0,
                            ctx: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """The absorbed decode over a 4-bit latent cache (planes as in mla_cache_append_fp4), one token per
    sequence (q_tilde [B, n_h, d_c], q_pe [B, n_h, d_r]) or T ([B, T, n_h, .], the last T cached rows of each
    sequence being those tokens).  Any n_h <= 128 in bf16.  Returns ctx of q_tilde's shape; lse float32
    [B, n_h] or [B, T, n_h]."""
    d = _fast_dims(dims)
    dtype = q_tilde.dtype
    B, n_max, c4b, c4r, scb, scr, krb, krr = _fp4_planes(d, c4, kv_scale, k_r, dtype)
    T, ldqt, ldqp = _queries(d, q_tilde, q_pe, B, lengths)
    if ctx is not None:
        _shape(ctx, q_tilde.shape, dtype, "ctx")
        if not ctx.is_contiguous():
            raise ValueError("ctx and lse must be contiguous")
    if lse is not None:
        _shape(lse, q_tilde.shape[:-1], torch.float32, "lse")
        if not lse.is_contiguous():
            raise ValueError("ctx and lse must be contiguous")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _flag(dev_err)
    dev = _on_device(q_tilde, q_pe, c4, kv_scale, k_r, lengths, ctx, lse, workspace, dev_err)
    on, st = _launch_on(stream, dev)
    with on:
        if ctx is None:
            ctx = torch.empty_like(q_tilde) if q_tilde.is_contiguous() else _empty(q_tilde, q_tilde.shape)
        if workspace is None:
            nbytes = max(_fp4kv_workspace(dev, d.n_h, d.d_c, d.d_r, dtype, B, T, n_max), 16)
            workspace = c4.new_empty(nbytes)
        else:
            nbytes = workspace.numel() * workspace.element_size()
        check(_fn("mla_decode_absorb_fp4kv")(
            d, _dtc(dtype), B, T, q_tilde.data_ptr(), ldqt, q_pe.data_ptr(), ldqp, c4.data_ptr(), c4b, c4r,
            kv_scale.data_ptr(), scb, scr, k_r.data_ptr(), krb, krr, latent_scale, n_max, lengths.data_ptr(), scale,
            ctx.data_ptr(), _at(lse), workspace.data_ptr(), nbytes, _at(dev_err), st), "mla_decode_absorb_fp4kv")
    return ctx


def _weight_array(t: Optional[torch.Tensor], shape: tuple, name: str) -> int:
    """Batch stride of acc or out."""
    if t is None:
        return shape[1]
    st = _shape(t, shape, torch.float32, name)
    return st[0] if shape[0] > 1 else shape[1]


def mla_cache_weights(dims, q_tilde: torch.Tensor, q_pe: torch.Tensor, c_kv: torch.Tensor, k_r: torch.Tensor,
                      lengths: torch.Tensor, scale: float, lse: torch.Tensor, acc: Optional[torch.Tensor] = None,
                      decay: float = 1.0, out: Optional[torch.Tensor] = None,
                      dev_err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The attention weight that each cached row received in a decode step, summed over heads and new
    tokens, added to decay * acc (float32 [B, n_max]; the step's own T rows start from nothing).  Queries
    [B, n_h, .] or [B, T, n_h, .]; lse is the decode's.  Returns out [B, n_max], which may be acc; entries
    at and behind lengths[b] are left as they were (zeros when out is allocated here)."""
    d = _fast_dims(dims)
    if c_kv.dim() != 3:
        raise ValueError("c_kv must be [B, n_max, d_c]")
    dtype = q_tilde.dtype
    B, n_max = c_kv.shape[0], c_kv.shape[1]
    ckv = _shape(c_kv, (B, n_max, d.d_c), dtype, "c_kv")
    kr = _shape(k_r, (B, n_max, d.d_r), dtype, "k_r")
    T, ldqt, ldqp = _queries(d, q_tilde, q_pe, B, lengths)
    _shape(lse, q_tilde.shape[:-1], torch.float32, "lse")
    if not lse.is_contiguous():
        raise ValueError("lse must be contiguous")
    rows = (B, n_max)
    acc_b, out_b = _weight_array(acc, rows, "acc"), _weight_array(out, rows, "out")
    _flag(dev_err)
    dev = _on_device(q_tilde, q_pe, c_kv, k_r, lengths, lse, acc, out, dev_err)
    on, st = _launch_on(stream, dev)
    with on:
        if out is None:
            out = torch.zeros(rows, dtype=torch.float32, device=dev)
        check(_fn("mla_cache_weights")(
            d, _dtc(dtype), B, T, q_tilde.data_ptr(), ldqt, q_pe.data_ptr(), ldqp, c_kv.data_ptr(), ckv[0], ckv[1],
            k_r.data_ptr(), kr[0], kr[1], n_max, lengths.data_ptr(), scale, lse.data_ptr(), _at(acc), acc_b, decay,
            out.data_ptr(), out_b, _at(dev_err), st), "mla_cache_weights")
    return out


def mla_cache_weights_fp4kv(dims, q_tilde: torch.Tensor, q_pe: torch.Tensor, c4: torch.Tensor, kv_scale: torch.Tensor,
                            k_r: torch.Tensor, lengths: torch.Tensor, scale: float, lse: torch.Tensor,
                            latent_scale: float = 1.0, acc: Optional[torch.Tensor] = None, decay: float = 1.0,
                            out: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """mla_cache_weights over a 4-bit latent cache (planes as in mla_cache_append_fp4)."""
    d = _fast_dims(dims)
    dtype = q_tilde.dtype
    B, n_max, c4b, c4r, scb, scr, krb, krr = _fp4_planes(d, c4, kv_scale, k_r, dtype)
    T, ldqt, ldqp = _queries(d, q_tilde, q_pe, B, lengths)
    _shape(lse, q_tilde.shape[:-1], torch.float32, "lse")
    if not lse.is_contiguous():
        raise ValueError("lse must be contiguous")
    rows = (B, n_max)
    acc_b, out_b = _weight_array(acc, rows, "acc"), _weight_array(out, rows, "out")
    _flag(dev_err)
    dev = _on_device(q_tilde, q_pe, c4, kv_scale, k_r, lengths, lse, acc, out, dev_err)
    on, st = _launch_on(stream, dev)
    with on:
        if out is None:
            out = torch.zeros(rows, dtype=torch.float32, device=dev)
        check(_fn("mla_cache_weights_fp4kv")(
            d, _dtc(dtype), B, T, q_tilde.data_ptr(), ldqt, q_pe.data_ptr(), ldqp, c4.data_ptr(), c4b, c4r,
            kv_scale.data_ptr(), scb, scr, k_r.data_ptr(), krb, krr, latent_scale, n_max, lengths.data_ptr(), scale,
            lse.data_ptr(), _at(acc), acc_b, decay, out.data_ptr(), out_b, _at(dev_err), st),
            "mla_cache_weights_fp4kv")
    return out


def mla_cache_evict(planes: Sequence[torch.Tensor], acc: torch.Tensor, lengths: torch.Tensor, keep: int,
                    sink: int = 0, recent: int = 0, new_lengths: Optional[torch.Tensor] = None,
                    row_map: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None, stream=None,
                    positions: Optional[torch.Tensor] = None):
    """Keep `keep` rows of every sequence that holds more: the first `sink`, the `recent` newest, and the
    heaviest of the rest by acc (float32 [B, n_max]); kept rows behind `keep` move, in place, into the rows
    before it that go.  planes: 1 to 4 tensors [B, n_max, width] of any type whose rows move together
    (e.g. [c_kv, k_r], [c4, kv_scale, k_r]; add acc.unsqueeze(-1) to keep it in step).
    positions: int32 [B, n_max], the position of the token that each row holds; it moves with the rows, and
    the newest are those of largest position.  Without it the last `recent` rows count as the newest, which
    is right only while rows stand in order of age: an eviction ends that order, so a cache that is cut more
    than once needs positions.  Returns (new_lengths int32 [B], which may be given as lengths itself, and
    row_map int32 [B, keep]: the row that row i held before, -1 from new_lengths[b] on)."""
    n_planes = len(planes)
    if not 1 <= n_planes <= _capi.MAX_PLANES:
        raise ValueError(f"need 1 to {_capi.MAX_PLANES} planes")
    if acc.dim() != 2:
        raise ValueError("acc must be [B, n_max]")
    B, n_max = lead = tuple(acc.shape)
    acc_b = _weight_array(acc, lead, "acc")
    pos_b = n_max
    if positions is not None:
        strides = _shape(positions, lead, torch.int32, "positions")
        pos_b = strides[0] if B > 1 else n_max
    _i32(lengths, (B,), "lengths")
    rows, fields = _PLANES(), []
    for i, p in enumerate(planes):
        shape = p.shape
        if len(shape) != 3 or shape[:2] != lead:
            raise ValueError(f"plane {i} must be [B, n_max, width] = [{B}, {n_max}, .], got {list(shape)}")
        bs, rs, one = p.stride()
        if one != 1 and shape[2] > 1:
            _rows(p, f"plane {i}")
        es = p.element_size()
        width = shape[2] * es
        fields += (p.data_ptr(), bs * es, rs * es if n_max > 1 else width, min(width, 0x7fffffff))  # (so wide a row is refused)
    _PACK_PLANES[n_planes](rows, 0, *fields)
    if new_lengths is not None:
        _i32(new_lengths, (B,), "new_lengths")
    if row_map is not None:
        _i32(row_map, (B, keep), "row_map")
    _flag(dev_err)
    dev = _on_device(acc, lengths, new_lengths, row_map, dev_err, positions, *planes)
    on, st = _launch_on(stream, dev)
    with on:
        if new_lengths is None:
            new_lengths = lengths.new_empty(B)
        if row_map is None:
            wide = max(keep, 0)
            row_map = torch.empty_strided((B, wide), (wide, 1), dtype=torch.int32, device=lengths.device)
        if positions is None:
            check(_fn("mla_cache_evict")(B, n_max, rows, n_planes, acc.data_ptr(), acc_b, lengths.data_ptr(), keep, sink,
                                         recent, new_lengths.data_ptr(), row_map.data_ptr(), _at(dev_err), st),
                  "mla_cache_evict")
        else:
            check(_fn("mla_cache_evict_at")(B, n_max, rows, n_planes, acc.data_ptr(), acc_b, lengths.data_ptr(), keep,
                                            sink, recent, positions.data_ptr(), pos_b, new_lengths.data_ptr(),
                                            row_map.data_ptr(), _at(dev_err), st), "mla_cache_evict_at")
    return new_lengths, row_map


def mla_clear_device_error(dev_err: torch.Tensor, stream=None) -> None:
    check(lib().mla_clear_device_error(_ptr(dev_err), _stream(stream)), "mla_clear_device_error")


def mla_get_device_error(dev_err: torch.Tensor) -> int:
    out = ctypes.c_int32(0)
    check(lib().mla_get_device_error(_ptr(dev_err), ctypes.byref(out)), "mla_get_device_error")
    return int(out.value)
