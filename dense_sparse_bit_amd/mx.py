"""Microscaled 4-bit matrices (include/mq.h): quantization, reading back, products.

32 consecutive inputs of a row share a power-of-two scale, values are 4-bit floats. The
functions check and marshal device tensors; all of the work runs in libmq.so.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import MQError, _lib

_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}   # MQ_F32, MQ_BF16, MQ_F16


class MX(NamedTuple):
    """A microscaled matrix, or a batch of them (experts' weights), in the library's
    device layout: `codes` u8 [(batch,) row tiles, groups, 1024], `scales` u8
    [(batch,) row tiles, quads, 256], and the matrix's own sizes."""
    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int


def _type(dtype, name):
    code = _TYPES.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {dtype}")
    return code


def _input(x, name, dims):
    """A strided device matrix whose last axis is contiguous."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _type(x.dtype, name)
    if x.dim() != dims:
        raise ValueError(f"{name} must have {dims} axes, got shape {tuple(x.shape)}")
    if x.stride(-1) != 1 and x.shape[-1] > 1:
        raise ValueError(f"{name}'s last axis must be contiguous")
    return code


def _check(t, name, dtype, shape, device):
    """A contiguous device tensor of this type and shape."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _mx(a, name, device, batch=None):
    """A microscaled operand: its tensors have the sizes its rows and cols ask for."""
    if not isinstance(a, MX):
        raise TypeError(f"{name} must be an MX matrix (mx_quantize)")
    lead = () if batch is None else (batch,)
    tiles, groups = (a.rows + 15) // 16, (a.cols + 127) // 128
    _check(a.codes, f"{name}.codes", torch.uint8, lead + (tiles, groups, 1024), device)
    _check(a.scales, f"{name}.scales", torch.uint8, lead + (tiles, (groups + 3) // 4, 256), device)
    return a


def _output(y, name, shape, dtype, device):
    _type(dtype, name)
    if y is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _check(y, name, dtype, shape, device)
    if y.data_ptr() % 16:
        raise ValueError(f"{name} must be 16-byte aligned")
    return y


class _Launch:
    """Makes the tensors' device and the launch stream current, so that what a call
    allocates belongs to the stream that uses it; `.stream` is the raw handle. With a
    stream of the caller's choice the operands are marked as used on it: their memory
    is not given away before its work is done."""

    def __init__(self, device, stream, *operands):
        if device.type != "cuda":
            raise ValueError("operands must be device tensors")
        self.ctx = None
        if stream is not None:
            self.ctx = torch.cuda.stream(stream)
            if stream.device != device:
                raise ValueError(f"the stream is on {stream.device}, the operands on {device}")
            for t in operands:
                for u in t if isinstance(t, tuple) else (t,):
                    if isinstance(u, torch.Tensor) and u.is_cuda:
                        u.record_stream(stream)
        elif device.index != torch.cuda.current_device():
            self.ctx = torch.cuda.device(device)
        self.index = device.index

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        self.stream = torch.cuda.current_stream(self.index).cuda_stream
        return self

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _call(name, *args):
    rc = getattr(_lib, name)(*args)
    if rc != 0:
        raise MQError(name, rc)


def mx_quantize(x, out=None, stream=None) -> MX:
    """x [R, K] or [B, R, K] (fp32, bf16, fp16; the last axis contiguous, other strides
    free) to microscaled 4-bit. A block of 32 with a NaN or an infinity reads back as NaN.
    out: an MX of the same sizes to write to."""
    batched = isinstance(x, torch.Tensor) and x.dim() == 3
    code = _input(x, "x", 3 if batched else 2)
    R, K = x.shape[-2:]
    if K == 0:
        raise ValueError("x has no columns")
    B = x.shape[0] if batched else 1
    if out is not None and (out.rows, out.cols) != (R, K):
        raise ValueError(f"out is {out.rows} x {out.cols}, x is {R} x {K}")
    with _Launch(x.device, stream, x) as at:
        if out is None:
            tiles, groups = (R + 15) // 16, (K + 127) // 128
            lead = (B,) if batched else ()
            out = MX(torch.empty(lead + (tiles, groups, 1024), dtype=torch.uint8, device=x.device),
                     torch.empty(lead + (tiles, (groups + 3) // 4, 256), dtype=torch.uint8, device=x.device), R, K)
        else:
            _mx(out, "out", x.device, B if batched else None)
        _call("mq_mx_quantize", x.data_ptr(), code, B, x.stride(0) if batched else 0, R, x.stride(-2), K,
              out.codes.data_ptr(), out.scales.data_ptr(), at.stream)
    return out


def mx_dequantize(a: MX, dtype=torch.float32, out=None, stream=None):
    """The values of a microscaled matrix (or batch), [(B,) R, K]."""
    if not isinstance(a, MX):
        raise TypeError("a must be an MX matrix (mx_quantize)")
    batch = a.codes.shape[0] if a.codes.dim() == 4 else None
    device = a.codes.device
    with _Launch(device, stream, a) as at:
        _mx(a, "a", device, batch)
        lead = () if batch is None else (batch,)
        out = _output(out, "out", lead + (a.rows, a.cols), dtype if out is None else out.dtype, device)
        _call("mq_mx_dequantize", a.codes.data_ptr(), a.scales.data_ptr(), 1 if batch is None else batch, a.rows, a.cols,
              out.data_ptr(), _TYPES[out.dtype], at.stream)
    return out


def mx_linear(x, w: MX, bias=None, out_dtype=torch.bfloat16, y=None, stream=None):
    """y = Q(x) w^T + bias: x [M, K] (fp32, bf16, fp16), quantized on the way, or an MX
    matrix; w an MX matrix [N, K]; bias fp32 [N]."""
    ready = isinstance(x, MX)
    device = x.codes.device if ready else x.device
    with _Launch(device, stream, x, w, bias) as at:
        _mx(w, "w", device)
        if ready:
            M, K = x.rows, x.cols
            _mx(x, "x", device)
        else:
            code = _input(x, "x", 2)
            M, K = x.shape
        if K != w.cols:
            raise ValueError(f"x has {K} inputs, w has {w.cols}")
        N = w.rows
        if bias is not None:
            _check(bias, "bias", torch.float32, (N,), device)
        y = _output(y, "y", (M, N), out_dtype if y is None else y.dtype, device)
        b = None if bias is None else bias.data_ptr()
        if ready:
            _call("mq_mx_gemm", x.codes.data_ptr(), x.scales.data_ptr(), w.codes.data_ptr(), w.scales.data_ptr(), M, N,
                  K, b, y.data_ptr(), _TYPES[y.dtype], at.stream)
        else:
            need = _lib.mq_mx_linear_workspace_bytes(M, N, K)
            work = torch.empty(need, dtype=torch.uint8, device=device) if need else None
            _call("mq_mx_linear", x.data_ptr(), code, x.stride(0), w.codes.data_ptr(), w.scales.data_ptr(), M, N, K, b,
                  y.data_ptr(), _TYPES[y.dtype], None if work is None else work.data_ptr(), need, at.stream)
    return y
