"""Microscaled 4-bit matrices (include/mq.h): quantization, reading back, products.

32 consecutive inputs of a row share a power-of-two scale, values are 4-bit floats. The
functions check and marshal device tensors; all of the work runs in libmq.so. A call
with all as it should be, on the current device and stream, is done by the extension
module _binding (csrc/binding.cpp), which costs the host about half of what the same
steps cost in Python; the rest of each function tells what is wrong, or makes another
device or stream current first. Where the module is not there, it does all calls.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import MQError, _binding, _lib

_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}   # MQ_F32, MQ_BF16, MQ_F16

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


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


def _check(t, name, dtype, shape, index):
    """A contiguous tensor of this type and shape on device `index`."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index \
            and t.is_contiguous():
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


def _whole(a, name):
    """The items of an MX, all of them."""
    if not isinstance(a, MX) or len(a) != 4:
        raise TypeError(f"{name} must be an MX matrix (mx_quantize)")
    return a


def _mx(a, name, index, batch=None):
    """A microscaled operand: its tensors have the sizes its rows and cols ask for."""
    codes, scales, rows, cols = _whole(a, name)
    tiles, groups = (rows + 15) // 16, (cols + 127) // 128
    if batch is None:
        _check(codes, f"{name}.codes", torch.uint8, (tiles, groups, 1024), index)
        _check(scales, f"{name}.scales", torch.uint8, (tiles, (groups + 3) // 4, 256), index)
    else:
        _check(codes, f"{name}.codes", torch.uint8, (batch, tiles, groups, 1024), index)
        _check(scales, f"{name}.scales", torch.uint8, (batch, tiles, (groups + 3) // 4, 256), index)
    return a


def _changed(*given):
    """The caller's outputs are about to be written: a gradient that kept what they held is told."""
    for t in given:
        if not t.is_inference():
            torch.autograd.graph.increment_version(t)


def _apart(y, name, x, other):
    """An output of the caller's is not memory that is still read."""
    spans = []
    for t in (y, x):
        last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
        spans.append((t.data_ptr(), t.data_ptr() + ((last + 1) * t.element_size() if t.numel() else 0)))
    if spans[0][0] < spans[1][1] and spans[1][0] < spans[0][1]:
        raise ValueError(f"{name} shares memory with {other}")
    return y


def _output(y, name, shape, dtype, index):
    if y is None:
        _type(dtype, name)
        return torch.empty(shape, dtype=dtype, device=f"cuda:{index}")
    _type(y.dtype if isinstance(y, torch.Tensor) else dtype, name)
    _check(y, name, dtype, shape, index)
    if y.data_ptr() % 16:
        raise ValueError(f"{name} must be 16-byte aligned")
    _changed(y)
    return y


def _on(index, stream, *operands):
    """The context in which device `index` and the launch stream are current, so that what
    a call allocates belongs to the stream that uses it. With a stream of the caller's
    choice the operands are marked as used on it: their memory is not given away before
    its work is done."""
    if index < 0:
        raise ValueError("operands must be device tensors")
    if stream is None:
        return torch.cuda.device(index)
    if stream.device.index != index:
        raise ValueError(f"the stream is on {stream.device}, the operands on cuda:{index}")
    for t in operands:
        for u in t if isinstance(t, tuple) else (t,):
            if isinstance(u, torch.Tensor) and u.is_cuda:
                u.record_stream(stream)
    return torch.cuda.stream(stream)


_quantize, _dequantize = _lib.mq_mx_quantize, _lib.mq_mx_dequantize
_gemm, _linear, _linear_workspace = _lib.mq_mx_gemm, _lib.mq_mx_linear, _lib.mq_mx_linear_workspace_bytes


def mx_quantize(x, out=None, stream=None) -> MX:
    """x [R, K] or [B, R, K] (fp32, bf16, fp16; the last axis contiguous, other strides
    free) to microscaled 4-bit. A block of 32 with a NaN or an infinity reads back as NaN.
    out: an MX of the same sizes to write to."""
    if stream is None and _binding is not None:
        done = _binding.quantize(x, out)
        if done is not None:
            return done
    batched = isinstance(x, torch.Tensor) and x.dim() == 3
    code = _input(x, "x", 3 if batched else 2)
    shape = x.shape
    R, K = shape[-2:]
    if K == 0:
        raise ValueError("x has no columns")
    index = x.get_device()
    if stream is not None or index < 0 or index != _current_device():
        with _on(index, stream, x, out):
            return mx_quantize(x, out)
    if out is None:
        tiles, groups = (R + 15) // 16, (K + 127) // 128
        quads = (groups + 3) // 4
        lead = (shape[0],) if batched else ()
        out = MX(torch.empty(lead + (tiles, groups, 1024), dtype=torch.uint8, device=x.device),
                 torch.empty(lead + (tiles, quads, 256), dtype=torch.uint8, device=x.device), R, K)
    else:
        if _whole(out, "out")[2:] != (R, K):
            raise ValueError(f"out is {out.rows} x {out.cols}, x is {R} x {K}")
        _mx(out, "out", index, shape[0] if batched else None)
    rc = _quantize(x.data_ptr(), code, shape[0] if batched else 1, x.stride(0) if batched else 0, R, x.stride(-2), K,
                   out[0].data_ptr(), out[1].data_ptr(), _raw_stream(index))
    if rc:
        raise MQError("mq_mx_quantize", rc)
    return out


def mx_dequantize(a: MX, dtype=torch.float32, out=None, stream=None):
    """The values of a microscaled matrix (or batch), [(B,) R, K]."""
    if stream is None and _binding is not None:
        done = _binding.dequantize(a, dtype, out)
        if done is not None:
            return done
    codes, scales, R, K = _whole(a, "a")
    index = codes.get_device()
    if stream is not None or index < 0 or index != _current_device():
        with _on(index, stream, a, out):
            return mx_dequantize(a, dtype, out)
    batch = codes.shape[0] if codes.dim() == 4 else None
    _mx(a, "a", index, batch)
    out = _output(out, "out", (R, K) if batch is None else (batch, R, K), dtype if out is None else out.dtype, index)
    rc = _dequantize(codes.data_ptr(), scales.data_ptr(), 1 if batch is None else batch, R, K, out.data_ptr(),
                     _TYPES[out.dtype], _raw_stream(index))
    if rc:
        raise MQError("mq_mx_dequantize", rc)
    return out


def mx_linear(x, w: MX, bias=None, out_dtype=torch.bfloat16, y=None, stream=None):
    """y = Q(x) w^T + bias: x [M, K] (fp32, bf16, fp16), quantized on the way, or an MX
    matrix; w an MX matrix [N, K]; bias fp32 [N]."""
    if stream is None and _binding is not None:
        done = _binding.linear(x, w, bias, out_dtype, y)
        if done is not None:
            return done
    ready = isinstance(x, MX)
    if ready:
        index = _whole(x, "x").codes.get_device()
    else:
        code = _input(x, "x", 2)
        index = x.get_device()
    if stream is not None or index < 0 or index != _current_device():
        with _on(index, stream, x, w, bias, y):
            return mx_linear(x, w, bias, out_dtype, y)
    _mx(w, "w", index)
    if ready:
        M, K = x.rows, x.cols
        _mx(x, "x", index)
    else:
        M, K = x.shape
    if K != w.cols:
        raise ValueError(f"x has {K} inputs, w has {w.cols}")
    N = w.rows
    b = None if bias is None else _check(bias, "bias", torch.float32, (N,), index).data_ptr()
    y = _output(y, "y", (M, N), out_dtype if y is None else y.dtype, index)
    if ready:
        rc = _gemm(x.codes.data_ptr(), x.scales.data_ptr(), w.codes.data_ptr(), w.scales.data_ptr(), M, N, K, b,
                   y.data_ptr(), _TYPES[y.dtype], _raw_stream(index))
    else:
        need = _linear_workspace(M, N, K)
        work = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
        rc = _linear(x.data_ptr(), code, x.stride(0), w.codes.data_ptr(), w.scales.data_ptr(), M, N, K, b, y.data_ptr(),
                     _TYPES[y.dtype], work.data_ptr() if need else None, need, _raw_stream(index))
    if rc:
        raise MQError("mq_mx_gemm" if ready else "mq_mx_linear", rc)
    return y
