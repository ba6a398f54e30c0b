"""Group-scaled 4-bit weights (include/mq.h): quantization, packing of a checkpoint's codes,
reading back, and products of rows that are not quantized, dense and by expert.

32, 64 or 128 consecutive inputs of a row share a 16-bit scale s and zero point z; a weight
is s * (code - z). As in mx.py, a call with all as it should be is done by the extension
module _binding; the rest of each function tells what is wrong, or makes another device or
stream current first.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import MQError, _binding, _lib
from .experts import ExpertPlan, _no_tangent, _plan
from .mx import _TYPES, _apart, _changed, _check, _current_device, _input, _on, _output, _raw_stream

GROUPS = (32, 64, 128)
_SCALE_TYPES = (torch.float16, torch.bfloat16)


class W4(NamedTuple):
    """A matrix of group-scaled 4-bit weights, or a batch of them (experts' weights), in the
    library's device layout: `codes` u8 [(batch,) row tiles, column tiles, 1024], `scales`
    (fp16 or bf16) [(batch,) row tiles, quads, 16, 512 / group], `zeros` the same or None (a zero
    point of 8 everywhere), the matrix's own sizes and its group."""
    codes: torch.Tensor
    scales: torch.Tensor
    zeros: torch.Tensor | None
    rows: int
    cols: int
    group: int


if _binding is not None:
    _binding.types_w4(W4)
_quantize, _pack, _dequantize = _lib.mq_w4_quantize, _lib.mq_w4_pack, _lib.mq_w4_dequantize
_linear, _linear_workspace = _lib.mq_w4_linear, _lib.mq_w4_linear_workspace_bytes
_experts, _experts_workspace = _lib.mq_w4_experts, _lib.mq_w4_experts_workspace_bytes


def _group(group):
    if isinstance(group, bool) or group not in GROUPS:
        raise ValueError(f"group must be one of {GROUPS}, got {group!r}")
    return group


def _scale_type(dtype, name):
    if dtype not in _SCALE_TYPES:
        raise TypeError(f"{name} must be float16 or bfloat16, got {dtype}")
    return _TYPES[dtype]


def _shapes(R, K, group, batch):
    lead = () if batch is None else (batch,)
    tiles = (R + 15) // 16
    return lead + (tiles, (K + 127) // 128, 1024), lead + (tiles, (K + 511) // 512, 16, 512 // group)


def _w4(a, name, index, batch=None):
    """A matrix, or a batch of this many: its tensors have the sizes its own sizes ask for."""
    if not isinstance(a, W4) or len(a) != 6:
        raise TypeError(f"{name} must be a W4 matrix (w4_quantize, w4_pack)")
    codes, scales, zeros, rows, cols, group = a
    c, s = _shapes(rows, cols, _group(group), batch)
    _check(codes, f"{name}.codes", torch.uint8, c, index)
    if not isinstance(scales, torch.Tensor):
        raise TypeError(f"{name}.scales must be a torch.Tensor")
    _scale_type(scales.dtype, f"{name}.scales")
    _check(scales, f"{name}.scales", scales.dtype, s, index)
    if zeros is not None:
        _check(zeros, f"{name}.zeros", scales.dtype, s, index)
    return a


def _pointers(a):
    return a.codes.data_ptr(), a.scales.data_ptr(), None if a.zeros is None else a.zeros.data_ptr()


def _new(R, K, group, batch, dtype, zeros, device):
    c, s = _shapes(R, K, group, batch)
    return W4(torch.empty(c, dtype=torch.uint8, device=device), torch.empty(s, dtype=dtype, device=device),
              torch.empty(s, dtype=dtype, device=device) if zeros else None, R, K, group)


def _no_gradient(*inputs):
    _no_tangent(*inputs)
    if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad for t in inputs):
        raise ValueError("this product has no gradient: detach its inputs, or call it under torch.no_grad()")


def w4_quantize(x, group: int = 128, zeros: bool = False, scale_dtype=torch.float16, out=None, stream=None) -> W4:
    """x [R, K] or [B, R, K] (fp32, bf16, fp16; the last axis contiguous, other strides free)
    to 4-bit codes: without zeros the scale is max|x| / 7 over the group, with them it and a
    zero point span the group's range (0 in it). A group with a NaN or an infinity reads back
    as NaN. out: a W4 of the same sizes, group and types to write to."""
    if stream is None and _binding is not None:
        done = _binding.w4_quantize(x, group, zeros, scale_dtype, out)
        if done is not None:
            return done
    batched = isinstance(x, torch.Tensor) and x.dim() == 3
    code = _input(x, "x", 3 if batched else 2)
    _group(group)
    scale_code = _scale_type(scale_dtype, "scale_dtype")
    R, K = x.shape[-2:]
    if K == 0:
        raise ValueError("x has no columns")
    index = x.get_device()
    if stream is not None or index < 0 or index != _current_device():
        with _on(index, stream, x, out):
            return w4_quantize(x, group, zeros, scale_dtype, out)
    batch = x.shape[0] if batched else None
    if out is None:
        out = _new(R, K, group, batch, scale_dtype, zeros, x.device)
    else:
        _w4(out, "out", index, batch)
        if out[3:] != (R, K, group) or out.scales.dtype != scale_dtype or (out.zeros is not None) != bool(zeros):
            raise ValueError(f"out is {out.rows} x {out.cols} of group {out.group}, {out.scales.dtype}, not what is asked for")
        _changed(out.codes, out.scales, *(() if out.zeros is None else (out.zeros,)))
    rc = _quantize(x.data_ptr(), code, batch if batched else 1, x.stride(0) if batched else 0, R, x.stride(-2), K, group,
                   scale_code, *_pointers(out), _raw_stream(index))
    if rc:
        raise MQError("mq_w4_quantize", rc)
    return out


def w4_pack(codes, scales, zeros=None, group: int = 128, stream=None) -> W4:
    """Weights that are quantized already: codes u8 [R, K] or [B, R, K], one to a byte (the low four
    bits count; a checkpoint that holds several in a word is unpacked first), scales and zeros (or None: 8) fp16 or bf16
    [(B,) R, ceil(K / group)]; a weight is scale * (code - zero)."""
    if stream is None and _binding is not None:
        done = _binding.w4_pack(codes, scales, zeros, group)
        if done is not None:
            return done
    if not isinstance(codes, torch.Tensor) or codes.dtype is not torch.uint8 or codes.dim() not in (2, 3):
        raise TypeError("codes must be a uint8 tensor [R, K] or [B, R, K]")
    if codes.stride(-1) != 1 and codes.shape[-1] > 1:
        raise ValueError("codes' last axis must be contiguous")
    _group(group)
    if not isinstance(scales, torch.Tensor):
        raise TypeError("scales must be a torch.Tensor")
    _scale_type(scales.dtype, "scales")
    index = codes.get_device()
    if stream is not None or index < 0 or index != _current_device():
        with _on(index, stream, codes, scales, zeros):
            return w4_pack(codes, scales, zeros, group)
    R, K = codes.shape[-2:]
    if K == 0:
        raise ValueError("codes have no columns")
    batch = codes.shape[0] if codes.dim() == 3 else None
    per = tuple(codes.shape[:-1]) + ((K + group - 1) // group,)
    _check(scales, "scales", scales.dtype, per, index)
    if zeros is not None:
        _check(zeros, "zeros", scales.dtype, per, index)
    out = _new(R, K, group, batch, scales.dtype, zeros is not None, codes.device)
    rc = _pack(codes.data_ptr(), 1 if batch is None else batch, 0 if batch is None else codes.stride(0), R, codes.stride(-2),
               K, group, scales.data_ptr(), None if zeros is None else zeros.data_ptr(), *_pointers(out), _raw_stream(index))
    if rc:
        raise MQError("mq_w4_pack", rc)
    return out


def w4_dequantize(a: W4, dtype=torch.float32, out=None, stream=None):
    """The weights of a matrix (or batch), [(B,) R, K]."""
    if stream is None and _binding is not None:
        done = _binding.w4_dequantize(a, dtype, out)
        if done is not None:
            return done
    if not isinstance(a, W4) or len(a) != 6:
        raise TypeError("a must be a W4 matrix (w4_quantize, w4_pack)")
    index = a.codes.get_device()
    if stream is not None or index < 0 or index != _current_device():
        with _on(index, stream, a, out):
            return w4_dequantize(a, dtype, out)
    batch = a.codes.shape[0] if a.codes.dim() == 4 else None
    _w4(a, "a", index, batch)
    R, K = a.rows, a.cols
    out = _output(out, "out", (R, K) if batch is None else (batch, R, K), dtype if out is None else out.dtype, index)
    rc = _dequantize(*_pointers(a), _TYPES[a.scales.dtype], 1 if batch is None else batch, R, K, a.group, out.data_ptr(),
                     _TYPES[out.dtype], _raw_stream(index))
    if rc:
        raise MQError("mq_w4_dequantize", rc)
    return out


def w4_linear(x, w: W4, bias=None, out_dtype=torch.bfloat16, y=None, stream=None):
    """y = x w^T + bias: x [M, K] (fp32, bf16, fp16) as it is, w a W4 matrix [N, K], bias fp32
    [N]. Without gradient: x and bias that ask for one, or carry a tangent, are refused."""
    if stream is None and _binding is not None:
        done = _binding.w4_linear(x, w, bias, out_dtype, y)
        if done is not None:
            return done
    code = _input(x, "x", 2)
    _no_gradient(x, bias)
    index = x.get_device()
    if stream is not None or index < 0 or index != _current_device():
        with _on(index, stream, x, w, bias, y):
            return w4_linear(x, w, bias, out_dtype, y)
    _w4(w, "w", index)
    M, K = x.shape
    if K != w.cols:
        raise ValueError(f"x has {K} inputs, w has {w.cols}")
    N = w.rows
    b = None if bias is None else _check(bias, "bias", torch.float32, (N,), index).data_ptr()
    y = _apart(_output(y, "y", (M, N), out_dtype if y is None else y.dtype, index), "y", x, "x")
    need = _linear_workspace(M, N, K, code, w.group)
    work = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
    rc = _linear(x.data_ptr(), code, x.stride(0), *_pointers(w), _TYPES[w.scales.dtype], w.group, M, N, K, b, y.data_ptr(),
                 _TYPES[y.dtype], work.data_ptr() if need else None, need, _raw_stream(index))
    if rc:
        raise MQError("mq_w4_linear", rc)
    return y


def w4_experts_linear(x, w: W4, plan: ExpertPlan, by_token: bool = False, out_dtype=torch.bfloat16, y=None, stream=None):
    """y [rows, N]: for each row p of the plan x[p] w[e]^T, e the row's expert, zero for rows of
    no token. x [rows, K], or by_token [T, K], where row p takes its token's; w: a W4 batch
    [experts, N, K]. Without gradient: an x that asks for one, or carries a tangent, is refused."""
    if stream is None and _binding is not None:
        done = _binding.w4_experts(x, w, plan, by_token, out_dtype, y)
        if done is not None:
            return done
    code = _input(x, "x", 2)
    _no_gradient(x)
    index = x.get_device()
    if stream is not None or index < 0 or index != _current_device():
        with _on(index, stream, x, w, plan, y):
            return w4_experts_linear(x, w, plan, by_token, out_dtype, y)
    T, k, E, rows = _plan(plan, index)
    _w4(w, "w", index, E)
    N, K = w.rows, w.cols
    need = (T if by_token else rows, K)
    if x.shape != need:
        raise ValueError(f"x must be [{need[0]}, {K}] for this plan and these weights, got {tuple(x.shape)}")
    y = _apart(_output(y, "y", (rows, N), out_dtype if y is None else y.dtype, index), "y", x, "x")
    size = _experts_workspace(T, k, E, N, K, bool(by_token), code, w.group)
    work = torch.empty(size, dtype=torch.uint8, device=x.device) if size else None
    rc = _experts(x.data_ptr(), code, x.stride(0), bool(by_token), T, k, E, N, K, plan.offsets.data_ptr(),
                  plan.row_token.data_ptr(), *_pointers(w), _TYPES[w.scales.dtype], w.group, y.data_ptr(), _TYPES[y.dtype],
                  work.data_ptr() if size else None, size, _raw_stream(index))
    if rc:
        raise MQError("mq_w4_experts", rc)
    return y
