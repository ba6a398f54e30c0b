"""Routing to experts, the plan of a batch's rows by expert, and the experts' products
over microscaled 4-bit weights (include/mq.h)."""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import MQError, _binding, _lib
from .mx import _TYPES, MX, _check, _current_device, _input, _mx, _on, _output, _raw_stream

_SCORES = {"softmax": 0, "sigmoid": 1}        # MQ_SCORE_*
_GROUP_SCORES = {"max": 0, "top2": 1}         # MQ_GROUP_*


class ExpertPlan(NamedTuple):
    """A batch's rows by expert: one row per (token, slot) with an expert, each expert's
    rows from a multiple of 16 on. offsets int32 [experts + 1], row_token int32 [rows]
    (-1: no token), row_of int32 [T, k] (-1: no row)."""
    offsets: torch.Tensor
    row_token: torch.Tensor
    row_of: torch.Tensor


if _binding is not None:
    _binding.types(MX, ExpertPlan)
_route, _plan_rows, _expert_plan = _lib.mq_route, _lib.mq_plan_rows, _lib.mq_expert_plan
_up, _up_workspace = _lib.mq_mx_experts_up, _lib.mq_mx_experts_up_workspace_bytes
_down, _down_workspace = _lib.mq_mx_experts_down, _lib.mq_mx_experts_down_workspace_bytes


def plan_rows(T: int, k: int, experts: int) -> int:
    """Rows of a plan of T tokens with k slots each: the most that any ids can take."""
    rows = _plan_rows(T, k, experts)
    if rows < 0:
        raise ValueError(f"no plan for {T} tokens of {k} slots and {experts} experts")
    return rows


def route(logits, k: int, score: str = "softmax", bias=None, groups: int = 1, top_groups: int | None = None,
          group_score: str = "max", renormalize: bool = True, scale: float = 1.0, ids=None, weights=None, stream=None):
    """The k experts of each token and their weights (ids int32 [T, k], weights fp32 [T, k])
    from logits [T, E]. Scores are softmax or sigmoid; a bias [E] (fp32) is added for the
    choice alone; with top_groups < groups only experts of the best groups are taken
    ("max": a group's largest key, "top2": the sum of its two largest). Logits of -inf mask
    experts: slots that none is left for have id -1 and weight 0. A NaN gives ids -1 and
    weights NaN."""
    if stream is None and _binding is not None:
        done = _binding.route(logits, k, _SCORES.get(score, -1), bias, groups, groups if top_groups is None else top_groups,
                              _GROUP_SCORES.get(group_score, -1), renormalize, float(scale), ids, weights)
        if done is not None:
            return done
    code = _input(logits, "logits", 2)
    T, E = logits.shape
    score_code, group_code = _SCORES.get(score), _GROUP_SCORES.get(group_score)
    if score_code is None:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    if group_code is None:
        raise ValueError(f"group_score must be one of {sorted(_GROUP_SCORES)}, got {group_score!r}")
    if top_groups is None:
        top_groups = groups
    if groups <= 0 or E % groups or not 0 < top_groups <= groups:
        raise ValueError(f"{E} experts do not make {groups} groups of which {top_groups} are kept")
    if not 0 < k <= top_groups * (E // groups):
        raise ValueError(f"k = {k} experts of {top_groups * (E // groups)}")
    index = logits.get_device()
    if stream is not None or index < 0 or index != _current_device():
        with _on(index, stream, logits, bias, ids, weights):
            return route(logits, k, score, bias, groups, top_groups, group_score, renormalize, scale, ids, weights)
    b = None if bias is None else _check(bias, "bias", torch.float32, (E,), index).data_ptr()
    if ids is None:
        ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    else:
        _check(ids, "ids", torch.int32, (T, k), index)
    if weights is None:
        weights = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    else:
        _check(weights, "weights", torch.float32, (T, k), index)
    rc = _route(logits.data_ptr(), code, T, logits.stride(0), E, b, score_code, groups, top_groups, group_code, k,
                1 if renormalize else 0, scale, ids.data_ptr(), weights.data_ptr(), _raw_stream(index))
    if rc:
        raise MQError("mq_route", rc)
    return ids, weights


def expert_plan(ids, experts: int, stream=None) -> ExpertPlan:
    """The plan of ids int32 [T, k]. Ids outside [0, experts), such as -1 or another
    rank's experts, get no row."""
    if stream is None and _binding is not None:
        done = _binding.expert_plan(ids, experts)
        if done is not None:
            return done
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2 or ids.dtype is not torch.int32:
        raise ValueError("ids must be an int32 tensor [T, k]")
    T, k = ids.shape
    index = ids.get_device()
    if stream is not None or index < 0 or index != _current_device():
        with _on(index, stream, ids):
            return expert_plan(ids, experts)
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    rows = _plan_rows(T, k, experts)
    if rows < 0:
        raise ValueError(f"no plan for {T} tokens of {k} slots and {experts} experts")
    offsets = torch.empty(experts + 1, dtype=torch.int32, device=ids.device)
    row_token = torch.empty(rows, dtype=torch.int32, device=ids.device)
    row_of = torch.empty_like(ids)
    rc = _expert_plan(ids.data_ptr(), T, k, experts, offsets.data_ptr(), row_token.data_ptr(), row_of.data_ptr(),
                      _raw_stream(index))
    if rc:
        raise MQError("mq_expert_plan", rc)
    return ExpertPlan(offsets, row_token, row_of)


def _plan(plan, index):
    """(T, k, experts, rows) of a plan, its tensors checked."""
    if not isinstance(plan, ExpertPlan) or len(plan) != 3:
        raise TypeError("plan must be an ExpertPlan (expert_plan)")
    offsets, row_token, row_of = plan
    T, k = row_of.shape
    E = offsets.shape[0] - 1
    rows = plan_rows(T, k, E)
    _check(offsets, "plan.offsets", torch.int32, (E + 1,), index)
    _check(row_token, "plan.row_token", torch.int32, (rows,), index)
    _check(row_of, "plan.row_of", torch.int32, (T, k), index)
    return T, k, E, rows


def mx_experts_up(x, w_gate: MX, w_up: MX, plan: ExpertPlan, out_dtype=torch.bfloat16, h=None, stream=None):
    """h [rows, I]: for each row of the plan silu(Q(x[t]) w_gate[e]^T) * (Q(x[t]) w_up[e]^T),
    zero for rows of no token. x [T, D]; w_gate, w_up: MX batches [experts, I, D]."""
    if stream is None and _binding is not None:
        done = _binding.experts_up(x, w_gate, w_up, plan, out_dtype, h)
        if done is not None:
            return done
    code = _input(x, "x", 2)
    index = x.get_device()
    if stream is not None or index < 0 or index != _current_device():
        with _on(index, stream, x, w_gate, w_up, plan, h):
            return mx_experts_up(x, w_gate, w_up, plan, out_dtype, h)
    T, k, E, rows = _plan(plan, index)
    _mx(w_gate, "w_gate", index, E)
    _mx(w_up, "w_up", index, E)
    D, I = w_gate.cols, w_gate.rows
    if (w_up.rows, w_up.cols) != (I, D):
        raise ValueError(f"w_gate is {I} x {D}, w_up is {w_up.rows} x {w_up.cols}")
    if x.shape != (T, D):
        raise ValueError(f"x must be [{T}, {D}] for this plan and these weights, got {tuple(x.shape)}")
    h = _output(h, "h", (rows, I), out_dtype if h is None else h.dtype, index)
    need = _up_workspace(T, k, E, D, I)
    work = torch.empty(need, dtype=torch.uint8, device=plan.offsets.device) if need else None
    rc = _up(x.data_ptr(), code, x.stride(0), T, k, E, D, I, plan.offsets.data_ptr(), plan.row_token.data_ptr(),
             plan.row_of.data_ptr(), w_gate.codes.data_ptr(), w_gate.scales.data_ptr(), w_up.codes.data_ptr(),
             w_up.scales.data_ptr(), h.data_ptr(), _TYPES[h.dtype], work.data_ptr() if need else None, need,
             _raw_stream(index))
    if rc:
        raise MQError("mq_mx_experts_up", rc)
    return h


def mx_experts_down(h, w_down: MX, plan: ExpertPlan, weights, out_dtype=torch.bfloat16, y=None, stream=None):
    """y[t] = sum over slots j of weights[t, j] * (Q(h[row_of[t, j]]) w_down[e]^T), in the order
    of the slots. h [rows, I], weights fp32 [T, k], w_down: MX batch [experts, D, I]."""
    if stream is None and _binding is not None:
        done = _binding.experts_down(h, w_down, plan, weights, out_dtype, y)
        if done is not None:
            return done
    code = _input(h, "h", 2)
    index = h.get_device()
    if stream is not None or index < 0 or index != _current_device():
        with _on(index, stream, h, w_down, plan, weights, y):
            return mx_experts_down(h, w_down, plan, weights, out_dtype, y)
    T, k, E, rows = _plan(plan, index)
    _mx(w_down, "w_down", index, E)
    D, I = w_down.rows, w_down.cols
    _check(h, "h", h.dtype, (rows, I), index)
    _check(weights, "weights", torch.float32, (T, k), index)
    y = _output(y, "y", (T, D), out_dtype if y is None else y.dtype, index)
    need = _down_workspace(T, k, E, D, I)
    work = torch.empty(need, dtype=torch.uint8, device=plan.offsets.device) if need else None
    rc = _down(h.data_ptr(), code, T, k, E, D, I, plan.offsets.data_ptr(), plan.row_of.data_ptr(), weights.data_ptr(),
               w_down.codes.data_ptr(), w_down.scales.data_ptr(), y.data_ptr(), _TYPES[y.dtype],
               work.data_ptr() if need else None, need, _raw_stream(index))
    if rc:
        raise MQError("mq_mx_experts_down", rc)
    return y


def mx_experts(x, w_gate: MX, w_up: MX, w_down: MX, plan: ExpertPlan, weights, out_dtype=torch.bfloat16, stream=None,
               h_dtype=torch.bfloat16):
    """A mixture's feed-forward layer of x [T, D]: mx_experts_up (its result in h_dtype), then
    mx_experts_down."""
    h = mx_experts_up(x, w_gate, w_up, plan, out_dtype=h_dtype, stream=stream)
    return mx_experts_down(h, w_down, plan, weights, out_dtype=out_dtype, stream=stream)
