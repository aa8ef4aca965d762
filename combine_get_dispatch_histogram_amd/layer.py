"""The block around the experts (``include/miep.h``, "the block around them").

  gate_topk(logits, num_topk) -> topk_idx, topk_weights       the router's choice, as dispatch takes it
  gate_topk_backward                                          gradient of the logits
  linear(x, w, bias, activation, residual)                    dense product with its epilogue: router, shared expert
  linear_backward                                             gradients of its rows, weight and bias
  expert_layer / expert_layer_fp8(x, topk_idx, topk_weights, w1, w2)
                                                              a few tokens through their experts and back, in place of
                                                              dispatch, the experts' products and combine (decoding)

As everywhere in this package the ``*_into`` variants take preallocated outputs and allocate nothing.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib
from ._call import _Args, _run

_BF16, _F32, _I64 = torch.bfloat16, torch.float32, torch.int64
_FP8 = (torch.float8_e4m3fn, torch.uint8)
_ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4, "swiglu": 5}
_SCORES = {"softmax": 0, "sigmoid": 1}


# --------------------------------------------------------------------------- router
def _gate(logits, num_topk, score, num_groups, topk_groups, group_best, renormalize, scale) -> _lib.GateC:
    if len(logits.shape) != 2:
        raise ValueError("logits must be [tokens, experts]")
    if score not in _SCORES:
        raise ValueError("score must be one of %s, got %r" % (sorted(_SCORES), score))
    kind = logits.dtype
    if kind != _F32 and kind != _BF16:
        raise TypeError("logits must be float32 or bfloat16, got %s" % kind)
    N, E = logits.shape
    return _lib.GateC(N, E, num_topk, _SCORES[score], bool(renormalize), num_groups, topk_groups, group_best, kind == _F32, scale)


def gate_topk_into(logits, topk_idx, topk_weights, score: str = "softmax", bias=None, num_groups: int = 1,
                   topk_groups: int = 1, group_best: int = 2, renormalize: bool = False, scale: float = 1.0) -> None:
    """gate_topk into topk_idx and topk_weights [tokens, K] (allocates nothing)."""
    if len(topk_idx.shape) != 2:
        raise ValueError("topk_idx must be [tokens, K]")
    K = topk_idx.shape[1]
    g = _gate(logits, K, score, num_groups, topk_groups, group_best, renormalize, scale)
    a = _Args()
    _run(a, "miep_gate_topk", ctypes.byref(g), a.arg(logits, "logits", logits.dtype), a.opt(bias, "bias", _F32, (g.num_experts,)),
         a.arg(topk_idx, "topk_idx", _I64, (g.num_tokens, K)), a.arg(topk_weights, "topk_weights", _F32, (g.num_tokens, K)))


def gate_topk(logits: torch.Tensor, num_topk: int, score: str = "softmax", bias: Optional[torch.Tensor] = None,
              num_groups: int = 1, topk_groups: int = 1, group_best: int = 2, renormalize: bool = False,
              scale: float = 1.0):
    """The K experts of each token: (topk_idx [tokens, K] int64 in descending order, topk_weights [tokens, K] fp32).

    logits [tokens, experts] float32 or bfloat16.  ``score``: "softmax" over the experts, or "sigmoid" of each.  The
    K largest scores + ``bias`` [experts] are chosen (the bias enters the choice alone), equal ones by the lower
    index, with ``num_groups`` among the experts of the ``topk_groups`` groups whose ``group_best`` (1 or 2) largest
    add up to most (of groups of one expert: whose expert has most).  Weights are the scores, divided by their sum with
    ``renormalize``, times ``scale``.  A logit of -inf or NaN masks an expert, a bias of them leaves it out of the choice
    (a group that has fewer than ``group_best`` left comes last); +inf counts as the type's largest number.  Where fewer
    than K are left the last entries are -1 with weight 0, which every dispatch skips.
    """
    shape = (logits.shape[0], num_topk)
    idx = torch.empty(shape, dtype=_I64, device=logits.device)
    weights = torch.empty(shape, dtype=_F32, device=logits.device)
    gate_topk_into(logits, idx, weights, score, bias, num_groups, topk_groups, group_best, renormalize, scale)
    return idx, weights


def gate_topk_backward_into(d_topk_weights, logits, topk_idx, d_logits, score: str = "softmax",
                            renormalize: bool = False, scale: float = 1.0) -> None:
    """gate_topk_backward into d_logits [tokens, experts], of the logits' type (allocates nothing)."""
    if len(topk_idx.shape) != 2:
        raise ValueError("topk_idx must be [tokens, K]")
    K = topk_idx.shape[1]
    g = _gate(logits, K, score, 1, 1, 1, renormalize, scale)
    a = _Args()
    _run(a, "miep_gate_topk_backward", ctypes.byref(g), a.arg(d_topk_weights, "d_topk_weights", _F32, (g.num_tokens, K)),
         a.arg(logits, "logits", logits.dtype), a.arg(topk_idx, "topk_idx", _I64, (g.num_tokens, K)),
         a.arg(d_logits, "d_logits", logits.dtype, logits.shape))


def gate_topk_backward(d_topk_weights: torch.Tensor, logits: torch.Tensor, topk_idx: torch.Tensor,
                       score: str = "softmax", renormalize: bool = False, scale: float = 1.0) -> torch.Tensor:
    """Gradient of gate_topk's logits from that of its weights (the choice itself has none, nor has the bias)."""
    d_logits = torch.empty_like(logits)
    gate_topk_backward_into(d_topk_weights, logits, topk_idx, d_logits, score, renormalize, scale)
    return d_logits


# --------------------------------------------------------------------------- dense products
def _activation(activation) -> int:
    if activation not in _ACTIVATIONS:
        raise ValueError("activation must be one of %s, got %r" % (list(_ACTIVATIONS)[1:], activation))
    return _ACTIVATIONS[activation]


def _linear_sizes(x, w, act):
    """(rows, N, K, columns of the result)"""
    if len(x.shape) != 2 or len(w.shape) != 2 or x.shape[1] != w.shape[1]:
        raise ValueError("x must be [rows, K] and w [N, K], got %s and %s" % (tuple(x.shape), tuple(w.shape)))
    (rows, K), N = x.shape, w.shape[0]
    if act == 5 and N % 2:
        raise ValueError("SwiGLU needs w [2 * inner, K]")
    return rows, N, K, N // 2 if act == 5 else N


def linear_into(x, w, y, bias=None, activation: Optional[str] = None, residual=None, z=None) -> None:
    """linear into y, bfloat16 or float32, and z [rows, N] bfloat16 when given (allocates nothing)."""
    act = _activation(activation)
    rows, N, K, width = _linear_sizes(x, w, act)
    kind = y.dtype
    if kind != _BF16 and kind != _F32:
        raise TypeError("y must be bfloat16 or float32, got %s" % kind)
    a = _Args()
    _run(a, "miep_linear", a.arg(x, "x", _BF16), rows, a.arg(w, "w", _BF16), N, K, a.opt(bias, "bias", _F32, (N,)), act,
         a.opt(residual, "residual", _BF16, (rows, width)), a.opt(z, "z", _BF16, (rows, N)), a.arg(y, "y", kind, (rows, width)),
         kind == _F32)


def linear(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, activation: Optional[str] = None,
           residual: Optional[torch.Tensor] = None, dtype=torch.bfloat16, save: bool = False):
    """y = f(x @ w.T + bias) + residual in fp32, rounded once to ``dtype`` (bfloat16 or float32).

    x [rows, K], w [N, K] bfloat16, bias [N] float32.  ``activation``: None, "relu", "silu", "gelu", "gelu_tanh", or
    "swiglu": w then is [gate | up] of 2 * inner rows and y [rows, inner] = silu(gate) * up.  residual [rows, N (inner)]
    bfloat16 (linear_into: may be y itself).  With ``save`` returns (y, z), z [rows, N] bfloat16 the values before the
    activation, which linear_backward takes.
    """
    width = _linear_sizes(x, w, _activation(activation))[3]
    y = torch.empty((x.shape[0], width), dtype=dtype, device=x.device)
    z = torch.empty((x.shape[0], w.shape[0]), dtype=_BF16, device=x.device) if save else None
    linear_into(x, w, y, bias, activation, residual, z)
    return (y, z) if save else y


def linear_backward_into(dy, x, w, activation: Optional[str] = None, z=None, dx=None, dw=None, dbias=None, dz=None,
                         workspace=None, accumulate: bool = False) -> None:
    """linear_backward into those of dx [rows, K] bfloat16, dw [N, K] (float32 or bfloat16), dbias [N] float32 and dz
    [rows, N] bfloat16 that are given (allocates nothing).  dz is the gradient before the activation, rounded: dx and dw
    need it where there is an activation, or dy is float32, as both products read it; elsewhere it is a copy of dy that
    costs its writing.  dbias needs a workspace [parts, N] float32 (parts: one for every 16 rows, up to 256, is enough),
    of one call at a time.  ``accumulate`` adds to dw (float32) and dbias."""
    act = _activation(activation)
    rows, N, K, width = _linear_sizes(x, w, act)
    kind = dy.dtype
    if kind != _BF16 and kind != _F32:
        raise TypeError("dy must be bfloat16 or float32, got %s" % kind)
    if act and z is None:
        raise ValueError("the activation's gradient needs z")
    if dw is not None and dw.dtype not in (_F32, _BF16):
        raise TypeError("dw must be float32 or bfloat16, got %s" % dw.dtype)
    if accumulate and dw is not None and dw.dtype != _F32:
        raise TypeError("accumulate needs a float32 dw")
    through = act != 0 or kind == _F32                      # the products read dz, not dy
    products = dx is not None or dw is not None
    if through and products and dz is None:
        raise ValueError("an activation, or a float32 dy, needs dz [%d, %d] bfloat16" % (rows, N))
    parts = 0
    if dbias is not None:
        if workspace is None or workspace.dim() != 2 or workspace.shape[0] < 1:
            raise ValueError("dbias needs a workspace [parts, %d] float32" % N)
        parts = workspace.shape[0]
    a = _Args()                                             # every tensor is looked at before the first launch
    dy_p, x_p, w_p = a.arg(dy, "dy", kind, (rows, width)), a.arg(x, "x", _BF16), a.arg(w, "w", _BF16)
    z_p, dz_p = a.opt(z, "z", _BF16, (rows, N)), a.opt(dz, "dz", _BF16, (rows, N))
    dx_p = a.opt(dx, "dx", _BF16, (rows, K))
    dw_p = None if dw is None else a.arg(dw, "dw", dw.dtype, (N, K))
    db_p, ws_p = a.opt(dbias, "dbias", _F32, (N,)), a.opt(workspace, "workspace", _F32, None if dbias is None else (parts, N))
    if dz is not None or dbias is not None:
        _run(a, "miep_linear_act_backward", dy_p, kind == _F32, z_p, rows, N, act, dz_p, db_p, bool(accumulate), ws_p, parts)
    grad = dz_p if through else dy_p
    if dx is not None:
        _run(a, "miep_linear_dgrad", grad, rows, w_p, N, K, dx_p)
    if dw is not None:
        _run(a, "miep_linear_wgrad", grad, x_p, rows, N, K, dw.dtype == _F32, bool(accumulate), dw_p)


def linear_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, activation: Optional[str] = None,
                    z: Optional[torch.Tensor] = None, bias: bool = False, dtype=torch.float32):
    """Gradients of linear at dy: (dx [rows, K] bfloat16, dw [N, K] in ``dtype``, dbias [N] float32 or None).

    ``z``: what the forward saved, where it had an activation.  The gradient before the activation is rounded to
    bfloat16 for the two products; dbias sums it unrounded.  A residual's gradient is dy itself."""
    rows, N, K, _ = _linear_sizes(x, w, _activation(activation))
    dev = x.device
    through = _activation(activation) != 0 or dy.dtype == _F32
    dx, dw = torch.empty((rows, K), dtype=_BF16, device=dev), torch.empty((N, K), dtype=dtype, device=dev)
    dz = torch.empty((rows, N), dtype=_BF16, device=dev) if through else None
    dbias = torch.empty((N,), dtype=_F32, device=dev) if bias else None
    workspace = torch.empty((max(1, min(256, -(-rows // 16))), N), dtype=_F32, device=dev) if bias else None
    linear_backward_into(dy, x, w, activation, z, dx, dw, dbias, dz, workspace)
    return dx, dw, dbias


# --------------------------------------------------------------------------- a few tokens
def _layer(x, topk_idx, w1, w2, first_expert, ue8m0) -> _lib.LayerC:
    if len(x.shape) != 2 or len(topk_idx.shape) != 2 or len(w1.shape) != 3:
        raise ValueError("x must be [tokens, H], topk_idx [tokens, K], w1 [experts, 2 * inner, H]")
    (N, H), K, (E, wide, h1) = x.shape, topk_idx.shape[1], w1.shape
    if wide % 2 or h1 != H or w2.shape != (E, H, wide // 2):
        raise ValueError("w1 must be [experts, 2 * inner, %d] and w2 [experts, %d, inner], got %s and %s" %
                         (H, H, tuple(w1.shape), tuple(w2.shape)))
    return _lib.LayerC(N, K, E, H, wide // 2, ue8m0, first_expert)


def expert_layer_into(x, topk_idx, topk_weights, w1, w2, y, workspace, first_expert: int = 0, residual=None) -> None:
    """expert_layer into y [tokens, H], with a workspace [tokens * K, inner] bfloat16 of one call at a time (allocates
    nothing)."""
    q = _layer(x, topk_idx, w1, w2, first_expert, 0)
    N, K, H = q.num_tokens, q.num_topk, q.hidden
    a = _Args()
    _run(a, "miep_expert_layer", ctypes.byref(q), a.arg(x, "x", _BF16), a.arg(topk_idx, "topk_idx", _I64, (N, K)),
         a.arg(topk_weights, "topk_weights", _F32, (N, K)), a.arg(w1, "w1", _BF16), a.arg(w2, "w2", _BF16),
         a.opt(residual, "residual", _BF16, (N, H)), a.arg(workspace, "workspace", _BF16, (N * K, q.inner)), a.arg(y, "y", _BF16, (N, H)))


def expert_layer(x: torch.Tensor, topk_idx: torch.Tensor, topk_weights: torch.Tensor, w1: torch.Tensor,
                 w2: torch.Tensor, first_expert: int = 0, residual: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[t] = residual[t] + sum over k of topk_weights[t, k] * w2[e] @ swiglu(w1[e] @ x[t]), e = topk_idx[t, k] -
    first_expert, for the entries whose expert is here; at most 128 tokens (more: dispatch and the grouped products).

    x [tokens, H] bfloat16, topk_idx / topk_weights [tokens, K] (gate_topk's), w1 [experts, 2 * inner, H] = [gate | up],
    w2 [experts, H, inner] bfloat16.  ``first_expert``: the first one that is here (a rank's share); other entries and
    masked ones add nothing.  Each chosen expert's weights are read once.  The activation is rounded to bfloat16."""
    y = torch.empty_like(x)
    workspace = torch.empty((x.shape[0] * topk_idx.shape[1], w1.shape[1] // 2), dtype=_BF16, device=x.device)
    expert_layer_into(x, topk_idx, topk_weights, w1, w2, y, workspace, first_expert, residual)
    return y


def expert_layer_fp8_into(x, topk_idx, topk_weights, w1, w1_scales, w2, w2_scales, y, workspace,
                          first_expert: int = 0, residual=None) -> None:
    """expert_layer_fp8 into y [tokens, H], with a workspace [tokens * K, inner] bfloat16 of one call at a time
    (allocates nothing)."""
    kind = w1_scales.dtype
    for t, name in ((w1, "w1"), (w2, "w2")):
        if t.dtype not in _FP8:
            raise TypeError("%s must be float8_e4m3fn/uint8 codes, got %s" % (name, t.dtype))
    if kind != _F32 and kind != torch.uint8:
        raise TypeError("w1_scales must be float32, or uint8 exponent bytes, got %s" % kind)
    q = _layer(x, topk_idx, w1, w2, first_expert, kind == torch.uint8)
    N, K, E, H, inner = q.num_tokens, q.num_topk, q.num_experts, q.hidden, q.inner
    if H % 128 or inner % 128:
        raise ValueError("E4M3 weights need H % 128 == 0 and inner % 128 == 0")
    a = _Args()
    _run(a, "miep_expert_layer_fp8", ctypes.byref(q), a.arg(x, "x", _BF16), a.arg(topk_idx, "topk_idx", _I64, (N, K)),
         a.arg(topk_weights, "topk_weights", _F32, (N, K)), a.arg(w1, "w1", w1.dtype),
         a.arg(w1_scales, "w1_scales", kind, (E, 2 * inner // 128, H // 128)), a.arg(w2, "w2", w2.dtype),
         a.arg(w2_scales, "w2_scales", kind, (E, H // 128, inner // 128)), a.opt(residual, "residual", _BF16, (N, H)),
         a.arg(workspace, "workspace", _BF16, (N * K, inner)), a.arg(y, "y", _BF16, (N, H)))


def expert_layer_fp8(x: torch.Tensor, topk_idx: torch.Tensor, topk_weights: torch.Tensor, w1: torch.Tensor,
                     w1_scales: torch.Tensor, w2: torch.Tensor, w2_scales: torch.Tensor, first_expert: int = 0,
                     residual: Optional[torch.Tensor] = None) -> torch.Tensor:
    """expert_layer with E4M3 weights, a scale for each 128 x 128 block: w1_scales [experts, 2 * inner / 128, H / 128],
    w2_scales [experts, H / 128, inner / 128], float32, or uint8 exponent bytes of powers of two.  x stays bfloat16:
    codes are multiplied as the bfloat16 numbers that they are."""
    y = torch.empty_like(x)
    workspace = torch.empty((x.shape[0] * topk_idx.shape[1], w1.shape[1] // 2), dtype=_BF16, device=x.device)
    expert_layer_fp8_into(x, topk_idx, topk_weights, w1, w1_scales, w2, w2_scales, y, workspace, first_expert, residual)
    return y
