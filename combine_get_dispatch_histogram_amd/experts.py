"""What the experts compute between dispatch and combine (``include/miep.h``, "experts").

  expert_order(recv_topk_idx, recv_rank_offset, num_experts) -> ExpertOrder   received rows -> slots in expert order
  grouped_gemm(x, w, groups, row_index)                     bf16 rows times their expert's weights
  grouped_gemm_dgrad / grouped_gemm_wgrad                   its gradients
  grouped_gemm_fp8(x, x_scales, w, w_scales, groups)        the same on E4M3 codes with a scale per 128 (x 128)
  swiglu / swiglu_fp8 / swiglu_backward                     the activation between an expert's two products
  expert_reduce / expert_reduce_backward                    slots -> received rows, gate-weighted

As everywhere in this package the ``*_into`` variants take preallocated outputs
and allocate nothing; rows of an output that lie in no group are left as they
were, so the allocating variants return uninitialised memory there.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib
from ._call import _Args, _run, check_status

_FP8 = (torch.float8_e4m3fn, torch.uint8)
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


@dataclass
class RowGroups:
    """The rows of a layout that belong to each expert: group g holds rows
    begin[g] .. begin[g] + rows[g] - 1, or with ``begin`` None the first
    rows[g] of the block of ``stride`` rows from g * stride (the packed layout
    of the low-latency dispatch).  Device int32, read when the kernels run."""
    rows: torch.Tensor
    begin: Optional[torch.Tensor] = None
    stride: int = 0

    @staticmethod
    def low_latency(recv: dict) -> "RowGroups":
        """The groups of ``low_latency_dispatch``'s packed_recv_x, one per local expert."""
        return RowGroups(rows=recv["packed_recv_count"], stride=recv["packed_recv_x"].shape[1])

    def c(self, a, num_rows: int) -> _lib.RowGroupsC:
        rows, begin = self.rows, self.begin
        shape = rows.shape
        if len(shape) != 1:
            raise ValueError("groups.rows must be [num_groups]")
        first = None if begin is None else a.arg(begin, "groups.begin", _I32, shape)
        return _lib.RowGroupsC(first, a.arg(rows, "groups.rows", _I32), num_rows, shape[0], int(self.stride))


@dataclass
class ExpertOrder:
    """Received rows in expert order: group_begin / group_rows [E] (first slot
    and slots of each global expert), slot_row [slots] (received row of each
    slot, -1 where there is none), row_slot [cap, K] (slot of each top-k entry,
    or -1), the dispatch's recv_rank_offset [R+1] and the workspace [parts, E]."""
    group_begin: torch.Tensor
    group_rows: torch.Tensor
    slot_row: torch.Tensor
    row_slot: torch.Tensor
    recv_rank_offset: torch.Tensor
    workspace: Optional[torch.Tensor] = None

    @property
    def groups(self) -> RowGroups:
        return RowGroups(rows=self.group_rows, begin=self.group_begin)

    @property
    def num_slots(self) -> int:
        return self.slot_row.numel()

    @staticmethod
    def allocate(recv_topk_idx: torch.Tensor, recv_rank_offset: torch.Tensor, num_experts: int,
                 expert_alignment: int = 1, num_slots: int = 0) -> "ExpertOrder":
        """Arrays for the order of recv_topk_idx; ``num_slots`` 0 takes the worst case (never overflows)."""
        cap, K = recv_topk_idx.shape
        R = recv_rank_offset.numel() - 1
        if R <= 0 or num_experts <= 0 or num_experts % R:
            raise ValueError("%d experts do not split over %d ranks" % (num_experts, R))
        if num_slots <= 0:
            num_slots = cap * K + (expert_alignment - 1) * num_experts
        i32 = dict(dtype=torch.int32, device=recv_topk_idx.device)
        return ExpertOrder(torch.empty((num_experts,), **i32), torch.empty((num_experts,), **i32),
                           torch.empty((num_slots,), **i32), torch.empty((cap, K), **i32), recv_rank_offset,
                           torch.empty((max(1, 256 // R), num_experts), **i32))


def _flat(t: torch.Tensor, name: str) -> torch.Tensor:
    """[rows, width], or [blocks, rows, width] seen as its rows."""
    if t.dim() == 2:
        return t
    if t.dim() == 3 and t.is_contiguous():
        return t.view(t.shape[0] * t.shape[1], t.shape[2])
    raise ValueError("%s must be [rows, width] or contiguous [groups, rows, width]" % name)


# --------------------------------------------------------------------------- expert order
def expert_order_into(recv_topk_idx, order: ExpertOrder, expert_alignment: int = 1, status=None) -> None:
    """expert_order into preallocated arrays (allocates nothing).  ``status`` ([1] int32, optional) receives 0 or
    MIEP_ECAPACITY where the experts need more than the slots given (read it with ``check_status``)."""
    if recv_topk_idx.dim() != 2:
        raise ValueError("recv_topk_idx must be [cap, K]")
    cap, K = recv_topk_idx.shape
    slots, workspace = order.num_slots, order.workspace
    parts = workspace.shape[0] if workspace is not None and workspace.dim() == 2 else 0
    E, R = order.group_begin.numel(), order.recv_rank_offset.numel() - 1
    if parts < 1:
        raise ValueError("expert_order needs a workspace [parts, %d] int32" % E)
    a = _Args()
    _run(a, "miep_expert_order", a.arg(recv_topk_idx, "recv_topk_idx", torch.int64),
         a.arg(order.recv_rank_offset, "recv_rank_offset", _I32, (R + 1,)), cap, K, E, R, int(expert_alignment),
         a.arg(workspace, "workspace", _I32, (parts, E)), parts, a.arg(order.group_begin, "group_begin", _I32, (E,)),
         a.arg(order.group_rows, "group_rows", _I32, (E,)), a.arg(order.slot_row, "slot_row", _I32, (slots,)), slots,
         a.arg(order.row_slot, "row_slot", _I32, (cap, K)), a.opt(status, "status", _I32, (1,)))


def expert_order(recv_topk_idx: torch.Tensor, recv_rank_offset: torch.Tensor, num_experts: int,
                 expert_alignment: int = 1, num_slots: int = 0, check_capacity: bool = True) -> ExpertOrder:
    """Slots in expert order for the rows of a normal dispatch.

    recv_topk_idx [cap, K] int64 and the handle's recv_rank_offset [R+1].  Slots are expert-major over the global
    experts, each expert's from a multiple of ``expert_alignment`` on, in (row, k) order inside an expert.
    ``order.slot_row`` is the row_index of the products, ``order.groups`` their groups.  The slots' number, and
    with it the size of everything in slot order, is the worst case cap * K + (expert_alignment - 1) * E, or
    ``num_slots`` (dispatch's num_recv_tokens_per_expert.sum() is exact); then, with ``check_capacity``, the device
    status word is read back (synchronously) and an overflow raises MiepError(MIEP_ECAPACITY).
    """
    order = ExpertOrder.allocate(recv_topk_idx, recv_rank_offset, num_experts, expert_alignment, num_slots)
    status = torch.empty((1,), dtype=torch.int32, device=recv_topk_idx.device) if num_slots > 0 else None
    expert_order_into(recv_topk_idx, order, expert_alignment, status)
    if status is not None and check_capacity:
        check_status(status)
    return order


def _reduce_args(a: _Args, order: ExpertOrder, topk_weights):
    """row_slot, cap, K, where the received rows' number is (recv_rank_offset's last entry), topk_weights."""
    cap, K = order.row_slot.shape
    off = order.recv_rank_offset
    if off.dim() != 1 or off.numel() < 2:
        raise ValueError("recv_rank_offset must be [R + 1]")
    return (a.arg(order.row_slot, "row_slot", _I32), cap, K,
            a.arg(off, "recv_rank_offset", _I32) + 4 * (off.numel() - 1),
            a.opt(topk_weights, "topk_weights", _F32, (cap, K)))


def expert_reduce_into(z, order: ExpertOrder, y, topk_weights=None) -> None:
    """expert_reduce into y [cap, H] (allocates nothing); rows behind the last received one are left as they were."""
    a = _Args()
    if z.dim() != 2 or z.shape[0] != order.num_slots:
        raise ValueError("z must be [%d, H]" % order.num_slots)
    slots, H = z.shape
    row_slot, cap, K, total, weights = _reduce_args(a, order, topk_weights)
    _run(a, "miep_expert_reduce", a.arg(z, "z", _BF16), slots, H, row_slot, cap, K, total, weights,
         a.arg(y, "y", _BF16, (cap, H)))


def expert_reduce(z: torch.Tensor, order: ExpertOrder, topk_weights: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Expert outputs z [slots, H] bf16 back to received rows [cap, H]: each row sums its entries' slots in
    ascending k in fp32, each times its gate weight (``topk_weights`` [cap, K], the received ones) when given."""
    y = torch.empty((order.row_slot.shape[0], z.shape[1]), dtype=torch.bfloat16, device=z.device)
    expert_reduce_into(z, order, y, topk_weights)
    return y


def expert_reduce_backward_into(dy, z, order: ExpertOrder, dz, topk_weights=None, d_topk_weights=None) -> None:
    """Gradients of expert_reduce (allocates nothing): dz [slots, H], and d_topk_weights [cap, K] fp32 when given
    (then z is needed).  Slots that no entry names and rows behind the last received one are left as they were."""
    a = _Args()
    row_slot, cap, K, total, weights = _reduce_args(a, order, topk_weights)
    if dy.dim() != 2 or dy.shape[0] != cap:
        raise ValueError("dy must be [%d, H]" % cap)
    H, slots = dy.shape[1], order.num_slots
    if d_topk_weights is not None and z is None:
        raise ValueError("d_topk_weights needs z")
    _run(a, "miep_expert_reduce_backward", a.arg(dy, "dy", _BF16), a.opt(z, "z", _BF16, (slots, H)), slots, H, row_slot,
         cap, K, total, weights, a.arg(dz, "dz", _BF16, (slots, H)),
         a.opt(d_topk_weights, "d_topk_weights", _F32, (cap, K)))


def expert_reduce_backward(dy: torch.Tensor, z: torch.Tensor, order: ExpertOrder,
                           topk_weights: Optional[torch.Tensor] = None):
    """Gradients of expert_reduce at dy [cap, H]: (dz [slots, H] bf16, d_topk_weights [cap, K] fp32 or None
    without weights)."""
    dz = torch.empty((order.num_slots, dy.shape[1]), dtype=torch.bfloat16, device=dy.device)
    dw = torch.empty_like(topk_weights) if topk_weights is not None else None
    expert_reduce_backward_into(dy, z, order, dz, topk_weights, dw)
    return dz, dw


# --------------------------------------------------------------------------- grouped products
def _check_product(x, w, groups: RowGroups, rows: int, row_index, wide: str):
    """(rows of x, N, K) of a product over x's channels, w's N or K."""
    shape, (x_rows, channels) = w.shape, x.shape
    if len(shape) != 3 or shape[0] != groups.rows.numel():
        raise ValueError("w must be [%d, N, K]" % groups.rows.numel())
    _, N, K = shape
    if channels != (K if wide == "K" else N):
        raise ValueError("rows of %d channels do not match w %s" % (channels, tuple(shape)))
    if row_index is None and x_rows != rows:
        raise ValueError("x has %d rows, the output %d (and there is no row_index)" % (x_rows, rows))
    return x_rows, N, K


def grouped_gemm_into(x, w, groups: RowGroups, y, row_index=None, expected_rows: int = 0) -> None:
    """grouped_gemm into y (allocates nothing)."""
    x, y = _flat(x, "x"), _flat(y, "y")
    rows = y.shape[0]
    x_rows, N, K = _check_product(x, w, groups, rows, row_index, "K")
    a = _Args()
    g = groups.c(a, rows)
    _run(a, "miep_grouped_gemm", ctypes.byref(g), a.arg(x, "x", _BF16), x_rows, a.arg(w, "w", _BF16), N, K,
         a.opt(row_index, "row_index", _I32, (rows,)), int(expected_rows), a.arg(y, "y", _BF16, (rows, N)))


def grouped_gemm(x: torch.Tensor, w: torch.Tensor, groups: RowGroups, row_index: Optional[torch.Tensor] = None,
                 expected_rows: int = 0) -> torch.Tensor:
    """y[i] = x[src(i)] @ w[g].T for the rows i of every group g, in bf16 with fp32 sums.

    x [rows, K] (or [G, block, K]), w [G, N, K].  ``row_index`` [slots] int32 gathers: src(i) = row_index[i] (a
    negative one gives a zero row) and y has one row per entry; without it src(i) = i.  ``expected_rows`` is the
    rows a group is expected to hold (default: the layout's rows / G); it only chooses the tile size, so give it
    where the layout is mostly empty, as the low-latency one is and an order's of worst-case slots.
    """
    lead = x.shape[:-1] if row_index is None else tuple(row_index.shape)
    y = torch.empty((*lead, w.shape[1]), dtype=torch.bfloat16, device=x.device)
    grouped_gemm_into(x, w, groups, y, row_index, expected_rows)
    return y


def grouped_gemm_dgrad_into(dy, w, groups: RowGroups, dx, expected_rows: int = 0) -> None:
    """grouped_gemm_dgrad into dx (allocates nothing)."""
    dy, dx = _flat(dy, "dy"), _flat(dx, "dx")
    rows = dx.shape[0]
    _, N, K = _check_product(dy, w, groups, rows, None, "N")
    a = _Args()
    g = groups.c(a, rows)
    _run(a, "miep_grouped_gemm_dgrad", ctypes.byref(g), a.arg(dy, "dy", _BF16), a.arg(w, "w", _BF16), N, K,
         int(expected_rows), a.arg(dx, "dx", _BF16, (rows, K)))


def grouped_gemm_dgrad(dy: torch.Tensor, w: torch.Tensor, groups: RowGroups, expected_rows: int = 0) -> torch.Tensor:
    """Gradient of grouped_gemm's rows, in layout rows: dx[i] = dy[i] @ w[g].  Where the forward gathered,
    ``expert_reduce`` without weights adds the slots' gradients up to the received rows'."""
    dx = torch.empty((*dy.shape[:-1], w.shape[2]), dtype=torch.bfloat16, device=dy.device)
    grouped_gemm_dgrad_into(dy, w, groups, dx, expected_rows)
    return dx


def grouped_gemm_wgrad_into(dy, x, groups: RowGroups, dw, row_index=None, accumulate: bool = False) -> None:
    """grouped_gemm_wgrad into dw [G, N, K], fp32 or bf16 (allocates nothing); ``accumulate`` (fp32) adds to it."""
    dy, x = _flat(dy, "dy"), _flat(x, "x")
    if dw.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("dw must be float32 or bfloat16, got %s" % dw.dtype)
    if accumulate and dw.dtype != torch.float32:
        raise TypeError("accumulate needs a float32 dw")
    rows = dy.shape[0]
    x_rows, N, K = _check_product(x, dw, groups, rows, row_index, "K")
    a = _Args()
    g = groups.c(a, rows)
    _run(a, "miep_grouped_gemm_wgrad", ctypes.byref(g), a.arg(dy, "dy", _BF16, (rows, N)), a.arg(x, "x", _BF16), x_rows,
         a.opt(row_index, "row_index", _I32, (rows,)), N, K, int(dw.dtype == _F32), int(bool(accumulate)),
         a.arg(dw, "dw", dw.dtype))


def grouped_gemm_wgrad(dy: torch.Tensor, x: torch.Tensor, groups: RowGroups, row_index: Optional[torch.Tensor] = None,
                       dtype=torch.float32) -> torch.Tensor:
    """Gradient of grouped_gemm's weights: dw[g] = dy[rows of g].T @ x[src(rows of g)], fp32 sums, in ``dtype``
    (float32 or bfloat16).  An empty group's gradient is zero."""
    dw = torch.empty((groups.rows.numel(), dy.shape[-1], x.shape[-1]), dtype=dtype, device=dy.device)
    grouped_gemm_wgrad_into(dy, x, groups, dw, row_index)
    return dw


def grouped_gemm_fp8_into(x, x_scales, w, w_scales, groups: RowGroups, y, row_index=None,
                          expected_rows: int = 0) -> None:
    """grouped_gemm_fp8 into y (allocates nothing)."""
    x, x_scales, y = _flat(x, "x"), _flat(x_scales, "x_scales"), _flat(y, "y")
    kind = x_scales.dtype
    for t, name in ((x, "x"), (w, "w")):
        if t.dtype not in _FP8:
            raise TypeError("%s must be float8_e4m3fn/uint8 codes, got %s" % (name, t.dtype))
    if kind != _F32 and kind != torch.uint8:
        raise TypeError("x_scales must be float32, or uint8 exponent bytes, got %s" % kind)
    rows = y.shape[0]
    x_rows, N, K = _check_product(x, w, groups, rows, row_index, "K")
    if K % 128:
        raise ValueError("FP8 products need K % 128 == 0")
    a = _Args()
    g = groups.c(a, rows)
    _run(a, "miep_grouped_gemm_fp8", ctypes.byref(g), a.arg(x, "x", x.dtype),
         a.arg(x_scales, "x_scales", kind, (x_rows, K // 128)), x_rows, a.arg(w, "w", w.dtype),
         a.arg(w_scales, "w_scales", kind, (w.shape[0], -(-N // 128), K // 128)), int(kind == torch.uint8), N, K,
         a.opt(row_index, "row_index", _I32, (rows,)), int(expected_rows), a.arg(y, "y", _BF16, (rows, N)))


def grouped_gemm_fp8(x: torch.Tensor, x_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
                     groups: RowGroups, row_index: Optional[torch.Tensor] = None,
                     expected_rows: int = 0) -> torch.Tensor:
    """grouped_gemm on E4M3 codes, to bf16.

    x [rows, K] with x_scales [rows, K/128], as an FP8 dispatch receives them (or [G, block, ...], packed by the
    low-latency dispatch); w [G, N, K] with w_scales [G, ceil(N/128), K/128], one per 128 x 128 block.  Both scales
    are float32, or both uint8: the exponent bytes of power-of-two scales (``use_ue8m0``).  Sums are fp32 but for the
    matrix instruction's cut: each 8 consecutive channels' products are held to 13 bits below the largest one's exponent.
    """
    lead = x.shape[:-1] if row_index is None else tuple(row_index.shape)
    y = torch.empty((*lead, w.shape[1]), dtype=torch.bfloat16, device=x.device)
    grouped_gemm_fp8_into(x, x_scales, w, w_scales, groups, y, row_index, expected_rows)
    return y


# --------------------------------------------------------------------------- activation
def _check_h(h):
    h = _flat(h, "h")
    rows, width = h.shape
    if width % 2:
        raise ValueError("h must be [rows, 2 * inner]")
    return h, rows, width // 2


def swiglu_into(h, groups: RowGroups, a_out) -> None:
    """swiglu into a_out [rows, inner] bf16 (allocates nothing)."""
    h, rows, inner = _check_h(h)
    out = _flat(a_out, "a")
    a = _Args()
    g = groups.c(a, rows)
    _run(a, "miep_swiglu", ctypes.byref(g), a.arg(h, "h", _BF16), inner, a.arg(out, "a", _BF16, (rows, inner)))


def swiglu(h: torch.Tensor, groups: RowGroups) -> torch.Tensor:
    """silu(gate) * up over the groups' rows of h [rows, 2 * inner] = [gate | up], to bf16."""
    out = torch.empty((*h.shape[:-1], h.shape[-1] // 2), dtype=torch.bfloat16, device=h.device)
    swiglu_into(h, groups, out)
    return out


def swiglu_fp8_into(h, groups: RowGroups, a_out, a_scales, round_scale: bool = False, a_scales_ue8m0=None) -> None:
    """swiglu_fp8 into E4M3 codes a_out [rows, inner], a_scales [rows, inner/128] fp32 and, when given (with
    round_scale), the scales' exponent bytes (allocates nothing)."""
    h, rows, inner = _check_h(h)
    if inner % 128:
        raise ValueError("the FP8 cast needs inner % 128 == 0")
    out, scales = _flat(a_out, "a"), _flat(a_scales, "a_scales")
    if out.dtype not in _FP8 or out.shape != (rows, inner):
        raise TypeError("a must be [%d, %d] E4M3 codes" % (rows, inner))
    ue = _flat(a_scales_ue8m0, "a_scales_ue8m0") if a_scales_ue8m0 is not None else None
    if ue is not None and not round_scale:
        raise ValueError("a_scales_ue8m0 needs round_scale=True")
    a = _Args()
    g = groups.c(a, rows)
    blocks = (rows, inner // 128)
    _run(a, "miep_swiglu_fp8", ctypes.byref(g), a.arg(h, "h", _BF16), inner, int(bool(round_scale)),
         a.arg(out, "a", out.dtype), a.arg(scales, "a_scales", _F32, blocks),
         a.opt(ue, "a_scales_ue8m0", torch.uint8, blocks))


def swiglu_fp8(h: torch.Tensor, groups: RowGroups, round_scale: bool = False, use_ue8m0: bool = False):
    """swiglu cast per 128 channels to E4M3 by the FP8 dispatch's rule, straight from the fp32 value.  Returns
    (codes [rows, inner], scales [rows, inner/128] fp32), plus the exponent bytes with ``use_ue8m0`` (needs
    round_scale)."""
    if use_ue8m0 and not round_scale:
        raise ValueError("use_ue8m0 needs round_scale=True")
    lead, inner = tuple(h.shape[:-1]), h.shape[-1] // 2
    out = torch.empty((*lead, inner), dtype=torch.float8_e4m3fn, device=h.device)
    scales = torch.empty((*lead, inner // 128), dtype=torch.float32, device=h.device)
    ue = torch.empty((*lead, inner // 128), dtype=torch.uint8, device=h.device) if use_ue8m0 else None
    swiglu_fp8_into(h, groups, out, scales, round_scale, ue)
    return (out, scales, ue) if use_ue8m0 else (out, scales)


def swiglu_backward_into(da, h, groups: RowGroups, dh) -> None:
    """swiglu_backward into dh [rows, 2 * inner], which may be h itself (allocates nothing)."""
    h, rows, inner = _check_h(h)
    da, out = _flat(da, "da"), _flat(dh, "dh")
    a = _Args()
    g = groups.c(a, rows)
    _run(a, "miep_swiglu_backward", ctypes.byref(g), a.arg(da, "da", _BF16, (rows, inner)), a.arg(h, "h", _BF16), inner,
         a.arg(out, "dh", _BF16, (rows, 2 * inner)))


def swiglu_backward(da: torch.Tensor, h: torch.Tensor, groups: RowGroups) -> torch.Tensor:
    """Gradient of swiglu's input h [rows, 2 * inner] from that of its output, da [rows, inner]."""
    dh = torch.empty_like(h)
    swiglu_backward_into(da, h, groups, dh)
    return dh
