"""CPU checks of the expert operators' argument validation, through the C ABI
and the Python binding.  No call here reaches a kernel launch."""
import ctypes

import pytest
import torch

import combine_get_dispatch_histogram_amd as miep
from combine_get_dispatch_histogram_amd import _lib

EINVAL, EUNSUPPORTED = _lib.MIEP_EINVAL, _lib.MIEP_EUNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(_lib.LIB_PATH):
        from combine_get_dispatch_histogram_amd import build
        build.build()
    return _lib.load()


def grp(**kw):
    d = dict(begin=16, rows=16, num_rows=100, num_groups=4, stride=0)
    d.update(kw)
    return _lib.RowGroupsC(**d)


BAD_GROUPS = [(dict(rows=None), EINVAL), (dict(num_rows=-1), EINVAL), (dict(num_rows=2 ** 31), EINVAL),
              (dict(num_groups=-1), EINVAL), (dict(num_groups=8193), EUNSUPPORTED), (dict(begin=None), EINVAL),
              (dict(begin=None, stride=-4), EINVAL)]


@pytest.mark.parametrize("kw,status", BAD_GROUPS)
def test_groups_are_checked_by_every_call(lib, kw, status):
    g = ctypes.byref(grp(**kw))
    rows = kw.get("num_rows", 100)
    calls = [lib.miep_grouped_gemm(g, 16, rows, 16, 64, 64, None, 0, 16, None),
             lib.miep_grouped_gemm_dgrad(g, 16, 16, 64, 64, 0, 16, None),
             lib.miep_grouped_gemm_wgrad(g, 16, 16, rows, None, 64, 64, 1, 0, 16, None),
             lib.miep_grouped_gemm_fp8(g, 16, 16, rows, 16, 16, 0, 64, 128, None, 0, 16, None),
             lib.miep_swiglu(g, 16, 64, 16, None), lib.miep_swiglu_fp8(g, 16, 128, 0, 16, 16, None, None),
             lib.miep_swiglu_backward(g, 16, 16, 64, 16, None)]
    assert calls == [status] * len(calls), lib.miep_last_error()
    assert lib.miep_last_error()


def test_null_groups(lib):
    assert lib.miep_grouped_gemm(None, 16, 1, 16, 64, 64, None, 0, 16, None) == EINVAL
    assert lib.miep_swiglu(None, 16, 64, 16, None) == EINVAL


@pytest.mark.parametrize("n,k,status", [(0, 64, EINVAL), (64, -8, EINVAL), (60, 64, EUNSUPPORTED), (64, 12, EUNSUPPORTED),
                                        ((1 << 21) + 8, 64, EUNSUPPORTED), (64, 1 << 22, EUNSUPPORTED)])
def test_product_sizes(lib, n, k, status):
    g = ctypes.byref(grp())
    assert lib.miep_grouped_gemm(g, 16, 100, 16, n, k, None, 0, 16, None) == status
    assert lib.miep_grouped_gemm_dgrad(g, 16, 16, n, k, 0, 16, None) == status
    assert lib.miep_grouped_gemm_wgrad(g, 16, 16, 100, None, n, k, 1, 0, 16, None) == status


def test_product_arguments(lib):
    g = ctypes.byref(grp())

    def gemm(x=16, rows=100, w=16, idx=None, exp=0, y=16):
        return lib.miep_grouped_gemm(g, x, rows, w, 64, 64, idx, exp, y, None)

    assert gemm(x=None) == EINVAL and gemm(w=None) == EINVAL and gemm(y=None) == EINVAL
    assert gemm(x=24) == EUNSUPPORTED and gemm(w=8) == EUNSUPPORTED and gemm(y=18) == EUNSUPPORTED
    assert gemm(rows=99) == EINVAL and b"row_index" in lib.miep_last_error()      # rows of another layout
    assert gemm(rows=-1, idx=16) == EINVAL and gemm(exp=-1) == EINVAL
    assert gemm(rows=(64 << 30) // 128 + 1, idx=16) == EUNSUPPORTED and b"64 GiB" in lib.miep_last_error()

    def wgrad(dw=16, f32=1, acc=0, dy=16):
        return lib.miep_grouped_gemm_wgrad(g, dy, 16, 100, None, 64, 64, f32, acc, dw, None)

    assert wgrad(dw=None) == EINVAL and wgrad(dw=8) == EUNSUPPORTED and wgrad(dy=None) == EINVAL
    assert wgrad(f32=0, acc=1) == EINVAL

    def fp8(xs=16, ws=16, k=128, x=16):
        return lib.miep_grouped_gemm_fp8(g, x, xs, 100, 16, ws, 0, 64, k, None, 0, 16, None)

    assert fp8(xs=None) == EINVAL and fp8(ws=None) == EINVAL and fp8(k=64) == EINVAL and fp8(x=20) == EUNSUPPORTED
    # tiles are counted in 32 bits
    big = ctypes.byref(grp(num_rows=2 ** 31 - 1))
    assert lib.miep_grouped_gemm(big, 16, 2 ** 31 - 1, 16, 1 << 20, 64, None, 0, 16, None) == EUNSUPPORTED
    wide = ctypes.byref(grp(num_groups=8192))
    assert lib.miep_grouped_gemm_wgrad(wide, 16, 16, 100, None, 1 << 20, 1 << 20, 1, 0, 16, None) == EUNSUPPORTED


def test_swiglu_arguments(lib):
    g = ctypes.byref(grp())
    assert lib.miep_swiglu(g, 16, 0, 16, None) == EINVAL
    assert lib.miep_swiglu(g, 16, 12, 16, None) == EUNSUPPORTED
    assert lib.miep_swiglu(g, None, 64, 16, None) == EINVAL
    assert lib.miep_swiglu(g, 16, 64, 8, None) == EUNSUPPORTED
    assert lib.miep_swiglu_fp8(g, 16, 64, 0, 16, 16, None, None) == EINVAL         # whole 128-channel groups
    assert lib.miep_swiglu_fp8(g, 16, 128, 0, 16, None, None, None) == EINVAL
    assert lib.miep_swiglu_fp8(g, 16, 128, 0, 16, 16, 16, None) == EINVAL          # exponent bytes need powers of two
    assert lib.miep_swiglu_backward(g, None, 16, 64, 16, None) == EINVAL


def test_expert_order_arguments(lib):
    def order(topk=16, off=16, rows=100, K=8, E=32, R=4, align=1, ws=16, parts=1, begin=16, cnt=16, sr=16, slots=800,
              rs=16):
        return lib.miep_expert_order(topk, off, rows, K, E, R, align, ws, parts, begin, cnt, sr, slots, rs, None, None)

    for kw in (dict(topk=None), dict(off=None), dict(ws=None), dict(begin=None), dict(cnt=None), dict(sr=None),
               dict(rs=None), dict(rows=-1), dict(slots=-1), dict(K=0), dict(E=0), dict(R=0), dict(align=0),
               dict(parts=0), dict(E=33), dict(rows=2 ** 31)):
        assert order(**kw) == EINVAL, kw
    for kw in (dict(K=65), dict(R=512, E=512), dict(E=16384, R=8), dict(E=4096, R=1), dict(rows=2 ** 28, slots=1),
               dict(align=2 ** 27)):
        assert order(**kw) == EUNSUPPORTED, kw


def test_expert_reduce_arguments(lib):
    def red(z=16, slots=10, H=64, rs=16, rows=5, K=2, y=16):
        return lib.miep_expert_reduce(z, slots, H, rs, rows, K, None, None, y, None)

    for kw in (dict(z=None), dict(rs=None), dict(y=None), dict(H=0), dict(K=0), dict(rows=-1), dict(slots=2 ** 31)):
        assert red(**kw) == EINVAL, kw
    for kw in (dict(H=12), dict(K=65), dict(z=8), dict(y=24 + 4), dict(H=(1 << 24) + 8)):
        assert red(**kw) == EUNSUPPORTED, kw

    def back(dy=16, z=16, dz=16, dw=16):
        return lib.miep_expert_reduce_backward(dy, z, 10, 64, 16, 5, 2, None, None, dz, dw, None)

    assert back(dy=None) == EINVAL and back(dz=None) == EINVAL and back(z=None) == EINVAL
    assert back(dy=8) == EUNSUPPORTED


# ------------------------------------------------------------------ binding
BF = torch.bfloat16


def test_binding_refuses_shapes_types_and_hosts():
    g = miep.RowGroups(rows=torch.zeros(2, dtype=torch.int32), begin=torch.zeros(2, dtype=torch.int32))
    x, w, y = torch.zeros((4, 64), dtype=BF), torch.zeros((2, 16, 64), dtype=BF), torch.zeros((4, 16), dtype=BF)
    with pytest.raises(ValueError, match="device tensors"):
        miep.grouped_gemm_into(x, w, g, y)
    with pytest.raises(TypeError):
        miep.grouped_gemm_into(x.float(), w, g, y)
    with pytest.raises(TypeError):
        miep.grouped_gemm_into(x, w, g, y.half())
    with pytest.raises(ValueError):
        miep.grouped_gemm_into(x, w[:1], g, y)                       # weights of another number of groups
    with pytest.raises(ValueError):
        miep.grouped_gemm_into(x[:, :32], w, g, y)
    with pytest.raises(ValueError):
        miep.grouped_gemm_into(x[:3], w, g, y)                       # rows of another layout
    with pytest.raises(TypeError):
        miep.grouped_gemm_into(x, w, g, y, row_index=torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        miep.grouped_gemm_into(x, w, g, y, row_index=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        miep.grouped_gemm_dgrad_into(y, w, g, x[:, :32])
    with pytest.raises(TypeError):
        miep.grouped_gemm_wgrad_into(y, x, g, w, accumulate=True)    # accumulate needs fp32
    with pytest.raises(TypeError):
        miep.grouped_gemm_wgrad_into(y, x, g, w.half())
    q, s = torch.zeros((4, 128), dtype=torch.uint8), torch.zeros((4, 1))
    wq, ws = torch.zeros((2, 16, 128), dtype=torch.uint8), torch.zeros((2, 1, 1))
    with pytest.raises(TypeError):
        miep.grouped_gemm_fp8_into(q, s.to(torch.uint8), wq, ws, g, y)   # both scales of one type
    with pytest.raises(TypeError):
        miep.grouped_gemm_fp8_into(q, s.half(), wq, ws, g, y)
    with pytest.raises(TypeError):
        miep.grouped_gemm_fp8_into(x, s, wq, ws, g, y)
    with pytest.raises(ValueError):
        miep.grouped_gemm_fp8_into(q, s[:3], wq, ws, g, y)
    h = torch.zeros((4, 256), dtype=BF)
    with pytest.raises(ValueError):
        miep.swiglu_into(h, g, torch.zeros((4, 64), dtype=BF))
    with pytest.raises(ValueError):
        miep.swiglu_fp8_into(h[:, :128], g, q[:, :64], s[:, :0])
    with pytest.raises(ValueError):
        miep.swiglu_fp8_into(h, g, q, s, a_scales_ue8m0=s.to(torch.uint8))
    with pytest.raises(ValueError):
        miep.swiglu_fp8(h, g, use_ue8m0=True)
    with pytest.raises(ValueError):
        miep.swiglu_backward_into(x, h, g, h)


def test_binding_refuses_orders():
    off, topk = torch.zeros(3, dtype=torch.int32), torch.zeros((5, 2), dtype=torch.int64)
    with pytest.raises(ValueError):
        miep.ExpertOrder.allocate(topk, off, 7)                      # experts do not split over the ranks
    order = miep.ExpertOrder.allocate(topk, off, 8, 4)
    assert order.num_slots == 10 + 24 and order.workspace.shape == (128, 8)
    with pytest.raises(TypeError):
        miep.expert_order_into(topk.int(), order)
    with pytest.raises(ValueError):
        miep.expert_order_into(topk[:4], order)
    order.workspace = None
    with pytest.raises(ValueError, match="workspace"):
        miep.expert_order_into(topk, order)
    z, y = torch.zeros((34, 16), dtype=BF), torch.zeros((5, 16), dtype=BF)
    with pytest.raises(ValueError):
        miep.expert_reduce_into(z[:3], order, y)
    with pytest.raises(ValueError):
        miep.expert_reduce_into(z, order, y, torch.zeros((5, 3)))
    with pytest.raises(ValueError):
        miep.expert_reduce_backward_into(y, None, order, z, d_topk_weights=torch.zeros((5, 2)))
