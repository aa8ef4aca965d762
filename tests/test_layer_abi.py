"""CPU checks of the block's argument validation (router, dense products, expert layer), through the C ABI and the
Python binding.  No call here reaches a kernel launch."""
import ctypes

import pytest
import torch

import combine_get_dispatch_histogram_amd as miep
from combine_get_dispatch_histogram_amd import _lib

EINVAL, EUNSUPPORTED, OK = _lib.MIEP_EINVAL, _lib.MIEP_EUNSUPPORTED, _lib.MIEP_OK


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(_lib.LIB_PATH):
        from combine_get_dispatch_histogram_amd import build
        build.build()
    return _lib.load()


def gate(**kw):
    d = dict(num_tokens=10, num_experts=64, num_topk=8, sigmoid=0, renormalize=0, num_groups=1, topk_groups=1, group_best=2,
             logits_f32=1, scale=1.0)
    d.update(kw)
    return ctypes.byref(_lib.GateC(**d))


@pytest.mark.parametrize("kw,status", [
    (dict(num_tokens=-1), EINVAL), (dict(num_experts=0), EINVAL), (dict(num_topk=0), EINVAL), (dict(num_topk=65), EINVAL),
    (dict(num_groups=0), EINVAL), (dict(num_groups=3), EINVAL), (dict(topk_groups=0), EINVAL),
    (dict(num_groups=4, topk_groups=5), EINVAL), (dict(group_best=0), EINVAL), (dict(group_best=3), EINVAL),
    (dict(num_experts=2049), EUNSUPPORTED), (dict(num_experts=128, num_topk=65), EUNSUPPORTED),
    (dict(num_experts=128, num_groups=128), EUNSUPPORTED), (dict(num_tokens=2 ** 31), EUNSUPPORTED)])
def test_gate_sizes(lib, kw, status):
    assert lib.miep_gate_topk(gate(**kw), 16, None, 16, 16, None) == status
    assert lib.miep_gate_topk_backward(gate(**kw), 16, 16, 16, 16, None) == status
    assert lib.miep_last_error()


def test_gate_pointers(lib):
    g = gate()
    assert lib.miep_gate_topk(None, 16, None, 16, 16, None) == EINVAL
    assert lib.miep_gate_topk(g, None, None, 16, 16, None) == EINVAL
    assert lib.miep_gate_topk(g, 24, None, 16, 16, None) == EUNSUPPORTED
    assert lib.miep_gate_topk(g, 16, None, None, 16, None) == EINVAL
    assert lib.miep_gate_topk(g, 16, None, 16, None, None) == EINVAL
    assert lib.miep_gate_topk_backward(g, None, 16, 16, 16, None) == EINVAL
    assert lib.miep_gate_topk_backward(g, 16, 16, None, 16, None) == EINVAL
    assert lib.miep_gate_topk_backward(g, 16, 16, 16, None, None) == EINVAL
    assert lib.miep_gate_topk_backward(g, 16, 16, 16, 8, None) == EUNSUPPORTED


@pytest.mark.parametrize("rows,n,k,status", [
    (-1, 64, 64, EINVAL), (8, 0, 64, EINVAL), (8, 64, -8, EINVAL), (8, 60, 64, EUNSUPPORTED), (8, 64, 12, EUNSUPPORTED),
    (8, (1 << 21) + 8, 64, EUNSUPPORTED), (8, 64, 1 << 22, EUNSUPPORTED), (2 ** 31 - 1, 64, 64, EUNSUPPORTED),
    (2 ** 30, 1 << 20, 64, EUNSUPPORTED)])
def test_linear_sizes(lib, rows, n, k, status):
    assert lib.miep_linear(16, rows, 16, n, k, None, 0, None, None, 16, 0, None) == status
    assert lib.miep_linear_dgrad(16, rows, 16, n, k, 16, None) == status
    assert lib.miep_linear_wgrad(16, 16, rows, n, k, 1, 0, 16, None) == status


def test_linear_arguments(lib):
    def linear(x=16, w=16, n=64, k=64, bias=None, act=0, res=None, z=None, y=16):
        return lib.miep_linear(x, 8, w, n, k, bias, act, res, z, y, 0, None)

    assert [linear(x=None), linear(w=None), linear(y=None), linear(act=6), linear(act=-1)] == [EINVAL] * 5
    assert [linear(x=8), linear(w=24), linear(bias=4), linear(res=8), linear(z=8), linear(y=8)] == [EUNSUPPORTED] * 6
    assert linear(act=5, n=72) == EUNSUPPORTED                                # gate and up of 36 columns
    assert linear(act=5, n=1 << 20, k=2048) == EUNSUPPORTED and b"4 GiB" in lib.miep_last_error()

    def back(dy=16, z=16, act=2, dz=16, db=None, ws=None, parts=0, n=64):
        return lib.miep_linear_act_backward(dy, 0, z, 8, n, act, dz, db, 0, ws, parts, None)

    assert [back(dy=None), back(z=None), back(act=9), back(db=16), back(db=16, parts=4)] == [EINVAL] * 5
    assert [back(dy=8), back(z=8), back(dz=8), back(db=8, ws=16, parts=1), back(act=5, n=72)] == [EUNSUPPORTED] * 5
    assert back(dz=None) == OK                                                # nothing asked for
    assert lib.miep_linear_wgrad(16, 16, 8, 64, 64, 0, 1, 16, None) == EINVAL    # accumulating into bf16
    assert lib.miep_linear_wgrad(16, 16, 8, 64, 64, 1, 0, None, None) == EINVAL
    assert lib.miep_linear_wgrad(16, 16, 8, 1 << 20, 1 << 20, 1, 0, 16, None) == EUNSUPPORTED
    assert lib.miep_linear_dgrad(16, 8, None, 64, 64, 16, None) == EINVAL


def layer(**kw):
    d = dict(num_tokens=4, num_topk=2, num_experts=8, hidden=256, inner=128, scales_ue8m0=0, first_expert=0)
    d.update(kw)
    return ctypes.byref(_lib.LayerC(**d))


@pytest.mark.parametrize("kw,status", [
    (dict(num_tokens=-1), EINVAL), (dict(num_topk=0), EINVAL), (dict(num_experts=0), EINVAL), (dict(hidden=0), EINVAL),
    (dict(inner=-8), EINVAL), (dict(num_tokens=129), EUNSUPPORTED), (dict(num_topk=65), EUNSUPPORTED),
    (dict(hidden=100), EUNSUPPORTED), (dict(inner=132), EUNSUPPORTED), (dict(hidden=1 << 22), EUNSUPPORTED),
    (dict(hidden=1 << 20, inner=2048), EUNSUPPORTED), (dict(num_experts=8192), EUNSUPPORTED),
    (dict(num_tokens=128, num_topk=64, inner=1 << 19, hidden=128), EUNSUPPORTED),
    (dict(num_tokens=128, num_experts=4096), EUNSUPPORTED)])
def test_layer_sizes(lib, kw, status):
    assert lib.miep_expert_layer(layer(**kw), 16, 16, 16, 16, 16, None, 16, 16, None) == status
    assert lib.miep_last_error()


@pytest.mark.parametrize("N,K,fits", [(128, 1, 2619), (128, 40, 604), (64, 8, 4157), (1, 1, 4898)])
def test_layer_lists(lib, N, K, fits):
    """E * (8 * ceil(N/64) + 2) + 8 * min(E, N*K) + 6.5 * N*K under 49,000 is accepted: the next check is another one's."""
    def call(E):
        return lib.miep_expert_layer(layer(num_tokens=N, num_topk=K, num_experts=E), 16, 16, 16, 16, 16, None, 16, 8, None)

    def size(E):
        return E * (8 * -(-N // 64) + 2) + 8 * min(E, N * K) + 6.5 * N * K

    assert size(fits) < 49000 <= size(fits + 1)
    assert call(fits) == EUNSUPPORTED and b"y" in lib.miep_last_error() and b"lists" not in lib.miep_last_error()
    for E in range(fits + 1, fits + 12):
        if size(E) >= 49016:                                                  # (the lists' own rounding up to 16)
            assert call(E) == EUNSUPPORTED and b"lists" in lib.miep_last_error()


def test_layer_first_expert(lib):
    assert lib.miep_expert_layer(layer(first_expert=-1), 16, 16, 16, 16, 16, None, 16, 16, None) == EINVAL


def test_layer_arguments(lib):
    q = layer()
    args = [16, 16, 16, 16, 16, None, 16, 16]
    assert lib.miep_expert_layer(None, *args, None) == EINVAL
    for i in (0, 1, 2, 3, 4, 6, 7):
        assert lib.miep_expert_layer(q, *args[:i], None, *args[i + 1:], None) == EINVAL, i
    for i in (0, 3, 4, 5, 6, 7):
        assert lib.miep_expert_layer(q, *args[:i], 8, *args[i + 1:], None) == EUNSUPPORTED, i
    fp8 = [16, 16, 16, 16, 16, 16, 16, None, 16, 16]
    assert lib.miep_expert_layer_fp8(layer(hidden=192), *fp8, None) == EUNSUPPORTED
    assert lib.miep_expert_layer_fp8(layer(inner=136), *fp8, None) == EUNSUPPORTED
    assert lib.miep_expert_layer_fp8(q, 16, 16, 16, 16, None, 16, 16, None, 16, 16, None) == EINVAL
    assert lib.miep_expert_layer_fp8(q, 16, 16, 16, 16, 16, 16, None, None, 16, 16, None) == EINVAL


def test_binding_refuses_before_it_calls():
    f, b, i = torch.float32, torch.bfloat16, torch.int64
    logits = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="score"):
        miep.gate_topk(logits, 2, score="tanh")
    with pytest.raises(TypeError, match="logits"):
        miep.gate_topk(logits.double(), 2)
    with pytest.raises(ValueError, match="logits"):
        miep.gate_topk(logits[0], 2)
    with pytest.raises(ValueError, match="bias"):
        miep.gate_topk(logits, 2, bias=torch.zeros(7))
    with pytest.raises(TypeError, match="topk_idx"):
        miep.gate_topk_into(logits, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
    with pytest.raises(ValueError, match="d_topk_weights"):
        miep.gate_topk_backward(torch.zeros(4, 3), logits, torch.zeros(4, 2, dtype=i))
    with pytest.raises(ValueError, match="device"):
        miep.gate_topk(logits, 2)
    x, w = torch.zeros(4, 64, dtype=b), torch.zeros(32, 64, dtype=b)
    with pytest.raises(ValueError, match="activation"):
        miep.linear(x, w, activation="tanh")
    with pytest.raises(ValueError, match="x must be"):
        miep.linear(x, w[:, :32].contiguous())
    with pytest.raises(TypeError, match="bias"):
        miep.linear(x, w, bias=torch.zeros(32, dtype=b))
    with pytest.raises(ValueError, match="residual"):
        miep.linear(x, w, activation="swiglu", residual=torch.zeros(4, 32, dtype=b))
    with pytest.raises(TypeError, match="y must be"):
        miep.linear(x, w, dtype=torch.float16)
    with pytest.raises(ValueError, match="device"):
        miep.linear(x, w)
    dy = torch.zeros(4, 32, dtype=b)
    with pytest.raises(ValueError, match="needs z"):
        miep.linear_backward(dy, x, w, activation="silu")
    with pytest.raises(ValueError, match="dz"):
        miep.linear_backward_into(dy.float(), x, w, dx=torch.zeros_like(x))
    with pytest.raises(ValueError, match="workspace"):
        miep.linear_backward_into(dy, x, w, dbias=torch.zeros(32))
    with pytest.raises(TypeError, match="accumulate"):
        miep.linear_backward_into(dy, x, w, dw=torch.zeros_like(w), accumulate=True)
    with pytest.raises(ValueError, match="dy"):
        miep.linear_backward(dy[:, :16].contiguous(), x, w)
    idx, wts = torch.zeros(4, 2, dtype=i), torch.zeros(4, 2)
    w1, w2 = torch.zeros(3, 256, 64, dtype=b), torch.zeros(3, 64, 128, dtype=b)
    with pytest.raises(ValueError, match="w1 must be"):
        miep.expert_layer(x, idx, wts, w1, torch.zeros(3, 128, 64, dtype=b))
    with pytest.raises(ValueError, match="topk_weights"):
        miep.expert_layer(x, idx, wts[:, :1].contiguous(), w1, w2)
    with pytest.raises(TypeError, match="topk_idx"):
        miep.expert_layer(x, idx.int(), wts, w1, w2)
    with pytest.raises(ValueError, match="workspace"):
        miep.expert_layer_into(x, idx, wts, w1, w2, x.clone(), torch.zeros(4, 128, dtype=b))
    with pytest.raises(ValueError, match="device"):
        miep.expert_layer(x, idx, wts, w1, w2)
    s = torch.zeros(3, 2, 1, dtype=f)
    with pytest.raises(TypeError, match="codes"):
        miep.expert_layer_fp8(x, idx, wts, w1, s, w2, s)
    u1, u2 = w1.to(torch.uint8), w2.to(torch.uint8)
    with pytest.raises(ValueError, match="128"):
        miep.expert_layer_fp8(x, idx, wts, u1, s, u2, s)
    with pytest.raises(TypeError, match="w1_scales"):
        miep.expert_layer_fp8(x, idx, wts, u1, s.double(), u2, s)
