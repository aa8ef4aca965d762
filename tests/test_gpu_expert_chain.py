"""The expert operators together, between dispatch and combine, as they are
used: a training step in normal mode with every gradient, and FP8 serving behind
the low-latency dispatch, eager and captured.

Tolerances: each bf16 rounding is off by at most 2^-8 of its array's norm, each
E4M3 one by 2^-4; a product with Gaussian weights passes an error on at no more
than about 3 times its share of the result (the weights' largest singular value
over their root mean square one, square matrices: 2; SwiGLU's slope: 1.1).  So
n roundings move a result by less than 3 n 2^-8 of its norm.
"""
import numpy as np
import pytest
import torch

from combine_get_dispatch_histogram_amd import workloads as wl

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_get_dispatch_histogram_amd as miep  # noqa: E402

DEV = torch.device("cuda:0")
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


def off(got, want):
    return float((got.detach().cpu().double() - want).norm() / want.norm())


@pytest.mark.parametrize("R,mask,align", [(4, 0.0, 1), (8, 0.15, 16)])
def test_training_step(R, mask, align):
    T, E, K, H, I = 32, 16, 4, 256, 192
    N = R * T
    g = torch.Generator().manual_seed(R)
    idx = wl.topk_uniform(N, E, K, g)
    idx[torch.rand((N, K), generator=g) < mask] = -1
    wts, x = wl.gate_weights(N, K, g), wl.activations(N, H, g)
    w1 = (torch.randn((E, 2 * I, H), generator=g) * H ** -0.5).to(BF)
    w2 = (torch.randn((E, H, I), generator=g) * I ** -0.5).to(BF)
    dout = wl.activations(N, H, g)
    w1d, w2d = w1.to(DEV), w2.to(DEV)

    ntpr, _, ntpe, itr = miep.get_dispatch_layout(idx.to(DEV), E, R)
    recv_x, _, recv_idx, recv_w, nrte, handle = miep.dispatch(x.to(DEV), idx.to(DEV), wts.to(DEV), ntpr, itr, ntpe, E, expert_alignment=align)
    order = miep.expert_order(recv_idx, handle.recv_rank_offset, E, align, num_slots=int(nrte.sum()))
    assert torch.equal(nrte.view(-1).long(), -(-order.group_rows.long() // align) * align)
    h = miep.grouped_gemm(recv_x, w1d, order.groups, row_index=order.slot_row)
    a = miep.swiglu(h, order.groups)
    z = miep.grouped_gemm(a, w2d, order.groups)
    y = miep.expert_reduce(z, order, recv_w)
    out, _ = miep.combine(y, handle)

    dy, _ = miep.cached_dispatch(dout.to(DEV), handle)                    # combine's gradient
    dz, d_recv_w = miep.expert_reduce_backward(dy, z, order, recv_w)
    da = miep.grouped_gemm_dgrad(dz, w2d, order.groups)
    dw2 = miep.grouped_gemm_wgrad(dz, a, order.groups)
    dh = miep.swiglu_backward(da, h, order.groups)
    dslots = miep.grouped_gemm_dgrad(dh, w1d, order.groups)
    dw1 = miep.grouped_gemm_wgrad(dh, recv_x, order.groups, row_index=order.slot_row)
    dx, dwts = miep.combine(miep.expert_reduce(dslots, order), handle, d_recv_w)

    xd, wd, w1r, w2r = (t.double().requires_grad_() for t in (x, wts, w1, w2))
    want = torch.zeros((N, H), dtype=torch.float64)
    for e in range(E):
        n, k = (idx == e).nonzero(as_tuple=True)
        v = xd[n] @ w1r[e].T
        act = torch.nn.functional.silu(v[:, :I]) * v[:, I:]
        want = want.index_add(0, n, wd[n, k, None] * (act @ w2r[e].T))
    (want * dout.double()).sum().backward()
    assert off(out, want.detach()) < 3 * 5 * 2.0 ** -8                    # h, a, z, y, out
    assert off(dwts, wd.grad * (idx >= 0)) < 3 * 4 * 2.0 ** -8            # dy is exact; h, a, z
    assert off(dw2, w2r.grad) < 3 * 3 * 2.0 ** -8                         # dz, h, a
    assert off(dw1, w1r.grad) < 3 * 4 * 2.0 ** -8                         # dz, da, h, dh
    assert off(dx, xd.grad) < 3 * 7 * 2.0 ** -8                           # those, dslots, rows, dx


def _weights(L, N, K, g, pow2):
    nb = N // 128
    v = (torch.randn((L, N, K), generator=g) * K ** -0.5).view(L, nb, 128, K // 128, 128)
    s = v.abs().amax((2, 4)) / 448
    s = torch.exp2(torch.ceil(torch.log2(s))) if pow2 else s
    q = (v / s.view(L, nb, 1, K // 128, 1)).to(F8).view(L, N, K)
    full = q.float().double() * s.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
    return q.to(DEV), ((torch.log2(s) + 127).to(torch.uint8) if pow2 else s).to(DEV), full


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("T,M", [(1, 4), (24, 32)])      # one token a rank, and more than a tile's rows an expert
def test_low_latency_serving(T, M, pow2):
    R, E, K, H, I, d = 4, 8, 3, 512, 256, 1
    L = E // R
    g = torch.Generator().manual_seed(T)
    idx, x, wts = wl.topk_uniform(R * T, E, K, g), wl.activations(R * T, H, g), wl.gate_weights(R * T, K, g)
    q1, s1, w1 = _weights(L, 2 * I, H, g, pow2)
    q2, s2, w2 = _weights(L, H, I, g, pow2)
    xd, idxd, wtsd = x.to(DEV), idx.to(DEV), wts.to(DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    recv = dict(packed_recv_x=torch.empty((L, R * M, H), dtype=F8, device=DEV),
                packed_recv_x_scales=torch.empty((L, R * M, H // 128), device=DEV),
                packed_recv_x_scales_ue8m0=torch.empty((L, R * M, H // 128), dtype=torch.uint8, device=DEV) if pow2 else None,
                packed_recv_src_info=torch.empty((L, R * M), **i32),
                packed_recv_layout_range=torch.empty((L, R), dtype=torch.int64, device=DEV),
                packed_recv_count=torch.empty((L,), **i32))
    msg = torch.empty((L, R, M, miep.ll_msg_bytes(H, True)), dtype=torch.uint8, device=DEV)
    cnt = torch.empty((L, R), **i32)
    h = torch.empty((L, R * M, 2 * I), dtype=BF, device=DEV)
    a = torch.empty((L, R * M, I), dtype=F8, device=DEV)
    sc = torch.empty((L, R * M, I // 128), device=DEV)
    ue = torch.empty((L, R * M, I // 128), dtype=torch.uint8, device=DEV) if pow2 else None
    y = torch.empty((L, R * M, H), dtype=BF, device=DEV)
    out = torch.empty((R * T, H), dtype=BF, device=DEV)
    groups = miep.RowGroups.low_latency(recv)
    expect = -(-T * K // L)

    def step():
        miep.low_latency_dispatch_into(xd, idxd, R, M, E, d, True, pow2, pow2, msg, cnt, **recv)
        xs = recv["packed_recv_x_scales_ue8m0"] if pow2 else recv["packed_recv_x_scales"]
        miep.grouped_gemm_fp8_into(recv["packed_recv_x"], xs, q1, s1, groups, h, expected_rows=expect)
        miep.swiglu_fp8_into(h, groups, a, sc, round_scale=pow2, a_scales_ue8m0=ue)
        miep.grouped_gemm_fp8_into(a, ue if pow2 else sc, q2, s2, groups, y, expected_rows=expect)
        miep.low_latency_combine_into(y, idxd, wtsd, recv["packed_recv_src_info"], recv["packed_recv_layout_range"], R, M, E, d, out)

    def reference():
        ref = torch.zeros((R * T, H), dtype=torch.float64)
        xr, ir, wr = xd.cpu().double(), idxd.cpu(), wtsd.cpu().double()
        for l in range(L):
            n, k = (ir == d * L + l).nonzero(as_tuple=True)
            v = xr[n] @ w1[l].T
            act = torch.nn.functional.silu(v[:, :I]) * v[:, I:]
            ref.index_add_(0, n, wr[n, k, None] * (act @ w2[l].T))
        return ref

    step()
    want = reference()
    assert want.norm() > 0
    assert off(out, want) < 3 * (2 * 2.0 ** -4 + 3 * 2.0 ** -8)           # x and a in E4M3; h, y, out in bf16

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for seed in range(4):                                                 # replays on new tokens and routing, each against eager
        g2 = torch.Generator().manual_seed(100 + seed)
        xd.copy_(wl.activations(R * T, H, g2))
        idxd.copy_(wl.topk_uniform(R * T, E, K, g2))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        out.fill_(-7.0)
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out)


def test_training_products_in_a_graph():
    """Order, products, gradients and reduction captured together; each replay on new routing equals the eager run."""
    cap, K, E, H, N = 300, 4, 8, 136, 264
    g = torch.Generator().manual_seed(1)
    topk = torch.randint(-1, E, (cap, K), generator=g).to(DEV)
    offs = torch.tensor([0, cap - 7], dtype=torch.int32, device=DEV)
    x = torch.randn((cap, H), generator=g).to(BF).to(DEV)
    w = torch.randn((E, N, H), generator=g).to(BF).to(DEV)
    wts = torch.rand((cap, K), generator=g).to(DEV)
    order = miep.ExpertOrder.allocate(topk, offs, E, 8)
    S = order.num_slots
    z = torch.zeros((S, N), dtype=BF, device=DEV)
    y = torch.zeros((cap, N), dtype=BF, device=DEV)
    dz, dxs = torch.zeros_like(z), torch.zeros((S, H), dtype=BF, device=DEV)
    dw, dwt = torch.zeros((E, N, H), device=DEV), torch.zeros_like(wts)
    dx = torch.zeros_like(x)
    outs = (z, y, dz, dxs, dw, dwt, dx)

    def step():
        miep.expert_order_into(topk, order, 8)
        miep.grouped_gemm_into(x, w, order.groups, z, row_index=order.slot_row)
        miep.expert_reduce_into(z, order, y, wts)
        miep.expert_reduce_backward_into(y, z, order, dz, wts, dwt)
        miep.grouped_gemm_dgrad_into(dz, w, order.groups, dxs)
        miep.grouped_gemm_wgrad_into(dz, x, order.groups, dw, row_index=order.slot_row)
        miep.expert_reduce_into(dxs, order, dx)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(4):
        topk.copy_(torch.randint(-1, E, (cap, K), generator=g))
        x.copy_(torch.randn((cap, H), generator=g))
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, outs))
