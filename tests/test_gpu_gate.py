"""GPU parity of the router's choice and its gradient against plain 64-bit formulas.

Choices have to be equal.  Weights: exp of l - m is off by |l - m| / 2 ulp (2^-23) for the rounded difference and 2
ulp for the function, a sum of up to 32 values a lane and 6 steps over lanes by at most one ulp a step and by its
terms' own errors, divisions and products by half an ulp each.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_get_dispatch_histogram_amd as miep  # noqa: E402

DEV = torch.device("cuda:0")
ULP = 2.0 ** -23


def gen(seed):
    return torch.Generator().manual_seed(seed)


def clean(l):
    """64-bit logits by the documented rule: NaN is masked, +inf the largest number."""
    l = l.double().numpy().copy()
    l[np.isnan(l)] = -np.inf
    return np.minimum(l, np.finfo(np.float32).max)


def scores(l, score):
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        top = l.max(1, keepdims=True)
        e = np.exp(l - np.where(np.isinf(top), 0.0, top))
        total = e.sum(1, keepdims=True)
        return np.divide(e, total, out=np.zeros_like(e), where=total > 0)


def choice(l, K, score, bias, groups, top_groups, best):
    v = l if bias is None and groups == 1 else scores(l, score) + (0.0 if bias is None else bias.double().numpy())
    v = np.where(np.isinf(l), -np.inf, v)
    if groups > 1:
        per = l.shape[1] // groups
        g = -np.sort(-v.reshape(len(v), groups, per), axis=2)[:, :, :best].sum(2)
        order = np.argsort(-g, axis=1, kind="stable")[:, :top_groups]
        out = np.ones(g.shape, bool)
        np.put_along_axis(out, order, False, 1)
        v = np.where(np.repeat(out, per, 1), -np.inf, v)
    idx = np.argsort(-v, axis=1, kind="stable")[:, :K]
    return np.where(np.isinf(np.take_along_axis(v, idx, 1)), -1, idx)


def weights(l, idx, score, renorm, scale):
    """In logarithms, so that far logits keep their ratios."""
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        if score == "sigmoid":
            v = np.minimum(l, 0.0) - np.log1p(np.exp(-np.abs(l)))
        else:
            top = l.max(1, keepdims=True)
            v = l - top - np.log(np.exp(l - top).sum(1, keepdims=True))
        v = np.where(idx < 0, -np.inf, np.take_along_axis(v, np.maximum(idx, 0), 1))
        if renorm:
            top = v.max(1, keepdims=True)
            v = v - top - np.log(np.exp(v - top).sum(1, keepdims=True))
        return np.where(idx < 0, 0.0, np.exp(v)) * scale


def check(logits, K, score="softmax", bias=None, groups=1, top_groups=1, best=2, renorm=False, scale=1.0):
    idx, w = miep.gate_topk(logits.to(DEV), K, score, None if bias is None else bias.to(DEV), groups, top_groups, best, renorm, scale)
    l = clean(logits.float())
    want = choice(l, K, score, bias, groups, top_groups, best)
    assert np.array_equal(idx.cpu().numpy(), want)
    ww = weights(l, want, score, renorm, scale)
    live = np.where(np.isinf(l), 0.0, l)
    spread = np.minimum(np.abs(live - live.max(1, keepdims=True)).max(1, keepdims=True), 104.0)    # farther ones are below fp32
    tol = ww * (2 * spread + 60) * ULP + 2.0 ** -125 * scale
    off = np.abs(w.double().cpu().numpy() - ww)
    assert (off <= tol).all(), (off / np.maximum(tol, 1e-300)).max()
    return want


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E", [1, 2, 7, 63, 64, 65, 128, 160, 250, 256, 257, 384, 512, 1000, 1024, 2047, 2048])
def test_experts(E, renorm, score):
    for dtype in (torch.float32, torch.bfloat16):
        logits = (torch.randn(37, E, generator=gen(E)) * 2).to(dtype)
        check(logits, min(8, E), score, renorm=renorm, scale=2.5)
        check(logits, min(8, E), score, bias=torch.randn(E, generator=gen(E + 1)) * 0.2, renorm=renorm)


@pytest.mark.parametrize("K", [1, 2, 31, 64])
def test_many_choices_and_few_experts(K):
    for E in (64, 100, 300):
        check(torch.randn(9, E, generator=gen(K)), K, "sigmoid", renorm=True)
    check(torch.randn(5, K, generator=gen(K)), K)                     # all of them


@pytest.mark.parametrize("N", [0, 1, 3, 4, 5, 64, 4099])
def test_tokens(N):
    check(torch.randn(N, 72, generator=gen(N)), 6, "softmax", renorm=True)


GROUPS = [(256, 8, 4, 2), (256, 8, 1, 2), (256, 8, 8, 1), (64, 64, 5, 2), (60, 4, 3, 1), (63, 7, 2, 2), (160, 5, 2, 2), (2048, 64, 9, 2),
          (12, 2, 1, 2), (24, 12, 3, 2)]


@pytest.mark.parametrize("E,groups,top,best", GROUPS)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups(E, groups, top, best, score):
    K = min(8, E // groups * top)
    for seed, dtype in ((1, torch.float32), (2, torch.bfloat16)):
        logits = torch.randn(65, E, generator=gen(seed)).to(dtype)
        check(logits, K, score, None, groups, top, best, True, 1.5)
        check(logits, K, score, torch.randn(E, generator=gen(9)) * 0.1, groups, top, best)
    # more choices than the chosen groups have experts: the rest is empty
    more = min(E, E // groups * top + 2, 64)
    got = check(logits, more, score, None, groups, top, best, True)
    if more > E // groups * top:
        assert (got[:, -1] == -1).all()


def test_equal_scores_take_the_lower_index():
    few = torch.randint(0, 3, (300, 256), generator=gen(3)).float()
    check(few, 8)
    check(few, 8, "sigmoid", torch.zeros(256), renorm=True)
    check(few, 8, "sigmoid", None, 8, 3, 2)
    check(torch.zeros(4, 130), 5)
    check(few.bfloat16(), 64, "softmax", torch.randint(0, 2, (256,), generator=gen(4)).float())


def test_scores_next_to_each_other():
    """s + bias a few 2^-40 apart: 32 bits would order them by chance."""
    E, N = 128, 64
    logits = torch.randn(N, E, generator=gen(5))
    s = 1.0 / (1.0 + torch.exp(-logits[0].double()))
    bias = (1.0 - s).float()                                          # of token 0: all within a rounding of 1
    logits[1:] = logits[0]
    got = check(logits, 8, "sigmoid", bias)
    assert len(set(map(tuple, got))) == 1
    check(logits, 8, "sigmoid", bias, 8, 2, 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("extra", ["plain", "bias", "groups"])
def test_masked_experts(score, dtype, extra):
    E = 96
    l = torch.randn(12, E, generator=gen(6))
    l[0] = float("-inf")                                              # a token that takes no part
    l[1, 3:] = float("-inf")                                          # fewer experts than choices
    l[2, ::2] = float("nan")
    l[3] = float("nan")
    l[4, 5] = float("inf")
    l[5, 7], l[5, 11] = float("inf"), float("inf")
    l[6] = -1e30
    l[7, :] = -200.0                                                  # sigmoids below fp32's smallest number
    l[7, 40] = -190.0
    l[8, 10] = 200.0
    l[9] = torch.finfo(dtype).min
    l[10, :32] = float("-inf")
    kw = dict(bias=torch.randn(E, generator=gen(8)) * 0.1) if extra == "bias" else dict(groups=6, top_groups=2) if extra == "groups" else {}
    for renorm in (False, True):
        if extra != "plain":                                          # rounded scores tie where real ones do not: both sides alike
            check(l.to(dtype)[[0, 1, 2, 3, 8, 10, 11]], 6, score, renorm=renorm, **kw)
        else:
            check(l.to(dtype), 6, score, renorm=renorm)


# ------------------------------------------------------------------ gradient
def gradient(l, idx, d, score, renorm, scale):
    """Of the formula in 64 bits, entry by entry."""
    p = scores(l, score)
    out = np.zeros_like(l)
    for n in range(len(l)):
        ks = [k for k in range(idx.shape[1]) if 0 <= idx[n, k] < l.shape[1]]
        g = {k: d[n, k] * scale for k in ks}
        if renorm:
            w = {k: p[n, idx[n, k]] for k in ks}
            total = sum(w.values())
            mean = sum(w[k] * g[k] for k in ks) / total if ks else 0.0
            ds = {k: (g[k] - mean) / total for k in ks}
        else:
            ds = g
        dp = np.zeros(l.shape[1])
        for k in ks:
            dp[idx[n, k]] += ds[k]
        out[n] = dp * p[n] * (1 - p[n]) if score == "sigmoid" else p[n] * (dp - (dp * p[n]).sum())
    return out


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_the_formula_agrees_with_differences(score, renorm):
    r = np.random.RandomState(3)
    l, d = r.randn(3, 9), r.randn(3, 4)
    idx = np.argsort(-l, 1)[:, :4].copy()
    idx[1, 2] = idx[1, 0]                                             # an expert named twice
    idx[2, 3] = -1

    def loss(x):
        return (weights(x, idx, score, renorm, 1.7) * d).sum()

    want, h = gradient(l, idx, d, score, renorm, 1.7), 1e-5
    for n in range(3):
        for e in range(9):
            up, down = l.copy(), l.copy()
            up[n, e] += h
            down[n, e] -= h
            assert abs((loss(up) - loss(down)) / (2 * h) - want[n, e]) < 1e-8


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,K", [(1, 1), (9, 4), (64, 6), (65, 8), (160, 6), (256, 8), (300, 3), (512, 64), (1024, 8), (2048, 5)])
def test_gradient(E, K, score, renorm):
    N = 33
    for dtype in (torch.float32, torch.bfloat16):
        logits = torch.randn(N, E, generator=gen(E)).to(dtype)
        if E > 8:
            logits[1, 2] = float("-inf")
        idx = torch.rand(N, E, generator=gen(E + 1)).topk(K, 1).indices
        idx[0, 0] = -1
        if K > 2:
            idx[2, 1] = idx[2, 0]
            idx[3] = -1
            idx[4, 2] = E + 5                                         # no such expert
        d = torch.randn(N, K, generator=gen(E + 2))
        got = miep.gate_topk_backward(d.to(DEV), logits.to(DEV), idx.to(DEV), score, renorm, 2.5)
        l = clean(logits.float())
        want = gradient(l, idx.numpy(), d.double().numpy(), score, renorm, 2.5)
        # every term is a product of numbers that are off by (2 * spread + 60) ulp; terms: the chosen ones
        size = np.abs(d.double().numpy()).sum(1, keepdims=True) * 2.5 * np.minimum(scores(l, score) if not renorm else 1.0, 1.0) * 2
        spread = np.abs(np.where(np.isinf(l), 0, l)).max() * 2
        tol = size * (2 * spread + 60) * ULP + np.abs(want) * (2.0 ** -8 if dtype == torch.bfloat16 else 0) + 1e-37
        assert got.dtype == dtype
        off = np.abs(got.double().cpu().numpy() - want)
        assert (off <= tol).all(), (off / tol).max()


def test_streams_graph_and_a_row_left_alone():
    N, E, K = 50, 128, 6
    logits = torch.randn(N, E, generator=gen(1)).to(DEV)
    want = miep.gate_topk(logits, K, "sigmoid", renormalize=True)
    idx, w = torch.full((N + 1, K), -7, dtype=torch.int64, device=DEV), torch.full((N + 1, K), -7.0, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        miep.gate_topk_into(logits, idx[:N], w[:N], "sigmoid", renormalize=True)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            miep.gate_topk_into(logits, idx[:N], w[:N], "sigmoid", renormalize=True)
    torch.cuda.current_stream().wait_stream(side)
    for turn in range(3):
        logits.copy_(torch.randn(N, E, generator=gen(turn + 10)))
        graph.replay()
        torch.cuda.synchronize()
        want = miep.gate_topk(logits, K, "sigmoid", renormalize=True)
        assert torch.equal(idx[:N], want[0]) and torch.equal(w[:N], want[1])
        assert (idx[N] == -7).all() and (w[N] == -7).all()


@pytest.mark.parametrize("E,groups,top", [(64, 1, 1), (64, 4, 2), (160, 8, 3), (256, 1, 1), (256, 8, 4), (384, 8, 4), (100, 5, 2), (512, 16, 5), (66, 1, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_near_neighbours(E, groups, top, score, dtype):
    """Many logits (and with them scores, and sums of two) a rounding or a few apart from another expert's, at every
    place of the order: a choice by 32 bits alone is by chance there."""
    N, K = 400, min(7, E // groups * top)
    g = gen(E + groups)
    l = torch.randn(N, E, generator=g)
    half = E // 2
    step = 2.0 ** -torch.randint(17, 25, (N, half), generator=g).float()
    near = l[:, :half] * (1 + step * torch.randint(-1, 2, (N, half), generator=g).float())
    l[:, half:2 * half] = torch.where(torch.rand(N, half, generator=g) < 0.6, near, l[:, half:2 * half])
    l = l[:, torch.randperm(E, generator=g)].to(dtype)
    check(l, K, score, None, groups, top, 2, True)
    check(l, K, score, None, groups, top, 1)
    b = (torch.randn(E, generator=g) * 0.05).float()
    b[::2] = 0.0
    check(l, K, score, b, groups, top, 2, True, 2.5)
    # all within a few roundings of each other: more candidates than 16
    if groups == 1:
        check((1 + l * 2.0 ** -21).float(), K, score, torch.zeros(E), 1, 1, 2)
        check((1 + l * 2.0 ** -21).float(), K, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K", [(64, 6), (160, 8), (700, 8)])
def test_a_bias_that_is_no_number(score, E, K):
    """leaves its expert out of the choice, and in the softmax's sum"""
    logits, bias = torch.randn(20, E, generator=gen(E)), torch.randn(E, generator=gen(E + 1)) * 0.2
    out = torch.zeros(E, dtype=torch.bool)
    out[::3] = True
    bias[::6], bias[3::6] = float("-inf"), float("nan")
    for groups in (1, 4):
        idx, w = miep.gate_topk(logits.to(DEV), K, score, bias.to(DEV), groups, groups // 2 or 1)
        l = clean(logits)
        v = scores(l, score) + bias.double().numpy()
        v[:, out.numpy()] = -np.inf
        if groups > 1:
            best = -np.sort(-v.reshape(20, groups, -1), axis=2)[:, :, :2].sum(2)
            keep = np.argsort(-best, axis=1, kind="stable")[:, :groups // 2]
            for n in range(20):
                for g in set(range(groups)) - set(keep[n]):
                    v[n, g * (E // groups):(g + 1) * (E // groups)] = -np.inf
        want = np.argsort(-v, axis=1, kind="stable")[:, :K]
        assert np.array_equal(idx.cpu().numpy(), want)
        ww = weights(l, want, score, False, 1.0)
        spread = 2 * np.abs(l).max()
        assert (np.abs(w.double().cpu().numpy() - ww) <= ww * (2 * spread + 60) * ULP).all()


def test_offsets_past_32_bits():
    """More than 2^31 logits: the last tokens, and their gradient."""
    N, E, K, last = 4200000, 512, 4, 50
    assert N * E > 2 ** 31
    logits = torch.zeros(N, E, dtype=torch.bfloat16, device=DEV)
    tail = (torch.randn(last, E, generator=gen(1)) * 2).bfloat16()
    logits[-last:] = tail.to(DEV)
    idx, w = miep.gate_topk(logits, K)
    assert np.array_equal(idx[-last:].cpu().numpy(), choice(clean(tail.float()), K, "softmax", None, 1, 1, 2))
    assert torch.equal(idx[N // 2], torch.arange(K, device=DEV)) and torch.equal(idx[:1], idx[N - last - 1:N - last])
    d = torch.ones(N, K, device=DEV)
    d[:, 0] = 2
    got = miep.gate_topk_backward(d, logits, idx)
    part = miep.gate_topk_backward(d[-last:].contiguous(), tail.to(DEV), idx[-last:].contiguous())
    assert torch.equal(got[-last:], part) and torch.equal(got[0], got[N - last - 1])
