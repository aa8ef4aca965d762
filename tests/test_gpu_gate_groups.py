"""GPU parity of the choice among groups where a group's score is at an edge, against the 64-bit choice."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_get_dispatch_histogram_amd as miep  # noqa: E402
from test_gpu_gate import check, choice, clean, gen, scores  # noqa: E402

DEV = torch.device("cuda:0")


def undecided(l, score, bias, groups, top, best):
    """Tokens whose groups 64 bits cannot order.  exp, the division and the softmax's sum (some 25 additions of equal signs
    one after the other, half an ulp each) leave s within 2^-48 of itself, s + b adds 2^-53 of itself and so does the sum of
    two: two evaluations of one score differ by less than tol = 2^-46 (1 + |b|).  Where a chosen group and another one are within that
    and are not of the very same numbers (which tie on either side), either is right."""
    v = np.where(np.isinf(l), -np.inf, scores(l, score) + bias.double().numpy()).reshape(len(l), groups, -1)
    places = np.argsort(-v, axis=2, kind="stable")[:, :, :best]
    g = np.take_along_axis(v, places, 2).sum(2)
    order = np.argsort(-g, axis=1, kind="stable")
    tol = 2.0 ** -46 * (1 + np.abs(bias.numpy()).max())
    out = np.zeros(len(l), bool)
    for n in np.flatnonzero((top < groups) & np.isfinite(g).all(1)):
        last, rest = g[n, order[n, top - 1]], g[n, order[n, min(top, groups - 1)]]
        if last - rest > tol:
            continue
        of = [i for i in range(groups) if rest - tol <= g[n, i] <= last + tol]
        what = {tuple(sorted((l[n].reshape(groups, -1)[i, p], bias.view(groups, -1)[i, p].item()) for p in places[n, i])) for i in of}
        out[n] = len(what) > 1
    return out


def same_choice(logits, K, score, bias, groups, top, best):
    print("[case]", tuple(logits.shape), logits.dtype, K, score, groups, top, best, flush=True)
    idx, _ = miep.gate_topk(logits.to(DEV), K, score, bias.to(DEV), groups, top, best)
    l = clean(logits.float())
    want = choice(l, K, score, bias, groups, top, best)
    wrong = (idx.cpu().numpy() != want).any(1)
    if wrong.any():
        wrong &= ~undecided(l, score, bias, groups, top, best)
    assert not wrong.any(), "%d of %d tokens, first %d: got %s want %s" % (wrong.sum(), len(wrong), wrong.argmax(), idx[int(wrong.argmax())].tolist(),
                                                                            want[wrong.argmax()].tolist())


# 16 lanes a token up to 16 groups, 64 lanes a token beyond
@pytest.mark.parametrize("E,top", [(1, 1), (2, 1), (3, 2), (4, 1), (8, 3), (8, 4), (12, 5), (16, 4), (16, 16), (17, 4), (32, 6), (64, 9)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_of_one_expert(E, top, best, score):
    """A group that has one member scores what it does, whatever number of members is asked for."""
    K = min(top, 8)
    for seed, dtype in ((1, torch.float32), (2, torch.bfloat16)):
        logits = torch.randn(133, E, generator=gen(seed)).to(dtype)
        logits[3] = float("-inf")
        logits[5, E // 2:] = float("-inf")
        check(logits, K, score, None, E, top, best, True, 1.5)
        check(logits, K, score, torch.randn(E, generator=gen(9)) * 0.3, E, top, best)
        check(logits, min(E, top + 2), score, None, E, top, best)     # more choices than groups are left


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [4.0, 16.0, 100.0, 1000.0, 1e5])
def test_sums_that_cancel(size, score):
    """One expert of every group at +size, the others at -size: a group's score is near 1 where its terms' roundings
    are those of `size`."""
    groups, per = 4, 16
    bias = torch.full((groups, per), -size)
    bias[:, 5] = size
    logits = torch.randn(100000, groups * per, generator=gen(int(size)))
    same_choice(logits, 6, score, bias.view(-1), groups, 2, 2)


@pytest.mark.parametrize("E,groups,top", [(64, 4, 2), (48, 8, 3), (256, 8, 4), (160, 5, 2), (512, 16, 5), (1024, 8, 3)])
@pytest.mark.parametrize("size", [16.0, 100.0, 1000.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_cancelling_sums_near_each_other(E, groups, top, size, dtype):
    """The same with the groups' scores a few of those roundings apart, and with one group of them so."""
    N, per, g = 4000, E // groups, gen(E)
    base = torch.randn(N, 1, per, generator=g)
    logits = (base + torch.randn(N, groups, per, generator=g) * size * 1e-5).to(dtype).view(N, E)
    bias = torch.full((groups, per), -size)
    bias[:, per // 2] = size
    for score in ("softmax", "sigmoid"):
        same_choice(logits, 3, score, bias.view(-1), groups, top, 2)
        one = bias.clone()
        one[1:] *= 2.0 ** -30
        same_choice(logits, 3, score, one.view(-1), groups, top, 2)


@pytest.mark.parametrize("E", [64, 1024])
@pytest.mark.parametrize("best", [1, 2])
def test_sums_past_the_type(E, best):
    """Groups' scores beyond fp32's largest number keep their order."""
    groups, per = 4, E // 4
    logits = torch.randn(37, E, generator=gen(E))
    for rows in ([2.9e38, 3.0e38, 3.1e38, 3.3e38], [3.3e38, 1.0, -3.3e38, 3.4e38], [-3.0e38, -3.1e38, -2.9e38, -3.3e38]):
        bias = torch.tensor(rows)[:, None].expand(groups, per).reshape(-1)
        same_choice(logits, 6, "sigmoid", bias, groups, 2, best)
        same_choice(logits, 6, "softmax", bias, groups, 1, best)


@pytest.mark.parametrize("E", [64, 1024])
def test_an_infinite_bias(E):
    """counts as fp32's largest number, as an infinite logit does: its group has a score, or none where it is the only
    expert that is left."""
    groups, per = 4, E // 4
    logits = torch.randn(37, E, generator=gen(E))
    bias = torch.zeros(E)
    bias[per + 3] = bias[2 * per + 1] = float("inf")
    logits[::2, per:2 * per] = float("-inf")
    logits[::2, per + 3] = 1.0                                        # the only one of its group
    number = bias.clamp(max=torch.finfo(torch.float32).max)
    for best in (1, 2):
        for score in ("softmax", "sigmoid"):
            idx, w = miep.gate_topk(logits.to(DEV), 5, score, bias.to(DEV), groups, 2, best)
            got, ww = miep.gate_topk(logits.to(DEV), 5, score, number.to(DEV), groups, 2, best)
            want = choice(clean(logits), 5, score, number, groups, 2, best)
            assert np.array_equal(got.cpu().numpy(), want)
            assert torch.equal(idx, got) and torch.equal(w, ww)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,K", [(9, 4), (64, 6), (256, 8), (300, 20), (1024, 8)])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf")])
def test_gradient_of_a_masked_experts_weight(E, K, score, renorm, what):
    """That weight is 0 whatever the logits are: its gradient reaches none of them, a number or not."""
    N, g = 21, gen(E)
    logits = torch.randn(N, E, generator=g)
    idx = torch.rand(N, E, generator=g).topk(K, 1).indices
    d = torch.randn(N, K, generator=g)
    for n in range(N):                                                # one, two .. all of a token's choices
        off = idx[n, :n % K + 1]
        logits[n, off] = float("-inf") if n % 2 else float("nan")
    masked = ~torch.isfinite(logits.gather(1, idx))
    for dtype in (torch.float32, torch.bfloat16):
        l = logits.to(dtype).to(DEV)
        got = miep.gate_topk_backward(d.masked_fill(masked, what).to(DEV), l, idx.to(DEV), score, renorm, 2.0)
        want = miep.gate_topk_backward(d.masked_fill(masked, 0.0).to(DEV), l, idx.to(DEV), score, renorm, 2.0)
        assert torch.isfinite(want).all() and torch.equal(got, want)
        assert (got.cpu()[~torch.isfinite(logits)] == 0).all()
