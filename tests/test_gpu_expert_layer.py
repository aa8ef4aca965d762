"""GPU parity of the expert layer for a few tokens against a plain 64-bit form.

Whole numbers: gates of 32 and more have a sigmoid of exactly 1 in fp32, so with small integers in x and the weights
the gates, the activation before its rounding to bf16, and every sum are exact in fp32; the rounding itself is the same
on both sides, and results have to agree with the 64-bit form's rounded once.
Normal numbers: the activation is off by its rounding (2^-8) and a few fp32 roundings, sums by an fp32 ulp an addition.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_get_dispatch_histogram_amd as miep  # noqa: E402

DEV = torch.device("cuda:0")
BF, F8 = torch.bfloat16, torch.float8_e4m3fn
ULP, BF_HALF = 2.0 ** -23, 2.0 ** -8


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rint(lo, hi, shape, seed):
    return torch.randint(lo, hi + 1, shape, generator=gen(seed), device=DEV).float()


def routing(N, K, experts, seed, kind="uniform"):
    score = torch.rand(N, experts, generator=gen(seed), device=DEV)
    if kind == "hot":                                                 # everyone takes the first experts
        score[:, :K] += 1
    idx = score.topk(K, 1).indices
    if kind == "masked":
        idx = torch.where(torch.rand(N, K, generator=gen(seed + 1), device=DEV) < 0.5, -1, idx)
        idx[N // 2] = -1
    if kind == "twice" and K > 1:
        idx[:, 1] = idx[:, 0]
    return idx


def plain(x, idx, wts, w1, w2, first=0, residual=None, exact=False):
    """64 bits; with `exact` the activation rounded to bf16 as the kernels round it.  Also the bound of its error."""
    N, H, I = x.shape[0], x.shape[1], w2.shape[2]
    y = torch.zeros(N, H, dtype=torch.float64, device=DEV) if residual is None else residual.double()
    tol = torch.zeros_like(y)
    for e in range(w1.shape[0]):
        n, k = (idx == first + e).nonzero(as_tuple=True)
        if not n.numel():
            continue
        h = x[n].double() @ w1[e].t()
        th = (H + 2) * ULP * (x[n].double().abs() @ w1[e].abs().t())
        g, u, tg, tu = h[:, :I], h[:, I:], th[:, :I], th[:, I:]
        s = torch.sigmoid(g)
        a = g * s * u
        ta = 1.1 * u.abs() * tg + (g * s).abs() * tu + 1.1 * tg * tu + 8 * ULP * (g * u).abs() + BF_HALF * a.abs()
        if exact:
            assert (g >= 32).all() and (g * u).abs().max() < 2 ** 24
            a, ta = (g * u).to(torch.float32).to(BF).double(), 0 * ta
        c = wts[n, k, None].double()
        y.index_add_(0, n, c * (a @ w2[e].t()))
        tol.index_add_(0, n, c.abs() * (ta @ w2[e].abs().t() + (I + 4) * ULP * (a.abs() @ w2[e].abs().t())))
    return y, tol + (2 ** -21 + BF_HALF) * y.abs()


def whole(N, K, E, H, I, seed, experts=None, kind="uniform", fp8=None):
    """Inputs whose every step is exact (see above); fp8: None, "f32" or "ue8m0" scales."""
    experts = experts or E
    dense = min(1.0, 400.0 / H)
    x = (torch.rand(N, H, generator=gen(seed), device=DEV) < dense).float()
    x[:, ::max(1, H // 48)] = 1                                       # 48 channels everyone has ...
    gate = rint(0, 1, (E, I, H), seed + 1)
    gate[:, :, ::max(1, H // 48)] = 1                                 # ... and every gate takes: 48 at least
    if H < 48:
        gate[:] = 48
    up = rint(-1, 1, (E, I, H), seed + 2) * (torch.rand(E, I, H, generator=gen(seed + 3), device=DEV) < 0.1)
    w2 = rint(-1, 1, (E, H, I), seed + 4)
    w1 = torch.cat([gate, up], 1)
    idx = routing(N, K, experts, seed + 5, kind)
    wts = 2.0 ** rint(-3, 0, (N, K), seed + 6)
    if not fp8:
        return x.to(BF), idx, wts, (w1.to(BF),), (w2.to(BF),), w1.double(), w2.double()

    def scaled(w, s):
        E_, n, k = w.shape
        e = rint(0, 2, (E_, n // 128, k // 128), s)
        v = (w.view(E_, n // 128, 128, k // 128, 128) * 2.0 ** e.view(E_, n // 128, 1, k // 128, 1)).view(w.shape)
        return (w.to(F8), 2.0 ** e if fp8 == "f32" else (e + 127).to(torch.uint8)), v.double()

    q1, v1 = scaled(w1, seed + 7)
    q2, v2 = scaled(w2, seed + 8)
    return x.to(BF), idx, wts, q1, q2, v1, v2


def run(x, idx, wts, q1, q2, **kw):
    f = miep.expert_layer if len(q1) == 1 else miep.expert_layer_fp8
    return f(x, idx, wts, *q1, *q2, **kw)


def check_whole(N, K, E, H, I, seed=1, experts=None, first=0, kind="uniform", fp8=None, residual=False):
    print("[case]", N, K, E, H, I, experts, first, kind, fp8, residual, flush=True)
    x, idx, wts, q1, q2, v1, v2 = whole(N, K, E, H, I, seed, experts, kind, fp8)
    r = rint(-9, 9, (N, H), seed + 20).to(BF) if residual else None
    y = run(x, idx, wts, q1, q2, first_expert=first, residual=r)
    want, tol = plain(x, idx, wts, v1, v2, first, r, exact=True)
    # Sums of whole numbers times eighths are exact in fp32 while their magnitudes add up to less than 2^24 eighths:
    # then the results are the exact ones rounded once.  Larger ones are off by an fp32 ulp of those magnitudes an
    # addition (the first product and the activation are exact all the same), and half a step of bf16.
    magnitudes = (tol - (2 ** -21 + BF_HALF) * want.abs()) / ((I + 4) * ULP)
    sums_exact = magnitudes + (0 if r is None else r.double().abs()) < 2 ** 21
    assert sums_exact.any() or I > 1000
    assert torch.equal(y[sums_exact], want.to(torch.float32).to(BF)[sums_exact]), (y.double() - want).abs().max()
    assert ((y.double() - want).abs() <= tol).all()


# tokens: columns of 16, 32 and 64 of an expert, one and two words of its token mask
@pytest.mark.parametrize("N", [1, 2, 7, 16, 17, 33, 63, 64, 65, 100, 128])
@pytest.mark.parametrize("kind", ["uniform", "hot", "masked", "twice"])
def test_tokens(N, kind):
    check_whole(N, 4, 12, 192, 72, kind=kind, residual=N % 2 == 0)
    check_whole(N, 2, 6, 256, 128, kind=kind, fp8="ue8m0" if N % 2 else "f32", residual=N % 2 == 1)


# channels: tiles' borders, contractions shorter than a step, not whole, and of many steps
@pytest.mark.parametrize("H,I", [(8, 8), (56, 16), (64, 24), (120, 200), (512, 64), (1000, 40), (2048, 136), (4104, 16), (40, 1032)])
@pytest.mark.parametrize("N", [1, 20])
def test_channels(N, H, I):
    check_whole(N, 3, 5, H, I)


@pytest.mark.parametrize("H,I", [(128, 128), (256, 384), (1152, 128), (384, 1408), (2048, 256)])
@pytest.mark.parametrize("N", [1, 5, 40])
@pytest.mark.parametrize("scales", ["f32", "ue8m0"])
def test_channels_fp8(N, H, I, scales):
    check_whole(N, 3, 5, H, I, fp8=scales)


@pytest.mark.parametrize("E,K,N", [(1, 1, 1), (1, 1, 40), (2, 2, 128), (64, 64, 3), (300, 8, 64), (513, 6, 100), (1030, 2, 9), (2000, 1, 128)])
def test_experts(E, K, N):
    check_whole(N, K, E, 64, 16)


@pytest.mark.parametrize("first", [0, 8, 24, 40])
def test_a_ranks_share(first):
    """Entries of other ranks' experts add nothing; a share that no token chose gives the residual, or zeros."""
    check_whole(30, 4, 8, 128, 64, experts=32, first=first, residual=True)
    check_whole(30, 4, 8, 128, 128, experts=32, first=first, fp8="f32")
    check_whole(5, 4, 8, 128, 64, experts=1000, first=2 ** 33 if first == 40 else first)


def test_no_tokens_and_untouched_rows():
    x, idx, wts, q1, q2, v1, v2 = whole(6, 2, 4, 64, 16, 3)
    assert run(x[:0], idx[:0], wts[:0], q1, q2).shape == (0, 64)
    y, ws = torch.full((7, 64), -77.0, dtype=BF, device=DEV), torch.full((13, 16), -77.0, dtype=BF, device=DEV)
    miep.expert_layer_into(x, idx, wts, *q1, *q2, y[:6], ws[:12])
    want, _ = plain(x, idx, wts, v1, v2, exact=True)
    assert torch.equal(y[:6], want.to(BF)) and (y[6] == -77).all() and (ws[12] == -77).all()
    y[:6] = 3
    miep.expert_layer_into(x, idx, wts, *q1, *q2, y[:6], ws[:12], residual=y[:6])      # in place
    assert torch.equal(y[:6], (want + 3).to(BF)) and (y[6] == -77).all()


def test_what_is_not_a_number_stays_where_it_is():
    """Experts that nobody chose, a token's own row, and the workspace's old values."""
    x, idx, wts, q1, q2, v1, v2 = whole(20, 2, 6, 128, 128, 5)
    idx = idx.clamp(max=4)
    idx[:, 1] = -1
    w1, w2 = q1[0].clone(), q2[0].clone()
    w1[5], w2[5] = float("nan"), float("nan")
    x[3] = float("nan")
    y, ws = torch.empty(20, 128, dtype=BF, device=DEV), torch.full((40, 128), float("nan"), dtype=BF, device=DEV)
    miep.expert_layer_into(x, idx, wts, w1, w2, y, ws)
    keep = [i for i in range(20) if i != 3]
    assert torch.isnan(y[3]).all()
    want, _ = plain(x[keep], idx[keep], wts[keep], v1, v2, exact=True)
    assert torch.equal(y[keep], want.to(BF))


@pytest.mark.parametrize("N,K,E,H,I", [(1, 8, 16, 1024, 768), (13, 4, 8, 512, 256), (64, 8, 16, 256, 384), (128, 2, 3, 384, 128)])
@pytest.mark.parametrize("fp8", [False, True])
def test_normal_numbers(N, K, E, H, I, fp8):
    x = torch.randn(N, H, generator=gen(1), device=DEV).to(BF)
    idx, wts = routing(N, min(K, E), E, 2), torch.softmax(torch.randn(N, min(K, E), generator=gen(3), device=DEV), 1)
    w1 = torch.randn(E, 2 * I, H, generator=gen(4), device=DEV) * H ** -0.5
    w2 = torch.randn(E, H, I, generator=gen(5), device=DEV) * I ** -0.5
    r = torch.randn(N, H, generator=gen(6), device=DEV).to(BF)
    if fp8:
        s1 = torch.rand(E, 2 * I // 128, H // 128, generator=gen(7), device=DEV) / 200 + 1e-3
        s2 = torch.rand(E, H // 128, I // 128, generator=gen(8), device=DEV) / 200 + 1e-3
        big = lambda s: s.repeat_interleave(128, 1).repeat_interleave(128, 2)  # noqa: E731
        c1, c2 = (w1 / big(s1)).clamp(-448, 448).to(F8), (w2 / big(s2)).clamp(-448, 448).to(F8)
        y = miep.expert_layer_fp8(x, idx, wts, c1, s1, c2, s2, residual=r)
        w1, w2 = c1.double() * big(s1).double(), c2.double() * big(s2).double()
    else:
        y = miep.expert_layer(x, idx, wts, w1.to(BF), w2.to(BF), residual=r)
        w1, w2 = w1.to(BF).double(), w2.to(BF).double()
    want, tol = plain(x, idx, wts, w1, w2, residual=r)
    off = (y.double() - want).abs()
    assert (off <= tol).all(), (off / tol).max()
    assert (y.double() - want).norm() < 2 ** -8 * want.norm()         # two roundings of at most 2^-9 on the average


def test_every_code_is_exact():
    """Each E4M3 code through the products: bf16 holds all of them."""
    H = I = 128
    codes = torch.arange(256, dtype=torch.uint8, device=DEV)
    codes = codes[(codes & 0x7f) != 0x7f]                             # without the two NaN
    w1 = torch.zeros(1, 2 * I, H, dtype=torch.uint8, device=DEV)
    one = torch.tensor(1.0).to(F8).view(torch.uint8).item()
    w1[0, :I, 0] = torch.tensor(64.0).to(F8).view(torch.uint8).item()                 # gate: 64
    w2 = torch.zeros(1, H, I, dtype=torch.uint8, device=DEV)
    w2[0, torch.arange(H), torch.arange(I)] = one                     # the identity
    s1, s2 = torch.ones(1, 2, 1, device=DEV), torch.ones(1, 1, 1, device=DEV)
    x = torch.zeros(1, H, dtype=BF, device=DEV)
    x[0, 0] = 1
    idx, wts = torch.zeros(1, 1, dtype=torch.int64, device=DEV), torch.ones(1, 1, device=DEV)
    for half in (codes[:128], codes[126:]):
        w1[0, I:, 0] = half
        y = miep.expert_layer_fp8(x, idx, wts, w1.view(F8), s1, w2.view(F8), s2)
        assert torch.equal(y[0].float(), 64.0 * half.view(F8).float())
        w2[0, torch.arange(H), torch.arange(I)] = half                # and through the second product
        w1[0, I:, 0] = one
        y = miep.expert_layer_fp8(x, idx, wts, w1.view(F8), s1, w2.view(F8), s2)
        assert torch.equal(y[0].float(), 64.0 * half.view(F8).float())
        w2[0, torch.arange(H), torch.arange(I)] = one


def test_streams_and_graphs():
    x, idx, wts, q1, q2, v1, v2 = whole(24, 4, 10, 256, 128, 9, fp8="f32")
    y, ws = torch.empty(24, 256, dtype=BF, device=DEV), torch.empty(96, 128, dtype=BF, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        miep.expert_layer_fp8_into(x, idx, wts, *q1, *q2, y, ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            miep.expert_layer_fp8_into(x, idx, wts, *q1, *q2, y, ws)
    torch.cuda.current_stream().wait_stream(side)
    for turn in range(3):                                             # another routing on every replay
        idx.copy_(routing(24, 4, 10, 30 + turn, ("uniform", "hot", "masked")[turn]))
        graph.replay()
        torch.cuda.synchronize()
        want, _ = plain(x, idx, wts, v1, v2, exact=True)
        assert torch.equal(y, want.to(BF))
    # the same bits on every call
    a = run(x, idx, wts, q1, q2)
    assert all(torch.equal(a, run(x, idx, wts, q1, q2)) for _ in range(5))


# the longest lists that are taken: two words a token mask and few entries, and many entries
@pytest.mark.parametrize("E,K", [(2619, 1), (604, 40)])
@pytest.mark.parametrize("H", [64, 4104])
def test_longest_lists(E, K, H):
    check_whole(128, K, E, H, 8)


def test_offsets_past_32_bits():
    """Weights of more than 4 GiB: the last expert's."""
    N, E, H, I = 3, 152, 4096, 2048
    assert 2 * E * I * H > 2 ** 31
    w1 = torch.zeros(E, 2 * I, H, dtype=BF, device=DEV)
    w2 = torch.zeros(E, H, I, dtype=BF, device=DEV)
    x, idx, wts, q1, q2, v1, v2 = whole(N, 1, 1, H, I, 4)
    w1[-1], w2[-1] = q1[0][0], q2[0][0]
    assert torch.equal(miep.expert_layer(x, idx + E - 1, wts, w1, w2), miep.expert_layer(x, idx, wts, *q1, *q2))


@pytest.mark.parametrize("product", [1, 2])
def test_exponent_bytes_at_their_ends(product):
    """0 is 2^-127, 254 2^127 and 255 NaN, in either product."""
    H = I = 128
    one = torch.tensor(1.0).to(F8).view(torch.uint8).item()
    w1 = torch.zeros(1, 2 * I, H, dtype=torch.uint8, device=DEV)
    w1[0, :I, 0], w1[0, I:, 1] = one, one                             # gate: x[0], up: x[1]
    w2 = torch.zeros(1, H, I, dtype=torch.uint8, device=DEV)
    w2[0, torch.arange(H), torch.arange(I)] = one
    idx, wts = torch.zeros(1, 1, dtype=torch.int64, device=DEV), torch.ones(1, 1, device=DEV)
    x = torch.zeros(1, H, dtype=BF, device=DEV)
    for byte in (0, 1, 254, 255):
        s1 = torch.full((1, 2, 1), 127, dtype=torch.uint8, device=DEV)
        s2 = torch.full((1, 1, 1), 127, dtype=torch.uint8, device=DEV)
        x[0, 0] = 64.0
        x[0, 1] = 2.0 ** 60 if byte < 128 else 2.0 ** -60
        (s1[0, 1:] if product == 1 else s2)[:] = byte
        y = miep.expert_layer_fp8(x, idx, wts, w1.view(F8), s1, w2.view(F8), s2)
        if byte == 255:
            assert torch.isnan(y).all()
        else:
            assert torch.equal(y.double(), torch.full_like(y.double(), 64.0 * float(x[0, 1]) * 2.0 ** (byte - 127)))


def test_two_streams_at_once():
    """Calls of two streams side by side, each with a workspace and an output of its own."""
    sides = [torch.cuda.Stream() for _ in range(2)]
    cases = []
    for N, fp8 in ((5, None), (40, "ue8m0")):
        x, idx, wts, q1, q2, v1, v2 = whole(N, 3, 8, 512, 256, N, fp8=fp8)
        want, _ = plain(x, idx, wts, v1, v2, exact=True)
        f = miep.expert_layer_fp8_into if fp8 else miep.expert_layer_into
        y, ws = torch.empty(N, 512, dtype=BF, device=DEV), torch.empty(N * 3, 256, dtype=BF, device=DEV)
        cases.append((lambda f=f, a=(x, idx, wts, *q1, *q2, y, ws): f(*a), y, want.to(BF)))
    torch.cuda.synchronize()
    for _ in range(10):
        for side, (call, y, _) in zip(sides, cases):
            with torch.cuda.stream(side):
                call()
    torch.cuda.synchronize()
    for _, y, want in cases:
        assert torch.equal(y, want)
