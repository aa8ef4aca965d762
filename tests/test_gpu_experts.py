"""GPU parity of the expert operators (expert order and reduction, grouped
products with their gradients, FP8 products, SwiGLU) against plain 64-bit
formulas.

Tolerances come from the arithmetic.  A sum of n products in fp32 is off by at
most one fp32 ulp (2^-23) of the sum of magnitudes per addition, whether the
adder rounds or truncates; a result rounded to bf16 by another half step,
2^-8 of its value; a product of factors in fp32 by half an ulp a factor.
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
ULP = 2.0 ** -23          # one fp32 ulp
BF_HALF = 2.0 ** -8       # half a bf16 step
F8_HALF = 2.0 ** -4       # half an E4M3 step
MARK = -77.0              # what an untouched place holds


def say(*a):
    print("[case]", *a, flush=True)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def d64(t):
    return t.detach().cpu().double()


def close(got, want, tol, what=""):
    got, want = d64(got), want.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what + ": NaN places"
    bad = ((got - want).abs() > tol) & ~torch.isnan(want)
    assert not bad.any(), "%s: %d of %d off, first %s got %r want %r tol %r" % (
        what, int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist(), float(got[bad][0]), float(want[bad][0]),
        float(tol[bad][0] if torch.is_tensor(tol) else tol))


# ------------------------------------------------------------------ layouts
# (rows of each group, gaps before each group): empty groups, one row, tile
# borders (32, 64, 128, 256 and one more or less), groups that touch and that do not
LAYOUTS = {
    "one": ([1], [0]),
    "empty": ([0, 0, 0], [0, 0, 2]),
    "ragged": ([0, 33, 1, 0, 129, 64, 7], [0, 0, 3, 0, 5, 0, 1]),
    "tiles": ([256, 32, 257, 128, 31], [0, 1, 0, 0, 9]),
}


def layout(name):
    rows, gaps = LAYOUTS[name]
    begin, at = [], 0
    for n, gap in zip(rows, gaps):
        at += gap
        begin.append(at)
        at += n
    return rows, begin, at + 3


def groups_of(rows, begin):
    return miep.RowGroups(rows=i32(rows), begin=i32(begin))


def members(rows, begin, total):
    live = torch.zeros(total, dtype=torch.bool)
    for n, b in zip(rows, begin):
        live[b:b + n] = True
    return live


def poison(x, live):
    """NaN in every row that no group names."""
    x = x.clone()
    x[~live] = float("nan")
    return x


# ------------------------------------------------------------------ grouped product, bf16
SIZES = [(8, 8), (136, 64), (264, 200), (128, 1000)]      # (N, K): below a tile, odd, past K steps of 64


@pytest.mark.parametrize("expected", [1, 100, 100000])   # three of the tiles; every one below
@pytest.mark.parametrize("N,K", SIZES)
@pytest.mark.parametrize("name", list(LAYOUTS))
def test_grouped_gemm(name, N, K, expected):
    say("grouped_gemm", name, N, K, expected)
    rows, begin, total = layout(name)
    g = gen(N + K)
    live = members(rows, begin, total)
    x = poison(torch.randn((total, K), generator=g), live).to(BF)
    w = torch.randn((len(rows), N, K), generator=g).to(BF)
    y = torch.full((total, N), MARK, dtype=BF, device=DEV)
    miep.grouped_gemm_into(x.to(DEV), w.to(DEV), groups_of(rows, begin), y, expected_rows=expected)
    assert bool((y.cpu()[~live] == MARK).all())
    for i, (n, b) in enumerate(zip(rows, begin)):
        xs, ws = x[b:b + n].double(), w[i].double()
        want, mag = xs @ ws.T, xs.abs() @ ws.abs().T
        close(y[b:b + n], want, BF_HALF * want.abs() + K * ULP * mag, "group %d" % i)


@pytest.mark.parametrize("expected", [1, 100, 100000])
@pytest.mark.parametrize("N,K", [(136, 72), (264, 128)])
def test_grouped_gemm_gathers_rows(N, K, expected):
    say("gather", N, K, expected)
    rows, begin, total = layout("ragged")
    g = gen(7)
    src = 41
    x = torch.randn((src, K), generator=g).to(BF)
    w = torch.randn((len(rows), N, K), generator=g).to(BF)
    index = torch.randint(0, src, (total,), generator=g, dtype=torch.int32)
    index[::5] = -1                                        # no source: zeros
    index[2::11] = src                                     # past the source: zeros as well
    index[3::13] = index[4::13][:index[3::13].numel()] if index[4::13].numel() >= index[3::13].numel() else 0
    y = torch.full((total, N), MARK, dtype=BF, device=DEV)
    miep.grouped_gemm_into(x.to(DEV), w.to(DEV), groups_of(rows, begin), y, row_index=index.to(DEV), expected_rows=expected)
    live = members(rows, begin, total)
    assert bool((y.cpu()[~live] == MARK).all())
    for i, (n, b) in enumerate(zip(rows, begin)):
        at = index[b:b + n].long()
        ok = ((at >= 0) & (at < src)).unsqueeze(1)
        xs, ws = torch.where(ok, x[at.clamp(0, src - 1)].double(), 0.0), w[i].double()
        want, mag = xs @ ws.T, xs.abs() @ ws.abs().T
        close(y[b:b + n], want, BF_HALF * want.abs() + K * ULP * mag, "group %d" % i)


def test_grouped_gemm_of_an_empty_source_is_zero():
    index = torch.full((5,), -1, dtype=torch.int32, device=DEV)
    y = miep.grouped_gemm(torch.empty((0, 64), dtype=BF, device=DEV), torch.ones((2, 16, 64), dtype=BF, device=DEV),
                          groups_of([2, 3], [0, 2]), row_index=index)
    assert y.shape == (5, 16) and not y.any()


def test_nan_and_infinity_stay_in_their_rows():
    g = gen(3)
    x = torch.randn((40, 96), generator=g)
    x[3, 5], x[17, 95], x[17, 0] = float("nan"), float("inf"), float("inf")
    x = x.to(BF)
    w = torch.rand((1, 40, 96), generator=g).to(BF) + 0.5
    y = miep.grouped_gemm(x.to(DEV), w.to(DEV), groups_of([40], [0])).cpu()
    assert y[3].isnan().all() and (y[17] == float("inf")).all()
    rest = [i for i in range(40) if i not in (3, 17)]
    assert y[rest].isfinite().all()


@pytest.mark.parametrize("expected", [1, 100, 100000])
def test_low_latency_blocks_and_wrong_counts(expected):
    """Blocks of a fixed stride; counts past the block, negative ones and begins outside the layout stay inside it."""
    G, stride, N, K = 4, 70, 72, 136
    g = gen(11)
    x = torch.randn((G, stride, K), generator=g).to(BF)
    w = torch.randn((G, N, K), generator=g).to(BF)
    counts = [70, 0, -5, 200]
    y = torch.full((G, stride, N), MARK, dtype=BF, device=DEV)
    miep.grouped_gemm_into(x.to(DEV), w.to(DEV), miep.RowGroups(rows=i32(counts), stride=stride), y, expected_rows=expected)
    for i, n in enumerate([70, 0, 0, 70]):
        want, mag = x[i, :n].double() @ w[i].double().T, x[i, :n].double().abs() @ w[i].double().abs().T
        close(y[i, :n], want, BF_HALF * want.abs() + K * ULP * mag, "block %d" % i)
        assert bool((y[i, n:].cpu() == MARK).all())
    y = torch.full((G * stride, N), MARK, dtype=BF, device=DEV)
    far = groups_of([10, 10, 2 ** 31 - 1, 5], [-3, G * stride, G * stride - 2, 2 ** 31 - 1])
    miep.grouped_gemm_into(x.view(-1, K).to(DEV), w.to(DEV), far, y, expected_rows=expected)
    assert bool((y.cpu()[:-2] == MARK).all()) and bool((y.cpu()[-2:] != MARK).any())


@pytest.mark.parametrize("expected", [1, 100, 100000])
@pytest.mark.parametrize("N,K", [(8, 8), (72, 136), (200, 264), (1000, 128)])
@pytest.mark.parametrize("name", list(LAYOUTS))
def test_grouped_gemm_dgrad(name, N, K, expected):
    say("dgrad", name, N, K, expected)
    rows, begin, total = layout(name)
    g = gen(N * K)
    live = members(rows, begin, total)
    dy = poison(torch.randn((total, N), generator=g), live).to(BF)
    w = torch.randn((len(rows), N, K), generator=g).to(BF)
    dx = torch.full((total, K), MARK, dtype=BF, device=DEV)
    miep.grouped_gemm_dgrad_into(dy.to(DEV), w.to(DEV), groups_of(rows, begin), dx, expected_rows=expected)
    assert bool((dx.cpu()[~live] == MARK).all())
    for i, (n, b) in enumerate(zip(rows, begin)):
        ds, ws = dy[b:b + n].double(), w[i].double()
        want, mag = ds @ ws, ds.abs() @ ws.abs()
        close(dx[b:b + n], want, BF_HALF * want.abs() + N * ULP * mag, "group %d" % i)


def _wgrad_want(dy, x, rows, begin, index=None):
    want, mag = [], []
    for n, b in zip(rows, begin):
        ds = dy[b:b + n].double()
        if index is None:
            xs = x[b:b + n].double()
        else:
            at = index[b:b + n].long()
            ok = ((at >= 0) & (at < x.shape[0])).unsqueeze(1)
            xs = torch.where(ok, x[at.clamp(0, x.shape[0] - 1)].double(), 0.0)
        want.append(ds.T @ xs)
        mag.append(ds.abs().T @ xs.abs())
    return torch.stack(want), torch.stack(mag)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("N,K", [(8, 8), (72, 136), (200, 264), (384, 128)])
@pytest.mark.parametrize("name", list(LAYOUTS))
def test_grouped_gemm_wgrad(name, N, K, gather):
    say("wgrad", name, N, K, gather)
    rows, begin, total = layout(name)
    g = gen(N + 3 * K)
    live = members(rows, begin, total)
    dy = poison(torch.randn((total, N), generator=g), live).to(BF)
    index = None
    if gather:
        x = torch.randn((50, K), generator=g).to(BF)
        index = torch.randint(-1, 51, (total,), generator=g, dtype=torch.int32)
    else:
        x = poison(torch.randn((total, K), generator=g), live).to(BF)
    want, mag = _wgrad_want(dy, x, rows, begin, index)
    grp, most = groups_of(rows, begin), max(rows)
    kw = dict(row_index=index.to(DEV)) if gather else {}
    dw = miep.grouped_gemm_wgrad(dy.to(DEV), x.to(DEV), grp, **kw)
    close(dw, want, (most + 1) * ULP * mag, "fp32")
    half = miep.grouped_gemm_wgrad(dy.to(DEV), x.to(DEV), grp, dtype=BF, **kw)
    close(half, want, BF_HALF * want.abs() + (most + 1) * ULP * mag * 2, "bf16")
    old = torch.randn(want.shape, generator=g)
    acc = old.to(DEV)
    miep.grouped_gemm_wgrad_into(dy.to(DEV), x.to(DEV), grp, acc, accumulate=True, **kw)
    close(acc, want + old.double(), (most + 2) * ULP * (mag + old.double().abs()), "accumulated")


@pytest.mark.parametrize("expected", [1, 100, 100000])
@pytest.mark.parametrize("K", [64, 3200])                 # steps in order, and split over wavefronts
def test_groups_that_overlap(K, expected):
    """Five groups over the same rows and one behind them: far more tiles than the layout's rows make."""
    say("overlap", K, expected)
    rows, begin, total, N = [200] * 5 + [33], [0] * 5 + [200], 240, 136
    g = gen(21)
    grp = groups_of(rows, begin)
    x, w = torch.randn((total, K), generator=g).to(BF), torch.randn((6, N, K), generator=g).to(BF)
    dy = torch.randn((total, N), generator=g).to(BF)
    y, dx = torch.full((total, N), MARK, dtype=BF, device=DEV), torch.full((total, K), MARK, dtype=BF, device=DEV)
    miep.grouped_gemm_into(x.to(DEV), w.to(DEV), grp, y, expected_rows=expected)
    miep.grouped_gemm_dgrad_into(dy.to(DEV), w.to(DEV), grp, dx, expected_rows=expected)
    for out, a, b, depth in ((y, x, w.transpose(1, 2), K), (dx, dy, w, N)):
        a, b = a.double(), b.double()
        assert bool((out[233:] == MARK).all())
        got = d64(out)
        fits = torch.zeros((200, out.shape[1]), dtype=torch.bool)
        for i in range(5):                                 # a shared row holds, place by place, one group's result
            want, mag = a[:200] @ b[i], a[:200].abs() @ b[i].abs()
            fits |= (got[:200] - want).abs() <= BF_HALF * want.abs() + depth * ULP * mag
        assert bool(fits.all())
        want, mag = a[200:233] @ b[5], a[200:233].abs() @ b[5].abs()
        close(out[200:233], want, BF_HALF * want.abs() + depth * ULP * mag)
    dw = miep.grouped_gemm_wgrad(dy.to(DEV), x.to(DEV), grp)
    want, mag = _wgrad_want(dy, x, rows, begin)
    close(dw, want, 201 * ULP * mag)
    h = _h(total, K, g)
    act = torch.full((total, K), MARK, dtype=BF, device=DEV)
    miep.swiglu_into(h.to(DEV), grp, act)
    want = swiglu64(h[:233])
    gate, up = factors(h[:233])
    close(act[:233], want, (BF_HALF + SIG) * want.abs() + TINY * (1 + gate * up))
    assert bool((act[233:] == MARK).all())


def test_layouts_without_rows():
    """No rows at all: outputs of no rows, weight gradients of zeros, or what they held."""
    grp = groups_of([3, 0], [0, 0])                        # counts that the layout does not hold
    x, w = torch.empty((0, 64), dtype=BF, device=DEV), torch.ones((2, 16, 64), dtype=BF, device=DEV)
    dy = torch.empty((0, 16), dtype=BF, device=DEV)
    assert miep.grouped_gemm(x, w, grp).shape == (0, 16) and miep.grouped_gemm_dgrad(dy, w, grp).shape == (0, 64)
    assert miep.swiglu(x, grp).shape == (0, 32) and miep.swiglu_backward(x[:, :32].contiguous(), x, grp).shape == (0, 64)
    assert not miep.grouped_gemm_wgrad(dy, x, grp).any()
    kept = torch.ones((2, 16, 64), device=DEV)
    miep.grouped_gemm_wgrad_into(dy, x, grp, kept, accumulate=True)
    assert bool((kept == 1).all())
    none = groups_of([], [])
    assert miep.grouped_gemm_wgrad(dy, x, none).shape == (0, 16, 64)
    y = torch.full((4, 16), MARK, dtype=BF, device=DEV)
    miep.grouped_gemm_into(torch.ones((4, 64), dtype=BF, device=DEV), w[:0], none, y)
    assert bool((y == MARK).all())


@pytest.mark.parametrize("expected", [1, 100, 100000])
def test_more_groups_than_lanes(expected):
    """150 groups, most of them empty: the walk over groups passes several blocks of 64."""
    rows = [(i * 7) % 40 if i % 3 == 0 else 0 for i in range(150)]
    begin = np.cumsum([0] + rows[:-1]).tolist()
    total, N, K = sum(rows), 72, 40
    g = gen(12)
    x, w = torch.randn((total, K), generator=g).to(BF), torch.randn((150, N, K), generator=g).to(BF)
    dy, h = torch.randn((total, N), generator=g).to(BF), torch.randn((total, 2 * K), generator=g).to(BF)
    grp = groups_of(rows, begin)
    y, dw = miep.grouped_gemm(x.to(DEV), w.to(DEV), grp, expected_rows=expected), miep.grouped_gemm_wgrad(dy.to(DEV), x.to(DEV), grp)
    a = miep.swiglu(h.to(DEV), grp)
    for i, (n, b) in enumerate(zip(rows, begin)):
        xs, ws = x[b:b + n].double(), w[i].double()
        close(y[b:b + n], xs @ ws.T, BF_HALF * (xs @ ws.T).abs() + K * ULP * (xs.abs() @ ws.abs().T), "group %d" % i)
        d = dy[b:b + n].double()
        close(dw[i], d.T @ xs, 41 * ULP * (d.abs().T @ xs.abs()))
    want = swiglu64(h)
    close(a, want, (BF_HALF + SIG) * want.abs() + TINY * (1 + factors(h)[0] * factors(h)[1]))


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("most", [70, 400])
def test_wgrad_large_tiles(most, gather):
    """Enough tiles for the large tile: 64 groups of up to ``most`` rows, 264 x 272 weights (edges in both)."""
    rows = [(37 * i) % most for i in range(64)]
    begin = np.cumsum([0] + rows[:-1]).tolist()
    total, N, K = sum(rows), 264, 272
    g = gen(5)
    dy = torch.randn((total, N), generator=g).to(BF)
    x = torch.randn((total, K), generator=g).to(BF)
    index = torch.randperm(total, generator=g).to(torch.int32) if gather else None
    want, mag = _wgrad_want(dy, x, rows, begin, index)
    dw = miep.grouped_gemm_wgrad(dy.to(DEV), x.to(DEV), groups_of(rows, begin),
                                 row_index=index.to(DEV) if gather else None)
    close(dw, want, (most + 1) * ULP * mag)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("N,K", [(8, 8), (136, 72), (192, 520)])
def test_wgrad_of_many_rows(N, K, gather):
    """Many rows under few tiles: the rows are split over wavefronts; groups of none, one, a few and many steps."""
    say("wgrad split", N, K, gather)
    rows = [0, 2600, 1, 33, 0, 1217]
    begin = np.cumsum([0] + rows[:-1]).tolist()
    total = sum(rows) + 5
    g = gen(N * K)
    dy = poison(torch.randn((total, N), generator=g), members(rows, begin, total)).to(BF)
    x = torch.randn((900, K) if gather else (total, K), generator=g).to(BF)
    index = torch.randint(-1, 901, (total,), generator=g, dtype=torch.int32) if gather else None
    want, mag = _wgrad_want(dy, x, rows, begin, index)
    grp, kw = groups_of(rows, begin), dict(row_index=index.to(DEV)) if gather else {}
    close(miep.grouped_gemm_wgrad(dy.to(DEV), x.to(DEV), grp, **kw), want, 2601 * ULP * mag)
    close(miep.grouped_gemm_wgrad(dy.to(DEV), x.to(DEV), grp, dtype=BF, **kw), want, BF_HALF * want.abs() + 2 * 2601 * ULP * mag)
    old = torch.randn(want.shape, generator=g)
    acc = old.to(DEV)
    miep.grouped_gemm_wgrad_into(dy.to(DEV), x.to(DEV), grp, acc, accumulate=True, **kw)
    close(acc, want + old.double(), 2602 * ULP * (mag + old.double().abs()))


def test_product_gradients_match_differences():
    """The formulas the gradients are held to, against central differences of the 64-bit product (linear: exact)."""
    g = gen(9)
    x, w, dy = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((5, 16), (8, 16), (5, 8)))
    h = 1e-3
    for t, grad in ((x, dy @ w), (w, dy.T @ x)):
        for at in ((0, 0), (3, 7), (4, 15)):
            d = torch.zeros_like(t)
            d[at] = h
            up = (x + d if t is x else x) @ (w + d if t is w else w).T
            dn = (x - d if t is x else x) @ (w - d if t is w else w).T
            assert abs(float(((up - dn) * dy).sum() / (2 * h) - grad[at])) < 1e-9
    dx = miep.grouped_gemm_dgrad(dy.to(BF).to(DEV), w.to(BF).unsqueeze(0).to(DEV), groups_of([5], [0]))
    a, b = dy.to(BF).double(), w.to(BF).double()
    close(dx, a @ b, BF_HALF * (a @ b).abs() + 8 * ULP * (a.abs() @ b.abs()))


# ------------------------------------------------------------------ FP8 product
def quant_rows(x, pow2):
    v = x.view(x.shape[0], -1, 128)
    s = v.abs().amax(2).clamp_min(1e-4) / 448
    s = torch.exp2(torch.ceil(torch.log2(s))) if pow2 else s
    return (v / s.unsqueeze(2)).to(F8).view(x.shape), s


def quant_blocks(w, pow2):
    G, N, K = w.shape
    nb = -(-N // 128)
    p = torch.zeros((G, nb * 128, K))
    p[:, :N] = w
    v = p.view(G, nb, 128, K // 128, 128)
    s = v.abs().amax((2, 4)).clamp_min(1e-4) / 448
    s = torch.exp2(torch.ceil(torch.log2(s))) if pow2 else s
    return (v / s.view(G, nb, 1, K // 128, 1)).to(F8).view(G, nb * 128, K)[:, :N].contiguous(), s


def expand_x(x, s):
    return x.to(torch.float32).double() * s.double().repeat_interleave(128, 1)


def expand_w(w, s):
    f = s.double().repeat_interleave(128, 0)[:w.shape[0]].repeat_interleave(128, 1)
    return w.to(torch.float32).double() * f


def fp8_tol(want, mag, K):
    # K additions, and per 128-block a product of two scales and one with the block's sum (3 half ulps)
    return BF_HALF * want.abs() + (K + K // 128 + 3) * ULP * mag


@pytest.mark.parametrize("expected", [1, 100, 100000])
@pytest.mark.parametrize("ue8m0", [False, True])
@pytest.mark.parametrize("N,K,gather", [(8, 128, False), (200, 384, False), (392, 256, True), (128, 1152, False)])
@pytest.mark.parametrize("name", ["one", "ragged", "tiles"])
def test_grouped_gemm_fp8(name, N, K, gather, ue8m0, expected):
    say("fp8", name, N, K, gather, ue8m0, expected)
    rows, begin, total = layout(name)
    g = gen(N + K)
    src = 37 if gather else total
    # rows and blocks of very different sizes: a scale of the wrong row or block is far off
    x, xs = quant_rows(torch.randn((src, K), generator=g) * torch.exp2(torch.randint(-6, 7, (src, 1), generator=g).float()), ue8m0)
    w, ws = quant_blocks(torch.randn((len(rows), N, K), generator=g) *
                         torch.exp2(torch.randint(-4, 5, (len(rows), 1, K // 128), generator=g).float()).repeat_interleave(128, 2), ue8m0)
    index = None
    live = members(rows, begin, total)
    if gather:
        index = torch.randint(-1, src + 1, (total,), generator=g, dtype=torch.int32)
    else:
        x.view(torch.uint8)[~live] = 0x7F                  # NaN codes and scales where no group reads
        xs[~live] = float("nan")
    byte = (lambda s: (torch.log2(s.nan_to_num(1.0)) + 127).to(torch.uint8)) if ue8m0 else (lambda s: s)
    y = torch.full((total, N), MARK, dtype=BF, device=DEV)
    miep.grouped_gemm_fp8_into(x.to(DEV), byte(xs).to(DEV), w.to(DEV), byte(ws).to(DEV), groups_of(rows, begin), y,
                               row_index=index.to(DEV) if gather else None, expected_rows=expected)
    assert bool((y.cpu()[~live] == MARK).all())
    xd = expand_x(x, xs)
    for i, (n, b) in enumerate(zip(rows, begin)):
        at = index[b:b + n].long() if gather else torch.arange(b, b + n)
        ok = ((at >= 0) & (at < src)).unsqueeze(1)
        a, c = torch.where(ok, xd[at.clamp(0, src - 1)], 0.0), expand_w(w[i], ws[i])
        want, mag = a @ c.T, a.abs() @ c.abs().T
        close(y[b:b + n], want, fp8_tol(want, mag, K), "group %d" % i)


KINDS = ["gemm", "gather", "dgrad", "fp8", "fp8 gather", "ue8m0", "ue8m0 gather"]


def check_product(kind, rows, N, K, expected):
    """Groups of these rows with gaps between them, N output channels, contractions of K."""
    G = len(rows)
    begin = np.cumsum([0] + [n + i % 3 for i, n in enumerate(rows)][:-1]).tolist()
    total = begin[-1] + rows[-1] + 2
    g, live, grp = gen(expected), members(rows, begin, total), groups_of(rows, begin)
    gather = "gather" in kind
    src = 500 if gather else total
    index = torch.randint(-1, src, (total,), generator=g, dtype=torch.int32) if gather else None
    kw = dict(row_index=index.to(DEV)) if gather else {}
    y = torch.full((total, N), MARK, dtype=BF, device=DEV)
    if kind in ("gemm", "gather", "dgrad"):
        x = torch.randn((src, K), generator=g).to(BF)
        w = torch.randn((G, K, N) if kind == "dgrad" else (G, N, K), generator=g).to(BF)
        if kind == "dgrad":
            miep.grouped_gemm_dgrad_into(x.to(DEV), w.to(DEV), grp, y, expected_rows=expected)
        else:
            miep.grouped_gemm_into(x.to(DEV), w.to(DEV), grp, y, expected_rows=expected, **kw)
        xd, wd = x.double(), [(t if kind == "dgrad" else t.T).double() for t in w]
    else:
        pow2 = "ue8m0" in kind
        x, xs = quant_rows(torch.randn((src, K), generator=g), pow2)
        w, ws = quant_blocks(torch.randn((G, N, K), generator=g), pow2)
        byte = (lambda s: (torch.log2(s) + 127).to(torch.uint8)) if pow2 else (lambda s: s)
        miep.grouped_gemm_fp8_into(x.to(DEV), byte(xs).to(DEV), w.to(DEV), byte(ws).to(DEV), grp, y, expected_rows=expected, **kw)
        xd, wd = expand_x(x, xs), [expand_w(w[i], ws[i]).T for i in range(G)]
    y = y.cpu()
    assert bool((y[~live] == MARK).all())
    for i, (n, b) in enumerate(zip(rows, begin)):
        a = xd[b:b + n]
        if gather:
            at = index[b:b + n].long()
            a = torch.where((at >= 0).unsqueeze(1), xd[at.clamp_min(0)], 0.0)
        want, mag = a @ wd[i], a.abs() @ wd[i].abs()
        close(y[b:b + n], want, fp8_tol(want, mag, K), "group %d" % i)


# 64 groups of 0 to 329 rows under 264 output channels: with these expectations every tile but 256 x 256 is taken in turn
@pytest.mark.parametrize("expected", [1, 60, 130, 190, 300, 1000])
@pytest.mark.parametrize("kind", KINDS)
def test_every_tile(kind, expected):
    say("every tile", kind, expected)
    check_product(kind, [(53 * i) % 330 if i % 9 else 0 for i in range(64)], 264, 640 if "8" in kind else 520, expected)


# More tiles of 256 channels than workgroups, some whole and some short: of 256 rows, and of 192
@pytest.mark.parametrize("most", [256, 192])
@pytest.mark.parametrize("kind", KINDS)
def test_rounds_of_wide_tiles(kind, most):
    say("wide tiles", kind, most)
    check_product(kind, [most - i % 7 for i in range(70)], 1040, 384 if "8" in kind else 264, 256)


@pytest.mark.parametrize("rows", [[1], [0, 33, 5], [70, 0, 1, 32]])
@pytest.mark.parametrize("kind", ["gemm", "gather", "dgrad", "fp8", "fp8 gather", "ue8m0", "ue8m0 gather"])
def test_few_tiles_over_a_long_contraction(kind, rows):
    """The contraction split over wavefronts: more than 24 steps of it, the last one short where the type allows."""
    say("split", kind, rows)
    begin = np.cumsum([1] + [n + 2 for n in rows])[:-1].tolist()
    total, G, N = begin[-1] + rows[-1] + 3, len(rows), 72
    g, live, grp = gen(len(kind)), members(rows, begin, total), groups_of(rows, begin)
    gather = "gather" in kind
    src = 50 if gather else total
    index = torch.randint(-1, src + 1, (total,), generator=g, dtype=torch.int32) if gather else None
    kw = dict(row_index=index.to(DEV)) if gather else {}
    y = torch.full((total, N), MARK, dtype=BF, device=DEV)
    if kind in ("gemm", "gather", "dgrad"):
        K = 1608
        x = torch.randn((src, K), generator=g)
        x = (x if gather else poison(x, live)).to(BF)
        w = torch.randn((G, K, N) if kind == "dgrad" else (G, N, K), generator=g).to(BF)
        if kind == "dgrad":
            miep.grouped_gemm_dgrad_into(x.to(DEV), w.to(DEV), grp, y, expected_rows=4)
        else:
            miep.grouped_gemm_into(x.to(DEV), w.to(DEV), grp, y, expected_rows=4, **kw)
        xd, wd = x.double(), [(t if kind == "dgrad" else t.T).double() for t in w]
    else:
        K, pow2 = 3200, "ue8m0" in kind
        x, xs = quant_rows(torch.randn((src, K), generator=g), pow2)
        w, ws = quant_blocks(torch.randn((G, N, K), generator=g), pow2)
        byte = (lambda s: (torch.log2(s) + 127).to(torch.uint8)) if pow2 else (lambda s: s)
        miep.grouped_gemm_fp8_into(x.to(DEV), byte(xs).to(DEV), w.to(DEV), byte(ws).to(DEV), grp, y, expected_rows=4, **kw)
        xd, wd = expand_x(x, xs), [expand_w(w[i], ws[i]).T for i in range(G)]
    y = y.cpu()
    assert bool((y[~live] == MARK).all())
    for i, (n, b) in enumerate(zip(rows, begin)):
        a = xd[b:b + n] if not gather else torch.where(((index[b:b + n] >= 0) & (index[b:b + n] < src)).unsqueeze(1),
                                                       xd[index[b:b + n].long().clamp(0, src - 1)], 0.0)
        want, mag = a @ wd[i], a.abs() @ wd[i].abs()
        close(y[b:b + n], want, fp8_tol(want, mag, K), "group %d" % i)


def test_fp8_codes_as_bytes():
    """uint8 codes are the same call as float8_e4m3fn ones."""
    g = gen(1)
    x, xs = quant_rows(torch.randn((9, 128), generator=g), False)
    w, ws = quant_blocks(torch.randn((1, 16, 128), generator=g), False)
    args = [t.to(DEV) for t in (x, xs, w, ws)]
    grp = groups_of([9], [0])
    a = miep.grouped_gemm_fp8(*args, grp)
    b = miep.grouped_gemm_fp8(args[0].view(torch.uint8), args[1], args[2].view(torch.uint8), args[3], grp)
    assert torch.equal(a, b)


# ------------------------------------------------------------------ SwiGLU
def swiglu64(h):
    I = h.shape[-1] // 2
    gate, up = h[..., :I].double(), h[..., I:].double()
    return gate * torch.sigmoid(gate) * up


# fp32: sigmoid's exp is exact to about 3 ulps (range split, exp2, correction), its sum and
# reciprocal 2 more, the two products 1 each
SIG = 8 * ULP
# A sigmoid below fp32's smallest normal number, 2^-126 (gate < -87.3), is held as zero (the hardware's
# reciprocal has no subnormal results), an absolute error of up to 2^-126 in s that gate * up (and the
# gradient's factors of s) multiply; a result below 2^-126 itself may be flushed as well.
TINY = 2.0 ** -126


def factors(h):
    I = h.shape[-1] // 2
    return h[..., :I].double().abs(), h[..., I:].double().abs()


def _h(total, I, g):
    h = torch.randn((total, 2 * I), generator=g) * 3
    h[:, 0] = torch.linspace(-120, 120, total)             # gates where exp overflows and underflows
    h[:, 1], h[:, 2] = 0.0, -0.0
    return h.to(BF)


@pytest.mark.parametrize("I", [8, 136, 640])
@pytest.mark.parametrize("name", list(LAYOUTS))
def test_swiglu(name, I):
    say("swiglu", name, I)
    rows, begin, total = layout(name)
    live = members(rows, begin, total)
    h = poison(_h(total, I, gen(I)), live)
    a = torch.full((total, I), MARK, dtype=BF, device=DEV)
    miep.swiglu_into(h.to(DEV), groups_of(rows, begin), a)
    assert bool((a.cpu()[~live] == MARK).all())
    want = swiglu64(h[live])
    gate, up = factors(h[live])
    close(a[live.to(DEV)], want, (BF_HALF + SIG) * want.abs() + TINY * (1 + gate * up))


@pytest.mark.parametrize("round_scale,ue", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("I", [128, 640])
@pytest.mark.parametrize("name", list(LAYOUTS))
def test_swiglu_fp8(name, I, round_scale, ue):
    say("swiglu_fp8", name, I, round_scale, ue)
    rows, begin, total = layout(name)
    live = members(rows, begin, total)
    h = _h(total, I, gen(I))
    h[total // 2] = 0                                      # a row of zeros: the floor of the scale
    h = poison(h, live)
    a = torch.full((total, I), 0x5A, dtype=torch.uint8, device=DEV)
    s = torch.full((total, I // 128), MARK, device=DEV)
    u = torch.full((total, I // 128), 9, dtype=torch.uint8, device=DEV) if ue else None
    miep.swiglu_fp8_into(h.to(DEV), groups_of(rows, begin), a, s, round_scale=round_scale, a_scales_ue8m0=u)
    a, s = a.cpu(), s.cpu()
    assert bool((a[~live] == 0x5A).all()) and bool((s[~live] == MARK).all())
    if not live.any():
        return
    want = swiglu64(h[live])
    top = want.view(want.shape[0], -1, 128).abs().amax(2).clamp_min(1e-4) / 448
    got = s[live].double()
    if round_scale:
        assert torch.equal(torch.log2(got), torch.log2(got).round())
        assert bool((got >= top * (1 - 16 * ULP)).all()) and bool((got < 2 * top * (1 + 16 * ULP)).all())
        if ue:
            assert torch.equal(u.cpu()[live].double(), torch.log2(got) + 127) and bool((u.cpu()[~live] == 9).all())
    else:
        close(got, top, 16 * ULP * top)
    val = a[live].view(F8).float().double() * got.repeat_interleave(128, 1)
    # half a step of the code, 2^-10 absolute below E4M3's smallest normal, in units of the scale
    close(val, want, F8_HALF * want.abs() * (1 + 1e-5) + 2.0 ** -10 * got.repeat_interleave(128, 1) + SIG * want.abs())


@pytest.mark.parametrize("I", [8, 136, 640])
@pytest.mark.parametrize("name", list(LAYOUTS))
def test_swiglu_backward(name, I):
    say("swiglu_backward", name, I)
    rows, begin, total = layout(name)
    live = members(rows, begin, total)
    g = gen(I)
    h, da = poison(_h(total, I, g), live), poison(torch.randn((total, I), generator=g), live).to(BF)
    dh = torch.full((total, 2 * I), MARK, dtype=BF, device=DEV)
    miep.swiglu_backward_into(da.to(DEV), h.to(DEV), groups_of(rows, begin), dh)
    assert bool((dh.cpu()[~live] == MARK).all())
    hd = h[live].double()
    gate, up, d = hd[:, :I], hd[:, I:], da[live].double()
    s = torch.sigmoid(gate)
    dgate, dup = d * up * s * (1 + gate * (1 - s)), d * gate * s
    got = dh[live.to(DEV)]
    # 1 + g (1 - s) cancels near g = -1.28: its absolute error is an ulp of 1 and 3 of g (1 - s) <= |g| + 1
    slack = d.abs() * up.abs() * s * (2 + gate.abs()) * SIG
    close(got[:, :I], dgate, BF_HALF * dgate.abs() + slack + TINY * (1 + d.abs() * up.abs() * (1 + gate.abs())), "gate")
    close(got[:, I:], dup, (BF_HALF + SIG) * dup.abs() + TINY * (1 + d.abs() * gate.abs()), "up")
    if live.any():                                         # the formula against central differences in 64 bits
        e = 1e-5
        num = (swiglu64(torch.cat([gate + e, up], 1)) - swiglu64(torch.cat([gate - e, up], 1))) / (2 * e) * d
        assert bool(((num - dgate).abs() <= 1e-8 * (1 + d.abs() * up.abs() * (1 + gate.abs()))).all())
        num = (swiglu64(torch.cat([gate, up + e], 1)) - swiglu64(torch.cat([gate, up - e], 1))) / (2 * e) * d
        assert bool(((num - dup).abs() <= 1e-8 * (1 + d.abs() * gate.abs() * (1 + up.abs()))).all())


def test_swiglu_backward_in_place():
    rows, begin, total = layout("ragged")
    g = gen(9)
    h, da = _h(total, 136, g).to(DEV), torch.randn((total, 136), generator=g).to(BF).to(DEV)
    want = h.clone()
    miep.swiglu_backward_into(da, h, groups_of(rows, begin), want)
    miep.swiglu_backward_into(da, h, groups_of(rows, begin), h)
    assert torch.equal(h, want)


def test_swiglu_of_infinities_and_nan():
    inf = float("inf")
    h = torch.zeros((1, 16))
    h[0, :5] = torch.tensor([inf, float("nan"), 2.0, 2.0, -500.0])
    h[0, 8:13] = torch.tensor([1.0, 1.0, inf, float("nan"), 1.0])
    a = miep.swiglu(h.to(BF).to(DEV), groups_of([1], [0])).cpu()[0]
    assert a[0] == inf and a[1].isnan() and a[2] == inf and a[3].isnan() and a[4] == 0 and not a[5:].any()


# ------------------------------------------------------------------ expert order
def order_want(topk, off, E, align, slots):
    topk = topk.numpy()
    cap, K = topk.shape
    R = len(off) - 1
    L = E // R
    lists = [[] for _ in range(E)]
    for r in range(R):
        for row in range(min(off[r], cap), min(off[r + 1], cap)):
            for k in range(K):
                if 0 <= topk[row, k] < L:
                    lists[r * L + topk[row, k]].append((row, k))
    begin, count = [], []
    slot_row, row_slot = np.full(slots, -1, np.int32), np.full((cap, K), -1, np.int32)
    at = 0
    for e in range(E):
        begin.append(at)
        count.append(len(lists[e]))
        for j, (row, k) in enumerate(lists[e]):
            if at + j < slots:
                slot_row[at + j] = row
                row_slot[row, k] = at + j
        at += -(-len(lists[e]) // align) * align
    return np.array(begin), np.array(count), slot_row, row_slot, at


def received(R, L, K, per_rank, cap, g, dead=0.3):
    """Received rows: every row names at least one local expert; some name one twice; the rest is -1 (or junk >= L)."""
    off = np.concatenate([[0], np.cumsum(per_rank)]).tolist()
    topk = torch.randint(0, L, (cap, K), generator=g)
    mask = torch.rand((cap, K), generator=g) < dead
    mask[:, 0] = False
    topk[mask] = -1
    topk[1::17, K - 1] = L + 3
    if K > 1:
        topk[::9, 1] = topk[::9, 0]
    return topk, off


@pytest.mark.parametrize("R,L,K,per_rank,spare,align,parts", [
    (1, 1, 1, [1], 0, 1, 1),
    (1, 8, 8, [300], 7, 1, 256),
    (1, 300, 3, [2000], 0, 16, 64),
    (4, 5, 8, [0, 130, 1, 64], 9, 8, 64),
    (8, 32, 8, [500] * 8, 0, 128, 32),
    (2, 2048, 2, [900, 5000], 3, 1, 128),
    (64, 4, 8, [17 * (i % 5) for i in range(64)], 40, 4, 4),
    (3, 64, 64, [0, 0, 333], 2, 1, 7),
    (2, 7, 4, [0, 0], 3, 1, 1),
    (2, 8, 4, [500, 524], 0, 1, 128),
    (2, 8, 4, [500, 525], 0, 1, 128),
    (16, 128, 2, [0, 9, 0, 0, 100] + [7] * 9 + [0, 0], 4, 8, 16),
])
def test_expert_order(R, L, K, per_rank, spare, align, parts):
    say("order", R, L, K, align, parts)
    cap, E = sum(per_rank) + spare, R * L
    topk, off = received(R, L, K, per_rank, cap, gen(R * L * K))
    order = miep.ExpertOrder.allocate(topk.to(DEV), i32(off), E, align)
    order.workspace = torch.full((parts, E), -9, dtype=torch.int32, device=DEV)
    for t in (order.group_begin, order.group_rows, order.slot_row, order.row_slot):
        t.fill_(-99)
    status = i32([-1])
    miep.expert_order_into(topk.to(DEV), order, align, status)
    begin, count, slot_row, row_slot, used = order_want(topk, off, E, align, order.num_slots)
    assert used <= order.num_slots
    assert np.array_equal(order.group_begin.cpu().numpy(), begin)
    assert np.array_equal(order.group_rows.cpu().numpy(), count)
    assert np.array_equal(order.slot_row.cpu().numpy(), slot_row)
    assert np.array_equal(order.row_slot.cpu().numpy(), row_slot)
    miep.check_status(status)


def test_expert_order_reports_too_few_slots():
    topk, off = received(2, 4, 4, [40, 30], 75, gen(2))
    need = order_want(topk, off, 8, 8, 10 ** 4)[4]
    for slots in (need, need - 9, 0):
        order = miep.ExpertOrder.allocate(topk.to(DEV), i32(off), 8, 8)
        order.slot_row = torch.full((slots,), -99, dtype=torch.int32, device=DEV)
        status = i32([0])
        miep.expert_order_into(topk.to(DEV), order, 8, status)
        _, _, slot_row, row_slot, _ = order_want(topk, off, 8, 8, slots)
        assert np.array_equal(order.slot_row.cpu().numpy(), slot_row)
        assert np.array_equal(order.row_slot.cpu().numpy(), row_slot)
        assert int(status) == (0 if slots >= need else miep.MIEP_ECAPACITY)


def test_expert_order_of_overflowed_receive_rows():
    """recv_rank_offset past the allocated rows (a dispatch that overflowed) reads only the rows there are."""
    topk, off = received(2, 4, 4, [40, 30], 50, gen(2))
    order = miep.expert_order(topk.to(DEV), i32(off), 8)
    begin, count, slot_row, row_slot, _ = order_want(topk, off, 8, 1, order.num_slots)
    assert np.array_equal(order.group_rows.cpu().numpy(), count)
    assert np.array_equal(order.row_slot.cpu().numpy(), row_slot)


def test_expert_order_of_offsets_out_of_order():
    """Offsets that no dispatch writes: whatever they hold, only the arrays' own places are written."""
    topk, _ = received(4, 3, 4, [20, 20, 20, 20], 80, gen(4))
    room = torch.full((3, 400), -99, dtype=torch.int32, device=DEV)
    for off in ([60, 0, 80, -7, 30], [2 ** 31 - 1, -2 ** 31, 5, 99, 0], [0, 80, 0, 80, 0]):
        room.fill_(-99)
        order = miep.ExpertOrder.allocate(topk.to(DEV), i32(off), 12, 4, 100)
        order.slot_row, order.row_slot = room[0, 150:250], room[2, 40:360].view(80, 4)
        miep.expert_order_into(topk.to(DEV), order, 4)
        assert bool((room[1] == -99).all()) and bool((room[0, :150] == -99).all()) and bool((room[0, 250:] == -99).all())
        assert bool((room[2, :40] == -99).all()) and bool((room[2, 360:] == -99).all())
        assert bool((order.slot_row >= -1).all()) and bool((order.slot_row < 80).all())
        assert bool((order.row_slot >= -1 - 98).all()) and bool((order.row_slot < 100).all())


@pytest.mark.parametrize("H,K,weighted", [(8, 1, True), (136, 8, True), (2056, 8, False), (264, 20, True), (7168, 3, True)])
def test_expert_reduce_and_backward(H, K, weighted):
    say("reduce", H, K, weighted)
    R, L, per_rank = 2, 6, [45, 30]
    cap = sum(per_rank) + 5
    g = gen(H + K)
    topk, off = received(R, L, K, per_rank, cap, g)
    topk[3] = -1                                           # a row that no expert took
    order = miep.expert_order(topk.to(DEV), i32(off), R * L, 4)
    wts = torch.rand((cap, K), generator=g) if weighted else None
    wdev = wts.to(DEV) if weighted else None
    rs = order.row_slot.cpu().long()
    used = torch.zeros(order.num_slots, dtype=torch.bool)
    used[rs[rs >= 0]] = True
    z = torch.randn((order.num_slots, H), generator=g)
    z[~used] = float("nan")
    z = z.to(BF)
    y = torch.full((cap, H), MARK, dtype=BF, device=DEV)
    miep.expert_reduce_into(z.to(DEV), order, y, wdev)
    w64 = wts.double() if weighted else torch.ones((cap, K), dtype=torch.float64)
    zz = torch.where((rs >= 0).unsqueeze(2), z[rs.clamp_min(0)].double(), 0.0)
    want, mag = (zz * w64.unsqueeze(2)).sum(1), (zz.abs() * w64.unsqueeze(2)).sum(1)
    n = off[-1]
    close(y[:n], want[:n], BF_HALF * want[:n].abs() + (K + 1) * ULP * mag[:n])
    assert not y[3].any() and bool((y[n:].cpu() == MARK).all())

    dy = torch.randn((cap, H), generator=g).to(BF)
    dz = torch.full((order.num_slots, H), MARK, dtype=BF, device=DEV)
    dw = torch.full((cap, K), MARK, device=DEV) if weighted else None
    miep.expert_reduce_backward_into(dy.to(DEV), z.to(DEV), order, dz, wdev, dw)
    assert bool((dz.cpu()[~used] == MARK).all())
    row = order.slot_row.cpu().long()
    at = {int(s): (r, k) for r in range(cap) for k, s in enumerate(rs[r].tolist()) if s >= 0}
    slots = sorted(at)
    ww = torch.tensor([float(w64[at[s]]) for s in slots], dtype=torch.float64)
    want = dy[row[slots]].double() * ww.unsqueeze(1)
    close(dz[slots], want, (BF_HALF + ULP) * want.abs())
    if weighted:
        prod = zz[:n] * dy[:n].double().unsqueeze(1)
        close(dw[:n], prod.sum(2), (H + 8) * ULP * prod.abs().sum(2))
        assert bool((dw[n:].cpu() == MARK).all())
        # the weights' gradient against central differences of the 64-bit sum (linear: exact)
        e = torch.zeros_like(w64)
        e[5, 0] = 1e-3
        f = lambda v: float((zz * v.unsqueeze(2)).sum(1)[:n].mul(dy[:n].double()).sum())  # noqa: E731
        assert abs((f(w64 + e) - f(w64 - e)) / 2e-3 - float(prod.sum(2)[5, 0])) < 1e-6


# ------------------------------------------------------------------ results that pass the caches by (128 MiB and more)
def test_large_swiglu_and_its_gradient():
    rows, I = 8200, 8200
    g = torch.Generator(device=DEV).manual_seed(4)
    h = torch.randn((rows, 2 * I), generator=g, device=DEV).to(BF)
    da = torch.randn((rows, I), generator=g, device=DEV).to(BF)
    grp = groups_of([8000, 0, 150], [0, 9, 8010])
    a = torch.full((rows, I), MARK, dtype=BF, device=DEV)
    dh = torch.full((rows, 2 * I), MARK, dtype=BF, device=DEV)
    miep.swiglu_into(h, grp, a)
    miep.swiglu_backward_into(da, h, grp, dh)
    at = [0, 1, 77, 4095, 7999, 8010, 8159]
    want = swiglu64(h[at].cpu())
    gate, up = factors(h[at].cpu())
    close(a[at], want, (BF_HALF + SIG) * want.abs() + TINY * (1 + gate * up))
    hd, d = h[at].cpu().double(), da[at].cpu().double()
    s = torch.sigmoid(hd[:, :I])
    dup = d * hd[:, :I] * s
    close(dh[at][:, I:], dup, (BF_HALF + SIG) * dup.abs() + TINY * (1 + d.abs() * gate), "up")
    dgate = d * hd[:, I:] * s * (1 + hd[:, :I] * (1 - s))
    close(dh[at][:, :I], dgate, BF_HALF * dgate.abs() + d.abs() * up * s * (2 + gate) * SIG + TINY * (1 + d.abs() * up * (1 + gate)), "gate")
    out = [8000, 8009, 8160, 8199]
    assert bool((a[out] == MARK).all()) and bool((dh[out] == MARK).all())


def test_large_reduce_backward():
    cap, K, H = 4200, 4, 8200
    g = torch.Generator(device=DEV).manual_seed(6)
    topk = torch.randint(0, 8, (cap, K), generator=g, device=DEV)
    order = miep.expert_order(topk, i32([0, cap - 3]), 8)
    z = torch.randn((order.num_slots, H), generator=g, device=DEV).to(BF)
    dy = torch.randn((cap, H), generator=g, device=DEV).to(BF)
    w = torch.rand((cap, K), generator=g, device=DEV)
    dz, dw = torch.full_like(z, MARK), torch.full_like(w, MARK)
    miep.expert_reduce_backward_into(dy, z, order, dz, w, dw)
    rs = order.row_slot.cpu().long()
    for r in (0, 1, 2000, cap - 4):
        want = d64(dy[r]) * d64(w[r]).unsqueeze(1)
        close(dz[rs[r]], want, (BF_HALF + ULP) * want.abs())
        prod = d64(z[rs[r]]) * d64(dy[r])
        close(dw[r], prod.sum(1), (H + 8) * ULP * prod.abs().sum(1))
    assert bool((dw[cap - 3:] == MARK).all())


# ------------------------------------------------------------------ offsets past 32 bits
def test_rows_past_four_gigabytes():
    """Source rows and results whose byte offsets pass 2^32, and an E4M3 source as large."""
    K, rows = 8192, 270000
    g = torch.Generator(device=DEV).manual_seed(8)
    x = torch.zeros((rows, K), dtype=BF, device=DEV)          # 4.4 GB
    at = [0, 131071, 262144, 269999]
    x[at] = torch.randn((4, K), generator=g, device=DEV).to(BF)
    w = torch.randn((2, 16, K), generator=g, device=DEV).to(BF)
    xs, ws = x[at].cpu().double(), w.cpu().double()
    tol = lambda a, b: BF_HALF * (a @ b.T).abs() + K * ULP * (a.abs() @ b.abs().T)  # noqa: E731
    y = miep.grouped_gemm(x, w, groups_of([3, 1], [0, 3]), row_index=i32([at[3], at[2], at[1], at[3]]))
    close(y[:3], xs[[3, 2, 1]] @ ws[0].T, tol(xs[[3, 2, 1]], ws[0]))
    close(y[3:], xs[[3]] @ ws[1].T, tol(xs[[3]], ws[1]))
    y = torch.full((rows, 16), MARK, dtype=BF, device=DEV)
    miep.grouped_gemm_into(x, w, groups_of([1, 2], [262144, 269998]), y, expected_rows=2)
    close(y[[262144, 269999]], torch.cat([xs[[2]] @ ws[0].T, xs[[3]] @ ws[1].T]), torch.cat([tol(xs[[2]], ws[0]), tol(xs[[3]], ws[1])]))
    assert bool((y[:262144] == MARK).all())
    dy = torch.randn((rows, 16), generator=g, device=DEV).to(BF)
    miep.grouped_gemm_dgrad_into(dy, w, groups_of([1, 2], [262144, 269998]), x, expected_rows=2)
    ds = dy[[262144, 269999]].cpu().double()
    want = torch.cat([ds[:1] @ ws[0], ds[1:] @ ws[1]])
    close(x[[262144, 269999]], want, BF_HALF * want.abs() + 16 * ULP * torch.cat([ds[:1].abs() @ ws[0].abs(), ds[1:].abs() @ ws[1].abs()]))
    dw = miep.grouped_gemm_wgrad(dy, x, groups_of([1, 2], [262144, 269998]))
    d, v = dy[269998:].cpu().double(), x[269998:].cpu().double()
    close(dw[1], d.T @ v, 3 * ULP * (d.abs().T @ v.abs()))


# ------------------------------------------------------------------ the same results every time, on any stream
def _problem(seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rows, begin, total = layout("ragged")
    x = torch.randn((total, 264), generator=g, device=DEV).to(BF)
    w = torch.randn((len(rows), 136, 264), generator=g, device=DEV).to(BF)
    dy = torch.randn((total, 136), generator=g, device=DEV).to(BF)
    return groups_of(rows, begin), x, w, dy


def test_results_do_not_depend_on_timing():
    grp, x, w, dy = _problem()
    live = members(*layout("ragged")).to(DEV)
    first = [miep.grouped_gemm(x, w, grp)[live], miep.grouped_gemm_dgrad(dy, w, grp)[live], miep.grouped_gemm_wgrad(dy, x, grp)]
    for _ in range(20):
        again = [miep.grouped_gemm(x, w, grp)[live], miep.grouped_gemm_dgrad(dy, w, grp)[live], miep.grouped_gemm_wgrad(dy, x, grp)]
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_two_streams_at_once():
    problems = [_problem(s) for s in (1, 2)]
    live = members(*layout("ragged")).to(DEV)
    want = [miep.grouped_gemm(x, w, grp)[live] for grp, x, w, _ in problems]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV) for _ in problems]
    outs = [[], []]
    for _ in range(10):
        for i, (st, (grp, x, w, dy)) in enumerate(zip(streams, problems)):
            with torch.cuda.stream(st):
                outs[i].append(miep.grouped_gemm(x, w, grp))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y[live], want[i]) for y in outs[i])
