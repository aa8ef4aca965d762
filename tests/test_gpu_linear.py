"""GPU parity of the dense products with their epilogue and of their gradients, against plain 64-bit formulas.

Sums of whole numbers: x and w hold small integers (w times a power of two), so that every sum and z itself are exact
in fp32 and only the epilogue's own roundings are left:
  identity, relu          exact; one rounding for the residual's sum, one to bf16 (half a step, 2^-8)
  silu, gelu, SwiGLU      a few fp32 roundings of the factors; gelu's distribution function is off by 0.75e-7
Sums of normal numbers: one fp32 ulp (2^-23) of the sum of magnitudes an addition.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_get_dispatch_histogram_amd as miep  # noqa: E402

DEV = torch.device("cuda:0")
BF = torch.bfloat16
ULP, BF_HALF = 2.0 ** -23, 2.0 ** -8
MARK = -77.0
ACTS = [None, "relu", "silu", "gelu", "gelu_tanh", "swiglu"]
# rows of the few-row kernel (1..64, its column tiles of 16), of the split one, of each tile, one more and one less
ROWS = [1, 2, 15, 16, 17, 32, 33, 48, 64, 65, 100, 129, 255, 257]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def ints(shape, hi, seed, scale=1.0, dtype=BF):
    return (torch.randint(-hi, hi + 1, shape, generator=gen(seed), device=DEV).float() * scale).to(dtype)


def f64(z, act):
    if act == "swiglu":
        g, u = z.chunk(2, 1)
        return g * torch.sigmoid(g) * u
    if act == "gelu_tanh":
        return torch.nn.functional.gelu(z, approximate="tanh")
    return {None: lambda v: v, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[act](z)


def own_error(z, act):
    """What f computes beside f(z) of an exact z, in fp32."""
    if act in (None, "relu"):
        return 0.0 * z[:, :1]
    if act == "swiglu":
        g, u = z.chunk(2, 1)
        # exp's argument is exact to 2^-40, exp2 and rcp an ulp each, the products half an ulp each
        return 8 * ULP * (g * u).abs()
    return (8 * ULP + (1e-7 if act == "gelu" else 0.0)) * z.abs() + (4 * ULP * z.abs() ** 3 if act == "gelu_tanh" else 0.0)


def close(got, want, tol, what):
    got = got.double()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), "%s: %d of %d off, first %s got %r want %r" % (what, int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist(),
                                                                         float(got[bad][0]), float(want[bad][0]))


def check(M, N, K, act, bias, residual, dtype, save, seed=1):
    print("[case]", M, N, K, act, bias, residual, dtype, save, flush=True)
    x, w = ints((M, K), 3, seed), ints((N, K), 3, seed + 1, 2.0 ** -5)
    b = ints((N,), 9, seed + 2, 2.0 ** -3, torch.float32) if bias else None
    width = N // 2 if act == "swiglu" else N
    r = ints((M, width), 50, seed + 3, 2.0 ** -4) if residual else None
    y = torch.full((M + 1, width), MARK, dtype=dtype, device=DEV)
    z = torch.full((M + 1, N), MARK, dtype=BF, device=DEV) if save else None
    miep.linear_into(x, w, y[:M], b, act, r, z[:M] if save else None)
    zz = x.double() @ w.double().t() + (0 if b is None else b.double())
    want = f64(zz, act) + (0 if r is None else r.double())
    tol = own_error(zz, act) + ULP * want.abs() + (BF_HALF * want.abs() if dtype == BF else 0)
    close(y[:M], want, tol, "y")
    assert (y[M] == MARK).all()
    if save:
        close(z[:M], zz, BF_HALF * zz.abs(), "z")
        assert (z[M] == MARK).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", ROWS)
def test_rows_and_activations(M, act):
    odd = M % 2 == 1
    check(M, 80, 136, act, odd, not odd, BF, not odd)
    check(M, 272, 200, act, not odd, odd, torch.float32, odd)


# one column of 8, tiles' borders, contractions shorter than a step and not whole ones
SIZES = [(8, 8), (16, 64), (24, 72), (48, 1000), (144, 40), (256, 1536), (264, 1544), (1040, 320), (4112, 128)]


@pytest.mark.parametrize("N,K", SIZES)
@pytest.mark.parametrize("M", [3, 40, 70, 300])
def test_sizes(M, N, K):
    check(M, N, K, None, True, True, BF, False)
    check(M, N, K, "gelu", False, False, torch.float32, True)
    if N % 16 == 0:
        check(M, N, K, "swiglu", True, True, BF, True)


# every tile of the many-rows kernels: wide ones of 192 and 256 rows, 128 x 128 / 192 / 256, the split one
@pytest.mark.parametrize("M,N,K", [(4096, 4096, 64), (6000, 2064, 128), (1500, 4096, 72), (190, 20000, 64), (180, 33000, 64),
                                   (250, 30000, 128), (128, 256, 2048), (70, 512, 7168), (1003, 7168, 256)])
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_tiles(M, N, K, act):
    if act == "swiglu" and N % 16:
        N -= 8
    check(M, N, K, act, True, True, BF, True)
    check(M, N, K, act, False, False, torch.float32, False)


@pytest.mark.parametrize("M", [16, 64, 200, 2000])
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_sums_of_normal_numbers(M, act):
    N, K = 512, 4096
    x, w = torch.randn(M, K, generator=gen(1), device=DEV).to(BF), (torch.randn(N, K, generator=gen(2), device=DEV) / 64).to(BF)
    y = miep.linear(x, w, activation=act, dtype=torch.float32)
    z = x.double() @ w.double().t()
    tz = (K + 2) * ULP * (x.double().abs() @ w.double().abs().t())
    if act:
        g, u = z.chunk(2, 1)
        tg, tu = tz.chunk(2, 1)
        tol = 1.1 * u.abs() * tg + (g * torch.sigmoid(g)).abs() * tu + 1.1 * tg * tu + own_error(z, act)
    else:
        tol = tz
    close(y, f64(z, act), tol, "y")
    # no sum is cut: the error is a small part of that bound
    assert (y.double() - f64(z, act)).norm() < 2e-6 * f64(z, act).norm()


def test_no_rows_and_values_that_are_no_numbers():
    x, w = torch.zeros(0, 64, dtype=BF, device=DEV), ints((32, 64), 3, 1)
    assert miep.linear(x, w, activation="swiglu").shape == (0, 16)
    for M in (5, 80):                                                 # a row of NaN and one of infinities stay in their rows
        x = ints((M, 72), 3, 2)
        x[1], x[3] = float("nan"), float("inf")
        y = miep.linear(x, w[:, :72] if w.shape[1] == 72 else ints((32, 72), 3, 1), dtype=torch.float32)
        assert torch.isnan(y[1]).all() and not torch.isfinite(y[3]).any()
        keep = [i for i in range(M) if i not in (1, 3)]
        assert torch.isfinite(y[keep]).all()
        v = ints((32, 72), 3, 1)
        v[7] = float("nan")
        y = miep.linear(x[keep].contiguous(), v, activation="relu")
        assert torch.isnan(y[:, 7]).all() and torch.isfinite(y[:, :7]).all() and torch.isfinite(y[:, 8:]).all()


@pytest.mark.parametrize("M", [20, 90, 700])
@pytest.mark.parametrize("act", ["silu", "swiglu"])
def test_residual_in_place(M, act):
    x, w = ints((M, 128), 3, 5), ints((256, 128), 3, 6, 2.0 ** -5)
    width = 128 if act == "swiglu" else 256
    r = ints((M, width), 50, 7)
    want = miep.linear(x, w, activation=act, residual=r)
    miep.linear_into(x, w, r, activation=act, residual=r)
    assert torch.equal(r, want)


# ------------------------------------------------------------------ gradient
def slope(z, act):
    z = z.double().requires_grad_()
    with torch.enable_grad():
        return torch.autograd.grad(f64(z, act).sum(), z)[0]


@pytest.mark.parametrize("act", ACTS[1:])
def test_slopes_agree_with_differences(act):
    z = torch.randn(50, 8, generator=gen(3), device=DEV).double() * 2
    h = 1e-6
    s = slope(z, act)
    for c in range(8):
        d = torch.zeros_like(z)
        d[:, c] = h
        assert ((f64(z + d, act) - f64(z - d, act)).sum(1) / (2 * h) - s[:, c]).abs().max() < 1e-7


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 3, 16, 65, 300, 1031])
def test_gradients(M, act):
    for N, K, dy_type, dw_type in ((80, 136, BF, torch.float32), (1040, 72, torch.float32, BF)):
        print("[case]", M, N, K, act, flush=True)
        width = N // 2 if act == "swiglu" else N
        x, w = ints((M, K), 3, 1), ints((N, K), 3, 2)
        z = (torch.randn(M, N, generator=gen(3), device=DEV) * 2).to(BF) if act else None
        dy = torch.randn(M, width, generator=gen(4), device=DEV).to(dy_type)
        dx, dw, db = miep.linear_backward(dy, x, w, act, z, bias=True, dtype=dw_type)
        if act == "swiglu":
            g, u = z.double().chunk(2, 1)
            s = torch.sigmoid(g)
            dz = torch.cat([dy.double() * u * s * (1 + g * (1 - s)), dy.double() * g * s], 1)
            size = torch.cat([(dy.double() * u).abs() * (1 + g.abs()), (dy.double() * g).abs()], 1)
        elif act:
            zd = z.double()
            dz = dy.double() * slope(z, act)
            size = dy.double().abs() * (1 + zd.abs()) * (1 + (zd * zd if act == "gelu_tanh" else 0))
        else:
            dz, size = dy.double(), 0 * dy.double()
        own = size * (12 * ULP + (2e-7 if act == "gelu" else 0))                    # fp32 factors of a slope
        half = BF_HALF if act or dy_type == torch.float32 else 0                    # what the products read
        tz = own + half * dz.abs()
        n = M + 4
        close(db, dz.sum(0), own.sum(0) + n * ULP * dz.abs().sum(0), "dbias")
        close(dx, dz @ w.double(), tz @ w.double().abs() + (N + 2) * ULP * (dz.abs() @ w.double().abs()) + BF_HALF * (dz @ w.double()).abs(), "dx")
        want = dz.t() @ x.double()
        close(dw, want, tz.t() @ x.double().abs() + (M + 2) * ULP * (dz.abs().t() @ x.double().abs()) + (BF_HALF * want.abs() if dw_type == BF else 0), "dw")
        assert dw.dtype == dw_type and db.dtype == torch.float32


def test_gradients_by_parts():
    """Any workspace gives the same sums up to their order; only what is asked for is written; sums can be added to."""
    M, N, K = 500, 96, 64
    x, w = ints((M, K), 3, 1), ints((N, K), 3, 2)
    dy = ints((M, N), 3, 3)
    z = ints((M, N), 2, 4)
    want_b = (dy.double() * (z.double() > 0)).sum(0)
    for parts in (1, 2, 31, 32, 200):
        ws = torch.full((parts + 1, N), MARK, device=DEV)
        db = torch.full((N,), MARK, device=DEV)
        miep.linear_backward_into(dy, x, w, "relu", z, dbias=db, workspace=ws[:parts])
        assert torch.equal(db.double(), want_b) and (ws[parts] == MARK).all()
        miep.linear_backward_into(dy, x, w, "relu", z, dbias=db, workspace=ws[:parts], accumulate=True)
        assert torch.equal(db.double(), 2 * want_b)
    dz = torch.empty(M, N, dtype=BF, device=DEV)
    dw = torch.full((N, K), 5.0, device=DEV)
    miep.linear_backward_into(dy, x, w, "relu", z, dw=dw, dz=dz, accumulate=True)
    exact = (dy.double() * (z.double() > 0))
    assert torch.equal(dz.double(), exact) and torch.equal(dw.double(), exact.t() @ x.double() + 5)
    dx = torch.empty(M, K, dtype=BF, device=DEV)
    miep.linear_backward_into(dy, x, w, dx=dx)                        # no activation, bf16 dy: no dz needed
    close(dx, dy.double() @ w.double(), BF_HALF * (dy.double() @ w.double()).abs(), "dx")


def test_gradients_of_no_rows():
    x, w, dy = torch.zeros(0, 64, dtype=BF, device=DEV), ints((32, 64), 3, 1), torch.zeros(0, 32, dtype=BF, device=DEV)
    dx, dw, db = miep.linear_backward(dy, x, w, bias=True)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()


def test_streams_and_graphs():
    M, N, K = 48, 128, 256
    x, w, b = ints((M, K), 3, 1), ints((N, K), 3, 2, 2.0 ** -5), ints((N,), 9, 3, 1.0, torch.float32)
    y, z = torch.empty(M, 64, dtype=BF, device=DEV), torch.empty(M, N, dtype=BF, device=DEV)
    dx, dw, db = torch.empty_like(x), torch.empty(N, K, device=DEV), torch.empty(N, device=DEV)
    dz, ws = torch.empty(M, N, dtype=BF, device=DEV), torch.empty(3, N, device=DEV)
    dy = ints((M, 64), 3, 4)

    def step():
        miep.linear_into(x, w, y, b, "swiglu", z=z)
        miep.linear_backward_into(dy, x, w, "swiglu", z, dx, dw, db, dz, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for turn in range(3):
        x.copy_(ints((M, K), 3, 10 + turn))
        dy.copy_(ints((M, 64), 3, 20 + turn))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, z, dx, dw, db)]
        wy, wz = miep.linear(x, w, b, "swiglu", save=True)
        wdx, wdw, wdb = miep.linear_backward(dy, x, w, "swiglu", wz, bias=True)
        for g, t in zip(got, (wy, wz, wdx, wdw, wdb)):
            assert torch.equal(g, t)


FAR = [64.0, 128.0, 1e4, 1e10, 1e20, 1e30, 3e38]


@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("M", [2, 100, 700])
def test_far_values(M, act):
    """Every f is z or 0 there and f' is 1 or 0, to a few fp32 roundings (2^-20 of them and the smallest normal number),
    with nothing that overflows between."""
    z = torch.tensor(FAR + [-v for v in FAR] + [0.0, 1.0], device=DEV).to(BF)
    n = z.numel()
    w = torch.zeros(2 * n if act == "swiglu" else n, 8, dtype=BF, device=DEV)
    w[:n, 0] = z
    w[n:, 0] = 1                                                      # SwiGLU's up
    x = torch.zeros(M, 8, dtype=BF, device=DEV)
    x[:, 0] = 1
    y, saved = miep.linear(x, w, activation=act, dtype=torch.float32, save=True)
    assert torch.equal(saved, w[:, 0].expand(M, -1))
    zz = saved.double()
    want = f64(zz, act)
    close(y, want, 2.0 ** -20 * want.abs() + 2.0 ** -126 + (1e-7 if act == "gelu" else 0), "y")
    dz = torch.empty_like(saved)
    miep.linear_backward_into(torch.ones_like(y), x, w, act, saved, dz=dz)
    s = slope(saved, act)
    close(dz, s, (BF_HALF + 2.0 ** -20) * s.abs() + 2.0 ** -126 + (1e-7 if act == "gelu" else 0), "dz")
    nan = torch.full_like(saved, float("nan"))
    miep.linear_backward_into(torch.ones_like(y), x, w, act, nan, dz=dz)
    assert act == "relu" or torch.isnan(dz).all()


def test_offsets_past_32_bits():
    """Results, saved values and gradients of more than 2^31 elements: the last rows."""
    M, N, K, last = 34000, 65536, 64, 40
    assert M * N > 2 ** 31
    x, w = torch.zeros(M, K, dtype=BF, device=DEV), ints((N, K), 3, 1)
    x[-last:] = ints((last, K), 3, 2)
    y, z = miep.linear(x, w, activation="relu", save=True)
    zz = x[-last:].double() @ w.double().t()
    assert torch.equal(z[-last:].double(), zz.to(BF).double()) and torch.equal(y[-last:], z[-last:].clamp(min=0))
    assert not y[:-last].any()
    y.zero_()
    y[-last:] = ints((last, N), 1, 3)
    dx, dw, db = miep.linear_backward(y, x, w, "relu", z, bias=True)
    dz = y[-last:].double() * (zz > 0)
    assert not dx[:-last].any()
    want = dz @ w.double()
    close(dx[-last:], want, (N + 2) * ULP * (dz.abs() @ w.double().abs()) + BF_HALF * want.abs(), "dx")
    assert torch.equal(dw.double(), dz.t() @ x[-last:].double()) and torch.equal(db.double(), dz.sum(0))


def test_two_streams_at_once():
    """Calls of two streams side by side, each with outputs of its own."""
    sides = [torch.cuda.Stream() for _ in range(2)]
    cases = []
    for M, N, K in ((16, 512, 2048), (200, 512, 1024)):
        x, w = ints((M, K), 3, M), ints((N, K), 3, M + 1, 2.0 ** -5)
        cases.append((x, w, torch.empty(M, N, device=DEV), x.double() @ w.double().t()))
    torch.cuda.synchronize()
    for _ in range(10):
        for side, (x, w, y, _) in zip(sides, cases):
            with torch.cuda.stream(side):
                miep.linear_into(x, w, y)
    torch.cuda.synchronize()
    for x, w, y, want in cases:
        assert torch.equal(y.double(), want)
