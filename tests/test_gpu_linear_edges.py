"""GPU parity of the dense products at their edges: what a gradient call writes, and the bound of gelu's formula."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_get_dispatch_histogram_amd as miep  # noqa: E402

DEV = torch.device("cuda:0")
BF = torch.bfloat16


@pytest.mark.parametrize("rows", [0, 1, 40, 300])
@pytest.mark.parametrize("wanted", [(), ("dx",), ("dw",), ("dx", "dw", "dbias"), ("dbias",)])
@pytest.mark.parametrize("kind", [BF, torch.float32])
def test_dz_is_written_where_it_is_given(rows, wanted, kind):
    """Without an activation too: it is dy, rounded where that is fp32."""
    N, K, g = 96, 64, torch.Generator(device=DEV).manual_seed(rows)
    x, w = torch.randint(-3, 4, (rows, K), generator=g, device=DEV).to(BF), torch.randint(-3, 4, (N, K), generator=g, device=DEV).to(BF)
    dy = torch.randn(rows, N, generator=g, device=DEV).to(kind)
    out = dict(dx=torch.empty(rows, K, dtype=BF, device=DEV), dw=torch.empty(N, K, device=DEV), dbias=torch.empty(N, device=DEV))
    out = {k: v for k, v in out.items() if k in wanted}
    alone = {k: torch.empty_like(v) for k, v in out.items()}
    ws = torch.empty(4, N, device=DEV)
    dz = torch.full((rows + 1, N), -77.0, dtype=BF, device=DEV)
    miep.linear_backward_into(dy, x, w, dz=dz[:rows], workspace=ws, **out)
    assert torch.equal(dz[:rows], dy.to(BF)) and (dz[rows] == -77).all()
    if kind == BF:                                                    # the same results as without it
        miep.linear_backward_into(dy, x, w, workspace=ws, **alone)
        for k in out:
            assert torch.equal(out[k], alone[k])


ULP = 2.0 ** -23


@pytest.mark.parametrize("rows", [1, 65, 300])
def test_gelu_holds_its_bound(rows):
    """The product is 0, so z is the bias, exactly.  Of the distribution function: its polynomial 4e-8, exp2 an ulp of the
    tail, 1 - tail half an ulp (2^-25); the product with z half an ulp of the result."""
    z = torch.cat([torch.linspace(-9, 9, 20001), torch.logspace(-30, 1, 3007)]).to(DEV)
    z = z[:z.numel() // 8 * 8]
    n = z.numel()
    y = miep.linear(torch.zeros(rows, 8, dtype=BF, device=DEV), torch.zeros(n, 8, dtype=BF, device=DEV), z.float(), "gelu", dtype=torch.float32)
    zd = z.float().double()
    p = 0.5 * torch.erfc(-zd / 2 ** 0.5)
    tail = 0.5 * torch.erfc(zd.abs() / 2 ** 0.5)
    tol = zd.abs() * (4e-8 + ULP * tail + 2.0 ** -25 * (zd > 0)) + ULP / 2 * (zd * p).abs() + 2.0 ** -126
    assert ((y.double() - zd * p).abs() <= tol).all()


def test_gelu_slope_holds_its_bound():
    """One row, so that dbias is the unrounded slope.  z is bf16, so z * z is exact; its product with log2(e) / 2 is off by
    2^-23 of itself (constant and product), exp2 an ulp, z / sqrt(2 pi) 2^-23, the last sum half an ulp."""
    z = torch.cat([torch.linspace(-9, 9, 6001), torch.logspace(-30, 1, 999)]).to(BF).to(DEV)
    n = z.numel()
    assert n % 8 == 0
    db, ws = torch.empty(n, device=DEV), torch.empty(1, n, device=DEV)
    x, w = torch.zeros(1, 8, dtype=BF, device=DEV), torch.zeros(n, 8, dtype=BF, device=DEV)
    miep.linear_backward_into(torch.ones(1, n, dtype=BF, device=DEV), x, w, "gelu", z[None].contiguous(), dbias=db, workspace=ws)
    zd = z.double()
    p, tail = 0.5 * torch.erfc(-zd / 2 ** 0.5), 0.5 * torch.erfc(zd.abs() / 2 ** 0.5)
    part = zd * torch.exp(-zd * zd / 2) / (2 * torch.pi) ** 0.5
    want = p + part
    tol = 4e-8 + ULP * tail + 2.0 ** -25 * (zd > 0) + part.abs() * (zd * zd / 2 + 2) * ULP + ULP / 2 * want.abs() + 2.0 ** -126
    assert ((db.double() - want).abs() <= tol).all()
