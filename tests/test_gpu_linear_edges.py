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
