"""Weights' gradients of gathered rows some of which have no source."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_get_dispatch_histogram_amd as miep  # noqa: E402
from test_gpu_experts import BF, BF_HALF, DEV, ULP, _wgrad_want, close, gen, groups_of, say  # noqa: E402


# (rows of each group, N, K): tiles of 128, of 256 with a group that ends on a whole step of 64, and rows split over wavefronts
@pytest.mark.parametrize("rows,N,K", [([1, 0, 200, 64, 77, 128, 130, 300], 136, 200), ([256 + 37 * (i % 3) for i in range(64)], 264, 272),
                                      ([2600, 1, 0, 1217, 33, 256], 72, 136)])
@pytest.mark.parametrize("where", ["some", "first and last", "a step", "all"])
def test_rows_without_a_source_contribute_nothing(where, rows, N, K):
    """Whatever their gradients hold: NaN and infinities, as in slots that nothing wrote."""
    say("no source", where, len(rows), N, K)
    begin = np.cumsum([2] + rows[:-1]).tolist()
    total, src = begin[-1] + rows[-1] + 3, 90
    g = gen(N)
    dy, x = torch.randn((total, N), generator=g).to(BF), torch.randn((src, K), generator=g).to(BF)
    index = torch.randint(0, src, (total,), generator=g, dtype=torch.int32)
    for n, b in zip(rows, begin):
        at = {"some": torch.arange(b, b + n)[torch.rand(n, generator=g) < 0.1],
              "first and last": torch.tensor([b, b + n - 1] if n else [], dtype=torch.int64),
              "a step": torch.arange(b + 64, b + max(min(n, 128), 64)), "all": torch.arange(b, b + n)}[where]
        index[at[::2]], index[at[1::2]] = -1, src + 5
    lost = (index < 0) | (index >= src)
    clean = torch.where(lost.unsqueeze(1), torch.zeros_like(dy), dy)
    dy[lost] = float("nan")
    dy[lost.nonzero()[::3, 0]] = float("inf")
    want, mag = _wgrad_want(clean, x, rows, begin, index)
    grp, kw, most = groups_of(rows, begin), dict(row_index=index.to(DEV)), max(rows)
    close(miep.grouped_gemm_wgrad(dy.to(DEV), x.to(DEV), grp, **kw), want, (most + 1) * ULP * mag, "fp32")
    close(miep.grouped_gemm_wgrad(dy.to(DEV), x.to(DEV), grp, dtype=BF, **kw), want,
          BF_HALF * want.abs() + (most + 1) * ULP * mag * 2, "bf16")
    old = torch.randn(want.shape, generator=g)
    acc = old.to(DEV)
    miep.grouped_gemm_wgrad_into(dy.to(DEV), x.to(DEV), grp, acc, accumulate=True, **kw)
    close(acc, want + old.double(), (most + 2) * ULP * (mag + old.double().abs()), "accumulated")
