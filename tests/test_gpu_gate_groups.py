"""GPU parity of the choice among groups where a group's score is at an edge, against the 64-bit choice."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_get_dispatch_histogram_amd as miep  # noqa: E402
from test_gpu_gate import check, choice, clean, gen  # noqa: E402

DEV = torch.device("cuda:0")


def same_choice(logits, K, score, bias, groups, top, best):
    print("[case]", tuple(logits.shape), logits.dtype, K, score, groups, top, best, flush=True)
    idx, _ = miep.gate_topk(logits.to(DEV), K, score, None if bias is None else bias.to(DEV), groups, top, best)
    want = choice(clean(logits.float()), K, score, bias, groups, top, best)
    wrong = (idx.cpu().numpy() != want).any(1)
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
