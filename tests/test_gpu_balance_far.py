"""The gradient of the z-loss where a logit comes near the end of FP32's range."""
import numpy as np
import pytest
import torch

from tests.test_gpu_balance import M, U, _score  # noqa: F401

pytestmark = pytest.mark.gpu

FLT_MAX = float(np.finfo(np.float32).max)


@pytest.mark.parametrize("E", [5, 64, 257, 1024])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top", [float("inf"), 3e38, 2e38])
def test_gradient_of_a_row_with_a_far_logit(M, E, score, top):  # noqa: F811
    """2 lse / N of a single row passes FP32's range: the experts whose scores vanish get 0, and d_add, all the same;
    halved by a second expert as far up, it is representable again."""
    print(f"[balance far] E={E} {score} top={top}", flush=True)
    for both in (False, True):
        l = torch.zeros(1, E, device="cuda")
        l[0, 2] = top
        if both:
            l[0, 4] = top
        rest = [e for e in range(E) if e not in ((2, 4) if both else (2,))]
        counts, tokens = torch.zeros(1, E, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
        for d in ([0.0, 1.0], [0.5, -1.0]):
            d = torch.tensor(d, device="cuda")
            add = torch.randn(1, E, device="cuda")
            got = M.moe_balance_loss_backward(l, counts, tokens, d, _score(M, score))
            assert not got[0, rest].any()
            assert torch.equal(M.moe_balance_loss_backward(l, counts, tokens, d, _score(M, score), d_add=add)[0, rest], add[0, rest])
            want = 2.0 * float(d[1]) * min(top, FLT_MAX) * (0.5 if both else 1.0)
            for e in (2, 4) if both else (2,):
                g = float(got[0, e])
                # (past the range by less than the rounding of q, either side is right)
                assert abs(g - want) <= 91 * U * abs(want) if abs(want) < 0.99 * FLT_MAX else abs(g) > 0.98 * FLT_MAX and g * want > 0
