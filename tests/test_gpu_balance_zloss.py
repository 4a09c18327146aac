"""The z-loss as the mean of squares whose sum passes FP32's range, or has FP32 steps of its own size."""
import numpy as np
import pytest
import torch

from oracle import block as B
from tests.test_gpu_balance import M, U, _f64  # noqa: F401

pytestmark = pytest.mark.gpu

FLT_MAX = float(np.finfo(np.float32).max)


@pytest.mark.parametrize("T,E,S", [(1, 8, 1), (7, 64, 1), (64, 257, 2), (5000, 384, 1), (4096, 1024, 4)])
def test_mean_square_within_range(M, T, E, S):  # noqa: F811
    """lse^2 of every row and their mean within FP32, not so their sum."""
    print(f"[balance far] T={T} E={E} S={S}", flush=True)
    g = torch.Generator().manual_seed(T)
    l = torch.randn(T, E, generator=g)
    l[:, E // 2] = 1.5e19 + 1e17 * torch.randn(T, generator=g)
    l = l.cuda()
    idx = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    losses = M.moe_balance_loss(l, idx, n_seqs=S)[0]
    want = float((_f64(l)[:, E // 2] ** 2).mean())
    assert want < 0.8 * FLT_MAX
    # lse is the logit itself to half a unit; its square and the FP64 sum are exact beside it
    assert abs(float(losses[1]) - want) <= 4 * U * want


def test_mean_square_of_many_rows(M):  # noqa: F811
    """As many rows as a call takes, all alike: the mean square of lse is the square of one row's, within the
    roundings of lse (4 U of it) and of the result, whatever the number of rows."""
    T, E = (1 << 22) - 1, 4
    l = torch.tensor([[0.3, -0.2, 1.1, 0.7]], device="cuda").repeat(T, 1)
    losses = M.moe_balance_loss(l, torch.zeros(T, 1, dtype=torch.int32, device="cuda"))[0]
    lse = B._lse(l[0].cpu().numpy(), np.ones(E, dtype=bool))
    one = float(M.moe_balance_loss(l[:1].contiguous(), torch.zeros(1, 1, dtype=torch.int32, device="cuda"))[0][1])
    assert abs(float(losses[1]) - lse ** 2) <= (8 + 1) * U * lse ** 2
    assert abs(float(losses[1]) - one) <= 2 * U * one
