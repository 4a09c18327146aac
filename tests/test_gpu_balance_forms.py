"""moe_balance_loss and its gradient at sizes of every form that the number of experts chooses: experts a lane
holds (one or pairs of neighbours, 1 to 16 of them), on either side of each border, with chunk ends inside a
step of rows and ragged last columns.  Bounds as in test_gpu_balance.py."""
import pytest
import torch

from tests.test_gpu_balance import M, _score, check_gradient, check_loss, make  # noqa: F401

pytestmark = pytest.mark.gpu

# odd E: to 63, 127, 255, 511, 1023; even E: to 128, 256, 384, 512, 768, 1024
SIZES = [(47, 63, 3, 1), (58, 127, 5, 2), (45, 255, 8, 3), (47, 257, 8, 1), (58, 385, 5, 2), (75, 511, 8, 3), (41, 513, 8, 1), (58, 769, 32, 2),
         (57, 1023, 8, 3), (47, 2, 1, 1), (58, 128, 8, 2), (57, 130, 8, 3), (47, 256, 8, 1), (58, 258, 8, 2), (57, 386, 8, 3),
         (47, 514, 8, 1), (58, 640, 8, 2), (57, 768, 8, 3), (47, 770, 8, 1), (58, 1022, 8, 2)]


@pytest.mark.parametrize("T,E,k,S", SIZES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("pad", [False, True])
def test_every_form(M, T, E, k, S, score, pad):  # noqa: F811
    print(f"[balance forms] T={T} E={E} k={k} S={S} {score} pad={pad}", flush=True)
    l, idx, mask = make(T, E, k, S, seed=T + E, pad=pad)
    got = M.moe_balance_loss(l, idx, _score(M, score), S, mask)
    check_loss(l, idx, mask, S, score, got)
    d = torch.tensor([0.8, -0.05], device="cuda")
    add = torch.randn(T, E, device="cuda") if T % 2 else None
    out = torch.full((T, E), float("nan"), device="cuda")
    M.moe_balance_loss_backward(l, got[1], got[3], d, _score(M, score), mask, d_add=add, dlogits=out)
    check_gradient(l, got[1], got[3], d, score, mask, add, out)


@pytest.mark.parametrize("E", [257, 513, 640])
def test_many_rows(M, E):  # noqa: F811
    """More rows than a chunk's first step: every chunk has a second one, the last chunk a ragged one."""
    print(f"[balance forms] many rows E={E}", flush=True)
    T, k = 40011, 4
    l, idx, mask = make(T, E, k, 1, seed=E, masked=False)
    losses, counts, probs, tokens = M.moe_balance_loss(l, idx, token_mask=mask)
    on = mask.bool()
    assert int(tokens) == int(on.sum())
    assert torch.equal(counts[0].long(), torch.bincount(idx[on].reshape(-1).long(), minlength=E))
    p = torch.softmax(l[on].double(), 1)
    # 28 U of a score, and at most (rows of a wave + 4) U of their FP32 sum: 40011 rows in 1024 chunks of 48 or less
    assert float(((probs[0].double() - p.mean(0)).abs() / p.mean(0)).max()) < (28 + 48 + 4) * 2.0 ** -24
    d = torch.tensor([1.0, 0.1], device="cuda")
    g = M.moe_balance_loss_backward(l, counts, tokens, d, token_mask=mask)
    c, n = counts[0].double(), int(tokens)
    f = E * c / c.sum()
    q, lse = torch.softmax(l.double(), 1), torch.logsumexp(l.double(), 1, keepdim=True)
    d1 = float(d[1].double())
    ref = (q * (f - (q * f).sum(1, keepdim=True)) / n + d1 * 2 / n * lse * q) * on.unsqueeze(1)
    size = q * 2 * f.max() / n + abs(d1) * 2 / n * torch.maximum(lse.abs(), l.double().abs().amax(1, keepdim=True)) * q
    assert bool(((g.double() - ref).abs() <= 91 * 2.0 ** -24 * size + 2.0 ** -24 * ref.abs() + 1e-37).all())
