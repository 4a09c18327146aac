"""moe_balance_loss_backward where the experts' counts are level, as the loss drives them.

With sum p = 1 the gradient p_e (c_e - sum_m p_m c_m) E / total does not change when one number is taken
from every count, so its rounding goes by how far the counts lie apart, not by how large they are."""
import numpy as np
import pytest
import torch

from oracle import block as B
from tests.test_gpu_balance import M, U, _f64, _score, make  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [2, 64, 129, 384, 768, 1024])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("count", [3, 1000, (1 << 24) + 1, (1 << 27) - 1])
def test_level_counts_have_no_gradient(M, E, score, count):  # noqa: F811
    """All counts alike: sum over e of f P is 1 whatever the scores are, so only the z-loss and d_add are left,
    to the bit what counts of 0 give.  Experts that no token is routed to, masked, change nothing."""
    print(f"[balance even] E={E} {score} count={count}", flush=True)
    T, S = 42, 3
    l, _, mask = make(T, E, 1, S, seed=E, masked=False)
    tokens = torch.full((S,), T // S, dtype=torch.int32, device="cuda")
    counts = torch.full((S, E), count, dtype=torch.int32, device="cuda")
    add = torch.randn(T, E, device="cuda")
    for off in ([], [E // 2]):
        l[:, off] = -float("inf")
        counts[:, off] = 0
        for d in ([0.7, 0.0], [1.0, -0.3], [-2.0 ** 20, 0.1]):
            d = torch.tensor(d, device="cuda")
            for a in (None, add):
                got = M.moe_balance_loss_backward(l, counts, tokens, d, _score(M, score), mask, d_add=a)
                none = M.moe_balance_loss_backward(l, torch.zeros_like(counts), tokens, d, _score(M, score), mask, d_add=a)
                assert torch.equal(got, none)
                if not d[1]:
                    assert torch.equal(got, torch.zeros_like(got) if a is None else a)


@pytest.mark.parametrize("T,E,S", [(40, 64, 1), (30, 257, 2), (33, 384, 3), (16, 1024, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("near", [12, 1000, 1 << 20, 1 << 26])
def test_nearly_level_counts(M, T, E, S, score, near):  # noqa: F811
    """Counts that differ by 1 and 2.  Their differences are exact; the scores are off by 28 U, the sum over the
    experts 28 + 21, slope 6, products 8: 91 U of |d0| E / (S N_s total) p 2 (max |c - mean| + 1)."""
    print(f"[balance even] T={T} E={E} S={S} {score} near={near}", flush=True)
    l, _, _ = make(T, E, 1, S, seed=E + T, masked=False, pad=False)
    g = torch.Generator().manual_seed(near)
    counts = (near + torch.randint(-1, 2, (S, E), generator=g)).int().cuda()
    tokens = torch.full((S,), T // S, dtype=torch.int32, device="cuda")
    d = torch.tensor([0.8, 0.0], device="cuda")
    got = _f64(M.moe_balance_loss_backward(l, counts, tokens, d, _score(M, score)))
    n = lambda t: t.cpu().numpy()  # noqa: E731
    c = n(counts).astype(np.float64)
    # the oracle on counts less their smallest would have another total: its gradient is scaled back
    low = c.min(axis=1, keepdims=True)
    ref = np.zeros((T, E))
    for s in range(S):
        rows = slice(s * (T // S), (s + 1) * (T // S))
        part = B.balance_loss_backward(n(l)[rows], (c - low)[s:s + 1], n(tokens)[s:s + 1], n(d), score)
        ref[rows] = part * (c - low)[s].sum() / c[s].sum() / S
    size = np.zeros((T, E))
    for t in range(T):
        s = t // (T // S)
        p = B._ratio(n(l)[t], np.ones(E, dtype=bool), score)
        size[t] = 0.8 * E / (S * (T // S) * c[s].sum()) * p * 2 * (np.abs(c[s] - c[s].mean()).max() + 1)
    over = np.abs(got - ref) - (91 * U * size + 1e-37)
    print(f"[balance even] worst {np.max(np.abs(got - ref) / size) / U:.1f} U", flush=True)
    assert np.all(over <= 0), f"{over.max():.3e} over, |ref| {np.abs(ref).max():.3e}"
