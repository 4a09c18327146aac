"""moe_balance_loss and its gradient against the FP64 oracle.

Bounds.  A score is a ratio of FP32 exponentials: 2 units in the last place each, their sum (6 adds
across lanes and up to 15 within one), a reciprocal and a product: 28 * 2^-24 relative.  Their mean is
summed in FP32 over a workgroup's rows (at most 2^12 of them to a wave) and in FP64 over
workgroups: a relative error of the rows of one wave, at most (rows + 4) 2^-24.  lse: 2 units of the
logarithm and of the sum of both parts, 4 * 2^-24 of the larger of the two, that is of
max(|largest logit|, log E).  The gradient adds the products' roundings, and the subtraction of two
numbers of the size of the largest f."""
import numpy as np
import pytest
import torch

from oracle import block as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def M():
    import mixture_experts_ffn_07_amd as M
    yield M
    M.moe_set_debug_options(0, 0)


def _f64(t):
    return t.detach().double().cpu().numpy()


def make(T, E, k, S, seed=0, masked=True, pad=True, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g) * spread
    idx = l.topk(k, dim=1).indices
    if masked and E > 2:
        l[:, torch.randint(0, E, (max(1, E // 16),), generator=g)] = -float("inf")
        l[T // 2] = -float("inf")                          # a token without experts
        l[0, 0] = float("nan")
        l[0, 1] = -3.3895313892515355e38
    mask = None
    if pad:
        L = T // S
        length = torch.randint(0, L + 1, (S, 1), generator=g)
        mask = (torch.arange(L) < length).reshape(T).to(torch.uint8)
        idx[mask == 0] = torch.tensor([-1, E, 2 ** 31 - 1])[torch.randint(0, 3, (int((mask == 0).sum()), k), generator=g)]
    return l.cuda(), idx.int().cuda(), None if mask is None else mask.cuda()


def _score(M, score):
    return M.MOE_SCORE_SIGMOID if score == "sigmoid" else M.MOE_SCORE_SOFTMAX


def check_loss(l, idx, mask, S, score, got):
    losses, counts, probs, tokens = got
    rl, rc, rp, rt = B.balance_loss(l.cpu().numpy(), idx.cpu().numpy(), score, S, None if mask is None else mask.cpu().numpy())
    assert np.array_equal(counts.cpu().numpy(), rc) and np.array_equal(tokens.cpu().numpy(), rt)
    T = l.shape[0]
    rel = (28 + 4 + min(T, 4096)) * U
    assert np.all(np.abs(_f64(probs) - rp) <= rp * rel + 1e-37)
    fin = l[torch.isfinite(l) & (l.abs() < 3e38)]
    big = max(float(fin.abs().max()) if fin.numel() else 0.0, np.log(l.shape[1]))
    g = _f64(losses)
    assert abs(g[0] - rl[0]) <= rl[0] * rel + 1e-37
    # lse is off by 4 U big, its square by 8 U big |lse| (+ the sum), |lse| <= root of the mean square
    # for the mean (Cauchy-Schwarz)
    assert abs(g[1] - rl[1]) <= 8 * U * big * np.sqrt(rl[1]) + rl[1] * rel + (4 * U * big) ** 2


SIZES = [(1, 1, 1, 1), (1, 8, 2, 1), (2, 64, 8, 2), (5, 65, 3, 1), (12, 129, 32, 3), (64, 384, 8, 1), (77, 1024, 10, 7), (300, 100, 4, 3),
         (1000, 512, 8, 8), (2048, 384, 8, 1), (2049, 256, 8, 3), (4096, 32, 2, 4096), (8192, 60, 6, 2)]


@pytest.mark.parametrize("T,E,k,S", SIZES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("pad", [False, True])
def test_loss_and_gradient(M, T, E, k, S, score, pad):
    print(f"[balance] T={T} E={E} k={k} S={S} {score} pad={pad}", flush=True)
    l, idx, mask = make(T, E, k, S, seed=T + E, pad=pad)
    got = M.moe_balance_loss(l, idx, _score(M, score), S, mask)
    check_loss(l, idx, mask, S, score, got)
    _, counts, _, tokens = got
    d = torch.tensor([0.8, -0.05], device="cuda")
    add = torch.randn(T, E, device="cuda") if T % 2 else None
    out = torch.full((T, E), float("nan"), device="cuda")
    M.moe_balance_loss_backward(l, counts, tokens, d, _score(M, score), mask, d_add=add, dlogits=out)
    check_gradient(l, counts, tokens, d, score, mask, add, out)


def check_gradient(l, counts, tokens, d, score, mask, add, out):
    n = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    ref = B.balance_loss_backward(n(l), n(counts), n(tokens), n(d), score, n(mask))
    T, E = l.shape
    S = counts.shape[0]
    # magnitudes of the parts: |d0| p max f / (S N_s), and |d1| 2/N lse q
    c = n(counts).astype(np.float64)
    f = E * c / np.maximum(1, c.sum(axis=1, keepdims=True))
    size = np.zeros((T, E))
    dd = n(d).astype(np.float64)
    for t in range(T):
        s = t // (T // S)
        on = (n(l)[t] > B.MASK)
        if not on.any() or (mask is not None and not mask[t]):
            continue
        p = B._ratio(n(l)[t], on, score)
        lse = B._lse(n(l)[t], on)
        big = max(abs(lse), float(np.abs(np.where(on, np.minimum(n(l)[t], B.FLT_MAX), 0)).max()), np.log(E))
        if tokens[s]:
            size[t] += abs(dd[0]) / (S * float(tokens[s])) * p * 2 * f[s].max()
        size[t] += abs(dd[1]) * 2 / max(1, int(tokens.sum())) * big * B._ratio(n(l)[t], on, "softmax")
    # scores 28 U, the dot product over the experts 28 + 21 more, slope 6, products 8: 91 U of a part
    base = np.zeros((T, E)) if add is None else n(add).astype(np.float64)
    bound = 91 * U * size + U * np.abs(ref + base) + 1e-37
    got = n(out).astype(np.float64)
    over = np.abs(got - (ref + base)) - bound
    assert np.all(np.isfinite(got)) and np.all(over <= 0), f"{over.max():.3e} over, |ref| {np.abs(ref).max():.3e}"


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_against_differences(M, score):
    """Central differences of the kernel's own loss: h = 2^-5, the loss off by up to 40 U of about 3 each
    way (2.3e-4 over 2 h), third derivatives up to 1 times h^2 / 6 (1.6e-4)."""
    T, E, k = 6, 12, 3
    l, idx, mask = make(T, E, k, 1, seed=3, masked=False, pad=False)
    d = torch.tensor([1.0, 0.25], device="cuda")
    value = lambda z: float((M.moe_balance_loss(z, idx, _score(M, score), 1, mask)[0].double() * d.double()).sum())  # noqa: E731
    _, counts, _, tokens = M.moe_balance_loss(l, idx, _score(M, score), 1, mask)
    g = M.moe_balance_loss_backward(l, counts, tokens, d, _score(M, score), mask)
    for t in range(T):
        for e in range(0, E, 3):
            up, down = l.clone(), l.clone()
            up[t, e] += 2.0 ** -5
            down[t, e] -= 2.0 ** -5
            h = float(up[t, e].double() - down[t, e].double())
            assert abs((value(up) - value(down)) / h - float(g[t, e])) < 4e-4


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_extreme_logits(M, score):
    l = torch.zeros(8, 70)
    l[0] = -1e30                                            # all far below: scores are ratios
    l[1] = 1e30
    l[2] = -104.0 - torch.arange(70) * 0.1
    l[3, 0], l[3, 1] = float("inf"), 3e38                   # +inf counts as FLT_MAX
    l[4, ::2] = -200.0
    l[5] = 88.0 + torch.arange(70) * 0.5
    l[6] = -float("inf")
    l[6, 9] = -50.0
    l[7] = torch.arange(70) - 35.0
    l = l.cuda()
    idx = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    idx[:, 1] = torch.arange(8, device="cuda") * 9
    for rows in ([0], [2], [4, 5], [6], [7], [2, 4, 5, 6, 7]):
        sub, ids = l[rows].contiguous(), idx[rows].contiguous()
        got = M.moe_balance_loss(sub, ids, _score(M, score))
        check_loss(sub, ids, None, 1, score, got) if rows != [0] else None
        assert torch.isfinite(got[2]).all()
        rp = B.balance_loss(sub.cpu().numpy(), ids.cpu().numpy(), score)[2]
        assert np.all(np.abs(_f64(got[2]) - rp) <= rp * 64 * U + 1e-37)
        d = torch.tensor([1.0, 0.0], device="cuda")
        out = M.moe_balance_loss_backward(sub, got[1], got[3], d, _score(M, score))
        check_gradient(sub, got[1], got[3], d, score, None, None, out)
    for rows in ([1], [3]):
        sub, ids = l[rows].contiguous(), idx[rows].contiguous()
        got = M.moe_balance_loss(sub, ids, _score(M, score))
        rp = B.balance_loss(sub.cpu().numpy(), ids.cpu().numpy(), score)[2]
        assert np.all(np.abs(_f64(got[2]) - rp) <= rp * 64 * U + 1e-37)


def test_nothing_takes_part(M):
    l, idx, _ = make(40, 24, 3, 4, pad=False)
    mask = torch.zeros(40, dtype=torch.bool, device="cuda")
    losses, counts, probs, tokens = M.moe_balance_loss(l, idx, n_seqs=4, token_mask=mask)
    assert not losses.any() and not counts.any() and not probs.any() and not tokens.any()
    d = torch.ones(2, device="cuda")
    add = torch.randn(40, 24, device="cuda")
    assert torch.equal(M.moe_balance_loss_backward(l, counts, tokens, d, token_mask=mask, d_add=add), add)
    assert not M.moe_balance_loss_backward(l, counts, tokens, d, token_mask=mask).any()
    # tokens, but no routed slot
    idx.fill_(-1)
    losses, counts, probs, tokens = M.moe_balance_loss(l, idx, n_seqs=4)
    assert losses[0] == 0 and losses[1] > 0 and not counts.any() and tokens.tolist() == [10] * 4


@pytest.mark.parametrize("S", [1, 5])
def test_empty_batch_writes_zeros(M, S):
    l, idx = torch.empty(0, 16, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda")
    full = dict(losses=torch.full((2,), 7.0, device="cuda"), counts=torch.full((S, 16), 7, dtype=torch.int32, device="cuda"),
                probs=torch.full((S, 16), 7.0, device="cuda"), tokens=torch.full((S,), 7, dtype=torch.int32, device="cuda"))
    for t in M.moe_balance_loss(l, idx, n_seqs=S, **full):
        assert not t.any()
    assert M.moe_balance_loss_backward(l, full["counts"], full["tokens"], full["losses"]).shape == (0, 16)


def test_masked_rows_may_hold_anything(M):
    T, E, k = 200, 96, 4
    l, idx, mask = make(T, E, k, 2, seed=9, masked=False)
    ref = M.moe_balance_loss(l, idx, n_seqs=2, token_mask=mask)
    d = torch.tensor([1.0, 1.0], device="cuda")
    g = M.moe_balance_loss_backward(l, ref[1], ref[3], d, token_mask=mask)
    l2, idx2 = l.clone(), idx.clone()
    l2[mask == 0] = float("nan")
    idx2[mask == 0] = 3
    for a, b in zip(ref, M.moe_balance_loss(l2, idx2, n_seqs=2, token_mask=mask)):
        assert torch.equal(a, b)
    assert torch.equal(M.moe_balance_loss_backward(l2, ref[1], ref[3], d, token_mask=mask), g)
    assert not g[mask == 0].any()


def test_in_place_addition(M):
    T, E = 333, 130
    l, idx, mask = make(T, E, 4, 1, seed=2)
    _, counts, _, tokens = M.moe_balance_loss(l, idx, token_mask=mask)
    d = torch.tensor([0.3, 0.1], device="cuda")
    add = torch.randn(T, E, device="cuda")
    ref = M.moe_balance_loss_backward(l, counts, tokens, d, token_mask=mask, d_add=add)
    same = add.clone()
    M.moe_balance_loss_backward(l, counts, tokens, d, token_mask=mask, d_add=same, dlogits=same)
    assert torch.equal(same, ref)


@pytest.mark.parametrize("T,E,k,S", [(1, 16, 2, 1), (2048, 384, 8, 1), (900, 200, 6, 3), (20000, 64, 4, 1)])
def test_deterministic_and_order_free(M, T, E, k, S):
    l, idx, mask = make(T, E, k, S, seed=4)
    d = torch.tensor([1.0, 0.1], device="cuda")
    ws = M.workspace(M.moe_balance_loss_workspace_bytes(T, E, S))
    ws.zero_()
    ref = M.moe_balance_loss(l, idx, n_seqs=S, token_mask=mask, ws=ws)
    g = M.moe_balance_loss_backward(l, ref[1], ref[3], d, token_mask=mask)
    ws.fill_(255)
    for seed in range(4):
        M.moe_set_debug_options(M.MOE_DEBUG_PERMUTE_ORDER if seed else 0, seed)
        for a, b in zip(ref, M.moe_balance_loss(l, idx, n_seqs=S, token_mask=mask, ws=ws)):
            assert torch.equal(a, b)
        assert torch.equal(M.moe_balance_loss_backward(l, ref[1], ref[3], d, token_mask=mask), g)
    M.moe_set_debug_options(0, 0)


def test_whole_batch_over_two_halves(M):
    """Counts and tokens summed over two GPUs' shares: the gradients of both are those of one batch."""
    T, E, k = 512, 48, 4
    l, idx, mask = make(T, E, k, 1, seed=6, masked=False)
    d = torch.tensor([1.0, 0.5], device="cuda")
    _, counts, _, tokens = M.moe_balance_loss(l, idx, token_mask=mask)
    g = M.moe_balance_loss_backward(l, counts, tokens, d, token_mask=mask)
    half = [slice(0, 300), slice(300, T)]
    parts = [M.moe_balance_loss(l[h], idx[h], token_mask=mask[h].clone()) for h in half]
    assert torch.equal(parts[0][1] + parts[1][1], counts) and torch.equal(parts[0][3] + parts[1][3], tokens)
    for h in half:
        assert torch.equal(M.moe_balance_loss_backward(l[h].clone(), counts, tokens, d, token_mask=mask[h].clone()), g[h])


@pytest.mark.parametrize("T,E,k,S", [(4, 32, 2, 1), (2048, 384, 8, 1), (1200, 256, 8, 4)])
def test_graph_replays(M, T, E, k, S):
    """Forward and gradient captured and replayed, two graphs on one workspace in turn."""
    print(f"[balance graph] T={T} E={E}", flush=True)
    sets = [make(T, E, k, S, seed=30 + j) for j in range(2)]
    d = torch.tensor([1.0, 0.1], device="cuda")
    ws = M.workspace(M.moe_balance_loss_workspace_bytes(T, E, S))

    def step(l, idx, mask, out=None):
        o = M.moe_balance_loss(l, idx, n_seqs=S, token_mask=mask, ws=ws)
        return (*o, M.moe_balance_loss_backward(l, o[1], o[3], d, token_mask=mask))
    ref = [step(*s) for s in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*sets[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*s))
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            for t in o:
                t.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, r in zip(outs, ref):
            for a, b in zip(o, r):
                assert torch.equal(a, b)
        step(*sets[1])
        torch.cuda.synchronize()


def test_more_rows_than_a_grid_of_waves(M):
    """2^22 - 1 rows, the most a call takes."""
    T, E, k = (1 << 22) - 1, 8, 2
    l = torch.randn(T, E, device="cuda")
    idx = l.topk(k, dim=1).indices.int().contiguous()
    losses, counts, probs, tokens = M.moe_balance_loss(l, idx)
    assert int(tokens) == T and torch.equal(counts[0].long(), torch.bincount(idx.reshape(-1).long(), minlength=E))
    p = torch.softmax(l.double(), 1).mean(0)
    assert float((probs[0].double() - p).abs().max()) < 4096 * U
    d = torch.tensor([1.0, 0.1], device="cuda")
    g = M.moe_balance_loss_backward(l, counts, tokens, d)
    sub = M.moe_balance_loss_backward(l[-7:].clone(), counts, tokens, d)
    assert torch.equal(g[-7:], sub)
