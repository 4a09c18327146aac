"""moe_route_scored and its backward against the FP64 oracle: indices exact, weights and
gradients to FP32's error (an exponential within 2 steps, a division, and sums of up to
1024 positive terms over 16 adds per lane and 6 across lanes: below 40 * 2^-24)."""
import numpy as np
import pytest
import torch

from oracle import block as B

pytestmark = pytest.mark.gpu

REL = 40 * 2.0 ** -24


@pytest.fixture(scope="module")
def M():
    import mixture_experts_ffn_07_amd as M
    yield M
    M.moe_set_debug_options(0, 0)


def _score(M, name):
    return M.MOE_SCORE_SOFTMAX if name == "softmax" else M.MOE_SCORE_SIGMOID


def _run(M, l, k, bias=None, score="softmax", G=1, tg=1, gt=1, renorm=True, scale=1.0, what=""):
    T, E = l.shape
    print(f"[route scored] {what} T={T} E={E} k={k} {score} G={G}/{tg}/{gt} bias={bias is not None} "
          f"renorm={renorm}", flush=True)
    idx, w = M.moe_route_scored(l.cuda(), k, bias=None if bias is None else bias.cuda(),
                                score=_score(M, score), n_groups=G, topk_groups=tg, group_top=gt,
                                renormalize=renorm, scale=scale)
    ridx, rw = B.route_scored(l.numpy(), k, None if bias is None else bias.numpy(), score, G, tg, gt,
                              renorm, scale)
    assert np.array_equal(idx.cpu().numpy(), ridx)
    assert np.all(np.abs(w.double().cpu().numpy() - rw) <= np.abs(rw) * REL + 1e-37)
    return idx, w


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k,G,tg,gt", [
    (1, 8, 2, 1, 1, 1), (5, 3, 3, 1, 1, 1), (33, 64, 6, 8, 3, 2), (65, 100, 7, 10, 4, 1),
    (17, 384, 8, 8, 4, 2), (9, 1024, 32, 64, 16, 2), (130, 256, 1, 2, 1, 2), (6, 60, 10, 60, 10, 2),
    (11, 511, 10, 7, 2, 1), (3, 1, 1, 1, 1, 2), (4, 65, 32, 1, 1, 1), (7, 96, 3, 3, 3, 2)])
def test_route_scored(M, score, bias, renorm, T, E, k, G, tg, gt):
    g = torch.Generator().manual_seed(T * 31 + E)
    l = torch.randn(T, E, generator=g) * 2
    b = 0.2 * torch.randn(E, generator=g) if bias else None
    _run(M, l, k, b, score, G, tg, gt, renorm, 1.0 if T % 2 else 2.5)


def test_route_scored_is_route_topk_without_options(M):
    l = torch.randn(500, 384, device="cuda")
    l[::3] = (l[::3] * 2).round() / 2                   # many ties
    a = M.moe_route_topk(l, 8)
    b = M.moe_route_scored(l, 8)
    assert torch.equal(a[0], b[0]) and (a[1] - b[1]).abs().max() <= 4 * 2.0 ** -24


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,tg,gt", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
def test_route_scored_ties_take_the_lowest_index(M, score, G, tg, gt):
    g = torch.Generator().manual_seed(5)
    l = (torch.randint(-2, 3, (200, 40), generator=g) / 2).float()
    b = (torch.randint(-1, 2, (40,), generator=g) / 4).float()
    l[::2][l[::2] == 0] = -0.0
    _run(M, l, 7, None, score, G, tg, gt, what="ties")
    _run(M, l, 7, b, score, G, tg, gt, what="ties")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("E,k,G,tg", [(256, 8, 1, 1), (384, 8, 8, 4), (130, 5, 1, 1), (1024, 32, 1, 1)])
def test_route_scored_equal_logits_across_a_lane(M, score, bias, E, k, G, tg):
    """Ties among experts that one lane holds (several per lane), of value 0, near 0 and not 0."""
    l = torch.zeros(7, E)
    l[1] = 0.75
    l[2] = -2.5
    l[3, ::3] = 1e-40                                  # below FP32's normal range, above 0
    l[4, 1::2] = -0.0
    l[5, 5:] = -1e-39
    l[6, ::2] = 2.0 ** -126
    _run(M, l, k, torch.zeros(E) if bias else None, score, G, tg, 2, what="equal logits")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("T,E,k,G,tg,gt", [(9, 1023, 16, 33, 7, 2), (6, 1020, 9, 17, 3, 2), (5, 1017, 9, 9, 2, 1),
                                           (8, 64, 2, 64, 5, 2), (4, 1024, 32, 2, 1, 2)])
def test_route_scored_odd_groups(M, score, bias, T, E, k, G, tg, gt):
    g = torch.Generator().manual_seed(E + G)
    l = torch.randn(T, E, generator=g) * 2
    _run(M, l, k, 0.2 * torch.randn(E, generator=g) if bias else None, score, G, tg, gt, True, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("G,tg,gt", [(1, 1, 1), (8, 3, 2), (8, 3, 1)])
def test_route_scored_masks(M, score, bias, renorm, G, tg, gt):
    g = torch.Generator().manual_seed(6)
    T, E, k = 64, 64, 6
    l = torch.randn(T, E, generator=g)
    u = torch.rand(T, E, generator=g)
    l[u < 0.5] = -float("inf")
    l[(u > 0.5) & (u < 0.55)] = float("nan")
    l[(u > 0.55) & (u < 0.6)] = torch.finfo(torch.float32).min
    l[(u > 0.6) & (u < 0.65)] = torch.finfo(torch.bfloat16).min
    l[0] = -float("inf")                                # nothing left
    l[1] = float("nan")
    l[2] = torch.finfo(torch.float32).min
    l[3] = -float("inf")
    l[3, 40] = 1.5                                      # one expert left
    l[4] = -float("inf")
    l[4, 9], l[4, 63] = -80.0, -85.0                    # scores near the end of FP32
    b = 0.2 * torch.randn(E, generator=g) if bias else None
    idx, w = _run(M, l, k, b, score, G, tg, gt, renorm, what="masks")
    assert not w[:3].any()
    i = idx.cpu().numpy()
    assert i.min() >= 0 and i.max() < E and all(len(set(r)) == k for r in i)


def test_route_scored_extreme_logits(M):
    l = torch.randn(6, 20)
    l[0, 3] = float("inf")
    l[1, 3] = l[1, 4] = float("inf")
    l[2] = 100 + 0.5 * torch.arange(20)
    l[3] = -100 - 0.01 * torch.arange(20)               # sigmoid scores of 4e-44: renormalised in FP32
    l[4, :10] = torch.finfo(torch.float32).max
    for score in ("softmax", "sigmoid"):
        for rows in (slice(0, 3), slice(4, 6)):
            _run(M, l[rows], 4, None, score, renorm=True, what="extremes")
            _run(M, l[rows], 4, None, score, renorm=False, what="extremes")
    idx, w = M.moe_route_scored(l.cuda(), 4, score=_score(M, "sigmoid"))
    assert torch.isfinite(w).all() and idx[3].tolist() == [0, 1, 2, 3]


def test_route_scored_near_ties_of_the_biased_choice(M):
    """Pairs of experts whose c differ by parts in 1e9: FP32 scores would not tell them apart."""
    g = torch.Generator().manual_seed(8)
    T, E = 300, 128
    l = torch.randn(T, E, generator=g)
    b = 0.1 * torch.randn(E, generator=g)
    p = torch.sigmoid(l[:, ::2].double())
    want = p + b[::2].double() - b[1::2].double()       # score that ties the neighbour's c
    want = want.clamp(0.05, 0.95)
    l[:, 1::2] = torch.log(want / (1 - want)).float()   # (rounded: c differs in its 8th to 9th digit)
    _run(M, l, 8, b, "sigmoid", what="near ties")


def test_route_scored_empty_batch_and_large(M):
    idx, w = M.moe_route_scored(torch.empty(0, 8, device="cuda"), 2)
    assert idx.shape == (0, 2) and w.shape == (0, 2)
    g = torch.Generator(device="cuda").manual_seed(9)
    l = torch.randn(70001, 16, generator=g, device="cuda")
    idx, w = M.moe_route_scored(l, 2, score=_score(M, "sigmoid"), renormalize=False)
    top = l.topk(2, dim=1)
    assert torch.equal(idx.long(), top.indices)         # (no ties among these)
    assert (w - torch.sigmoid(top.values.double())).abs().max() <= REL


BACK = [(1, 8, 2), (5, 3, 3), (33, 64, 6), (65, 100, 7), (17, 384, 8), (9, 1024, 32), (130, 256, 1), (6, 511, 10)]


def _back(M, l, idx, dw, score, renorm, scale):
    got = M.moe_route_scored_backward(l.cuda(), idx.cuda(), dw.cuda(), score=_score(M, score),
                                      renormalize=renorm, scale=scale).double().cpu().numpy()
    ref = B.route_scored_backward(l.numpy(), idx.numpy(), dw.numpy(), score, renorm, scale)
    p, _ = B.scores(l.numpy(), score)
    # size of the terms that are subtracted: p_e (|dw_e| + sum w |dw|), over the scores' sum if renormalised
    mag = np.zeros_like(ref)
    for t in range(l.shape[0]):
        sel = [int(e) for e in idx[t] if 0 <= e < l.shape[1]]
        a = {}
        for e, d in zip(idx[t].tolist(), dw[t].tolist()):
            if 0 <= e < l.shape[1]:
                a[e] = a.get(e, 0.0) + abs(d)
        z = sum(p[t, e] for e in sel) if renorm else 1.0
        mean = sum(p[t, e] * v for e, v in a.items()) / (z if z > 0 else 1.0)
        for e in (range(l.shape[1]) if score == "softmax" and not renorm else sel):
            mag[t, e] = abs(scale) * p[t, e] / (z if z > 0 else 1.0) * (a.get(e, 0.0) + mean)
    assert np.all(np.isfinite(got))
    # the oracle's own error: p_e (dp_e - sum dp p) in FP64, where for renormalised softmax scores
    # the sum is 0 but for the rounding of at most 3 * 32 terms, each no larger than the row's mag
    # summed: below 128 * 2^-53 of that
    own = mag.sum(axis=1, keepdims=True) * 2.0 ** -46
    assert np.all(np.abs(got - ref) <= 2 * REL * mag + own + 1e-37)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", BACK)
def test_route_scored_backward(M, score, renorm, T, E, k):
    print(f"[route scored backward] T={T} E={E} k={k} {score} renorm={renorm}", flush=True)
    g = torch.Generator().manual_seed(T + E)
    l = torch.randn(T, E, generator=g) * 2
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    _back(M, l, idx, torch.randn(T, k, generator=g), score, renorm, 2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_scored_backward_masks_and_ids(M, score, renorm):
    g = torch.Generator().manual_seed(3)
    l = torch.randn(8, 20, generator=g)
    l[0] = -float("inf")
    l[1, :15] = -float("inf")
    l[2, 4] = float("nan")
    l[3, 1] = torch.finfo(torch.float32).min
    idx = torch.stack([torch.randperm(20, generator=g)[:5] for _ in range(8)]).int()
    idx[1] = torch.tensor([0, 1, 15, 16, 17])            # two masked ones among the selected
    idx[2, 0] = 4
    idx[3, 2] = 1
    idx[5, 3] = -1                                       # ids that are no expert
    idx[6] = torch.tensor([20, -7, 2 ** 31 - 1, 3, 9])
    _back(M, l, idx, torch.randn(8, 5, generator=g), score, renorm, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_scored_gradient_against_differences(M, score, renorm):
    """<dlogits, v> against the difference of sum(dw w) along v, the selection held fixed."""
    g = torch.Generator().manual_seed(12)
    T, E, k = 10, 48, 5
    l, v, dw = torch.randn(T, E, generator=g), torch.randn(T, E, generator=g), torch.randn(T, k, generator=g)
    idx, _ = M.moe_route_scored(l.cuda(), k, score=_score(M, score), renormalize=renorm, scale=1.5)
    d = M.moe_route_scored_backward(l.cuda(), idx, dw.cuda(), score=_score(M, score), renormalize=renorm, scale=1.5)
    i = idx.long().cpu()

    def f(z):
        p = torch.softmax(z, 1) if score == "softmax" else torch.sigmoid(z)
        w = p.gather(1, i)
        w = w / w.sum(1, keepdim=True) if renorm else w
        return float((1.5 * w * dw.double()).sum())

    h = 1e-4
    num = (f(l.double() + h * v.double()) - f(l.double() - h * v.double())) / (2 * h)
    got = float((d.double().cpu() * v.double()).sum())
    tol = float((d.double().cpu() * v.double()).abs().sum()) * 1e-5 + 1e-6
    assert abs(got - num) <= tol


def test_route_scored_is_deterministic_and_order_free(M):
    l = torch.randn(999, 384, device="cuda")
    b = 0.1 * torch.randn(384, device="cuda")
    dw = torch.randn(999, 8, device="cuda")

    def call():
        i, w = M.moe_route_scored(l, 8, bias=b, score=_score(M, "sigmoid"), n_groups=8, topk_groups=4, group_top=2)
        return i, w, M.moe_route_scored_backward(l, i, dw, score=_score(M, "sigmoid"))
    ref = call()
    for seed in range(4):
        M.moe_set_debug_options(M.MOE_DEBUG_PERMUTE_ORDER if seed else 0, seed)
        for a, c in zip(ref, call()):
            assert torch.equal(a.view(torch.int32), c.view(torch.int32))
    M.moe_set_debug_options(0, 0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_scored_weights_of_low_logits(M, score, renorm):
    """Selected logits tens below the largest (a bias picks them): the difference's rounding
    alone, half a step of it, would be up to 64 steps of the exponential.  All logits far
    below 0 and above the masks: sigmoid scores that vanish in FP32 still have their ratio."""
    g = torch.Generator().manual_seed(3)
    l = -torch.rand(64, 96, generator=g) * 65
    l[:, 0] = 6.28125 + torch.rand(64, generator=g)
    b = torch.zeros(96)
    b[64:] = 2.0
    _run(M, l, 32, b, score, renorm=renorm, what="low")
    _run(M, l, 96 // 3, None, score, renorm=renorm, what="low")
    idx, w = M.moe_route_scored((l - 600).cuda(), 8, score=_score(M, "sigmoid"), renormalize=True)
    top = torch.gather((l - 600).double(), 1, idx.cpu().long())
    ref = torch.softmax(top, 1)
    assert ((w.cpu().double() - ref).abs() <= ref * REL + 1e-37).all()


def test_route_scored_backward_of_low_logits(M):
    """Softmax, not renormalised: the gradient of experts tens below the largest."""
    g = torch.Generator().manual_seed(4)
    l = -torch.rand(32, 96, generator=g) * 65
    l[:, 0] = 6.28125
    idx, _ = M.moe_route_scored(l.cuda(), 8, renormalize=False)
    d = torch.randn(32, 8, generator=g)
    got = M.moe_route_scored_backward(l.cuda(), idx, d.cuda(), renormalize=False).cpu().double()
    p = torch.softmax(l.double(), 1)
    sel = idx.cpu().long()
    mean = (torch.gather(p, 1, sel) * d).sum(1, keepdim=True)
    full = torch.zeros(32, 96, dtype=torch.float64).scatter(1, sel, d.double())
    size = full.abs() + (torch.gather(p, 1, sel) * d.abs()).sum(1, keepdim=True)   # (the terms' magnitudes)
    assert ((got - p * (full - mean)).abs() <= 2 * REL * p * size + 1e-37).all()


def test_route_scored_most_tokens(M):
    T, E, k = (1 << 22) - 1, 4, 2
    l = torch.randn(T, E, device="cuda")
    idx, w = M.moe_route_scored(l, k)
    d = torch.randn(T, k, device="cuda")
    g = M.moe_route_scored_backward(l, idx, d)
    for a in (0, 1 << 21, T - 9):
        n = lambda t: t[a:a + 9].clone()  # noqa: E731
        i1, w1 = M.moe_route_scored(n(l), k)
        assert torch.equal(n(idx), i1) and torch.equal(n(w), w1)
        assert torch.equal(n(g), M.moe_route_scored_backward(n(l), i1, n(d)))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,tg,gt", [(1, 1, 1), (2, 1, 2), (8, 3, 1), (8, 3, 2), (32, 9, 2)])
def test_route_scored_infinite_biases(M, score, G, tg, gt):
    """A bias of -inf: the expert comes after all others that take part, before the masked
    ones, and a group that has to count it scores -inf, still above a group without experts."""
    if G == 2:                                          # one group's second largest is the -inf
        l = torch.tensor([[0.1, 0.2, -3.0, -3.0]])
        idx, _ = _run(M, l, 1, torch.tensor([5.0, -float("inf"), 0.0, 0.0]), score, 2, 1, 2, what="-inf")
        assert idx.tolist() == [[2]]
    g = torch.Generator().manual_seed(G + gt)
    T, E, k = 96, 64, 6
    l = torch.randn(T, E, generator=g)
    b = 0.2 * torch.randn(E, generator=g)
    b[torch.rand(E, generator=g) < 0.5] = -float("inf")
    _run(M, l, k, b, score, G, tg, gt, what="-inf")
    u = torch.rand(T, E, generator=g)
    l[u < 0.5] = -float("inf")
    l[:4] = -float("inf")
    l[2, 63] = l[3, 3] = 1.0
    l[8:16, :32] = -float("inf")
    _run(M, l, k, b, score, G, tg, gt, renorm=False, what="-inf and masks")
    _run(M, l, k, torch.full((E,), -float("inf")), score, G, tg, gt, what="all -inf and masks")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("sign", [1, -1])
def test_route_scored_group_sums_past_fp32(M, score, sign):
    """Two biases whose sum FP32 does not hold: group scores are compared all the same."""
    g = torch.Generator().manual_seed(10)
    l = torch.randn(8, 4, generator=g)
    b = sign * torch.tensor([2e38, 2e38, 3e38, 3e38])
    idx, _ = _run(M, l, 1, b, score, 2, 1, 2, what="sums past FP32")
    assert all(i >= 2 for i in idx[:, 0].tolist()) == (sign > 0)
    _run(M, l, 1, b.flip(0), score, 2, 1, 2, what="sums past FP32")
    # both groups just past FP32's range, the second by more
    hi, lo = 1.5 * 2.0 ** 127 + 7 * 2.0 ** 104, 2.0 ** 126 - 2.0 ** 102
    b = sign * torch.tensor([hi, lo, hi + 2.0 ** 107, lo])
    idx, _ = _run(M, l, 1, b, score, 2, 1, 2, what="sums just past FP32")
    assert idx[:, 0].tolist() == ([2] * 8 if sign > 0 else [1] * 8)
    l = torch.randn(40, 64, generator=g)
    b = sign * (1.6 + 1.8 * torch.rand(64, generator=g)) * 1e38
    b[torch.rand(64, generator=g) < 0.3] = 0.5
    for G, tg in ((4, 2), (16, 5), (32, 7)):
        _run(M, l, 2, b, score, G, tg, 2, what="sums past FP32")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [64.0, 1000.0, 1e5])
def test_route_scored_group_sums_that_cancel(M, score, size):
    """Each group's two largest have large biases of opposite sign: the sum keeps the rounding
    of its terms (2^-24 of the bias), far above that of the sum itself.  Groups apart by
    about that much."""
    g = torch.Generator().manual_seed(int(size))
    T, G = 400, 8
    l = torch.randn(T, 1, 2, generator=g).expand(T, G, 2) + size * 2.0 ** -22 * torch.randn(T, G, 2, generator=g)
    b = torch.tensor([size, -size]).repeat(G)
    _run(M, l.reshape(T, 2 * G).contiguous(), 2, b, score, G, 1, 2, what=f"cancelling {size}")
    # groups of three, the third masked or far below
    l3 = torch.full((T, G, 3), -float("inf"))
    l3[:, :, :2] = l
    l3[::2, :, 2] = -4.0
    b3 = torch.tensor([size, -size, -3 * size]).repeat(G)
    _run(M, l3.reshape(T, 3 * G), 4, b3, score, G, 3, 2, what=f"cancelling {size}")
