"""Pins of oracle/block.py: differences, brute force, library routines, other forms of the
same formula - never the oracle's own steps."""
import itertools

import numpy as np
import pytest
import torch

from oracle import block as B
from oracle import route


def _diff(f, x, h=1e-5):
    """Central differences of the scalar f at x, element by element."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


def test_norm_against_torch():
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.normal(size=(5, 64))).to(torch.bfloat16)
    r = torch.from_numpy(rng.normal(size=(5, 64))).to(torch.bfloat16)
    w = torch.from_numpy(rng.normal(size=64))
    s, y = B.add_rmsnorm(x.double().numpy(), w.numpy(), 1e-6, r.double().numpy())
    ref_s = (x.double() + r.double()).to(torch.bfloat16).double()
    assert np.array_equal(s, ref_s.numpy())
    ref = torch.nn.functional.rms_norm(ref_s, (64,), w, 1e-6)
    assert np.allclose(y, ref.numpy(), rtol=1e-13, atol=0)


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(1)
    s, dy, ds = (rng.normal(size=(3, 8)) for _ in range(3))
    w = rng.normal(size=8)
    f = lambda s_, w_: (dy * B.add_rmsnorm(s_, w_, 1e-3)[1]).sum() + (ds * s_).sum()  # noqa: E731
    dx, dw = B.add_rmsnorm_backward(s, w, dy, 1e-3, ds)
    assert np.allclose(dx, _diff(lambda v: f(v, w), s), atol=1e-8)
    assert np.allclose(dw, _diff(lambda v: f(s, v), w), atol=1e-8)


def test_route_scored_softmax_is_the_plain_route():
    l = np.random.default_rng(2).normal(size=(40, 24)).astype(np.float32)
    a, aw = route(l, 5)
    b, bw = B.route_scored(l, 5)
    assert np.array_equal(a, b) and np.allclose(aw, bw, rtol=1e-12)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
def test_route_scored_by_brute_force(score, group_top):
    """Groups and experts as the subset with the largest total, over all subsets."""
    rng = np.random.default_rng(3)
    E, G, tg, k = 12, 4, 2, 3
    size = E // G
    l = rng.normal(size=(20, E)).astype(np.float32)
    b = (0.3 * rng.normal(size=E)).astype(np.float32)
    idx, w = B.route_scored(l, k, b, score, G, tg, group_top, True, 2.5)
    for t in range(20):
        z = torch.from_numpy(l[t]).double()
        p = (torch.softmax(z, 0) if score == "softmax" else torch.sigmoid(z)).numpy()
        c = p + b.astype(np.float64)
        value = lambda g: max(sum(s) for s in itertools.combinations(c[g * size:(g + 1) * size], group_top))  # noqa: E731
        groups = max(itertools.combinations(range(G), tg), key=lambda q: sum(value(g) for g in q))
        pool = [e for e in range(E) if e // size in groups]
        chosen = max(itertools.combinations(pool, k), key=lambda q: sum(c[e] for e in q))
        assert sorted(idx[t]) == sorted(chosen)
        assert all(c[idx[t][i]] >= c[idx[t][i + 1]] for i in range(k - 1))
        assert np.allclose(w[t], 2.5 * p[idx[t]] / p[list(chosen)].sum(), rtol=1e-12)


def test_route_scored_masks_and_ties():
    l = np.zeros((1, 6), dtype=np.float32)
    l[0, 2] = -np.inf
    l[0, 0] = np.nan
    idx, w = B.route_scored(l, 6, renorm=False)
    assert idx.tolist() == [[1, 3, 4, 5, 0, 2]] and np.allclose(w, [[0.25] * 4 + [0, 0]])
    idx, w = B.route_scored(np.full((1, 4), -np.inf, dtype=np.float32), 3, score="sigmoid")
    assert idx.tolist() == [[0, 1, 2]] and not w.any()
    # a group with nothing to offer ranks last, one with a single expert by that expert
    l = np.array([[-np.inf, -np.inf, 3.0, -np.inf, 1.0, 1.0]], dtype=np.float32)
    idx, _ = B.route_scored(l, 2, score="sigmoid", groups=3, top_groups=2, group_top=2)
    assert idx.tolist() == [[2, 4]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_scored_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(4)
    l = rng.normal(size=(4, 10))
    idx = np.stack([rng.permutation(10)[:3] for _ in range(4)])
    dw = rng.normal(size=(4, 3))

    def f(v):                                      # selection held fixed, torch's own scores
        z = torch.from_numpy(v)
        p = torch.softmax(z, 1) if score == "softmax" else torch.sigmoid(z)
        w = p.gather(1, torch.from_numpy(idx))
        w = w / w.sum(1, keepdim=True) if renorm else w
        return float((1.5 * w * torch.from_numpy(dw)).sum())

    l32 = l.astype(np.float32).astype(np.float64)
    got = B.route_scored_backward(l32, idx, dw, score, renorm, 1.5)
    assert np.allclose(got, _diff(f, l32), atol=1e-8)


def test_int8_rows():
    v = np.array([[127.0, 0.5, 1.5, -2.5, -127.0], [0.0] * 5, [2.0 ** -101] * 5])
    c, s = B.int8_rows(v)
    assert c.tolist() == [[127, 0, 2, -2, -127], [0] * 5, [0] * 5] and s.tolist() == [1.0, 0.0, 0.0]


def test_experts_int8_against_a_scalar_loop():
    rng = np.random.default_rng(5)
    T, H, I, E, k = 3, 6, 4, 3, 2
    x = rng.integers(-127, 128, size=(T, H))
    xs = rng.uniform(0.01, 0.02, size=T)
    wg, wd = rng.integers(-127, 128, size=(E, 2 * I, H)), rng.integers(-127, 128, size=(E, H, I))
    sg, sd = rng.uniform(1e-3, 2e-3, size=(E, 2 * I)), rng.uniform(1e-3, 2e-3, size=(E, H))
    idx = np.array([[0, 2], [1, -1], [7, 9]])
    w = rng.uniform(size=(T, k))
    got, _ = B.experts_int8(x, xs, wg, sg, wd, sd, idx, w)
    for t in range(T):
        ref = np.zeros(H)
        for j in range(k):
            e = idx[t, j]
            if not 0 <= e < E:
                continue
            a = []
            for n in range(I):
                g = xs[t] * sg[e, n] * sum(int(x[t, c]) * int(wg[e, n, c]) for c in range(H))
                u = xs[t] * sg[e, I + n] * sum(int(x[t, c]) * int(wg[e, I + n, c]) for c in range(H))
                a.append(g * torch.sigmoid(torch.tensor(g, dtype=torch.float64)).item() * u)
            top = max(abs(v) for v in a)
            q = [round(v * 127 / top) for v in a]
            for h in range(H):
                ref[h] += w[t, j] * top / 127 * sd[e, h] * sum(q[n] * int(wd[e, h, n]) for n in range(I))
        assert np.allclose(got[t], ref, rtol=1e-12, atol=1e-15)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_scored_infinite_biases(score):
    inf = np.inf
    l = np.array([[0.1, 0.2, -3.0, -3.0]], dtype=np.float32)
    b = np.array([5.0, -inf, 0.0, 0.0])
    # c of -inf: the group that counts it scores -inf, the one that counts one expert does not
    assert B.route_scored(l, 1, b, score, 2, 1, 2)[0].tolist() == [[2]]
    assert B.route_scored(l, 1, b, score, 2, 1, 1)[0].tolist() == [[0]]
    assert B.route_scored(l, 4, b, score)[0].tolist() == [[0, 2, 3, 1]]
    # above masked experts and groups, by index among equals
    l = np.array([[-inf, -inf, 1.0, 2.0, 0.0, 0.0]], dtype=np.float32)
    b = np.array([9.0, 9.0, -inf, -inf, -inf, -inf])
    assert B.route_scored(l, 2, b, score, 3, 1, 2)[0].tolist() == [[2, 3]]
    assert B.route_scored(l, 6, b, score)[0].tolist() == [[2, 3, 4, 5, 0, 1]]
    idx, w = B.route_scored(l, 4, b, score, 3, 2, 2)
    assert idx.tolist() == [[2, 3, 4, 5]] and np.all(w > 0)
