"""Pins of the oracle's E2M1 codec, of its MXFP4 blocks and of the layer on them: the definition by
search over exact rationals, library routines, the INT8 layer's arithmetic where both are exact."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import block as B
from oracle import formats as F

GRID = [Fraction(0), Fraction(1, 2), Fraction(1), Fraction(3, 2), Fraction(2), Fraction(3), Fraction(4), Fraction(6)]


def _nearest(x):
    """Code of the nearest grid value by search; of two as near, the even one."""
    f = abs(Fraction(x))
    best = min(range(8), key=lambda c: (abs(GRID[c] - f), c & 1))
    return best | (8 if np.signbit(x) else 0)


def test_e2m1_values_follow_the_definition():
    for c in range(16):
        ex, man = (c >> 1) & 3, c & 1
        v = Fraction(man, 2) if ex == 0 else (1 + Fraction(man, 2)) * Fraction(2) ** (ex - 1)
        assert Fraction(float(F.e2m1_decode(c))) == (-v if c & 8 else v)


def test_e2m1_encode_by_search():
    rng = np.random.default_rng(0)
    edges = [float((a + b) / 2) for a, b in zip(GRID, GRID[1:])] + [float(g) for g in GRID]
    v = np.array(edges + [np.nextafter(e, 9) for e in edges] + [np.nextafter(e, -9) for e in edges]
                 + list(rng.uniform(0, 8, 500)) + [7.0, 100.0, 1e300, 0.0])
    v = np.concatenate([v, -v])
    got = F.e2m1_encode(v)
    assert [int(c) for c in got] == [_nearest(x) for x in v]


def test_mxfp4_blocks_by_search():
    rng = np.random.default_rng(1)
    v = rng.normal(size=(6, 96)) * np.exp2(rng.integers(-30, 30, size=(6, 96)))
    v[0, :32] = 0
    v[1, 32:64] = 2.0 ** -140
    v[2, :32] = 2.0 ** 100
    packed, s = F.mxfp4_quantize(v)
    for r in range(6):
        for b in range(3):
            blk = v[r, 32 * b:32 * b + 32]
            top = max(abs(Fraction(x)) for x in blk)
            e = -127
            while top and e < 127 and Fraction(2) ** (e + 3) <= top:
                e += 1
            assert s[r, b] == e + 127
            for i, x in enumerate(blk):
                c = packed[r, 16 * b + i // 2] >> (4 * (i % 2)) & 15
                assert c == _nearest(float(Fraction(x) / Fraction(2) ** e))
    back = F.mxfp4_dequantize(packed, s)
    assert back.shape == v.shape and np.array_equal(F.mxfp4_quantize(back)[0][3:], packed[3:])


def test_experts_against_torch():
    rng = np.random.default_rng(2)
    T, H, I, E, k = 7, 64, 32, 3, 2
    x = rng.integers(-4, 5, (T, H)) / 2.0
    wg, wd = rng.integers(-3, 4, (E, 2 * I, H)) / 8.0, rng.integers(-3, 4, (E, H, I)) / 4.0
    idx = rng.integers(-1, E, (T, k))
    w = rng.random((T, k))
    for four in (False, True):
        out, slack = B.experts_mxfp4(x, wg, wd, idx, w, four)
        ref = torch.zeros(T, H, dtype=torch.float64)
        for t in range(T):
            for j in range(k):
                e = idx[t, j]
                if e < 0:
                    continue
                gu = torch.from_numpy(wg[e] @ x[t])
                a = torch.nn.functional.silu(gu[:I]) * gu[I:]
                top = float(a.abs().max())
                s = 2.0 ** (np.floor(np.log2(top)) - (2 if four else 8))
                if four:
                    h = torch.tensor([float(GRID[_nearest(float(v) / s) & 7]) * np.sign(float(v)) for v in a]) * s
                else:
                    h = (a / s).clamp(-448, 448).float().to(torch.float8_e4m3fn).double() * s
                ref[t] += w[t, j] * (torch.from_numpy(wd[e]) @ h.double())
        # the float32 cast may move a value next to a border of E4M3: none here
        assert np.allclose(out, ref.numpy(), rtol=1e-12, atol=1e-12)
        assert (slack >= 0).all() and slack.max() < 0.3 * np.abs(out).max()


def test_slack_covers_a_small_error_of_the_activations():
    rng = np.random.default_rng(3)
    T, H, I = 5, 64, 64
    x, wg, wd = rng.normal(size=(T, H)), rng.normal(size=(1, 2 * I, H)) / 8, rng.normal(size=(1, H, I)) / 8
    idx, w = np.zeros((T, 1), dtype=int), np.ones((T, 1))
    for four, rel in ((True, 2.0 ** -23), (False, 2.0 ** -12)):
        out, slack = B.experts_mxfp4(x, wg, wd, idx, w, four)
        for seed in range(20):
            move = 1 + rel * np.random.default_rng(seed).uniform(-1, 1, wg.shape)
            assert np.all(np.abs(B.experts_mxfp4(x, wg * move, wd, idx, w, four)[0] - out) <= slack * (1 + 1e-9))


def _loss(l, idx, seqs, mask, score, d):
    return float(np.dot(d, B.balance_loss(l, idx, score, seqs, mask)[0]))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_against_torch_autograd(score):
    rng = np.random.default_rng(4)
    T, E, k, S = 12, 7, 3, 3
    l = rng.normal(size=(T, E)).astype(np.float32)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    idx[4, 1] = E
    idx[5, 0] = -1
    mask = np.ones(T, dtype=np.uint8)
    mask[[1, 6]] = 0
    mask[8:12] = 0                                         # the last sequence is empty
    d = np.array([0.7, -0.3])
    z = torch.tensor(l, dtype=torch.float64, requires_grad=True)
    p = torch.softmax(z, 1) if score == "softmax" else torch.sigmoid(z) / torch.sigmoid(z).sum(1, keepdim=True)
    on = torch.tensor(mask, dtype=torch.bool)
    total = 0.0
    for s in range(S):
        rows = [t for t in range(4 * s, 4 * s + 4) if on[t]]
        if not rows:
            continue
        c = np.bincount([e for t in rows for e in idx[t] if 0 <= e < E], minlength=E)
        total = total + (p[rows].mean(0) * torch.tensor(E * c / c.sum())).sum()
    lse = torch.logsumexp(z, 1)[on]
    value = d[0] * total / S + d[1] * (lse ** 2).mean()
    value.backward()
    losses, counts, probs, tokens = B.balance_loss(l, idx, score, S, mask)
    assert np.isclose(np.dot(d, losses), float(value), rtol=1e-6)
    assert tokens.tolist() == [3, 3, 0] and counts[2].sum() == 0 and not probs[2].any()
    g = B.balance_loss_backward(l, counts, tokens, d, score, mask)
    assert np.allclose(g, z.grad.numpy(), atol=1e-12)
    add = rng.normal(size=(T, E))
    assert np.allclose(B.balance_loss_backward(l, counts, tokens, d, score, mask, add), add + g, atol=1e-15)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_against_differences(score):
    rng = np.random.default_rng(5)
    T, E, k = 4, 5, 2
    l = rng.normal(size=(T, E))
    l[2, 3] = -np.inf                                      # a masked expert
    l[3] = -np.inf                                         # a token without experts
    idx = np.argsort(-l, axis=1)[:, :k]
    d = np.array([1.0, 0.5])
    _, counts, _, tokens = B.balance_loss(l, idx, score)
    g = B.balance_loss_backward(l, counts, tokens, d, score)
    assert not g[3].any() and g[2, 3] == 0
    for t in range(3):
        for e in range(E):
            if not np.isfinite(l[t, e]):
                continue
            h = 2.0 ** -7                                  # (the oracle reads logits as FP32)
            a, b = np.float32(l[t, e]) + np.float32(h), np.float32(l[t, e]) - np.float32(h)
            up, down = l.copy(), l.copy()
            up[t, e], down[t, e] = a, b
            slope = (_loss(up, idx, 1, None, score, d) - _loss(down, idx, 1, None, score, d)) / (float(a) - float(b))
            assert abs(slope - g[t, e]) < 1e-4             # third derivatives of order 1 times h^2
