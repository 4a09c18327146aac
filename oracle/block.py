"""The operators around the routed experts, written out in float64: residual sum
and RMS norm with its gradients, routing by scores with its gradient, INT8 rows
and the INT8 experts, the experts with MXFP4 weights, and the router's balance loss
with its gradient.  Plain NumPy, one token or one expert at a time where that
reads better."""
from __future__ import annotations

import numpy as np

from . import formats as F
from .formats import bf16_round

MASK = float(np.float32(-3.3895313892515355e38))   # BF16's lowest finite value
FLT_MAX = float(np.finfo(np.float32).max)


def add_rmsnorm(x, weight, eps: float, residual=None):
    """(s, y): s = the BF16-rounded sum (x without a residual), y = s w / rms(s)."""
    s = np.asarray(x, dtype=np.float64)
    if residual is not None:
        s = bf16_round(s + np.asarray(residual, dtype=np.float64))
    rms = np.sqrt((s * s).sum(axis=1, keepdims=True) / s.shape[1] + eps)
    return s, s / rms * np.asarray(weight, dtype=np.float64)


def add_rmsnorm_backward(s, weight, dy, eps: float, ds=None):
    """(dx, dweight) for sum(dy y) + sum(ds s)."""
    s, w, dy = (np.asarray(v, dtype=np.float64) for v in (s, weight, dy))
    H = s.shape[1]
    rms = np.sqrt((s * s).sum(axis=1, keepdims=True) / H + eps)
    g = w * dy
    dx = g / rms - s * (g * s).sum(axis=1, keepdims=True) / (H * rms ** 3)
    if ds is not None:
        dx = dx + np.asarray(ds, dtype=np.float64)
    return dx, (dy * s / rms).sum(axis=0)


def scores(logits, score: str):
    """(p, takes_part) of logits [T, E]."""
    l = np.asarray(logits, dtype=np.float32).astype(np.float64)
    on = l > MASK                                  # (NaN compares false)
    l = np.where(on, np.minimum(l, FLT_MAX), 0.0)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            p = 1.0 / (1.0 + np.exp(-l))
    else:
        top = np.max(np.where(on, l, -np.inf), axis=1, keepdims=True)
        with np.errstate(invalid="ignore", over="ignore"):
            e = np.where(on, np.exp(np.where(on, l, 0.0) - np.where(np.isfinite(top), top, 0.0)), 0.0)
        z = e.sum(axis=1, keepdims=True)
        p = e / np.where(z > 0, z, 1.0)
    return np.where(on, p, 0.0), on


def route_scored(logits, k: int, bias=None, score: str = "softmax", groups: int = 1,
                 top_groups: int = 1, group_top: int = 1, renorm: bool = True, scale: float = 1.0):
    """(idx [T, k], w [T, k]): experts by (choice descending, index ascending) within the
    best groups; masked experts after all others, in index order."""
    p, on = scores(logits, score)
    T, E = p.shape
    size = E // groups
    b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float32).astype(np.float64)
    l = np.asarray(logits, dtype=np.float32).astype(np.float64)
    idx = np.zeros((T, k), dtype=np.int64)
    w = np.zeros((T, k))
    for t in range(T):
        c = p[t] + b
        value = []
        for g in range(groups):
            mine = sorted((c[e] for e in range(g * size, (g + 1) * size) if on[t, e]), reverse=True)
            value.append((not mine, -sum(mine[:group_top])))   # a group with nothing to offer comes last
        best = sorted(range(groups), key=lambda g: (value[g], g))[:top_groups]
        pool = [e for e in range(E) if e // size in best]
        # without a bias the order is the logits' own
        order = lambda e: (not on[t, e], (-c[e] if bias is not None else -l[t, e]) if on[t, e] else 0.0, e)  # noqa: E731
        pool.sort(key=order)
        idx[t] = pool[:k]
        w[t] = p[t, idx[t]]
        if renorm:
            z = w[t].sum()
            w[t] = w[t] / z if z > 0 else 0.0
    return idx, scale * w


def route_scored_backward(logits, idx, dw, score: str = "softmax", renorm: bool = True,
                          scale: float = 1.0):
    """dlogits from the Jacobian of the weights, slot by slot: w_j = scale p_j / z."""
    p, on = scores(logits, score)
    T, E = p.shape
    out = np.zeros((T, E))
    for t in range(T):
        dp = np.zeros(E)
        sel = [(int(e), float(d)) for e, d in zip(idx[t], dw[t]) if 0 <= e < E]
        z = sum(p[t, e] for e, _ in sel) if renorm else 1.0
        if z <= 0:
            continue
        for e, d in sel:
            dp[e] += scale * d / z
        if renorm:
            back = sum(d * p[t, e] for e, d in sel) * scale / z ** 2
            for e, _ in sel:
                dp[e] -= back
        if score == "sigmoid":
            out[t] = dp * p[t] * (1.0 - p[t])
        else:
            out[t] = p[t] * (dp - (dp * p[t]).sum())
        out[t][~on[t]] = 0.0
    return out


def int8_rows(v):
    """(codes, scale) of rows: scale = amax / 127, codes to the nearest even."""
    v = np.asarray(v, dtype=np.float64)
    amax = np.abs(v).max(axis=-1, keepdims=True)
    live = amax >= 2.0 ** -100
    codes = np.rint(v * np.where(live, 127.0 / np.where(live, amax, 1.0), 0.0))
    return codes, np.where(live, amax / 127.0, 0.0)[..., 0]


def experts_int8(x, x_scales, w_gate_up, w_gate_up_scales, w_down, w_down_scales, idx, w):
    """(out [T, H], slack [T, H]): the INT8 layer, and how far out may move when activations
    that lie within 2.5e-3 codes of a rounding border (FP32's error of a 127 / amax, 2e-5
    relative with the exponential's) are coded the other way: each such code moves y by
    sh sd |wd|, |wd| that of its weight (128 for a weight of -128)."""
    x = np.asarray(x, dtype=np.float64)
    T, H = x.shape
    E, I = w_down.shape[0], w_down.shape[2]
    out, slack = np.zeros((T, H)), np.zeros((T, H))
    for e in range(E):
        t, j = np.nonzero(np.asarray(idx) == e)
        if not t.size:
            continue
        gu = (x[t] @ np.asarray(w_gate_up[e], dtype=np.float64).T) * np.asarray(x_scales, dtype=np.float64)[t, None] \
            * np.asarray(w_gate_up_scales[e], dtype=np.float64)
        g, u = gu[:, :I], gu[:, I:]
        with np.errstate(over="ignore"):
            a = g / (1.0 + np.exp(-g)) * u
        hq, sh = int8_rows(a)
        amax = np.abs(a).max(axis=1, keepdims=True)
        code = np.abs(a) * np.where(amax > 0, 127.0 / np.where(amax > 0, amax, 1.0), 0.0)
        near = (np.abs(code - np.floor(code) - 0.5) < 2.5e-3).astype(np.float64)
        sd = np.asarray(w_down_scales[e], dtype=np.float64)
        y = (hq @ np.asarray(w_down[e], dtype=np.float64).T) * sh[:, None] * sd
        wt = np.asarray(w, dtype=np.float64)[t, j][:, None]
        np.add.at(out, t, wt * y)
        np.add.at(slack, t, np.abs(wt) * (near @ np.abs(np.asarray(w_down[e], dtype=np.float64)).T) * sh[:, None] * sd
                  + np.abs(wt * y) * 2.0 ** -16)      # FP32: a (2e-5) through sh, the products, the sum
    return out, slack


def _mx_round(v, four: bool, s=None):
    """v rounded to its MX codes' values, blocks of 32 along the last axis (s: the scale exponents)."""
    b = v.reshape(v.shape[:-1] + (v.shape[-1] // 32, 32))
    if s is None:
        s = _mx_exp(np.abs(b).max(axis=-1), four)
    step = np.exp2(s.astype(np.float64))[..., None]
    c = F.e2m1_decode(F.e2m1_encode(b / step)) if four else F.e4m3_decode(F.e4m3_encode(b / step))
    return (c * step).reshape(v.shape)


def _mx_exp(amax, four: bool):
    _, ex = np.frexp(amax)
    return np.where(amax == 0.0, -127, np.clip(ex.astype(np.int64) - (3 if four else 9), -127, 127))


# How far the matrix instruction may be off, relative to the summed magnitudes of its products:
# 4-bit operands add up exactly while the products span less than 24 bits (measured 2^-22.8 where
# they span more); with an 8-bit operand runs of eight are added on a grid of 2^-13 of the run's
# largest product (measured 2^-11.8 at most over 32x32x64 and 16x16x128 products of random codes;
# seven products just below the grid would make it 2^-10.2).
MFMA4_ERROR, MFMA8_ERROR = 2.0 ** -22, 2.0 ** -11


def experts_mxfp4(x, w_gate_up, w_down, idx, w, four: bool, mfma=None):
    """(out [T, H], slack [T, H]) of the layer on decoded operands: x [T, H], w_gate_up [E, 2I, H],
    w_down [E, H, I] (a callable e -> (2I x H, H x I) is also taken for both).  slack: how far FP32
    and the matrix instruction may move out, activations that change their code by it included.
    mfma: the instruction's share of it, where the inputs keep it below MFMA4_ERROR or MFMA8_ERROR."""
    x = np.asarray(x, dtype=np.float64)
    T, H = x.shape
    idx, w = np.asarray(idx), np.asarray(w, dtype=np.float64)
    out, slack = np.zeros((T, H)), np.zeros((T, H))
    if mfma is None:
        mfma = MFMA4_ERROR if four else MFMA8_ERROR
    for e in range(w_gate_up.shape[0]):
        t, j = np.nonzero(idx == e)
        if not t.size:
            continue
        wg, wd = np.asarray(w_gate_up[e], dtype=np.float64), np.asarray(w_down[e], dtype=np.float64)
        I = wd.shape[1]
        gu = x[t] @ wg.T
        # an FP32 rounding per 64 products, and the instruction's own
        err = (np.abs(x[t]) @ np.abs(wg).T) * (mfma + H / 64 * 2.0 ** -24)
        g, u, dg, du = gu[:, :I], gu[:, I:], err[:, :I], err[:, I:]
        with np.errstate(over="ignore"):
            silu = g / (1.0 + np.exp(-g))
        a = silu * u
        # |silu'| <= 1.1; the exponential, the reciprocal and three products: 2^-19 (|g| up to 16)
        da = 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du + np.abs(a) * 2.0 ** -19 * (1.0 + np.abs(g) / 16)
        h = _mx_round(a, four)
        blocks = a.shape[:-1] + (I // 32, 32)
        top, dtop = np.abs(a).reshape(blocks).max(axis=-1), da.reshape(blocks).max(axis=-1)
        dh = np.zeros_like(a)
        for s in (_mx_exp(np.maximum(top - dtop, 0.0), four), _mx_exp(top + dtop, four)):
            for v in (a - da, a + da):
                dh = np.maximum(dh, np.abs(_mx_round(v, four, s) - h))
        y = h @ wd.T
        dy = dh @ np.abs(wd).T + ((np.abs(h) + dh) @ np.abs(wd).T) * (mfma + I / 64 * 2.0 ** -24)
        wt = w[t, j][:, None]
        np.add.at(out, t, wt * y)
        np.add.at(slack, t, np.abs(wt) * (dy + np.abs(y) * 2.0 ** -20))     # (up to 16 roundings of the slot sum)
    return out, slack


def balance_loss(logits, idx, score: str = "softmax", seqs: int = 1, mask=None):
    """(losses [2], counts [S, E], probs [S, E], tokens [S]), token by token."""
    _, on = scores(logits, score)
    T, E = on.shape
    L = T // seqs
    counts, probs = np.zeros((seqs, E), dtype=np.int64), np.zeros((seqs, E))
    tokens = np.zeros(seqs, dtype=np.int64)
    z = 0.0
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        s = t // L
        tokens[s] += 1
        for e in idx[t]:
            if 0 <= e < E:
                counts[s, e] += 1
        probs[s] += _ratio(logits[t], on[t], score) if on[t].any() else 0.0
        z += _lse(logits[t], on[t]) ** 2
    balance = 0.0
    for s in range(seqs):
        probs[s] /= max(1, tokens[s])
        balance += E * float((counts[s] * probs[s]).sum()) / max(1, counts[s].sum())
    return np.array([balance / seqs, z / max(1, tokens.sum())]), counts, probs, tokens


def _values(row):
    return np.minimum(np.asarray(row, dtype=np.float32).astype(np.float64), FLT_MAX)


def _lse(row, on):
    if not on.any():
        return 0.0
    l = _values(row)[on]
    return float(l.max() + np.log(np.exp(l - l.max()).sum()))


def _ratio(row, on, score):
    """One token's scores over their sum, also where all of them vanish in FP64."""
    l = np.where(on, _values(row), 0.0)
    if score == "softmax":
        top = l[on].max()
        v = np.where(on, np.exp(np.where(on, l, top) - top), 0.0)
    else:
        # sigma(l) = exp(min(l, 0)) / (1 + exp(-|l|)); the common factor exp(min(largest, 0)) drops out
        t = min(l[on].max(), 0.0)
        v = np.where(on, np.exp(np.minimum(l, 0.0) - t) / (1.0 + np.exp(-np.abs(l))), 0.0)
    return v / v.sum()


def balance_loss_backward(logits, counts, tokens, d_losses, score: str = "softmax", mask=None, d_add=None):
    """dlogits [T, E] from the Jacobians, token by token."""
    _, on = scores(logits, score)
    T, E = on.shape
    S = len(tokens)
    L = T // S
    out = np.zeros((T, E)) if d_add is None else np.array(d_add, dtype=np.float64)
    d0, d1 = (float(v) for v in d_losses)
    N = int(np.sum(tokens))
    for t in range(T):
        s = t // L
        if (mask is not None and not mask[t]) or not on[t].any():
            continue
        p = _ratio(logits[t], on[t], score)
        l = np.where(on[t], _values(logits[t]), 0.0)
        total = int(np.sum(counts[s]))
        if total and tokens[s]:
            up = d0 * E * np.asarray(counts[s], dtype=np.float64) / (total * S * float(tokens[s]))
            d = p * (up - (p * up).sum())
            if score == "sigmoid":
                with np.errstate(over="ignore"):
                    d = d / (1.0 + np.exp(l))
            out[t] += np.where(on[t], d, 0.0)
        if N:
            out[t] += 2.0 * d1 / N * _lse(logits[t], on[t]) * _ratio(logits[t], on[t], "softmax")
    return out
