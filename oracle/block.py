"""The operators around the routed experts, written out in float64: residual sum
and RMS norm with its gradients, routing by scores with its gradient, INT8 rows
and the INT8 experts.  Plain NumPy, one token or one expert at a time where that
reads better."""
from __future__ import annotations

import numpy as np

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
