"""The bound that the MXFP8 experts are held to on inputs that are exact in runs (tests/_mxfp4.py) tells a
wrong kernel from a right one, also at the longest reductions: mistakes planted in the oracle's weights
are found, one at a time."""
import numpy as np
import pytest

from oracle import block as B
from oracle import formats as F
from oracle.formats import bf16_round
from tests._mxfp4 import RUNS_ERROR, excess, one_in_eight

T = 4


def _weights(rng, rows, K):
    """Codes' values [rows, K / 32, 32] and their scales [rows, K / 32, 1], about 1 / sqrt(K)."""
    e = -int(round(np.log2(2.9 * K ** 0.5)))
    return F.e2m1_decode(rng.integers(0, 16, (rows, K // 32, 32))), np.exp2(rng.integers(e - 2, e + 2, (rows, K // 32, 1)).astype(float))


def _mat(w):
    c, s = w
    return (c * s).reshape(c.shape[0], -1)


def _out(x, wg, wd, **kw):
    return B.experts_mxfp4(x, _mat(wg)[None], _mat(wd)[None], np.zeros((T, 1), dtype=int), np.ones((T, 1)), False, **kw)


@pytest.mark.parametrize("H,I", [(256, 256), (1024, 4096), (4096, 1024), (1792, 3840), (2048, 2048), (256, 16384), (16384, 256)])
def test_planted_mistakes_are_found(H, I):
    rng = np.random.default_rng(H + I)
    x = rng.normal(size=(T, H))
    x[:, ::61] *= 8
    x = F.mx_dequantize(*F.mx_quantize(x)) * one_in_eight(rng, T, H)
    wg, wd = _weights(rng, 2 * I, H), _weights(rng, H, I)
    on = one_in_eight(rng, I)
    wg[0][:I][~on] = 0
    ref, slack = _out(x, wg, wd, mfma=RUNS_ERROR)
    rms = lambda v: float(np.sqrt((v * v).mean()))  # noqa: E731
    assert rms(slack) < 0.05 * rms(ref), rms(slack) / rms(ref)
    assert (excess(bf16_round(ref), ref, slack) <= 0).all()

    def found(what, x=x, wg=wg, wd=wd):
        assert (excess(bf16_round(_out(x, wg, wd)[0]), ref, slack) > 0).any(), what

    def changed(w, **kw):
        c, s = w[0].copy(), w[1].copy()
        for rows, b, f in kw.values():
            s[rows, b] *= f
        return c, s
    row = I // 2 // 16 * 16                                  # sixteen neurons, as many rows as an operand holds
    for b in (0, H // 64, H // 32 - 1):                     # blocks of the gate/up reduction
        found("block left out", wg=changed(wg, a=(slice(None), b, 0.0)))
        found("block twice", wg=changed(wg, a=(slice(None), b, 2.0)))
        found("gate scales of an operand doubled", wg=changed(wg, a=(slice(row, row + 16), b, 2.0)))
        found("up scales of an operand doubled", wg=changed(wg, a=(slice(I + row, I + row + 16), b, 2.0)))
    for b in (0, I // 64, I // 32 - 1):                     # blocks of the down reduction
        found("block left out", wd=changed(wd, a=(slice(None), b, 0.0)))
        found("scales doubled", wd=changed(wd, a=(slice(None), b, 2.0)))
        found("one row's scale doubled", wd=changed(wd, a=(H // 2 + 3, b, 2.0)))
    for w, n in ((wg, "wg"), (wd, "wd")):                   # neighbouring scales for each other
        s = w[1].copy()
        b = s.shape[1] // 2
        s[:, [b - 1, b]] = s[:, [b, b - 1]]
        found("scales swapped", **{n: (w[0], s)})
    found("tokens swapped", x=x[::-1])
    found("gate and up swapped", wg=(np.concatenate([wg[0][I:], wg[0][:I]]), np.concatenate([wg[1][I:], wg[1][:I]])))
    moved = x.copy()
    moved[:, :-8] = x[:, 8:]
    found("x moved by a run", x=moved)
