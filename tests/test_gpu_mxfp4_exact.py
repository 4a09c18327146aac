"""moe_experts_mxfp4 with MXFP8 activations on inputs that are exact in the matrix instruction's runs
(tests/_mxfp4.py), held to FP32 element by element at every tile height and form; on dense inputs, as a
whole; and its forms against each other."""
import numpy as np
import pytest
import torch

from oracle import block as B
from oracle import formats as F
from tests._mxfp4 import RUNS_ERROR, excess, one_in_eight
from tests.test_gpu_mxfp4 import SIZES, M, _f64, Lazy, call, make, part_of, reference  # noqa: F401

pytestmark = pytest.mark.gpu


# The longest reductions of either product, with few pairs, on 32- and 96-row tiles; many slots
LONG = [(1, 16384, 256, 4, 1), (1, 256, 16384, 4, 2), (3, 16384, 512, 64, 2), (1, 7168, 2048, 40, 8), (3, 4096, 14336, 2, 1),
        (70, 16384, 256, 2, 1), (70, 256, 16384, 2, 2), (40, 7168, 2048, 3, 2), (9, 512, 256, 64, 32), (300, 512, 256, 40, 32)]


def make_runs(M, T, H, I, E, k, seed, **kw):  # noqa: F811
    d = make(M, T, H, I, E, k, False, seed=seed, **kw)
    rng = np.random.default_rng(seed)
    d["x"] = d["x"] * torch.from_numpy(one_in_eight(rng, T, H)).cuda()
    d["wg"][:, :I] *= torch.from_numpy(one_in_eight(rng, E, I)).cuda().unsqueeze(2)
    return d


def check_runs(d, out, rows=slice(None)):
    n = lambda t: t.cpu().numpy()  # noqa: E731
    ref, slack = B.experts_mxfp4(F.mx_dequantize(n(d["x"])[rows], n(d["xs"])[rows]), Lazy(d["wg"], d["sg"]), Lazy(d["wd"], d["sd"]),
                                 n(d["idx"])[rows], n(d["w"])[rows], False, mfma=RUNS_ERROR)
    got = _f64(out)[rows]
    over = excess(got, ref, slack)
    rms = lambda v: float(np.sqrt((v * v).mean()))  # noqa: E731
    print(f"[mxfp4 runs] rms slack / rms {rms(slack) / max(rms(ref), 1e-300):.1e}", flush=True)
    assert np.all(np.isfinite(got)) and np.all(over <= 0), f"{over.max():.3e} over, |ref| {np.abs(ref).max():.3e}"


@pytest.mark.parametrize("T,H,I,E,k", SIZES + LONG)
def test_exact_runs(M, T, H, I, E, k):  # noqa: F811
    print(f"[mxfp4 runs] T={T} H={H} I={I} E={E} k={k}", flush=True)
    d = make_runs(M, T, H, I, E, k, seed=T + H)
    check_runs(d, call(M, d))


@pytest.mark.parametrize("T,H,I", [(16500, 16384, 256), (1500, 256, 16384)])
def test_exact_runs_on_large_tiles_and_the_longest_reductions(M, T, H, I):  # noqa: F811
    print(f"[mxfp4 runs] large T={T} H={H} I={I}", flush=True)
    d = make_runs(M, T, H, I, 1, 1, seed=T)
    out = call(M, d)
    for rows in (slice(0, 40), slice(T - 40, T)):
        check_runs(d, out, rows)


@pytest.mark.parametrize("T,H,I,E,k", [(6, 512, 256, 4, 2), (200, 512, 256, 8, 3), (900, 512, 256, 3, 1), (2400, 2048, 2048, 3, 1),
                                       (1200, 2048, 2048, 3, 2), (1600, 1024, 4096, 2, 1), (1200, 512, 512, 72, 2)])
def test_exact_runs_and_ids_out_of_range(M, T, H, I, E, k):  # noqa: F811
    """Slots of experts held elsewhere, most of them: tiles with few rows, experts with none."""
    print(f"[mxfp4 runs] ids out of range T={T} H={H} I={I} E={E} k={k}", flush=True)
    d = make_runs(M, T, H, I, E, k, seed=T)
    g = torch.Generator().manual_seed(3)
    off = torch.rand(T, k, generator=g) < 0.8
    off |= d["idx"].cpu() == E - 1                          # an expert without a row
    d["idx"] = torch.where(off, torch.tensor(E), d["idx"].cpu()).int().cuda()
    out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    call(M, d, out=out)
    assert not out[off.all(dim=1).cuda()].view(torch.int16).any()
    check_runs(d, out)


@pytest.mark.parametrize("T,H,I,E,k", [s for s in SIZES if s[0] * s[4] >= 500])
def test_dense_activations_as_a_whole(M, T, H, I, E, k):  # noqa: F811
    """The relative error of all outputs together.  Their rounding to BF16: 2^-8 / sqrt(3) at most.  A product of a
    run is cut by less than 2^-13 of the run's largest, whose mean square on these inputs (unit noise, one
    channel in 61 eight times as large) is below (5.5 rms)^2: a gate/up sum is off by 2^-13 5.5 / sqrt(3) of its
    rms, an activation by sqrt(2) times that, in the mean 0.8 of it, 4.4e-4.  It takes the other of two codes
    with the probability of that over their distance, 2^-3 of it at most: a mean square of 4.4e-4 / 8, a root
    of 0.0074.  The down product adds 2^-13 5.5 / sqrt(3).  Together 0.0078."""
    print(f"[mxfp4 dense] T={T} H={H} I={I} E={E} k={k}", flush=True)
    d = make(M, T, H, I, E, k, False, seed=T)
    ref, _ = reference(d)
    rel = float(np.linalg.norm(_f64(call(M, d)) - ref) / np.linalg.norm(ref))
    print(f"[mxfp4 dense] {rel:.5f}", flush=True)
    assert rel < 0.008


@pytest.mark.parametrize("H,I,E,k", [(512, 256, 16, 1), (512, 256, 16, 3), (2560, 1280, 128, 1), (2560, 1280, 128, 3), (2304, 1792, 128, 4)])
@pytest.mark.parametrize("four", [False, True])
def test_few_pairs_have_the_bits_of_a_larger_batch(M, H, I, E, k, four):  # noqa: F811
    """Every pair on its own (48 pairs at most) against the 32-row tiles: the same products in the same order."""
    print(f"[mxfp4] few pairs H={H} I={I} E={E} k={k} four={four}", flush=True)
    T = 48 // k
    d = make(M, T + 14, H, I, E, k, four, seed=17)
    d["idx"][2, 0] = E                                      # a slot without an expert
    full = call(M, d)
    for n in (1, 5, T):
        part = call(M, part_of(d, slice(0, n)))
        assert torch.equal(part, full[:n]), n
