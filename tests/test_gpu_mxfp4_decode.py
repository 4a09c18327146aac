"""moe_experts_mxfp4 with MXFP8 activations for few rows to an expert: the gate/up sums are exact to FP32 on
any activations (the instruction's runs of eight drop bits, tests/_mxfp4.py; these forms multiply the codes
below 2 and the others apart, which leaves none to drop).  Dense activations, and one neuron in eight, so
that the down product, which is not taken apart, is exact too: held to FP32 element by element."""
import numpy as np
import pytest
import torch

from tests._mxfp4 import one_in_eight
from tests.test_gpu_mxfp4 import M, call, make, part_of  # noqa: F401
from tests.test_gpu_mxfp4_exact import check_runs

pytestmark = pytest.mark.gpu


def make_neurons(M, T, H, I, E, k, seed, spread=0):  # noqa: F811
    d = make(M, T, H, I, E, k, False, seed=seed)
    rng = np.random.default_rng(seed)
    d["wg"][:, :I] *= torch.from_numpy(one_in_eight(rng, E, I)).cuda().unsqueeze(2)
    if spread:                                              # codes of every size, down to the lowest, in every run
        d["x"] = torch.from_numpy(rng.integers(0, 0x7F, (T, H)).astype(np.uint8) | (rng.integers(0, 2, (T, H)) << 7).astype(np.uint8)).cuda()
        d["xs"] = torch.from_numpy(rng.integers(118 - spread, 119 + spread, (T, H // 32)).astype(np.uint8)).cuda()
    return d


# every pair on its own; 32-row tiles; both with long reductions, odd numbers of steps, padded slots
SIZES = [(1, 256, 256, 1, 1), (1, 2048, 768, 128, 8), (8, 512, 256, 16, 3), (2, 16384, 256, 64, 2), (1, 256, 16384, 4, 2), (1, 7168, 2048, 40, 8),
         (20, 512, 256, 16, 4), (64, 1024, 256, 32, 8), (64, 2048, 768, 64, 4), (50, 2304, 512, 40, 3), (70, 16384, 256, 5, 1), (70, 512, 4096, 9, 2),
         (17, 768, 512, 4, 1), (300, 512, 512, 64, 1)]


@pytest.mark.parametrize("T,H,I,E,k", SIZES)
@pytest.mark.parametrize("spread", [0, 3])
def test_dense_activations(M, T, H, I, E, k, spread):  # noqa: F811
    print(f"[mxfp4 decode] T={T} H={H} I={I} E={E} k={k} spread={spread}", flush=True)
    d = make_neurons(M, T, H, I, E, k, seed=T + H, spread=spread)
    if T > 2:
        d["idx"][1, 0] = E
    check_runs(d, call(M, d))


@pytest.mark.parametrize("T", [5, 40, 300])
def test_activations_of_one_size(M, T):  # noqa: F811
    """All codes on one side of 2, and every code once."""
    H, I, E, k = 512, 256, 24, 1
    for lo, hi in ((0, 0x40), (0x40, 0x7F)):
        d = make_neurons(M, T, H, I, E, k, seed=lo, spread=1)
        g = torch.Generator(device="cuda").manual_seed(lo)
        d["x"] = torch.randint(lo, hi, (T, H), generator=g, device="cuda", dtype=torch.uint8)
        check_runs(d, call(M, d))
    d = make_neurons(M, T, H, I, E, k, seed=3, spread=1)
    codes = torch.arange(256, dtype=torch.uint8)
    codes[codes & 0x7F == 0x7F] = 0                         # (NaN)
    d["x"] = codes.repeat(T, 2).cuda()
    check_runs(d, call(M, d))
