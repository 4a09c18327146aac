"""moe_experts_int8 against the FP64 oracle.  Its dot products are exact; the bound is half
a BF16 step of the result, FP32's error and what activations at a rounding border of their
codes may move (oracle/block.py: experts_int8 gives the latter two)."""
import numpy as np
import pytest
import torch

from oracle import block as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import mixture_experts_ffn_07_amd as M
    yield M
    M.moe_set_debug_options(0, 0)


def make(T, H, I, E, k, seed=0, skew=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ri = lambda *s: torch.randint(-128, 128, s, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    ru = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    d = dict(x=ri(T, H), xs=(0.5 + ru(T)) * 0.02, wg=ri(E, 2 * I, H), sg=(0.5 + ru(E, 2 * I)) * 0.6 / (73 * H ** 0.5),
             wd=ri(E, H, I), sd=(0.5 + ru(E, H)) * 3e-4)
    l = torch.randn(T, E, generator=g, device="cuda")
    if skew:
        l[:, 0] += 100                                    # every token takes expert 0
    d["w"], idx = torch.softmax(l, 1).topk(k, dim=1)
    d["w"], d["idx"] = d["w"].contiguous(), idx.int().contiguous()
    return d


def call(M, d, **kw):
    return M.moe_experts_int8(d["x"], d["xs"], d["wg"], d["sg"], d["wd"], d["sd"], d["idx"], d["w"], **kw)


def check(M, d, out, tokens=None):
    n = lambda t: t.cpu().numpy()  # noqa: E731
    rows = slice(None) if tokens is None else tokens
    ref, slack = B.experts_int8(n(d["x"])[rows], n(d["xs"])[rows], n(d["wg"]), n(d["sg"]), n(d["wd"]), n(d["sd"]),
                                n(d["idx"])[rows], n(d["w"])[rows])
    got = out.double().cpu().numpy()[rows]
    # out is the BF16 value next to some v with |v - ref| <= slack: |out - ref| <= half a step of
    # v + slack, half a step <= 2^-8 |v| <= 2^-8 (|ref| + slack), and 2^-134 below the normal
    # range (steps of 2^-133 there: a weight of 1e-43 times y has no nearer BF16 value)
    over = np.abs(got - ref) - ((np.abs(ref) + slack) * 2.0 ** -8 + 2.0 ** -134 + slack)
    assert np.all(np.isfinite(got)) and np.all(over <= 0), f"{over.max():.3e} over, |ref| {np.abs(ref).max():.3e}"


@pytest.mark.parametrize("T,H,I,E,k", [
    (1, 256, 256, 1, 1), (1, 512, 256, 8, 2), (1, 2048, 768, 128, 8), (2, 256, 512, 4, 4), (8, 512, 256, 16, 3),
    (17, 768, 512, 4, 2), (33, 512, 768, 6, 1), (64, 1024, 256, 32, 8), (65, 512, 256, 5, 2), (130, 256, 256, 2, 2),
    (300, 512, 512, 3, 1), (777, 256, 512, 16, 6), (600, 512, 256, 1, 1), (513, 768, 256, 2, 2),
    (1025, 1024, 512, 4, 1),
    # 256-row tiles: one ragged expert, several with tail slices along K, k = 1 and more
    (700, 4096, 1024, 1, 1), (1300, 2048, 2048, 2, 1), (900, 4096, 1024, 4, 2), (1500, 4096, 1024, 9, 2),
    (2200, 1024, 2048, 3, 1), (1500, 1024, 2048, 4, 2), (2601, 1792, 1792, 2, 1)])
def test_experts_int8(M, T, H, I, E, k):
    print(f"[int8] T={T} H={H} I={I} E={E} k={k}", flush=True)
    d = make(T, H, I, E, k, seed=T)
    check(M, d, call(M, d))


@pytest.mark.parametrize("T", [5, 63, 200, 900])
def test_experts_int8_skewed(M, T):
    print(f"[int8] skewed T={T}", flush=True)
    d = make(T, 512, 256, 12, 2, seed=1, skew=True)
    check(M, d, call(M, d))


@pytest.mark.parametrize("T,E,k,H,I", [
    (6, 4, 2, 512, 256), (50, 8, 3, 512, 256), (200, 8, 3, 512, 256), (9, 4, 1, 512, 256), (300, 4, 1, 512, 256),
    (900, 3, 1, 512, 256), (1200, 3, 2, 512, 256), (1100, 3, 1, 2048, 2048), (600, 3, 2, 4096, 1024),
    (2200, 3, 1, 1024, 2048), (1100, 3, 2, 1024, 2048)])
def test_experts_int8_ids_out_of_range(M, T, E, k, H, I):
    print(f"[int8] ids out of range T={T} E={E} k={k} H={H}", flush=True)
    d = make(T, H, I, E, k, seed=2)
    g = torch.Generator().manual_seed(7)
    off = torch.rand(T, k, generator=g) < 0.4
    off[1] = True                                          # a token without an expert
    bad = torch.tensor([-1, E, 2 ** 31 - 1, -2 ** 31])[torch.randint(0, 4, (T, k), generator=g)].int()
    d["idx"] = torch.where(off, bad, d["idx"].cpu()).int().cuda()
    out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    call(M, d, out=out)
    assert not out[1].any()
    check(M, d, out)
    d["idx"].fill_(-1)
    out.fill_(float("nan"))
    assert not call(M, d, out=out).any()


@pytest.mark.parametrize("T,H,I,E,k", [
    (14, 2560, 1792, 5, 5), (100, 4096, 1024, 4, 2), (300, 4096, 1024, 4, 1), (40, 4096, 256, 3, 3), (60, 512, 2048, 4, 4),
    (90, 1536, 1792, 2, 1), (20, 512, 4096, 16, 12), (131, 7168, 256, 1, 1)])
def test_experts_int8_split_reductions(M, T, H, I, E, k):
    """Few rows and few experts: reductions in slices, on either or both projections."""
    print(f"[int8] split T={T} H={H} I={I} E={E} k={k}", flush=True)
    d = make(T, H, I, E, k, seed=12)
    ws = M.workspace(M.moe_experts_int8_workspace_bytes(T, H, I, E, k))
    ws.fill_(255)
    ref = call(M, d, ws=ws)
    check(M, d, ref)
    one = {n: (t[3:4].clone() if n in ("x", "xs", "idx", "w") else t) for n, t in d.items()}
    assert torch.equal(call(M, one), ref[3:4])              # exact sums: the bits of an unsplit form
    for seed in (1, 2, 3):
        M.moe_set_debug_options(M.MOE_DEBUG_PERMUTE_ORDER, seed)
        assert torch.equal(call(M, d), ref)
    M.moe_set_debug_options(0, 0)
    d["idx"][1] = E                                         # a token without an expert, a slot without one
    d["idx"][2, 0] = -1
    out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    call(M, d, out=out)
    assert not out[1].any()
    check(M, d, out)


def test_experts_int8_same_expert_twice(M):
    d = make(40, 512, 256, 6, 3, seed=3)
    d["idx"][:, 2] = d["idx"][:, 0]
    check(M, d, call(M, d))


@pytest.mark.parametrize("T", [4, 90, 700])
def test_experts_int8_zero_rows(M, T):
    d = make(T, 512, 256, 4, 2, seed=4)
    d["x"][0] = 0
    d["xs"][1] = 0
    d["wg"][2] = 0                                          # an expert that answers 0
    out = call(M, d)
    assert not out[:2].any()
    check(M, d, out)


def test_experts_int8_extreme_codes(M):
    """Every code at the end of its range over the longest reduction: the INT32 sums' largest."""
    T, H, I, E, k = 3, 16384, 256, 2, 1
    d = make(T, H, I, E, k, seed=5)
    d["x"].fill_(-128)
    d["wg"].fill_(-128)
    d["sg"].fill_(1e-9)
    check(M, d, call(M, d))
    T, H, I = 3, 256, 16384
    d = make(T, H, I, E, k, seed=6)
    d["wd"].fill_(-128)
    check(M, d, call(M, d))


def test_experts_int8_rows_do_not_depend_on_the_batch(M):
    """A token's bits are the same alone, in a decode batch and in a large batch (exact sums,
    one order of the slots), on any form of the kernels."""
    d = make(2100, 4096, 1024, 4, 2, seed=8)
    full = call(M, d)
    for rows in (slice(0, 1), slice(5, 12), slice(0, 64), slice(100, 190), slice(0, 400), slice(1400, 2099)):
        part = {n: (t[rows].clone() if n in ("x", "xs", "idx", "w") else t) for n, t in d.items()}
        assert torch.equal(call(M, part), full[rows]), rows


@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 512, 512), (40, 8, 2, 512, 512), (500, 8, 2, 512, 512),
                                       (900, 2, 1, 2048, 2048), (700, 2, 2, 4096, 1024),
                                       (2100, 2, 1, 1024, 2048), (1050, 2, 2, 1024, 2048)])
def test_experts_int8_deterministic_and_order_free(M, T, E, k, H, I):
    d = make(T, H, I, E, k, seed=9)
    ref = call(M, d)
    for seed in range(4):
        M.moe_set_debug_options(M.MOE_DEBUG_PERMUTE_ORDER if seed else 0, seed)
        assert torch.equal(call(M, d), ref)
    M.moe_set_debug_options(0, 0)


def test_experts_int8_workspace_contents_do_not_matter(M):
    for T, E, k, H, I in ((2, 8, 2, 512, 256), (70, 8, 2, 512, 256), (300, 8, 2, 512, 256), (700, 2, 1, 4096, 1024),
                          (500, 2, 2, 4096, 1024), (2100, 2, 1, 1024, 2048), (1050, 2, 2, 1024, 2048)):
        d = make(T, H, I, E, k, seed=10)
        ws = M.workspace(M.moe_experts_int8_workspace_bytes(T, H, I, E, k))
        ws.zero_()
        a = call(M, d, ws=ws)
        ws.fill_(255)
        b = call(M, d, ws=ws)
        assert torch.equal(a, b)


def test_experts_int8_large_offsets(M):
    """An expert array beyond 2^31 elements and the last expert in it."""
    T, H, I, E, k = 4, 2048, 1024, 540, 2
    d = make(T, H, I, 2, k, seed=11)
    big = {"wg": torch.zeros(E, 2 * I, H, dtype=torch.int8, device="cuda"), "sg": torch.zeros(E, 2 * I, device="cuda"),
           "wd": torch.zeros(E, H, I, dtype=torch.int8, device="cuda"), "sd": torch.zeros(E, H, device="cuda")}
    for n, t in big.items():
        t[E - 2:] = d[n]
    moved = dict(d, **big, idx=d["idx"] + (E - 2))
    assert torch.equal(call(M, moved), call(M, d))
    assert E * 2 * I * H > 2 ** 31


@pytest.mark.parametrize("T,E,k,H,I", [(1, 16, 4, 512, 256), (60, 16, 4, 512, 256), (300, 8, 2, 512, 256),
                                       (900, 2, 1, 2048, 2048), (700, 2, 2, 4096, 1024),
                                       (2100, 2, 1, 1024, 2048), (1050, 2, 2, 1024, 2048)])
def test_experts_int8_graph_replays(M, T, E, k, H, I):
    """Captured and replayed, with eager work of the program's own between the replays; two
    graphs that share one workspace, replayed in turn."""
    print(f"[int8 graph] T={T} E={E} k={k}", flush=True)
    ds = [make(T, H, I, E, k, seed=20 + j) for j in range(2)]
    ref = [call(M, d) for d in ds]
    ws = M.workspace(M.moe_experts_int8_workspace_bytes(T, H, I, E, k))
    outs = [torch.empty(T, H, dtype=torch.bfloat16, device="cuda") for _ in ds]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for d, o in zip(ds, outs):
            call(M, d, out=o, ws=ws)
    torch.cuda.synchronize()
    graphs = []
    for d, o in zip(ds, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(M, d, out=o, ws=ws)
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, r in zip(outs, ref):
            assert torch.equal(o, r)
        call(M, ds[0], ws=ws)
        _ = (outs[0].float() * 2).sum()
        torch.cuda.synchronize()


@pytest.mark.parametrize("H,I,E", [(512, 256, 8), (4096, 1024, 4), (2048, 2048, 2)])
def test_experts_int8_one_slot_zero_and_negative_weights(M, H, I, E):
    """k = 1: a token's bits, the sign of a zero included, are the same in every form (weight 0
    is what routing gives a masked expert that fills a slot)."""
    print(f"[int8] one slot H={H} I={I} E={E}", flush=True)
    d = make(2100, H, I, E, 1, seed=13)
    d["w"][::3] = 0
    d["w"][1::3] *= -1
    full = call(M, d)
    check(M, d, full)
    zero = full[::3].view(torch.int16)
    assert ((zero == 0) | (zero == -2 ** 15)).all() and (zero == 0).any() and (zero != 0).any()
    for rows in (slice(0, 1), slice(3, 4), slice(5, 12), slice(0, 20), slice(0, 48), slice(100, 190), slice(0, 400)):
        part = {n: (t[rows].clone() if n in ("x", "xs", "idx", "w") else t) for n, t in d.items()}
        assert torch.equal(call(M, part).view(torch.int16), full[rows].view(torch.int16)), rows


@pytest.mark.parametrize("H,I,E,k", [(2560, 1792, 5, 5), (2048, 2048, 2, 1), (4096, 1024, 4, 2)])
def test_experts_int8_one_workspace_for_all_batches(M, H, I, E, k):
    """Sized once, for the largest batch: every smaller one is taken, and its outputs are
    those with a workspace of its own."""
    print(f"[int8] one workspace H={H} I={I} E={E} k={k}", flush=True)
    most = 2100
    d = make(most, H, I, E, k, seed=14)
    ws = M.workspace(M.moe_experts_int8_workspace_bytes(most, H, I, E, k))
    ws.fill_(255)
    for T in (1, 2, 3, 9, 14, 40, 48, 100, 123, 300, 383, 700, 1025, most):
        part = {n: (t[:T].clone() if n in ("x", "xs", "idx", "w") else t) for n, t in d.items()}
        assert torch.equal(call(M, part, ws=ws), call(M, part)), T
