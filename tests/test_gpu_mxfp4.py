"""moe_quantize_mxfp4, moe_dequantize_mxfp4 and moe_experts_mxfp4 against the FP64 oracle.

Rows: codes, scales and values are exact.  Experts: the bound is half a BF16 step of the result and
what FP32, the matrix instruction and activations that change their code by it may move
(oracle/block.py: experts_mxfp4 gives the latter)."""
import numpy as np
import pytest
import torch

from oracle import block as B
from oracle import formats as F

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import mixture_experts_ffn_07_amd as M
    yield M
    M.moe_set_debug_options(0, 0)


def _f64(t):
    return t.detach().double().cpu().numpy()


# ---------------------------------------------------------------------------
# rows

@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (7, 64), (8, 4096), (1001, 2080), (2, 16416), (513, 7168), (40000, 32)])
def test_quantize_rows(M, rows, K):
    print(f"[mxfp4] rows={rows} K={K}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, K, generator=g, device="cuda") * torch.exp2(
        torch.randint(-20, 20, (rows, K // 32), generator=g, device="cuda").float()).repeat_interleave(32, dim=1)
    x[0, :32] = 0
    x = x.bfloat16()
    codes, scales = M.moe_quantize_mxfp4(x)
    rc, rs = F.mxfp4_quantize(_f64(x))
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), rc)
    v = M.moe_dequantize_mxfp4(codes, scales)
    assert np.array_equal(_f64(v), F.mxfp4_dequantize(rc, rs))
    for seed in (1, 2):
        M.moe_set_debug_options(M.MOE_DEBUG_PERMUTE_ORDER, seed)
        c2, s2 = M.moe_quantize_mxfp4(x)
        assert torch.equal(c2, codes) and torch.equal(s2, scales)
        assert torch.equal(M.moe_dequantize_mxfp4(codes, scales), v)
    M.moe_set_debug_options(0, 0)


def test_quantize_every_finite_bf16(M):
    """Every finite value in a block of its own (its scale) and in blocks whose largest is 2^9 above."""
    bits = torch.arange(1 << 16, dtype=torch.int32)
    bits = bits[(bits & 0x7F80) != 0x7F80].to(torch.int16)
    v = bits.view(torch.bfloat16)
    x = torch.zeros(v.numel(), 32, dtype=torch.bfloat16)
    x[:, 5] = v
    y = v[: v.numel() // 32 * 32].reshape(-1, 32)
    z = torch.randn(4096, 32).bfloat16() * 2.0 ** 120
    z[::3] *= 2.0 ** -118
    z[1::3] *= 2.0 ** -250                                 # down to subnormal values and the lowest scale
    for t in (x, y, z):
        codes, scales = M.moe_quantize_mxfp4(t.cuda())
        rc, rs = F.mxfp4_quantize(t.double().numpy())
        assert np.array_equal(scales.cpu().numpy(), rs) and np.array_equal(codes.cpu().numpy(), rc)
        got = _f64(M.moe_dequantize_mxfp4(codes, scales))
        assert np.array_equal(got, F.mxfp4_dequantize(rc, rs))


def test_dequantize_every_code_and_scale(M):
    codes = torch.arange(16, dtype=torch.uint8)
    row = (codes[0::2] | codes[1::2] << 4).repeat(2)
    c = row.repeat(256, 1).contiguous().cuda()
    s = torch.arange(256, dtype=torch.uint8).reshape(256, 1).cuda()
    got = _f64(M.moe_dequantize_mxfp4(c, s))
    ref = F.mxfp4_dequantize(c.cpu().numpy(), s.cpu().numpy())
    big = np.abs(ref) >= 2.0 ** 128
    assert np.isnan(got[255]).all() and np.isnan(ref[255]).all()
    ref = np.where(big, np.sign(ref) * np.inf, ref)
    assert np.array_equal(got[:255], ref[:255])
    assert np.array_equal(np.signbit(got[:255]), np.signbit(ref[:255]))


def test_quantize_row_with_infinity_leaves_the_others(M):
    x = torch.randn(6, 128, device="cuda").bfloat16()
    ref = M.moe_quantize_mxfp4(x)
    bad = x.clone()
    bad[2, 40], bad[4, 3] = float("inf"), float("nan")
    got = M.moe_quantize_mxfp4(bad)
    keep = torch.ones(6, 4, dtype=torch.bool, device="cuda")
    keep[2, 1] = keep[4, 0] = False
    assert torch.equal(got[1][keep], ref[1][keep])
    assert torch.equal(got[0].view(6, 4, 16)[keep], ref[0].view(6, 4, 16)[keep])


def test_rows_empty(M):
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    codes, scales = M.moe_quantize_mxfp4(x)
    assert codes.shape == (0, 32) and scales.shape == (0, 2)
    assert M.moe_dequantize_mxfp4(codes, scales).shape == (0, 64)


def test_rows_past_2_31_elements(M):
    rows, K = (1 << 31) // 4096 + 3, 4096
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.arange(K, device="cuda").bfloat16()
    x[-2, 7] = -3.0
    codes, scales = M.moe_quantize_mxfp4(x)
    v = M.moe_dequantize_mxfp4(codes, scales)
    rc, rs = F.mxfp4_quantize(_f64(x[-3:]))
    assert np.array_equal(codes[-3:].cpu().numpy(), rc) and np.array_equal(scales[-3:].cpu().numpy(), rs)
    assert np.array_equal(_f64(v[-3:]), F.mxfp4_dequantize(rc, rs))
    assert not v[:-3].any()


# ---------------------------------------------------------------------------
# experts

class Lazy:
    """Experts' MXFP4 weights, decoded by the oracle's codec one at a time."""

    def __init__(self, codes, scales):
        self.c, self.s, self.shape = codes, scales, codes.shape

    def __getitem__(self, e):
        return F.mxfp4_dequantize(self.c[e].cpu().numpy(), self.s[e].cpu().numpy())


def make(M, T, H, I, E, k, four, seed=0, skew=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ri = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    d = dict(four=four, wg=ri(0, 256, E, 2 * I, H // 2), wd=ri(0, 256, E, H, I // 2))
    # weights of about 1 / sqrt(row): |code| is 2.9 in the mean square, scales differ from block to block
    e = lambda n: 127 - int(round(np.log2(2.9 * n ** 0.5)))  # noqa: E731
    d["sg"], d["sd"] = ri(e(H) - 2, e(H) + 2, E, 2 * I, H // 32), ri(e(I) - 2, e(I) + 2, E, H, I // 32)
    x = torch.randn(T, H, generator=g, device="cuda")
    x[:, ::61] *= 8
    d["x"], d["xs"] = (M.moe_quantize_mxfp4 if four else M.moe_quantize_mxfp8)(x.bfloat16())
    l = torch.randn(T, E, generator=g, device="cuda")
    if skew:
        l[:, 0] += 100                                    # every token takes expert 0
    d["w"], idx = torch.softmax(l, 1).topk(k, dim=1)
    d["w"], d["idx"] = d["w"].contiguous(), idx.int().contiguous()
    return d


TOKENS = ("x", "xs", "idx", "w")


def part_of(d, rows):
    return {n: (t[rows].clone() if n in TOKENS else t) for n, t in d.items()}


def call(M, d, **kw):
    return M.moe_experts_mxfp4(d["x"], d["xs"], d["wg"], d["sg"], d["wd"], d["sd"], d["idx"], d["w"],
                               xtype=M.MOE_MXFP4 if d["four"] else M.MOE_MXFP8, **kw)


def reference(d, rows=slice(None)):
    n = lambda t: t.cpu().numpy()  # noqa: E731
    x = (F.mxfp4_dequantize if d["four"] else F.mx_dequantize)(n(d["x"])[rows], n(d["xs"])[rows])
    return B.experts_mxfp4(x, Lazy(d["wg"], d["sg"]), Lazy(d["wd"], d["sd"]), n(d["idx"])[rows], n(d["w"])[rows], d["four"])


def check(d, out, rows=slice(None)):
    ref, slack = reference(d, rows)
    got = _f64(out)[rows]
    # out is the BF16 value next to some v with |v - ref| <= slack: half a step of v is at most
    # 2^-8 (|ref| + slack), and 2^-134 below the normal range
    over = np.abs(got - ref) - ((np.abs(ref) + slack) * 2.0 ** -8 + 2.0 ** -134 + slack)
    print(f"[mxfp4] rel l2 {np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-300):.2e}", flush=True)
    assert np.all(np.isfinite(got)) and np.all(over <= 0), f"{over.max():.3e} over, |ref| {np.abs(ref).max():.3e}"


SIZES = [
    (1, 256, 256, 1, 1), (1, 512, 256, 8, 2), (1, 2048, 768, 128, 8), (2, 256, 512, 4, 4), (8, 512, 256, 16, 3),
    (17, 768, 512, 4, 2), (33, 512, 768, 6, 1), (64, 1024, 256, 32, 8), (65, 512, 256, 5, 2), (130, 256, 256, 2, 2),
    (300, 512, 512, 3, 1), (777, 256, 512, 16, 6), (600, 512, 256, 1, 1), (513, 768, 256, 2, 2), (1025, 1024, 512, 4, 1),
    (700, 4096, 1024, 1, 1), (1300, 2048, 2048, 2, 1), (900, 4096, 1024, 4, 2), (1500, 1024, 2048, 4, 2),
    # 96-row tiles with enough of them for 64 weight rows a wave: on the gate/up product, on the down product, on both
    (700, 512, 512, 72, 2), (1900, 512, 512, 72, 1), (500, 512, 1280, 18, 2), (333, 2304, 256, 15, 3), (2500, 256, 2048, 24, 1), (2600, 512, 512, 40, 1), (1500, 512, 768, 40, 2),
    # 256-row tiles: k = 1 and more, ragged experts, odd numbers of steps, slices of the last round's tiles on
    # either product
    (2400, 2048, 2048, 3, 1), (1600, 2048, 2048, 4, 2), (2048, 2048, 2048, 1, 1), (2305, 2304, 2048, 1, 1),
    (1600, 1024, 4096, 2, 1), (700, 1280, 4096, 2, 2), (1500, 1792, 3840, 3, 1)]


@pytest.mark.parametrize("T,H,I,E,k", SIZES)
@pytest.mark.parametrize("four", [False, True])
def test_experts(M, T, H, I, E, k, four):
    print(f"[mxfp4] T={T} H={H} I={I} E={E} k={k} four={four}", flush=True)
    d = make(M, T, H, I, E, k, four, seed=T)
    check(d, call(M, d))


@pytest.mark.parametrize("T", [5, 63, 200, 900])
@pytest.mark.parametrize("four", [False, True])
def test_experts_skewed(M, T, four):
    print(f"[mxfp4] skewed T={T} four={four}", flush=True)
    d = make(M, T, 512, 256, 12, 2, four, seed=1, skew=True)
    check(d, call(M, d))


@pytest.mark.parametrize("T,E,k,H,I", [
    (6, 4, 2, 512, 256), (50, 8, 3, 512, 256), (200, 8, 3, 512, 256), (9, 4, 1, 512, 256), (300, 4, 1, 512, 256),
    (900, 3, 1, 512, 256), (1200, 3, 2, 512, 256), (1100, 3, 1, 2048, 2048),
    (600, 3, 2, 4096, 1024),
    (2400, 3, 1, 2048, 2048), (1200, 3, 2, 2048, 2048), (1600, 2, 1, 1024, 4096), (1200, 72, 2, 512, 512), (2500, 72, 1, 512, 512)])
@pytest.mark.parametrize("four", [False, True])
def test_experts_ids_out_of_range(M, T, E, k, H, I, four):
    print(f"[mxfp4] ids out of range T={T} E={E} k={k} H={H} four={four}", flush=True)
    d = make(M, T, H, I, E, k, four, seed=2)
    g = torch.Generator().manual_seed(7)
    off = torch.rand(T, k, generator=g) < 0.4
    off[1] = True                                          # a token without an expert
    bad = torch.tensor([-1, E, 2 ** 31 - 1, -2 ** 31])[torch.randint(0, 4, (T, k), generator=g)].int()
    d["idx"] = torch.where(off, bad, d["idx"].cpu()).int().cuda()
    out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    call(M, d, out=out)
    assert not out[1].view(torch.int16).any()
    check(d, out)
    d["idx"].fill_(-1)
    out.fill_(float("nan"))
    assert not call(M, d, out=out).view(torch.int16).any()


@pytest.mark.parametrize("T,H,I,E,k", [
    (14, 2560, 1792, 5, 5), (100, 4096, 1024, 4, 2), (300, 4096, 1024, 4, 1), (40, 4096, 256, 3, 3), (60, 512, 2048, 4, 4),
    (90, 1536, 1792, 2, 1), (20, 512, 4096, 16, 12), (131, 7168, 256, 1, 1), (70, 16384, 256, 2, 1), (70, 256, 16384, 2, 2)])
@pytest.mark.parametrize("four", [False, True])
def test_experts_few_rows_and_long_reductions(M, T, H, I, E, k, four):
    print(f"[mxfp4] long T={T} H={H} I={I} E={E} k={k} four={four}", flush=True)
    d = make(M, T, H, I, E, k, four, seed=12)
    ws = M.workspace(M.moe_experts_mxfp4_workspace_bytes(T, H, I, E, k, M.MOE_MXFP4 if four else M.MOE_MXFP8))
    ws.fill_(255)
    ref = call(M, d, ws=ws)
    check(d, ref)
    for seed in (1, 2, 3):
        M.moe_set_debug_options(M.MOE_DEBUG_PERMUTE_ORDER, seed)
        assert torch.equal(call(M, d), ref)
    M.moe_set_debug_options(0, 0)
    d["idx"][1] = E                                         # a token without an expert, a slot without one
    d["idx"][2, 0] = -1
    out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    call(M, d, out=out)
    assert not out[1].view(torch.int16).any()
    check(d, out)


@pytest.mark.parametrize("four", [False, True])
def test_experts_same_expert_twice(M, four):
    for T in (3, 40, 500):
        d = make(M, T, 512, 256, 6, 3, four, seed=3)
        d["idx"][:, 2] = d["idx"][:, 0]
        check(d, call(M, d))


@pytest.mark.parametrize("T,H,I", [(4, 512, 256), (90, 512, 256), (700, 512, 256), (1600, 2048, 2048)])
@pytest.mark.parametrize("four", [False, True])
def test_experts_zero_rows(M, T, H, I, four):
    d = make(M, T, H, I, 4, 2, four, seed=4)
    d["x"][0] = 0
    d["xs"][0] = 0                                          # as a row of zeros is coded
    d["xs"][1] = 0                                          # values of 2^-127
    d["wg"][2] = 0                                          # an expert that answers 0
    out = call(M, d)
    assert not out[0].any()
    check(d, out)


@pytest.mark.parametrize("T,H,I", [(6, 512, 512), (70, 512, 512), (300, 512, 512), (1200, 2048, 2048)])
@pytest.mark.parametrize("four", [False, True])
def test_experts_far_apart_scales(M, T, H, I, four):
    """Blocks whose scales lie far apart, on both operands; activations that saturate silu."""
    d = make(M, T, H, I, 3, 2, four, seed=5)
    g = torch.Generator(device="cuda").manual_seed(1)
    d["sg"] = (d["sg"].int() + torch.randint(-18, 3, d["sg"].shape, generator=g, device="cuda")).to(torch.uint8)
    d["xs"] = (d["xs"].int() + torch.randint(-12, 4, d["xs"].shape, generator=g, device="cuda")).to(torch.uint8)
    d["sd"] = (d["sd"].int() + torch.randint(-12, 4, d["sd"].shape, generator=g, device="cuda")).to(torch.uint8)
    check(d, call(M, d))


@pytest.mark.parametrize("T,E,k,H,I", [(3, 8, 2, 512, 256), (90, 8, 2, 512, 256), (700, 4, 2, 512, 256),
                                       (2400, 3, 1, 2048, 2048), (1300, 3, 2, 2048, 2048), (800, 72, 2, 512, 512), (1800, 72, 1, 512, 512)])
@pytest.mark.parametrize("four", [False, True])
def test_experts_bad_token_leaves_the_others(M, T, E, k, H, I, four):
    """A token with a NaN scale, and an expert with one: only that token's, and that expert's tokens'
    outputs change."""
    d = make(M, T, H, I, E, k, four, seed=6)
    ref = call(M, d)
    xs = d["xs"].clone()
    xs[2, 1] = 255
    got = call(M, dict(d, xs=xs))
    keep = torch.arange(T, device="cuda") != 2
    assert torch.equal(got[keep], ref[keep])
    sg = d["sg"].clone()
    sg[1] = 255
    got = call(M, dict(d, sg=sg))
    keep = ~(d["idx"] == 1).any(dim=1)
    assert torch.equal(got[keep], ref[keep])


@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 512, 512), (40, 8, 2, 512, 512), (500, 8, 2, 512, 512), (900, 2, 1, 2048, 2048),
                                       (700, 2, 2, 4096, 1024), (2100, 2, 1, 2048, 2048), (1050, 2, 2, 2048, 2048),
                                       (1600, 2, 1, 1024, 4096), (2305, 1, 1, 2304, 2048), (800, 72, 2, 512, 512), (1800, 72, 1, 512, 512),
                                       (2400, 72, 2, 512, 512), (5000, 72, 1, 512, 512)])
@pytest.mark.parametrize("four", [False, True])
def test_experts_deterministic_and_order_free(M, T, E, k, H, I, four):
    print(f"[mxfp4] order T={T} E={E} k={k} four={four}", flush=True)
    d = make(M, T, H, I, E, k, four, seed=9)
    ws = M.workspace(M.moe_experts_mxfp4_workspace_bytes(T, H, I, E, k, M.MOE_MXFP4 if four else M.MOE_MXFP8))
    ws.zero_()
    ref = call(M, d, ws=ws)
    ws.fill_(255)                                           # its contents do not matter
    assert torch.equal(call(M, d, ws=ws), ref)
    for seed in range(4):
        M.moe_set_debug_options(M.MOE_DEBUG_PERMUTE_ORDER if seed else 0, seed)
        assert torch.equal(call(M, d), ref)
    M.moe_set_debug_options(0, 0)


@pytest.mark.parametrize("T", [4, 90, 600, 164000, 404000])
@pytest.mark.parametrize("four", [False, True])
def test_experts_large_offsets(M, T, four):
    """An expert array beyond 2^32 bytes and the last experts in it."""
    H, I, E, k = 2048, 2048, 1024, 2
    d = make(M, T, H, I, 2, k, four, seed=11)
    big = {"wg": torch.zeros(E, 2 * I, H // 2, dtype=torch.uint8, device="cuda"),
           "sg": torch.zeros(E, 2 * I, H // 32, dtype=torch.uint8, device="cuda"),
           "wd": torch.zeros(E, H, I // 2, dtype=torch.uint8, device="cuda"),
           "sd": torch.zeros(E, H, I // 32, dtype=torch.uint8, device="cuda")}
    for n, t in big.items():
        t[E - 2:] = d[n]
    moved = dict(d, **big, idx=d["idx"] + (E - 2))
    out = call(M, moved)                                    # (404000: 256-row tiles)
    check(d, out, rows=slice(T - 40 if T > 40 else 0, T))
    assert E * I * H >= 2 ** 32


@pytest.mark.parametrize("four", [False, True])
def test_experts_many_rows_and_short_reductions(M, four):
    d = make(M, 41000, 512, 512, 2, 1, four, seed=16)
    out = call(M, d)
    check(d, out, rows=slice(0, 200))
    check(d, out, rows=slice(40800, 41000))


@pytest.mark.parametrize("T,E,k,H,I", [(1, 16, 4, 512, 256), (60, 16, 4, 512, 256), (300, 8, 2, 512, 256), (900, 2, 1, 2048, 2048),
                                       (700, 2, 2, 4096, 1024), (2100, 2, 1, 2048, 2048), (1050, 2, 2, 2048, 2048)])
@pytest.mark.parametrize("four", [False, True])
def test_experts_graph_replays(M, T, E, k, H, I, four):
    """Captured and replayed, with eager work of the program's own between the replays; two
    graphs that share one workspace, replayed in turn."""
    print(f"[mxfp4 graph] T={T} E={E} k={k} four={four}", flush=True)
    ds = [make(M, T, H, I, E, k, four, seed=20 + j) for j in range(2)]
    ref = [call(M, d) for d in ds]
    ws = M.workspace(M.moe_experts_mxfp4_workspace_bytes(T, H, I, E, k, M.MOE_MXFP4 if four else M.MOE_MXFP8))
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
@pytest.mark.parametrize("four", [False, True])
def test_experts_one_slot_zero_and_negative_weights(M, H, I, E, four):
    """k = 1: a weight of 0 or less; a zero's sign is that of the product in every form."""
    print(f"[mxfp4] one slot H={H} I={I} E={E} four={four}", flush=True)
    d = make(M, 2100, H, I, E, 1, four, seed=13)                # (256-row tiles at H 2048 I 2048)
    d["w"][::3] = 0
    d["w"][1::3] *= -1
    full = call(M, d)
    check(d, full, rows=slice(0, 300))
    zero = full[::3].view(torch.int16)
    assert ((zero == 0) | (zero == -2 ** 15)).all() and (zero == 0).any() and (zero != 0).any()
    for rows in (slice(0, 1), slice(3, 4), slice(5, 12), slice(0, 20), slice(0, 48), slice(100, 190), slice(0, 400)):
        part = call(M, part_of(d, rows))
        check(part_of(d, rows), part, rows=slice(0, 20))
        none = (d["w"][rows] == 0).reshape(-1)
        assert not part[none].any() and (torch.signbit(part[none]).any() or none.sum() == 0)


@pytest.mark.parametrize("H,I,E,k", [(2560, 1792, 5, 5), (2048, 2048, 2, 1), (4096, 1024, 4, 2)])
@pytest.mark.parametrize("four", [False, True])
def test_experts_one_workspace_for_all_batches(M, H, I, E, k, four):
    """Sized once, for the largest batch: every smaller one is taken, and its outputs are
    those with a workspace of its own."""
    print(f"[mxfp4] one workspace H={H} I={I} E={E} k={k} four={four}", flush=True)
    most = 2100
    d = make(M, most, H, I, E, k, four, seed=14)
    ws = M.workspace(M.moe_experts_mxfp4_workspace_bytes(most, H, I, E, k, M.MOE_MXFP4 if four else M.MOE_MXFP8))
    ws.fill_(255)
    for T in (1, 2, 3, 9, 14, 40, 48, 100, 123, 300, 383, 700, 1025, most):
        part = part_of(d, slice(0, T))
        assert torch.equal(call(M, part, ws=ws), call(M, part)), T


def test_experts_empty_batch(M):
    for four in (False, True):
        d = make(M, 4, 512, 256, 4, 2, four)
        assert call(M, part_of(d, slice(0, 0))).shape == (0, 512)


def test_experts_small_workspace_is_refused(M):
    d = make(M, 100, 512, 256, 4, 2, True)
    n = M.moe_experts_mxfp4_workspace_bytes(100, 512, 256, 4, 2, M.MOE_MXFP4)
    with pytest.raises(M.MoeError) as e:
        call(M, d, ws=M.workspace(n - 1))
    assert e.value.status == M.MOE_ERR_WORKSPACE


def test_experts_against_the_batched_mxfp8_layer(M):
    """Weights that both formats hold exactly: E2M1 codes as E4M3 codes give the layer of the batched
    MXFP8 calls, up to the order of sums."""
    T, H, I, E, k = 300, 512, 256, 6, 2
    d = make(M, T, H, I, E, k, False, seed=15)
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    lut = torch.cat([lut, -lut]).to(torch.float8_e4m3fn).view(torch.uint8)
    wide = lambda c: lut[torch.stack([c & 15, c >> 4], dim=-1).flatten(-2).int()]  # noqa: E731
    h, hs, ws = M.moe_gate_up_3d_batched(d["x"], wide(d["wg"]), d["idx"], k, M.MOE_MXFP8, x_scales=d["xs"],
                                         w_gate_up_scales=d["sg"])
    ref = M.moe_down_3d_batched(h, wide(d["wd"]), d["idx"], d["w"], ws, k, M.MOE_MXFP8, h_scales=hs, w_down_scales=d["sd"])
    out, slack = reference(d)
    both = np.abs(_f64(call(M, d)) - _f64(ref))
    assert np.all(both <= 2 * ((np.abs(out) + slack) * 2.0 ** -8 + slack))
