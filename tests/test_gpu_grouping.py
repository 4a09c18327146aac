"""The expert grouping behind the batched calls, over batches around the sizes where its kernel
changes form: the rows of h come expert by expert, ascending pairs within one.  Inputs whose
products and sums are exact in FP32, so that a row out of place shows at once."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import mixture_experts_ffn_07_amd as M
    return M


SIZES = [(1, 1), (65, 1), (1023, 1), (1024, 1), (1025, 1), (512, 2), (4095, 1), (1024, 4), (4097, 1), (2731, 6), (16384, 1),
         (16385, 1), (2100, 8)]


@pytest.mark.parametrize("T,k,E", [(T, k, E) for T, k in SIZES for E in (1, 7, 9, 384) if k <= E])
@pytest.mark.parametrize("skew", [False, True])
def test_rows_by_expert(M, T, k, E, skew):
    print(f"[grouping] T={T} k={k} E={E} skew={skew}", flush=True)
    H = I = 256
    g = torch.Generator(device="cuda").manual_seed(T + E)
    x = torch.randint(-1, 2, (T, H), generator=g, device="cuda").bfloat16()
    w = (torch.randint(-4, 5, (E, 2 * I, H), generator=g, device="cuda") / 64).bfloat16()
    l = torch.randn(T, E, generator=g, device="cuda")
    if skew:
        l[:, E // 2:] -= 100                            # half of the experts get nothing (but where slots run out)
    idx = l.topk(k, dim=1).indices.int().contiguous()
    h, _, _ = M.moe_gate_up_3d_batched(x, w, idx, k)
    pair_expert = idx.reshape(-1).long()
    order = torch.argsort(pair_expert, stable=True)
    xs, es = x.float()[order // k], pair_expert[order]
    for e in range(E):
        rows = (es == e).nonzero().reshape(-1)
        if rows.numel() == 0:
            continue
        gu = xs[rows] @ w[e].float().t()
        ref = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        # half a BF16 step, and FP32's error of silu (an exponential of an argument below 16 and a division)
        assert ((h[rows].float() - ref).abs() <= ref.abs() * (2.0 ** -8 + 32 * 2.0 ** -24)).all(), e


@pytest.mark.parametrize("T,H", [(3, 512), (70, 1024), (700, 256)])
def test_slot_sums_of_any_number_of_slots(M, T, H):
    """Further slots of weight 0 leave the output's bits as they are, whichever form of the slot
    sum their number selects."""
    I, E, most = 256, 256, 13
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, wg, wd = r(T, H).bfloat16(), (r(E, 2 * I, H) / 16).bfloat16(), (r(E, H, I) / 16).bfloat16()
    idx = r(T, E).topk(most, dim=1).indices.int()
    w = torch.rand(T, most, generator=g, device="cuda")

    def layer(n, k):
        i = idx[:, :k].contiguous()
        wk = w[:, :k].clone()
        wk[:, n:] = 0
        h, _, ws = M.moe_gate_up_3d_batched(x, wg, i, k)
        return M.moe_down_3d_batched(h, wd, i, wk, ws, k)
    for n in (2, 3, 4, 5, 8, 9):
        ref = layer(n, n)
        assert ref.any()
        for k in range(n + 1, most + 1):
            assert torch.equal(layer(n, k), ref), (n, k)
