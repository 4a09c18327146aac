"""Workloads of the operators for MXFP4 experts and for balancing the router, case by case.

Four operators of a block with routed experts:

  mxfp4             BF16 rows to MXFP4 (4-bit codes, one scale per 32) and back to their values
  experts_mxfp4     the routed experts' products with MXFP4 weights and MXFP8 or MXFP4
                    activations (gate/up, SwiGLU, down, weighted sum)
  balance           the router's balance loss and z-loss, tokens per expert, mean scores
  balance_backward  their gradient, added to the one that reaches the logits elsewhere

`run` computes a case in elementary torch operations (`own` false) or with the
library's kernels (`own` true); `exact` computes it once more in 64 bits.
"""
import math

import torch

own = False

BF16 = torch.bfloat16


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # a decode step's few activation rows on their way into MXFP4 experts: latency
        dict(name="mxfp4-T8", op="mxfp4", rows=8, K=4096),
        # a ragged batch of rows whose length fills no tile
        dict(name="mxfp4-T1001", op="mxfp4", rows=1001, K=2080),
        # weights on their way into memory: gate/up of six experts
        dict(name="mxfp4-weights", op="mxfp4", rows=24576, K=7168),
        # one token in decode: the touched experts' weights once
        dict(name="experts-T1-a8", op="experts_mxfp4", T=1, H=2048, I=768, E=128, k=8, x="mxfp8", padded=0),
        # a decode batch that touches nearly every expert, some of its places empty
        dict(name="experts-T64-a4", op="experts_mxfp4", T=64, H=2048, I=768, E=128, k=8, x="mxfp4", padded=5),
        # a ragged batch of some hundred tokens, tens of rows to an expert
        dict(name="experts-T777-a8", op="experts_mxfp4", T=777, H=4096, I=1024, E=64, k=6, x="mxfp8", padded=0),
        # one GPU's share under expert parallelism: thousands of rows to each of a few experts
        dict(name="experts-T16384-a4", op="experts_mxfp4", T=16384, H=7168, I=2048, E=6, k=1, x="mxfp4", padded=0),
        # a prefill batch with MXFP8 activations, about a thousand rows to an expert
        dict(name="experts-T4095-a8", op="experts_mxfp4", T=4095, H=2048, I=1024, E=16, k=4, x="mxfp8", padded=0),
        # a training micro-batch, sigmoid scores, one sequence
        dict(name="balance-T2048", op="balance", T=2048, E=384, k=8, score="sigmoid", seqs=1, padded=False),
        # a large batch of eight sequences with padding, softmax scores
        dict(name="balance-T32768", op="balance", T=32768, E=256, k=8, score="softmax", seqs=8, padded=True),
        # the gradients of both, the second on top of the gradient of the routing weights
        dict(name="balance-bwd-T2048", op="balance_backward", T=2048, E=384, k=8, score="sigmoid", seqs=1,
             padded=False, add=False),
        dict(name="balance-bwd-T32768", op="balance_backward", T=32768, E=256, k=8, score="softmax", seqs=8,
             padded=True, add=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["mxfp4", "experts_mxfp4", "experts_mxfp4", "experts_mxfp4", "balance", "balance_backward"])
    if op == "mxfp4":
        K = 32 * _log(rng, 4, 512)
        return dict(op=op, rows=_log(rng, 1, (1 << 27) // K), K=K)
    if op == "experts_mxfp4":
        H, I = 256 * rng.randint(2, 16), 256 * rng.randint(1, 8)
        E = _log(rng, 4, 128)
        k = rng.randint(1, min(8, E))
        T = _log(rng, 1, min(8192, (1 << 37) // (k * H * I)))
        return dict(op=op, T=T, H=H, I=I, E=E, k=k, x=rng.choice(["mxfp8", "mxfp4"]),
                    padded=rng.choice([0, 0, T // 10]))
    seqs = rng.choice([1, 1, 2, 3, 8])
    E = _log(rng, 4, 512)
    c = dict(op=op, T=seqs * _log(rng, 1, 32768 // seqs), E=E, k=rng.randint(1, min(8, E)),
             score=rng.choice(["softmax", "sigmoid"]), seqs=seqs, padded=rng.random() < 0.4)
    if op == "balance_backward":
        c["add"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------------------
# formats

def _nearest_e2m1(a):
    """Indexes 0..7 of the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 to magnitudes a, ties to the even index."""
    fine = torch.round(a * 2.0)                  # steps of 0.5 up to 2
    mid = torch.round(a) + 2.0                   # of 1 up to 4
    wide = torch.round(a * 0.5) + 4.0            # of 2 up to 6 (torch.round: ties to even)
    return torch.where(a < 2.0, fine, torch.where(a < 4.0, mid, wide)).clamp_max(7.0).to(torch.uint8)


def _table(dtype, device):
    v = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(v + [-x for x in v], dtype=dtype, device=device)


def _blocks(v):
    return v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)


def _mx_exp(amax, emax):
    """floor(log2 amax) - emax in [-127, 127]; -127 for an all-zero block."""
    _, e = torch.frexp(amax)                     # amax = m 2^e, m in [0.5, 1)
    return torch.where(amax == 0, -127, e - 1 - emax).clamp(-127, 127)


def _power(e):
    """2^e in 32 bits, e in [-127, 127], as its bit pattern (2^-127 lies below the normal range)."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _to_mxfp4(v):
    """FP32 [..., K] -> nibbles [..., K] uint8 and scale codes [..., K/32] uint8."""
    b = _blocks(v)
    e = _mx_exp(b.abs().amax(dim=-1), 2)
    y = b * _power(-e).unsqueeze(-1)
    return (_nearest_e2m1(y.abs()) | torch.signbit(y).to(torch.uint8) << 3).view(v.shape), (e + 127).to(torch.uint8)


def _to_mxfp8(v):
    """FP32 [..., K] -> E4M3 values as uint8 codes [..., K] and scale codes [..., K/32] uint8."""
    b = _blocks(v)
    e = _mx_exp(b.abs().amax(dim=-1), 8)
    y = (b * _power(-e).unsqueeze(-1)).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn).view(torch.uint8).view(v.shape), (e + 127).to(torch.uint8)


def _pack(n):
    """Nibbles, two to a byte: the even element in the low half."""
    return n[..., 0::2] | n[..., 1::2] << 4


def _unpack(codes):
    return torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)


def _scale(scales, dtype):
    e = scales.to(torch.int32) - 127
    return _power(e).unsqueeze(-1) if dtype == torch.float32 else torch.ldexp(
        torch.ones((), dtype=dtype, device=e.device), e).unsqueeze(-1)


def _values4(codes, scales, dtype=torch.float32):
    """MXFP4 [..., K/2], [..., K/32] -> values [..., K]."""
    v = _table(dtype, codes.device)[_unpack(codes).int()]
    return (_blocks(v) * _scale(scales, dtype)).view(v.shape)


def _values8(codes, scales, dtype=torch.float32):
    v = codes.view(torch.float8_e4m3fn).to(dtype)
    return (_blocks(v) * _scale(scales, dtype)).view(v.shape)


# ---------------------------------------------------------------------------
# inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 29)
    return g


def _stream(T, H, g):
    """Normed activations: unit noise, a few channels much larger than the rest."""
    gain = torch.ones(H, device="cuda")
    gain[torch.randint(0, H, (max(1, H // 512),), generator=g, device="cuda")] = 12.0
    return torch.randn(T, H, generator=g, device="cuda") * gain


def _weights(E, R, K, g):
    """MXFP4 weights of N(0, 0.02^2), some experts at a time."""
    codes = torch.empty(E, R, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, R, K // 32, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (R * K))
    for e in range(0, E, step):
        n, s = _to_mxfp4(torch.randn(min(step, E - e), R, K, generator=g, device="cuda") * 0.02)
        codes[e:e + step], scales[e:e + step] = _pack(n), s
    return codes, scales


def _logits(T, E, g):
    return torch.randn(T, E, generator=g, device="cuda") * 1.5 + torch.randn(E, generator=g, device="cuda") * 0.5


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    op = case["op"]
    if op == "mxfp4":
        rows, K = case["rows"], case["K"]
        s["v"] = _stream(rows, K, g).to(BF16)
        s["codes"] = torch.empty(rows, K // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(rows, K // 32, dtype=torch.uint8, device="cuda")
        s["values"] = torch.empty(rows, K, dtype=BF16, device="cuda")
    elif op == "experts_mxfp4":
        T, H, I, E, k = (case[n] for n in "THIEk")
        x = _stream(T, H, g)
        if case["x"] == "mxfp4":
            n, s["x_scales"] = _to_mxfp4(x)
            s["x_codes"] = _pack(n)
        else:
            s["x_codes"], s["x_scales"] = _to_mxfp8(x)
        s["wgu"], s["wgu_scales"] = _weights(E, 2 * I, H, g)
        s["wd"], s["wd_scales"] = _weights(E, H, I, g)
        top, idx = _logits(T, E, g).topk(k, dim=1)
        if case["padded"]:           # empty places of the batch: routed to no expert
            idx[torch.randperm(T, generator=g, device="cuda")[:case["padded"]]] = -1
        s["idx"] = idx.to(torch.int32)
        s["w"] = torch.softmax(top, dim=1)
        # the most rows an expert gets, known to whoever lays rows out by expert
        s["most"] = int(torch.bincount(idx[idx >= 0], minlength=E).max()) if T > case["padded"] else 1
        s["out"] = torch.empty(T, H, dtype=BF16, device="cuda")
        if own:
            import mixture_experts_ffn_07_amd as M
            s["ws"] = M.workspace(M.moe_experts_mxfp4_workspace_bytes(T, H, I, E, k, _type(M, s)))
    else:
        T, E, k, S = case["T"], case["E"], case["k"], case["seqs"]
        s["logits"] = _logits(T, E, g)
        idx = s["logits"].topk(k, dim=1).indices
        s["mask"] = None
        if case["padded"]:           # every sequence has a length of its own; the rest of it is padding
            length = torch.randint(0, T // S + 1, (S, 1), generator=g, device="cuda")
            s["mask"] = (torch.arange(T // S, device="cuda") < length).reshape(T).to(torch.uint8)
            idx[s["mask"] == 0] = -1
        s["idx"] = idx.to(torch.int32)
        if op == "balance":
            s["losses"] = torch.empty(2, device="cuda")
            s["counts"] = torch.empty(S, E, dtype=torch.int32, device="cuda")
            s["probs"] = torch.empty(S, E, device="cuda")
            s["tokens"] = torch.empty(S, dtype=torch.int32, device="cuda")
            if own:
                import mixture_experts_ffn_07_amd as M
                s["ws"] = M.workspace(M.moe_balance_loss_workspace_bytes(T, E, S))
        else:
            s["counts"], s["tokens"] = _counts(s)
            s["d_losses"] = torch.tensor([1e-2, 1e-3], device="cuda")
            s["d_add"] = torch.randn(T, E, generator=g, device="cuda") * (1e-3 / T) if case["add"] else None
            s["dlogits"] = torch.empty(T, E, device="cuda")
    return s


# ---------------------------------------------------------------------------
# the library's kernels

def _type(M, s):
    return M.MOE_MXFP4 if s["x"] == "mxfp4" else M.MOE_MXFP8


def _score(M, s):
    return M.MOE_SCORE_SOFTMAX if s["score"] == "softmax" else M.MOE_SCORE_SIGMOID


def _own_mxfp4(s):
    import mixture_experts_ffn_07_amd as M
    M.moe_quantize_mxfp4(s["v"], codes=s["codes"], scales=s["scales"])
    M.moe_dequantize_mxfp4(s["codes"], s["scales"], out=s["values"])
    return {"values": s["values"], "scales": s["scales"].view(torch.float8_e8m0fnu)}


def _own_experts_mxfp4(s):
    import mixture_experts_ffn_07_amd as M
    M.moe_experts_mxfp4(s["x_codes"], s["x_scales"], s["wgu"], s["wgu_scales"], s["wd"], s["wd_scales"],
                        s["idx"], s["w"], xtype=_type(M, s), out=s["out"], ws=s["ws"])
    return {"out": s["out"]}


def _own_balance(s):
    import mixture_experts_ffn_07_amd as M
    M.moe_balance_loss(s["logits"], s["idx"], score=_score(M, s), n_seqs=s["seqs"], token_mask=s["mask"],
                       losses=s["losses"], counts=s["counts"], probs=s["probs"], tokens=s["tokens"], ws=s["ws"])
    return {n: s[n] for n in ("losses", "counts", "probs", "tokens")}


def _own_balance_backward(s):
    import mixture_experts_ffn_07_amd as M
    M.moe_balance_loss_backward(s["logits"], s["counts"], s["tokens"], s["d_losses"], score=_score(M, s),
                                token_mask=s["mask"], d_add=s["d_add"], dlogits=s["dlogits"])
    return {"dlogits": s["dlogits"]}


# ---------------------------------------------------------------------------
# plain forms

def _plain_mxfp4(s):
    n, scales = _to_mxfp4(s["v"].float())
    codes = _pack(n)                             # as it is kept
    return {"values": _values4(codes, scales).to(BF16), "scales": scales.view(torch.float8_e8m0fnu)}


def _plain_experts_mxfp4(s):
    T, H, I, E, k = (s[n] for n in "THIEk")
    four = s["x"] == "mxfp4"
    x = (_values4 if four else _values8)(s["x_codes"], s["x_scales"])
    pair = torch.nonzero(s["idx"].reshape(-1) >= 0).reshape(-1)
    expert = s["idx"].reshape(-1)[pair].long()
    P = pair.numel()
    if P <= E:            # few pairs: each pair's own expert
        wg, wd = _values4(s["wgu"][expert], s["wgu_scales"][expert]), _values4(s["wd"][expert], s["wd_scales"][expert])
        n, cap, where = P, 1, torch.arange(P, device="cuda")
    else:                 # rows laid out by expert, padded to the most rows an expert gets
        wg, wd = _values4(s["wgu"], s["wgu_scales"]), _values4(s["wd"], s["wd_scales"])
        n, cap = E, s["most"]
        order = torch.argsort(expert, stable=True)
        counts = torch.bincount(expert, minlength=E)
        first = torch.cumsum(counts, 0) - counts
        by_expert = expert[order]
        where = torch.empty_like(order)
        where[order] = by_expert * cap + torch.arange(P, device="cuda") - first[by_expert]
    rows = torch.zeros(n * cap, H, device="cuda")
    rows[where] = x[pair // k]
    gu = torch.bmm(rows.view(n, cap, H), wg.transpose(1, 2))
    gate, up = gu[:, :, :I], gu[:, :, I:]
    a = gate / (1.0 + torch.exp(-gate)) * up
    if four:
        codes, scales = _to_mxfp4(a)
        h = _values4(_pack(codes), scales)
    else:
        h = _values8(*_to_mxfp8(a))
    y = torch.zeros(T * k, H, device="cuda")
    y[pair] = torch.bmm(h, wd.transpose(1, 2)).view(n * cap, H)[where]
    return {"out": (y.view(T, k, H) * s["w"].unsqueeze(2)).sum(dim=1).to(BF16)}


def _counts(s):
    """Pairs per sequence and expert, and tokens per sequence."""
    T, E, S = s["T"], s["E"], s["seqs"]
    seq = torch.arange(T, device="cuda") // (T // S)
    on = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"] != 0
    take = on.unsqueeze(1) & (s["idx"] >= 0) & (s["idx"] < E)
    at = (seq.unsqueeze(1) * E + s["idx"])[take]
    return (torch.bincount(at, minlength=S * E).view(S, E).to(torch.int32),
            torch.bincount(seq[on], minlength=S).to(torch.int32))


def _scores(l, score):
    """Normalised scores, log of the summed exponentials and softmax of logits l, in their type."""
    top = l.amax(dim=1, keepdim=True)
    e = torch.exp(l - top)
    z = e.sum(dim=1, keepdim=True)
    q = e / z
    lse = (top + torch.log(z)).squeeze(1)
    if score == "softmax":
        return q, lse, q
    p = 1.0 / (1.0 + torch.exp(-l))
    return p / p.sum(dim=1, keepdim=True), lse, q


def _plain_balance(s):
    T, E, S = s["T"], s["E"], s["seqs"]
    p, lse, _ = _scores(s["logits"], s["score"])
    on = torch.ones(T, device="cuda") if s["mask"] is None else s["mask"].float()
    counts, tokens = _counts(s)
    # long sums in 64 bits
    P = (p * on.unsqueeze(1)).view(S, T // S, E).sum(dim=1, dtype=torch.float64) / tokens.clamp_min(1).unsqueeze(1)
    f = E * counts.double() / counts.sum(dim=1, keepdim=True).clamp_min(1)
    z = (lse * lse * on).sum(dtype=torch.float64) / tokens.sum().clamp_min(1)
    return {"losses": torch.stack([(f * P).sum() / S, z]).float(), "counts": counts, "probs": P.float(), "tokens": tokens}


def _plain_balance_backward(s):
    T, E, S = s["T"], s["E"], s["seqs"]
    l = s["logits"]
    p, lse, q = _scores(l, s["score"])
    f = E * s["counts"].float() / s["counts"].sum(dim=1, keepdim=True).clamp_min(1)
    f = f.repeat_interleave(T // S, dim=0)
    d = p * (f - (p * f).sum(dim=1, keepdim=True))
    if s["score"] == "sigmoid":
        d = d * (1.0 / (1.0 + torch.exp(l)))
    N = s["tokens"].clamp_min(1).float().repeat_interleave(T // S).unsqueeze(1)
    d = s["d_losses"][0] / S * d / N
    d = d + s["d_losses"][1] * 2.0 / s["tokens"].sum().clamp_min(1) * lse.unsqueeze(1) * q
    if s["mask"] is not None:
        d = torch.where(s["mask"].unsqueeze(1) != 0, d, 0.0)
    return {"dlogits": d if s["d_add"] is None else d + s["d_add"]}


def run(state):
    op = state["op"]
    if own:
        return {"mxfp4": _own_mxfp4, "experts_mxfp4": _own_experts_mxfp4, "balance": _own_balance,
                "balance_backward": _own_balance_backward}[op](state)
    return {"mxfp4": _plain_mxfp4, "experts_mxfp4": _plain_experts_mxfp4, "balance": _plain_balance,
            "balance_backward": _plain_balance_backward}[op](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "mxfp4":
        n = case["rows"] * case["K"]
        return {"bytes": 4 * n + n // 32, "flops": 4 * n}        # rows in, their values and scales out
    if op == "experts_mxfp4":
        T, H, I, E, k = (case[n] for n in "THIEk")
        live = T - case["padded"]
        touched = E * (1.0 - (1.0 - k / E) ** live)              # experts that some token is routed to
        row = H // 2 if case["x"] == "mxfp4" else H
        return {"bytes": touched * 3 * H * I * (0.5 + 1 / 32) + T * (row + H // 32 + 2 * H) + 8 * T * k,
                "flops": 6.0 * live * k * H * I}
    T, E, k, S = case["T"], case["E"], case["k"], case["seqs"]
    if op == "balance":
        return {"bytes": 4 * T * E + 4 * T * k + 8 * S * E + (T if case["padded"] else 0), "flops": 8 * T * E}
    return {"bytes": (12 if case["add"] else 8) * T * E + 4 * S * E + (T if case["padded"] else 0), "flops": 12 * T * E}


# ---------------------------------------------------------------------------
# 64 bits

def _grid_round(v, emax, edges, lowest):
    """Blocks of 32 of v (64 bits) rounded to a grid of `edges` steps to a binade: exact values."""
    b = _blocks(v)
    amax = b.abs().amax(dim=-1, keepdim=True)
    s = (torch.floor(torch.log2(amax.clamp_min(2.0 ** -1000))) - emax).clamp(-127, 127)
    y = b * torch.exp2(-s)
    binade = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** lowest))).clamp_min(lowest)
    step = torch.exp2(binade) / edges
    most = 6.0 if emax == 2 else 448.0
    return ((torch.round(y / step) * step).clamp(-most, most) * torch.exp2(s)).view(v.shape), (s + 127).squeeze(-1)


def _exact_mxfp4(s):
    v, scales = _grid_round(s["v"].double(), 2, 2.0, 0)
    return {"values": v, "scales": torch.exp2(scales - 127.0)}


def _exact_experts_mxfp4(s):
    T, H, I, E = (s[n] for n in "THIE")
    four = s["x"] == "mxfp4"
    x = (_values4 if four else _values8)(s["x_codes"], s["x_scales"], torch.float64)
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = torch.nonzero(s["idx"] == e, as_tuple=True)
        if not t.numel():
            continue
        gu = x[t] @ _values4(s["wgu"][e], s["wgu_scales"][e], torch.float64).t()
        a = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        h = _grid_round(a, 2, 2.0, 0)[0] if four else _grid_round(a, 8, 8.0, -6)[0]
        y = h @ _values4(s["wd"][e], s["wd_scales"][e], torch.float64).t()
        out.index_add_(0, t, s["w"][t, j].double().unsqueeze(1) * y)
    return {"out": out}


def _exact_scores(s):
    l = s["logits"].double()
    lse = torch.logsumexp(l, dim=1)
    q = torch.exp(l - lse.unsqueeze(1))
    if s["score"] == "softmax":
        return q, lse, q, 1.0
    p = torch.sigmoid(l)
    return p / p.sum(dim=1, keepdim=True), lse, q, torch.sigmoid(-l)


def _exact_balance(s):
    T, E, S = s["T"], s["E"], s["seqs"]
    L = T // S
    p, lse, _, _ = _exact_scores(s)
    P = torch.zeros(S, E, dtype=torch.float64, device="cuda")
    counts = torch.zeros(S, E, dtype=torch.int32, device="cuda")
    tokens = torch.zeros(S, dtype=torch.int32, device="cuda")
    total, z, n = 0.0, 0.0, 0
    for i in range(S):
        rows = slice(i * L, (i + 1) * L)
        on = torch.nonzero(s["mask"][rows]).reshape(-1) + i * L if s["mask"] is not None else torch.arange(i * L, (i + 1) * L, device="cuda")
        if not on.numel():
            continue
        ids = s["idx"][on].reshape(-1)
        counts[i] = torch.bincount(ids[ids >= 0], minlength=E).to(torch.int32)
        tokens[i] = on.numel()
        P[i] = p[on].mean(dim=0)
        total += float((P[i] * counts[i]).sum()) * E / max(1, int(counts[i].sum()))
        z += float(lse[on].square().sum())
        n += on.numel()
    return {"losses": torch.tensor([total / S, z / max(1, n)], dtype=torch.float64), "counts": counts, "probs": P,
            "tokens": tokens}


def _exact_balance_backward(s):
    T, E, S = s["T"], s["E"], s["seqs"]
    p, lse, q, slope = _exact_scores(s)
    c = s["counts"].double()
    d0, d1 = (float(v) for v in s["d_losses"])
    total = max(1, int(s["tokens"].sum()))
    d = 2.0 * d1 / total * lse.unsqueeze(1) * q
    for i in range(S):
        rows = slice(i * (T // S), (i + 1) * (T // S))
        up = c[i] * (d0 * E / (S * max(1.0, float(c[i].sum())) * max(1, int(s["tokens"][i]))))
        d[rows] += p[rows] * up - p[rows] * (p[rows] @ up).unsqueeze(1) if s["score"] == "softmax" else \
            p[rows] * slope[rows] * (up - (p[rows] @ up).unsqueeze(1))
    if s["mask"] is not None:
        d[s["mask"] == 0] = 0.0
    return {"dlogits": d if s["d_add"] is None else d + s["d_add"].double()}


def exact(case, seed):
    s = prepare(case, seed)
    return {"mxfp4": _exact_mxfp4, "experts_mxfp4": _exact_experts_mxfp4, "balance": _exact_balance,
            "balance_backward": _exact_balance_backward}[case["op"]](s)
