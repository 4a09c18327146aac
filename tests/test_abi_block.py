"""Refusals of the norm, scored-routing and INT8 calls: arguments are checked on the
host before anything is enqueued (no GPU needed)."""
import os

import pytest
import torch


@pytest.fixture(scope="module")
def m():
    import mixture_experts_ffn_07_amd as M
    return M


FAKE = 0x10000        # a 16-byte aligned address that is never dereferenced
OFF = FAKE + 8


def _norm(m, x=FAKE, r=None, w=FAKE, T=4, H=512, eps=1e-6, ro=None, y=FAKE, q=0, codes=None, scales=None):
    return m.lib.moe_add_rmsnorm(x, r, w, T, H, eps, ro, y, q, codes, scales, None)


def test_norm_refusals(m):
    for T in (-1, 1 << 22, 2 ** 31 - 1):
        assert _norm(m, T=T) == m.MOE_ERR_SHAPE, T
    for H in (0, -32, 31, 48, 16384 + 32):
        assert _norm(m, H=H) == m.MOE_ERR_SHAPE, H
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert _norm(m, eps=eps) == m.MOE_ERR_SHAPE, eps
    assert _norm(m, q=3) == m.MOE_ERR_SHAPE
    assert _norm(m, q=-1) == m.MOE_ERR_SHAPE
    assert _norm(m, ro=FAKE) == m.MOE_ERR_NULL                    # no residual to sum
    assert _norm(m, x=None) == m.MOE_ERR_NULL
    assert _norm(m, w=None) == m.MOE_ERR_NULL
    assert _norm(m, y=None) == m.MOE_ERR_NULL
    assert _norm(m, y=None, q=1, codes=FAKE) == m.MOE_ERR_NULL
    assert _norm(m, y=None, q=2, scales=FAKE) == m.MOE_ERR_NULL
    assert _norm(m, r=FAKE, ro=2 * FAKE, y=2 * FAKE) == m.MOE_ERR_UNSUPPORTED
    for bad in (dict(x=OFF), dict(w=OFF), dict(y=OFF), dict(r=OFF), dict(r=FAKE, ro=OFF),
                dict(q=1, codes=OFF, scales=FAKE), dict(q=2, codes=FAKE, scales=OFF)):
        assert _norm(m, **bad) == m.MOE_ERR_ALIGN, bad
    assert _norm(m, x=None, w=None, y=None, T=0) == m.MOE_OK       # nothing to do


def test_norm_backward_refusals(m):
    def call(s=FAKE, w=FAKE, dy=FAKE, ds=None, T=4, H=512, eps=1e-6, dx=FAKE, dw=FAKE, ws=FAKE, n=None):
        n = m.lib.moe_add_rmsnorm_backward_workspace_bytes(T, H) if n is None else n
        return m.lib.moe_add_rmsnorm_backward(s, w, dy, ds, T, H, eps, dx, dw, ws, n, None)
    need = m.lib.moe_add_rmsnorm_backward_workspace_bytes(4, 512)
    assert need >= 4 * 512 * 4
    assert m.lib.moe_add_rmsnorm_backward_workspace_bytes(-1, 512) == 0
    for T in (-1, 1 << 22, 2 ** 31 - 1):
        assert call(T=T, n=1 << 40) == m.MOE_ERR_SHAPE, T
    assert call(H=40) == m.MOE_ERR_SHAPE
    assert call(eps=0.0) == m.MOE_ERR_SHAPE
    for bad in (dict(s=None), dict(w=None), dict(dy=None), dict(dx=None), dict(dw=None)):
        assert call(**bad) == m.MOE_ERR_NULL, bad
    assert call(ws=None) == m.MOE_ERR_WORKSPACE
    assert call(n=need - 1) == m.MOE_ERR_WORKSPACE
    for bad in (dict(s=OFF), dict(w=OFF), dict(dy=OFF), dict(ds=OFF), dict(dx=OFF), dict(dw=OFF), dict(ws=OFF)):
        assert call(**bad) == m.MOE_ERR_ALIGN, bad


def _route(m, l=FAKE, b=None, T=4, E=32, k=4, G=1, tg=1, gt=1, score=0, rn=1, sc=1.0, i=FAKE, w=FAKE):
    return m.lib.moe_route_scored(l, b, T, E, k, G, tg, gt, score, rn, sc, i, w, None)


def test_route_scored_refusals(m):
    for bad in (dict(T=-1), dict(T=1 << 22), dict(T=2 ** 31 - 1), dict(E=0), dict(E=1025), dict(k=0), dict(k=33, E=64), dict(k=5, E=4),
                dict(G=0), dict(G=5), dict(G=128, E=1024), dict(G=4, tg=0), dict(G=4, tg=5),
                dict(gt=0), dict(gt=3), dict(G=8, tg=1, k=5), dict(score=2), dict(score=-1),
                dict(sc=float("nan")), dict(sc=float("inf"))):
        assert _route(m, **bad) == m.MOE_ERR_SHAPE, bad
    for bad in (dict(l=None), dict(i=None), dict(w=None)):
        assert _route(m, **bad) == m.MOE_ERR_NULL, bad
    for bad in (dict(l=OFF), dict(b=OFF), dict(i=OFF), dict(w=OFF)):
        assert _route(m, **bad) == m.MOE_ERR_ALIGN, bad
    assert _route(m, l=None, i=None, w=None, T=0) == m.MOE_OK


def test_route_scored_backward_refusals(m):
    def call(l=FAKE, i=FAKE, d=FAKE, T=4, E=32, k=4, score=1, sc=1.0, o=FAKE):
        return m.lib.moe_route_scored_backward(l, i, d, T, E, k, score, 1, sc, o, None)
    for bad in (dict(T=-1), dict(T=1 << 22), dict(T=2 ** 31 - 1), dict(E=1025), dict(k=0), dict(k=33), dict(score=7), dict(sc=float("inf"))):
        assert call(**bad) == m.MOE_ERR_SHAPE, bad
    for bad in (dict(l=None), dict(i=None), dict(d=None), dict(o=None)):
        assert call(**bad) == m.MOE_ERR_NULL, bad
    for bad in (dict(l=OFF), dict(i=OFF), dict(d=OFF), dict(o=OFF)):
        assert call(**bad) == m.MOE_ERR_ALIGN, bad
    assert call(l=None, i=None, d=None, o=None, T=0) == m.MOE_OK


def test_quantize_int8_refusals(m):
    q = m.lib.moe_quantize_int8
    for rows, K in ((-1, 64), (1 << 29, 64), (4, 0), (4, 48), (4, 16384 + 32)):
        assert q(FAKE, rows, K, FAKE, FAKE, None) == m.MOE_ERR_SHAPE, (rows, K)
    for a in ((None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None)):
        assert q(a[0], 4, 64, a[1], a[2], None) == m.MOE_ERR_NULL
    assert q(OFF, 4, 64, FAKE, FAKE, None) == m.MOE_ERR_ALIGN
    assert q(None, 0, 64, None, None, None) == m.MOE_OK


def test_experts_int8_refusals(m):
    def call(T=4, H=512, I=256, E=8, k=2, ws=FAKE, n=None, **p):
        a = {n_: FAKE for n_ in ("x", "xs", "wg", "sg", "wd", "sd", "i", "w", "out")}
        a.update(p)
        n = m.lib.moe_experts_int8_workspace_bytes(T, H, I, E, k) if n is None else n
        return m.lib.moe_experts_int8(a["x"], a["xs"], a["wg"], a["sg"], a["wd"], a["sd"], a["i"], a["w"],
                                      T, H, I, E, k, a["out"], ws, n, None)
    need = m.lib.moe_experts_int8_workspace_bytes(4, 512, 256, 8, 2)
    assert need > 4 * 2 * 256 * 4
    assert m.lib.moe_experts_int8_workspace_bytes(0, 512, 256, 8, 2) == 0
    big = 1 << 40
    for bad in (dict(T=-1, n=big), dict(H=384), dict(I=128), dict(H=16640), dict(I=16640), dict(E=0, n=big),
                dict(E=1025), dict(k=0, n=big), dict(k=9), dict(k=33, E=64), dict(T=1 << 22, H=1024, n=big),
                dict(T=1 << 17, H=16384, k=8, n=big)):
        assert call(**bad) == m.MOE_ERR_SHAPE, bad
    for name in ("x", "xs", "wg", "sg", "wd", "sd", "i", "w", "out"):
        assert call(**{name: None}) == m.MOE_ERR_NULL, name
        assert call(**{name: OFF}) == m.MOE_ERR_ALIGN, name
    assert call(ws=None) == m.MOE_ERR_WORKSPACE
    assert call(n=need - 1) == m.MOE_ERR_WORKSPACE
    assert call(T=0, ws=None, x=None, out=None) == m.MOE_OK


@pytest.mark.parametrize("T", [-5, 0, 1, 3, 1000, 2 ** 31 - 1])
@pytest.mark.parametrize("E,k", [(1, 1), (8, 2), (1024, 32), (2 ** 31 - 1, 2 ** 31 - 1), (0, 0), (-1, -1)])
def test_workspace_queries_answer_for_any_sizes(m, T, E, k):
    """Sizes that the calls themselves refuse come in through the queries too."""
    for H in (-256, 0, 1, 64, 255, 256, 4096, 2 ** 31 - 1):
        assert m.lib.moe_add_rmsnorm_backward_workspace_bytes(T, H) >= 0
        for I in (-128, 0, 1, 64, 127, 128, 255, 256, 2 ** 31 - 1):
            n = m.lib.moe_experts_int8_workspace_bytes(T, H, I, E, k)
            assert n >= 0 and (n == 0 or min(T, H, I, E, k) >= 1)


def test_int8_is_not_a_type_of_the_batched_calls(m):
    assert m.lib.moe_workspace_bytes(4, 512, 256, 8, 2, m.MOE_INT8) == 0
    assert m.lib.moe_gate_up_3d_batched(FAKE, None, FAKE, None, FAKE, 4, 512, 256, 8, 2, m.MOE_INT8, FAKE,
                                        None, FAKE, 1 << 30, None) == m.MOE_ERR_SHAPE


def test_binding_refuses_before_a_pointer_is_handed_over(m):
    x = torch.zeros(4, 512, dtype=torch.bfloat16)
    w = torch.zeros(512, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                 # on the host
        m.moe_add_rmsnorm(x, w, 1e-6)
    with pytest.raises(TypeError):
        m.moe_add_rmsnorm(x.float(), w, 1e-6)
    with pytest.raises(ValueError):
        m.moe_add_rmsnorm(x, w[:256], 1e-6)
    with pytest.raises(ValueError):
        m.moe_add_rmsnorm(x, w, 1e-6, residual=x[:3])
    with pytest.raises(ValueError):
        m.moe_add_rmsnorm_backward(x, w, x, 1e-6, ws=torch.zeros(16, dtype=torch.uint8))
    with pytest.raises(TypeError):
        m.moe_route_scored(torch.zeros(4, 8, dtype=torch.float64), 2)
    with pytest.raises(ValueError):
        m.moe_route_scored(torch.zeros(4, 8), 2, bias=torch.zeros(7))
    with pytest.raises(TypeError):
        m.moe_route_scored_backward(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2))
    with pytest.raises(TypeError):
        m.moe_quantize_int8(x.float())
    i8 = lambda *s: torch.zeros(*s, dtype=torch.int8)  # noqa: E731
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    idx, tw = torch.zeros(4, 2, dtype=torch.int32), f(4, 2)
    with pytest.raises(ValueError):                 # scales of the wrong length
        m.moe_experts_int8(i8(4, 512), f(4), i8(8, 512, 512), f(8, 511), i8(8, 512, 256), f(8, 512), idx, tw)
    with pytest.raises(ValueError):                 # an odd number of gate/up rows
        m.moe_experts_int8(i8(4, 512), f(4), i8(8, 513, 512), f(8, 512), i8(8, 512, 256), f(8, 512), idx, tw)


def test_header_names_every_binding(m):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "moe_mi355x.h")).read()
    for name in m._SIGS:
        assert name + "(" in text, name


@pytest.mark.parametrize("H,I,E,k", [
    (7168, 2048, 6, 1), (7168, 2048, 2, 1), (2048, 768, 128, 8), (4096, 1024, 6, 4), (2560, 1792, 5, 5), (4096, 1024, 64, 6),
    (512, 256, 8, 2), (16384, 256, 1, 1), (256, 16384, 3, 2), (1536, 4096, 32, 12), (1024, 2048, 3, 1)])
def test_int8_workspace_for_a_batch_serves_smaller_ones(m, H, I, E, k):
    q = lambda T: m.lib.moe_experts_int8_workspace_bytes(T, H, I, E, k)  # noqa: E731
    T = list(range(1, 2500)) + list(range(2500, 40000, 37))
    n = [q(t) for t in T]
    worse = [(T[i], n[i], T[i + 1], n[i + 1]) for i in range(len(T) - 1) if n[i + 1] < n[i]]
    assert not worse, worse[:3]


@pytest.mark.parametrize("H", [32, 512, 4096, 7168])
def test_norm_backward_workspace_for_a_batch_serves_smaller_ones(m, H):
    n = [m.lib.moe_add_rmsnorm_backward_workspace_bytes(t, H) for t in range(3000)]
    assert n == sorted(n)
