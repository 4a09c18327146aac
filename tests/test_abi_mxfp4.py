"""Refusals of the MXFP4 and balance-loss calls: arguments are checked on the host before anything
is enqueued (no GPU needed)."""
import pytest
import torch


@pytest.fixture(scope="module")
def m():
    import mixture_experts_ffn_07_amd as M
    return M


FAKE = 0x10000        # a 16-byte aligned address that is never dereferenced
OFF = FAKE + 8
BIG = 1 << 50


@pytest.mark.parametrize("name", ["moe_quantize_mxfp4", "moe_dequantize_mxfp4"])
def test_row_refusals(m, name):
    def call(rows=4, K=64, a=FAKE, b=FAKE, c=FAKE):
        if name == "moe_quantize_mxfp4":
            return m.lib.moe_quantize_mxfp4(a, rows, K, b, c, None)
        return m.lib.moe_dequantize_mxfp4(a, b, rows, K, c, None)
    for bad in (dict(rows=-1), dict(K=0), dict(K=-32), dict(K=31), dict(K=48), dict(rows=1 << 40), dict(rows=2 ** 62),
                dict(rows=(1 << 40) // 64, K=64)):
        assert call(**bad) == m.MOE_ERR_SHAPE, bad
    for n in "abc":
        assert call(**{n: None}) == m.MOE_ERR_NULL
        assert call(**{n: OFF}) == m.MOE_ERR_ALIGN
    assert call(rows=0, a=None, b=None, c=None) == m.MOE_OK


def test_experts_refusals(m):
    names = ("x", "xs", "wg", "sg", "wd", "sd", "i", "w", "out")

    def call(T=4, H=512, I=256, E=8, k=2, q=m.MOE_MXFP4, ws=FAKE, n=BIG, **p):
        a = {n_: FAKE for n_ in names}
        a.update(p)
        return m.lib.moe_experts_mxfp4(a["x"], a["xs"], q, a["wg"], a["sg"], a["wd"], a["sd"], a["i"], a["w"],
                                       T, H, I, E, k, a["out"], ws, n, None)
    for q in (m.MOE_BF16, m.MOE_INT8, 4, -1, 2 ** 31 - 1):
        assert call(q=q) == m.MOE_ERR_SHAPE, q
    for bad in (dict(T=-1), dict(H=384), dict(H=0), dict(I=128), dict(I=-256), dict(H=16640), dict(I=16640), dict(E=0),
                dict(E=1025), dict(k=0), dict(k=9), dict(k=33, E=64), dict(T=1 << 22, H=1024),
                dict(T=1 << 17, H=16384, k=8), dict(H=16384, I=16384 * 4)):
        for q in (m.MOE_MXFP8, m.MOE_MXFP4):
            assert call(q=q, **bad) == m.MOE_ERR_SHAPE, bad
    for name in names:
        assert call(**{name: None}) == m.MOE_ERR_NULL, name
        assert call(**{name: OFF}) == m.MOE_ERR_ALIGN, name
    for q in (m.MOE_MXFP8, m.MOE_MXFP4):
        need = m.lib.moe_experts_mxfp4_workspace_bytes(4, 512, 256, 8, 2, q)
        assert need > 4 * 2 * 512 * 4
        assert call(q=q, n=need - 1) == m.MOE_ERR_WORKSPACE
    assert call(ws=None) == m.MOE_ERR_WORKSPACE
    assert call(ws=OFF) == m.MOE_ERR_ALIGN
    assert call(T=0, ws=None, n=0, **{n_: None for n_ in names}) == m.MOE_OK


def test_experts_workspace_query(m):
    q = m.lib.moe_experts_mxfp4_workspace_bytes
    for T, H, I, E, k, t in ((0, 512, 256, 8, 2, 1), (4, 0, 256, 8, 2, 1), (4, 512, 0, 8, 2, 1), (4, 512, 256, 0, 2, 1),
                             (4, 512, 256, 8, 0, 1), (4, 512, 256, 8, 2, 0), (4, 512, 256, 8, 2, 2), (4, 300, 256, 8, 2, 3),
                             (4, 512, 100, 8, 2, 3), (-1, 512, 256, 8, 2, 3), (4, 512, 256, 8, 9, 3)):
        assert q(T, H, I, E, k, t) == 0
    # it does not fall as T grows
    for H, I, E, k in ((256, 256, 1, 1), (2048, 768, 128, 8), (4096, 1024, 4, 2), (7168, 2048, 6, 1), (2560, 1792, 5, 5),
                       (16384, 256, 3, 3), (256, 16384, 2, 1), (1024, 512, 1024, 32)):
        for t in (m.MOE_MXFP8, m.MOE_MXFP4):
            last = 0
            for T in list(range(1, 700)) + list(range(700, 9000, 37)):
                n = q(T, H, I, E, k, t)
                assert n >= last, (T, H, I, E, k, t)
                last = n


def test_balance_refusals(m):
    names = ("l", "i", "losses", "counts", "probs", "tokens")

    def call(T=12, E=32, k=4, S=3, score=0, mask=None, ws=FAKE, n=BIG, **p):
        a = {n_: FAKE for n_ in names}
        a.update(p)
        return m.lib.moe_balance_loss(a["l"], a["i"], mask, T, E, k, S, score, a["losses"], a["counts"], a["probs"],
                                      a["tokens"], ws, n, None)
    for bad in (dict(T=-3), dict(T=1 << 22, S=1), dict(E=0), dict(E=1025), dict(k=0), dict(k=33, E=64), dict(k=5, E=4),
                dict(S=0), dict(S=-1), dict(S=5), dict(T=8194, S=4097), dict(score=2), dict(score=-1)):
        assert call(**bad) == m.MOE_ERR_SHAPE, bad
    for name in names:
        assert call(**{name: None}) == m.MOE_ERR_NULL, name
        assert call(**{name: OFF}) == m.MOE_ERR_ALIGN, name
    assert call(mask=OFF) == m.MOE_ERR_ALIGN
    assert call(ws=None) == m.MOE_ERR_WORKSPACE
    assert call(ws=OFF) == m.MOE_ERR_ALIGN
    need = m.lib.moe_balance_loss_workspace_bytes(12, 32, 3)
    assert need > 0 and call(n=need - 1) == m.MOE_ERR_WORKSPACE
    for T, E, S in ((-1, 32, 1), (1 << 22, 32, 1), (12, 0, 1), (12, 1025, 1), (12, 32, 0), (12, 32, 4097)):
        assert m.lib.moe_balance_loss_workspace_bytes(T, E, S) == 0


@pytest.mark.parametrize("S", [1, 2, 3, 8, 1000, 4096])
def test_balance_workspace_does_not_fall(m, S):
    last = 0
    for L in list(range(0, 600)) + list(range(600, 1000000 // S, 977)):
        if L * S < 1 << 22:
            n = m.lib.moe_balance_loss_workspace_bytes(L * S, 384, S)
            assert n >= last
            last = n


def test_balance_backward_refusals(m):
    names = ("l", "counts", "tokens", "d", "o")

    def call(T=12, E=32, S=3, score=1, mask=None, add=None, **p):
        a = {n_: FAKE for n_ in names}
        a.update(p)
        return m.lib.moe_balance_loss_backward(a["l"], mask, a["counts"], a["tokens"], a["d"], add, T, E, S, score,
                                               a["o"], None)
    for bad in (dict(T=-3), dict(T=1 << 22, S=1), dict(E=0), dict(E=1025), dict(S=0), dict(S=5), dict(T=8194, S=4097),
                dict(score=2)):
        assert call(**bad) == m.MOE_ERR_SHAPE, bad
    for name in names:
        assert call(**{name: None}) == m.MOE_ERR_NULL, name
        assert call(**{name: OFF}) == m.MOE_ERR_ALIGN, name
    assert call(mask=OFF) == m.MOE_ERR_ALIGN
    assert call(add=OFF) == m.MOE_ERR_ALIGN
    assert call(T=0, S=1, **{n_: None for n_ in names}) == m.MOE_OK


def test_binding_refuses_before_a_pointer_is_taken(m):
    u8, i32 = torch.uint8, torch.int32
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype)  # noqa: E731
    with pytest.raises(ValueError):                        # not on a GPU
        m.moe_quantize_mxfp4(z(4, 64, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        m.moe_quantize_mxfp4(z(4, 64))
    with pytest.raises(ValueError):
        m.moe_quantize_mxfp4(z(4, 64, 1, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        m.moe_quantize_mxfp4(z(4, 64, dtype=torch.bfloat16), codes=z(4, 64, dtype=u8))
    with pytest.raises(ValueError):
        m.moe_dequantize_mxfp4(z(4, 32, dtype=u8), z(4, 4, dtype=u8))
    e = dict(x=z(4, 512, dtype=u8), xs=z(4, 16, dtype=u8), wg=z(8, 512, 256, dtype=u8), sg=z(8, 512, 16, dtype=u8),
             wd=z(8, 512, 128, dtype=u8), sd=z(8, 512, 8, dtype=u8), i=z(4, 2, dtype=i32), w=z(4, 2))
    for name, t in (("x", z(4, 256, dtype=u8)), ("x", z(4, 512)), ("xs", z(4, 8, dtype=u8)), ("wg", z(8, 256, 256, dtype=u8)),
                    ("sg", z(8, 512, 8, dtype=u8)), ("sd", z(8, 512, 16, dtype=u8)), ("i", z(4, 2, dtype=torch.int64)),
                    ("i", z(8, dtype=i32)), ("w", z(4, 1)), ("wd", z(512, 128, dtype=u8))):
        with pytest.raises((TypeError, ValueError)):
            m.moe_experts_mxfp4(*{**e, name: t}.values())
    with pytest.raises(ValueError):                        # MXFP4 activations are half as wide
        m.moe_experts_mxfp4(*e.values(), xtype=m.MOE_MXFP4)
    l, idx = z(12, 32), z(12, 4, dtype=i32)
    for kw in (dict(token_mask=z(12)), dict(token_mask=z(11, dtype=u8)), dict(counts=z(1, 32)), dict(losses=z(3)),
               dict(probs=z(2, 32)), dict(tokens=z(1))):
        with pytest.raises((TypeError, ValueError)):
            m.moe_balance_loss(l, idx, **kw)
    with pytest.raises((TypeError, ValueError)):
        m.moe_balance_loss_backward(l, z(1, 32, dtype=i32), z(2, dtype=i32), z(2))
    with pytest.raises((TypeError, ValueError)):
        m.moe_balance_loss_backward(l, z(1, 31, dtype=i32), z(1, dtype=i32), z(2))
