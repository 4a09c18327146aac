"""Memory that the binding allocates for a call, looked at without a GPU: tensors on the host,
and a stand-in where the library would be called."""
import weakref

import pytest
import torch

EPS = 1e-6


@pytest.fixture
def m(monkeypatch):
    import mixture_experts_ffn_07_amd as M
    made, make = [], M.workspace

    def note(nbytes, device="cuda"):
        t = make(nbytes, device)
        made.append((weakref.ref(t), t.data_ptr()))
        return t

    def enqueue(name, dev, stream, *args):
        calls.append(name)
        assert made and all(r() is not None for r, _ in made), f"{name}: its workspace is gone before the launch"
        assert made[-1][1] in args
    calls = []
    monkeypatch.setattr(M, "workspace", note)
    monkeypatch.setattr(M, "_enqueue", enqueue)
    yield M
    assert len(calls) == len(made) == 1


def test_norm_backward_holds_its_workspace(m):
    x = torch.zeros(4, 512, dtype=torch.bfloat16)
    m.moe_add_rmsnorm_backward(x, x[0].clone(), x.clone(), EPS)


def test_experts_int8_holds_its_workspace(m):
    i8 = lambda *s: torch.zeros(*s, dtype=torch.int8)  # noqa: E731
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    m.moe_experts_int8(i8(4, 512), f(4), i8(8, 512, 512), f(8, 512), i8(8, 512, 256), f(8, 512),
                       torch.zeros(4, 2, dtype=torch.int32), f(4, 2))
