"""The workspaces that the MXFP4 and balance calls make for themselves live until their kernels are
enqueued (no GPU: tensors on the host, and a stand-in where the library would be called)."""
import torch

from tests.test_binding_memory import m  # noqa: F401


def test_experts_mxfp4_holds_its_workspace(m):  # noqa: F811
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    m.moe_experts_mxfp4(u8(4, 512), u8(4, 16), u8(8, 512, 256), u8(8, 512, 16), u8(8, 512, 128), u8(8, 512, 8),
                        torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))


def test_balance_loss_holds_its_workspace(m):  # noqa: F811
    m.moe_balance_loss(torch.zeros(12, 32), torch.zeros(12, 4, dtype=torch.int32), n_seqs=3)
