"""moe_quantize_mxfp4 and moe_dequantize_mxfp4 on more rows than one launch takes (2^31 pieces of eight values)."""
import numpy as np
import pytest
import torch

from oracle import formats as F
from tests.test_gpu_mxfp4 import M, _f64  # noqa: F401

pytestmark = pytest.mark.gpu


def test_rows_of_two_launches(M):  # noqa: F811
    K = 16384
    rows = (1 << 34) // K + 3                               # 34 GB in, 9 GB of codes and scales, 34 GB out
    border = (1 << 34) // K
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    some = [0, border - 1, border, border + 1, rows - 1]
    for r in some:
        x[r] = torch.randn(K, generator=g, device="cuda").bfloat16()
    print("[mxfp4] two launches", flush=True)
    codes = torch.full((rows, K // 2), 255, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, K // 32), 255, dtype=torch.uint8, device="cuda")
    out = torch.full((rows, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    M.moe_quantize_mxfp4(x, codes=codes, scales=scales)
    M.moe_dequantize_mxfp4(codes, scales, out=out)
    rc, rs = F.mxfp4_quantize(_f64(x[some]))
    assert np.array_equal(codes[some].cpu().numpy(), rc) and np.array_equal(scales[some].cpu().numpy(), rs)
    assert np.array_equal(_f64(out[some]), F.mxfp4_dequantize(rc, rs))
    del x
    for r in range(0, rows, 1 << 16):                       # the other rows are zeros: every one was written
        e = min(rows, r + (1 << 16))
        keep = [i for i in some if r <= i < e]
        codes[keep], scales[keep], out[keep] = 0, 0, 0
        assert not codes[r:e].any() and not scales[r:e].any() and not out[r:e].any()
