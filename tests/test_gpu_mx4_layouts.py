"""4-bit matrices in memory layouts that the header allows, against the 64-bit
definitions (tests/mx4_ref.py): bit for bit."""
import numpy as np
import pytest
import torch

import fsdp_sharded_state_amd as fs
import mx4_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu

CANARY = 0xA5
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _side_by_side(rows, cols):
    """A matrix whose rows hold their codes and then their scales, in one buffer with bytes between the rows."""
    nb = ref.blocks(cols)
    buf = torch.full((rows, (17 * nb + 15) // 16 * 16 + 16), CANARY, dtype=torch.uint8, device="cuda")
    return fs.Mx4Matrix(buf[:, :16 * nb], buf[:, 16 * nb:17 * nb], cols), buf


@pytest.mark.parametrize("rows,cols", [(2, 33), (77, 130), (300, 1000), (17000, 530)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_codes_and_scales_side_by_side(rows, cols, dtype):
    say("side by side", rows, cols, dtype)
    x = torch.randn(rows, cols, generator=_gen(rows + cols), device="cuda").to(DT[dtype])
    by_row, by_col = fs.fs_mx4_empty(rows, cols), fs.fs_mx4_empty(cols, rows)
    fs.fs_mx4_quantize(x, by_row, by_col)
    for want, x_out in ((by_row, (0, None)), (by_col, (None, 0))):
        q, buf = _side_by_side(*want.shape)
        fs.fs_mx4_quantize(x, q if x_out[0] == 0 else None, q if x_out[1] == 0 else None)
        nb = ref.blocks(want.shape[1])
        assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales) and (buf[:, 17 * nb:] == CANARY).all()
        a, b = (torch.empty(want.shape, dtype=DT[dtype], device="cuda") for _ in range(2))
        fs.fs_mx4_dequantize(q, a)
        fs.fs_mx4_dequantize(want, b)
        assert torch.equal(a, b)
        other = fs.fs_mx4_empty(40, want.shape[1])
        fs.fs_mx4_quantize(torch.randn(40, want.shape[1], generator=_gen(3), device="cuda"), other)
        a, b = (torch.empty(want.shape[0], 40, device="cuda") for _ in range(2))
        fs.fs_mx4_matmul(q, other, a)
        fs.fs_mx4_matmul(want, other, b)
        assert torch.equal(a, b)
    assert np.array_equal(by_row.codes[:50].cpu().numpy(), ref.encode_matrix(x[:50].float().cpu().double().numpy())[0])
