"""The sign of what quant_fp8 (include/mswz_fp8.h) rounds to zero: that of the
value, whichever way the block's scale was rounded."""
import pytest
import torch

import mma_swizzled_operand_amd as mswz

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.parametrize("scales", ["f32", "pow2"])
@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_zeros_keep_their_sign(dt, block, scales):
    """Zeros of both signs, and values far below half of the smallest step, in blocks whose largest value runs through
    the mantissas (m / 448 is rounded up for some of them and down for others) and is infinite in one."""
    rows = cols = 128 * 17
    x = torch.zeros(rows, cols)
    x[:, 0::4] = -0.0
    x[:, 1::4] = 2.0 ** -18     # (448 / 255 * 2^-18 is far below the smallest step's half, 2^-10)
    x[:, 2::4] = -2.0 ** -18
    # one largest value a block along a row, along a column and of a tile
    i, j = torch.arange(17)[:, None], torch.arange(17)[None, :]
    most = 128.0 + (31 * i + 7 * j) % 128
    most[16, 16] = float("inf")
    for r in range(128):
        x[128 * i + r, 128 * j + r] = most
    x = x.to(DT[dt])
    plan = mswz.quant_fp8_plan_create(rows, cols, dt, block, scales)
    tiles = (17, 17)
    Q, QT = (torch.full((rows, cols), 0x55, dtype=torch.uint8, device="cuda") for _ in range(2))
    S, ST = (torch.zeros(tiles if block == "tile" else (17, rows), device="cuda") for _ in range(2))
    mswz.quant_fp8(plan, x.cuda(), Q=Q, S=S, QT=QT, ST=ST)
    want = torch.where(torch.signbit(x), 0x80, 0).to(torch.uint8)
    small = x.abs() < 1
    assert torch.equal(Q.cpu()[small], want[small])
    assert torch.equal(QT.cpu().t()[small], want[small])
    assert (Q.cpu()[~small] & 0x7F >= 0x70).all()     # (the largest are not zeros)
