"""What a product of E4M3 operands writes (include/mswz_fp8.h): its columns of D
and nothing else, in every kernel that a plan may take, whatever D's width,
pitch and alignment.

Values are 0, +-1, +-2 and scales 1, 2, 4, so every sum is a whole number below
2^24 (K 6160 at most: 6160 * 4 * 16) and exact on every way through the matrix
unit; D is its one rounding and is compared bit for bit, with its surroundings.
"""
import pytest
import torch

import mma_swizzled_operand_amd as mswz
from test_gpu_fp8 import close, fp8_inputs, fp8_reference, fp8_run, gen

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
GUARD = 7.5   # what the buffer holds where nothing may be written

# rows, columns (a multiple of 8, to which up to 4 are added) and K by kernel: the
# tile, or the rows that the kernel without barriers holds, or the split of K
SHAPES = {
    "few16": (5, 200, 272), "few32": (22, 200, 272), "split": (70, 200, 6160), "32x64": (40, 200, 272),
    "64x64": (70, 6000, 272), "128x64": (700, 1512, 1040), "128x128": (700, 3000, 528), "128x128 twice": (700, 6000, 272),
    "256x256": (1500, 6000, 272),
}
# fp32 D: other tiles are worth their time
SHAPES_F32 = {**SHAPES, "128x64": (97, 12400, 3520), "128x128": (1500, 2512, 272)}
del SHAPES_F32["256x256"]

CASES = [(kernel, d) for d in DT for kernel in (SHAPES_F32 if d == "f32" else SHAPES)]


def shape_of(kernel, d):
    return (SHAPES_F32 if d == "f32" else SHAPES)[kernel]


def blocks(n):
    return -(-n // 128)


@pytest.mark.parametrize("more", [1, 2, 3, 4])
@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("kernel,d", CASES)
def test_product_writes_its_columns_only(kernel, d, block, more):
    """N of 1, 2 and 3 past a multiple of four, and of 4 past one of eight; pitches that are multiples of 4 and of 8;
    D aligned to 16 bytes, to four elements, and to one."""
    M, N, K = shape_of(kernel, d)
    N += more
    kb = blocks(K)
    g = torch.Generator(device="cuda").manual_seed(N + K)
    A = torch.randint(-2, 3, (M, K), generator=g, device="cuda").float().to(E4M3)
    B = torch.randint(-2, 3, (N, K), generator=g, device="cuda").float().to(E4M3)
    SA = torch.exp2(torch.randint(0, 3, (kb, M), generator=g, device="cuda").float())
    SB = torch.exp2(torch.randint(0, 3, (blocks(N), kb) if block == "tile" else (kb, N), generator=g, device="cuda").float())
    s = SB.repeat_interleave(128, 0)[:N] if block == "tile" else SB.t()
    a = A.double() * SA.t().double().repeat_interleave(128, 1)[:, :K]
    ref = a @ (B.double() * s.double().repeat_interleave(128, 1)[:, :K]).t()
    old = torch.randint(-8, 9, (M, N), generator=g, device="cuda")
    fours, eights = (N // 8 + 1) * 8 + 4, (N // 8 + 1) * 8
    for pitch, start in ((fours, 32), (eights, 32), (eights, 36), (eights, 33)):
        plan = mswz.gemm_fp8_plan_create(M, N, K, d, block, ldd=pitch)
        ws = torch.empty(max(16, plan.workspace_bytes()), dtype=torch.uint8, device="cuda")
        flat, want = (torch.full((start + M * pitch + 64,), GUARD, dtype=DT[d], device="cuda") for _ in range(2))
        assert flat.data_ptr() % 16 == 0
        D, E = (t[start:start + M * pitch].view(M, pitch)[:, :N] for t in (flat, want))
        E.copy_(ref.to(DT[d]))
        mswz.gemm_run_fp8(plan, A, SA, B, SB, D, workspace=ws)
        assert torch.equal(flat, want), (pitch, start)
        D.copy_(old)
        E.copy_((ref + old).to(DT[d]))
        mswz.gemm_run_fp8(plan, A, SA, B, SB, D, beta=1, workspace=ws)
        assert torch.equal(flat, want), (pitch, start, "beta")


@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("kernel,d", CASES)
def test_all_codes_by_every_kernel(kernel, d, block):
    """Every finite code of both operands, subnormal ones and zeros among them: rows and columns at the edges of
    tiles and in between, within the tolerance that test_gpu_fp8.py derives."""
    M, N, K = shape_of(kernel, d)
    N += 3
    x = fp8_inputs(gen(M + N), M, N, K, block, subnormal=True)
    x["SA"] *= 0.1      # (sums stay inside fp16)
    plan = mswz.gemm_fp8_plan_create(M, N, K, d, block)
    got = fp8_run(plan, x, torch.full((M, N), float("nan"), dtype=DT[d], device="cuda")).cpu()
    assert torch.isfinite(got).all()
    rows = torch.tensor(sorted({0, M // 2, M - 1, min(31, M - 1), min(64, M - 1)}))
    ref, tol = fp8_reference(x["A"][rows], x["SA"][:, rows], x["B"], x["SB"], block == "tile", d == "f32")
    close(got[rows], ref, tol, d, "rows")
    cols = torch.tensor([0, 15, 63, 64, 127, 128, N // 2, N - 2, N - 1])
    sb = x["SB"][cols // 128].t().contiguous() if block == "tile" else x["SB"][:, cols]
    ref, tol = fp8_reference(x["A"], x["SA"], x["B"][cols], sb, False, d == "f32")
    close(got[:, cols], ref, tol, d, "columns")
