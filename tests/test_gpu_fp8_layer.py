"""A linear layer Y = X W^T and its gradients on the E4M3 operators
(include/mswz_fp8.h), against the tensors that were quantised.

Whole numbers up to 8 are E4M3 values at every power-of-two scale up to 64, and
so are those up to 7 at the scale 7 / 448 = 2^-6, so their quantisation loses
nothing, and their products' sums, below 2^24, are exact: Y and the gradients,
and the change of <dY, Y> from one W or X to another, have to be those of the
formulas, bit for bit.

With values of all sizes a quantised value is within 2^-4 |v| + 2^-10 s of v:
half a step of three mantissa bits, or of the smallest subnormal values.  A sum
of products a b of such values is within
    sum (|a| + da) (|b| + db) - |a| |b|,  da = 2^-4 |a| + 2^-10 sa
of the sum of the values' own, and the product's own error comes on top.
"""
import pytest
import torch

import mma_swizzled_operand_amd as mswz
from test_gpu_fp8 import DT, E4M3, blocks, expand, fp8_reference, gen, mp

pytestmark = pytest.mark.gpu

SIZES = [(100, 144, 272), (256, 128, 256), (1, 160, 128), (333, 528, 400), (515, 1040, 784)]   # M, N, K


def quantised(t, block, scales):
    """t as it lies and transposed: {"q": (values, scales), "t": ...}."""
    R, C = t.shape
    plan = mswz.quant_fp8_plan_create(R, C, {v: k for k, v in DT.items()}[t.dtype], block, scales)
    Q, QT = torch.empty(R, C, dtype=E4M3, device="cuda"), torch.empty(C, mp(R), dtype=E4M3, device="cuda")
    if block == "row":
        S, ST = torch.empty(blocks(C), R, device="cuda"), torch.empty(blocks(R), C, device="cuda")
    else:
        S, ST = torch.empty(blocks(R), blocks(C), device="cuda"), torch.empty(blocks(C), blocks(R), device="cuda")
    mswz.quant_fp8(plan, t, Q=Q, S=S, QT=QT, ST=ST)
    return {"q": (Q, S), "t": (QT, ST)}


def product(a, b, block, d, D=None):
    """A . B^T, added to D where one is given."""
    m, k, n = a[0].shape[0], a[0].shape[1], b[0].shape[0]
    plan = mswz.gemm_fp8_plan_create(m, n, k, d, block)
    ws = torch.empty(max(16, plan.workspace_bytes()), dtype=torch.uint8, device="cuda")
    out = torch.empty(m, n, dtype=DT[d], device="cuda") if D is None else D
    mswz.gemm_run_fp8(plan, *a, *b, out, beta=0 if D is None else 1, workspace=ws)
    return out


def whole_numbers(g, scales, *shape):
    """Of few bits; with scales that are no powers of two every block's largest is 7."""
    most = 8 if scales == "pow2" else 7
    t = torch.randint(-most, most + 1, shape, generator=g)
    if scales == "f32":      # one in every block along a row, along a column and of a tile
        t[:, ::128] = 7
        t[::128, :] = -7
    return t.to(torch.bfloat16).cuda()


@pytest.mark.parametrize("scales", ["f32", "pow2"])
@pytest.mark.parametrize("d", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_layer_of_whole_numbers(M, N, K, d, scales):
    """The formulas' Y, dX and dW, a second batch added to dW, and the differences of <dY, Y>."""
    g = gen(M * N + K)
    X, X1, W, W1, dY = (whole_numbers(g, scales, *s) for s in ((M, K), (M, K), (N, K), (N, K), (M, N)))
    x, x1, dy = (quantised(t, "row", scales) for t in (X, X1, dY))
    w, w1 = (quantised(t, "tile", scales) for t in (W, W1))
    dX = product(dy["q"], w["t"], "tile", d)
    dW = product(dy["t"], x["t"], "row", d)
    Y = product(x["q"], w["q"], "tile", d)
    v = {name: t.double() for name, t in (("X", X), ("X1", X1), ("W", W), ("W1", W1), ("dY", dY))}
    assert torch.equal(Y, (v["X"] @ v["W"].t()).to(DT[d]))
    assert torch.equal(dX, (v["dY"] @ v["W"]).to(DT[d]))
    assert torch.equal(dW, (v["dY"].t() @ v["X"]).to(DT[d]))
    if d == "f32":
        # <dY, Y> is linear in W and in X: its differences are the gradients' products with the steps
        def of(y):
            return (v["dY"] * y.double()).sum()

        assert of(product(x["q"], w1["q"], "tile", d)) - of(Y) == (dW.double() * (v["W1"] - v["W"])).sum()
        assert of(product(x1["q"], w["q"], "tile", d)) - of(Y) == (dX.double() * (v["X1"] - v["X"])).sum()
    before = dW.double()
    product(dy["t"], x1["t"], "row", d, D=dW)
    assert torch.equal(dW, (before + v["dY"].t() @ v["X1"]).to(DT[d]))


@pytest.mark.parametrize("scales", ["f32", "pow2"])
@pytest.mark.parametrize("d", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SIZES[:4])
def test_layer_of_any_values(M, N, K, d, scales):
    """Operands near the tensors that they were made from, as they lie and transposed; Y, dX and dW near the formulas'
    of those tensors."""
    g = gen(M + N * K)
    tensors = {"X": (M, K, "row"), "W": (N, K, "tile"), "dY": (M, N, "row")}
    value, size, q = {}, {}, {}
    for name, (R, C, block) in tensors.items():
        t = (torch.randn(R, C, generator=g) * torch.exp(torch.randn(C, generator=g))).to(torch.bfloat16).cuda()
        q[name], value[name] = quantised(t, block, scales), t.double().cpu()
        for form in ("q", "t"):
            code, s = (u.cpu() for u in q[name][form])
            v = value[name] if form == "q" else value[name].t()
            S = expand(s, code.shape[1], block == "tile", code.shape[0])[:, :v.shape[1]]
            off = 2.0 ** -4 * v.abs() + 2.0 ** -10 * S
            assert ((code.double()[:, :v.shape[1]] * S - v).abs() <= off).all(), (name, form)
            assert not code[:, v.shape[1]:].view(torch.uint8).any()
            size[name, form] = v, v.abs() + off
    for a, af, b, bf, block in (("X", "q", "W", "q", "tile"), ("dY", "q", "W", "t", "tile"), ("dY", "t", "X", "t", "row")):
        got = product(q[a][af], q[b][bf], block, d).double().cpu()
        (va, ma), (vb, mb) = size[a, af], size[b, bf]
        tol = ma @ mb.t() - va.abs() @ vb.abs().t()
        codes = [u.cpu().view(torch.uint8) if u.dtype is E4M3 else u.cpu() for u in (*q[a][af], *q[b][bf])]
        tol = tol + fp8_reference(*codes, block == "tile", d == "f32")[1]
        if d != "f32":
            tol = tol * (1 + torch.finfo(DT[d]).eps) + torch.finfo(DT[d]).eps / 2 * (va @ vb.t()).abs()
        assert ((got - va @ vb.t()).abs() <= tol).all(), (a, b)
