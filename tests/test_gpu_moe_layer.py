"""The layer of experts for a few tokens (include/mswz_moe_layer.h) against the
definition in 64 bits, through the binding.

Tolerance of an output, from the arithmetic:
* the two sums of the first product, g and u, are fp32: each within
  d = 2 (H + 8) 2^-24 S, S the sum of its terms' magnitudes;
* the activation's slope is at most 1.2, its own error at most
  (16 + 2 |z|) 2^-22 of its value, z the exponential's argument (its argument's
  rounding is an error in the exponent); the value between the products keeps 16
  significant bits (2^-16): a = act(g) u is within
  1.2 d_g |u| + |act(g)| d_u + |a| ((16 + 2 |z|) 2^-22 + 2^-16);
* the second product's sum, and the weighted sum over choices, are fp32 sums of
  up to 4 I + topk terms (a value's two parts, a weight's two);
* the output's rounding is half a step, eps / 2 (fp16: 2^-25 at least).
"""
import math

import pytest
import torch

import mma_swizzled_operand_amd as mswz

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
GUARD = 7.5


def blocks(n):
    return -(-n // 128)


def inputs(seed, T, k, E, H, I, dt, w):
    g = torch.Generator().manual_seed(seed)
    x = {"X": torch.randn(T, H, generator=g).to(DT[dt]), "weights": torch.rand(T, k, generator=g),
         "ids": torch.randint(0, E, (T, k), generator=g, dtype=torch.int32), "S1": None, "S2": None}
    if w == "e4m3":
        for name, rows, cols in (("W1", 2 * I, H), ("W2", H, I)):
            x[name] = (torch.randn(E, rows, cols, generator=g) * 112).clamp(-448, 448).to(E4M3)
        x["S1"] = (0.5 + torch.rand(E, 2, blocks(I), blocks(H), generator=g)) * H ** -0.5 / 112
        x["S2"] = (0.5 + torch.rand(E, blocks(H), blocks(I), generator=g)) * I ** -0.5 / 112
    else:
        x["W1"] = (torch.randn(E, 2 * I, H, generator=g) * H ** -0.5).to(DT[w])
        x["W2"] = (torch.randn(E, H, I, generator=g) * I ** -0.5).to(DT[w])
    return x


def values(x, E, H, I):
    """The weights' values in 64 bits."""
    W1, W2 = x["W1"].double(), x["W2"].double()
    if x["S1"] is not None:
        s1 = x["S1"].double().repeat_interleave(128, 2)[:, :, :I].repeat_interleave(128, 3)[..., :H]
        W1 = W1 * s1.reshape(E, 2 * I, H)
        W2 = W2 * x["S2"].double().repeat_interleave(128, 1)[:, :H].repeat_interleave(128, 2)[..., :I]
    return W1, W2


def reference(x, T, k, E, H, I, act):
    W1, W2 = values(x, E, H, I)
    Y, tol = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        v = x["X"][t].double()
        total = torch.zeros(H, dtype=torch.float64)
        for j in range(k):
            e = int(x["ids"][t, j])
            if not 0 <= e < E:
                continue
            w = float(x["weights"][t, j])
            s, S = W1[e] @ v, W1[e].abs() @ v.abs()
            d = 2 * (H + 8) * 2.0 ** -24 * S
            gate, up = s[:I], s[I:]
            z = gate if act == "silu" else 2 * math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3)
            on = gate / (1 + torch.exp(-z))
            a = on * up
            da = 1.2 * d[:I] * up.abs() + on.abs() * d[I:] + 1.2 * d[:I] * d[I:] + a.abs() * ((16 + 2 * z.abs()) * 2.0 ** -22 + 2.0 ** -16)
            Y[t] += w * (W2[e] @ a)
            mag = W2[e].abs() @ (a.abs() + da)
            tol[t] += abs(w) * (W2[e].abs() @ da + 2 * (4 * I + 8) * 2.0 ** -24 * mag)
            total += abs(w) * mag
        tol[t] += 2 * (k + 8) * 2.0 ** -24 * total
    return Y, tol


def run(plan, x, Y, stream=None, ws=None):
    c = {n: None if v is None else v.cuda() for n, v in x.items()}
    if ws is None:
        ws = torch.full((plan.workspace_bytes(),), 0xFF, dtype=torch.uint8, device="cuda")
    mswz.moe_layer(plan, c["X"], c["ids"], c["weights"], c["W1"], c["W2"], Y, S1=c["S1"], S2=c["S2"], workspace=ws, stream=stream)
    torch.cuda.synchronize()
    return Y


def close(got, ref, tol, dt):
    got = got.double().cpu()
    eps = torch.finfo(DT[dt]).eps
    tol = tol * (1 + eps) + eps / 2 * ref.abs() + (2.0 ** -25 if dt == "f16" else 0)
    assert torch.isfinite(got).all()
    bad = (got - ref).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((got - ref).abs() / tol.clamp(min=1e-300)).max()))


CASES = [  # T, k, E, H, I, dt, w, act
    (1, 1, 1, 8, 8, "f16", "f16", "silu"),
    (1, 1, 1, 16, 16, "bf16", "e4m3", "gelu"),
    (1, 2, 8, 1024, 512, "f16", "f16", "silu"),
    (1, 8, 16, 264, 136, "bf16", "bf16", "silu"),
    (2, 3, 5, 1000, 328, "bf16", "bf16", "gelu"),
    (5, 3, 6, 400, 72, "f16", "f16", "gelu"),
    (16, 4, 32, 512, 256, "bf16", "bf16", "silu"),
    (17, 1, 2, 136, 200, "f16", "f16", "silu"),
    (33, 2, 3, 128, 128, "bf16", "bf16", "silu"),
    (40, 2, 1, 72, 40, "bf16", "bf16", "gelu"),
    (64, 8, 64, 256, 96, "f16", "f16", "silu"),
    (100, 10, 40, 64, 48, "bf16", "bf16", "silu"),
    (1024, 1, 7, 24, 24, "f16", "f16", "silu"),
    (1, 1024, 1000, 16, 16, "bf16", "bf16", "silu"),
    (1, 4, 8, 2048, 1024, "bf16", "e4m3", "silu"),
    (3, 2, 4, 400, 272, "f16", "e4m3", "gelu"),
    (16, 4, 16, 1040, 144, "bf16", "e4m3", "silu"),
    (33, 3, 5, 144, 400, "f16", "e4m3", "silu"),
    (64, 8, 32, 256, 128, "bf16", "e4m3", "gelu"),
    # many rows an expert: the tokens' values by way of LDS, in one kernel or both
    (40, 8, 64, 264, 136, "bf16", "bf16", "silu"),
    (60, 8, 64, 1032, 72, "f16", "f16", "gelu"),
    (64, 8, 16, 1160, 520, "bf16", "bf16", "silu"),
    (128, 8, 12, 1416, 712, "f16", "f16", "silu"),
    (64, 8, 64, 272, 144, "bf16", "e4m3", "gelu"),
    (96, 10, 40, 528, 208, "f16", "e4m3", "silu"),
    (128, 8, 16, 1040, 528, "bf16", "e4m3", "silu"),
    (100, 4, 2, 264, 4104, "bf16", "bf16", "silu"),
    (100, 4, 2, 8208, 72, "f16", "f16", "gelu"),
]


def skewed(x, T, k, E, seed):
    """Choices of very unequal experts: one with half of them, some with one, some left out."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    ids[torch.rand(T, k, generator=g) < 0.5] = E // 2
    ids[torch.rand(T, k, generator=g) < 0.05] = -1
    ids[ids == E - 1] = E
    x["ids"] = ids


@pytest.mark.parametrize("T,k,E,H,I,dt,w", [
    (64, 8, 64, 264, 136, "bf16", "bf16"), (64, 8, 64, 264, 136, "f16", "f16"), (64, 8, 64, 272, 144, "bf16", "e4m3"),
    (64, 8, 64, 272, 144, "f16", "e4m3"), (70, 6, 5, 136, 72, "bf16", "bf16"), (70, 6, 5, 144, 80, "f16", "e4m3"),
    (128, 8, 40, 520, 264, "bf16", "bf16"), (17, 1, 3, 72, 40, "f16", "f16"),
])
def test_unequal_experts(T, k, E, H, I, dt, w):
    x = inputs(T * E, T, k, E, H, I, dt, w)
    skewed(x, T, k, E, T)
    plan = mswz.moe_layer_plan_create(T, k, E, H, I, dt, w)
    ref, tol = reference(x, T, k, E, H, I, "silu")
    got = run(plan, x, torch.full((T, H), float("nan"), dtype=DT[dt], device="cuda"))
    close(got, ref, tol, dt)
    again = run(plan, x, torch.zeros((T, H), dtype=DT[dt], device="cuda"))
    assert torch.equal(got, again)


@pytest.mark.parametrize("T,k,E,H,I,dt,w,act", CASES)
def test_layer(T, k, E, H, I, dt, w, act):
    x = inputs(T + H, T, k, E, H, I, dt, w)
    plan = mswz.moe_layer_plan_create(T, k, E, H, I, dt, w, act)
    ref, tol = reference(x, T, k, E, H, I, act)
    got = run(plan, x, torch.full((T, H), float("nan"), dtype=DT[dt], device="cuda"))
    close(got, ref, tol, dt)
    again = run(plan, x, torch.zeros((T, H), dtype=DT[dt], device="cuda"))
    assert torch.equal(got, again)


@pytest.mark.parametrize("T,k,E,H,I,w", [(64, 8, 48, 1032, 520, "bf16"), (64, 8, 48, 1040, 528, "e4m3"), (20, 4, 36, 1096, 600, "bf16"),
                                         (20, 4, 36, 1104, 592, "e4m3")])
def test_layer_starts_inside_rows(T, k, E, H, I, w):
    """Two choices an expert and more, many experts: workgroups that start at every place of a row whose last chunk is
    not whole."""
    test_layer(T, k, E, H, I, "bf16", w, "gelu")


@pytest.mark.parametrize("w", ["bf16", "e4m3"])
def test_choices_left_out(w):
    """Ids of other devices, tokens without any expert, all tokens to one expert, the same expert twice."""
    T, k, E, H, I = 37, 3, 6, 144, 80
    for what in ("some", "none", "one", "twice", "bad"):
        x = inputs(7, T, k, E, H, I, "bf16", w)
        if what == "some":
            x["ids"][::3] = -1
            x["ids"][1::3, 1] = E
        elif what == "none":
            x["ids"][:] = -1
        elif what == "one":
            x["ids"][:] = 4
        elif what == "twice":
            x["ids"][:, 1] = x["ids"][:, 0]
        else:
            x["ids"][::2, 0] = -2 ** 31
            x["ids"][1::2, 1] = 2 ** 31 - 1
            x["weights"][::2, 0] = float("nan")     # of a choice left out: not read into the sum
        x["ids"][5] = E + 9
        plan = mswz.moe_layer_plan_create(T, k, E, H, I, "bf16", w)
        ref, tol = reference(x, T, k, E, H, I, "silu")
        got = run(plan, x, torch.full((T, H), float("nan"), dtype=DT["bf16"], device="cuda"))
        close(got, ref, tol, "bf16")
        assert (got[5] == 0).all()


def test_wide_range():
    """fp16 values whose product between the two matrices is beyond fp16's range, and gates far out on both sides."""
    T, k, E, H, I = 4, 2, 3, 64, 64
    x = inputs(11, T, k, E, H, I, "f16", "f16")
    x["X"] *= 600
    x["W1"] *= 4
    x["W2"] *= 2.0 ** -12
    plan = mswz.moe_layer_plan_create(T, k, E, H, I, "f16")
    ref, tol = reference(x, T, k, E, H, I, "silu")
    W1, _ = values(x, E, H, I)
    s = W1[int(x["ids"][0, 0])] @ x["X"][0].double()
    assert float((s[:I] * s[I:]).max()) > 1e6 and float(ref.abs().max()) < 6e4
    close(run(plan, x, torch.empty((T, H), dtype=DT["f16"], device="cuda")), ref, tol, "f16")


@pytest.mark.parametrize("T,H", [(20, 144), (8, 144), (256, 5120)])
@pytest.mark.parametrize("w", ["bf16", "e4m3"])
def test_bad_values_stay_apart(w, T, H):
    """A NaN token and an expert with infinite weights or scales reach the tokens that they belong to only (a few
    choices, more, and many for an expert with wide rows)."""
    k, E, I = 2, 5, 144 if T < 100 else 2064
    x = inputs(13, T, k, E, H, I, "bf16", w)
    x["ids"] = torch.stack([torch.arange(T) % 4, torch.full((T,), -1)], 1).to(torch.int32).contiguous()
    plan = mswz.moe_layer_plan_create(T, k, E, H, I, "bf16", w)
    clean = run(plan, x, torch.empty((T, H), dtype=DT["bf16"], device="cuda"))
    x["X"][6, 3] = float("nan")
    if w == "e4m3":
        x["S1"][3] = float("inf")
        x["S2"][1, 0, 1] = float("nan")
    else:
        x["W1"][3] = float("inf")
        x["W2"][1, :, 5] = float("nan")
    got = run(plan, x, torch.empty((T, H), dtype=DT["bf16"], device="cuda"))
    bad = torch.zeros(T, dtype=torch.bool)
    bad[6] = True
    bad[3::4] = True
    bad[1::4] = True
    assert torch.equal(got[~bad.cuda()], clean[~bad.cuda()])
    assert not torch.isfinite(got[bad.cuda()][:, :128]).any()


@pytest.mark.parametrize("T,k,E,H,I", [(1, 2, 4, 136, 72), (18, 2, 4, 136, 72), (64, 8, 64, 264, 136)])
def test_pitch_and_surroundings(T, k, E, H, I):
    ld = H + 16
    x = inputs(17, T, k, E, H, I, "bf16", "bf16")
    plan = mswz.moe_layer_plan_create(T, k, E, H, I, "bf16", ldx=ld)
    ref, tol = reference(x, T, k, E, H, I, "silu")
    wide = torch.full((T, ld), float("nan"), dtype=DT["bf16"])
    wide[:, :H] = x["X"]
    flat = torch.full((T * ld + 64,), GUARD, dtype=DT["bf16"], device="cuda")
    Y = flat[32:32 + T * ld].view(T, ld)[:, :H]
    need = plan.workspace_bytes()
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    c = {n: v.cuda() for n, v in x.items() if v is not None}
    mswz.moe_layer(plan, wide.cuda()[:, :H], c["ids"], c["weights"], c["W1"], c["W2"], Y, workspace=ws[32:32 + need])
    close(Y, ref, tol, "bf16")
    Y.fill_(GUARD)
    assert (flat == GUARD).all()
    assert (ws[:32] == 0xA5).all() and (ws[32 + need:] == 0xA5).all()


@pytest.mark.parametrize("T,k,E,H,I", [(6, 2, 8, 512, 256), (20, 2, 8, 512, 256), (64, 8, 64, 256, 136)])
def test_streams_and_graph(T, k, E, H, I):
    x = inputs(19, T, k, E, H, I, "bf16", "bf16")
    other = inputs(20, T, k, E, H, I, "bf16", "bf16")
    plan = mswz.moe_layer_plan_create(T, k, E, H, I, "bf16")
    want = run(plan, x, torch.empty((T, H), dtype=DT["bf16"], device="cuda")).clone()
    want2 = run(plan, other, torch.empty((T, H), dtype=DT["bf16"], device="cuda")).clone()
    c = {n: v.cuda() for n, v in x.items() if v is not None}
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros((T, H), dtype=DT["bf16"], device="cuda") for _ in range(2)]
    ws = [torch.empty(plan.workspace_bytes(), dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, Y, w in zip(streams, outs, ws):
            mswz.moe_layer(plan, c["X"], c["ids"], c["weights"], c["W1"], c["W2"], Y, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(Y, want) for Y in outs)
    Y = torch.zeros((T, H), dtype=DT["bf16"], device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mswz.moe_layer(plan, c["X"], c["ids"], c["weights"], c["W1"], c["W2"], Y, workspace=ws[2])
    for i in range(4):   # the graph reads what its buffers hold: other tokens and choices on every second replay
        src = other if i % 2 else x
        for n in ("X", "ids", "weights", "W1", "W2"):
            c[n].copy_(src[n])
        Y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want2 if i % 2 else want)


def test_past_4_gib():
    """Experts whose weights lie beyond 32 bits of offset, and their scales: as the chosen ones alone."""
    T, k, E, H, I = 4, 2, 300, 4096, 1024
    ids = torch.tensor([[299, 0], [150, 299], [1, 298], [299, 299]], dtype=torch.int32)
    used = torch.unique(ids)
    small = torch.searchsorted(used, ids).to(torch.int32)
    g = torch.Generator(device="cuda").manual_seed(5)
    for w in ("bf16", "e4m3"):
        W1 = torch.randint(0, 120, (E, 2 * I, H * (2 if w == "bf16" else 1)), generator=g, device="cuda", dtype=torch.uint8)
        W2 = torch.randint(0, 120, (E, H, I * (2 if w == "bf16" else 1)), generator=g, device="cuda", dtype=torch.uint8)
        if w == "bf16":      # exponents of moderate size
            W1.view(E, -1, 2)[..., 1] = W1.view(E, -1, 2)[..., 1] % 4 + 58
            W2.view(E, -1, 2)[..., 1] = W2.view(E, -1, 2)[..., 1] % 4 + 58
            W1, W2, S1, S2 = W1.view(DT[w]), W2.view(DT[w]), None, None
        else:
            S1, S2 = torch.rand(E, 2, 8, 32, generator=g, device="cuda"), torch.rand(E, 32, 8, generator=g, device="cuda")
        X = (torch.randn(T, H, generator=g, device="cuda") / 64).to(DT["bf16"])
        weights = torch.rand(T, k, generator=g, device="cuda") / 4096
        out = []
        for n, i, pick in ((E, ids, slice(None)), (used.numel(), small, used.long().cuda())):
            plan = mswz.moe_layer_plan_create(T, k, n, H, I, "bf16", w)
            Y = torch.empty(T, H, dtype=DT["bf16"], device="cuda")
            ws = torch.empty(plan.workspace_bytes(), dtype=torch.uint8, device="cuda")
            mswz.moe_layer(plan, X, i.cuda(), weights, W1[pick].contiguous(), W2[pick].contiguous(), Y,
                           S1=None if S1 is None else S1[pick].contiguous(), S2=None if S2 is None else S2[pick].contiguous(), workspace=ws)
            out.append(Y)
        assert torch.isfinite(out[0]).all() and out[0].abs().max() > 0
        # the waves' shares of a sum may differ with the number of experts: by fp32's rounding, below a step of bf16
        assert (out[0].double() - out[1].double()).abs().max() <= 2.0 ** -7 * out[1].double().abs().max()


def test_quantised_weights_and_the_sorted_way():
    """The layer next to the operators it stands for: weights quantised by quant_fp8 (tiles), tokens sorted by
    moe_dispatch, the 16-bit products of the dequantised weights by gemm_run_grouped, and back by moe_combine; the
    two ways differ by the sorted way's roundings to bf16 (dequantised weights 2^-9 of each term, h and the rows of
    the last product 2^-9 each, and the output's)."""
    T, k, E, H, I = 24, 2, 4, 256, 128
    x = inputs(23, T, k, E, H, I, "bf16", "bf16")
    c = {n: v.cuda() for n, v in x.items() if v is not None}
    q1, q2 = torch.empty(E * 2 * I, H, dtype=E4M3, device="cuda"), torch.empty(E * H, I, dtype=E4M3, device="cuda")
    s1 = torch.empty(E, 2, blocks(I), blocks(H), device="cuda")
    s2 = torch.empty(E, blocks(H), blocks(I), device="cuda")
    mswz.quant_fp8(mswz.quant_fp8_plan_create(E * 2 * I, H, "bf16", "tile"), c["W1"].view(E * 2 * I, H), Q=q1, S=s1.view(-1, blocks(H)))
    mswz.quant_fp8(mswz.quant_fp8_plan_create(E * H, I, "bf16", "tile"), c["W2"].view(E * H, I), Q=q2, S=s2.view(-1, blocks(I)))
    plan = mswz.moe_layer_plan_create(T, k, E, H, I, "bf16", "e4m3")
    Y = torch.empty(T, H, dtype=DT["bf16"], device="cuda")
    ws = torch.empty(plan.workspace_bytes(), dtype=torch.uint8, device="cuda")
    mswz.moe_layer(plan, c["X"], c["ids"], c["weights"], q1.view(E, 2 * I, H), q2.view(E, H, I), Y, S1=s1, S2=s2, workspace=ws)
    y = dict(x, W1=q1.cpu().view(E, 2 * I, H), W2=q2.cpu().view(E, H, I), S1=s1.cpu(), S2=s2.cpu())
    ref, tol = reference(y, T, k, E, H, I, "silu")
    close(Y, ref, tol, "bf16")

    W1, W2 = (v.to(DT["bf16"]).cuda().contiguous() for v in values(y, E, H, I))
    n = T * k
    Xs, offsets = torch.empty(n, H, dtype=DT["bf16"], device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    order, pos = torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")
    moe = mswz.moe_plan_create(T, k, E, H, "bf16")
    mswz.moe_dispatch(moe, c["ids"], c["X"], Xs, offsets, order, pos, torch.empty(max(16, moe.workspace_bytes()), dtype=torch.uint8, device="cuda"))
    up = torch.empty(n, 2 * I, device="cuda")
    mswz.gemm_run_grouped(mswz.gemm_grouped_plan_create(E, n, 2 * I, H, "bf16", "f32"), Xs, W1, offsets, up)
    h = (torch.nn.functional.silu(up[:, :I]) * up[:, I:]).to(DT["bf16"])
    Ys = torch.empty(n, H, dtype=DT["bf16"], device="cuda")
    mswz.gemm_run_grouped(mswz.gemm_grouped_plan_create(E, n, H, I, "bf16", "bf16"), h, W2, offsets, Ys)
    Y2 = torch.empty(T, H, dtype=DT["bf16"], device="cuda")
    mswz.moe_combine(moe, Ys, pos, Y2, weights=c["weights"])
    # first order: each of the sums moves by 2^-9 of its terms' magnitudes
    V1, V2 = values(y, E, H, I)
    bound = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(x["ids"][t, j])
            v = x["X"][t].double()
            s, S = V1[e] @ v, V1[e].abs() @ v.abs()
            on, up_ = s[:I] * torch.sigmoid(s[:I]), s[I:]
            da = 2.0 ** -9 * (1.2 * S[:I] * (up_.abs() + 2.0 ** -9 * S[I:]) + on.abs() * S[I:] + (on * up_).abs())
            a = (on * up_).abs() + da
            bound[t] += float(x["weights"][t, j]) * (V2[e].abs() @ da + 2.0 ** -9 * (V2[e].abs() @ a) + 2.0 ** -9 * (V2[e].abs() @ a))
    bound += 2.0 ** -8 * ref.abs() + tol
    assert ((Y2.double().cpu() - Y.double().cpu()).abs() <= 1.05 * bound).all()


def test_refusals_on_the_gpu():
    T, k, E, H, I = 2, 2, 3, 64, 32
    x = inputs(29, T, k, E, H, I, "bf16", "bf16")
    c = {n: v.cuda() for n, v in x.items() if v is not None}
    plan = mswz.moe_layer_plan_create(T, k, E, H, I, "bf16")
    Y = torch.zeros(T, H, dtype=DT["bf16"], device="cuda")
    ws = torch.empty(plan.workspace_bytes(), dtype=torch.uint8, device="cuda")
    good = dict(X=c["X"], ids=c["ids"], weights=c["weights"], W1=c["W1"], W2=c["W2"], Y=Y, workspace=ws)
    mswz.moe_layer(plan, **good)
    torch.cuda.synchronize()
    for name, bad in (("X", c["X"].float()), ("ids", c["ids"].long()), ("ids", c["ids"][:1]), ("weights", c["weights"].half()),
                      ("W1", c["W1"][:2]), ("W2", c["W1"]), ("Y", Y[:, :32]), ("workspace", ws[:-1]), ("workspace", None),
                      ("X", c["X"].cpu()), ("S1", c["weights"])):
        with pytest.raises(ValueError):
            mswz.moe_layer(plan, **dict(good, **{name: bad}))
