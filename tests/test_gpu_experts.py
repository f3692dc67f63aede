"""The expert operators against plain computations in 64 bits, through the
binding (include/mswz_experts.h).

Tolerances, from the arithmetic:
* a product's fp32 sum of n terms, in any order and with adders that truncate,
  is within 2 (n + 8) 2^-24 S of the exact sum, S the sum of the terms'
  magnitudes (the 8 covers the scale, the zero-point correction and beta).
  With bf16 activations and u4 weights the terms are a s (16 + q) and
  a s (16 + z), so S is taken over those;
* D in 16 bits adds one rounding, half a step: eps / 2 of the value;
* copies, integers and single products rounded once are compared exactly.
"""
import numpy as np
import pytest
import torch

import mma_swizzled_operand_amd as mswz

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
GUARD = 7.5   # what a buffer holds where nothing may be written


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, dt="bf16"):
    return torch.randn(*shape, generator=g, dtype=torch.float32).to(DT[dt])


def bounds_of(counts, rows=None):
    b = torch.zeros(len(counts) + 1, dtype=torch.int32)
    b[1:] = torch.tensor(counts).cumsum(0)
    return b


def check(got, ref, mag, n, dt, what=""):
    got, ref, mag = got.double().cpu(), ref.double(), mag.double()
    assert torch.isfinite(got).all(), what
    tol = 2 * (n + 8) * 2.0 ** -24 * mag + (torch.finfo(DT[dt]).eps / 2 if dt != "f32" else 0) * ref.abs()
    if dt == "f16":
        tol = tol + 2.0 ** -25   # half a step below the smallest normal number
    bad = (got - ref).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), float(((got - ref).abs() / tol.clamp(min=1e-300)).max()))


# ---- 4-bit weights --------------------------------------------------------------

def w4_inputs(g, M, N, K, E, a, w, G, zeros):
    groups = -(-K // G)
    x = {"A": normal(g, M, K, dt=a), "B": torch.randint(0, 256, (max(1, E), N, K // 2), generator=g, dtype=torch.uint8), "Z": None}
    if w == "u4":
        x["S"] = ((0.5 + torch.rand(max(1, E), N, groups, generator=g)) * 0.02).to(DT[a])
        if zeros:
            x["Z"] = torch.randint(0, 16, (max(1, E), N, groups), generator=g, dtype=torch.uint8)
    else:
        x["S"] = torch.randint(118, 130, (max(1, E), N, groups), generator=g, dtype=torch.uint8)
    return x


def w4_reference(x, w, G, a, bounds=None):
    """The exact result and the sum of the terms' magnitudes, rows outside every group NaN."""
    A, B = x["A"].double(), x["B"]
    E, N, half = B.shape
    K = 2 * half
    q = torch.stack((B & 15, B >> 4), -1).reshape(E, N, K)
    group = torch.arange(K) // G
    if w == "u4":
        s = x["S"].double()[:, :, group]
        z = x["Z"].double()[:, :, group] if x["Z"] is not None else torch.full_like(s, 8)
        W = (q.double() - z) * s
        mag = (32 + q.double() + z) * s if a == "bf16" else W.abs()
    else:
        W = E2M1[q.long()] * torch.pow(2.0, x["S"].double() - 127)[:, :, group]
        mag = W.abs()
    D = torch.full((A.shape[0], N), float("nan"), dtype=torch.float64)
    S = D.clone()
    for e in range(E):
        lo, hi = (bounds[e], bounds[e + 1]) if bounds is not None else (0, A.shape[0])
        D[lo:hi] = A[lo:hi] @ W[e].t()
        S[lo:hi] = A[lo:hi].abs() @ mag[e].abs().t()
    return D, S


def w4_run(plan, x, D, offsets=None, beta=0, stream=None):
    c = {k: None if v is None else v.cuda() for k, v in x.items()}
    ws = torch.full((max(16, plan.workspace_bytes()),), 0xFF, dtype=torch.uint8, device="cuda")
    mswz.gemm_run_w4(plan, c["A"], c["B"], c["S"], D, Z=c["Z"], offsets=None if offsets is None else offsets.cuda(),
                     beta=beta, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    return D


W4_CASES = [  # M, N, K, G, a, w, d, zeros
    (1, 1, 32, 32, "f16", "u4", "f16", True),
    (1, 16, 32, 128, "bf16", "u4", "bf16", True),
    (1, 1000, 4096, 128, "bf16", "u4", "f32", False),
    (3, 77, 96, 64, "f16", "u4", "f32", True),
    (16, 130, 1056, 64, "bf16", "u4", "f32", True),
    (17, 48, 1056, 32, "f16", "u4", "f16", True),
    (33, 31, 160, 128, "f16", "u4", "f32", True),
    (64, 272, 2080, 32, "bf16", "u4", "bf16", True),
    (64, 513, 512, 256, "f16", "u4", "f32", False),
    (65, 40, 384, 384, "bf16", "u4", "f32", True),
    (200, 64, 256, 128, "f16", "u4", "f16", False),
    (1, 4099, 2048, 32, "bf16", "e2m1", "bf16", False),
    (5, 33, 32, 32, "f16", "e2m1", "f32", False),
    (31, 65, 544, 32, "bf16", "e2m1", "f32", False),
    (64, 512, 1024, 32, "f16", "e2m1", "f16", False),
    (130, 17, 96, 32, "bf16", "e2m1", "f32", False),
    (1, 8192, 8192, 64, "bf16", "u4", "f32", True),
    (2, 9000, 2048, 128, "f16", "u4", "f32", True),
    # each width of a workgroup, with and without K split over workgroups
    (3, 16500, 1088, 128, "bf16", "u4", "f32", True),
    (16, 16500, 544, 32, "f16", "e2m1", "f32", False),
    (15, 4100, 1152, 64, "f16", "u4", "f16", True),
    (2, 65700, 288, 32, "bf16", "u4", "bf16", True),
    (40, 16400, 416, 128, "bf16", "u4", "f32", True),
    (64, 16400, 1056, 32, "bf16", "e2m1", "f32", False),
    (50, 32900, 96, 32, "f16", "u4", "f32", True),
    (64, 300, 8192, 32, "f16", "e2m1", "f32", False),
    (64, 1000, 6176, 128, "f16", "u4", "f16", True),
]


@pytest.mark.parametrize("M,N,K,G,a,w,d,zeros", W4_CASES)
def test_w4(M, N, K, G, a, w, d, zeros):
    g = gen(M + N + K)
    x = w4_inputs(g, M, N, K, 0, a, w, G, zeros)
    plan = mswz.gemm_w4_plan_create(M, N, K, a, w, d, group=G)
    ref, mag = w4_reference(x, w, G, a)
    got = w4_run(plan, x, torch.full((M, N), float("nan"), dtype=DT[d], device="cuda"))
    check(got, ref, mag, K, d)
    again = w4_run(plan, x, torch.zeros((M, N), dtype=DT[d], device="cuda"))
    assert torch.equal(got, again)
    D0 = normal(g, M, N, dt=d)
    got = w4_run(plan, x, D0.cuda(), beta=1)
    check(got, ref + D0.double(), mag + D0.double().abs(), K, d, "beta")


@pytest.mark.parametrize("a,w,G", [("f16", "u4", 128), ("bf16", "u4", 32), ("bf16", "e2m1", 32)])
def test_w4_row_pitches(a, w, G):
    g = gen(5)
    M, N, K, lda, ldd = 19, 50, 160, 176, 53
    x = w4_inputs(g, M, N, K, 0, a, w, G, w == "u4")
    wide = torch.full((M, lda), float("nan"), dtype=DT[a])
    wide[:, :K] = x["A"]
    D = torch.full((M, ldd), GUARD, device="cuda")
    plan = mswz.gemm_w4_plan_create(M, N, K, a, w, "f32", group=G, lda=lda, ldd=ldd)
    c = {k: None if v is None else v.cuda() for k, v in x.items()}
    ws = torch.empty(max(16, plan.workspace_bytes()), dtype=torch.uint8, device="cuda")
    mswz.gemm_run_w4(plan, wide.cuda()[:, :K], c["B"], c["S"], D[:, :N], Z=c["Z"], workspace=ws)
    ref, mag = w4_reference(x, w, G, a)
    check(D[:, :N], ref, mag, K, "f32")
    assert (D[:, N:] == GUARD).all()


W4_EXPERTS = [  # counts, rows, N, K, G, a, w, d
    ([1], 1, 48, 64, 64, "bf16", "u4", "bf16"),
    ([0, 3, 0, 1, 0], 9, 70, 160, 32, "f16", "u4", "f32"),
    ([5, 0, 17, 64, 65, 2], 160, 100, 288, 128, "bf16", "u4", "f32"),
    ([130, 1, 0, 0], 131, 33, 96, 64, "f16", "u4", "f16"),
    ([2] * 70, 150, 32, 128, 32, "bf16", "e2m1", "f32"),
    ([0, 0, 0], 4, 32, 64, 32, "f16", "e2m1", "f16"),
    ([70, 0, 100, 33, 64], 280, 6600, 160, 64, "bf16", "u4", "f32"),
    ([1, 3, 0, 9, 16, 17, 2, 5] * 4, 220, 2100, 320, 128, "f16", "u4", "f16"),
]


@pytest.mark.parametrize("counts,rows,N,K,G,a,w,d", W4_EXPERTS)
def test_w4_experts(counts, rows, N, K, G, a, w, d):
    g = gen(rows + N)
    E = len(counts)
    x = w4_inputs(g, rows, N, K, E, a, w, G, True)
    offsets = bounds_of(counts)
    x["A"][offsets[-1]:] = float("nan")   # rows behind the last group are not read
    plan = mswz.gemm_w4_plan_create(rows, N, K, a, w, d, group=G, experts=E)
    ref, mag = w4_reference(x, w, G, a, offsets.tolist())
    got = w4_run(plan, x, torch.full((rows, N), GUARD, dtype=DT[d], device="cuda"), offsets)
    used = int(offsets[-1])
    check(got[:used], ref[:used], mag[:used], K, d)
    assert (got[used:] == GUARD).all()


@pytest.mark.parametrize("counts,N,a,w", [([2, 0, 3], 37, "bf16", "u4"), ([9, 20, 1], 37, "f16", "u4"), ([2, 1, 1], 67, "bf16", "e2m1"),
                                          ([40, 30, 1], 70, "f16", "e2m1")])
def test_w4_scales_at_any_alignment(counts, N, a, w):
    """Scales and zero points that start and end between words, NaN and 255 around them."""
    M, K, E = sum(counts), 160, 3
    x, bounds = w4_inputs(gen(N + M), M, N, K, E, a, w, 32, w == "u4"), bounds_of(counts)
    ref, mag = w4_reference(x, w, 32, a, bounds.tolist())
    plan = mswz.gemm_w4_plan_create(M, N, K, a, w, "f32", group=32, experts=E)
    ws = torch.empty(max(16, plan.workspace_bytes()), dtype=torch.uint8, device="cuda")

    def inside(t, off):
        wide = torch.full((t.numel() + 8,), float("nan") if t.dtype.is_floating_point else 255, dtype=t.dtype)
        wide[off:off + t.numel()] = t.reshape(-1)
        return wide.cuda()[off:off + t.numel()]

    for off in (1, 2, 3, 5):
        D = torch.full((M, N), float("nan"), device="cuda")
        mswz.gemm_run_w4(plan, x["A"].cuda(), x["B"].cuda(), inside(x["S"], off), D, Z=None if x["Z"] is None else inside(x["Z"], 6 - off),
                         offsets=bounds.cuda(), workspace=ws)
        check(D, ref, mag, K, "f32", off)


def test_w4_weights_past_4_gib():
    E, N, K = 1024, 4128, 2112
    x = w4_inputs(gen(50), 8, N, K, 2, "bf16", "u4", 64, True)
    B = torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda")
    S, Z = torch.zeros(E, N, K // 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(E, N, K // 64, dtype=torch.uint8, device="cuda")
    for e, i in ((0, 0), (E - 1, 1)):
        B[e], S[e], Z[e] = x["B"][i].cuda(), x["S"][i].cuda(), x["Z"][i].cuda()
    offsets = torch.full((E + 1,), 3, dtype=torch.int32)
    offsets[0], offsets[E] = 0, 8
    D = torch.full((8, N), float("nan"), device="cuda")
    plan = mswz.gemm_w4_plan_create(8, N, K, "bf16", "u4", "f32", group=64, experts=E)
    mswz.gemm_run_w4(plan, x["A"].cuda(), B, S, D, Z=Z, offsets=offsets.cuda())
    check(D, *w4_reference(x, "u4", 64, "bf16", [0, 3, 8]), K, "f32")


def test_w4_rows_past_4_gib():
    M, N, K, ld = 600, 24, 96, 1 << 22
    x = w4_inputs(gen(51), M, N, K, 0, "bf16", "u4", 32, True)
    A = torch.empty(M, ld, dtype=torch.bfloat16, device="cuda")
    A[:, :K] = x["A"].cuda()
    A[:, K:K + 64] = float("nan")
    D = torch.empty(M, ld, dtype=torch.bfloat16, device="cuda")
    D[:, :64] = GUARD
    plan = mswz.gemm_w4_plan_create(M, N, K, "bf16", "u4", "bf16", group=32, lda=ld, ldd=ld)
    ws = torch.empty(max(16, plan.workspace_bytes()), dtype=torch.uint8, device="cuda")
    mswz.gemm_run_w4(plan, A[:, :K], x["B"].cuda(), x["S"].cuda(), D[:, :N], Z=x["Z"].cuda(), workspace=ws)
    check(D[:, :N], *w4_reference(x, "u4", 32, "bf16"), K, "bf16")
    assert (D[:, N:64] == GUARD).all()


def test_w4_bounds_that_do_not_ascend_stay_inside_the_buffers():
    g = gen(3)
    x = w4_inputs(g, 8, 32, 64, 4, "bf16", "u4", 64, True)
    plan = mswz.gemm_w4_plan_create(8, 32, 64, "bf16", "u4", "f32", group=64, experts=4)
    room = torch.full((24, 32), GUARD, device="cuda")
    w4_run(plan, x, room[8:16], torch.tensor([-5, 3, 2, 1 << 30, 9], dtype=torch.int32))
    assert (room[:8] == GUARD).all() and (room[16:] == GUARD).all()
    # group 0 is rows 0..2, group 1 empty, group 2 rows 2..7 (clamped), group 3 none
    ref, mag = w4_reference(x, "u4", 64, "bf16", [0, 2, 2, 8, 8])
    check(room[8:10], ref[:2], mag[:2], 64, "f32")
    ref2, mag2 = w4_reference(x, "u4", 64, "bf16", [0, 0, 2, 8, 8])
    check(room[11:16], ref2[3:], mag2[3:], 64, "f32")


@pytest.mark.parametrize("a", ["f16", "bf16"])
def test_w4_scales_and_zero_points_at_their_limits(a):
    M, N, K = 2, 16, 64
    g = gen(4)
    x = w4_inputs(g, M, N, K, 0, a, "e2m1", 32, False)
    x["S"][0, :, 0] = 0          # 2^-127
    x["S"][0, :, 1] = 1
    x["S"][0, 3, 1] = 255        # NaN
    x["S"][0, 5, 1] = 254
    plan = mswz.gemm_w4_plan_create(M, N, K, a, "e2m1", "f32", group=32)
    got = w4_run(plan, x, torch.zeros(M, N, device="cuda")).cpu()
    ref, mag = w4_reference(x, "e2m1", 32, a)
    assert torch.isnan(got[:, 3]).all()
    keep = [n for n in range(N) if n != 3]
    big = ref[:, 5].abs() > torch.finfo(torch.float32).max
    assert torch.equal(torch.isinf(got[:, 5]), big)
    small = [n for n in keep if n != 5]
    # results next to fp32's smallest normal number: each of the two groups' sums may lose a step of 2^-149
    assert ((got.double() - ref)[:, small].abs() <= 2 * (K + 8) * 2.0 ** -24 * mag[:, small] + 2 ** -148.0).all()

    y = w4_inputs(g, M, N, K, 0, a, "u4", 64, True)
    y["Z"] = torch.arange(240, 256, dtype=torch.uint8).reshape(1, N, 1)
    plan = mswz.gemm_w4_plan_create(M, N, K, a, "u4", "f32", group=64)
    ref, mag = w4_reference(y, "u4", 64, a)
    check(w4_run(plan, y, torch.zeros(M, N, device="cuda")), ref, mag, K, "f32")


def test_w4_nan_stays_in_its_row():
    x = w4_inputs(gen(6), 20, 40, 256, 0, "f16", "u4", 128, True)
    x["A"][7, 13] = float("nan")
    x["A"][9, 200] = float("inf")
    x["B"][0, :, 100] = 0x00     # elements 200 and 201: q = 0
    x["Z"][0, :, 1] = 3
    plan = mswz.gemm_w4_plan_create(20, 40, 256, "f16", "u4", "f32", group=128)
    got = w4_run(plan, x, torch.zeros(20, 40, device="cuda")).cpu()
    assert torch.isnan(got[7]).all() and (got[9] == -float("inf")).all()
    keep = [m for m in range(20) if m not in (7, 9)]
    ref, mag = w4_reference({**x, "A": x["A"][keep]}, "u4", 128, "f16")
    check(got[keep], ref, mag, 256, "f32")


# ---- products over groups of rows ---------------------------------------------------

GROUPED = [  # counts, rows, N, K, dt, d
    ([1], 1, 8, 8, "f16", "f16"),
    ([0, 5, 0], 7, 24, 72, "bf16", "f32"),
    ([256, 0, 257, 3], 520, 264, 64, "bf16", "bf16"),
    ([100, 1, 30, 0, 70], 201, 520, 264, "f16", "f16"),
    ([700, 20], 800, 256, 520, "f16", "f32"),
    ([3] * 100, 333, 40, 136, "bf16", "f32"),
    ([0, 0], 5, 16, 128, "bf16", "f32"),
    ([64, 128, 65, 1, 190], 448, 776, 320, "bf16", "bf16"),
    # more tiles than a round of workgroups holds, with a full and with a halved last one
    ([2100, 1900], 4000, 2304, 64, "bf16", "bf16"),
    ([4100, 0, 4090], 8200, 2304, 72, "f16", "f32"),
]


def grouped_reference(A, B, bounds):
    """rows of A times their group's B (E, N, K): result and magnitudes, NaN outside the groups."""
    D = torch.full((A.shape[0], B.shape[1]), float("nan"), dtype=torch.float64)
    S = D.clone()
    for e in range(B.shape[0]):
        lo, hi = bounds[e], bounds[e + 1]
        D[lo:hi] = A[lo:hi].double() @ B[e].double().t()
        S[lo:hi] = A[lo:hi].double().abs() @ B[e].double().abs().t()
    return D, S


@pytest.mark.parametrize("b_major", ["k", "mn"])
@pytest.mark.parametrize("counts,rows,N,K,dt,d", GROUPED)
def test_grouped_rows(counts, rows, N, K, dt, d, b_major):
    g = gen(rows + N + K)
    E, offsets = len(counts), bounds_of(counts)
    used = int(offsets[-1])
    A, B = normal(g, rows, K, dt=dt), normal(g, E, N, K, dt=dt)
    A[used:] = float("nan")
    plan = mswz.gemm_grouped_plan_create(E, rows, N, K, dt, d, b_major=b_major)
    stored = B.cuda() if b_major == "k" else B.transpose(1, 2).contiguous().cuda()
    ref, mag = grouped_reference(A, B, offsets.tolist())
    D = torch.full((rows, N), GUARD, dtype=DT[d], device="cuda")
    mswz.gemm_run_grouped(plan, A.cuda(), stored, offsets.cuda(), D)
    check(D[:used], ref[:used], mag[:used], K, d)
    assert (D[used:] == GUARD).all()
    D0 = normal(g, rows, N, dt=d)
    D1 = D0.cuda()
    mswz.gemm_run_grouped(plan, A.cuda(), stored, offsets.cuda(), D1, beta=1)
    check(D1[:used], (ref + D0.double())[:used], (mag + D0.double().abs())[:used], K, d, "beta")
    assert torch.equal(D1[used:].cpu(), D0[used:])


@pytest.mark.parametrize("counts,rows,N,K,dt,d", GROUPED)
def test_grouped_along_k(counts, rows, N, K, dt, d):
    """The weight gradient: D[e] (N, K) = sum over the group's rows of dY^T X."""
    g = gen(rows * N + K)
    E, offsets = len(counts), bounds_of(counts)
    used = int(offsets[-1])
    dY, X = normal(g, rows, N, dt=dt), normal(g, rows, K, dt=dt)
    dY[used:] = float("nan")
    X[used:] = float("inf")
    plan = mswz.gemm_grouped_plan_create(E, N, K, rows, dt, d, axis="k")
    b = offsets.tolist()
    ref = torch.stack([dY[b[e]:b[e + 1]].double().t() @ X[b[e]:b[e + 1]].double() for e in range(E)])
    mag = torch.stack([dY[b[e]:b[e + 1]].double().abs().t() @ X[b[e]:b[e + 1]].double().abs() for e in range(E)])
    D = torch.full((E, N, K), float("nan"), dtype=DT[d], device="cuda")
    mswz.gemm_run_grouped(plan, dY.cuda(), X.cuda(), offsets.cuda(), D)
    check(D, ref, mag, max(counts) + 1, d)
    D0 = normal(g, E, N, K, dt=d)
    D1 = D0.cuda()
    mswz.gemm_run_grouped(plan, dY.cuda(), X.cuda(), offsets.cuda(), D1, beta=1)
    check(D1, ref + D0.double(), mag + D0.double().abs(), max(counts) + 1, d, "beta")


def test_grouped_bounds_that_do_not_ascend_stay_inside_the_buffers():
    g = gen(8)
    E, rows, N, K = 4, 300, 16, 64
    A, B = normal(g, rows, K), normal(g, E, N, K)
    bad = torch.tensor([-9, 280, 2, 1 << 30, -7], dtype=torch.int32).cuda()
    room = torch.full((rows + 600, N), GUARD, device="cuda")
    mswz.gemm_run_grouped(mswz.gemm_grouped_plan_create(E, rows, N, K, "bf16", "f32"), A.cuda(), B.cuda(), bad,
                          room[300:600])
    assert (room[:300] == GUARD).all() and (room[600:] == GUARD).all()
    dW = torch.full((E + 2, N, K), GUARD, device="cuda")
    dY = normal(g, rows, N)
    mswz.gemm_run_grouped(mswz.gemm_grouped_plan_create(E, N, K, rows, "bf16", "f32", axis="k"), dY.cuda(), A.cuda(),
                          bad, dW[1:-1])
    assert (dW[0] == GUARD).all() and (dW[-1] == GUARD).all()
    assert (dW[2] == 0).all() and (dW[4] == 0).all()   # groups 1 and 3 have no rows


def test_grouped_rows_past_4_gib():
    """The last rows of an operand and a result larger than 32-bit offsets reach."""
    E, rows, N, K = 3, 1 << 20, 2112, 2112
    A = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda").fill_(0.5)
    B = normal(gen(9), E, N, K).cuda()
    g = gen(10)
    tail = normal(g, 300, K)
    A[-300:] = tail.cuda()
    D = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
    offsets = torch.tensor([0, 1000, rows - 300, rows], dtype=torch.int32)
    mswz.gemm_run_grouped(mswz.gemm_grouped_plan_create(E, rows, N, K, "bf16", "bf16"), A, B, offsets.cuda(), D)
    ref = tail.double() @ B[2].double().cpu().t()
    mag = tail.double().abs() @ B[2].double().cpu().abs().t()
    check(D[-300:], ref, mag, K, "bf16")
    row = torch.full((1, K), 0.5, dtype=torch.float64)
    check(D[rows - 301:rows - 300], row @ B[1].double().cpu().t(), row @ B[1].double().cpu().abs().t(), K, "bf16")


# ---- tokens to their experts and back --------------------------------------------------

def sorted_reference(ids, E):
    flat = ids.reshape(-1).numpy()
    keep = (flat >= 0) & (flat < E)
    slots = np.nonzero(keep)[0]
    slots = slots[np.argsort(flat[slots], kind="stable")]
    order = np.full(flat.size, -1, np.int32)
    order[:slots.size] = slots
    pos = np.full(flat.size, -1, np.int32)
    pos[slots] = np.arange(slots.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[keep], minlength=E))]).astype(np.int32)
    return offsets, order, pos.reshape(ids.shape)


def dispatch(plan, ids, X, Xs=None):
    n = plan.choices
    out = [torch.full((m,), -99, dtype=torch.int32, device="cuda") for m in (plan.E + 1, n, n)]
    if X is not None and Xs is None:
        Xs = torch.full((n, plan.H), GUARD, dtype=plan.type, device="cuda")
    ws = torch.full((max(16, plan.workspace_bytes()),), 0xFF, dtype=torch.uint8, device="cuda")
    mswz.moe_dispatch(plan, ids.cuda(), X, Xs, *out, workspace=ws)
    torch.cuda.synchronize()
    return out[0], out[1], out[2].reshape(plan.T, plan.topk), Xs


MOE = [  # T, topk, E, H, dt, share of ids outside
    (1, 1, 1, 8, "f16", 0.0),
    (1, 8, 3, 72, "bf16", 0.3),
    (7, 2, 8, 1024, "f16", 0.0),
    (5, 3, 1024, 64, "f32", 0.2),
    (64, 8, 64, 520, "bf16", 0.0),
    (255, 4, 5, 136, "f16", 0.1),
    (256, 8, 256, 64, "bf16", 0.05),
    (1000, 3, 1000, 8, "f32", 0.5),
    (2049, 1, 2, 24, "bf16", 0.0),
    (3000, 9, 40, 16, "f16", 0.02),
    (9000, 8, 128, 64, "bf16", 0.02),
    (40, 33, 7, 2064, "bf16", 0.1),
    (20, 4, 4, 64, "f32", 1.0),
    (1024, 8, 300, 8, "bf16", 0.01),    # the most choices that the sort does not count first
    (8193, 1, 70, 16, "f16", 0.0),
    (2100, 8, 1000, 8, "bf16", 0.05),
]


def ids_for(g, T, topk, E, out):
    ids = torch.randint(0, E, (T, topk), generator=g, dtype=torch.int32)   # the same expert twice is allowed
    if out:
        wrong = torch.tensor([-1, E, -(1 << 31), (1 << 31) - 1], dtype=torch.int64).to(torch.int32)
        hit = torch.rand(T, topk, generator=g) < out
        ids[hit] = wrong[torch.randint(0, 4, (int(hit.sum()),), generator=g)]
    return ids


@pytest.mark.parametrize("T,topk,E,H,dt,out", MOE)
def test_dispatch(T, topk, E, H, dt, out):
    g = gen(T * topk + E)
    ids, X = ids_for(g, T, topk, E, out), normal(g, T, H, dt=dt)
    offsets, order, pos = sorted_reference(ids, E)
    plan = mswz.moe_plan_create(T, topk, E, H, dt)
    got = dispatch(plan, ids, X.cuda())
    assert np.array_equal(got[0].cpu().numpy(), offsets)
    assert np.array_equal(got[1].cpu().numpy(), order)
    assert np.array_equal(got[2].cpu().numpy(), pos)
    used = int(offsets[-1])
    assert torch.equal(got[3][:used].cpu(), X[torch.from_numpy(order[:used].astype(np.int64) // topk)])
    assert (got[3][used:] == GUARD).all()
    only = dispatch(plan, ids, None)   # the sort alone
    assert all(torch.equal(a, b) for a, b in zip(only[:3], got[:3]))


@pytest.mark.parametrize("T,topk,E,H,dt,out", MOE)
def test_combine_and_its_gradient(T, topk, E, H, dt, out):
    g = gen(T + topk * E)
    n = T * topk
    pos = torch.from_numpy(sorted_reference(ids_for(g, T, topk, E, out), E)[2])
    Ys, dY, w = normal(g, n, H, dt=dt), normal(g, T, H, dt=dt), torch.randn(T, topk, generator=g)
    held = pos >= 0
    used = int(held.sum())
    Ys[used:] = float("nan")              # rows that no choice names
    w[~held] = float("nan")               # weights of choices left out
    rows = torch.where(held[:, :, None], Ys[pos.clamp(min=0).long()].double(), 0.0)
    wk = torch.where(held, w, 0.0).double()
    plan = mswz.moe_plan_create(T, topk, E, H, dt)
    for weights, wd in ((w, wk), (None, held.double())):
        Y = torch.full((T, H), float("nan"), dtype=DT[dt], device="cuda")
        mswz.moe_combine(plan, Ys.cuda(), pos.cuda(), Y, weights=None if weights is None else weights.cuda())
        check(Y, (rows * wd[:, :, None]).sum(1), (rows * wd[:, :, None]).abs().sum(1), topk, dt)
    dYs = torch.full((n, H), GUARD, dtype=DT[dt], device="cuda")
    dw = torch.full((T, topk), float("nan"), device="cuda")
    mswz.moe_combine_grad(plan, dY.cuda(), Ys.cuda(), pos.cuda(), w.cuda(), dYs, dw)
    terms = rows * dY.double()[:, None, :]
    check(dw, terms.sum(2), terms.abs().sum(2), H, "f32")
    assert (dw.cpu()[~held] == 0).all()
    want = (w[:, :, None] * dY.float()[:, None, :]).to(DT[dt])
    assert torch.equal(dYs[:used].cpu()[pos[held].long()], want[held])
    assert (dYs[used:] == GUARD).all()


def test_gradients_against_differences():
    """Each pass is linear in what it is differentiated by, so a difference of two passes is the gradient's
    product with the step, to rounding."""
    g = gen(12)
    T, topk, E, H, N = 50, 3, 6, 64, 48
    ids = ids_for(g, T, topk, E, 0.1)
    n = T * topk
    plan = mswz.moe_plan_create(T, topk, E, H, "f32")
    X, w = normal(g, T, H, dt="f32"), torch.rand(T, topk, generator=g)
    c, dX = normal(g, n, H, dt="f32"), normal(g, T, H, dt="f32")
    offsets, order, pos, Xs = dispatch(plan, ids, X.cuda(), torch.zeros(n, H, device="cuda"))
    # dispatch: <c, d(Xs)> = <dispatch's gradient of c, dX>
    _, _, _, Xs2 = dispatch(plan, ids, (X + dX).cuda(), torch.zeros(n, H, device="cuda"))
    grad = torch.zeros(T, H, device="cuda")
    mswz.moe_combine(plan, c.cuda(), pos, grad)
    a = (c.double() * (Xs2.double() - Xs.double()).cpu()).sum()
    b = (grad.double().cpu() * ((X + dX).double() - X.double())).sum()
    assert abs(a - b) <= 2 * topk * 2.0 ** -24 * (c.double().abs().sum() * dX.abs().max().double())
    # combine: both gradients
    cy = normal(g, T, H, dt="f32")
    Ys, dYs_step, dw_step = normal(g, n, H, dt="f32"), normal(g, n, H, dt="f32"), normal(g, T, topk, dt="f32")
    used = int(offsets[-1])
    Ys[used:] = dYs_step[used:] = 0
    gy, gw = torch.zeros(n, H, device="cuda"), torch.zeros(T, topk, device="cuda")
    mswz.moe_combine_grad(plan, cy.cuda(), Ys.cuda(), pos, w.cuda(), gy, gw)

    def value(ys, ww):
        Y = torch.zeros(T, H, device="cuda")
        mswz.moe_combine(plan, ys.cuda(), pos, Y, weights=ww.cuda())
        return (Y.double().cpu() * cy.double()).sum()

    base = value(Ys, w)
    size = 2 * (topk + 8) * 2.0 ** -24 * 4 * T * topk * H * 16   # terms below 4 sigma each
    assert abs(value(Ys + dYs_step, w) - base - (gy.double().cpu() * ((Ys + dYs_step).double() - Ys.double())).sum()) <= size
    assert abs(value(Ys, w + dw_step) - base - (gw.double().cpu() * ((w + dw_step).double() - w.double())).sum()) <= size
    # grouped product: both gradients of <cd, Xs . B^T>
    A, B, cd = normal(g, n, H, dt="bf16"), normal(g, E, N, H, dt="bf16"), normal(g, n, N, dt="bf16")
    A[used:] = 0
    cd[used:] = 0
    fwd = mswz.gemm_grouped_plan_create(E, n, N, H, "bf16", "f32")
    dA, dB = torch.zeros(n, H, device="cuda"), torch.zeros(E, N, H, device="cuda")
    mswz.gemm_run_grouped(mswz.gemm_grouped_plan_create(E, n, H, N, "bf16", "f32", b_major="mn"), cd.cuda(), B.cuda(), offsets, dA)
    mswz.gemm_run_grouped(mswz.gemm_grouped_plan_create(E, N, H, n, "bf16", "f32", axis="k"), cd.cuda(), A.cuda(), offsets, dB)

    def product(a, b):
        D = torch.zeros(n, N, device="cuda")
        mswz.gemm_run_grouped(fwd, a.cuda(), b.cuda(), offsets, D)
        return (D.double().cpu() * cd.double()).sum()

    A2, B2 = (A.float() + normal(g, n, H, dt="f32")).bfloat16(), (B.float() + normal(g, E, N, H, dt="f32")).bfloat16()
    A2[used:] = 0
    base = product(A, B)
    size = 2 * (H + 8) * 2.0 ** -24 * n * N * H * 4.0   # mean magnitude of a term below 4
    assert abs(product(A2, B) - base - (dA.double().cpu() * (A2.double() - A.double())).sum()) <= size
    assert abs(product(A, B2) - base - (dB.double().cpu() * (B2.double() - B.double())).sum()) <= size


def test_token_row_pitch():
    g = gen(13)
    T, topk, E, H, ld = 37, 2, 5, 40, 64
    plan = mswz.moe_plan_create(T, topk, E, H, "f16", ldx=ld)
    wide = torch.full((T, ld), GUARD, dtype=torch.float16, device="cuda")
    X = normal(g, T, H, dt="f16")
    wide[:, :H] = X.cuda()
    ids = ids_for(g, T, topk, E, 0.1)
    offsets, order, pos, Xs = dispatch(plan, ids, wide[:, :H])
    used = int(offsets[-1])
    assert torch.equal(Xs[:used].cpu(), X[order[:used].cpu().long() // topk])
    out = torch.full((T, ld), GUARD, dtype=torch.float16, device="cuda")
    mswz.moe_combine(plan, Xs, pos, out[:, :H])
    held = (pos >= 0).sum(1).cpu()
    check(out[:, :H], X.double() * held[:, None], X.double().abs() * held[:, None], topk, "f16")
    assert (out[:, H:] == GUARD).all()
    gx, gw = torch.zeros(T * topk, H, dtype=torch.float16, device="cuda"), torch.zeros(T, topk, device="cuda")
    w = torch.rand(T, topk, generator=g)
    mswz.moe_combine_grad(plan, wide[:, :H], Xs, pos, w.cuda(), gx, gw)
    want = (w[:, :, None] * X.float()[:, None, :]).half()[(pos >= 0).cpu()]
    assert torch.equal(gx.cpu()[pos[pos >= 0].cpu().long()], want)


def test_rows_past_4_gib():
    T, topk, E, H = 150000, 4, 16, 4096
    plan = mswz.moe_plan_create(T, topk, E, H, "bf16")
    ids = torch.randint(0, E, (T, topk), generator=gen(14), dtype=torch.int32)
    X = torch.randint(-8, 8, (T, H), device="cuda").to(torch.bfloat16)
    offsets, order, pos, Xs = dispatch(plan, ids, X)
    at = torch.tensor([0, 1, T * topk // 2, T * topk - 2, T * topk - 1], device="cuda")
    assert torch.equal(Xs[at], X[order[at].long() // topk])
    Y = torch.empty_like(X)
    mswz.moe_combine(plan, Xs, pos, Y)
    assert torch.equal(Y, X * topk)   # small integers: exact
    w = torch.full((T, topk), 0.5, device="cuda")
    dw, dYs = torch.empty_like(w), torch.empty_like(Xs)
    mswz.moe_combine_grad(plan, X, Xs, pos, w, dYs, dw)
    assert torch.equal(dYs[at], Xs[at] * 0.5)
    last = X[-100:].double()
    assert torch.equal(dw[-100:].double(), (last * last).sum(1, keepdim=True).expand(-1, topk))


# ---- together, as a layer of experts -----------------------------------------------------

def layer(g, T, topk, E, H, N, dt="bf16"):
    """Everything a layer's forward and backward pass needs, on the GPU."""
    s = {"ids": ids_for(g, T, topk, E, 0.05).cuda(), "w": torch.rand(T, topk, generator=g).cuda(), "X": normal(g, T, H, dt=dt).cuda(),
         "B1": (normal(g, E, N, H, dt="f32") * H ** -0.5).to(DT[dt]).cuda(),
         "B2": (normal(g, E, H, N, dt="f32") * N ** -0.5).to(DT[dt]).cuda(), "dY": normal(g, T, H, dt=dt).cuda()}
    n = T * topk
    s["moe"] = mswz.moe_plan_create(T, topk, E, H, dt)
    s["fwd1"] = mswz.gemm_grouped_plan_create(E, n, N, H, dt, dt)
    s["fwd2"] = mswz.gemm_grouped_plan_create(E, n, H, N, dt, dt)
    s["bwd2"] = mswz.gemm_grouped_plan_create(E, n, N, H, dt, dt, b_major="mn")
    s["bwd1"] = mswz.gemm_grouped_plan_create(E, n, H, N, dt, dt, b_major="mn")
    s["dw2"] = mswz.gemm_grouped_plan_create(E, H, N, n, dt, "f32", axis="k")
    s["dw1"] = mswz.gemm_grouped_plan_create(E, N, H, n, dt, "f32", axis="k")
    s["ws"] = torch.empty(max(16, s["moe"].workspace_bytes()), dtype=torch.uint8, device="cuda")
    i32 = lambda *sh: torch.zeros(*sh, dtype=torch.int32, device="cuda")
    z = lambda *sh: torch.zeros(*sh, dtype=DT[dt], device="cuda")
    s.update(offsets=i32(E + 1), order=i32(n), pos=i32(T, topk), Xs=z(n, H), Hs=z(n, N), Ys=z(n, H), Y=z(T, H),
             dYs=z(n, H), dHs=z(n, N), dXs=z(n, H), dX=z(T, H), dw=torch.zeros(T, topk, device="cuda"),
             dB1=torch.zeros(E, N, H, device="cuda"), dB2=torch.zeros(E, H, N, device="cuda"))
    return s


def layer_pass(s):
    mswz.moe_dispatch(s["moe"], s["ids"], s["X"], s["Xs"], s["offsets"], s["order"], s["pos"], s["ws"])
    mswz.gemm_run_grouped(s["fwd1"], s["Xs"], s["B1"], s["offsets"], s["Hs"])
    mswz.gemm_run_grouped(s["fwd2"], s["Hs"], s["B2"], s["offsets"], s["Ys"])
    mswz.moe_combine(s["moe"], s["Ys"], s["pos"], s["Y"], weights=s["w"])
    mswz.moe_combine_grad(s["moe"], s["dY"], s["Ys"], s["pos"], s["w"], s["dYs"], s["dw"])
    mswz.gemm_run_grouped(s["bwd2"], s["dYs"], s["B2"], s["offsets"], s["dHs"])
    mswz.gemm_run_grouped(s["dw2"], s["dYs"], s["Hs"], s["offsets"], s["dB2"])
    mswz.gemm_run_grouped(s["bwd1"], s["dHs"], s["B1"], s["offsets"], s["dXs"])
    mswz.gemm_run_grouped(s["dw1"], s["dHs"], s["Xs"], s["offsets"], s["dB1"])
    mswz.moe_combine(s["moe"], s["dXs"], s["pos"], s["dX"])


OUT = ("Y", "dX", "dw", "dB1", "dB2")


def test_layer_of_experts_against_64_bits():
    s = layer(gen(20), 300, 2, 5, 128, 200)
    layer_pass(s)
    X, B1, B2, w = (s[k].double().cpu().requires_grad_() for k in ("X", "B1", "B2", "w"))
    ids = s["ids"].cpu()
    Y = torch.zeros(300, 128, dtype=torch.float64)
    for e in range(5):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        Y = Y.index_add(0, t, (X[t] @ B1[e].t() @ B2[e].t()) * w[t, j][:, None])
    Y.backward(s["dY"].double().cpu())
    # each of the chain's at most five 16-bit roundings moves a result by eps / 2 of intermediate values
    # whose errors add like independent ones; 4 x 5 x eps / 2 of the norm bounds them with room
    for name, ref in zip(OUT, (Y.detach(), X.grad, w.grad, B1.grad, B2.grad)):
        rel = float((s[name].double().cpu() - ref).norm() / ref.norm())
        assert rel <= 20 * torch.finfo(torch.bfloat16).eps / 2, (name, rel)


def test_layer_captured_and_replayed():
    s = layer(gen(21), 700, 4, 16, 256, 264)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer_pass(s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer_pass(s)
    for seed in (30, 31, 32):
        other = layer(gen(seed), 700, 4, 16, 256, 264)
        for k in ("ids", "w", "X", "B1", "B2", "dY"):
            s[k].copy_(other[k])
        for k in OUT:
            s[k].fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        layer_pass(other)
        torch.cuda.synchronize()
        for k in OUT + ("offsets", "order", "pos"):
            assert torch.equal(s[k], other[k]), (seed, k)


def test_w4_layer_captured_on_another_stream():
    """Sort, 4-bit experts, weighted sum: a decode step, replayed with new inputs."""
    g = gen(22)
    T, topk, E, H, N = 9, 4, 12, 256, 128
    moe_in, moe_out = mswz.moe_plan_create(T, topk, E, H, "bf16"), mswz.moe_plan_create(T, topk, E, N, "bf16")
    plan = mswz.gemm_w4_plan_create(T * topk, N, H, "bf16", "u4", "bf16", group=64, experts=E)
    x = w4_inputs(g, 1, N, H, E, "bf16", "u4", 64, True)
    c = {k: x[k].cuda() for k in ("B", "S", "Z")}
    i32 = lambda *sh: torch.zeros(*sh, dtype=torch.int32, device="cuda")
    ids, X, w = i32(T, topk), torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, topk, device="cuda")
    offsets, order, pos = i32(E + 1), i32(T * topk), i32(T, topk)
    Xs, Ys = (torch.zeros(T * topk, k, dtype=torch.bfloat16, device="cuda") for k in (H, N))
    Y = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(16, moe_in.workspace_bytes()), dtype=torch.uint8, device="cuda")
    ws4 = torch.empty(max(16, plan.workspace_bytes()), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        mswz.moe_dispatch(moe_in, ids, X, Xs, offsets, order, pos, ws, stream=stream)
        mswz.gemm_run_w4(plan, Xs, c["B"], c["S"], Ys, Z=c["Z"], offsets=offsets, workspace=ws4, stream=stream)
        mswz.moe_combine(moe_out, Ys, pos, Y, weights=w, stream=stream)

    graph = torch.cuda.CUDAGraph()
    step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    other = torch.cuda.Stream()
    for seed in range(3):
        g = gen(40 + seed)
        ids.copy_(ids_for(g, T, topk, E, 0.1))
        X.copy_(normal(g, T, H))
        w.copy_(torch.rand(T, topk, generator=g))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        replayed = Y.clone()
        Y.zero_()
        torch.cuda.synchronize()
        step(other)
        torch.cuda.synchronize()
        assert torch.equal(Y, replayed)
        ref = torch.zeros(T, N, dtype=torch.float64)
        for t in range(T):
            for j in range(topk):
                e = int(ids[t, j])
                if 0 <= e < E:
                    one = {"A": X[t:t + 1].cpu(), "B": x["B"][e:e + 1], "S": x["S"][e:e + 1], "Z": x["Z"][e:e + 1]}
                    ref[t] += float(w[t, j]) * w4_reference(one, "u4", 64, "bf16")[0][0]
        # Ys and Y are rounded to bf16: half a step of each of the topk rows and of the sum
        assert float((Y.double().cpu() - ref).norm() / ref.norm()) <= 2 * torch.finfo(torch.bfloat16).eps / 2


def test_two_streams_at_once():
    """One plan of each kind, used on two streams with a workspace each."""
    T, topk, E, H, N = 3000, 4, 24, 512, 264
    n = T * topk
    moe, up = mswz.moe_plan_create(T, topk, E, H, "bf16"), mswz.gemm_grouped_plan_create(E, n, N, H, "bf16", "f32")
    plan = mswz.gemm_w4_plan_create(64, 300, 8192, "f16", "e2m1", "f32", group=32)
    assert moe.workspace_bytes() and plan.workspace_bytes()

    def state(seed):
        g = gen(seed)
        x = {k: v.cuda() for k, v in w4_inputs(g, 64, 300, 8192, 0, "f16", "e2m1", 32, False).items() if v is not None}
        i32 = lambda *sh: torch.zeros(*sh, dtype=torch.int32, device="cuda")
        return dict(x=x, ids=ids_for(g, T, topk, E, 0.1).cuda(), X=normal(g, T, H).cuda(), w=torch.rand(T, topk, generator=g).cuda(),
                    B=normal(g, E, N, H).cuda(), offsets=i32(E + 1), order=i32(n), pos=i32(T, topk),
                    Xs=torch.zeros(n, H, dtype=torch.bfloat16, device="cuda"), Ys=torch.zeros(n, N, device="cuda"),
                    Y=torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"), D=torch.zeros(64, 300, device="cuda"),
                    ws=torch.zeros(moe.workspace_bytes(), dtype=torch.uint8, device="cuda"),
                    ws4=torch.zeros(plan.workspace_bytes(), dtype=torch.uint8, device="cuda"))

    def run(s, stream=None):
        mswz.moe_dispatch(moe, s["ids"], s["X"], s["Xs"], s["offsets"], s["order"], s["pos"], s["ws"], stream=stream)
        mswz.gemm_run_grouped(up, s["Xs"], s["B"], s["offsets"], s["Ys"], stream=stream)
        mswz.moe_combine(moe, s["Xs"], s["pos"], s["Y"], weights=s["w"], stream=stream)
        mswz.gemm_run_w4(plan, s["x"]["A"], s["x"]["B"], s["x"]["S"], s["D"], workspace=s["ws4"], stream=stream)

    states, out = [state(60), state(61)], ("offsets", "order", "pos", "Xs", "Ys", "Y", "D")
    alone = []
    for s in states:
        run(s)
        torch.cuda.synchronize()
        alone.append({k: s[k].clone() for k in out})
        for k in out:
            s[k].zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, stream in zip(states, streams):
            run(s, stream)
    torch.cuda.synchronize()
    for s, want in zip(states, alone):
        for k in out:
            assert torch.equal(s[k], want[k]), k


def test_tensors_that_do_not_fit_are_refused():
    plan = mswz.gemm_w4_plan_create(2, 16, 64, "bf16", "u4", "f32", group=64)
    A, B = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(16, 32, dtype=torch.uint8, device="cuda")
    S, D = torch.zeros(16, 1, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 16, device="cuda")
    mswz.gemm_run_w4(plan, A, B, S, D)
    for bad in (dict(A=A.half()), dict(A=A[:1]), dict(B=B[:8]), dict(S=S.half()), dict(D=D.half()), dict(D=D.t()),
                dict(A=A.cpu()), dict(B=B.cpu()), dict(Z=S), dict(offsets=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            mswz.gemm_run_w4(**{**dict(plan=plan, A=A, B=B, S=S, D=D), **bad})
    with pytest.raises(mswz.MswzError):
        mswz.gemm_run_w4(plan, A, B, S, D, beta=2)
    big = mswz.moe_plan_create(5000, 2, 4, 8, "f32")
    n = 10000
    i32 = lambda m: torch.zeros(m, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):   # no workspace
        mswz.moe_dispatch(big, i32(n), None, None, i32(5), i32(n), i32(n))
    with pytest.raises(ValueError):
        mswz.moe_dispatch(big, i32(n), torch.zeros(5000, 8, device="cuda"), None, i32(5), i32(n), i32(n),
                          torch.zeros(1 << 20, device="cuda"))


@pytest.mark.parametrize("a", ["bf16", "f16"])
@pytest.mark.parametrize("M", [1, 4, 16, 40, 64])
def test_w4_largest_e8m0_scales(M, a):
    """Scale bytes 249 .. 254 in any block of 32, with A small enough for finite results, and an infinity of A in
    a block whose neighbours have such scales."""
    g, N, K = gen(70 + M), 70, 416
    x = w4_inputs(g, M, N, K, 0, a, "e2m1", 32, False)
    x["A"] = (torch.randn(M, K, generator=g) * 2.0 ** -20).to(DT[a])
    x["S"] = torch.randint(249, 255, (1, N, K // 32), generator=g, dtype=torch.uint8)
    plan = mswz.gemm_w4_plan_create(M, N, K, a, "e2m1", "f32", group=32)
    ref, mag = w4_reference(x, "e2m1", 32, a)
    assert float(mag.max()) < torch.finfo(torch.float32).max
    got = w4_run(plan, x, torch.full((M, N), float("nan"), device="cuda"))
    check(got, ref, mag, K, "f32")
    at = torch.randint(0, K, (M,), generator=g)
    odd = torch.arange(M) % 2 == 1 if M > 1 else torch.ones(1, dtype=torch.bool)
    for m in torch.nonzero(odd)[:, 0].tolist():
        x["A"][m, at[m]] = float("inf") if m % 4 == 1 else -float("inf")
        pair = x["B"][0, :, int(at[m]) // 2]   # no zero weight meets it
        pair[pair % 8 == 0] |= 1
        pair[pair // 16 % 8 == 0] |= 16
    ref, mag = w4_reference(x, "e2m1", 32, a)
    got = w4_run(plan, x, torch.full((M, N), float("nan"), device="cuda")).cpu()
    assert torch.isinf(ref[odd]).all()
    assert torch.equal(got[odd].double(), ref[odd])
    check(got[~odd], ref[~odd], mag[~odd], K, "f32")


@pytest.mark.parametrize("M,N,K,G", [(1, 16, 128, 1024), (3, 40, 32, 128), (16, 33, 160, 256), (20, 70, 160, 384), (64, 100, 8096, 8192),
                                     (2, 70000, 96, 256)])
@pytest.mark.parametrize("a", ["f16", "bf16"])
def test_w4_scales_that_are_not_finite(M, N, K, G, a):
    """An infinite scale gives an infinite sum and NaN a NaN in its own column only; the chunks of 128 values
    that lie behind K add nothing."""
    x = w4_inputs(gen(K + G), M, N, K, 0, a, "u4", G, True)
    x["A"] = x["A"].abs() + 0.5            # sums of one sign
    x["B"] |= 0x88                         # weights 8 .. 15
    x["Z"] %= 8                            # zero points 0 .. 7
    x["S"][0, ::5, -1] = float("inf")
    x["S"][0, 1::5, 0] = -float("inf")
    x["S"][0, 2::5, -1] = float("nan")
    plan = mswz.gemm_w4_plan_create(M, N, K, a, "u4", "f32", group=G)
    got = w4_run(plan, x, torch.zeros((M, N), device="cuda")).cpu()
    assert (got[:, ::5] == float("inf")).all() and (got[:, 1::5] == -float("inf")).all() and torch.isnan(got[:, 2::5]).all()
    x["S"][~torch.isfinite(x["S"])] = 0.0
    ref, mag = w4_reference(x, "u4", G, a)
    for i in (3, 4):
        check(got[:, i::5], ref[:, i::5], mag[:, i::5], K, "f32")


@pytest.mark.parametrize("T,topk,E", [
    (16 * 1024, 1, 1024), (16 * 1024 + 1, 1, 1024),          # the edges between the ways of adding up counts
    (128 * 1024, 1, 128), (128 * 1024, 1, 129), (256 * 1024, 1, 3), (256 * 1024 + 1, 1, 3),
    (40000, 7, 1), (70001, 5, 17), (90000, 8, 300), (1 << 21, 2, 1000), ((1 << 24) - 1, 1, 1024), ((1 << 21) - 1, 8, 2),
])
def test_sort_of_many_choices(T, topk, E):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    ids = torch.randint(-1, E + 1, (T, topk), generator=g, device="cuda", dtype=torch.int32)
    plan, n = mswz.moe_plan_create(T, topk, E, 8, "bf16"), T * topk
    key = torch.where((ids < 0) | (ids >= E), E, ids).reshape(-1)
    key, slot = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device="cuda", dtype=torch.int32)).to(torch.int32)
    order = torch.where(key < E, slot, -1).to(torch.int32)
    pos = torch.empty_like(order)
    pos[slot] = torch.where(key < E, torch.arange(n, device="cuda"), -1).to(torch.int32)
    need = plan.workspace_bytes()
    out = [torch.full((m,), -99, dtype=torch.int32, device="cuda") for m in (E + 1, n, n)]
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    mswz.moe_dispatch(plan, ids, None, None, *out, workspace=ws[:need])
    for got, want in zip(out, (offsets, order, pos)):
        assert torch.equal(got, want)
    assert (ws[need:] == 0xFF).all()


def test_sort_of_many_choices_captured_and_replayed():
    T, topk, E, H = 50000, 8, 200, 16
    plan, n = mswz.moe_plan_create(T, topk, E, H, "f16"), T * topk
    ids, X = torch.zeros(T, topk, dtype=torch.int32, device="cuda"), torch.zeros(T, H, dtype=torch.float16, device="cuda")
    i32 = lambda m: torch.zeros(m, dtype=torch.int32, device="cuda")
    out, Xs = [i32(E + 1), i32(n), i32(n)], torch.zeros(n, H, dtype=torch.float16, device="cuda")
    ws = torch.empty(plan.workspace_bytes(), dtype=torch.uint8, device="cuda")
    mswz.moe_dispatch(plan, ids, X, Xs, *out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mswz.moe_dispatch(plan, ids, X, Xs, *out, workspace=ws)
    for seed in (80, 81, 82):
        g = gen(seed)
        new, rows = ids_for(g, T, topk, E, 0.1), normal(g, T, H, dt="f16")
        ids.copy_(new)
        X.copy_(rows)
        Xs.fill_(GUARD)
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        want = dispatch(plan, new, X)
        assert all(torch.equal(a, b.reshape(-1)) for a, b in zip(out, want))
        assert torch.equal(Xs, want[3])
        ref = sorted_reference(new, E)
        assert all(np.array_equal(a.cpu().numpy(), b.reshape(-1)) for a, b in zip(out, ref))


def test_sort_does_not_grow_with_the_square_of_the_choices():
    """Four times the choices take at most eight times as long (they took 12.8 times with every workgroup adding up
    the counts of all others)."""
    E, times = 1024, []
    for T in (1 << 17, 1 << 19):
        plan, n = mswz.moe_plan_create(T, 8, E, 8, "bf16"), T * 8
        ids = torch.randint(0, E, (T, 8), device="cuda", dtype=torch.int32)
        out = [torch.zeros(m, dtype=torch.int32, device="cuda") for m in (E + 1, n, n)]
        ws = torch.empty(plan.workspace_bytes(), dtype=torch.uint8, device="cuda")
        best = float("inf")
        for _ in range(8):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            mswz.moe_dispatch(plan, ids, None, None, *out, workspace=ws)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        times.append(best)
    assert times[1] <= 8 * times[0], times


W4_FORMS = [  # rows an expert, experts, N, steps' K: the widths and stages that the sizes choose (gemm_w4_kernel.hpp)
    (2, 64, 1000, 256), (3, 32, 510, 512), (4, 33, 250, 512), (2, 5, 100, 1024),           # tiles of 4 rows
    (7, 64, 1000, 256), (16, 32, 510, 512), (9, 17, 286, 512), (5, 4, 100, 1024),          # of 16
    (17, 64, 510, 256), (40, 5, 130, 512),                                                 # of 64
]


def w4_large_inputs(seed, M, N, K, E, a, w, G):
    """w4_inputs, made on the GPU."""
    g, x, sh = torch.Generator(device="cuda").manual_seed(seed), {"Z": None}, (max(1, E), N, -(-K // G))
    x["A"] = torch.randn(M, K, generator=g, device="cuda").to(DT[a])
    x["B"] = torch.randint(0, 256, (sh[0], N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    if w == "u4":
        x["S"] = ((0.5 + torch.rand(sh, generator=g, device="cuda")) * 0.02).to(DT[a])
        x["Z"] = torch.randint(0, 16, sh, generator=g, device="cuda", dtype=torch.uint8)
    else:
        x["S"] = torch.randint(118, 130, sh, generator=g, device="cuda", dtype=torch.uint8)
    return x


def w4_columns(x, cols):
    """The inputs of some columns of D, on the CPU."""
    return {k: v if v is None else (v if k == "A" else v[:, cols.cuda()]).cpu() for k, v in x.items()}


@pytest.mark.parametrize("steps", [2.6, 4, 5.2, 7, 8.5, 9])
@pytest.mark.parametrize("a,w,G", [("f16", "u4", 32), ("bf16", "u4", 64), ("f16", "u4", 128), ("bf16", "u4", 384),
                                   ("bf16", "e2m1", 32), ("f16", "e2m1", 32)])
def test_w4_many_steps(a, w, G, steps):
    """Every form of the kernel over whole and partial rounds of its stages, the last step whole and partly filled."""
    for rows, E, N, step in W4_FORMS:
        K = int(steps * step) // 32 * 32
        M, cols = rows * E, torch.cat((torch.arange(0, N - 16, 9), torch.arange(N - 16, N)))
        counts = torch.randint(0, 2 * rows + 1, (E,), generator=gen(K + E))
        while int(counts.sum()) > M:
            counts[int(counts.argmax())] //= 2
        bounds = bounds_of(counts.tolist())
        x = w4_large_inputs(K + E, M, N, K, E, a, w, G)
        plan = mswz.gemm_w4_plan_create(M, N, K, a, w, "f32", group=G, experts=E)
        assert plan.workspace_bytes() == 0
        got = w4_run(plan, x, torch.full((M, N), GUARD, device="cuda"), bounds.cuda())
        used = int(bounds[-1])
        ref, mag = w4_reference(w4_columns(x, cols), w, G, a, bounds.tolist())
        check(got[:used][:, cols.cuda()], ref[:used], mag[:used], K, "f32", (rows, E, N, K))
        assert torch.isfinite(got).all() and (got[used:] == GUARD).all()
        again = w4_run(plan, x, torch.full((M, N), GUARD, device="cuda"), bounds.cuda())
        assert torch.equal(got, again)


@pytest.mark.parametrize("M,N,K,G,a,w,d", [
    (64, 16400, 4640, 32, "bf16", "e2m1", "bf16"), (50, 16400, 4640, 64, "bf16", "u4", "bf16"),
    (64, 16390, 2560, 128, "f16", "u4", "f32"), (64, 32900, 1120, 32, "bf16", "e2m1", "f32"),
    (33, 32800, 1536, 32, "f16", "e2m1", "f32"), (130, 16400, 1312, 128, "bf16", "u4", "f32"),
    (64, 9000, 4640, 32, "bf16", "e2m1", "bf16"), (50, 12100, 2560, 64, "bf16", "u4", "f32"),
    (64, 8200, 3584, 128, "f16", "u4", "f32"), (64, 8190, 3584, 32, "f16", "e2m1", "f32"),
    (64, 700, 8224, 32, "bf16", "e2m1", "bf16"), (20, 260, 12320, 64, "bf16", "u4", "f32"),
])
def test_w4_one_matrix_many_steps(M, N, K, G, a, w, d):
    """17 rows and more by one matrix: two and three stages, K whole and split over workgroups."""
    cols = torch.cat((torch.arange(0, N - 70, 23), torch.arange(N - 70, N)))
    x = w4_large_inputs(K + N, M, N, K, 0, a, w, G)
    plan = mswz.gemm_w4_plan_create(M, N, K, a, w, d, group=G)
    got = w4_run(plan, x, torch.full((M, N), float("nan"), dtype=DT[d], device="cuda"))
    ref, mag = w4_reference(w4_columns(x, cols), w, G, a)
    check(got[:, cols.cuda()], ref, mag, K, d)
    assert torch.isfinite(got).all()
    again = w4_run(plan, x, torch.zeros((M, N), dtype=DT[d], device="cuda"))
    assert torch.equal(got, again)


# ---- calls that the header allows ----------------------------------------------------------

@pytest.mark.parametrize("T,topk,E,H,ld,dt", [(1, 1024, 30, 16, 0, "f16"), (3, 300, 1024, 4200, 4304, "bf16"), (9, 2, 4, 8200, 0, "f32"),
                                              (700, 2, 9, 72, 96, "f16"), (300, 5, 6, 4200, 4304, "bf16"), (9000, 1, 6, 520, 528, "f32")])
def test_dispatch_of_wide_and_pitched_rows(T, topk, E, H, ld, dt):
    g = gen(T + H)
    ids, X = ids_for(g, T, topk, E, 0.1), normal(g, T, H, dt=dt)
    plan = mswz.moe_plan_create(T, topk, E, H, dt, ldx=ld)
    wide = torch.full((T, ld or H), float("nan"), dtype=DT[dt], device="cuda")
    wide[:, :H] = X.cuda()
    offsets, order, pos, Xs = dispatch(plan, ids, wide[:, :H])
    want = sorted_reference(ids, E)
    assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip((offsets, order, pos), want))
    used = int(want[0][-1])
    assert torch.equal(Xs[:used].cpu(), X[torch.from_numpy(want[1][:used].astype(np.int64) // topk)])
    assert (Xs[used:] == GUARD).all()


@pytest.mark.parametrize("T,topk,H,dt", [(40, 3, 72, "bf16"), (700, 9, 264, "f32")])
def test_combine_of_any_positions(T, topk, H, dt):
    """A row named twice counts twice; positions outside the rows add nothing and leave dYs as it was."""
    g, n = gen(T + 90), T * topk
    Ys, dY, w = normal(g, n, H, dt=dt), normal(g, T, H, dt=dt), torch.randn(T, topk, generator=g)
    plan = mswz.moe_plan_create(T, topk, 4, H, dt)
    wrong = torch.tensor([-1, n, n + 1, -(1 << 31), (1 << 31) - 1])
    pos = torch.randint(0, n, (T, topk), generator=g)
    out = torch.rand(T, topk, generator=g) < 0.2
    pos[out] = wrong[torch.randint(0, 5, (int(out.sum()),), generator=g)]
    w[out] = float("inf")
    rows, wk = Ys[pos.clamp(0, n - 1)].double(), torch.where(out, 0.0, w).double()
    Y = torch.full((T, H), float("nan"), dtype=DT[dt], device="cuda")
    mswz.moe_combine(plan, Ys.cuda(), pos.int().cuda(), Y, weights=w.cuda())
    check(Y, (rows * wk[:, :, None]).sum(1), (rows * wk[:, :, None]).abs().sum(1), topk, dt)
    pos = torch.randperm(n, generator=g).reshape(T, topk)   # each row once, in any order
    pos[out] = wrong[torch.randint(0, 5, (int(out.sum()),), generator=g)]
    dYs = torch.full((n, H), GUARD, dtype=DT[dt], device="cuda")
    dw = torch.full((T, topk), float("nan"), device="cuda")
    mswz.moe_combine_grad(plan, dY.cuda(), Ys.cuda(), pos.int().cuda(), w.cuda(), dYs, dw)
    terms = torch.where(out[:, :, None], 0.0, Ys[pos.clamp(0, n - 1)].double() * dY.double()[:, None, :])
    check(dw, terms.sum(2), terms.abs().sum(2), H, "f32")
    want = torch.full((n, H), GUARD, dtype=DT[dt])
    want[pos[~out]] = (w[:, :, None] * dY.float()[:, None, :]).to(DT[dt])[~out]
    assert torch.equal(dYs.cpu(), want)


def test_most_tokens():
    """2^24 - 1 tokens through every call of the token movement."""
    T, E, H = (1 << 24) - 1, 5, 8
    plan, g = mswz.moe_plan_create(T, 1, E, H, "f16"), torch.Generator(device="cuda").manual_seed(91)
    ids = torch.randint(0, E, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    X = torch.randint(-8, 9, (T, H), generator=g, device="cuda").half()
    offsets, order, pos, Xs = dispatch(plan, ids, X)
    assert torch.equal(Xs, X[order.long()]) and torch.equal(order[pos[:, 0].long()].long(), torch.arange(T, device="cuda"))
    w = torch.full((T, 1), 2.0, device="cuda")
    Y, dYs, dw = torch.full_like(X, GUARD), torch.full_like(X, GUARD), torch.full_like(w, GUARD)
    mswz.moe_combine(plan, Xs, pos, Y, weights=w)
    assert torch.equal(Y, 2 * X)
    mswz.moe_combine_grad(plan, X, Xs, pos, w, dYs, dw)
    assert torch.equal(dYs, 2 * Xs) and torch.equal(dw[:, 0], (X.float() ** 2).sum(1))


@pytest.mark.parametrize("a,w,G,per", [("f16", "u4", 64, 3), ("bf16", "u4", 128, 12), ("bf16", "e2m1", 32, 30), ("f16", "e2m1", 32, 2)])
def test_w4_experts_with_pitches_beta_and_unaligned_d(a, w, G, per):
    E, N, K, lda, ldd = 6, 45, 352, 368, 47
    counts = [per, 0, 2 * per, 1, per - 1, 2 * per - 2]
    M, g = 6 * per + 3, gen(per)
    first = 2                              # rows before the first group and behind the last are left alone
    bounds = bounds_of(counts) + first
    x = w4_inputs(g, M, N, K, E, a, w, G, True)
    ref, mag = w4_reference(x, w, G, a, bounds.tolist())
    wide = torch.full((M, lda), float("nan"), dtype=DT[a])
    wide[first:int(bounds[-1]), :K] = x["A"][first:int(bounds[-1])]
    D0 = normal(g, M, ldd, dt=a)
    room = torch.zeros(M * ldd + 1, dtype=DT[a], device="cuda")
    D = room[1:].reshape(M, ldd)           # 2 bytes past a 16-byte boundary
    D.copy_(D0)
    plan = mswz.gemm_w4_plan_create(M, N, K, a, w, a, group=G, experts=E, lda=lda, ldd=ldd)
    c = {k: None if v is None else v.cuda() for k, v in x.items()}
    mswz.gemm_run_w4(plan, wide.cuda()[:, :K], c["B"], c["S"], D[:, :N], Z=c["Z"], offsets=bounds.cuda(), beta=1)
    used = slice(first, int(bounds[-1]))
    check(D[used, :N], (ref + D0[:, :N].double())[used], (mag + D0[:, :N].double().abs())[used], K, a)
    D = D.cpu()
    assert torch.equal(D[:, N:], D0[:, N:]) and torch.equal(D[:first], D0[:first]) and torch.equal(D[used.stop:], D0[used.stop:])


@pytest.mark.parametrize("E", [0, 1024])
def test_w4_most_rows(E):
    M, N, K = 1 << 16, 24, 64
    x = w4_large_inputs(92, M, N, K, E, "f16", "u4", 32)
    bounds = None
    if E:
        cuts = torch.randint(0, M + 1, (E - 1,), generator=gen(93)).sort()[0]
        bounds = torch.cat((torch.zeros(1), cuts, torch.full((1,), M))).int()
    plan = mswz.gemm_w4_plan_create(M, N, K, "f16", "u4", "f32", group=32, experts=E)
    got = w4_run(plan, x, torch.full((M, N), float("nan"), device="cuda"), bounds)
    ref, mag = w4_reference(w4_columns(x, torch.arange(N)), "u4", 32, "f16", None if bounds is None else bounds.tolist())
    check(got, ref, mag, K, "f32")


def test_w4_split_captured_and_replayed():
    """The product whose K is split over workgroups, with its workspace, as a graph."""
    M, N, K = 40, 300, 8192
    plan = mswz.gemm_w4_plan_create(M, N, K, "bf16", "u4", "bf16", group=128)
    x = {k: torch.empty_like(v) for k, v in w4_large_inputs(94, M, N, K, 0, "bf16", "u4", 128).items()}
    D, ws = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty(plan.workspace_bytes(), dtype=torch.uint8, device="cuda")
    run = lambda: mswz.gemm_run_w4(plan, x["A"], x["B"], x["S"], D, Z=x["Z"], workspace=ws)
    assert plan.workspace_bytes() > 0
    new = w4_large_inputs(95, M, N, K, 0, "bf16", "u4", 128)
    for k in x:
        x[k].copy_(new[k])
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in (96, 97, 98):
        new = w4_large_inputs(seed, M, N, K, 0, "bf16", "u4", 128)
        for k in x:
            x[k].copy_(new[k])
        D.fill_(float("nan"))
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        eager = w4_run(plan, new, torch.zeros_like(D))
        assert torch.equal(D, eager)
        check(D, *w4_reference(w4_columns(new, torch.arange(N)), "u4", 128, "bf16"), K, "bf16")


@pytest.mark.parametrize("first,gap", [(1, 0), (70, 0), (5, 9)])
def test_grouped_rows_before_the_first_group(first, gap):
    """Bounds may start behind row 0: rows before the first group are neither read nor written."""
    g, E, N, K, counts = gen(first), 3, 40, 136, [30, 0, 300]
    rows = first + sum(counts) + gap
    bounds = bounds_of(counts) + first
    used = slice(first, first + sum(counts))
    A, B = torch.full((rows, K), float("nan"), dtype=torch.bfloat16), normal(g, E, N, K)
    A[used] = normal(g, sum(counts), K)
    ref, mag = grouped_reference(A, B, bounds.tolist())
    for b_major, stored in (("k", B), ("mn", B.transpose(1, 2).contiguous())):
        D = torch.full((rows, N), GUARD, device="cuda")
        mswz.gemm_run_grouped(mswz.gemm_grouped_plan_create(E, rows, N, K, b_major=b_major), A.cuda(), stored.cuda(), bounds.cuda(), D)
        check(D[used], ref[used], mag[used], K, "f32")
        assert (D[:first] == GUARD).all() and (D[used.stop:] == GUARD).all()
    dY = torch.full((rows, N), float("inf"), dtype=torch.bfloat16)
    dY[used] = normal(g, sum(counts), N)
    dW = torch.full((E, N, K), float("nan"), device="cuda")
    mswz.gemm_run_grouped(mswz.gemm_grouped_plan_create(E, N, K, rows, axis="k"), dY.cuda(), A.cuda(), bounds.cuda(), dW)
    b = bounds.tolist()
    parts = [(dY[b[e]:b[e + 1]].double(), A[b[e]:b[e + 1]].double()) for e in range(E)]
    check(dW, torch.stack([y.t() @ a for y, a in parts]), torch.stack([y.abs().t() @ a.abs() for y, a in parts]), max(counts), "f32")
