"""Cases of the expert and 4-bit-weight operators: what is measured, in plain
torch (``own`` false) or through the package's entry points (``own`` true).

A case is a dict of plain values.  ``op`` names the pass:

    w4             D = A . dequant(B)^T, M rows, 4-bit B with group scales
    w4_experts     the same for rows sorted by expert, one B per expert
    dispatch       expert ids -> sorted order, and the token rows in that order
    combine        sorted rows back to tokens, weighted
    combine_train  combine and its gradients (rows and weights)
    experts        grouped 16-bit product over sorted rows
    experts_grad   its two gradients (rows and weights)
"""
import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # one token through a small projection: latency
        dict(name="w4_m1_small", op="w4", M=1, N=1024, K=1024, a="f16", w="u4", d="f16", G=128, zeros=True),
        # one token through the largest projection of the weight-streaming workload's sizes
        dict(name="w4_m1_large", op="w4", M=1, N=16384, K=8192, a="bf16", w="u4", d="bf16", G=128, zeros=True),
        # a decode batch of 64 against FP4 weights with power-of-two scales, the same sizes
        dict(name="w4_m64_e2m1", op="w4", M=64, N=16384, K=8192, a="bf16", w="e2m1", d="bf16", G=32, zeros=False),
        # a decode batch of 16 tokens, 4 experts each, through 4-bit experts
        dict(name="w4_experts_decode", op="w4_experts", M=64, E=32, N=4096, K=2048, a="bf16", w="u4", d="bf16",
             G=64, zeros=False, fill=1.0),
        # odd sizes, few of the sorted rows in use, a last scale group that is half a group
        dict(name="w4_experts_odd", op="w4_experts", M=37, E=6, N=1003, K=1056, a="f16", w="u4", d="f32",
             G=64, zeros=True, fill=0.8),
        # a few decode tokens to their experts: one short call
        dict(name="dispatch_decode", op="dispatch", T=7, k=2, E=8, H=1024, dt="f16", drop=0.0),
        # a training batch to its experts, some tokens padding
        dict(name="dispatch_train", op="dispatch", T=8192, k=8, E=128, H=2048, dt="bf16", drop=0.02),
        # a decode batch back from its experts
        dict(name="combine_decode", op="combine", T=33, k=4, E=32, H=4096, dt="f16", drop=0.0),
        # a training batch back from its experts, with the gradients of rows and weights
        dict(name="combine_train", op="combine_train", T=4096, k=8, E=64, H=2048, dt="bf16", drop=0.02),
        # a short ragged batch through small experts
        dict(name="experts_small", op="experts", M=203, E=8, N=520, K=264, a="f16", d="f16", fill=0.9),
        # a training batch through the experts
        dict(name="experts_train", op="experts", M=16384, E=16, N=4096, K=2048, a="bf16", d="bf16", fill=0.98),
        # the gradients of such a product: the rows' in 16 bits, the weights' in 32
        dict(name="experts_grad", op="experts_grad", M=8192, E=8, N=2048, K=2048, a="bf16", d="bf16", fill=1.0),
    ]


def _spread(rng, lo, hi, step=1):
    """A whole multiple of step, spread over the logarithm of lo .. hi."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v))) // step * step or step


def draw(rng):
    op = rng.choice(["w4", "w4_experts", "dispatch", "combine", "combine_train", "experts", "experts_grad"])
    if op in ("w4", "w4_experts"):
        a, w = rng.choice(["f16", "bf16"]), rng.choice(["u4", "u4", "e2m1"])
        case = dict(op=op, a=a, w=w, d=rng.choice([a, "f32"]), G=32 if w == "e2m1" else rng.choice([32, 64, 128]),
                    zeros=w == "u4" and rng.random() < 0.7)
        if op == "w4":
            return dict(case, M=_spread(rng, 1, 64), N=_spread(rng, 250, 16384), K=_spread(rng, 256, 8192, 32))
        case.update(M=_spread(rng, 1, 256), E=_spread(rng, 2, 32), K=_spread(rng, 128, 4096, 32),
                    fill=rng.choice([1.0, 0.8]))
        return dict(case, N=_spread(rng, 64, min(8192, (1 << 28) // (case["E"] * case["K"]))))
    if op in ("dispatch", "combine", "combine_train"):
        dt, E = rng.choice(["f16", "bf16", "bf16", "f32"]), _spread(rng, 4, 256)
        k, H = rng.randint(1, min(8, E)), _spread(rng, 64, 4096, 8)
        most = (1 << 27 if op == "dispatch" else 1 << 26) // (k * H * SIZE[dt] // 2)
        return dict(op=op, T=_spread(rng, 1, min(8192, most)), k=k, E=E, H=H, dt=dt, drop=rng.choice([0.0, 0.05]))
    a, E, K = rng.choice(["f16", "bf16"]), _spread(rng, 2, 32), _spread(rng, 64, 2048, 8)
    N = _spread(rng, 64, min(4096, (1 << 26) // (E * K)), 8)
    most = 1 << 15 if op == "experts_grad" else 1 << 14
    M = _spread(rng, 8, min(16384, most * 2048 // K * 2048 // N))
    return dict(op=op, M=M, E=E, N=N, K=K, a=a, d=rng.choice([a, "f32"]), fill=rng.choice([1.0, 0.9]))


def _offsets(g, rows, E, fill):
    """Group bounds of sorted rows: experts of unequal use, rows behind the last group left over."""
    used = max(1, int(rows * fill))
    pull = torch.randn(E, generator=g, device="cuda") * 0.5
    ids = (pull - torch.log(-torch.log(torch.rand(used, E, generator=g, device="cuda").clamp(1e-6, 1 - 1e-6)))).argmax(1)
    counts = torch.zeros(E, dtype=torch.int64, device="cuda").index_add_(0, ids, torch.ones_like(ids))
    bounds = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    bounds[1:] = counts.cumsum(0)
    return bounds, int(counts.max())


def _routing(g, T, k, E, drop):
    """k different experts for each token, unevenly liked, and their weights; dropped tokens have id -1."""
    score = torch.randn(T, E, generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
    top, ids = score.topk(k, dim=1)
    ids = ids.to(torch.int32)
    ids[torch.rand(T, generator=g, device="cuda") < drop] = -1
    return ids.contiguous(), torch.softmax(top, 1).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, s = case, {"case": case}

    def normal(*shape, dt, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(DT[dt])

    if c["op"] in ("w4", "w4_experts"):
        E = c.get("E", 1)
        groups = -(-c["K"] // c["G"])
        s["A"] = normal(c["M"], c["K"], dt=c["a"])
        s["B"] = torch.randint(0, 256, (E, c["N"], c["K"] // 2), generator=g, device="cuda", dtype=torch.uint8)
        if c["w"] == "u4":
            s["S"] = ((0.5 + torch.rand(E, c["N"], groups, generator=g, device="cuda")) * 0.01).to(DT[c["a"]])
        else:
            s["S"] = torch.randint(117, 122, (E, c["N"], groups), generator=g, device="cuda", dtype=torch.uint8)
        s["Z"] = torch.randint(5, 11, (E, c["N"], groups), generator=g, device="cuda", dtype=torch.uint8) if c["zeros"] else None
        s["offsets"] = None
        if c["op"] == "w4_experts":
            s["offsets"], s["most"] = _offsets(g, c["M"], E, c["fill"])
        s["D"] = torch.zeros(c["M"], c["N"], dtype=DT[c["d"]], device="cuda")
        if own:
            import mma_swizzled_operand_amd as mswz
            s["plan"] = mswz.gemm_w4_plan_create(c["M"], c["N"], c["K"], c["a"], c["w"], c["d"], group=c["G"],
                                                 experts=c.get("E", 0))
            s["ws"] = torch.empty(max(16, s["plan"].workspace_bytes()), dtype=torch.uint8, device="cuda")
    elif c["op"] in ("dispatch", "combine", "combine_train"):
        T, k, E, H = c["T"], c["k"], c["E"], c["H"]
        s["ids"], s["w"] = _routing(g, T, k, E, c["drop"])
        if c["op"] == "dispatch":
            s["X"] = normal(T, H, dt=c["dt"])
            s["Xs"] = torch.zeros(T * k, H, dtype=DT[c["dt"]], device="cuda")
            s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
            s["order"] = torch.zeros(T * k, dtype=torch.int32, device="cuda")
            s["pos"] = torch.zeros(T, k, dtype=torch.int32, device="cuda")
        else:
            s["pos"] = _sorted_by_expert(s["ids"], E)[2]
            s["Ys"] = normal(T * k, H, dt=c["dt"])
            s["Y"] = torch.zeros(T, H, dtype=DT[c["dt"]], device="cuda")
            if c["op"] == "combine_train":
                s["dY"] = normal(T, H, dt=c["dt"])
                s["dYs"] = torch.zeros(T * k, H, dtype=DT[c["dt"]], device="cuda")
                s["dw"] = torch.zeros(T, k, dtype=torch.float32, device="cuda")
        if own:
            import mma_swizzled_operand_amd as mswz
            s["plan"] = mswz.moe_plan_create(T, k, E, H, c["dt"])
            s["ws"] = torch.empty(max(16, s["plan"].workspace_bytes()), dtype=torch.uint8, device="cuda")
    else:
        M, E, N, K = c["M"], c["E"], c["N"], c["K"]
        s["offsets"], s["most"] = _offsets(g, M, E, c["fill"])
        s["A"] = normal(M, K, dt=c["a"])
        s["B"] = normal(E, N, K, dt=c["a"], scale=K ** -0.5)
        if c["op"] == "experts":
            s["D"] = torch.zeros(M, N, dtype=DT[c["d"]], device="cuda")
        else:
            s["dD"] = normal(M, N, dt=c["a"])
            s["dA"] = torch.zeros(M, K, dtype=DT[c["d"]], device="cuda")
            s["dB"] = torch.zeros(E, N, K, dtype=torch.float32, device="cuda")
        if own:
            import mma_swizzled_operand_amd as mswz
            if c["op"] == "experts":
                s["plan"] = mswz.gemm_grouped_plan_create(E, M, N, K, c["a"], c["d"], b_major="k")
            else:
                s["plan"] = mswz.gemm_grouped_plan_create(E, M, K, N, c["a"], c["d"], b_major="mn")
                s["plan_w"] = mswz.gemm_grouped_plan_create(E, N, K, M, c["a"], "f32", axis="k")
    return s


# ---- the plain forms ---------------------------------------------------------------

def _sorted_by_expert(ids, E):
    """offsets [E+1], order [T k] (slot of each sorted row, -1 behind the last) and pos [T][k] (sorted row of
    each slot, -1 for an id outside 0 .. E-1), by a stable sort."""
    n = ids.numel()
    key = torch.where((ids < 0) | (ids >= E), E, ids).reshape(-1)
    key, slot = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device=ids.device, dtype=key.dtype)).to(torch.int32)
    kept = key < E
    row = torch.arange(n, device=ids.device)
    order = torch.where(kept, slot, -1).to(torch.int32)
    pos = torch.empty(n, device=ids.device, dtype=torch.int32)
    pos[slot] = torch.where(kept, row, -1).to(torch.int32)
    return offsets, order, pos.reshape(ids.shape)


def _weights(s):
    """The 4-bit weights' values in 32 bits, [E][N][K]."""
    c, B = s["case"], s["B"]
    q = torch.stack((B & 15, B >> 4), -1).reshape(B.shape[0], B.shape[1], c["K"])
    group = torch.arange(c["K"], device="cuda") // c["G"]
    if c["w"] == "u4":
        z = s["Z"].float()[:, :, group] if s["Z"] is not None else 8.0
        return (q.float() - z) * s["S"].float()[:, :, group]
    table = torch.tensor(E2M1, device="cuda")
    return table[q.int()] * torch.exp2(s["S"].float() - 127.0)[:, :, group]


def _padded(offsets, most, rows):
    """Row of each (group, place) in groups of `most` places, and which of them hold a row."""
    row = offsets[:-1, None].long() + torch.arange(most, device="cuda")
    return row.clamp(max=rows - 1), row < offsets[1:, None]


def _grouped(A, B, s):
    """sorted rows of A (R, K) times their group's B (E, N, K), in 32 bits; rows behind the last group zero."""
    row, held = _padded(s["offsets"], s["most"], A.shape[0])
    out = torch.bmm(A.float()[row], B.transpose(1, 2))
    D = torch.zeros(A.shape[0], B.shape[1], device="cuda")
    D[row[held]] = out[held]
    return D


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import mma_swizzled_operand_amd as mswz
        if op in ("w4", "w4_experts"):
            mswz.gemm_run_w4(s["plan"], s["A"], s["B"], s["S"], s["D"], Z=s["Z"], offsets=s["offsets"], workspace=s["ws"])
            return s["D"]
        if op == "dispatch":
            mswz.moe_dispatch(s["plan"], s["ids"], s["X"], s["Xs"], s["offsets"], s["order"], s["pos"], s["ws"])
            return {"xs": s["Xs"], "offsets": s["offsets"], "order": s["order"], "pos": s["pos"]}
        if op in ("combine", "combine_train"):
            mswz.moe_combine(s["plan"], s["Ys"], s["pos"], s["Y"], weights=s["w"])
            if op == "combine":
                return s["Y"]
            mswz.moe_combine_grad(s["plan"], s["dY"], s["Ys"], s["pos"], s["w"], s["dYs"], s["dw"])
            return {"y": s["Y"], "dys": s["dYs"], "dw": s["dw"]}
        if op == "experts":
            mswz.gemm_run_grouped(s["plan"], s["A"], s["B"], s["offsets"], s["D"])
            return s["D"]
        mswz.gemm_run_grouped(s["plan"], s["dD"], s["B"], s["offsets"], s["dA"])
        mswz.gemm_run_grouped(s["plan_w"], s["dD"], s["A"], s["offsets"], s["dB"])
        return {"da": s["dA"], "db": s["dB"]}

    if op == "w4":
        return (s["A"].float() @ _weights(s)[0].t()).to(DT[c["d"]])
    if op == "w4_experts":
        return _grouped(s["A"], _weights(s), s).to(DT[c["d"]])
    if op == "dispatch":
        offsets, order, pos = _sorted_by_expert(s["ids"], c["E"])
        xs = torch.where(order[:, None] >= 0, s["X"][order.clamp(min=0).long() // c["k"]], 0)
        return {"xs": xs, "offsets": offsets, "order": order, "pos": pos}
    if op in ("combine", "combine_train"):
        pos, held = s["pos"].clamp(min=0).long(), s["pos"] >= 0
        w = torch.where(held, s["w"], 0.0)
        rows = torch.where(held[:, :, None], s["Ys"][pos].float(), 0.0)
        y = (rows * w[:, :, None]).sum(1).to(DT[c["dt"]])
        if op == "combine":
            return y
        dY = s["dY"].float()
        dw = (rows * dY[:, None, :]).sum(2)
        dys = torch.zeros(s["Ys"].shape, device="cuda", dtype=DT[c["dt"]])
        dys[pos[held]] = (w[:, :, None] * dY[:, None, :])[held].to(DT[c["dt"]])
        return {"y": y, "dys": dys, "dw": dw}
    if op == "experts":
        return _grouped(s["A"], s["B"].float(), s).to(DT[c["d"]])
    dA = _grouped(s["dD"], s["B"].float().transpose(1, 2), s)
    row, held = _padded(s["offsets"], s["most"], c["M"])
    rows = torch.where(held[:, :, None], s["dD"].float()[row], 0.0)
    dB = torch.bmm(rows.transpose(1, 2), s["A"].float()[row])
    return {"da": dA.to(DT[c["d"]]), "db": dB}


def work(case):
    c = case
    if c["op"] in ("w4", "w4_experts"):
        rows = max(1, int(c["M"] * c.get("fill", 1.0)))
        # experts that rows reach on average when they choose evenly
        E = c.get("E", 1)
        hit = E * (1 - (1 - 1 / E) ** rows) if E > 1 else 1
        groups = -(-c["K"] // c["G"])
        per = (2 if c["w"] == "u4" else 1) + (1 if c["zeros"] else 0)
        return {"bytes": hit * c["N"] * (c["K"] / 2 + groups * per) + rows * (2 * c["K"] + SIZE[c["d"]] * c["N"]),
                "flops": 2.0 * rows * c["N"] * c["K"]}
    if c["op"] in ("dispatch", "combine", "combine_train"):
        T, k, H, b = c["T"], c["k"], c["H"], SIZE[c["dt"]]
        sorted_rows = T * k * (1 - c["drop"])
        if c["op"] == "dispatch":
            return {"bytes": T * H * b + sorted_rows * H * b + T * k * 12 + 4 * (c["E"] + 1), "flops": 0.0}
        fwd = {"bytes": T * H * b + sorted_rows * H * b + T * k * 8, "flops": 2.0 * sorted_rows * H}
        if c["op"] == "combine":
            return fwd
        return {"bytes": fwd["bytes"] + T * H * b + sorted_rows * H * b + T * k * 4, "flops": 5.0 * sorted_rows * H}
    rows, b = max(1, int(c["M"] * c["fill"])), SIZE[c["d"]]
    one = 2.0 * rows * c["N"] * c["K"]
    A, B, D = rows * c["K"], c["E"] * c["N"] * c["K"], rows * c["N"]
    if c["op"] == "experts":
        return {"bytes": 2 * (A + B) + b * D, "flops": one}
    return {"bytes": 2 * (A + B + D) + b * A + 4 * B, "flops": 2 * one}


# ---- the definitions in 64 bits, apart from the plain forms --------------------------

def exact(case, seed):
    s, c = prepare(case, seed), case
    op = c["op"]
    if op in ("w4", "w4_experts"):
        E, N, K, G = c.get("E", 1), c["N"], c["K"], c["G"]
        bounds = s["offsets"].tolist() if s["offsets"] is not None else [0, c["M"]]
        D = torch.zeros(c["M"], N, dtype=torch.float64, device="cuda")
        for e in range(E):
            lo, hi = bounds[e], bounds[e + 1]
            if lo == hi:
                continue
            q = torch.empty(N, K, dtype=torch.int64, device="cuda")
            q[:, 0::2], q[:, 1::2] = s["B"][e] % 16, s["B"][e] // 16
            if c["w"] == "e2m1":
                mag = q % 8
                value = torch.where(mag < 2, mag * 0.5, (2 + mag % 2) * torch.pow(2.0, (mag // 2 - 2).double()))
                value = torch.where(q >= 8, -value, value)
                scale = torch.pow(2.0, s["S"][e].double() - 127)
            else:
                value, scale = q.double(), s["S"][e].double()
            for k in range(0, K, G):   # one scale group after the other
                v = value[:, k:k + G]
                if c["w"] == "u4":
                    v = v - (s["Z"][e][:, k // G].double()[:, None] if s["Z"] is not None else 8)
                D[lo:hi] += (s["A"][lo:hi, k:k + G].double() @ v.t()) * scale[:, k // G]
        return D
    if op == "dispatch":
        ids, T, k, E = s["ids"].cpu(), c["T"], c["k"], c["E"]
        lists = [[] for _ in range(E)]
        for slot, e in enumerate(ids.reshape(-1).tolist()):
            if 0 <= e < E:
                lists[e].append(slot)
        flat = [slot for one in lists for slot in one]
        xs = torch.zeros(T * k, c["H"], dtype=torch.float64, device="cuda")
        xs[:len(flat)] = s["X"].double()[torch.tensor([f // k for f in flat], dtype=torch.int64, device="cuda")]
        return {"xs": xs, "offsets": None, "order": None, "pos": None}
    if op in ("combine", "combine_train"):
        T, k, H = c["T"], c["k"], c["H"]
        y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        dys = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
        dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            t = (s["pos"][:, j] >= 0).nonzero()[:, 0]
            p = s["pos"][t, j].long()
            w, ys = s["w"][t, j].double()[:, None], s["Ys"][p].double()
            y[t] += w * ys
            if op == "combine_train":
                dY = s["dY"][t].double()
                dys[p] = w * dY
                dw[t, j] = torch.linalg.vecdot(dY, ys)
        return y if op == "combine" else {"y": y, "dys": dys, "dw": dw}
    b = s["offsets"].tolist()
    if op == "experts":
        D = torch.zeros(c["M"], c["N"], dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            D[b[e]:b[e + 1]] = s["A"][b[e]:b[e + 1]].double() @ s["B"][e].double().t()
        return D
    dA = torch.zeros(c["M"], c["K"], dtype=torch.float64, device="cuda")
    dB = torch.zeros(c["E"], c["N"], c["K"], dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        dD = s["dD"][b[e]:b[e + 1]].double()
        dA[b[e]:b[e + 1]] = dD @ s["B"][e].double()
        dB[e] = dD.t() @ s["A"][b[e]:b[e + 1]].double()
    return {"da": dA, "db": dB}
