"""Cases of the FP8 operators and of the one-call layer of experts: what is
measured, in plain torch (``own`` false) or through the package's entry points
(``own`` true).

A case is a dict of plain values.  ``op`` names the pass:

    fp8        D = A . B^T, A and B in E4M3 with an fp32 scale per block of 128
    fp8_grad   a linear layer's two gradients as such products (rows and weights)
    quant      16-bit rows to E4M3 with a scale per block, as they lie, transposed, or both
    layer      a gated layer of experts for a few tokens, 16-bit or E4M3 weights
"""
import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4, "e4m3": 1}
E4M3 = torch.float8_e4m3fn
BLOCK = 128


def listed():
    return [
        # one token through a projection: latency
        dict(name="fp8_m1", op="fp8", M=1, N=4096, K=4096, block="tile", d="bf16"),
        # a decode batch of 64 through the largest projection of the weight-streaming workload's sizes
        dict(name="fp8_m64", op="fp8", M=64, N=16384, K=8192, block="tile", d="bf16"),
        # a short ragged prompt, odd output columns, a last block of 16 values, 32-bit results
        dict(name="fp8_ragged", op="fp8", M=333, N=1003, K=2064, block="row", d="f32"),
        # the headline square product
        dict(name="fp8_square", op="fp8", M=8192, N=8192, K=8192, block="tile", d="bf16"),
        # a training step's gradients of a 4096 x 4096 projection over 8192 tokens
        dict(name="fp8_grad", op="fp8_grad", M=8192, N=4096, K=4096, d="bf16"),
        # a few decode tokens' activations
        dict(name="quant_decode", op="quant", M=17, K=4096, dt="f16", block="row", scales="f32", out="q"),
        # a training batch's activations, for the product and, transposed, for the weights' gradient
        dict(name="quant_train", op="quant", M=16384, K=4096, dt="bf16", block="row", scales="f32", out="both"),
        # a weight, for the product and, transposed, for the rows' gradient, power-of-two scales
        dict(name="quant_weight", op="quant", M=8192, K=8192, dt="bf16", block="tile", scales="pow2", out="both"),
        # one token through small experts: latency
        dict(name="layer_one_token", op="layer", T=1, k=2, E=8, H=1024, I=512, dt="f16", w="f16", act="silu", drop=0.0),
        # a decode batch of 16 tokens, 4 experts each, through 16-bit experts
        dict(name="layer_decode", op="layer", T=16, k=4, E=32, H=4096, I=2048, dt="bf16", w="bf16", act="silu", drop=0.0),
        # a decode batch of 64 tokens through many smaller E4M3 experts
        dict(name="layer_e4m3", op="layer", T=64, k=8, E=64, H=2048, I=1024, dt="bf16", w="e4m3", act="silu", drop=0.0),
        # odd sizes, some choices left out (experts that other devices hold)
        dict(name="layer_odd", op="layer", T=5, k=3, E=6, H=1000, I=328, dt="bf16", w="bf16", act="gelu", drop=0.3),
    ]


def _spread(rng, lo, hi, step=1):
    """A whole multiple of step, spread over the logarithm of lo .. hi."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v))) // step * step or step


def draw(rng):
    op = rng.choice(["fp8", "fp8", "fp8_grad", "quant", "layer", "layer"])
    if op == "fp8":
        N, K = _spread(rng, 100, 16384), _spread(rng, 128, 8192, 16)
        M = _spread(rng, 1, min(8192, (1 << 39) // (N * K)))
        return dict(op=op, M=M, N=N, K=K, block=rng.choice(["tile", "tile", "row"]), d=rng.choice(["bf16", "f16", "f32"]))
    if op == "fp8_grad":
        N, K = _spread(rng, 128, 8192, 16), _spread(rng, 128, 8192, 16)
        M = _spread(rng, 16, min(8192, (1 << 37) // (N * K)))
        return dict(op=op, M=M, N=N, K=K, d=rng.choice(["bf16", "bf16", "f32"]))
    if op == "quant":
        K = _spread(rng, 64, 8192, 16)
        return dict(op=op, M=_spread(rng, 1, min(16384, (1 << 26) // K)), K=K, dt=rng.choice(["f16", "bf16", "bf16", "f32"]),
                    block=rng.choice(["row", "row", "tile"]), scales=rng.choice(["f32", "pow2"]),
                    out=rng.choice(["q", "t", "both"]))
    dt = rng.choice(["f16", "bf16"])
    w = rng.choice([dt, dt, "e4m3"])
    step = 16 if w == "e4m3" else 8
    E, H = _spread(rng, 2, 64), _spread(rng, 128, 4096, step)
    I = _spread(rng, 64, min(4096, (1 << 28) // (E * H)), step)
    return dict(op=op, T=_spread(rng, 1, 64), k=rng.randint(1, min(8, E)), E=E, H=H, I=I, dt=dt, w=w,
                act=rng.choice(["silu", "gelu"]), drop=rng.choice([0.0, 0.1]))


def _blocks(n):
    return -(-n // BLOCK)


def _padded16(n):
    return -(-n // 16) * 16


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, s = case, {"case": case}

    def normal(*shape, dt, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(DT[dt])

    def e4m3(*shape):
        """Quantised values: each block's largest close to the format's."""
        return (torch.randn(*shape, generator=g, device="cuda") * 112).clamp(-448, 448).to(E4M3)

    def scales(*shape, size=1.0):
        return (0.5 + torch.rand(*shape, generator=g, device="cuda")) * (size / 112)

    if c["op"] == "fp8":
        M, N, K, kb = c["M"], c["N"], c["K"], _blocks(c["K"])
        s["A"], s["B"] = e4m3(M, K), e4m3(N, K)
        s["SA"] = scales(kb, M) * torch.exp(torch.randn(M, generator=g, device="cuda"))
        s["SB"] = scales(_blocks(N), kb, size=K ** -0.5) if c["block"] == "tile" else scales(kb, N, size=K ** -0.5)
        s["D"] = torch.zeros(M, N, dtype=DT[c["d"]], device="cuda")
        if own:
            import mma_swizzled_operand_amd as mswz
            s["plan"] = mswz.gemm_fp8_plan_create(M, N, K, c["d"], c["block"])
            s["ws"] = torch.empty(max(16, s["plan"].workspace_bytes()), dtype=torch.uint8, device="cuda")
    elif c["op"] == "fp8_grad":
        M, N, K, mp, mb = c["M"], c["N"], c["K"], _padded16(c["M"]), _blocks(c["M"])
        s["dY"], s["SdY"] = e4m3(M, N), scales(_blocks(N), M)
        s["Wt"], s["SWt"] = e4m3(K, N), scales(_blocks(K), _blocks(N), size=N ** -0.5)
        s["dYt"], s["SdYt"] = e4m3(N, mp), scales(mb, N)
        s["Xt"], s["SXt"] = e4m3(K, mp), scales(mb, K)
        for t in (s["dYt"], s["Xt"]):   # the tokens' tail of the transposed rows
            t.view(torch.uint8)[:, M:] = 0
        s["dX"] = torch.zeros(M, K, dtype=DT["bf16"], device="cuda")
        s["dW"] = torch.zeros(N, K, dtype=DT[c["d"]], device="cuda")
        if own:
            import mma_swizzled_operand_amd as mswz
            s["plan"] = mswz.gemm_fp8_plan_create(M, K, N, "bf16", "tile")
            s["plan_w"] = mswz.gemm_fp8_plan_create(N, K, mp, c["d"], "row")
            need = max(16, s["plan"].workspace_bytes(), s["plan_w"].workspace_bytes())
            s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    elif c["op"] == "quant":
        M, K, row = c["M"], c["K"], c["block"] == "row"
        # features of unequal size, a few tokens of padding
        x = torch.randn(M, K, generator=g, device="cuda") * torch.exp(torch.randn(K, generator=g, device="cuda"))
        x[torch.rand(M, generator=g, device="cuda") < 0.01] = 0
        s["X"] = x.to(DT[c["dt"]])
        s["Q"] = s["S"] = s["QT"] = s["ST"] = None
        if c["out"] != "t":
            s["Q"] = torch.zeros(M, K, dtype=E4M3, device="cuda")
            s["S"] = torch.zeros((_blocks(K), M) if row else (_blocks(M), _blocks(K)), device="cuda")
        if c["out"] != "q":
            s["QT"] = torch.zeros(K, _padded16(M), dtype=E4M3, device="cuda")
            s["ST"] = torch.zeros((_blocks(M), K) if row else (_blocks(K), _blocks(M)), device="cuda")
        if own:
            import mma_swizzled_operand_amd as mswz
            s["plan"] = mswz.quant_fp8_plan_create(M, K, c["dt"], c["block"], c["scales"])
    else:
        T, k, E, H, I = c["T"], c["k"], c["E"], c["H"], c["I"]
        # k different experts for each token, unevenly liked, and their weights; choices left out have id -1
        score = torch.randn(T, E, generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
        top, ids = score.topk(k, dim=1)
        ids = ids.to(torch.int32)
        ids[torch.rand(T, k, generator=g, device="cuda") < c["drop"]] = -1
        s["ids"], s["weights"] = ids.contiguous(), torch.softmax(top, 1).contiguous()
        s["most"] = int(torch.bincount(ids[ids >= 0].long(), minlength=E).max())
        s["X"] = normal(T, H, dt=c["dt"])
        s["S1"] = s["S2"] = None
        if c["w"] == "e4m3":
            s["W1"], s["W2"] = e4m3(E, 2 * I, H), e4m3(E, H, I)
            s["S1"] = scales(E, 2, _blocks(I), _blocks(H), size=H ** -0.5)
            s["S2"] = scales(E, _blocks(H), _blocks(I), size=I ** -0.5)
        else:
            s["W1"], s["W2"] = normal(E, 2 * I, H, dt=c["w"], scale=H ** -0.5), normal(E, H, I, dt=c["w"], scale=I ** -0.5)
        s["Y"] = torch.zeros(T, H, dtype=DT[c["dt"]], device="cuda")
        if own:
            import mma_swizzled_operand_amd as mswz
            s["plan"] = mswz.moe_layer_plan_create(T, k, E, H, I, c["dt"], c["w"], c["act"])
            s["ws"] = torch.empty(max(16, s["plan"].workspace_bytes()), dtype=torch.uint8, device="cuda")
    return s


# ---- the plain forms ---------------------------------------------------------------

def _rows_value(Q, S):
    """E4M3 rows (R, K) with scales (ceil(K/128), R), in 32 bits."""
    return Q.float() * S.t().repeat_interleave(BLOCK, 1)[:, :Q.shape[1]]


def _tiles_value(Q, S):
    """E4M3 matrices (..., R, K) with scales (..., ceil(R/128), ceil(K/128)), in 32 bits."""
    s = S.repeat_interleave(BLOCK, -1)[..., :Q.shape[-1]].repeat_interleave(BLOCK, -2)[..., :Q.shape[-2], :]
    return Q.float() * s


def _power(e):
    """2^e in 64 bits, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest(v):
    """v (64 bits) rounded to the nearest E4M3 value, ties to even, saturated; NaN stays."""
    step = _power(torch.frexp(v)[1].clamp(min=-5) - 4)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0).float().to(E4M3)


def _scale_of(largest, kind):
    """The scale of blocks whose largest magnitude (64 bits) is given."""
    s = largest.clamp(min=2.0 ** -90) / 448.0
    if kind == "f32":
        return s.float()
    fraction, exponent = torch.frexp(s)
    return _power(exponent - (fraction == 0.5).to(exponent.dtype)).float()


def _quantised_rows(x, kind):
    """Blocks of 128 along the last axis of x (64 bits): E4M3 values and their scales (blocks first)."""
    R, K = x.shape
    b = torch.nn.functional.pad(x, (0, _blocks(K) * BLOCK - K)).reshape(R, _blocks(K), BLOCK)
    S = _scale_of(b.abs().amax(2), kind)
    return _nearest(b / S.double()[:, :, None]).reshape(R, -1)[:, :K].contiguous(), S.t().contiguous()


def _quantised_tiles(x, kind):
    """Blocks of 128 x 128 of x (64 bits): E4M3 values and their scales."""
    R, K = x.shape
    b = torch.nn.functional.pad(x, (0, _blocks(K) * BLOCK - K, 0, _blocks(R) * BLOCK - R))
    b = b.reshape(_blocks(R), BLOCK, _blocks(K), BLOCK)
    S = _scale_of(b.abs().amax((1, 3)), kind)
    q = _nearest(b / S.double()[:, None, :, None]).reshape(_blocks(R) * BLOCK, -1)
    return q[:R, :K].contiguous(), S


def _quantised(s):
    c, x = s["case"], s["X"].double()
    form = _quantised_rows if c["block"] == "row" else _quantised_tiles
    out = {}
    if c["out"] != "t":
        out["q"], out["s"] = form(x, c["scales"])
    if c["out"] != "q":
        qt, out["st"] = form(x.t(), c["scales"])
        tail = _padded16(c["M"]) - c["M"]
        out["qt"] = torch.nn.functional.pad(qt.view(torch.uint8), (0, tail)).view(E4M3)
    return out


def _act(v, kind):
    if kind == "silu":
        return v / (1.0 + torch.exp(-v))
    return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))


def _layer(s):
    """Choices sorted by expert, every expert's rows in as many places as the fullest has, and back."""
    c = s["case"]
    T, k, E, I = c["T"], c["k"], c["E"], c["I"]
    if c["w"] == "e4m3":
        W1 = _tiles_value(s["W1"].view(E, 2, I, c["H"]), s["S1"]).reshape(E, 2 * I, c["H"])
        W2 = _tiles_value(s["W2"], s["S2"])
    else:
        W1, W2 = s["W1"].float(), s["W2"].float()
    ids = s["ids"].reshape(-1).long()
    key, slot = torch.sort(torch.where((ids >= 0) & (ids < E), ids, E), stable=True)
    first = torch.searchsorted(key, torch.arange(E + 1, device=key.device))
    row = first[:-1, None] + torch.arange(max(1, s["most"]), device=key.device)
    held = row < first[1:, None]
    choice = slot[row.clamp(max=T * k - 1)]
    up = torch.bmm(s["X"].float()[choice // k], W1.transpose(1, 2))
    ys = torch.bmm(_act(up[..., :I], c["act"]) * up[..., I:], W2.transpose(1, 2))
    of_choice = torch.zeros(T * k, c["H"], device=key.device)
    of_choice[choice[held]] = ys[held] * s["weights"].reshape(-1)[choice[held]][:, None]
    return of_choice.reshape(T, k, -1).sum(1).to(DT[c["dt"]])


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import mma_swizzled_operand_amd as mswz
        if op == "fp8":
            mswz.gemm_run_fp8(s["plan"], s["A"], s["SA"], s["B"], s["SB"], s["D"], workspace=s["ws"])
            return s["D"]
        if op == "fp8_grad":
            mswz.gemm_run_fp8(s["plan"], s["dY"], s["SdY"], s["Wt"], s["SWt"], s["dX"], workspace=s["ws"])
            mswz.gemm_run_fp8(s["plan_w"], s["dYt"], s["SdYt"], s["Xt"], s["SXt"], s["dW"], workspace=s["ws"])
            return {"dx": s["dX"], "dw": s["dW"]}
        if op == "quant":
            mswz.quant_fp8(s["plan"], s["X"], Q=s["Q"], S=s["S"], QT=s["QT"], ST=s["ST"])
            out = {"q": s["Q"], "s": s["S"], "qt": s["QT"], "st": s["ST"]}
            return {name: t for name, t in out.items() if t is not None}
        mswz.moe_layer(s["plan"], s["X"], s["ids"], s["weights"], s["W1"], s["W2"], s["Y"], S1=s["S1"], S2=s["S2"],
                       workspace=s["ws"])
        return s["Y"]

    if op == "fp8":
        B = _tiles_value(s["B"], s["SB"]) if c["block"] == "tile" else _rows_value(s["B"], s["SB"])
        return (_rows_value(s["A"], s["SA"]) @ B.t()).to(DT[c["d"]])
    if op == "fp8_grad":
        dX = _rows_value(s["dY"], s["SdY"]) @ _tiles_value(s["Wt"], s["SWt"]).t()
        dW = _rows_value(s["dYt"], s["SdYt"]) @ _rows_value(s["Xt"], s["SXt"]).t()
        return {"dx": dX.to(DT["bf16"]), "dw": dW.to(DT[c["d"]])}
    if op == "quant":
        return _quantised(s)
    return _layer(s)


def work(case):
    c = case
    if c["op"] == "fp8":
        M, N, K, kb = c["M"], c["N"], c["K"], _blocks(c["K"])
        sb = kb * (_blocks(N) if c["block"] == "tile" else N)
        return {"bytes": (M + N) * K + 4 * (kb * M + sb) + SIZE[c["d"]] * M * N, "flops": 2.0 * M * N * K}
    if c["op"] == "fp8_grad":
        M, N, K, mp, mb = c["M"], c["N"], c["K"], _padded16(c["M"]), _blocks(c["M"])
        rows = M * N + K * N + 2 * M * K + 4 * (_blocks(N) * M + _blocks(K) * _blocks(N))
        weights = (N + K) * mp + SIZE[c["d"]] * N * K + 4 * mb * (N + K)
        return {"bytes": rows + weights, "flops": 4.0 * M * N * K}
    if c["op"] == "quant":
        M, K = c["M"], c["K"]
        one = M * K + (4 * M * _blocks(K) if c["block"] == "row" else 4 * _blocks(M) * _blocks(K))
        return {"bytes": SIZE[c["dt"]] * M * K + one * (2 if c["out"] == "both" else 1), "flops": 3.0 * M * K}
    T, k, E, H, I = c["T"], c["k"], c["E"], c["H"], c["I"]
    choices = T * k * (1 - c["drop"])
    # experts that the choices reach on average when each token takes k different ones evenly
    hit = E * (1 - (1 - (1 - c["drop"]) * k / E) ** T)
    weights = 3 * H * I * SIZE[c["w"]]
    if c["w"] == "e4m3":
        weights += 4 * _blocks(H) * 3 * _blocks(I)
    return {"bytes": hit * weights + 2 * T * H * SIZE[c["dt"]] + 8 * T * k, "flops": 6.0 * choices * H * I}


# ---- the definitions in 64 bits, apart from the plain forms --------------------------

def _product64(A, SA, B, SB, tiles):
    """One block of 128 values of K after the other."""
    D = torch.zeros(A.shape[0], B.shape[0], dtype=torch.float64, device="cuda")
    column = torch.arange(B.shape[0], device="cuda")
    for b in range(SA.shape[0]):
        part = A[:, b * BLOCK:(b + 1) * BLOCK].double() @ B[:, b * BLOCK:(b + 1) * BLOCK].double().t()
        sb = SB[column // BLOCK, b] if tiles else SB[b]
        D += part * SA[b].double()[:, None] * sb.double()[None, :]
    return D


def _e4m3_table():
    """The format's finite magnitudes, ascending."""
    small = [m / 512 for m in range(8)]
    return torch.tensor(small + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)],
                        dtype=torch.float64, device="cuda")


def _quantised64(x, tall, wide, kind):
    """Blocks of tall x wide values of x: the nearest of all values of the format, ties to the even code."""
    R, K = x.shape
    table = _e4m3_table()
    middle = (table[1:] + table[:-1]) / 2
    row, col = torch.arange(R, device="cuda") // tall, torch.arange(K, device="cuda") // wide
    S = torch.empty(int(row[-1]) + 1, int(col[-1]) + 1, dtype=torch.float64, device="cuda")
    Q = torch.empty(R, K, dtype=torch.float64, device="cuda")
    for b in range(S.shape[1]):
        part = x[:, b * wide:(b + 1) * wide]
        most = torch.zeros(S.shape[0], dtype=torch.float64, device="cuda").scatter_reduce(0, row, part.abs().amax(1), "amax")
        most = torch.where(most < 2.0 ** -90, 2.0 ** -90, most)
        if kind == "f32":
            S[:, b] = (most / 448).float().double()
        else:
            # the smallest power of two that brings the largest into the format
            e = torch.floor(torch.log2(most)) - 9
            while bool((torch.exp2(e) * 448 < most).any()):
                e = torch.where(torch.exp2(e) * 448 < most, e + 1, e)
            S[:, b] = torch.exp2(e)
        ratio = part / S[row, b][:, None]
        code = torch.searchsorted(middle, ratio.abs().contiguous())
        # searchsorted puts a tie below; the even code is the one above where the one below is odd
        tie = middle[code.clamp(max=middle.numel() - 1)] == ratio.abs()
        code = torch.where(tie & (code % 2 == 1), code + 1, code)
        Q[:, b * wide:(b + 1) * wide] = torch.where(ratio < 0, -table[code], table[code])
    return Q, S


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "fp8":
        return _product64(s["A"], s["SA"], s["B"], s["SB"], c["block"] == "tile")
    if c["op"] == "fp8_grad":
        return {"dx": _product64(s["dY"], s["SdY"], s["Wt"], s["SWt"], True),
                "dw": _product64(s["dYt"], s["SdYt"], s["Xt"], s["SXt"], False)}
    if c["op"] == "quant":
        x, row, out = s["X"].double(), c["block"] == "row", {}
        if c["out"] != "t":
            out["q"], S = _quantised64(x, 1 if row else BLOCK, BLOCK, c["scales"])
            out["s"] = S.t().contiguous() if row else S
        if c["out"] != "q":
            qt, ST = _quantised64(x.t().contiguous(), 1 if row else BLOCK, BLOCK, c["scales"])
            out["st"] = ST.t().contiguous() if row else ST
            out["qt"] = torch.zeros(c["K"], _padded16(c["M"]), dtype=torch.float64, device="cuda")
            out["qt"][:, :c["M"]] = qt
        return out
    T, k, E, H, I = c["T"], c["k"], c["E"], c["H"], c["I"]
    Y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = (s["ids"] == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        W1, W2 = s["W1"][e].double(), s["W2"][e].double()
        if c["w"] == "e4m3":
            i, h = torch.arange(I, device="cuda") // BLOCK, torch.arange(H, device="cuda") // BLOCK
            W1[:I] *= s["S1"][e, 0].double()[i][:, h]
            W1[I:] *= s["S1"][e, 1].double()[i][:, h]
            W2 *= s["S2"][e].double()[h][:, i]
        x = s["X"][t].double()
        gate, up = x @ W1[:I].t(), x @ W1[I:].t()
        if c["act"] == "silu":
            gate = gate * torch.sigmoid(gate)
        else:
            gate = gate * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3))
        Y.index_add_(0, t, ((gate * up) @ W2.t()) * s["weights"][t, j].double()[:, None])
    return Y
