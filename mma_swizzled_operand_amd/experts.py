"""Binding of the expert operators (include/mswz_experts.h and
mswz_moe_layer.h): products with 4-bit weights, products over rows grouped by
expert, the token movement around them, and a whole layer of experts for a few
tokens.  Names and arguments are the C ABI's.  Tensors are checked against the
plan's sizes and types and must share one GPU; a call runs on that GPU, on
``stream`` (default: torch's current stream of that GPU).

    moe = moe_plan_create(T, topk, E, H, "bf16")
    moe_dispatch(moe, ids, X, Xs, offsets, order, pos, workspace)
    up = gemm_grouped_plan_create(E, T * topk, N, H, "bf16", "bf16")
    gemm_run_grouped(up, Xs, B, offsets, Ys)                  # Ys[p] = Xs[p] . B[e]^T
    moe_combine(moe_plan_create(T, topk, E, N, "bf16"), Ys, pos, Y, weights=w)

    layer = moe_layer_plan_create(T, topk, E, H, I, "bf16")   # decoding
    moe_layer(layer, X, ids, w, W1, W2, Y, workspace=workspace)
"""
from __future__ import annotations

import ctypes
import functools

torch = None    # imported by the first call that takes tensors; the package and its plans work without it

__all__ = ["W4Plan", "GroupedPlan", "MoePlan", "LayerPlan", "gemm_w4_plan_create", "gemm_run_w4", "gemm_grouped_plan_create",
           "gemm_run_grouped", "moe_plan_create", "moe_dispatch", "moe_combine", "moe_combine_grad",
           "moe_layer_plan_create", "moe_layer"]

_TORCH = {"f16": "float16", "bf16": "bfloat16", "f32": "float32"}
_WEIGHTS = {"u4": 9, "e2m1": 5}
_AXES = {"m": 0, "k": 1}
_ACTS = {"silu": 0, "gelu": 1}


def declare(h):
    """Argument types of the library's functions (called once when it is loaded)."""
    i64, i32, vp, c_int = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int
    out = ctypes.POINTER(vp)
    for name, args, res in (
            ("gemm_w4_plan_create", [out, i64, i64, i64, i64, c_int, c_int, c_int, i32, i64, i64], c_int),
            ("gemm_w4_plan_destroy", [vp], None),
            ("gemm_w4_plan_workspace_size", [vp], i64),
            ("gemm_run_w4", [vp, vp, vp, vp, vp, vp, vp, c_int, vp, i64, vp], c_int),
            ("gemm_grouped_plan_create", [out, i64, i64, i64, i64, c_int, c_int, c_int, c_int], c_int),
            ("gemm_grouped_plan_destroy", [vp], None),
            ("gemm_run_grouped", [vp, vp, vp, vp, vp, c_int, vp], c_int),
            ("moe_plan_create", [out, i64, i64, i64, i64, c_int, i64], c_int),
            ("moe_plan_destroy", [vp], None),
            ("moe_plan_workspace_size", [vp], i64),
            ("moe_dispatch", [vp, vp, vp, vp, vp, vp, vp, vp, i64, vp], c_int),
            ("moe_combine", [vp, vp, vp, vp, vp, vp], c_int),
            ("moe_combine_grad", [vp, vp, vp, vp, vp, vp, vp, vp], c_int),
            ("moe_layer_plan_create", [out, i64, i64, i64, i64, i64, c_int, c_int, c_int, i64], c_int),
            ("moe_layer_plan_destroy", [vp], None),
            ("moe_layer_plan_workspace_size", [vp], i64),
            ("moe_layer", [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, vp], c_int)):
        f = getattr(h, name)
        f.argtypes, f.restype = args, res


def _need_torch():
    global torch, _current_stream
    if torch is None:
        import torch as module
        # The handle of torch's current stream of a GPU.  (torch.cuda.current_stream
        # makes a stream object first: 1.1 us of a call that takes 6.)
        _current_stream = getattr(module._C, "_cuda_getCurrentRawStream", None) or (
            lambda dev: module.cuda.current_stream(dev).cuda_stream)
        torch = module   # (last: another thread goes by it)


def _type(name):
    """torch's name of an element type, looked up when it is first asked for."""
    def get(plan):
        _need_torch()
        return getattr(torch, _TORCH[getattr(plan, name)])
    return functools.cached_property(get)


class _Plan:
    """Owns a C plan handle, made by ``<_make>`` and freed by ``<_free>``."""
    _h = None
    _make = _free = ""

    def _create(self, *args):
        from . import MswzError, load
        lib, h = load(), ctypes.c_void_p()
        make = getattr(lib, self._make)
        # (ctypes would cut a number off to the argument's bits)
        if any(t(v).value != v for t, v in zip(make.argtypes[1:], args)):
            raise MswzError(-1, self._make)
        rc = make(ctypes.byref(h), *args)
        if rc != 0:
            raise MswzError(rc, self._make)
        self._lib, self._h = lib, h

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("plan has been destroyed")
        return self._h

    def destroy(self):
        if self._h is not None:
            getattr(self._lib, self._free)(self._h)
            self._h = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def _dt(name):
    from . import DTYPES
    if name not in DTYPES:
        raise ValueError(f"unknown dtype {name!r}")
    return DTYPES[name]


def _pick(table, name, what):
    if name not in table:
        raise ValueError(f"unknown {what} {name!r}")
    return table[name]


class W4Plan(_Plan):
    """A product with 4-bit weights (gemm_w4_plan_create)."""
    _make, _free = "gemm_w4_plan_create", "gemm_w4_plan_destroy"
    a_type, d_type = _type("a_dt"), _type("d_dt")

    @functools.cached_property
    def s_type(self):
        _need_torch()
        return self.a_type if self.w_dt == "u4" else torch.uint8

    def __init__(self, M, N, K, a_dt="bf16", w_dt="u4", d_dt="bf16", group=128, experts=0, lda=0, ldd=0):
        self.M, self.N, self.K, self.E = int(M), int(N), int(K), int(experts)
        self._create(self.M, self.N, self.K, self.E, _dt(a_dt), _pick(_WEIGHTS, w_dt, "weight format"), _dt(d_dt),
                     int(group), int(lda), int(ldd))
        self.a_dt, self.w_dt, self.d_dt, self.group = a_dt, w_dt, d_dt, int(group)
        self.lda, self.ldd = int(lda) or self.K, int(ldd) or self.N
        matrices = max(1, self.E)
        self.b_numel = matrices * self.N * (self.K // 2)
        self.s_numel = matrices * self.N * (-(-self.K // self.group))
        self.ws_bytes, self._run = int(self._lib.gemm_w4_plan_workspace_size(self._h)), self._lib.gemm_run_w4

    def workspace_bytes(self) -> int:
        """Device workspace gemm_run_w4 needs for this plan (0: none)."""
        return self.ws_bytes


class GroupedPlan(_Plan):
    """A product over groups of rows (gemm_grouped_plan_create)."""
    _make, _free = "gemm_grouped_plan_create", "gemm_grouped_plan_destroy"
    type, d_type = _type("dt"), _type("d_dt")

    def __init__(self, E, M, N, K, dt="bf16", d_dt="f32", axis="m", b_major=None):
        from . import MAJORS
        b_major = b_major or ("mn" if axis == "k" else "k")
        self.E, self.M, self.N, self.K = int(E), int(M), int(N), int(K)
        self._create(self.E, self.M, self.N, self.K, _dt(dt), _dt(d_dt), _pick(_AXES, axis, "axis"),
                     _pick(MAJORS, b_major, "major"))
        self.dt, self.d_dt, self.axis, self.b_major = dt, d_dt, axis, b_major
        self.a_numel = self.M * self.K
        self.b_numel = self.K * self.N * (1 if axis == "k" else self.E)
        self.d_numel = self.M * self.N * (self.E if axis == "k" else 1)
        self._run = self._lib.gemm_run_grouped


class MoePlan(_Plan):
    """The token movement of T tokens of H elements and topk choices among E experts (moe_plan_create)."""
    _make, _free = "moe_plan_create", "moe_plan_destroy"
    type = _type("dt")

    def __init__(self, T, topk, E, H, dt="bf16", ldx=0):
        self.T, self.topk, self.E, self.H = int(T), int(topk), int(E), int(H)
        self._create(self.T, self.topk, self.E, self.H, _dt(dt), int(ldx))
        self.dt, self.ldx = dt, int(ldx) or self.H
        self.choices = self.T * self.topk
        self.ws_bytes = int(self._lib.moe_plan_workspace_size(self._h))
        self._dispatch, self._combine = self._lib.moe_dispatch, self._lib.moe_combine
        self._combine_grad = self._lib.moe_combine_grad

    def workspace_bytes(self) -> int:
        """Device workspace moe_dispatch needs for this plan (0: none)."""
        return self.ws_bytes


class LayerPlan(_Plan):
    """A whole gated layer of E experts for T tokens of topk choices each (moe_layer_plan_create)."""
    _make, _free = "moe_layer_plan_create", "moe_layer_plan_destroy"
    type = _type("dt")

    def __init__(self, T, topk, E, H, I, dt="bf16", w_dt=None, act="silu", ldx=0):
        w_dt = w_dt or dt
        self.T, self.topk, self.E, self.H, self.I = int(T), int(topk), int(E), int(H), int(I)
        self._create(self.T, self.topk, self.E, self.H, self.I, _dt(dt), _dt(w_dt), _pick(_ACTS, act, "activation"),
                     int(ldx))
        self.dt, self.w_dt, self.act, self.ldx = dt, w_dt, act, int(ldx) or self.H
        self.choices = self.T * self.topk
        self.w1_numel = self.E * 2 * self.I * self.H
        tiles = self.E * -(-self.I // 128) * -(-self.H // 128)
        self.s1_numel, self.s2_numel = 2 * tiles, tiles
        self.ws_bytes, self._run = int(self._lib.moe_layer_plan_workspace_size(self._h)), self._lib.moe_layer

    def workspace_bytes(self) -> int:
        """Device workspace moe_layer needs for this plan."""
        return self.ws_bytes


def gemm_w4_plan_create(M, N, K, a_dt="bf16", w_dt="u4", d_dt="bf16", group=128, experts=0, lda=0, ldd=0) -> W4Plan:
    """Plan of D = beta*D + A . dequant(B)^T, B in 4 bits with group scales; experts > 0: one B per expert and
    rows sorted by expert."""
    return W4Plan(M, N, K, a_dt, w_dt, d_dt, group, experts, lda, ldd)


def gemm_grouped_plan_create(E, M, N, K, dt="bf16", d_dt="f32", axis="m", b_major=None) -> GroupedPlan:
    """Plan of a product over E groups of rows: axis "m", D[p] = beta*D[p] + A[p] . B[e]^T, or "k",
    D[e] = beta*D[e] + sum_p A[p]^T B[p]."""
    return GroupedPlan(E, M, N, K, dt, d_dt, axis, b_major)


def moe_plan_create(T, topk, E, H, dt="bf16", ldx=0) -> MoePlan:
    """Plan of moe_dispatch, moe_combine and moe_combine_grad."""
    return MoePlan(T, topk, E, H, dt, ldx)


def moe_layer_plan_create(T, topk, E, H, I, dt="bf16", w_dt=None, act="silu", ldx=0) -> LayerPlan:
    """Plan of moe_layer: W1 [E][2I][H] and W2 [E][H][I] in w_dt (dt, or "e4m3" with a scale per 128 x 128 tile),
    activation "silu" or "gelu" of the gate."""
    return LayerPlan(T, topk, E, H, I, dt, w_dt, act, ldx)


def _packed(t, dtype, numel, dev, name):
    """Device pointer of a contiguous tensor of ``numel`` elements on GPU ``dev``."""
    if t.dtype is dtype and t.numel() == numel and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    raise ValueError(f"{name}: expected a contiguous {dtype} tensor of {numel} elements on GPU {dev}, got "
                     f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")


def _rows(t, dtype, rows, cols, ld, dev, name):
    """Device pointer of ``rows`` rows of ``cols`` elements, ``ld`` elements apart: packed rows in any contiguous
    tensor, others in a 2-D view."""
    if ld == cols:
        return _packed(t, dtype, rows * cols, dev, name)
    if (t.dtype != dtype or t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols or t.get_device() != dev or
            (rows > 1 and t.stride(0) != ld) or (cols > 1 and t.stride(1) != 1)):
        raise ValueError(f"{name}: expected a ({rows}, {cols}) {dtype} view with rows {ld} elements apart on GPU "
                         f"{dev}, got {t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")
    return t.data_ptr()


def _workspace(t, need, dev):
    if not need:
        return None
    if t is None:
        raise ValueError(f"workspace: the plan needs {need} bytes")
    if t.numel() * t.element_size() >= need and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    raise ValueError(f"workspace: expected a contiguous tensor of at least {need} bytes on GPU {dev}, got "
                     f"{t.numel() * t.element_size()} bytes on {t.device}")


def _device(plan, kind, t, name):
    """The GPU that tensor ``t`` lives on, after checking the plan."""
    if not isinstance(plan, kind):
        raise TypeError(f"expected a {kind.__name__}, got {type(plan).__name__}")
    if plan._h is None:
        raise ValueError("plan has been destroyed")
    if torch is None:
        _need_torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name}: tensor must live in GPU memory")
    return dev


def _call(fn, what, dev, stream, *args):
    """Call a run function with the stream's handle last, on GPU ``dev``."""
    if stream is None:
        stream = _current_stream(dev)
    elif not isinstance(stream, int):
        if stream.device.index != dev:
            raise ValueError(f"stream: on {stream.device}, the tensors are on GPU {dev}")
        stream = stream.cuda_stream
    if torch.cuda.current_device() == dev:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, stream)
    if rc != 0:
        from . import MswzError
        raise MswzError(rc, what)


def gemm_run_w4(plan: W4Plan, A, B, S, D, Z=None, offsets=None, beta: int = 0, workspace=None, stream=None) -> None:
    """Enqueue D = beta*D + A . dequant(B)^T.  B uint8 [E][N][K/2]; S and Z [E][N][ceil(K/group)], Z uint8 or None
    (u4: zero point 8); offsets int32 [E+1] for a plan with experts, else None."""
    dev = _device(plan, W4Plan, A, "A")
    if (offsets is None) != (plan.E == 0):
        raise ValueError("offsets: given exactly for a plan with experts")
    if Z is not None and plan.w_dt != "u4":
        raise ValueError("Z: only u4 weights have zero points")
    _call(plan._run, "gemm_run_w4", dev, stream, plan._h,
          _rows(A, plan.a_type, plan.M, plan.K, plan.lda, dev, "A"),
          _packed(B, torch.uint8, plan.b_numel, dev, "B"), _packed(S, plan.s_type, plan.s_numel, dev, "S"),
          None if Z is None else _packed(Z, torch.uint8, plan.s_numel, dev, "Z"),
          None if offsets is None else _packed(offsets, torch.int32, plan.E + 1, dev, "offsets"),
          _rows(D, plan.d_type, plan.M, plan.N, plan.ldd, dev, "D"), int(beta),
          _workspace(workspace, plan.ws_bytes, dev), plan.ws_bytes)


def gemm_run_grouped(plan: GroupedPlan, A, B, offsets, D, beta: int = 0, stream=None) -> None:
    """Enqueue the grouped product (axis "m": A [M][K], B [E][N][K] or [E][K][N], D [M][N]; axis "k": A [K][M],
    B [K][N], D [E][M][N])."""
    dev = _device(plan, GroupedPlan, A, "A")
    _call(plan._run, "gemm_run_grouped", dev, stream, plan._h,
          _packed(A, plan.type, plan.a_numel, dev, "A"), _packed(B, plan.type, plan.b_numel, dev, "B"),
          _packed(offsets, torch.int32, plan.E + 1, dev, "offsets"),
          _packed(D, plan.d_type, plan.d_numel, dev, "D"), int(beta))


def moe_dispatch(plan: MoePlan, ids, X, Xs, offsets, order, pos, workspace=None, stream=None) -> None:
    """Enqueue the sort of ids [T][topk] by expert (offsets, order and pos are written) and, unless X and Xs are
    None, Xs[pos[t][j]] = X[t]."""
    dev = _device(plan, MoePlan, ids, "ids")
    if (X is None) != (Xs is None):
        raise ValueError("X and Xs: both or neither")
    n = plan.choices
    _call(plan._dispatch, "moe_dispatch", dev, stream, plan._h, _packed(ids, torch.int32, n, dev, "ids"),
          None if X is None else _rows(X, plan.type, plan.T, plan.H, plan.ldx, dev, "X"),
          None if X is None else _packed(Xs, plan.type, n * plan.H, dev, "Xs"),
          _packed(offsets, torch.int32, plan.E + 1, dev, "offsets"), _packed(order, torch.int32, n, dev, "order"),
          _packed(pos, torch.int32, n, dev, "pos"), _workspace(workspace, plan.ws_bytes, dev), plan.ws_bytes)


def moe_combine(plan: MoePlan, Ys, pos, Y, weights=None, stream=None) -> None:
    """Enqueue Y[t] = sum_j weights[t][j] Ys[pos[t][j]] (weights None: ones, the gradient of moe_dispatch)."""
    dev = _device(plan, MoePlan, Ys, "Ys")
    n = plan.choices
    _call(plan._combine, "moe_combine", dev, stream, plan._h,
          _packed(Ys, plan.type, n * plan.H, dev, "Ys"), _packed(pos, torch.int32, n, dev, "pos"),
          None if weights is None else _packed(weights, torch.float32, n, dev, "weights"),
          _rows(Y, plan.type, plan.T, plan.H, plan.ldx, dev, "Y"))


def moe_combine_grad(plan: MoePlan, dY, Ys, pos, weights, dYs, dw, stream=None) -> None:
    """Enqueue moe_combine's gradients: dYs[pos[t][j]] = weights[t][j] dY[t] and dw[t][j] = <dY[t], Ys[pos[t][j]]>."""
    dev = _device(plan, MoePlan, dY, "dY")
    n = plan.choices
    _call(plan._combine_grad, "moe_combine_grad", dev, stream, plan._h,
          _rows(dY, plan.type, plan.T, plan.H, plan.ldx, dev, "dY"), _packed(Ys, plan.type, n * plan.H, dev, "Ys"),
          _packed(pos, torch.int32, n, dev, "pos"), _packed(weights, torch.float32, n, dev, "weights"),
          _packed(dYs, plan.type, n * plan.H, dev, "dYs"), _packed(dw, torch.float32, n, dev, "dw"))


def moe_layer(plan: LayerPlan, X, ids, weights, W1, W2, Y, S1=None, S2=None, workspace=None, stream=None) -> None:
    """Enqueue Y[t] = sum_j weights[t][j] W2[e] (act(W1[e][:I] X[t]) * (W1[e][I:] X[t])), e = ids[t][j].  S1 fp32
    [E][2][ceil(I/128)][ceil(H/128)] and S2 [E][ceil(H/128)][ceil(I/128)] for E4M3 weights, else None."""
    dev = _device(plan, LayerPlan, X, "X")
    e4m3 = plan.w_dt == "e4m3"
    if (S1 is None) == e4m3 or (S2 is None) == e4m3:
        raise ValueError("S1 and S2: given exactly for E4M3 weights")
    bytes_ok = (torch.float8_e4m3fn, torch.uint8)
    t1, t2 = ((w.dtype if w.dtype in bytes_ok else bytes_ok[0]) if e4m3 else plan.type for w in (W1, W2))
    n = plan.choices
    _call(plan._run, "moe_layer", dev, stream, plan._h, _rows(X, plan.type, plan.T, plan.H, plan.ldx, dev, "X"),
          _packed(ids, torch.int32, n, dev, "ids"), _packed(weights, torch.float32, n, dev, "weights"),
          _packed(W1, t1, plan.w1_numel, dev, "W1"),
          None if S1 is None else _packed(S1, torch.float32, plan.s1_numel, dev, "S1"),
          _packed(W2, t2, plan.w1_numel // 2, dev, "W2"),
          None if S2 is None else _packed(S2, torch.float32, plan.s2_numel, dev, "S2"),
          _rows(Y, plan.type, plan.T, plan.H, plan.ldx, dev, "Y"), _workspace(workspace, plan.ws_bytes, dev),
          plan.ws_bytes)
