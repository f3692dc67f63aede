"""Binding of the E4M3 operators (include/mswz_fp8.h): products of operands with
an fp32 scale per block of 128 values, and the quantisation that makes them.
Names and arguments are the C ABI's; tensors, streams and errors as in
experts.py.  E4M3 tensors are torch.float8_e4m3fn or uint8.

    rows, tiles = quant_fp8_plan_create(M, K, "bf16", "row"), quant_fp8_plan_create(N, K, "bf16", "tile")
    quant_fp8(rows, X, Q=Xq, S=SX)
    quant_fp8(tiles, W, Q=Wq, S=SW, QT=Wt, ST=SWt)            # W^T for the gradient of X
    plan = gemm_fp8_plan_create(M, N, K, "bf16", "tile")
    gemm_run_fp8(plan, Xq, SX, Wq, SW, Y, workspace=workspace)   # Y = X . W^T
"""
from __future__ import annotations

from . import experts as _x

__all__ = ["Fp8Plan", "QuantPlan", "gemm_fp8_plan_create", "gemm_run_fp8", "quant_fp8_plan_create", "quant_fp8"]

_BLOCKS = {"row": 0, "tile": 1}
_SCALES = {"f32": 0, "pow2": 1}


def declare(h):
    """Argument types of the library's functions (called once when it is loaded)."""
    import ctypes
    i64, vp, c_int = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    out = ctypes.POINTER(vp)
    for name, args, res in (
            ("gemm_fp8_plan_create", [out, i64, i64, i64, c_int, c_int, i64, i64, i64], c_int),
            ("gemm_fp8_plan_destroy", [vp], None),
            ("gemm_fp8_plan_workspace_size", [vp], i64),
            ("gemm_run_fp8", [vp, vp, vp, vp, vp, vp, c_int, vp, i64, vp], c_int),
            ("quant_fp8_plan_create", [out, i64, i64, c_int, c_int, c_int, i64], c_int),
            ("quant_fp8_plan_destroy", [vp], None),
            ("quant_fp8", [vp, vp, vp, vp, vp, vp, vp], c_int)):
        f = getattr(h, name)
        f.argtypes, f.restype = args, res


def _blocks(n):
    return -(-n // 128)


class Fp8Plan(_x._Plan):
    """A product of E4M3 operands with a scale per block of 128 (gemm_fp8_plan_create)."""
    _make, _free = "gemm_fp8_plan_create", "gemm_fp8_plan_destroy"
    d_type = _x._type("d_dt")

    def __init__(self, M, N, K, d_dt="bf16", b_block="tile", lda=0, ldb=0, ldd=0):
        self.M, self.N, self.K = int(M), int(N), int(K)
        self._create(self.M, self.N, self.K, _x._dt(d_dt), _x._pick(_BLOCKS, b_block, "block"), int(lda), int(ldb),
                     int(ldd))
        self.d_dt, self.b_block = d_dt, b_block
        self.lda, self.ldb, self.ldd = int(lda) or self.K, int(ldb) or self.K, int(ldd) or self.N
        kb = _blocks(self.K)
        self.sa_numel = kb * self.M
        self.sb_numel = kb * (_blocks(self.N) if b_block == "tile" else self.N)
        self.ws_bytes, self._run = int(self._lib.gemm_fp8_plan_workspace_size(self._h)), self._lib.gemm_run_fp8

    def workspace_bytes(self) -> int:
        """Device workspace gemm_run_fp8 needs for this plan (0: none)."""
        return self.ws_bytes


class QuantPlan(_x._Plan):
    """The quantisation of a matrix to E4M3 with a scale per block of 128 (quant_fp8_plan_create)."""
    _make, _free = "quant_fp8_plan_create", "quant_fp8_plan_destroy"
    type = _x._type("dt")

    def __init__(self, M, K, dt="bf16", block="row", scales="f32", ldx=0):
        self.M, self.K = int(M), int(K)
        self._create(self.M, self.K, _x._dt(dt), _x._pick(_BLOCKS, block, "block"), _x._pick(_SCALES, scales, "scales"),
                     int(ldx))
        self.dt, self.block, self.scales, self.ldx = dt, block, scales, int(ldx) or self.K
        self.mp = -(-self.M // 16) * 16     # elements of a row of QT
        tiles = _blocks(self.M) * _blocks(self.K)
        self.s_numel = tiles if block == "tile" else _blocks(self.K) * self.M
        self.st_numel = tiles if block == "tile" else _blocks(self.M) * self.K
        self._run = self._lib.quant_fp8


def gemm_fp8_plan_create(M, N, K, d_dt="bf16", b_block="tile", lda=0, ldb=0, ldd=0) -> Fp8Plan:
    """Plan of D = beta*D + A . B^T, both E4M3 with a scale per block of 128 along K (b_block "tile": B's scales
    per 128 x 128 tile)."""
    return Fp8Plan(M, N, K, d_dt, b_block, lda, ldb, ldd)


def quant_fp8_plan_create(M, K, dt="bf16", block="row", scales="f32", ldx=0) -> QuantPlan:
    """Plan of quant_fp8 of a matrix [M][K]."""
    return QuantPlan(M, K, dt, block, scales, ldx)


def _e4m3(t):
    """The type an E4M3 tensor may have: its own if it is one of the two."""
    return t.dtype if t.dtype in (_x.torch.float8_e4m3fn, _x.torch.uint8) else _x.torch.float8_e4m3fn


def gemm_run_fp8(plan: Fp8Plan, A, SA, B, SB, D, beta: int = 0, workspace=None, stream=None) -> None:
    """Enqueue D = beta*D + A . B^T.  SA fp32 [ceil(K/128)][M]; SB fp32 [ceil(K/128)][N], or for plans of "tile"
    [ceil(N/128)][ceil(K/128)]."""
    dev = _x._device(plan, Fp8Plan, A, "A")
    f32 = _x.torch.float32
    _x._call(plan._run, "gemm_run_fp8", dev, stream, plan._h,
             _x._rows(A, _e4m3(A), plan.M, plan.K, plan.lda, dev, "A"), _x._packed(SA, f32, plan.sa_numel, dev, "SA"),
             _x._rows(B, _e4m3(B), plan.N, plan.K, plan.ldb, dev, "B"), _x._packed(SB, f32, plan.sb_numel, dev, "SB"),
             _x._rows(D, plan.d_type, plan.M, plan.N, plan.ldd, dev, "D"), int(beta),
             _x._workspace(workspace, plan.ws_bytes, dev), plan.ws_bytes)


def quant_fp8(plan: QuantPlan, X, Q=None, S=None, QT=None, ST=None, stream=None) -> None:
    """Enqueue the quantisation of X into Q [M][K] with scales S, and of its transpose into QT [K][M rounded up to
    16] with scales ST; either pair may be left out."""
    dev = _x._device(plan, QuantPlan, X, "X")
    if (Q is None) != (S is None) or (QT is None) != (ST is None) or (Q is None and QT is None):
        raise ValueError("Q and S, QT and ST: both or neither of a pair, and one pair at least")
    f32 = _x.torch.float32
    _x._call(plan._run, "quant_fp8", dev, stream, plan._h, _x._rows(X, plan.type, plan.M, plan.K, plan.ldx, dev, "X"),
             None if Q is None else _x._packed(Q, _e4m3(Q), plan.M * plan.K, dev, "Q"),
             None if S is None else _x._packed(S, f32, plan.s_numel, dev, "S"),
             None if QT is None else _x._packed(QT, _e4m3(QT), plan.K * plan.mp, dev, "QT"),
             None if ST is None else _x._packed(ST, f32, plan.st_numel, dev, "ST"))
