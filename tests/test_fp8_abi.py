"""C ABI checks of the E4M3 operators (include/mswz_fp8.h) and of the layer of
experts (include/mswz_moe_layer.h) that need no GPU: the headers' functions are
exported, and everything they refuse is refused on the host, before any GPU
work (fake, never-dereferenced pointer values are enough to reach the checks)."""
import ctypes
import os
import re

import pytest
import torch

import mma_swizzled_operand_amd as mswz

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F16, BF16, E4M3, F32, E2M1 = 1, 2, 3, 4, 5
ROW, TILE = 0, 1
P = 0x10000   # an aligned address that no refused call reads


@pytest.mark.parametrize("header,count", [("mswz_fp8.h", 7), ("mswz_moe_layer.h", 4)])
def test_library_exports_every_declared_symbol(header, count):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*[A-Za-z_][A-Za-z0-9_]*\s*\**\s*([a-z_][a-z0-9_]*)\s*\(", text, flags=re.M)))
    assert len(names) == count
    lib = ctypes.CDLL(mswz.library_path())
    for name in names:
        assert hasattr(lib, name), name
        assert hasattr(mswz.load(), name)


def create(name, *args):
    lib, h = mswz.load(), ctypes.c_void_p(1)
    rc = getattr(lib, name + "_create")(ctypes.byref(h), *args)
    if rc == 0:
        return rc, h
    assert not h.value
    return rc, None


@pytest.mark.parametrize("args,expect", [
    ((1, 1, 16, BF16, TILE, 0, 0, 0), 0),
    ((333, 1003, 2064, F32, ROW, 2080, 4096, 1004), 0),
    ((1 << 20, 64, 128, F16, TILE, 0, 0, 0), 0),
    ((0, 16, 128, BF16, TILE, 0, 0, 0), -1),
    ((1, -4, 128, BF16, TILE, 0, 0, 0), -1),
    ((1, 16, (1 << 20) + 16, BF16, TILE, 0, 0, 0), -1),
    ((1, 16, 128, 9, TILE, 0, 0, 0), -1),                 # no such dtype
    ((1, 16, 128, BF16, 2, 0, 0, 0), -1),
    ((1, 16, 128, BF16, TILE, 112, 0, 0), -1),            # pitches below a row
    ((1, 16, 128, BF16, TILE, 0, 112, 0), -1),
    ((1, 16, 128, BF16, TILE, 0, 0, 15), -1),
    ((1, 16, 128, BF16, TILE, 0, -128, 0), -1),
    ((1, 16, 136, BF16, TILE, 0, 0, 0), -2),              # rows not 16-byte pieces
    ((1, 16, 128, BF16, TILE, 136, 0, 0), -2),
    ((1, 16, 128, BF16, TILE, 0, 136, 0), -2),
    ((1, 16, 128, BF16, TILE, 0, (1 << 22) + 16, 0), -2),
    ((1, 16, 128, BF16, TILE, 0, 0, (1 << 22) + 1), -2),
    ((1, 16, 128, E4M3, TILE, 0, 0, 0), -2),
    ((1, 16, 128, E2M1, ROW, 0, 0, 0), -2),
    ((1 << 20, 64, 1 << 18, BF16, TILE, 0, 0, 0), -2),    # 8 GiB of scales
    ((64, 1 << 20, 1 << 18, BF16, ROW, 0, 0, 0), -2),
    ((1 << 20, 1 << 20, 128, BF16, TILE, 0, 0, 0), -2),   # too many tiles
])
def test_gemm_plan(args, expect):
    rc, h = create("gemm_fp8_plan", *args)
    assert rc == expect
    if h:
        assert mswz.load().gemm_fp8_plan_workspace_size(h) >= 0
        mswz.load().gemm_fp8_plan_destroy(h)


def test_gemm_run():
    lib = mswz.load()
    rc, h = create("gemm_fp8_plan", 1, 4096, 4096, BF16, TILE, 0, 0, 0)
    assert rc == 0
    need = lib.gemm_fp8_plan_workspace_size(h)
    good = [h, P, P, P, P, P, 0, P, max(need, 16), None]
    for at in (0, 1, 2, 3, 4, 5):
        args = list(good)
        args[at] = None
        assert lib.gemm_run_fp8(*args) == -1
    for at, value in ((6, 2), (6, -1)):
        args = list(good)
        args[at] = value
        assert lib.gemm_run_fp8(*args) == -1
    if need:
        assert lib.gemm_run_fp8(*good[:7], None, need, None) == -1
        assert lib.gemm_run_fp8(*good[:8], need - 1, None) == -1
        assert lib.gemm_run_fp8(*good[:7], P + 8, need, None) == -3
    for at, off in ((1, 8), (2, 2), (3, 4), (4, 1), (5, 1)):
        args = list(good)
        args[at] = P + off
        assert lib.gemm_run_fp8(*args) == -3
    assert lib.gemm_fp8_plan_create(None, 1, 1, 16, BF16, TILE, 0, 0, 0) == -1
    assert lib.gemm_fp8_plan_workspace_size(None) == -1
    lib.gemm_fp8_plan_destroy(h)
    lib.gemm_fp8_plan_destroy(None)


@pytest.mark.parametrize("args,expect", [
    ((1, 16, F16, ROW, 0, 0), 0),
    ((16384, 4096, F32, TILE, 1, 4104), 0),
    ((0, 16, F16, ROW, 0, 0), -1),
    ((16, 0, F16, ROW, 0, 0), -1),
    ((16, 16, 99, ROW, 0, 0), -1),
    ((16, 16, F16, 2, 0, 0), -1),
    ((16, 16, F16, ROW, 2, 0), -1),
    ((16, 32, F16, ROW, 0, 24), -1),
    ((16, 32, F16, ROW, 0, -32), -1),
    ((16, 24, F16, ROW, 0, 0), -2),
    ((16, 32, E4M3, ROW, 0, 0), -2),
    ((16, 32, BF16, ROW, 0, 36), -2),
    ((16, 32, BF16, ROW, 0, (1 << 22) + 8), -2),
    ((1 << 20, 1 << 20, BF16, ROW, 0, 0), -2),
])
def test_quant_plan(args, expect):
    rc, h = create("quant_fp8_plan", *args)
    assert rc == expect
    if h:
        mswz.load().quant_fp8_plan_destroy(h)


def test_quant_run():
    lib = mswz.load()
    rc, h = create("quant_fp8_plan", 16, 32, BF16, ROW, 0, 0)
    assert rc == 0
    for args in ((None, P, P, P, P, P), (h, None, P, P, P, P), (h, P, None, P, P, P), (h, P, P, None, P, P),
                 (h, P, P, P, None, P), (h, P, P, P, P, None), (h, P, None, None, None, None)):
        assert lib.quant_fp8(*args, None) == -1
    for args in ((P + 8, P, P, P, P), (P, P + 8, P, P, P), (P, P, P + 2, P, P), (P, P, P, P + 4, P), (P, P, P, P, P + 1)):
        assert lib.quant_fp8(h, *args, None) == -3
    assert lib.quant_fp8_plan_create(None, 16, 32, BF16, ROW, 0, 0) == -1
    lib.quant_fp8_plan_destroy(h)
    lib.quant_fp8_plan_destroy(None)


@pytest.mark.parametrize("args,expect", [
    ((1, 1, 1, 8, 8, F16, F16, 0, 0), 0),
    ((128, 8, 1024, 4096, 2048, BF16, E4M3, 1, 4104), 0),
    ((0, 1, 1, 8, 8, F16, F16, 0, 0), -1),
    ((1, 0, 1, 8, 8, F16, F16, 0, 0), -1),
    ((1, 1, 0, 8, 8, F16, F16, 0, 0), -1),
    ((1, 1, 1, -8, 8, F16, F16, 0, 0), -1),
    ((1, 1, 1, 8, 0, F16, F16, 0, 0), -1),
    ((1, 1, 1, 8, 8, 17, F16, 0, 0), -1),
    ((1, 1, 1, 8, 8, F16, 17, 0, 0), -1),
    ((1, 1, 1, 8, 8, F16, F16, 2, 0), -1),
    ((1, 1, 1, 16, 8, F16, F16, 0, 8), -1),
    ((129, 8, 16, 64, 64, F16, F16, 0, 0), -2),           # more than 1024 choices
    ((1 << 40, 1 << 40, 16, 64, 64, F16, F16, 0, 0), -2),
    ((1, 1, 1025, 8, 8, F16, F16, 0, 0), -2),
    ((1, 1, 1, 8, 8, F32, F32, 0, 0), -2),
    ((1, 1, 1, 8, 8, F16, BF16, 0, 0), -2),
    ((1, 1, 1, 8, 8, F16, E2M1, 0, 0), -2),
    ((1, 1, 1, 12, 8, F16, F16, 0, 0), -2),
    ((1, 1, 1, 8, 12, F16, F16, 0, 0), -2),
    ((1, 1, 1, 24, 16, F16, E4M3, 0, 0), -2),
    ((1, 1, 1, 16, 24, F16, E4M3, 0, 0), -2),
    ((1, 1, 1, 16, 16, F16, F16, 0, 20), -2),
    ((1, 1, 1, 1 << 16, 1 << 14, F16, F16, 0, 0), -2),    # an expert's W1 of 4 GiB
    ((1024, 1, 1, 8, 1 << 20, F16, F16, 0, 0), -2),       # 4 GiB between the products
])
def test_layer_plan(args, expect):
    rc, h = create("moe_layer_plan", *args)
    assert rc == expect
    if h:
        assert mswz.load().moe_layer_plan_workspace_size(h) > 0
        mswz.load().moe_layer_plan_destroy(h)


def test_layer_run():
    lib = mswz.load()
    for w_dt in (BF16, E4M3):
        rc, h = create("moe_layer_plan", 4, 2, 8, 64, 128, BF16, w_dt, 0, 0)
        assert rc == 0
        s = P if w_dt == E4M3 else None
        need = lib.moe_layer_plan_workspace_size(h)
        good = [h, P, P, P, P, s, P, s, P, P, need, None]
        for at in (0, 1, 2, 3, 4, 6, 8, 9):
            args = list(good)
            args[at] = None
            assert lib.moe_layer(*args) == -1, at
        for at in (5, 7):   # scales are given exactly for E4M3
            args = list(good)
            args[at] = None if s else P
            assert lib.moe_layer(*args) == -1
        args = list(good)
        args[10] = need - 1
        assert lib.moe_layer(*args) == -1
        for at, off in ((1, 8), (2, 2), (3, 1), (4, 8), (6, 2), (8, 8), (9, 8)):
            args = list(good)
            args[at] = P + off
            assert lib.moe_layer(*args) == -3, at
        if s:
            for at in (5, 7):
                args = list(good)
                args[at] = P + 2
                assert lib.moe_layer(*args) == -3
        lib.moe_layer_plan_destroy(h)
    assert lib.moe_layer_plan_create(None, 1, 1, 1, 8, 8, F16, F16, 0, 0) == -1
    assert lib.moe_layer_plan_workspace_size(None) == -1
    lib.moe_layer_plan_destroy(None)


def test_binding_refuses_before_any_call():
    with pytest.raises(mswz.MswzError):
        mswz.gemm_fp8_plan_create(1, 16, 136)
    with pytest.raises(mswz.MswzError):
        mswz.gemm_fp8_plan_create(1 << 64, 16, 128)      # wider than the argument
    with pytest.raises(ValueError):
        mswz.gemm_fp8_plan_create(1, 16, 128, b_block="column")
    with pytest.raises(ValueError):
        mswz.gemm_fp8_plan_create(1, 16, 128, d_dt="f64")
    with pytest.raises(ValueError):
        mswz.quant_fp8_plan_create(1, 16, scales="log")
    with pytest.raises(ValueError):
        mswz.moe_layer_plan_create(1, 1, 1, 8, 8, act="relu")
    x = torch.zeros(1, 128, dtype=torch.uint8)
    s = torch.zeros(1)
    gemm = mswz.gemm_fp8_plan_create(1, 16, 128)
    with pytest.raises(ValueError):                       # host tensors
        mswz.gemm_run_fp8(gemm, x, s, x, s, x)
    with pytest.raises(TypeError):
        mswz.gemm_run_fp8(gemm, 1, s, x, s, x)
    quant = mswz.quant_fp8_plan_create(1, 128)
    with pytest.raises(TypeError):                        # another operator's plan
        mswz.gemm_run_fp8(quant, x, s, x, s, x)
    with pytest.raises(ValueError):
        mswz.quant_fp8(quant, x, Q=x, S=s)
    layer = mswz.moe_layer_plan_create(1, 1, 1, 128, 128)
    with pytest.raises(ValueError):
        mswz.moe_layer(layer, x, s, s, x, x, x)
    layer.destroy()
    with pytest.raises(ValueError):
        mswz.moe_layer(layer, x, s, s, x, x, x)
