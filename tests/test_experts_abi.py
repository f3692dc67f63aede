"""C ABI checks of the expert operators that need no GPU: the header's
functions are exported, and everything include/mswz_experts.h refuses is
refused on the host, before any GPU work (fake, never-dereferenced pointer
values are enough to reach the checks)."""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

import mma_swizzled_operand_amd as mswz

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mswz_experts.h")
F16, BF16, E4M3, F32, E2M1, U4 = 1, 2, 3, 4, 5, 9
K_, MN = 0, 1
P = 0x10000   # an aligned address that no refused call reads


def declared_functions():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^\s*[A-Za-z_][A-Za-z0-9_]*\s*\**\s*([a-z_][a-z0-9_]*)\s*\(", text, flags=re.M)))


def test_library_exports_every_declared_symbol():
    names = declared_functions()
    assert len(names) == 13
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
    ((1, 1000, 1024, 0, BF16, U4, BF16, 128, 0, 0), 0),
    ((65536, 7, 32, 0, F16, U4, F32, 32, 0, 0), 0),
    ((5, 16, 1056, 1024, F16, E2M1, F16, 32, 2048, 24), 0),
    ((1, 16, 1024, 0, BF16, U4, F32, 2048, 0, 0), 0),          # one scale per row
    ((0, 16, 1024, 0, BF16, U4, BF16, 128, 0, 0), -1),
    ((1, -1, 1024, 0, BF16, U4, BF16, 128, 0, 0), -1),
    ((1, 16, 1024, -1, BF16, U4, BF16, 128, 0, 0), -1),
    ((1, 16, 1024, 0, BF16, 10, BF16, 128, 0, 0), -1),         # no such dtype
    ((1, 16, 1024, 0, BF16, U4, BF16, 0, 0, 0), -1),
    ((1, 16, 1024, 0, BF16, U4, BF16, 128, 1016, 0), -1),      # pitch below a row
    ((1, 16, 1024, 0, BF16, U4, BF16, 128, 0, 15), -1),
    ((65537, 16, 1024, 0, BF16, U4, BF16, 128, 0, 0), -2),
    ((1, 16, 1040, 0, BF16, U4, BF16, 128, 0, 0), -2),         # K % 32
    ((1, 16, 1024, 0, BF16, U4, BF16, 96, 0, 0), -2),
    ((1, 16, 1024, 0, BF16, E2M1, BF16, 64, 0, 0), -2),
    ((1, 16, 1024, 0, BF16, E4M3, BF16, 32, 0, 0), -2),
    ((1, 16, 1024, 0, F32, U4, F32, 128, 0, 0), -2),
    ((1, 16, 1024, 0, BF16, U4, F16, 128, 0, 0), -2),
    ((1, 16, 1024, 1025, BF16, U4, BF16, 128, 0, 0), -2),
    ((1, 16, 1024, 0, BF16, U4, BF16, 128, 1028, 0), -2),      # rows of A not 16-byte aligned
    ((1, 1 << 20, 1 << 14, 0, BF16, U4, BF16, 128, 0, 0), -2),  # 8 GiB of weights
])
def test_w4_plan(args, expect):
    rc, h = create("gemm_w4_plan", *args)
    assert rc == expect
    if h:
        assert mswz.load().gemm_w4_plan_workspace_size(h) >= 0
        mswz.load().gemm_w4_plan_destroy(h)


@pytest.mark.parametrize("args,expect", [
    ((8, 100, 264, 520, F16, F16, 0, K_), 0),
    ((1024, 1, 8, 8, BF16, F32, 0, MN), 0),
    ((8, 264, 520, 100, BF16, F32, 1, MN), 0),
    ((0, 100, 264, 520, F16, F16, 0, K_), -1),
    ((8, 0, 264, 520, F16, F16, 0, K_), -1),
    ((8, 100, 264, 520, 0, F16, 0, K_), -1),
    ((8, 100, 264, 520, F16, F16, 2, K_), -1),
    ((8, 100, 264, 520, F16, F16, 0, 2), -1),
    ((1025, 100, 264, 520, F16, F16, 0, K_), -2),
    ((8, 100, 264, 520, E4M3, F32, 0, K_), -2),
    ((8, 100, 264, 520, F16, BF16, 0, K_), -2),
    ((8, 264, 520, 100, BF16, F32, 1, K_), -2),                # along K both operands are MN-major
    ((8, 100, 260, 520, F16, F16, 0, K_), -2),                 # N % 8
    ((8, 100, 264, 516, F16, F16, 0, K_), -2),                 # K % 8
    ((8, 260, 520, 100, BF16, F32, 1, MN), -2),                # M % 8
    ((8, 100, 1 << 18, 1 << 14, F16, F16, 0, MN), -2),         # a [K][N] of 8 GiB
])
def test_grouped_plan(args, expect):
    rc, h = create("gemm_grouped_plan", *args)
    assert rc == expect
    if h:
        mswz.load().gemm_grouped_plan_destroy(h)


@pytest.mark.parametrize("args,expect", [
    ((7, 2, 8, 1024, F16, 0), 0),
    ((1, 1, 1, 4, F32, 8), 0),
    ((1 << 20, 8, 1024, 64, BF16, 128), 0),
    ((0, 2, 8, 1024, F16, 0), -1),
    ((7, 0, 8, 1024, F16, 0), -1),
    ((7, 2, 0, 1024, F16, 0), -1),
    ((7, 2, 8, 0, F16, 0), -1),
    ((7, 2, 8, 1024, F16, 1016), -1),
    ((7, 2, 8, 1024, 0, 0), -1),
    ((1 << 22, 4, 8, 1024, F16, 0), -2),                       # 2^24 choices
    ((1 << 40, 1 << 30, 8, 1024, F16, 0), -2),
    ((7, 2, 1025, 1024, F16, 0), -2),
    ((7, 2, 8, 1028, F16, 0), -2),                             # rows not whole 16-byte pieces
    ((7, 2, 8, 1022, F32, 0), -2),
    ((7, 2, 8, 1024, F16, 1028), -2),
    ((7, 2, 8, 1024, E4M3, 0), -2),
])
def test_moe_plan(args, expect):
    rc, h = create("moe_plan", *args)
    assert rc == expect
    if h:
        assert mswz.load().moe_plan_workspace_size(h) >= 0
        mswz.load().moe_plan_destroy(h)


def test_grouped_plan_beyond_a_launch():
    """512 threads for every tile of 256 x 256: 2^23 of them are one launch too many."""
    tiles = (1 << 23) - 256
    most = (tiles // 4096 - 8) * 256 + 255   # rows of 8 experts, 4096 tiles side by side
    assert create("gemm_grouped_plan", 8, most, 1 << 20, 264, F16, F16, 0, K_)[0] == 0
    assert create("gemm_grouped_plan", 8, most + 1, 1 << 20, 264, F16, F16, 0, K_)[0] == -2
    # along K every expert has all the tiles of its matrix
    assert create("gemm_grouped_plan", 15, 1 << 18, 1 << 17, 8, BF16, F32, 1, MN)[0] == 0
    assert create("gemm_grouped_plan", 16, 1 << 18, 1 << 17, 8, BF16, F32, 1, MN)[0] == -2


def test_null_plans_and_out_pointers():
    lib = mswz.load()
    assert lib.gemm_w4_plan_create(None, 1, 16, 1024, 0, BF16, U4, BF16, 128, 0, 0) == -1
    assert lib.gemm_grouped_plan_create(None, 8, 100, 264, 520, F16, F16, 0, K_) == -1
    assert lib.moe_plan_create(None, 7, 2, 8, 1024, F16, 0) == -1
    assert lib.gemm_w4_plan_workspace_size(None) == -1 and lib.moe_plan_workspace_size(None) == -1
    for name in ("gemm_w4_plan", "gemm_grouped_plan", "moe_plan"):
        getattr(lib, name + "_destroy")(None)


def refusals(fn, good, cases):
    """Each case replaces arguments of a good call, by index, with ones that are refused."""
    for change, expect in cases:
        args = list(good)
        for i, v in change.items():
            args[i] = v
        assert fn(*args) == expect, change


def test_w4_run_refusals():
    lib = mswz.load()
    big = 1 << 40
    for E, w in ((0, U4), (4, U4), (0, E2M1)):
        rc, h = create("gemm_w4_plan", 3, 16, 64, E, BF16, w, BF16, 32, 0, 0)
        assert rc == 0
        good = [h, P, P, P, P if w == U4 else None, P if E else None, P, 0, P, big, None]
        refusals(lib.gemm_run_w4, good, [
            ({0: None}, -1), ({1: None}, -1), ({2: None}, -1), ({3: None}, -1), ({6: None}, -1),
            ({5: None if E else P}, -1), ({7: 2}, -1), ({7: -1}, -1),
            ({1: P + 8}, -3), ({2: P + 8}, -3), ({6: P + 1}, -3)])
        if w == U4:
            refusals(lib.gemm_run_w4, good, [({3: P + 1}, -3)])
        else:
            refusals(lib.gemm_run_w4, good, [({4: P}, -1)])
        if E:
            refusals(lib.gemm_run_w4, good, [({5: P + 2}, -3)])
        if lib.gemm_w4_plan_workspace_size(h):
            refusals(lib.gemm_run_w4, good, [({8: None}, -1), ({9: 0}, -1), ({8: P + 4}, -3)])
        lib.gemm_w4_plan_destroy(h)


def test_grouped_run_refusals():
    lib = mswz.load()
    _, h = create("gemm_grouped_plan", 8, 100, 264, 520, F16, F16, 0, K_)
    refusals(lib.gemm_run_grouped, [h, P, P, P, P, 0, None], [
        ({0: None}, -1), ({1: None}, -1), ({2: None}, -1), ({3: None}, -1), ({4: None}, -1), ({5: 2}, -1),
        ({1: P + 8}, -3), ({2: P + 8}, -3), ({3: P + 2}, -3), ({4: P + 8}, -3)])
    lib.gemm_grouped_plan_destroy(h)


def test_moe_run_refusals():
    lib = mswz.load()
    big = 1 << 40
    for T in (3, 5000):
        _, h = create("moe_plan", T, 2, 8, 64, F16, 0)
        good = [h, P, P, P, P, P, P, P, big, None]
        refusals(lib.moe_dispatch, good, [
            ({0: None}, -1), ({1: None}, -1), ({2: None}, -1), ({3: None}, -1), ({4: None}, -1), ({5: None}, -1),
            ({6: None}, -1), ({1: P + 2}, -3), ({2: P + 8}, -3), ({3: P + 8}, -3), ({4: P + 2}, -3), ({5: P + 2}, -3),
            ({6: P + 2}, -3)])
        if lib.moe_plan_workspace_size(h):
            refusals(lib.moe_dispatch, good, [({7: None}, -1), ({8: 3}, -1), ({7: P + 4}, -3)])
        refusals(lib.moe_combine, [h, P, P, P, P, None], [
            ({0: None}, -1), ({1: None}, -1), ({2: None}, -1), ({4: None}, -1), ({1: P + 8}, -3), ({2: P + 2}, -3),
            ({3: P + 2}, -3), ({4: P + 8}, -3)])
        refusals(lib.moe_combine_grad, [h, P, P, P, P, P, P, None],
                 [({i: None}, -1) for i in range(7)] +
                 [({1: P + 8}, -3), ({2: P + 8}, -3), ({3: P + 2}, -3), ({4: P + 2}, -3), ({5: P + 8}, -3), ({6: P + 2}, -3)])
        lib.moe_plan_destroy(h)


def test_binding_refusals():
    with pytest.raises(ValueError):
        mswz.gemm_w4_plan_create(1, 16, 64, w_dt="u5")
    with pytest.raises(ValueError):
        mswz.gemm_grouped_plan_create(2, 8, 8, 8, axis="n")
    with pytest.raises(ValueError):
        mswz.moe_plan_create(1, 1, 1, 8, dt="half")
    with pytest.raises(mswz.MswzError):
        mswz.gemm_w4_plan_create(1, 16, 63)
    plan = mswz.moe_plan_create(2, 2, 4, 8, "f32")
    with pytest.raises(TypeError):   # another operator's plan
        mswz.gemm_run_grouped(plan, torch.zeros(1), torch.zeros(1), torch.zeros(1), torch.zeros(1))
    with pytest.raises(ValueError):  # not in GPU memory
        mswz.moe_combine(plan, torch.zeros(4, 8), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 8))
    plan.destroy()
    with pytest.raises(ValueError):
        plan.handle


@pytest.mark.parametrize("make", [
    lambda wide: mswz.gemm_w4_plan_create(4, 16, 256, group=128 + (wide << 32)),
    lambda wide: mswz.gemm_w4_plan_create(4 + (wide << 64), 16, 256),
    lambda wide: mswz.gemm_grouped_plan_create(2, 64, 64, 64 + (wide << 64)),
    lambda wide: mswz.moe_plan_create(4, 2, 8, 64, ldx=64 + (wide << 64)),
])
def test_numbers_wider_than_the_argument_are_refused(make):
    make(0)
    for wide in (1, -1):
        with pytest.raises(mswz.MswzError):
            make(wide)


def test_package_and_plans_work_without_torch():
    """torch supplies memory and streams to the run calls; nothing before them asks for it."""
    code = """
import sys
sys.modules["torch"] = None    # importing it raises
import mma_swizzled_operand_amd as mswz
assert mswz.tile_offset(3, 1) >= 0 and mswz.desc_check(16, 1024, 2) is not None
assert mswz.gemm_plan_create(256, 256, 64, "bf16", "bf16").describe()["tile_m"] > 0
assert mswz.gemm_w4_plan_create(64, 300, 8192).workspace_bytes() > 0
assert mswz.gemm_grouped_plan_create(2, 64, 64, 64).d_numel == 64 * 64
assert mswz.moe_plan_create(5000, 2, 8, 64).workspace_bytes() > 0
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_types_of_a_plan():
    w4 = mswz.gemm_w4_plan_create(1, 16, 64, "f16", "u4", "f32", group=64)
    assert (w4.a_type, w4.s_type, w4.d_type) == (torch.float16, torch.float16, torch.float32)
    assert mswz.gemm_w4_plan_create(1, 16, 64, "bf16", "e2m1", "bf16", group=32).s_type is torch.uint8
    grouped = mswz.gemm_grouped_plan_create(2, 64, 64, 64, "bf16", "f32")
    assert (grouped.type, grouped.d_type) == (torch.bfloat16, torch.float32)
    assert mswz.moe_plan_create(1, 1, 1, 8, "f16").type is torch.float16
