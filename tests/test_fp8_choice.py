"""Which kernel a product of E4M3 operands takes (csrc/fp8_choice.hpp), asked
on the host: the shapes of tests/test_gpu_fp8_stores.py reach the kernels that
they are named after, and every kernel there is.  (A choice that moves away from
under them fails here.)"""
import ctypes
import os

import pytest

import test_gpu_fp8_stores as shapes

LIB = os.path.join(os.path.dirname(os.path.abspath(__file__)), "probes", "libprobes.so")
KERNELS = ["few", "split", "32x64", "64x64", "128x64", "128x128", "128x128 twice", "256x256"]   # Fp8Kernel's order
KINDS = {"f32": 0, "bf16": 1, "f16": 2}


@pytest.fixture(scope="module")
def kernel_of():
    if not os.path.exists(LIB):
        raise RuntimeError(f"{LIB} is missing: run __graft_entry__.build()")
    h = ctypes.CDLL(LIB)
    h.probe_fp8_kernel.argtypes = [ctypes.c_int] * 4 + [ctypes.c_int64] * 2
    return lambda M, N, K, d, lda=0, ldb=0: KERNELS[h.probe_fp8_kernel(M, N, K, KINDS[d], lda or K, ldb or K)]


@pytest.mark.parametrize("kernel,d", shapes.CASES)
def test_shapes_reach_the_kernel_they_name(kernel_of, kernel, d):
    M, N, K = shapes.shape_of(kernel, d)
    for more in range(5):
        assert kernel_of(M, N + more, K, d) == (kernel if kernel in KERNELS else "few")
    if kernel in ("few16", "few32"):    # one tile of 16 rows, and two
        assert M <= 16 if kernel == "few16" else 16 < M <= 32


def test_every_kernel_has_a_shape():
    reached = {(k if k in KERNELS else "few", d) for k, d in shapes.CASES}
    assert reached == {(k, d) for k in KERNELS for d in KINDS} - {("256x256", "f32")}   # (no registers for it)
    assert {(k, d) for k in ("few16", "few32") for d in KINDS} <= set(shapes.CASES)


@pytest.mark.parametrize("M,N,K,d,kernel", [
    (1, 4096, 4096, "bf16", "few"), (16, 4096, 4096, "bf16", "few"), (16, 4160, 4096, "bf16", "32x64"),
    (16, 8192, 4096, "f32", "few"), (16, 8256, 4096, "f32", "32x64"), (32, 4096, 4096, "bf16", "few"),
    (33, 4096, 4096, "bf16", "32x64"), (32, 4096, 6144, "bf16", "split"), (16, 4096, 6144, "bf16", "few"),
    (128, 4096, 6016, "bf16", "32x64"), (128, 4096, 6144, "bf16", "split"), (129, 4096, 6144, "bf16", "64x64"),
    (64, 16384, 8192, "bf16", "64x64"), (333, 1003, 2064, "f32", "32x64"), (1024, 4096, 4096, "bf16", "128x128"),
    (2048, 4096, 4096, "bf16", "128x128 twice"), (8192, 8192, 8192, "bf16", "256x256"),
    (8192, 8192, 8192, "f32", "128x128 twice"), (22, 1185, 560, "f32", "few"), (105, 14480, 3520, "f32", "128x64"),
    (1017, 1304, 2848, "bf16", "128x64"),
])
def test_choice(kernel_of, M, N, K, d, kernel):
    """Both sides of the rules' limits, and ordinary sizes."""
    assert kernel_of(M, N, K, d) == kernel


def test_rows_that_are_not_whole_lines_count(kernel_of):
    """A pitch of A or of B that is no multiple of 128 makes a step longer, that of small tiles most."""
    assert kernel_of(400, 4096, 1024, "bf16") == "64x64"
    for pitches in ((1040, 1024), (1024, 1040), (1040, 1040)):
        assert kernel_of(400, 4096, 1024, "bf16", *pitches) == "128x64"
