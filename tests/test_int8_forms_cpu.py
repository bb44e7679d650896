"""Which kernel each size in the tests of the integer products reaches, by the library's own rule: together they reach
every one that a call can launch, so that a rule that changes shows which of them no size reaches any longer."""
import ctypes

import pytest

import test_gpu_int8
import test_gpu_int8_forms
from non_uniform_weight_amd import int8

SIZES = test_gpu_int8.SHAPES + test_gpu_int8.FEW + test_gpu_int8_forms.FORMS


def kernel(batch, rows, cols, gated, stored):
    p = int8.int8_plan(rows, cols, batch, gated, stored)
    if p["form"] == "vector":
        return gated, "vector", not stored and not p["rounded_first"], p["held"], p["chunks"]
    if p["form"] == "matrix":
        return gated, "matrix", p["blocks"]
    return gated, p["tile"], "split" if p["splits"] > 1 else "halves" if p["whole"] else "whole"


def kernels(gated):
    """Every product kernel of the library: (gated, form, what tells it from the others of its form)."""
    for held in (1, 2, 4):  # x in integers
        for chunks in (1, 2, 3):
            yield gated, "vector", False, held, chunks
    inside = [(1, 1), (1, 2), (1, 3), (2, 1), (2, 2), (4, 1)]  # x in fp16, rounded in the kernel
    for held, chunks in inside if gated else [*inside, (2, 3)]:
        yield gated, "vector", True, held, chunks
    for blocks in (2, 4, 8, 16):
        yield gated, "matrix", blocks
    for tile in int8.TILES:
        yield gated, tile, "whole"
    for tile in ("256x128", "128x128", "128x64", "64x64", "64x32"):
        yield gated, tile, "split"
    yield gated, "256x256", "halves"


@pytest.mark.parametrize("gated", [False, True], ids=["gemm", "glu"])
def test_every_kernel_is_reached(gated):
    reached = {kernel(*size, gated, stored) for size in SIZES for stored in (False, True)}
    assert reached == set(kernels(gated))


@pytest.mark.parametrize("gated", [False, True], ids=["gemm", "glu"])
def test_the_sizes_of_one_form_reach_it(gated):
    """What the comment at FORMS says of its sizes."""
    for batch, rows, cols in test_gpu_int8_forms.FORMS:
        p = int8.int8_plan(rows, cols, batch, gated, True)
        if batch <= 4:
            assert p["form"] == "vector" and p["chunks"] == (2 if cols <= 16384 else 3)
        elif gated:
            assert p == {"rounded_first": False, "form": "tiles", "tile": "256x128", "splits": 1, "whole": 0}


@pytest.mark.parametrize("batch,cols,gemm,glu", [(1, 49152, False, False), (2, 16384, False, False), (2, 16385, False, True),
                                                 (2, 49152, False, True), (3, 8192, False, False), (3, 8193, True, True),
                                                 (4, 8192, False, False), (4, 20000, True, True), (5, 300, True, True)])
def test_where_x_is_rounded(batch, cols, gemm, glu):
    """x in fp16 is rounded in a launch before the product where the kernel that would do it has no registers left."""
    for rows in (1, 300, 20000):
        for gated, first in ((False, gemm), (True, glu)):
            assert int8.int8_plan(rows, cols, batch, gated)["rounded_first"] is first
            assert int8.int8_plan(rows, cols, batch, gated, stored=True)["rounded_first"] is False


def test_plan_argument_errors():
    plan = int8._lib.sqllm_test_int8_plan
    out = (ctypes.c_int * 5)()
    assert plan(64, 300, 3, 0, 0, out) == 0
    assert plan(64, 300, 3, 0, 0, None) == 1
    assert plan(0, 300, 3, 0, 0, out) == plan(64, 131072, 3, 0, 0, out) == plan(64, 300, 0, 0, 0, out) == 3
    assert plan(1 << 20, 300, 1 << 19, 0, 0, out) == 3
