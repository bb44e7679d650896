"""The forms of the integer products that the sizes of test_gpu_int8.py do not reach, against the same exact sums; rows of
x that hold an infinity or a NaN, one at a time, in every form that rounds x itself.

FORMS is what test_int8_forms_cpu.py adds to those sizes to have every kernel that a call can launch."""
import pytest
import torch

import test_gpu_int8 as base
from gpu_util import nw, step

pytestmark = pytest.mark.gpu

# Up to four rows of x, a wave holding two chunks of 1024 columns (9 to 16 in a row of W) or three (17 to 48): whole
# chunks and rows of W that end inside one, odd numbers of them (the last wave has one less), so many rows of W that a
# workgroup takes several groups, and numbers of rows that end inside a group.  Then gated 256x128 tiles.
FORMS = [(1, 4099, 11008), (1, 301, 8320), (1, 4096, 14336), (1, 5, 8193), (1, 3001, 16384), (1, 77, 16385),
         (2, 301, 9001), (2, 515, 14336), (2, 1501, 12300), (2, 3, 8193), (2, 130, 20008), (2, 77, 49152), (2, 1101, 22016),
         (2, 9, 16385), (3, 301, 9001), (3, 77, 24001), (4, 50, 49152), (4, 1030, 17000), (4, 901, 16384),
         (1000, 4001, 260), (747, 5003, 1300)]


@pytest.mark.parametrize("batch,rows,cols", FORMS)
def test_gemm(batch, rows, cols):
    base.test_gemm(batch, rows, cols)


@pytest.mark.parametrize("batch,rows,cols", FORMS)
def test_glu(batch, rows, cols):
    base.test_glu(batch, rows, cols)


@pytest.mark.parametrize("batch,cols", [(2, 600), (3, 150), (4, 8000), (4, 8192), (2, 9001), (2, 16384), (2, 17001),
                                        (2, 40000), (3, 9001), (4, 20008), (5, 700), (17, 700)])
def test_a_bad_row_leaves_the_others(batch, cols):
    """One row of x with an infinity or a NaN, first, inside or last: its products are NaN, all others have the bits
    that they have without it."""
    step(f"int8 one bad row batch {batch} cols {cols}")
    rows = 133
    (q, scale), (u, us) = base.codes(rows, cols, 8), base.codes(rows, cols, 9)
    x = base.acts(batch, cols, 9)
    y, h = nw().int8_gemm(q, scale, x), nw().int8_glu(q, scale, u, us, x)
    assert not y.isnan().any() and not h.isnan().any()
    values = [float("inf"), float("-inf"), float("nan")]
    for bad in range(min(batch, 5)):
        for k, value in enumerate(values):
            other = x.clone()
            other[bad, (0, cols // 2, cols - 1)[(bad + k) % 3]] = value
            rest = [b for b in range(batch) if b != bad]
            for got, want in ((nw().int8_gemm(q, scale, other), y), (nw().int8_glu(q, scale, u, us, other), h)):
                assert got[bad].isnan().all() and torch.equal(got[rest], want[rest])
