"""The forms of the integer products that the sizes of test_gpu_int8.py do not reach, against the same exact sums.

FORMS is what test_int8_forms_cpu.py adds to those sizes to have every kernel that a call can launch."""
import pytest

import test_gpu_int8 as base
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
