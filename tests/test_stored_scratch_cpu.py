"""Scratch of the products of activations that come in 8 bits: no room for a rounded copy of x, which only those of
activations in fp16 make.  Asked for and checked on the host, before any launch."""
import ctypes

import pytest

import non_uniform_weight_amd as nw

P = ctypes.c_void_p
A, B = P(0x100000), P(0x200000)  # aligned addresses that are never read
LIB = nw.library()

# rows, cols, batch: streaming, tiles, halves, and split columns
SIZES = [(8192, 22016, 1), (300, 9001, 3), (8192, 8192, 16), (4096, 8192, 4096), (8192, 24576, 8192), (13824, 5120, 2048),
         (200, 17000, 40), (2097, 16542, 17), (1300, 9000, 390), (64, 1000, 33)]


def gemm(rows, cols, batch, size, ws=A):
    return LIB.sqllm_int8_gemm(A, B, rows, cols, A, B, batch, B, ws, size, None)


def glu(rows, cols, batch, size, ws=A):
    return LIB.sqllm_int8_glu(A, B, A, B, rows, cols, A, B, batch, B, ws, size, None)


@pytest.mark.parametrize("call,query,words", [(gemm, nw.int8_workspace_bytes, 1), (glu, nw.int8_glu_workspace_bytes, 2)],
                         ids=["gemm", "glu"])
@pytest.mark.parametrize("rows,cols,batch", SIZES)
def test_integer_products(rows, cols, batch, call, query, words):
    splits = nw.int8.int8_plan(rows, cols, batch, words == 2, True).get("splits", 1)
    sums = splits * batch * (-(-rows // 4) * 4) * 4 * words  # of 32 bits, rows in fours
    need = query(rows, cols, batch, stored=True)
    assert need == (sums if splits > 1 else 256)
    assert query(rows, cols, batch) >= need + batch * nw.int8_cols(cols)
    assert call(rows, cols, batch, need - 1) == call(rows, cols, batch, need, None) == 8
    assert call(rows, cols, batch, need, P(0x100080)) == 8


@pytest.mark.parametrize("query", [nw.int8_workspace_bytes, nw.int8_glu_workspace_bytes])
def test_sizes_out_of_range(query):
    assert query(0, 300, 1, stored=True) == query(64, 131072, 1, stored=True) == query(64, 300, 0, stored=True) == 0
    assert query(1 << 20, 300, 1 << 19, stored=True) == query(64 + 2 ** 64, 300, 3, stored=True) == 0


def fp8(rows, cols, batch, size, ws=A):
    return LIB.sqllm_fp8_gemm_stored(A, B, rows, cols, A, B, batch, B, ws, size, None)


@pytest.mark.parametrize("rows,cols,batch", SIZES)
def test_e4m3_product(rows, cols, batch):
    need = nw.fp8_workspace_bytes(rows, cols, batch, stored=True)
    assert need == 256 or any(need == splits * batch * rows * 4 for splits in range(2, 9))
    assert nw.fp8_workspace_bytes(rows, cols, batch) >= batch * nw.fp8_cols(cols) + (need if need > 256 else 0)
    assert fp8(rows, cols, batch, need - 1) == fp8(rows, cols, batch, need, None) == 8
    assert fp8(rows, cols, batch, need, P(0x100080)) == 8


def test_e4m3_sizes_out_of_range():
    query = nw.fp8_workspace_bytes
    assert query(0, 300, 1, stored=True) == query(64, 1 << 25, 1, stored=True) == query(64, 300, 0, stored=True) == 0
    assert query(1 << 20, 300, 1 << 19, stored=True) == query(64 + 2 ** 64, 300, 3, stored=True) == 0
