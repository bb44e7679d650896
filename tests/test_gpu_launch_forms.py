"""Launch forms of the expert products and of the 8-bit calls that small sizes do not reach."""
import numpy as np
import pytest
import torch

from gpu_util import nw, step
from test_gpu_fp8 import acts, check_product, check_quantized, weights, wide
from test_gpu_moe import Layer, choices, tokens
from test_gpu_moe_outliers import set_lut

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("kw", [{"density": 0}, {"density": 0.005}, {"density": 0.01, "skew": True}])
@pytest.mark.parametrize("batch,inter", [(1, 8192), (1, 16384), (6, 16384), (12, 8192)])
def test_down_columns_split_between_workgroups(batch, inter, kw, bits):
    """Few rows and long columns: four and eight workgroups share a tile of down."""
    step(f"moe down splits {bits}-bit batch {batch} 256x{inter} {kw}")
    layer = Layer(2, 256, inter, bits, 5, **kw)
    x = tokens(batch, 256, 1)
    ids, w = choices(batch, 2, 1, 2)
    y = layer.run(x, ids, w)
    layer.check(x, ids, w, y)
    assert torch.equal(y, layer.run(x, ids, w))


@pytest.mark.parametrize("bits", [2, 3, 4])
def test_activations_beyond_fp16(bits):
    """a = 256 * 255.875 = 65504 is kept; one of 65536 is infinite, and so is every y that it enters."""
    step(f"moe activations at the end of fp16, {bits}-bit")
    layer = Layer(1, 256, 256, bits, 1, density=0)
    n, codes = 1 << bits, np.zeros((1, 256, 256), dtype=np.uint8)
    for p in (layer.gate, layer.up, layer.down):
        p.bits = bits
    set_lut(layer.gate, np.full((1, 256, n), 1.0, dtype=np.float16), codes)
    set_lut(layer.down, np.full((1, 256, n), 2.0 ** -10, dtype=np.float16), codes)
    up = np.full((1, 256, n), 1 - 2.0 ** -11, dtype=np.float16)
    x = torch.zeros(2, 256, dtype=torch.float16, device="cuda")
    x[0, 3], x[1, 7] = 256, 1
    ids, w = torch.zeros(2, 1, dtype=torch.int32, device="cuda"), torch.ones(2, 1, device="cuda")
    set_lut(layer.up, up, codes)
    y = layer.run(x, ids, w)
    layer.check(x, ids, w, y)
    assert (y[0] == 16376).all()
    up[0, 200] = 1
    set_lut(layer.up, up, codes)
    z = layer.run(x, ids, w)
    assert (z[0] == float("inf")).all()
    layer.check(x[1:], ids[1:], w[1:], z[1:])


def test_quantize_more_rows_than_a_launch_has_groups():
    """1.1 million rows of one word of scales: each group of lanes takes a second row."""
    step("fp8 quantize 1100000x5")
    base = wide(1000, 5, 9)
    x = torch.from_numpy(base).cuda().repeat(1100, 1)
    q, scale = nw().fp8_quantize(x)
    check_quantized(base, q[-1000:], scale[-1000:])
    assert torch.equal(q.view(1100, 1000, 128), q[-1000:].expand(1100, 1000, 128))
    assert torch.equal(scale.view(1100, 1000, 4), scale[-1000:].expand(1100, 1000, 4))


@pytest.mark.parametrize("batch,rows,cols", [(4400, 4200, 200), (2305, 8192, 640)])
def test_more_large_tiles_than_compute_units(batch, rows, cols):
    """306 and 320 tiles of 256x256 on 256 compute units."""
    step(f"fp8 gemm batch {batch} {rows}x{cols}")
    q, scale = weights(rows, cols, 3)
    x = acts(batch, cols, 4)
    y = nw().fp8_gemm(q, scale, x)
    check_product(q, scale, x, y)
    assert torch.equal(y, nw().fp8_gemm(q, scale, x))


@pytest.mark.parametrize("rows,cols,batches", [(2048, 8192, (7, 8, 16)), (1300, 12800, (14, 15)), (2700, 6016, (10, 11)),
                                               (500, 7168, (16,)), (4096, 4096, (15, 16)), (1600, 10240, (6, 7))])
def test_small_matrices_on_both_sides_of_one_launch(rows, cols, batches):
    """The streaming form that rounds x itself, up to the batch where the rounding outweighs a launch, and past it."""
    q, scale = weights(rows, cols, 5)
    for batch in batches:
        step(f"fp8 gemm batch {batch} {rows}x{cols}")
        x = acts(batch, cols, 6)
        y = nw().fp8_gemm(q, scale, x)
        check_product(q, scale, x, y)
        assert torch.equal(y, nw().fp8_gemm(q, scale, x))
