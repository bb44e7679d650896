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


def test_weights_past_four_gigabytes():
    """300000 x 16384 in 8 bits, 4.9 GB: the last rows' codes and products."""
    base = (torch.randn(1000, 16384, generator=torch.Generator().manual_seed(1)) * 0.02).half().cuda()
    step("fp8 quantize 300000x16384")
    q, scale = nw().fp8_quantize(base.repeat(300, 1))
    want, wscale = nw().fp8_quantize(base)
    assert torch.equal(q[-1000:], want) and torch.equal(scale[-1000:], wscale)
    for batch in (1, 16, 40, 300):
        step(f"fp8 gemm batch {batch} 300000x16384")
        x = acts(batch, 16384, batch)
        y = nw().fp8_gemm(q, scale, x)
        check_product(want, wscale, x, y[:, -1000:].contiguous())


@pytest.mark.parametrize("bits,experts", [(3, 200), (4, 136)])
def test_experts_past_four_gigabytes(bits, experts):
    """Copies of one expert of 8192x8192, more than 4 GB a projection: the last one's y is the first one's."""
    r = np.random.default_rng(bits)
    parts = {}
    for name in ("gate", "up", "down"):
        codes = torch.from_numpy(r.integers(0, 1 << bits, (8192, 8192), dtype=np.uint8)).cuda()
        lut = torch.from_numpy((r.standard_normal((1, 8192, 1 << bits)) * 0.02).astype(np.float16)).cuda()
        counts = r.binomial(8192, 0.001, 8192)
        nnz = int(counts.sum())
        row_ptr = np.concatenate([[0], np.cumsum(np.tile(counts, experts))])
        col, val = r.integers(0, 8192, nnz).astype(np.uint16), (r.standard_normal(nnz) * 0.1).astype(np.float16)
        parts[name] = {"packed": nw().pack(codes, bits).repeat(experts), "lut": lut.repeat(experts, 1, 1),
                       "row_ptr": torch.from_numpy(row_ptr.astype(np.int32)).cuda(),
                       "col": torch.from_numpy(col.view(np.int16)).cuda().repeat(experts),
                       "val": torch.from_numpy(val).cuda().repeat(experts)}
        assert parts[name]["packed"].numel() > 1 << 32
    for batch in (1, 9):
        step(f"moe experts {bits}-bit batch {batch} {experts} of 8192x8192")
        x = tokens(batch, 8192, 3)
        w = torch.ones(batch, 1, device="cuda")
        first = nw().moe_experts(x, torch.zeros(batch, 1, dtype=torch.int32, device="cuda"), w, **parts, bits=bits)
        last = nw().moe_experts(x, torch.full((batch, 1), experts - 1, dtype=torch.int32, device="cuda"), w, **parts, bits=bits)
        assert first.isfinite().all() and first.abs().max() > 0 and torch.equal(first, last)


def test_calls_on_two_streams_at_once():
    """Calls that follow each other on two streams with nothing between them: each stream has scratch of its own."""
    step("two streams at once")
    layer = Layer(7, 512, 768, 3, 23)
    router = (tokens(7, 512, 42).float() / 512 ** 0.5).half()
    q, scale = weights(1000, 512, 4)

    def step_of(x, **kw):
        y = nw().moe_layer(x, router, 2, layer.gate.dev, layer.up.dev, layer.down.dev, 3, **kw)[0]
        return y, nw().fp8_gemm(q, scale, x, **kw)

    xs = [tokens(b, 512, 50 + b) for b in (3, 16)]
    want = [step_of(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [(k, step_of(xs[k], stream=streams[k])) for _ in range(40) for k in range(2)]
    torch.cuda.synchronize()
    for k, out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want[k]))


def test_quantize_in_a_graph():
    step("fp8 quantize captured")
    x = torch.from_numpy(wide(33, 700, 1)).cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q, scale = nw().fp8_quantize(x)
    for seed in (2, 3, 4):
        xh = wide(33, 700, seed)
        x.copy_(torch.from_numpy(xh))
        g.replay()
        torch.cuda.synchronize()
        check_quantized(xh, q, scale)
