"""Products of activations that come in 8 bits in scratch of just the bytes that they ask for."""
import pytest
import torch

import test_gpu_int8 as base
from gpu_util import nw, step

pytestmark = pytest.mark.gpu

# batch, rows, cols: streaming in both forms, tiles, halves; then every tile with split columns, of one product or both
SIZES = [(1, 300, 9001), (9, 515, 4097), (64, 1000, 385), (512, 768, 2000), (3400, 3841, 640), (8, 30, 33000),
         (370, 216, 16669), (130, 2500, 9000), (462, 1029, 9409), (437, 1745, 17094), (291, 141, 16682), (614, 179, 16510),
         (401, 473, 16406), (643, 1236, 11607)]


def scratch(need):
    """need bytes of noise between guards."""
    buf = torch.full((need + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
    return buf, buf[512:512 + need]


def kept(buf, need):
    return bool((buf[:512] == 0xA5).all()) and bool((buf[512 + need:] == 0xA5).all())


@pytest.mark.parametrize("batch,rows,cols", SIZES)
def test_integer_products(batch, rows, cols):
    step(f"int8 stored scratch batch {batch} {rows}x{cols}")
    (q, scale), (u, us) = base.codes(rows, cols, 1), base.codes(rows, cols, 2)
    xq, xs = nw().int8_quantize(base.acts(batch, cols, 3))
    want = base.number(q, scale, xq, xs)
    need = nw().int8_workspace_bytes(rows, cols, batch, stored=True)
    buf, ws = scratch(need)
    base.same(nw().int8_gemm(q, scale, xq, xs, ws=ws), want)
    assert kept(buf, need)
    need = nw().int8_glu_workspace_bytes(rows, cols, batch, stored=True)
    buf, ws = scratch(need)
    base.check_glu(nw().int8_glu(q, scale, u, us, xq, xs, ws=ws), want, base.number(u, us, xq, xs))
    assert kept(buf, need)


def test_integer_products_hold_no_room_for_x():
    """What the calls keep for a stream, and what a captured call takes: not the 33 MB of a copy of x."""
    step("int8 stored scratch kept")
    rows, cols, batch = 256, 8192, 4096
    (q, scale), (xq, xs) = base.codes(rows, cols, 1), nw().int8_quantize(base.acts(batch, cols, 3))
    y, h = (torch.empty(batch, rows, dtype=torch.float16, device="cuda") for _ in range(2))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    nw().int8_gemm(q, scale, xq, xs, y=y, stream=stream)
    nw().int8_glu(q, scale, q, scale, xq, xs, h=h, stream=stream)
    stream.synchronize()
    assert torch.cuda.memory_allocated() - before <= 1 << 20
    want = y.clone(), h.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    before = torch.cuda.memory_reserved()
    with torch.cuda.graph(graph):
        nw().int8_gemm(q, scale, xq, xs, y=y)
        nw().int8_glu(q, scale, q, scale, xq, xs, h=h)
    assert torch.cuda.memory_reserved() - before <= 4 << 20
    for _ in range(3):
        y.fill_(1), h.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(h, want[1])


# batch, rows, cols: streaming, tiles, and both with split columns
@pytest.mark.parametrize("batch,rows,cols", [(1, 5000, 9000), (3, 300, 9001), (16, 1000, 16400), (12, 8200, 8300), (16, 500, 2048),
                                             (40, 300, 6000), (100, 300, 16500), (300, 600, 5001), (600, 5000, 400)])
def test_e4m3_product(batch, rows, cols):
    """The bits that the call gives with a full workspace, in bytes of the smaller one between guards."""
    step(f"fp8 stored scratch batch {batch} {rows}x{cols}")
    g = torch.Generator(device="cuda").manual_seed(rows)
    q, scale = nw().fp8_quantize((torch.randn(rows, cols, generator=g, device="cuda") * 0.02).half())
    xq, xs = nw().fp8_quantize(base.acts(batch, cols, 1))
    full = torch.empty(nw().fp8_workspace_bytes(rows, cols, batch), dtype=torch.uint8, device="cuda")
    want = nw().fp8_gemm(q, scale, xq, x_scale=xs, ws=full)
    need = nw().fp8_workspace_bytes(rows, cols, batch, stored=True)
    buf, ws = scratch(need)
    assert torch.equal(nw().fp8_gemm(q, scale, xq, x_scale=xs, ws=ws), want)
    assert kept(buf, need)
    assert torch.equal(nw().fp8_gemm(q, scale, xq, x_scale=xs), want)


def test_e4m3_product_holds_no_room_for_x():
    step("fp8 stored scratch kept")
    rows, cols, batch = 256, 8192, 4096
    q, scale = nw().fp8_quantize(base.acts(rows, cols, 1))
    xq, xs = nw().fp8_quantize(base.acts(batch, cols, 3))
    y = torch.empty(batch, rows, dtype=torch.float16, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    nw().fp8_gemm(q, scale, xq, x_scale=xs, y=y, stream=stream)
    stream.synchronize()
    assert torch.cuda.memory_allocated() - before <= 1 << 20
