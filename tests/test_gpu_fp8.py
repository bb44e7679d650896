"""Block-scaled e4m3 quantiser and product on the GPU against 64-bit references.

Tolerances: codes and scales are exact.  A product's sums run in fp32: cols additions of terms of total magnitude
M = sum |wx| are off by at most cols * 2^-23 * M (half of that for round-to-nearest adds; the matrix cores' adds may
truncate), and the result is rounded once: 2^-11 of its value, 2^-25 among the subnormals.

Before that the matrix cores add the products of each eight adjacent columns on one grid: with 2^e the product of the
powers of two of the group's largest term (its operands' mantissas multiply to 1 <= m < 4, so 2^e <= |term|), every
term is cut to a multiple of 2^(e - 13) towards zero.  The largest term itself has at most 6 bits after its point (two
3-bit fractions) and is not cut; the seven others lose less than 2^-13 * |largest| each.  So a group is off by less than
7 * 2^-13 * max |wx| over its eight columns, whatever the data (test_matrix_core_grid holds the grid itself)."""
import numpy as np
import pytest
import torch

from gpu_util import nw, step

pytestmark = pytest.mark.gpu

GRID = None


def e4m3_values():
    """The 256 codes' values, from the format: sign, 4 exponent bits (bias 7), 3 mantissa bits, 0x7F NaN."""
    global GRID
    if GRID is None:
        c = np.arange(128)
        e, m = c >> 3, c & 7
        v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
        v[127] = np.nan
        GRID = np.concatenate([v, -v])
    return GRID


def reference(x):
    """(values, exponents) of float64 x [rows, cols]: nearest e4m3 by distance over the whole grid, ties to the
    even code, at the smallest exponent that keeps the block within 448."""
    rows, cols = x.shape
    pad = -cols % 128
    b = np.pad(x, ((0, 0), (0, pad))).reshape(rows, -1, 128)
    top = np.where(np.isfinite(b), np.abs(b), 0).max(axis=2)
    s = np.zeros(top.shape, dtype=np.int64)
    live = top > 0
    s[live] = -60
    for k in range(-60, 20):
        s[live & (top > 448 * 2.0 ** s)] = k + 1
    grid = e4m3_values()[:127]
    a = np.abs(b) * 2.0 ** -s[..., None].astype(np.float64)
    fin = np.isfinite(a)
    hi = np.clip(np.searchsorted(grid, np.where(fin, a, 0)), 1, 126)
    lo = hi - 1
    dl, dh = np.where(fin, a, 0) - grid[lo], grid[hi] - np.where(fin, a, 0)
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    v = np.where(fin, np.sign(b) * grid[code], np.nan)
    return v.reshape(rows, -1), s


def stored(q, scale, cols):
    v = e4m3_values()[q.cpu().numpy()]
    nb = (cols + 127) // 128
    sb = scale.cpu().numpy().astype(np.int64)
    assert (sb[:, nb:] == 127).all()
    return v, sb[:, :nb] - 127


def dequantized(q, scale, cols):
    v, s = stored(q, scale, cols)
    return v * np.repeat(2.0 ** s.astype(np.float64), 128, axis=1)


def wide(rows, cols, seed):
    """fp16 values over the whole exponent range, zeros, halves and block borders among them."""
    r = np.random.default_rng(seed)
    x = r.standard_normal((rows, cols)) * 2.0 ** r.integers(-24, 12, (rows, (cols + 127) // 128)).repeat(128, axis=1)[:, :cols]
    x[r.random((rows, cols)) < 0.05] = 0
    x[r.random((rows, cols)) < 0.02] = 448 * 2.0 ** -7
    return np.clip(x, -65504, 65504).astype(np.float16)


def check_quantized(xh, q, scale):
    rows, cols = xh.shape
    v, s = stored(q, scale, cols)
    rv, rs = reference(xh.astype(np.float64))
    np.testing.assert_array_equal(s, rs)
    np.testing.assert_array_equal(v, rv)


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 127), (3, 128), (2, 129), (5, 511), (7, 513), (64, 1000), (33, 2048),
                                       (130, 2056), (1, 20001), (5000, 130)])
def test_quantize(rows, cols):
    step(f"fp8 quantize {rows}x{cols}")
    xh = wide(rows, cols, rows * 7 + cols)
    q, scale = nw().fp8_quantize(torch.from_numpy(xh).cuda())
    assert tuple(q.shape) == (rows, nw().fp8_cols(cols)) and tuple(scale.shape) == (rows, nw().fp8_scale_pitch(cols))
    check_quantized(xh, q, scale)


def test_quantize_borders():
    """Every positive fp16 value as a block's largest, among the values that it scales."""
    step("fp8 quantize borders")
    bits = np.arange(1, 0x7C00, dtype=np.uint16)
    r = np.random.default_rng(3)
    x = np.zeros((bits.size, 128), dtype=np.float16)
    x[:] = (bits.view(np.float16)[:, None].astype(np.float64) * r.uniform(-1, 1, (1, 128))).astype(np.float16)
    x[:, 5] = bits.view(np.float16)
    x[:, 6] = -bits.view(np.float16)
    q, scale = nw().fp8_quantize(torch.from_numpy(x).cuda())
    check_quantized(x, q, scale)


def test_quantize_special_values():
    step("fp8 quantize specials")
    x = wide(4, 300, 1)
    x[0, 5], x[0, 200], x[1, 7] = np.inf, -np.inf, np.nan
    x[2, :128] = np.nan   # nothing finite in the block
    x[3, 128:256] = 0     # nothing but zeros
    q, scale = nw().fp8_quantize(torch.from_numpy(x).cuda())
    check_quantized(x, q, scale)
    assert stored(q, scale, 300)[1][2, 0] == 0 and stored(q, scale, 300)[1][3, 1] == 0


@pytest.mark.parametrize("offset,width", [(0, 640), (1, 515), (8, 648), (3, 640)])
def test_quantize_strided_rows(offset, width):
    step(f"fp8 quantize strided {offset} {width}")
    full = wide(9, width, offset)
    view = torch.from_numpy(full).cuda()[:, offset:offset + 500]
    q, scale = nw().fp8_quantize(view)
    check_quantized(full[:, offset:offset + 500], q, scale)


def weights(rows, cols, seed):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(rows, cols, generator=g) * 0.02).half().cuda()
    return nw().fp8_quantize(w)


def acts(batch, cols, seed):
    g = torch.Generator().manual_seed(seed + 1)
    x = torch.randn(batch, cols, generator=g)
    x[:, :: max(1, cols // 3)] *= 30
    return x.half().cuda()


def check_product(q, scale, x, y):
    cols = x.shape[1]
    w = dequantized(q, scale, cols)
    xq = dequantized(*nw().fp8_quantize(x), cols)
    ref, mag = xq @ w.T, np.abs(xq) @ np.abs(w).T
    ax, aw = torch.from_numpy(np.abs(xq)).cuda(), torch.from_numpy(np.abs(w)).cuda()
    cut = torch.stack([(row * aw).view(len(w), -1, 8).amax(dim=2).sum(dim=1) for row in ax]).cpu().numpy()
    tol = cols * 2.0 ** -23 * mag + 7 * 2.0 ** -13 * cut + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25
    err = np.abs(y.float().cpu().numpy().astype(np.float64) - ref)
    assert (err <= tol).all(), f"{(err / tol).max():.3f} of the tolerance at {np.unravel_index((err / tol).argmax(), err.shape)}"


SHAPES = [(1, 1, 1), (1, 16, 128), (1, 300, 4096), (2, 129, 127), (3, 64, 8320), (7, 1, 1000), (15, 257, 640), (16, 512, 2048),
          (17, 64, 256), (17, 300, 130), (31, 1000, 1300), (33, 130, 512), (64, 256, 4096), (65, 127, 700),
          (128, 128, 128), (129, 513, 1024), (200, 70, 3000), (255, 256, 640), (257, 255, 1152), (512, 768, 2000),
          (1000, 300, 300), (1, 5000, 22016), (40, 2304, 6400), (300, 2560, 1536),
          (1, 130, 20008), (11, 300, 24000), (16, 2000, 16500), (16, 8200, 512), (5, 8193, 300),
          (3600, 3590, 130), (3400, 3841, 640), (3585, 3500, 1000),
          (500, 6100, 300), (100, 300, 16500), (130, 129, 20000), (40, 200, 17000), (2, 8200, 2100), (16, 8193, 2176),
          (9, 2050, 16400), (24, 2100, 5000), (90, 4100, 640), (16, 8200, 8200), (1, 8193, 9000), (5, 700, 8300),
          (16, 4100, 4100), (3, 2000, 5001), (16, 6000, 700)]


@pytest.mark.parametrize("batch,rows,cols", SHAPES)
def test_gemm(batch, rows, cols):
    step(f"fp8 gemm batch {batch} {rows}x{cols}")
    q, scale = weights(rows, cols, batch + rows)
    x = acts(batch, cols, cols)
    guard = torch.full((batch * rows + 512,), 7.0, dtype=torch.float16, device="cuda")
    y = guard[256:256 + batch * rows].view(batch, rows)
    out = nw().fp8_gemm(q, scale, x, y=y)
    check_product(q, scale, x, out)
    assert (guard[:256] == 7).all() and (guard[256 + batch * rows:] == 7).all()
    assert torch.equal(out, nw().fp8_gemm(q, scale, x))  # the same bits again


@pytest.mark.parametrize("batch", [1, 20, 140])
def test_matrix_core_grid(batch):
    """A term of 2^3 survives beside one of 2^16 in its group of eight columns, and 2^-1 does not where it would be
    seen (the large terms cancel between two groups); apart from it both survive."""
    step(f"fp8 gemm grid batch {batch}")
    w = torch.zeros(1, 128, dtype=torch.float16, device="cuda")
    w[0, 0], w[0, 8] = 256, -256
    w[0, 1] = w[0, 17] = 1
    q, scale = nw().fp8_quantize(w)
    for small, near, far in ((8.0, 8.0, 8.0), (0.5, 0.0, 0.5)):
        for col, want in ((1, near), (17, far)):
            x = torch.zeros(batch, 128, dtype=torch.float16, device="cuda")
            x[:, 0], x[:, 8], x[:, col] = 256, 256, small
            assert (nw().fp8_gemm(q, scale, x) == want).all()


@pytest.mark.parametrize("batch", [1, 5, 16, 24, 130])
def test_gemm_misaligned_inputs(batch):
    """x and y that begin at odd addresses of 16-bit values."""
    step(f"fp8 gemm misaligned batch {batch}")
    q, scale = weights(200, 777, 5)
    x = torch.empty(batch * 777 + 3, dtype=torch.float16, device="cuda")[3:].view(batch, 777)
    x.copy_(acts(batch, 777, 6))
    y = torch.empty(batch * 200 + 1, dtype=torch.float16, device="cuda")[1:].view(batch, 200)
    check_product(q, scale, x, nw().fp8_gemm(q, scale, x, y=y))


@pytest.mark.parametrize("batch", [2, 16, 20, 150])
def test_gemm_keeps_nan_in_its_row(batch):
    step(f"fp8 gemm NaN batch {batch}")
    q, scale = weights(150, 600, 8)
    x = acts(batch, 600, 9)
    clean = nw().fp8_gemm(q, scale, x)
    x[batch - 1, 300] = float("nan")
    x[0, 599] = float("inf")
    y = nw().fp8_gemm(q, scale, x)
    assert y[0].isnan().all() and y[batch - 1].isnan().all()
    assert torch.equal(y[1:batch - 1], clean[1:batch - 1])


def test_gemm_large_values_overflow_to_infinity():
    step("fp8 gemm overflow")
    w = torch.full((3, 256), 200.0, dtype=torch.float16, device="cuda")
    w[1] = -200.0
    q, scale = nw().fp8_quantize(w)
    for batch in (1, 20, 140):
        y = nw().fp8_gemm(q, scale, torch.full((batch, 256), 100.0, dtype=torch.float16, device="cuda"))
        assert (y[:, 0] == float("inf")).all() and (y[:, 1] == float("-inf")).all()


def test_gemm_one_dimensional_x_and_own_workspace():
    step("fp8 gemm workspace")
    q, scale = weights(96, 384, 2)
    x = acts(1, 384, 3)
    ws = torch.full((nw().fp8_workspace_bytes(96, 384, 1),), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(nw().fp8_gemm(q, scale, x[0], ws=ws), nw().fp8_gemm(q, scale, x))


@pytest.mark.parametrize("batch", [1, 24, 140])
def test_gemm_on_another_stream_and_in_graphs(batch):
    """Two captured graphs replayed in turn, on two streams, with eager calls between."""
    step(f"fp8 gemm streams and graphs batch {batch}")
    q, scale = weights(520, 1500, 4)
    xs = [acts(batch, 1500, 20 + k) for k in range(3)]
    want = [nw().fp8_gemm(q, scale, x).clone() for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = nw().fp8_gemm(q, scale, xs[1], stream=side)
    side.synchronize()
    assert torch.equal(got, want[1])
    graphs = []
    for k in range(2):
        x = xs[k].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = nw().fp8_gemm(q, scale, x)
        graphs.append((g, x, y))
    for turn in range(4):
        for k, (g, x, y) in enumerate(graphs):
            x.copy_(xs[(k + turn) % 3])
            y.fill_(3)
        torch.cuda.synchronize()
        other = torch.cuda.Stream()
        graphs[0][0].replay()
        with torch.cuda.stream(other):
            graphs[1][0].replay()
        eager = nw().fp8_gemm(q, scale, xs[2])
        torch.cuda.synchronize()
        assert torch.equal(eager, want[2])
        for k, (g, x, y) in enumerate(graphs):
            assert torch.equal(y, want[(k + turn) % 3])


def test_quantize_and_gemm_from_two_threads():
    """Calls of two host threads on one stream, which share its scratch."""
    import threading
    step("fp8 gemm threads")
    q, scale = weights(300, 900, 4)
    xs = [acts(b, 900, 40 + b) for b in (3, 40)]
    want = [nw().fp8_gemm(q, scale, x) for x in xs]
    got = [[], []]

    def work(k):
        for _ in range(20):
            got[k].append(nw().fp8_gemm(q, scale, xs[k]))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[k]) for k in range(2) for y in got[k])
