"""Products in 8-bit integers on the GPU against exact sums.

The sum of products is an integer below 2^31: exact.  y is its conversion to fp32, a product with the fp32 product of
the two scales and a rounding to fp16, each to nearest: numpy does the same steps, so y has to have the same bits.

int8_glu's two products are those fp32 numbers g and u.  silu(g) u after them: the exponent -g log2(e) is rounded in
fp32, |g| 2^-24 of e^-g; exponential, sum, quotient and product round four times more (2^-23 each at worst).  So h is
off by (|g| + 8) 2^-23 of its value (a g beyond -88 gives 0 for less than 2^-25), and one rounding to fp16."""
import threading

import numpy as np
import pytest
import torch

from gpu_util import nw, step

pytestmark = pytest.mark.gpu


def codes(rows, cols, seed, whole=False):
    """Random stored matrices: codes over the whole range and scales of different sizes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    wide = nw().int8_cols(cols)
    q = torch.randint(-128 if whole else -127, 128, (rows, wide), generator=g, device="cuda", dtype=torch.int8)
    q[:, cols:] = 0
    return q, torch.rand(rows, generator=g, device="cuda") * 0.02 / cols ** 0.5 + 1e-6


def acts(batch, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn(batch, cols, generator=g, device="cuda")
    x[:, :: max(1, cols // 3)] *= 30
    return x.half()


def sums(q, xq):
    """Exact sums: 64-bit floating point holds every integer below 2^53, and these stay below 2^31."""
    return (xq.double() @ q.double().t().contiguous()).cpu().numpy()


def number(q, scale, xq, xs):
    s = (xs.cpu().numpy()[:, None] * scale.cpu().numpy()[None]).astype(np.float32)
    return sums(q, xq).astype(np.float32) * s


def same(y, want):
    with np.errstate(over="ignore"):
        want = want.astype(np.float16)
    got = y.cpu().numpy()
    assert np.array_equal(got, want, equal_nan=True), np.argwhere(got != want)[:5]


def check_glu(h, g, u):
    g, u = g.astype(np.float64), u.astype(np.float64)
    with np.errstate(over="ignore"):
        ref = g / (1 + np.exp(-g)) * u
    got = h.cpu().numpy().astype(np.float64)
    over = np.abs(ref) >= 65520
    assert (np.isinf(got) == over).all() or np.abs(ref[np.isinf(got) != over] / 65520 - 1).max() < 1e-4
    tol = (2.0 ** -11 + (np.abs(g) + 8) * 2.0 ** -23) * np.abs(ref) + 2.0 ** -25
    err = np.abs(np.where(over, 0, got - ref))
    assert (err <= tol).all(), (err / tol).max()


SHAPES = [(1, 1, 1), (1, 16, 128), (1, 300, 4096), (2, 129, 127), (3, 64, 8320), (7, 1, 1000), (15, 257, 640),
          (16, 512, 2048), (17, 64, 256), (17, 300, 130), (31, 1000, 1300), (33, 130, 512), (64, 256, 4096), (65, 127, 700),
          (128, 128, 128), (129, 513, 1024), (200, 70, 3000), (255, 256, 640), (257, 255, 1152), (512, 768, 2000),
          (1000, 300, 300), (1, 5000, 22016), (40, 2304, 6400), (300, 2560, 1536), (1, 130, 20008), (11, 300, 24000),
          (16, 2000, 16500), (16, 8200, 512), (5, 8193, 300), (3600, 3590, 130), (3400, 3841, 640), (3585, 3500, 1000),
          (500, 6100, 300), (100, 300, 16500), (40, 200, 17000), (2, 8200, 2100), (16, 8193, 2176), (9, 2050, 16400),
          (24, 2100, 5000), (90, 4100, 640), (16, 8200, 8200), (5, 700, 8300), (16, 4100, 4100), (3, 40, 131071),
          (130, 140, 60000), (8, 30, 33000), (700, 4300, 900), (4, 4096, 4096), (2, 600, 200),
          (4200, 8100, 1500), (4200, 6100, 700), (4200, 500, 300), (390, 4300, 300), (390, 2000, 300), (130, 3900, 9000),
          (2000, 3900, 300), (130, 8100, 17000), (130, 2500, 9000), (130, 6100, 9000), (390, 1300, 9000), (390, 200, 9000),
          (1300, 1100, 9100), (1000, 2050, 130)]


def guarded(batch, rows):
    g = torch.full((batch * rows + 512,), 7.0, dtype=torch.float16, device="cuda")
    return g, g[256:256 + batch * rows].view(batch, rows)


@pytest.mark.parametrize("batch,rows,cols", SHAPES)
def test_gemm(batch, rows, cols):
    """Activations in integers, and in fp16: the same as rounding them first, bit for bit."""
    step(f"int8 gemm batch {batch} {rows}x{cols}")
    q, scale = codes(rows, cols, batch + rows)
    x = acts(batch, cols, cols)
    xq, xs = nw().int8_quantize(x)
    want = number(q, scale, xq, xs)
    guard, y = guarded(batch, rows)
    nw().int8_gemm(q, scale, xq, xs, y=y)
    same(y, want)
    assert (guard[:256] == 7).all() and (guard[256 + batch * rows:] == 7).all()
    guard, y = guarded(batch, rows)
    nw().int8_gemm(q, scale, x, y=y)
    same(y, want)
    assert (guard[:256] == 7).all() and (guard[256 + batch * rows:] == 7).all()


@pytest.mark.parametrize("batch,rows,cols", SHAPES)
def test_glu(batch, rows, cols):
    step(f"int8 glu batch {batch} {rows}x{cols}")
    (gq, gs), (uq, us) = codes(rows, cols, batch + rows), codes(rows, cols, batch + rows + 1)
    x = acts(batch, cols, cols)
    xq, xs = nw().int8_quantize(x)
    g, u = number(gq, gs, xq, xs), number(uq, us, xq, xs)
    guard, h = guarded(batch, rows)
    nw().int8_glu(gq, gs, uq, us, xq, xs, h=h)
    check_glu(h, g, u)
    assert (guard[:256] == 7).all() and (guard[256 + batch * rows:] == 7).all()
    assert torch.equal(nw().int8_glu(gq, gs, uq, us, x), h)


# Tiles of a few rows of W whose waves share the blocks (one to 128 blocks, so that some groups of waves have one less
# or none; rows and batches that end inside a tile), and split columns with the tiles above them.
FEW = [(17, 32, 100), (17, 33, 128), (20, 4097, 129), (32, 4096, 4096), (48, 2700, 4000), (64, 1000, 385), (32, 4090, 11008),
       (129, 700, 7000), (295, 210, 128), (582, 193, 136), (60, 2040, 8192), (300, 500, 9000), (29, 2300, 13900),
       (26, 8465, 6456), (19, 4483, 16399), (17, 2097, 16542), (656, 778, 9159), (428, 577, 4998), (370, 216, 16669),
       (553, 466, 9433), (376, 342, 5449), (291, 141, 16682), (462, 1029, 9409), (451, 857, 7459), (401, 473, 16406),
       (437, 1745, 17094), (480, 433, 7598), (614, 179, 16510), (177, 2637, 11906), (708, 1185, 129), (620, 3281, 129),
       (643, 1236, 11607), (545, 1848, 5886), (516, 3196, 129), (40, 10990, 4200), (130, 5001, 4999), (70, 2900, 8190)]


@pytest.mark.parametrize("batch,rows,cols", FEW)
def test_few_tiles(batch, rows, cols):
    test_gemm(batch, rows, cols)
    test_glu(batch, rows, cols)


@pytest.mark.parametrize("batch", [1, 16, 40, 300])
def test_largest_sums(batch):
    """Rows of codes of one sign at both ends of their range, up to the longest row: the sums stay within 32 bits."""
    step(f"int8 gemm largest sums batch {batch}")
    cols, wide = 131071, 131072
    q = torch.full((20, wide), -128, dtype=torch.int8, device="cuda")
    q[1::2] = 127
    xq = torch.full((batch, wide), -128, dtype=torch.int8, device="cuda")
    xq[1::3] = 127
    q[:, cols:] = 0
    xq[:, cols:] = 0
    scale, xs = torch.full((20,), 2.0 ** -20, device="cuda"), torch.full((batch,), 2.0 ** -4, device="cuda")
    want = number(q, scale, xq, xs)
    assert np.abs(sums(q, xq)).max() == 128 * 128 * cols
    same(nw().int8_gemm(q, scale, xq, xs), want)
    check_glu(nw().int8_glu(q, scale * 2.0 ** -3, q, scale, xq, xs), want / 8, want)


@pytest.mark.parametrize("batch", [1, 5, 16, 24, 130, 700])
def test_misaligned(batch):
    """x and y that begin at odd addresses of 16-bit values; every value of the code range."""
    step(f"int8 misaligned batch {batch}")
    q, scale = codes(203, 777, 5, whole=True)
    x = torch.empty(batch * 777 + 3, dtype=torch.float16, device="cuda")[3:].view(batch, 777)
    x.copy_(acts(batch, 777, 6))
    y = torch.empty(batch * 203 + 1, dtype=torch.float16, device="cuda")[1:].view(batch, 203)
    xq, xs = nw().int8_quantize(x)
    same(nw().int8_gemm(q, scale, x, y=y), number(q, scale, xq, xs))
    h = torch.empty(batch * 203 + 1, dtype=torch.float16, device="cuda")[1:].view(batch, 203)
    check_glu(nw().int8_glu(q, scale, q, scale, x, h=h), *[number(q, scale, xq, xs)] * 2)


@pytest.mark.parametrize("batch,rows,cols", [(1, 150, 600), (2, 150, 600), (16, 150, 600), (20, 150, 600), (150, 150, 600),
                                             (2, 700, 9000), (600, 5000, 300)])
def test_nan_stays_in_its_row(batch, rows, cols):
    step(f"int8 NaN batch {batch}")
    q, scale = codes(rows, cols, 8)
    x = acts(batch, cols, 9)
    clean = nw().int8_gemm(q, scale, x)
    x[batch - 1, cols // 2] = float("nan")
    x[0, cols - 1] = float("inf")
    y, h = nw().int8_gemm(q, scale, x), nw().int8_glu(q, scale, q, scale, x)
    assert y[0].isnan().all() and y[batch - 1].isnan().all() and h[0].isnan().all() and h[batch - 1].isnan().all()
    assert torch.equal(y[1:batch - 1], clean[1:batch - 1]) and not h[1:batch - 1].isnan().any()
    scale[rows // 2] = float("nan")  # a weight row that held one
    y = nw().int8_gemm(q, scale, acts(batch, cols, 9))
    assert y[:, rows // 2].isnan().all() and not y[:, :rows // 2].isnan().any() and not y[:, rows // 2 + 1:].isnan().any()


@pytest.mark.parametrize("batch", [1, 20, 140, 600])
def test_large_values_overflow_to_infinity(batch):
    step(f"int8 overflow batch {batch}")
    w = torch.full((3, 256), 200.0, dtype=torch.float16, device="cuda")
    w[1] = -200.0
    q, scale = nw().int8_quantize(w)
    x = torch.full((batch, 256), 100.0, dtype=torch.float16, device="cuda")
    y = nw().int8_gemm(q, scale, x)
    assert (y[:, 0] == float("inf")).all() and (y[:, 1] == float("-inf")).all()
    h = nw().int8_glu(q, scale, q, scale, x)  # silu of a large negative number is 0
    assert (h[:, 0] == float("inf")).all() and (h[:, 1] == 0).all() and (h[:, 2] == float("inf")).all()


def test_zeros():
    step("int8 zeros")
    for batch in (1, 18, 200):
        q, scale = nw().int8_quantize(torch.zeros(70, 300, dtype=torch.float16, device="cuda"))
        x = torch.zeros(batch, 300, dtype=torch.float16, device="cuda")
        assert (scale == 0).all() and (nw().int8_gemm(q, scale, x) == 0).all()
        assert (nw().int8_glu(q, scale, q, scale, x) == 0).all()


def test_one_dimensional_x_and_own_workspace():
    step("int8 workspace")
    q, scale = codes(96, 384, 2)
    x = acts(1, 384, 3)
    ws = torch.full((nw().int8_workspace_bytes(96, 384, 1),), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(nw().int8_gemm(q, scale, x[0], ws=ws), nw().int8_gemm(q, scale, x))
    ws = torch.full((nw().int8_glu_workspace_bytes(96, 384, 1),), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(nw().int8_glu(q, scale, q, scale, x[0], ws=ws), nw().int8_glu(q, scale, q, scale, x))


def block(s, x, residual):
    """The feed-forward half of a decoder layer in integers: the norm's residual comes back too."""
    q, xs, total = nw().rms_norm_int8(x, s["norm"], 1e-5, residual=residual)
    h = nw().int8_glu(*s["gate"], *s["up"], q, xs)
    return nw().int8_gemm(*s["down"], h), total, (q, xs, h)


def block_of(hidden, inter, seed):
    norm = (1 + 0.1 * torch.randn(hidden, generator=torch.Generator().manual_seed(seed))).half().cuda()
    return {"norm": norm, "gate": codes(inter, hidden, seed), "up": codes(inter, hidden, seed + 1),
            "down": codes(hidden, inter, seed + 2)}


@pytest.mark.parametrize("batch", [1, 3, 16, 50, 400])
def test_block(batch):
    """The calls as they are used together: each against its own reference on what the one before left."""
    step(f"int8 block batch {batch}")
    s = block_of(768, 2100, 4)
    x, res = acts(batch, 768, 1), acts(batch, 768, 2)
    y, total, (q, xs, h) = block(s, x, res)
    assert torch.equal(total, x + res)
    v = total.double()
    v = v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + 1e-5) * s["norm"].double()
    top = v.abs().amax(dim=1)
    e = 25 * 2.0 ** -24  # as for the norm alone
    assert ((xs.double() - top / 127).abs() <= e * top / 127).all()
    assert ((q[:, :768].double() - v * 127 / top[:, None]).abs() <= 0.5 + 127 * (2 * e + 2.0 ** -23)).all()
    check_glu(h, number(*s["gate"], q, xs), number(*s["up"], q, xs))
    same(y, number(*s["down"], *nw().int8_quantize(h)))


@pytest.mark.parametrize("batch", [1, 24, 140, 600])
def test_block_on_another_stream_and_in_graphs(batch):
    """Two captured graphs replayed in turn, on two streams, with eager calls between."""
    step(f"int8 block streams and graphs batch {batch}")
    s = block_of(640, 1500, 9)
    res = acts(batch, 640, 3)
    xs = [acts(batch, 640, 20 + k) for k in range(3)]
    want = [block(s, x, res)[0] for x in xs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = block(s, xs[1], res)[0]
    side.synchronize()
    assert torch.equal(got, want[1])
    got = nw().int8_gemm(*s["gate"], xs[1], stream=side)
    side.synchronize()
    assert torch.equal(got, nw().int8_gemm(*s["gate"], xs[1]))
    graphs = []
    for k in range(2):
        x = xs[k].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = block(s, x, res)[0]
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
        eager = block(s, xs[2], res)[0]
        torch.cuda.synchronize()
        assert torch.equal(eager, want[2])
        for k, (g, x, y) in enumerate(graphs):
            assert torch.equal(y, want[(k + turn) % 3])


def test_from_two_threads():
    """Calls of two host threads on one stream, which share its scratch."""
    step("int8 threads")
    q, scale = codes(300, 900, 4)
    xs = [acts(b, 900, 40 + b) for b in (3, 40)]
    want = [nw().int8_gemm(q, scale, x) for x in xs]
    got = [[], []]

    def work(k):
        for _ in range(20):
            got[k].append(nw().int8_gemm(q, scale, xs[k]))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[k]) for k in range(2) for y in got[k])


# ------------------------------------------------------------------------- e4m3 products of what the norm leaves
@pytest.mark.parametrize("batch,rows,cols", [(1, 300, 1000), (5, 700, 9000), (16, 8200, 8300), (40, 300, 2000),
                                             (16, 500, 2048), (300, 600, 5001), (600, 5000, 400), (100, 300, 16500)])
def test_fp8_gemm_of_stored_activations(batch, rows, cols):
    """fp8_gemm of activations in the stored form: as of the fp16 values that the form stands for, which it rounds to
    the same form (sums in another order where one launch serves both: those are held to the sums' own bound)."""
    step(f"fp8 gemm stored batch {batch} {rows}x{cols}")
    g = torch.Generator(device="cuda").manual_seed(rows)
    q, scale = nw().fp8_quantize((torch.randn(rows, cols, generator=g, device="cuda") * 0.02).half())
    x, res = acts(batch, cols, 1), acts(batch, cols, 2)
    w = (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).half()
    xq, xs, _ = nw().rms_norm_fp8(x, w, 1e-5, residual=res)
    guard, y = guarded(batch, rows)
    nw().fp8_gemm(q, scale, xq, x_scale=xs, y=y)

    def values(q, s):
        v = q.view(torch.float8_e4m3fn).double().view(q.shape[0], -1, 128)
        return (v * torch.exp2(s[:, :v.shape[1], None].double() - 127)).flatten(1)

    a, b = values(xq, xs), values(q, scale)
    ref, mag = a @ b.t().contiguous(), a.abs() @ b.abs().t().contiguous()
    # groups of eight columns on a grid 2^-13 below their largest product, sums in fp32, one rounding
    cut = torch.stack([(row.abs() * b.abs()).view(rows, -1, 8).amax(dim=2).sum(dim=1) for row in a])
    tol = cols * 2.0 ** -23 * mag + 7 * 2.0 ** -13 * cut + 2.0 ** -11 * ref.abs() + 2.0 ** -25
    assert ((y.double() - ref).abs() <= tol).all()
    assert (guard[:256] == 7).all() and (guard[256 + batch * rows:] == 7).all()


# ------------------------------------------------------------------------------------------- beyond 32-bit offsets
@pytest.mark.parametrize("batch", [1, 3, 16, 40, 300])
def test_weights_past_four_gigabytes(batch):
    """The last rows of a matrix whose codes lie past 2^32 bytes."""
    step(f"int8 weights past 4 GB, batch {batch}")
    rows, cols = 200003, 24000  # 24064 stored columns: 4.8 GB
    q, scale = codes(rows, cols, 3)
    x = acts(batch, cols, 5)
    xq, xs = nw().int8_quantize(x)
    at = torch.arange(rows - 77, rows, device="cuda")
    want = number(q[at], scale[at], xq, xs)
    for y in (nw().int8_gemm(q, scale, xq, xs), nw().int8_gemm(q, scale, x)):
        same(y[:, at], want)
        same(y[:, :50], number(q[:50], scale[:50], xq, xs))
    # gate from the front of the same memory, up from its end: both matrices of 178 000 rows
    n = 178000
    g, u, first = q[:n], q[rows - n:], torch.arange(n - 60, n, device="cuda")
    h = nw().int8_glu(g, scale[:n], u, scale[rows - n:], xq, xs)
    check_glu(h[:, first], number(g[first], scale[first], xq, xs), number(u[first], scale[rows - n:][first], xq, xs))


def test_results_past_four_gigabytes():
    step("int8 results past 4 GB")
    batch, rows, cols = 70000, 33000, 128
    q, scale = codes(rows, cols, 3)
    xq, xs = nw().int8_quantize(acts(batch, cols, 5))
    y = nw().int8_gemm(q, scale, xq, xs)
    b, r = torch.tensor([0, 1, 35000, batch - 2, batch - 1], device="cuda"), torch.arange(rows - 300, rows, device="cuda")
    same(y[b][:, r], number(q[r], scale[r], xq[b], xs[b]))
    del y
    h = nw().int8_glu(q, scale, q, scale, xq, xs)
    check_glu(h[b][:, r], *[number(q[r], scale[r], xq[b], xs[b])] * 2)


def test_first_calls_inside_a_capture():
    """Shapes that no call before took (each launch's one-time settings are made there), captured at once."""
    step("int8 captured first")
    made = []
    for batch, rows, cols in ((6, 900, 17000), (77, 900, 9000), (900, 6000, 200), (300, 2000, 300)):
        q, scale = codes(rows, cols, batch)
        xq, xs = nw().int8_quantize(acts(batch, cols, 2))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = nw().int8_gemm(q, scale, xq, xs)
            h = nw().int8_glu(q, scale, q, scale, xq, xs)
        made.append((g, y, h, number(q, scale, xq, xs), (q, scale, xq, xs)))  # a graph's inputs live as long as it
    for _ in range(3):
        for g, y, h, *_ in made:
            y.fill_(1), h.fill_(1)
            g.replay()
        torch.cuda.synchronize()
        for _, y, h, want, _ in made:
            same(y, want)
            check_glu(h, want, want)
