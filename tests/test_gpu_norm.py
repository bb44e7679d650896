"""The norm and the quantiser to 8-bit integers on the GPU against 64-bit references.

Tolerances.  total is one fp16 addition: exact.  Squares of fp16 values are exact in fp32.  Their sum, were it in fp32
throughout, would run through at most `adds` additions on a path from a square to the total (8 in a piece of eight values, the pieces of a thread, 4 + 2
in a wave, one for each wave; rows beyond 32768 columns add the pieces of a thread in one chain), each 2^-24 relative
at worst (all terms are positive); mean and eps add two, and the root halves them; the product with the root rounds
once more and the quotient of the int8 scale once.  So y in fp32 is off by e = (adds / 2 + 4) * 2^-24 relative.

fp16: e and one rounding (2^-11 of the value, 2^-25 among the subnormals).  int8: the scale is off by e; a code is
within half a step of y * 127 / max in steps, 127 * (2 e + 2^-23) more for the two factors' errors and the reciprocal.
e4m3: the exponent is exact unless the block's largest lies within e of a border; a code is within half a step of its
own binade, and e of the value.

The quantiser has no e: its scale is exact, a code within 0.5 + 127 * 2^-24 (the reciprocal rounds once)."""
import numpy as np
import pytest
import torch

from gpu_util import nw, step

pytestmark = pytest.mark.gpu

EPS = 1e-5


def e_of(cols):
    adds = 8 + 4 + 6 + 16 if cols <= 32768 else 8 * (-(-cols // 8192)) + 6 + 16
    return (adds / 2 + 4) * 2.0 ** -24


def rows_of(rows, cols, seed, loud=True):
    r = np.random.default_rng(seed)
    x = r.standard_normal((rows, cols)) * 2.0 ** r.integers(-6, 6, (rows, 1))
    if loud:
        x[:, r.random(cols) < 0.01] *= 20
    return np.clip(x, -60000, 60000).astype(np.float16)


def weight_of(cols, seed):
    return (1 + 0.3 * np.random.default_rng(seed + 77).standard_normal(cols)).astype(np.float16)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def reference(xh, wh, eps=EPS, res=None):
    """(y in 64 bits, the fp16 sums)."""
    total = xh if res is None else (xh.astype(np.float64) + res.astype(np.float64)).astype(np.float16)
    s = total.astype(np.float64)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        return s / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps) * wh.astype(np.float64), total


def check_half(y, ref, e):
    got = y.cpu().numpy().astype(np.float64)
    tol = (2.0 ** -11 + e) * np.abs(ref) + 2.0 ** -25
    assert np.isfinite(got).all() and (np.abs(got - ref) <= tol).all(), np.max(np.abs(got - ref) / tol)


def check_int8(q, scale, ref, e, code_e=None):
    cols = ref.shape[1]
    got, s = q.cpu().numpy().astype(np.float64), scale.cpu().numpy().astype(np.float64)
    assert (got[:, cols:] == 0).all() and got.shape[1] == nw().int8_cols(cols)
    top = np.abs(ref).max(axis=1)
    assert (np.abs(s - top / 127) <= e * top / 127).all()
    live = top > 0
    assert (got[~live] == 0).all()
    steps = ref[live] * 127 / top[live, None]
    off = np.abs(got[live][:, :cols] - steps)
    assert (off <= 0.5 + (127 * (2 * e + 2.0 ** -23) if code_e is None else code_e)).all(), off.max()


def e4m3(q):
    c = np.arange(128)
    ex, m = c >> 3, c & 7
    v = np.where(ex == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (ex - 10.0))
    v[127] = np.nan
    return np.concatenate([v, -v])[q.cpu().numpy()]


def check_fp8(q, scale, ref, e):
    rows, cols = ref.shape
    blocks = -(-cols // 128)
    sb = scale.cpu().numpy().astype(np.int64)
    assert (sb[:, blocks:] == 127).all()
    a = np.pad(ref, ((0, 0), (0, -cols % 128))).reshape(rows, blocks, 128)
    top = np.abs(a).max(axis=2)
    s = sb[:, :blocks] - 127
    live = top > 0
    assert (s[~live] == 0).all()
    t = top[live] / 2.0 ** s[live]
    assert (t <= 448 * (1 + e)).all() and (t * (1 + e) > 224).all()
    a = a / 2.0 ** s[..., None].astype(np.float64)
    v = e4m3(q).reshape(a.shape)
    half = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(a) * (1 + e), 2.0 ** -6))) - 4)
    assert (np.abs(v - a) <= half + e * np.abs(a)).all()
    assert (v.reshape(rows, -1)[:, cols:] == 0).all()


def check(form, got, ref, total, e):
    if form == "fp16":
        got = got if isinstance(got, tuple) else (got,)
        check_half(got[0], ref, e)
        rest = got[1:]
    else:
        (check_int8 if form == "int8" else check_fp8)(got[0], got[1], ref, e)
        rest = got[2:]
    if total is not None:
        assert np.array_equal(rest[0].cpu().numpy().view(np.uint16), total.view(np.uint16))
    else:
        assert not rest


def call(form):
    return {"fp16": nw().rms_norm, "int8": nw().rms_norm_int8, "fp8": nw().rms_norm_fp8}[form]


SHAPES = [(1, 1), (1, 7), (3, 8), (5, 127), (2, 128), (7, 129), (1, 513), (33, 1000), (6, 1024), (5, 1025), (9, 2049),
          (4, 4096), (130, 5001), (2, 8192), (3, 8200), (2, 16385), (1, 32768), (2, 32769), (1, 40003), (300, 64), (2, 16500), (2, 24600), (1100, 2600)]


@pytest.mark.parametrize("form", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(form, rows, cols, residual):
    step(f"norm {form} {rows}x{cols} residual {residual}")
    xh, wh = rows_of(rows, cols, cols + rows), weight_of(cols, cols)
    res = rows_of(rows, cols, cols + 1, loud=False) if residual else None
    ref, total = reference(xh, wh, res=res)
    got = call(form)(dev(xh), dev(wh), EPS, residual=None if res is None else dev(res))
    check(form, got, ref, total if residual else None, e_of(cols))


@pytest.mark.parametrize("form", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("cols", [1, 500, 1100, 6000, 33000])
def test_norm_writes_only_its_outputs(form, cols):
    """Outputs between guards, at odd addresses where they may be; inputs at odd addresses, rows further apart."""
    step(f"norm {form} guards {cols}")
    rows, lead = 5, 3
    xh, rh = rows_of(rows, cols + 11, 1), rows_of(rows, cols + 6, 2)
    x, r = dev(xh)[:, lead:lead + cols], dev(rh)[:, 1:1 + cols]
    wh = weight_of(cols + 1, 3)
    w = dev(wh)[1:]
    ref, total = reference(xh[:, lead:lead + cols], wh[1:], res=rh[:, 1:1 + cols])

    def guarded(n, dtype, at):
        g = torch.full((n + 512,), 7, dtype=dtype, device="cuda")
        return g, g[at:at + n]

    kept = []
    g, t = guarded(rows * cols, torch.float16, 257)
    kept.append((g, 257, rows * cols))
    if form == "fp16":
        g, y = guarded(rows * cols, torch.float16, 255)
        kept.append((g, 255, rows * cols))
        out = {"y": y.view(rows, cols)}
    else:
        wide = nw().int8_cols(cols) if form == "int8" else nw().fp8_cols(cols)
        g, q = guarded(rows * wide, torch.int8 if form == "int8" else torch.uint8, 256)
        kept.append((g, 256, rows * wide))
        n = rows if form == "int8" else rows * nw().fp8_scale_pitch(cols)
        h, s = guarded(n, torch.float32 if form == "int8" else torch.uint8, 256)
        kept.append((h, 256, n))
        out = {"q": q.view(rows, wide), "scale": s if form == "int8" else s.view(rows, -1)}
    got = call(form)(x, w, EPS, residual=r, total=t.view(rows, cols), **out)
    check(form, got, ref, total, e_of(cols))
    for g, at, n in kept:
        assert (g[:at] == 7).all() and (g[at + n:] == 7).all()


@pytest.mark.parametrize("form", ["fp16", "int8", "fp8"])
@pytest.mark.parametrize("cols", [300, 5000, 20000, 33001])
@pytest.mark.parametrize("which", ["x", "residual"])
def test_norm_adds_in_place(form, cols, which):
    step(f"norm {form} in place {cols} {which}")
    xh, rh, wh = rows_of(6, cols, 1), rows_of(6, cols, 2), weight_of(cols, 3)
    x, r, w = dev(xh), dev(rh), dev(wh)
    want = call(form)(x, w, EPS, residual=r)
    place = x if which == "x" else r
    got = call(form)(x, w, EPS, residual=r, total=place)
    assert got[-1].data_ptr() == place.data_ptr()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    check(form, got, *reference(xh, wh, res=rh), e_of(cols))
    # the norm of the sum alone: the same bits
    alone = call(form)(got[-1], w, EPS)
    for a, b in zip(alone if form != "fp16" else (alone,), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("cols", [256, 3000, 9000, 33000])
def test_norm_special_rows(cols):
    """Zeros, an infinity, a NaN, values at both ends of fp16, and a sum that overflows; the rows beside them are as
    they are without them."""
    step(f"norm special rows {cols}")
    xh, wh = rows_of(9, cols, 5), weight_of(cols, 6)
    clean = xh.copy()
    xh[1] = 0
    xh[2, 5], xh[3, 7], xh[4] = np.inf, np.nan, 65504
    xh[5] = 0
    xh[5, 9] = 2.0 ** -24
    xh[7] = -(2.0 ** -24)
    x, w = dev(xh), dev(wh)
    y = nw().rms_norm(x, w, EPS).cpu().numpy()
    ref, _ = reference(xh, wh)
    plain = [0, 1, 4, 5, 6, 7, 8]
    check_half(torch.from_numpy(y[plain]), ref[plain], e_of(cols))
    assert (y[1] == 0).all() and np.isnan(y[2, 5]) and (np.delete(y[2], 5) == 0).all() and np.isnan(y[3]).all()
    q, scale = nw().rms_norm_int8(x, w, EPS)
    assert scale[2].isnan() and scale[3].isnan() and (q[2:4] == 0).all() and scale[1] == 0 and (q[1] == 0).all()
    check_int8(q[plain], scale[plain], ref[plain], e_of(cols))
    q, scale = nw().rms_norm_fp8(x, w, EPS)
    check_fp8(q[plain], scale[plain], ref[plain], e_of(cols))
    v = e4m3(q)
    assert np.isnan(v[2, 5]) and (np.delete(v[2], 5)[:cols - 1] == 0).all() and np.isnan(v[3, :cols]).all()
    assert (v[:, cols:] == 0).all()
    for form in ("fp16", "int8", "fp8"):  # and the other rows' bits do not depend on these
        a, b = call(form)(x, w, EPS), call(form)(dev(clean), w, EPS)
        for u, v in zip(a if isinstance(a, tuple) else (a,), b if isinstance(b, tuple) else (b,)):
            assert all(torch.equal(u[k], v[k]) for k in (0, 6, 8))
    big = torch.full((1, cols), 40000.0, dtype=torch.float16, device="cuda")
    y, total = nw().rms_norm(big, w, EPS, residual=big)
    assert (total == float("inf")).all() and y.isnan().all()


@pytest.mark.parametrize("eps", [0.0, 1e-12, 1.0, 1e30])
def test_norm_eps(eps):
    step(f"norm eps {eps}")
    xh, wh = rows_of(4, 700, 8), weight_of(700, 9)
    if eps == 0:
        xh[2] = 0
    ref, _ = reference(xh, wh, eps)
    y = nw().rms_norm(dev(xh), dev(wh), eps)
    q, scale = nw().rms_norm_int8(dev(xh), dev(wh), eps)
    f, fs = nw().rms_norm_fp8(dev(xh), dev(wh), eps)
    keep = [0, 1, 3] if eps == 0 else [0, 1, 2, 3]
    check_half(y[keep], ref[keep], e_of(700))
    check_int8(q[keep], scale[keep], ref[keep], e_of(700))
    check_fp8(f[keep], fs[keep], ref[keep], e_of(700))
    if eps == 0:  # 0 / 0
        assert y[2].isnan().all() and scale[2].isnan() and np.isnan(e4m3(f)[2, :700]).all()


def nearest_even(p, top):
    """The integers nearest to 127 p / top, ties to even, without rounding: products of 22-bit numbers with small
    integers are exact in 64 bits."""
    low = np.floor(127 * p / top)
    low = np.where(127 * p < low * top, low - 1, low)          # should the quotient have been rounded up
    low = np.where(127 * p >= (low + 1) * top, low + 1, low)   # or down
    side = 254 * p - (2 * low + 1) * top
    return np.where(side > 0, low + 1, np.where(side < 0, low, low + low % 2))


@pytest.mark.parametrize("rows,cols", [(400, 1000), (200, 8192), (3, 40000)])
def test_norm_int8_integers_are_exact(rows, cols):
    """The root falls out of the integers: nearest to 127 sum weight / the row's largest."""
    step(f"norm int8 exact {rows}x{cols}")
    xh, wh = rows_of(rows, cols, 4), weight_of(cols, 5)
    wh[::3] = np.round(wh[::3] * 8) / 8  # and where many quotients are half way
    xh[:rows // 2] = np.round(xh[:rows // 2].astype(np.float64) * 4) / 4
    q, _ = nw().rms_norm_int8(dev(xh), dev(wh), EPS)
    p = xh.astype(np.float64) * wh.astype(np.float64)
    top = np.abs(p).max(axis=1, keepdims=True)
    assert np.array_equal(q.cpu().numpy()[:, :cols], nearest_even(p, np.where(top > 0, top, 1)).astype(np.int8))


@pytest.mark.parametrize("cols", [32768, 65536])
def test_norm_beside_the_borders_of_e4m3(cols):
    """y a quarter of an fp32 step beside a border between two codes: to the code of its own side, not to the even one."""
    step(f"norm e4m3 borders {cols}")
    w = np.ones(cols, np.float16)
    w[:8] = [1.0625, 1.1875, 1.3125, 1.4375, -1.0625, -1.1875, -1.3125, -1.4375]  # borders, even codes below and above
    below = [1.0, 1.125, 1.25, 1.375]
    above = [1.125, 1.25, 1.375, 1.5]
    # all ones: the root is 1 / sqrt(1 + eps), 5e-8 below 1
    q, scale = nw().rms_norm_fp8(dev(np.ones((1, cols), np.float16)), dev(w), 1e-7)
    v = e4m3(q)[0, :8] * 2.0 ** (int(scale[0, 0]) - 127)
    assert v.tolist() == below + [-b for b in below]
    # one value 2^-11 below 1: the root is 2^-11 / cols above 1
    x = np.ones((1, cols), np.float16)
    x[0, -1] -= 2.0 ** -11
    q, scale = nw().rms_norm_fp8(dev(x), dev(w), 0.0)
    v = e4m3(q)[0, :8] * 2.0 ** (int(scale[0, 0]) - 127)
    assert v.tolist() == above + [-b for b in above]
    # on the border: to the even code
    q, scale = nw().rms_norm_fp8(dev(np.ones((1, cols), np.float16)), dev(w), 0.0)
    v = e4m3(q)[0, :8] * 2.0 ** (int(scale[0, 0]) - 127)
    even = [1.0, 1.25, 1.25, 1.5]
    assert v.tolist() == even + [-b for b in even]


def test_norm_and_quantize_many_rows():
    """More rows than one launch takes."""
    step("norm of 2^21 + 3 rows")
    rows, cols = (1 << 21) + 3, 8
    x = (torch.arange(rows * cols, device="cuda").view(rows, cols) % 2039 - 1000).half()
    w = torch.ones(cols, dtype=torch.float16, device="cuda")
    y, total = nw().rms_norm(x, w, EPS, residual=x)
    q, scale, _ = nw().rms_norm_int8(x, w, EPS, residual=x)
    f, fs, _ = nw().rms_norm_fp8(x, w, EPS, residual=x)
    k, ks = nw().int8_quantize(x)
    at = torch.tensor([0, 1, (1 << 21) - 1, 1 << 21, (1 << 21) + 2], device="cuda")
    assert torch.equal(total, x + x)
    xh = x[at].cpu().numpy()
    ref, _ = reference(xh, np.ones(cols, np.float16), res=xh)
    check_half(y[at], ref, e_of(cols))
    check_int8(q[at], scale[at], ref, e_of(cols))
    check_fp8(f[at], fs[at], ref, e_of(cols))
    check_int8(k[at], ks[at], xh.astype(np.float64), 2.0 ** -24, 127 * 2.0 ** -24)


@pytest.mark.parametrize("form", ["fp16", "int8", "fp8"])
def test_norm_on_another_stream_and_in_graphs(form):
    step(f"norm {form} streams and graphs")
    w = dev(weight_of(1500, 1))
    xs = [dev(rows_of(20, 1500, 30 + k)) for k in range(3)]
    want = [call(form)(x, w, EPS, residual=xs[0]) for x in xs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(form)(xs[1], w, EPS, residual=xs[0], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))
    x = xs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call(form)(x, w, EPS, residual=xs[0])
    for turn in range(4):
        x.copy_(xs[turn % 3])
        for o in out:
            o.fill_(3)
        g.replay()
        eager = call(form)(xs[2], w, EPS, residual=xs[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[turn % 3]))
        assert all(torch.equal(a, b) for a, b in zip(eager, want[2]))


# ------------------------------------------------------------------------------------------------ the quantiser
@pytest.mark.parametrize("rows,cols", SHAPES + [(1, 131071), (3000, 130)])
def test_quantize(rows, cols):
    step(f"int8 quantize {rows}x{cols}")
    xh = rows_of(rows, cols, rows * 3 + cols)
    xh[rows // 2, cols // 2] = 0
    q, scale = nw().int8_quantize(dev(xh))
    check_int8(q, scale, xh.astype(np.float64), 0 if cols == 0 else 2.0 ** -24, 127 * 2.0 ** -24)
    exact = np.abs(xh).max(axis=1).astype(np.float32) / np.float32(127)
    assert np.array_equal(scale.cpu().numpy(), exact)


def test_quantize_every_largest():
    """Every positive fp16 value as a row's largest: its code is 127, and ties go to the even integer."""
    step("int8 quantize borders")
    bits = np.arange(1, 0x7C00, dtype=np.uint16)
    top = bits.view(np.float16).astype(np.float64)
    r = np.random.default_rng(3).uniform(-1, 1, (1, 96))
    x = (top[:, None] * r).astype(np.float16)
    x[:, 5], x[:, 6] = top, -top
    q, scale = nw().int8_quantize(dev(x))
    assert (q[:, 5] == 127).all() and (q[:, 6] == -127).all()
    check_int8(q, scale, x.astype(np.float64), 2.0 ** -24, 127 * 2.0 ** -24)
    ties = np.zeros((1, 20), dtype=np.float16)
    ties[0, 0] = 127
    ties[0, 1:9] = [0.5, 1.5, 2.5, 3.5, -0.5, -1.5, -2.5, 126.5]
    q, scale = nw().int8_quantize(dev(ties))
    assert scale[0] == 1 and q[0, :9].tolist() == [127, 0, 2, 2, 4, 0, -2, -2, 126]
    for m in range(1, 9):  # steps of m / 2^k, no power of two: halves of an odd number of them are ties all the same
        n = np.arange(0, 127)
        x = np.append(127 * m, (n + 0.5) * m)
        x = np.concatenate([x, -x])[None] * 2.0 ** -8
        assert np.array_equal(x.astype(np.float16), x)
        q, scale = nw().int8_quantize(dev(x.astype(np.float16)))
        want = np.append(127, n + n % 2)
        assert np.array_equal(q.cpu().numpy()[0, :256], np.concatenate([want, -want])), m


@pytest.mark.parametrize("cols", [300, 5000, 20000, 40000])
def test_quantize_special_rows(cols):
    step(f"int8 quantize specials {cols}")
    xh = rows_of(6, cols, 4)
    xh[1, 3], xh[2, cols - 1], xh[3, 0], xh[4] = np.inf, -np.inf, np.nan, 0
    q, scale = nw().int8_quantize(dev(xh))
    assert scale[1:4].isnan().all() and (q[1:5] == 0).all() and scale[4] == 0
    check_int8(q[[0, 5]], scale[[0, 5]], xh[[0, 5]].astype(np.float64), 2.0 ** -24, 127 * 2.0 ** -24)


@pytest.mark.parametrize("offset,width", [(0, 640), (1, 515), (8, 648), (3, 640)])
def test_quantize_strided_rows(offset, width):
    step(f"int8 quantize strided {offset} {width}")
    full = rows_of(9, width, offset)
    q, scale = nw().int8_quantize(dev(full)[:, offset:offset + 500])
    check_int8(q, scale, full[:, offset:offset + 500].astype(np.float64), 2.0 ** -24, 127 * 2.0 ** -24)


def test_rows_past_four_gigabytes():
    """The last rows of activations that lie past 2^32 bytes, inputs and outputs."""
    step("norm past 4 GB")
    rows, cols = 290001, 8000  # 4.6 GB
    x = torch.empty(rows, cols, dtype=torch.float16, device="cuda")
    for part in x.split(20000):
        part.normal_(generator=torch.Generator(device="cuda").manual_seed(part.shape[0]))
    w = dev(weight_of(cols, 2))
    at = torch.tensor([0, 1, rows // 2, rows - 2, rows - 1], device="cuda")
    xh = x[at].cpu().numpy()
    ref, total = reference(xh, w.cpu().numpy(), res=xh)
    for form in ("fp16", "int8", "fp8"):
        got = call(form)(x, w, EPS, residual=x)
        check(form, tuple(t[at] for t in got), ref, total, e_of(cols))
        del got
    q, scale = nw().int8_quantize(x)
    check_int8(q[at], scale[at], xh.astype(np.float64), 2.0 ** -24, 127 * 2.0 ** -24)
