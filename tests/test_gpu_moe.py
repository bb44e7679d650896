"""The mixture-of-experts calls on the GPU against 64-bit references.

Tolerance of the experts' products, with M the sum of a product's |w||v| and n = cols + the row's outliers: an fp32
sum is off by at most n 2^-23 M (its adds may truncate on the matrix cores).  For a = silu(g) u,
|da| <= 1.1 |u| dg + |silu(g)| du + 2^-19 |a| + 2^-25 (|silu'| <= 1.1; the last terms cover the exponential and the
storing of a as two fp16 values).  A y is off by sum_k |w_k| (|down| da + n 2^-23 |down||a|), a few fp32 roundings of
the sum over k (2^-20 of its magnitude) and its own rounding, 2^-11 |y| + 2^-25.  Router weights come from 64-bit
scores: 2^-22 of the value covers the rounding to fp32."""
import threading

import numpy as np
import pytest
import torch

from gpu_util import nw, step

pytestmark = pytest.mark.gpu


class Proj:
    """One projection of every expert, on the host in 64 bits and on the device in the stored form."""

    def __init__(self, experts, rows, cols, bits, seed, density=0.005, skew=False, few=0, lut_sigma=0.05):
        r = np.random.default_rng(seed)
        codes = r.integers(0, 1 << bits, (experts, rows, cols), dtype=np.uint8)
        lut = np.sort(r.standard_normal((experts, rows, 1 << bits)) * lut_sigma, axis=2).astype(np.float16)
        self.dense = np.take_along_axis(lut.astype(np.float64), codes.astype(np.int64), axis=2)
        self.abs = np.abs(self.dense)
        self.n = np.full((experts, rows), cols)
        packed = torch.cat([nw().pack(torch.from_numpy(codes[e]).cuda(), bits) for e in range(experts)])
        self.dev = {"packed": packed, "lut": torch.from_numpy(lut).cuda()}
        if density:
            counts = r.binomial(cols, density, experts * rows)
            if skew:  # a few rows with far more than the rest, many with none
                counts[:] = 0
                counts[r.integers(0, counts.size, 3)] = cols // 2
                counts[-1] = 5
            if few:  # hardly any, among them the first and the last row's
                counts[:] = 0
                counts[[0, -1, -2][:few]] = 1
            row_ptr = np.concatenate([[0], np.cumsum(counts)])
            col = r.integers(0, cols, row_ptr[-1])  # repeated entries are summed
            val = (r.standard_normal(row_ptr[-1]) * 0.2).astype(np.float16)
            at = np.repeat(np.arange(experts * rows), counts)
            np.add.at(self.dense.reshape(-1, cols), (at, col), val.astype(np.float64))
            np.add.at(self.abs.reshape(-1, cols), (at, col), np.abs(val.astype(np.float64)))
            self.n = self.n + counts.reshape(experts, rows)
            self.dev["row_ptr"] = torch.from_numpy(row_ptr.astype(np.int32)).cuda()
            self.dev["col"] = torch.from_numpy(col.astype(np.uint16).view(np.int16)).cuda()
            self.dev["val"] = torch.from_numpy(val).cuda()


class Layer:
    def __init__(self, experts, hidden, inter, bits, seed, **kw):
        self.experts, self.hidden, self.inter, self.bits = experts, hidden, inter, bits
        self.gate = Proj(experts, inter, hidden, bits, seed, **kw)
        self.up = Proj(experts, inter, hidden, bits, seed + 1, **kw)
        self.down = Proj(experts, hidden, inter, bits, seed + 2, **kw)

    def run(self, x, ids, weights, **kw):
        return nw().moe_experts(x, ids, weights, self.gate.dev, self.up.dev, self.down.dev, self.bits, **kw)

    def check(self, x, ids, weights, y, floor=2.0 ** -25):
        x64, w64 = x.cpu().numpy().astype(np.float64), weights.cpu().numpy().astype(np.float64)
        ids, y = ids.cpu().numpy(), y.float().cpu().numpy().astype(np.float64)
        eps = 2.0 ** -23
        for t in range(x64.shape[0]):
            ref, err, mag = (np.zeros(self.hidden) for _ in range(3))
            any_expert = False
            for k in range(ids.shape[1]):
                e = ids[t, k]
                if e < 0 or e >= self.experts:
                    continue
                any_expert = True
                v, av = x64[t], np.abs(x64[t])
                g, u = self.gate.dense[e] @ v, self.up.dense[e] @ v
                dg, du = self.gate.n[e] * eps * (self.gate.abs[e] @ av), self.up.n[e] * eps * (self.up.abs[e] @ av)
                s = g / (1 + np.exp(-g))
                a = s * u
                da = 1.1 * np.abs(u) * dg + np.abs(s) * du + 2.0 ** -19 * np.abs(a) + floor
                down = self.down.abs[e]
                ref += w64[t, k] * (self.down.dense[e] @ a)
                err += abs(w64[t, k]) * (down @ da + self.down.n[e] * eps * (down @ np.abs(a)))
                mag += abs(w64[t, k]) * (down @ np.abs(a))
            if not any_expert:
                assert (y[t] == 0).all(), f"token {t} has no expert"
                continue
            tol = err + 2.0 ** -20 * mag + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25
            off = np.abs(y[t] - ref)
            assert (off <= tol).all(), f"token {t}: {np.nanmax(off / tol):.3f} of the tolerance, {np.isnan(off).sum()} NaN"


def tokens(batch, hidden, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(batch, hidden, generator=g).half().cuda()


def choices(batch, experts, topk, seed):
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand(batch, experts, generator=g).argsort(dim=1)[:, :topk].int().contiguous()
    return ids.cuda(), (torch.rand(batch, topk, generator=g) + 0.1).cuda()


@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("batch,experts,topk,hidden,inter", [(1, 1, 1, 256, 256), (1, 8, 2, 512, 768), (2, 5, 3, 768, 512),
                                                             (4, 4, 4, 256, 1280), (5, 9, 2, 1024, 256), (8, 3, 2, 512, 256),
                                                             (9, 2, 1, 256, 512), (13, 6, 6, 512, 512), (16, 40, 8, 256, 256),
                                                             (16, 1, 1, 512, 512), (3, 2, 2, 256, 4352), (1, 2, 1, 4608, 256),
                                                             (16, 1, 1, 1280, 2304), (12, 2, 2, 2048, 2048), (16, 3, 1, 1024, 512),
                                                             (16, 1, 1, 4096, 256), (7, 12, 4, 1792, 2048), (6, 48, 8, 2048, 512),
                                                             (16, 24, 4, 2048, 768)])
def test_experts(bits, batch, experts, topk, hidden, inter):
    step(f"moe experts {bits}-bit batch {batch} E {experts} K {topk} {hidden}x{inter}")
    layer = Layer(experts, hidden, inter, bits, batch + hidden)
    x = tokens(batch, hidden, 1)
    ids, weights = choices(batch, experts, topk, 2)
    guard = torch.full((batch * hidden + 512,), 7.0, dtype=torch.float16, device="cuda")
    y = guard[256:256 + batch * hidden].view(batch, hidden)
    out = layer.run(x, ids, weights, y=y)
    layer.check(x, ids, weights, out)
    assert (guard[:256] == 7).all() and (guard[256 + batch * hidden:] == 7).all()
    assert torch.equal(out, layer.run(x, ids, weights))


@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("kw", [{"density": 0}, {"density": 0.05}, {"density": 0.01, "skew": True},
                                {"few": 1}, {"few": 3}])
def test_outliers(bits, kw):
    step(f"moe outliers {bits}-bit {kw}")
    layer = Layer(3, 512, 768, bits, 11, **kw)
    for batch in (1, 6, 16):
        x = tokens(batch, 512, 3)
        ids, weights = choices(batch, 3, 2, 4)
        layer.check(x, ids, weights, layer.run(x, ids, weights))


def test_down_tiles_shared_by_four_waves():
    step("moe down by four waves")
    layer = Layer(22, 2048, 1536, 3, 29)
    x = tokens(8, 2048, 30)
    ids, weights = choices(8, 22, 4, 31)
    layer.check(x, ids, weights, layer.run(x, ids, weights))


@pytest.mark.parametrize("density", [0, 0.005])
def test_small_activations(density):
    """Entries of a around 2^-17, below fp16's normal range, with weights that lift y well above it: they are stored
    to 2^-36, and what the fp32 sums of gate and up are off by is far smaller still."""
    step("moe small activations")
    layer = Layer(3, 512, 768, 3, 23, density=density)
    x = tokens(5, 512, 5) / 256
    ids, weights = choices(5, 3, 2, 6)
    weights *= 4096
    y = layer.run(x, ids, weights)
    assert y.float().abs().median() > 2.0 ** -8
    layer.check(x, ids, weights, y, floor=2.0 ** -36)


def test_outliers_in_one_projection_only():
    step("moe outliers in one projection")
    layer = Layer(3, 512, 512, 3, 17, density=0)
    layer.up = Proj(3, 512, 512, 3, 18, density=0.01)
    x = tokens(3, 512, 3)
    ids, weights = choices(3, 3, 2, 4)
    layer.check(x, ids, weights, layer.run(x, ids, weights))


@pytest.fixture(scope="module")
def small():
    return Layer(7, 512, 768, 3, 23)


def test_ids_that_take_no_part(small):
    """Padded rows and dropped choices: whatever stands in x and the weights there, nothing of it is seen."""
    step("moe masked ids")
    for batch in (1, 4, 7, 16):
        x = tokens(batch, 512, 5)
        ids, weights = choices(batch, 7, 3, 6)
        ids[0, 1] = -1
        ids[batch - 1] = torch.tensor([7, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32)
        x[batch - 1] = float("nan")
        weights[batch - 1] = float("inf")
        if batch > 2:
            ids[1, 0], weights[1, 0] = -5, float("nan")
        small.check(x, ids, weights, small.run(x, ids, weights))


def test_no_expert_at_all(small):
    step("moe nothing chosen")
    x = torch.full((3, 512), float("nan"), dtype=torch.float16, device="cuda")
    ids = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    y = small.run(x, ids, torch.ones(3, 2, device="cuda"), y=torch.full_like(x, 9))
    assert (y == 0).all()


@pytest.mark.parametrize("batch", [1, 3, 16])
def test_repeated_ids(small, batch):
    """One expert in several of a token's choices counts with the sum of its weights."""
    step(f"moe repeated ids batch {batch}")
    x = tokens(batch, 512, 8)
    g = torch.Generator().manual_seed(9)
    ids = torch.randint(0, 3, (batch, 7), generator=g).int().cuda()
    ids[0] = 2
    weights = torch.rand(batch, 7, generator=g).cuda()
    small.check(x, ids, weights, small.run(x, ids, weights))


def test_every_token_to_one_expert(small):
    step("moe one expert")
    for batch in range(1, 17):
        x = tokens(batch, 512, 30 + batch)
        ids = torch.full((batch, 1), 4, dtype=torch.int32, device="cuda")
        weights = torch.full((batch, 1), -0.75, device="cuda")
        small.check(x, ids, weights, small.run(x, ids, weights))


def test_a_nan_token_stays_alone(small):
    step("moe NaN token")
    for batch in (2, 9):
        x = tokens(batch, 512, 5)
        ids, weights = choices(batch, 7, 2, 6)
        clean = small.run(x, ids, weights)
        x[1, 77] = float("nan")
        y = small.run(x, ids, weights)
        assert y[1].isnan().all()
        keep = [t for t in range(batch) if t != 1]
        assert torch.equal(y[keep], clean[keep])


def route64(x, router, topk, bias=None, sigmoid=False, renormalize=True, scale=1.0):
    l = x.cpu().numpy().astype(np.float64) @ router.cpu().numpy().astype(np.float64).T
    s = 1 / (1 + np.exp(-l)) if sigmoid else np.exp(l - l.max(axis=1, keepdims=True))
    if not sigmoid:
        s /= s.sum(axis=1, keepdims=True)
    rank = s if bias is None else s + bias.cpu().numpy().astype(np.float64)
    ids = np.argsort(-rank, axis=1, kind="stable")[:, :topk]
    w = np.take_along_axis(s, ids, axis=1)
    return ids, scale * (w / w.sum(axis=1, keepdims=True) if renormalize else w)


@pytest.mark.parametrize("batch,experts,topk,hidden", [(1, 1, 1, 256), (1, 8, 2, 4096), (2, 3, 3, 512), (5, 64, 6, 2048),
                                                       (16, 65, 8, 768), (16, 512, 8, 1024), (7, 200, 1, 256), (11, 129, 5, 65536)])
@pytest.mark.parametrize("kw", [{}, {"sigmoid": True}, {"renormalize": False}, {"sigmoid": True, "renormalize": False, "scale": 2.5}])
def test_route(batch, experts, topk, hidden, kw):
    step(f"moe route batch {batch} E {experts} K {topk} H {hidden} {kw}")
    x = tokens(batch, hidden, 1)
    router = (tokens(experts, hidden, 2).float() / hidden ** 0.5).half()
    g = torch.Generator().manual_seed(3)
    for bias in (None, (torch.randn(experts, generator=g) * 0.1).cuda()):
        ids, weights = nw().moe_route(x, router, topk, bias=bias, **kw)
        rid, rw = route64(x, router, topk, bias, **kw)
        np.testing.assert_array_equal(ids.cpu().numpy(), rid)
        w = weights.cpu().numpy().astype(np.float64)
        assert (np.abs(w - rw) <= 2.0 ** -22 * np.abs(rw)).all()


def test_route_ties_go_to_the_lowest_expert():
    step("moe route ties")
    x = tokens(3, 512, 1)
    one = tokens(2, 512, 2)
    router = one[torch.tensor([0, 1] * 50 + [0])].contiguous()  # two values only
    ids, weights = nw().moe_route(x, router, 4)
    rid, _ = route64(x, router, 4)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    zero = torch.zeros(4, 512, dtype=torch.float16, device="cuda")
    ids, weights = nw().moe_route(zero, router, 8, sigmoid=True)
    assert (ids.cpu() == torch.arange(8, dtype=torch.int32)).all() and (weights == 0.125).all()


@pytest.mark.parametrize("offset", [-3000.0, 0.0, 700.0])
def test_route_large_sums(offset):
    """Sums whose exponentials over- and underflow by themselves; all of a token's sums negative."""
    step(f"moe route offset {offset}")
    x = torch.ones(2, 256, dtype=torch.float16, device="cuda")
    router = tokens(100, 256, 2) * 0.1
    router[:, 0] += offset
    for sigmoid in (False, True):
        ids, weights = nw().moe_route(x, router, 5, sigmoid=sigmoid, renormalize=False)
        with np.errstate(over="ignore"):
            rid, rw = route64(x, router, 5, sigmoid=sigmoid, renormalize=False)
        if rw.min() > 1e-300 and rw.max() < 1:  # distinct scores
            np.testing.assert_array_equal(ids.cpu().numpy(), rid)
        w = weights.cpu().numpy().astype(np.float64)
        assert (np.abs(w - rw) <= 2.0 ** -22 * np.abs(rw) + 2.0 ** -149).all()


def test_route_with_values_that_are_no_numbers():
    """Ids stay distinct and in range; a NaN score ranks below every other."""
    step("moe route NaN")
    x = tokens(2, 512, 1)
    router = tokens(70, 512, 2)
    router[5] = float("nan")
    ids, _ = nw().moe_route(x, router, 8, sigmoid=True)
    keep = torch.tensor([e for e in range(70) if e != 5], dtype=torch.int32)
    rid, _ = route64(x, router[keep.long().cuda()], 8, sigmoid=True)
    np.testing.assert_array_equal(ids.cpu().numpy(), keep.numpy()[rid])
    x[1] = float("nan")
    ids, _ = nw().moe_route(x, router, 8)
    for row in ids.cpu().tolist():
        assert len(set(row)) == 8 and min(row) >= 0 and max(row) < 70
    assert ids[1].tolist() == list(range(8))


def make_router(layer, seed):
    return (tokens(layer.experts, layer.hidden, seed).float() / layer.hidden ** 0.5).half()


@pytest.mark.parametrize("batch", [1, 3, 8, 16])
def test_layer_is_the_two_calls(small, batch):
    step(f"moe layer batch {batch}")
    x, router = tokens(batch, 512, 41), make_router(small, 42)
    bias = torch.linspace(-0.2, 0.2, 7).cuda()
    kw = dict(bias=bias, sigmoid=True, scale=1.5)
    y, ids, weights = nw().moe_layer(x, router, 3, small.gate.dev, small.up.dev, small.down.dev, 3, **kw)
    rid, rw = nw().moe_route(x, router, 3, **kw)
    assert torch.equal(ids, rid) and torch.equal(weights, rw)
    assert torch.equal(y, small.run(x, rid, rw))
    small.check(x, ids, weights, y)


def test_layers_from_two_threads_on_one_stream(small):
    """The launches of a call that shares the stream's scratch stay together."""
    step("moe two threads")
    router = (torch.randn(300, 512, generator=torch.Generator().manual_seed(43)) / 16).half().cuda()
    xs = [tokens(4, 512, 50 + i) for i in range(2)]
    want = [nw().moe_route(x, router, 4) for x in xs]
    bad = []

    def run(i):
        for _ in range(200):
            ids, weights = nw().moe_route(xs[i], router, 4)
            if not (torch.equal(ids, want[i][0]) and torch.equal(weights, want[i][1])):
                bad.append(i)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_arguments_by_name(small):
    step("moe arguments by name")
    x, router = tokens(2, 512, 41), make_router(small, 42)
    parts = dict(gate=small.gate.dev, up=small.up.dev, down=small.down.dev, bits=3)
    y, ids, weights = nw().moe_layer(topk=2, router=router, x=x, **parts)
    assert torch.equal(y, nw().moe_experts(weights=weights, ids=ids, x=x, **parts))


def test_own_workspace_with_any_contents(small):
    step("moe workspace")
    x, router = tokens(9, 512, 41), make_router(small, 42)
    args = (x, router, 2, small.gate.dev, small.up.dev, small.down.dev, 3)
    ws = torch.full((nw().moe_workspace_bytes(9, 7, 2, 512, 768),), 255, dtype=torch.uint8, device="cuda")
    want = nw().moe_layer(*args)
    for _ in range(2):  # the second call finds what the first left
        assert all(torch.equal(a, b) for a, b in zip(nw().moe_layer(*args, ws=ws), want))


@pytest.mark.parametrize("batch", [1, 12])
def test_streams_and_graphs(small, batch):
    """Two captured graphs replayed in turn on two streams, with eager calls between."""
    step(f"moe streams and graphs batch {batch}")
    router = make_router(small, 42)
    xs = [tokens(batch, 512, 50 + k) for k in range(3)]
    call = lambda x, **kw: nw().moe_layer(x, router, 2, small.gate.dev, small.up.dev, small.down.dev, 3, **kw)  # noqa: E731
    want = [[t.clone() for t in call(x)] for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(xs[1], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))
    graphs = []
    for k in range(2):
        x = xs[k].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call(x)
        graphs.append((g, x, out))
    for turn in range(4):
        for k, (g, x, out) in enumerate(graphs):
            x.copy_(xs[(k + turn) % 3])
            out[0].fill_(3)
        torch.cuda.synchronize()
        other = torch.cuda.Stream()
        graphs[0][0].replay()
        with torch.cuda.stream(other):
            graphs[1][0].replay()
        eager = call(xs[2])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, want[2]))
        for k, (g, x, out) in enumerate(graphs):
            assert all(torch.equal(a, b) for a, b in zip(out, want[(k + turn) % 3]))


def test_a_decoding_step(small):
    """The operators as a step uses them: projections in 8 bits, the layer, the output head in 8 bits."""
    step("moe decoding step")
    g = torch.Generator().manual_seed(77)
    mix = nw().fp8_quantize((torch.randn(512, 512, generator=g) / 20).half().cuda())
    head = nw().fp8_quantize((torch.randn(1000, 512, generator=g) / 20).half().cuda())
    router = make_router(small, 42)
    for batch in (1, 5, 16):
        x = tokens(batch, 512, 60 + batch)
        hid = nw().fp8_gemm(*mix, x)
        y, ids, weights = nw().moe_layer(hid, router, 2, small.gate.dev, small.up.dev, small.down.dev, 3)
        logits = nw().fp8_gemm(*head, y)
        rid, _ = route64(hid, router, 2)
        np.testing.assert_array_equal(ids.cpu().numpy(), rid)
        small.check(hid, ids, weights, y)
        assert logits.shape == (batch, 1000) and logits.isfinite().all()
