"""Outliers of the experts' products: a row's sum is that of its own entries, whatever its neighbours hold."""
import numpy as np
import pytest
import torch

from gpu_util import nw, step
from test_gpu_moe import Layer, Proj, choices, tokens

pytestmark = pytest.mark.gpu


def set_lut(p, lut, codes):
    p.dense = np.take_along_axis(lut.astype(np.float64), codes.astype(np.int64), axis=2)
    p.abs = np.abs(p.dense)
    p.dev["lut"] = torch.from_numpy(lut).cuda()
    p.dev["packed"] = torch.cat([nw().pack(torch.from_numpy(c).cuda(), p.bits) for c in codes])


def set_outliers(p, counts, col, val):
    """counts [experts * rows], and the entries of all rows in order."""
    cols = p.dense.shape[2]
    row_ptr, at = np.concatenate([[0], np.cumsum(counts)]), np.repeat(np.arange(len(counts)), counts)
    np.add.at(p.dense.reshape(-1, cols), (at, col), val.astype(np.float64))
    np.add.at(p.abs.reshape(-1, cols), (at, col), np.abs(val.astype(np.float64)))
    p.n = p.n + counts.reshape(p.n.shape)
    p.dev["row_ptr"] = torch.from_numpy(row_ptr.astype(np.int32)).cuda()
    p.dev["col"] = torch.from_numpy(col.astype(np.uint16).view(np.int16)).cuda()
    p.dev["val"] = torch.from_numpy(val.astype(np.float16)).cuda()


def projection(experts, rows, cols, bits, seed, heavy=None, zero=None):
    """Centroids around 1e-3 and one outlier around 0.3 a row; row `heavy` of each expert has 320 instead that cancel,
    30000 and -30000 at the same columns; row `zero` is empty and zero."""
    p = Proj(experts, rows, cols, bits, seed, density=0)
    p.bits = bits
    r = np.random.default_rng(seed + 100)
    lut = (r.standard_normal((experts, rows, 1 << bits)) * 1e-3).astype(np.float16)
    counts = np.ones((experts, rows), dtype=np.int64)
    if zero is not None:
        lut[:, zero], counts[:, zero] = 0, 0
    if heavy is not None:
        counts[:, heavy] = 320
    set_lut(p, lut, r.integers(0, 1 << bits, (experts, rows, cols), dtype=np.uint8))
    col, val = [], []
    for e in range(experts):
        for row in range(rows):
            if counts[e, row] > 1:
                c = r.choice(cols, 160, replace=False)
                col += [c, c]
                val += [np.full(160, 30000.0), np.full(160, -30000.0)]
            elif counts[e, row]:
                col.append(r.integers(0, cols, 1))
                val.append(r.standard_normal(1) * 0.3)
    set_outliers(p, counts.reshape(-1), np.concatenate(col), np.concatenate(val).astype(np.float16))
    return p


@pytest.mark.parametrize("hidden,inter", [(512, 768), (1024, 512)])
@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("where", ["gate", "up", "down"])
def test_light_rows_beside_a_heavy_one(where, bits, hidden, inter):
    """A row of 320 outliers whose partial sums are millions of times its neighbours': they lose nothing by it.  (In
    gate or up it meets a row of zeros of the other, so that its own error does not enter y.)"""
    step(f"moe heavy row in {where} {bits}-bit {hidden}x{inter}")
    layer = Layer(2, hidden, inter, bits, 3, density=0)
    layer.gate = projection(2, inter, hidden, bits, 1, **{"gate": dict(heavy=3), "up": dict(zero=3)}.get(where, {}))
    layer.up = projection(2, inter, hidden, bits, 2, **{"up": dict(heavy=3), "gate": dict(zero=3)}.get(where, {}))
    layer.down = projection(2, hidden, inter, bits, 4, **(dict(heavy=3) if where == "down" else {}))
    for batch in (1, 6, 16):
        x = tokens(batch, hidden, 3)
        ids, weights = choices(batch, 2, 1, 4)
        weights *= 64
        layer.check(x, ids, weights, layer.run(x, ids, weights), floor=2.0 ** -36)


@pytest.mark.parametrize("hidden,inter", [(512, 768), (1024, 512)])
@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("kw", [{"density": 0.005}, {"density": 0.01, "skew": True}])
def test_an_infinite_x_gives_infinity(kw, bits, hidden, inter):
    """One infinite entry of x among positive weights and activations: every sum of that token is infinite and none is
    NaN, since no row meets another's column; the other tokens are as they were."""
    step(f"moe infinite x {bits}-bit {kw} {hidden}x{inter}")
    layer = Layer(3, hidden, inter, bits, 7, **kw)
    for p in (layer.gate, layer.up, layer.down):
        p.dev["lut"] = p.dev["lut"].abs() * 0.25 + 0.002
        p.dev["val"] = p.dev["val"].abs() + 0.01
    for batch in (2, 6, 16):
        x = tokens(batch, hidden, 3).abs()
        ids, weights = choices(batch, 3, 2, 4)
        clean = layer.run(x, ids, weights)
        assert clean.isfinite().all()
        x[1, int(layer.gate.dev["col"][5].item())] = float("inf")
        y = layer.run(x, ids, weights)
        assert (y[1] == float("inf")).all(), f"{y[1].isnan().sum()} NaN"
        keep = [t for t in range(batch) if t != 1]
        assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("bits", [2, 3, 4])
def test_arrays_longer_than_the_rows_entries(bits):
    """Behind the last row's entries the arrays may hold anything: it is of no row."""
    step(f"moe outlier arrays with a tail, {bits}-bit")
    layer = Layer(2, 512, 768, bits, 9, density=0.004)
    for p in (layer.gate, layer.up, layer.down):
        for name, fill in (("col", -1), ("val", float("nan"))):
            t = p.dev[name]
            p.dev[name] = torch.cat([t, torch.full((37,), fill, dtype=t.dtype, device="cuda")])
    for batch in (1, 6, 16):
        x = tokens(batch, 512, 3)
        ids, weights = choices(batch, 2, 1, 4)
        layer.check(x, ids, weights, layer.run(x, ids, weights))
