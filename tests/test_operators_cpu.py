"""Refusals of the mixture-of-experts and 8-bit calls, on the host before any launch, and their size queries."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
A, B = P(0x100000), P(0x200000)  # aligned addresses that are never read
ODD = P(0x200001)


@pytest.fixture(scope="module")
def nw():
    import non_uniform_weight_amd
    return non_uniform_weight_amd


@pytest.fixture(scope="module")
def lib(nw):
    return nw.library()


@pytest.mark.parametrize("header,module", [("sqllm_fp8.h", "fp8"), ("sqllm_moe.h", "moe")])
def test_every_declared_function_is_bound(lib, nw, header, module):
    text = open(os.path.join(ROOT, "include", header)).read()
    names = set(re.findall(r"\b(sqllm_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert names == set(getattr(nw, module).EXPORTS)
    for n in names:
        assert getattr(lib, n).argtypes is not None


def test_fp8_sizes(nw):
    assert [nw.fp8_cols(c) for c in (1, 128, 129, 5001)] == [128, 128, 256, 5120]
    assert [nw.fp8_scale_pitch(c) for c in (1, 512, 513, 5001)] == [4, 4, 8, 40]
    assert nw.fp8_cols(0) == nw.fp8_scale_pitch(-1) == nw.fp8_cols((1 << 24) + 1) == 0
    assert nw.fp8_workspace_bytes(8192, 8192, 0) == nw.fp8_workspace_bytes(0, 8192, 1) == 0
    assert nw.fp8_workspace_bytes(64, 1000, 33) >= 33 * 1024 + 33 * 8


def quantize(lib, x=A, rows=8, cols=300, ldx=300, q=A, scale=B):
    return lib.sqllm_fp8_quantize(x, rows, cols, ldx, q, scale, None)


def gemm(lib, q=A, scale=B, rows=64, cols=300, x=A, batch=3, y=B, ws=A, wsb=1 << 20):
    return lib.sqllm_fp8_gemm(q, scale, rows, cols, x, batch, y, ws, wsb, None)


def test_fp8_argument_errors(lib):
    for name in ("x", "q", "scale"):
        assert quantize(lib, **{name: None}) == 1
    assert quantize(lib, rows=0) == quantize(lib, cols=0) == quantize(lib, ldx=299) == 3
    assert quantize(lib, cols=(1 << 24) + 1, ldx=1 << 30) == 3
    assert quantize(lib, rows=1 << 29) == 3            # scales beyond the bound
    assert quantize(lib, x=ODD) == quantize(lib, q=P(0x100008)) == quantize(lib, scale=P(0x100002)) == 5
    for name in ("q", "scale", "x", "y"):
        assert gemm(lib, **{name: None}) == 1
    assert gemm(lib, rows=0) == gemm(lib, cols=-1) == gemm(lib, rows=1 << 29) == 3
    assert gemm(lib, batch=0) == gemm(lib, batch=1 << 29) == 4
    assert quantize(lib, rows=(1 << 28) - 63, cols=5, ldx=5) == gemm(lib, rows=(1 << 28) - 63, cols=5) == 3
    assert gemm(lib, rows=1 << 20, batch=1 << 19) == 3  # more of y than the launches count
    assert lib.sqllm_fp8_workspace_bytes(1 << 20, 300, 1 << 19) == 0
    assert gemm(lib, q=P(0x100008)) == gemm(lib, scale=P(0x100002)) == gemm(lib, x=ODD) == gemm(lib, y=ODD) == 5
    assert gemm(lib, ws=None) == gemm(lib, ws=P(0x100010)) == gemm(lib, wsb=16) == 8


def test_moe_sizes(nw):
    good = dict(batch=4, experts=8, topk=2, hidden=512, inter=768)
    size = lambda **kw: nw.moe_workspace_bytes(**{**good, **kw})  # noqa: E731
    assert size() > 0 and size(batch=16) >= size()
    for bad in ({"batch": 0}, {"batch": 17}, {"experts": 0}, {"experts": 513}, {"topk": 0}, {"topk": 9}, {"hidden": 500},
                {"hidden": 0}, {"inter": 128}, {"hidden": 65792}, {"experts": 1}):
        assert size(**bad) == 0, bad


def test_sizes_beyond_the_c_types(nw):
    """Sizes that the low bits alone would make good ones."""
    assert nw.fp8_cols(2 ** 64 + 5) == nw.fp8_scale_pitch(2 ** 64 + 5) == nw.fp8_cols(5 - 2 ** 64) == 0
    for at in range(3):
        sizes = [64, 1000, 33]
        sizes[at] += 2 ** 64
        assert nw.fp8_workspace_bytes(*sizes) == 0
    for at in range(5):
        sizes = [4, 8, 2, 512, 768]
        sizes[at] += 2 ** 32 if at < 3 else 2 ** 64
        assert nw.moe_workspace_bytes(*sizes) == 0


def projection(nw, **kw):
    f = dict(packed=A.value, lut=B.value, row_ptr=A.value, col_idx=A.value, val=A.value, nnz=10)
    return nw.moe.Experts(**{**f, **kw})


def route(lib, x=A, router=B, bias=A, batch=4, experts=8, hidden=512, topk=2, flags=0, ids=A, weights=B, ws=A, wsb=1 << 20):
    return lib.sqllm_moe_route(x, router, bias, batch, experts, hidden, topk, flags, 1.0, ids, weights, ws, wsb, None)


def experts(lib, nw, x=A, ids=A, weights=B, gate=None, up=None, down=None, bits=3, batch=4, experts=8, topk=2, hidden=512,
            inter=768, y=B, ws=A, wsb=1 << 24):
    g, u, d = (p or projection(nw) for p in (gate, up, down))
    return lib.sqllm_moe_experts(x, ids, weights, g, u, d, bits, batch, experts, topk, hidden, inter, y, ws, wsb, None)


def layer(lib, nw, x=A, router=B, bias=None, flags=0, bits=3, batch=4, experts=8, topk=2, hidden=512, inter=768, ids=A,
          weights=B, y=B, ws=A, wsb=1 << 24, down=None):
    g, u, d = projection(nw), projection(nw), down or projection(nw)
    return lib.sqllm_moe_layer(x, router, bias, flags, 1.0, g, u, d, bits, batch, experts, topk, hidden, inter, ids, weights,
                               y, ws, wsb, None)


SIZES = [({"batch": 0}, 4), ({"batch": 17}, 4), ({"experts": 0}, 3), ({"experts": 513}, 3), ({"topk": 0}, 3),
         ({"topk": 9, "experts": 16}, 3), ({"topk": 3, "experts": 2}, 3), ({"hidden": 500}, 3), ({"hidden": 1 << 20}, 3),
         ({"ws": None}, 8), ({"ws": P(0x100010)}, 8), ({"wsb": 16}, 8)]


def test_moe_route_argument_errors(lib):
    for name in ("x", "router", "ids", "weights"):
        assert route(lib, **{name: None}) == 1
    for kw, status in SIZES:
        assert route(lib, **kw) == status, kw
    assert route(lib, flags=4) == 3
    assert route(lib, x=P(0x100008)) == route(lib, router=P(0x100008)) == route(lib, bias=ODD) == 5
    assert route(lib, ids=ODD) == route(lib, weights=ODD) == 5


def test_moe_experts_argument_errors(lib, nw):
    for name in ("x", "ids", "weights", "y"):
        assert experts(lib, nw, **{name: None}) == 1
        if name != "y":
            assert experts(lib, nw, **{name: ODD}) == 5
    for kw, status in SIZES + [({"inter": 128}, 3), ({"bits": 1}, 2), ({"bits": 5}, 2), ({"y": P(0x100002)}, 5)]:
        assert experts(lib, nw, **kw) == status, kw
    for which in ("gate", "up", "down"):
        for kw, status in ({"packed": None}, 1), ({"lut": None}, 1), ({"row_ptr": None}, 1), ({"col_idx": None}, 1), \
                ({"val": None}, 1), ({"nnz": -1}, 3), ({"nnz": 1 << 31}, 3), ({"packed": 0x100008}, 5), \
                ({"lut": 0x100004}, 5), ({"row_ptr": 0x100002}, 5), ({"col_idx": 0x100001}, 5), ({"val": 0x100001}, 5):
            assert experts(lib, nw, **{which: projection(nw, **kw)}) == status, (which, kw)
    assert lib.sqllm_moe_experts(A, A, B, None, projection(nw), projection(nw), 3, 4, 8, 2, 512, 768, B, A, 1 << 24, None) == 1


def test_moe_layer_argument_errors(lib, nw):
    for name in ("x", "router", "ids", "weights", "y"):
        assert layer(lib, nw, **{name: None}) == 1
    for kw, status in SIZES + [({"inter": 128}, 3), ({"bits": 5}, 2), ({"flags": 8}, 3)]:
        assert layer(lib, nw, **kw) == status, kw
    assert layer(lib, nw, down=projection(nw, packed=None)) == 1


def test_python_refuses_host_tensors(nw):
    h = torch.zeros(4, 512, dtype=torch.float16)
    u8 = torch.zeros(4, 512, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device tensor"):
        nw.fp8_quantize(h)
    with pytest.raises(ValueError, match="device tensor"):
        nw.fp8_gemm(u8, u8, h)
    with pytest.raises(ValueError, match="device tensor"):
        nw.moe_route(h, h, 2)
    with pytest.raises(TypeError, match="torch.Tensor"):
        nw.moe_route([1.0], h, 2)
    p = {"packed": u8, "lut": h}
    with pytest.raises(ValueError, match="device tensor"):
        nw.moe_experts(h, u8, h, p, p, p, 3)
