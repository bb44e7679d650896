"""Refusals of the integer products, the norm and the stored e4m3 product, on the host before any launch, and their
size queries."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
A, B = P(0x100000), P(0x200000)  # aligned addresses that are never read
ODD = P(0x200001)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def nw():
    import non_uniform_weight_amd
    return non_uniform_weight_amd


@pytest.fixture(scope="module")
def lib(nw):
    return nw.library()


@pytest.mark.parametrize("header,module", [("sqllm_int8.h", "int8"), ("sqllm_norm.h", "norm"), ("sqllm_fp8.h", "fp8")])
def test_every_declared_function_is_bound(lib, nw, header, module):
    text = open(os.path.join(ROOT, "include", header)).read()
    names = set(re.findall(r"\b(sqllm_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert names == set(getattr(nw, module).EXPORTS)
    for n in names:
        assert getattr(lib, n).argtypes is not None


def test_sizes(nw):
    assert [nw.int8_cols(c) for c in (1, 128, 129, 5001, 131071)] == [128, 128, 256, 5120, 131072]
    assert nw.int8_cols(0) == nw.int8_cols(-1) == nw.int8_cols(131072) == nw.int8_cols(2 ** 64 + 5) == 0
    for size in (nw.int8_workspace_bytes, nw.int8_glu_workspace_bytes):
        assert size(8192, 8192, 0) == size(0, 8192, 1) == size(64, 131072, 1) == size(1 << 31, 128, 1) == 0
        assert size(1 << 20, 300, 1 << 19) == 0
        assert size(64, 1000, 33) >= 33 * 1024 + 33 * 4
        for at in range(3):
            sizes = [64, 1000, 33]
            sizes[at] += 2 ** 64
            assert size(*sizes) == 0


def quantize(lib, x=A, rows=8, cols=300, ldx=300, q=A, scale=B):
    return lib.sqllm_int8_quantize(x, rows, cols, ldx, q, scale, None)


def test_quantize_argument_errors(lib):
    for name in ("x", "q", "scale"):
        assert quantize(lib, **{name: None}) == 1
    assert quantize(lib, rows=0) == quantize(lib, cols=0) == quantize(lib, ldx=299) == 3
    assert quantize(lib, cols=131072, ldx=131072) == quantize(lib, rows=(1 << 30) + 1) == 3
    assert quantize(lib, x=ODD) == quantize(lib, q=P(0x100008)) == quantize(lib, scale=P(0x100002)) == 5


def gemm(lib, q=A, scale=B, rows=64, cols=300, x=A, xscale=None, batch=3, y=B, ws=A, wsb=1 << 20):
    return lib.sqllm_int8_gemm(q, scale, rows, cols, x, xscale, batch, y, ws, wsb, None)


def glu(lib, q=A, scale=B, up=A, up_scale=B, rows=64, cols=300, x=A, xscale=None, batch=3, y=B, ws=A, wsb=1 << 20):
    return lib.sqllm_int8_glu(q, scale, up, up_scale, rows, cols, x, xscale, batch, y, ws, wsb, None)


@pytest.mark.parametrize("call", [gemm, glu])
def test_product_argument_errors(lib, call):
    for name in ("q", "scale", "x", "y") + (("up", "up_scale") if call is glu else ()):
        assert call(lib, **{name: None}) == 1
    assert call(lib, rows=0) == call(lib, cols=-1) == call(lib, cols=131072) == call(lib, rows=(1 << 30) + 1) == 3
    assert call(lib, batch=0) == call(lib, batch=(1 << 30) + 1) == 4
    assert call(lib, rows=1 << 20, batch=1 << 19) == 3
    assert call(lib, q=P(0x100008)) == call(lib, scale=P(0x100002)) == call(lib, x=ODD) == call(lib, y=ODD) == 5
    assert call(lib, x=P(0x100002), xscale=A) == call(lib, xscale=P(0x100002)) == 5
    if call is glu:
        assert call(lib, up=P(0x100008)) == call(lib, up_scale=P(0x100002)) == 5
    assert call(lib, ws=None) == call(lib, ws=P(0x100010)) == call(lib, wsb=16) == 8


def stored(lib, q=A, scale=B, rows=64, cols=300, x=A, xscale=A, batch=3, y=B, ws=A, wsb=1 << 20):
    return lib.sqllm_fp8_gemm_stored(q, scale, rows, cols, x, xscale, batch, y, ws, wsb, None)


def test_stored_fp8_product_argument_errors(lib):
    for name in ("q", "scale", "x", "xscale", "y"):
        assert stored(lib, **{name: None}) == 1
    assert stored(lib, rows=0) == stored(lib, cols=-1) == stored(lib, rows=1 << 29) == 3
    assert stored(lib, batch=0) == stored(lib, batch=1 << 29) == 4
    assert stored(lib, q=P(0x100008)) == stored(lib, x=P(0x100008)) == stored(lib, xscale=P(0x100002)) == stored(lib, y=ODD) == 5
    assert stored(lib, ws=None) == stored(lib, ws=P(0x100010)) == stored(lib, wsb=16) == 8


NORMS = {"sqllm_rms_norm": 1, "sqllm_rms_norm_int8": 2, "sqllm_rms_norm_fp8": 2}


def norm(lib, name, x=A, ldx=300, residual=A, ldr=300, weight=A, rows=8, cols=300, eps=1e-5, total=B, out=None):
    out = out or [B] * NORMS[name]
    return getattr(lib, name)(x, ldx, residual, ldr, weight, rows, cols, eps, total, *out, None)


@pytest.mark.parametrize("name", NORMS)
def test_norm_argument_errors(lib, name):
    assert norm(lib, name, x=None) == norm(lib, name, weight=None) == 1
    assert norm(lib, name, residual=None) == 1  # a sum, but nothing to add
    for k in range(NORMS[name]):
        out = [B] * NORMS[name]
        out[k] = None
        assert norm(lib, name, out=out) == 1
        out[k] = ODD
        assert norm(lib, name, out=out) == 5
    assert norm(lib, name, rows=0) == norm(lib, name, cols=0) == norm(lib, name, ldx=299) == norm(lib, name, ldr=299) == 3
    assert norm(lib, name, rows=(1 << 30) + 1) == 3
    for eps in (-1e-9, NAN, INF, -INF):
        assert norm(lib, name, eps=eps) == 3
    most = 131072 if name.endswith("int8") else (1 << 24) + 1
    assert norm(lib, name, cols=most, ldx=most, ldr=most) == 3
    for bad in ("x", "residual", "weight", "total"):
        assert norm(lib, name, **{bad: ODD}) == 5
    if name.endswith("fp8"):
        assert norm(lib, name, rows=1 << 29) == 3  # scales beyond the bound


def test_python_refuses_host_tensors(nw):
    h, w = torch.zeros(4, 512, dtype=torch.float16), torch.zeros(512, dtype=torch.float16)
    q, s = torch.zeros(4, 512, dtype=torch.int8), torch.zeros(4)
    for call in (nw.rms_norm, nw.rms_norm_int8, nw.rms_norm_fp8):
        with pytest.raises(ValueError, match="device tensor"):
            call(h, w, 1e-5)
        with pytest.raises(TypeError, match="torch.Tensor"):
            call([1.0], w, 1e-5)
    with pytest.raises(ValueError, match="device tensor"):
        nw.int8_quantize(h)
    with pytest.raises(ValueError, match="device tensor"):
        nw.int8_gemm(q, s, h)
    with pytest.raises(ValueError, match="device tensor"):
        nw.int8_glu(q, s, q, s, h)
    u = q.view(torch.uint8)
    with pytest.raises(ValueError, match="device tensor"):
        nw.fp8_gemm(u, u, u, x_scale=u)
