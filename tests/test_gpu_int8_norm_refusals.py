"""What the integer products, the norm and the stored e4m3 product refuse of device tensors, before any launch: types,
shapes, strides, other devices and scratch that is too small.  The outputs stay as they were."""
import pytest
import torch

from gpu_util import nw

pytestmark = pytest.mark.gpu

B, R, C = 3, 40, 300


def zeros(*shape, dtype=torch.float16):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def products():
    lib, wide = nw(), nw().int8_cols(C)
    q, s = zeros(R, wide, dtype=torch.int8), zeros(R, dtype=torch.float32)
    yield lambda **k: lib.int8_gemm(**{"q": q, "scale": s, **k}), "q", "scale", "y", lib.int8_workspace_bytes
    yield (lambda **k: lib.int8_glu(**{"gate": q, "gate_scale": s, "up": q, "up_scale": s, **k}), "up", "up_scale", "h",
           lib.int8_glu_workspace_bytes)


@pytest.mark.parametrize("which", [0, 1], ids=["gemm", "glu"])
def test_integer_products(which):
    call, q, scale, out, size = list(products())[which]
    wide = nw().int8_cols(C)
    x, xq, xs = zeros(B, C), zeros(B, wide, dtype=torch.int8), zeros(B, dtype=torch.float32)
    call(x=x), call(x=xq, x_scale=xs)  # allowed
    for bad in (x.float(), xq, x.tolist(), None):
        with pytest.raises(TypeError):
            call(x=bad)
    for bad in (zeros(B, wide + 1), zeros(B, wide - 128), zeros(B, 2, C), zeros(B, 131072), zeros(C, B).t(), x.cpu()):
        with pytest.raises(ValueError):
            call(x=bad)
    for bad in ((x, xs), (xq, xs.half()), (xq.view(torch.uint8), xs), (xq, [1.0] * B)):
        with pytest.raises(TypeError):
            call(x=bad[0], x_scale=bad[1])
    for bad in ((xq[:, :C], xs), (zeros(B, wide + 128, dtype=torch.int8), xs), (xq, xs[:2]), (xq, xs.cpu()),
                (xq, zeros(2 * B, dtype=torch.float32)[::2])):
        with pytest.raises(ValueError):
            call(x=bad[0], x_scale=bad[1])
    for bad in (zeros(R, wide, dtype=torch.uint8), zeros(R, wide)):
        with pytest.raises(TypeError):
            call(x=x, **{q: bad})
    for bad in (zeros(R, C, dtype=torch.int8), zeros(R + 1, wide, dtype=torch.int8), zeros(wide, R, dtype=torch.int8).t(),
                zeros(wide, dtype=torch.int8)):
        with pytest.raises(ValueError):
            call(x=x, **{q: bad})
    with pytest.raises(TypeError):
        call(x=x, **{scale: zeros(R)})
    with pytest.raises(ValueError):
        call(x=x, **{scale: zeros(R + 1, dtype=torch.float32)})
    y = torch.full((B, R), 7.0, dtype=torch.float16, device="cuda")
    with pytest.raises(TypeError):
        call(x=x, **{out: y.float()})
    for bad in (y[:2], y.t(), zeros(R, B).t()):
        with pytest.raises(ValueError):
            call(x=x, **{out: bad})
    need = size(R, C, B)
    with pytest.raises(RuntimeError):
        call(x=x, ws=zeros(need - 1, dtype=torch.uint8), **{out: y})
    with pytest.raises(RuntimeError):  # (16 bytes past a multiple of 256)
        call(x=x, ws=zeros(need + 256, dtype=torch.uint8)[16:], **{out: y})
    with pytest.raises(TypeError):
        call(x=x, ws=zeros(need), **{out: y})
    with pytest.raises(RuntimeError):
        call(x=zeros(0, C))
    assert (y == 7).all()


@pytest.mark.parametrize("form", ["rms_norm", "rms_norm_int8", "rms_norm_fp8"])
def test_norms(form):
    call = getattr(nw(), form)
    x, w = zeros(B, C), zeros(C)
    call(x, w, 1e-5), call(x, w, 1e-5, residual=x)  # allowed
    for bad in (x.float(), x.bfloat16()):
        with pytest.raises(TypeError):
            call(bad, w, 1e-5)
        with pytest.raises(TypeError):
            call(x, w, 1e-5, residual=bad)
    for bad in (zeros(C), zeros(0, C), zeros(B, 0), zeros(C, B).t(), zeros(1, C).expand(B, C), zeros(B, C, 1)):
        with pytest.raises((ValueError, RuntimeError)):
            call(bad, zeros(bad.shape[-1]), 1e-5)
    for bad in (zeros(B, C + 1), zeros(B + 1, C), zeros(C), zeros(1, C).expand(B, C), x.cpu()):
        with pytest.raises((ValueError, RuntimeError)):
            call(x, w, 1e-5, residual=bad)
    with pytest.raises(TypeError):
        call(x, w, 1e-5, residual=1.0)
    with pytest.raises(TypeError):
        call(x, w.float(), 1e-5)
    for bad in (zeros(C + 1), zeros(1, C), zeros(2 * C)[::2], w.cpu()):
        with pytest.raises(ValueError):
            call(x, bad, 1e-5)
    for eps in (-1e-9, float("nan"), float("inf")):
        with pytest.raises(RuntimeError):
            call(x, w, eps)
    with pytest.raises(ValueError):
        call(x, w, 1e-5, total=zeros(B, C))
    for bad in (zeros(B, C + 1), zeros(B, 2 * C)[:, ::2], zeros(B, C + 8)[:, :C]):
        with pytest.raises(ValueError):
            call(x, w, 1e-5, residual=x, total=bad)
    with pytest.raises(TypeError):
        call(x, w, 1e-5, residual=x, total=zeros(B, C, dtype=torch.float32))
    if form == "rms_norm":
        with pytest.raises(ValueError):
            call(x, w, 1e-5, y=zeros(B, C + 1))
    else:
        with pytest.raises(ValueError):
            call(x, w, 1e-5, q=zeros(B, C, dtype=torch.int8 if form.endswith("int8") else torch.uint8))
        with pytest.raises(ValueError):
            call(x, w, 1e-5, scale=zeros(B + 1, dtype=torch.float32))


def test_quantize():
    call = nw().int8_quantize
    with pytest.raises(TypeError):
        call(zeros(B, C, dtype=torch.float32))
    for bad in (zeros(C), zeros(0, C), zeros(C, B).t(), zeros(1, 131072), zeros(1, C).expand(B, C)):
        with pytest.raises((ValueError, RuntimeError)):
            call(bad)
    with pytest.raises(ValueError):
        call(zeros(B, C), q=zeros(B, C, dtype=torch.int8))
    with pytest.raises(TypeError):
        call(zeros(B, C), scale=zeros(B))


def test_stored_fp8_product():
    lib = nw()
    wide, pitch = lib.fp8_cols(C), lib.fp8_scale_pitch(C)
    u8 = torch.uint8
    q, s, x, xs = zeros(R, wide, dtype=u8), zeros(R, pitch, dtype=u8), zeros(B, wide, dtype=u8), zeros(B, pitch, dtype=u8)
    lib.fp8_gemm(q, s, x, x_scale=xs)  # allowed
    for bad in ((zeros(B, wide), xs), (x, xs.half()), (x, 1.0)):
        with pytest.raises(TypeError):
            lib.fp8_gemm(q, s, bad[0], x_scale=bad[1])
    for bad in ((x[:, :C], xs), (zeros(B, wide + 128, dtype=u8), xs), (x, xs[:2]), (x, xs[:, :1]), (x.cpu(), xs),
                (x, zeros(pitch, B, dtype=u8).t())):
        with pytest.raises(ValueError):
            lib.fp8_gemm(q, s, bad[0], x_scale=bad[1])
    with pytest.raises(TypeError):
        lib.fp8_gemm(q, s, x)
