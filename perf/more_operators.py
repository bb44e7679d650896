"""Cases that measure the norm in front of the products and the products in 8-bit integers.

Four operators: the root-mean-square norm with the residual's addition, its output in fp16, in 8-bit integers with a
scale for each token or in e4m3 with a power-of-two scale for each block of 128 columns (rms_norm, rms_norm_int8,
rms_norm_fp8); the quantiser to 8-bit integers (int8_quantize); the product with scales for each token and channel
(int8_gemm), its activations in fp16 or already in integers; and the gated half of a feed-forward block, both
projections, the activation and the product in one call (int8_glu).  `own` chooses between their plain form in torch
and this package's calls.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5


# --------------------------------------------------------------------------------------------------- the cases
def _norm(name, rows, cols, form, residual):
    return {"name": name, "op": "rms_norm", "rows": rows, "cols": cols, "form": form, "residual": residual}


def _product(name, op, batch, rows, cols, stored):
    return {"name": name, "op": op, "batch": batch, "rows": rows, "cols": cols, "stored": stored}


def listed():
    return [
        # one token between two blocks of a layer: nothing but latency
        _norm("norm_1", 1, 4096, "fp16", True),
        # sixteen users, in front of an integer product
        _norm("norm_16_int8", 16, 8192, "int8", True),
        # a prompt's first norm, no residual yet
        _norm("norm_prompt", 2000, 5120, "fp16", False),
        # a long prompt in front of an e4m3 product: the largest
        _norm("norm_prompt_e4m3", 4096, 8192, "e4m3", True),
        # sixteen tokens' activations in front of a down projection
        {"name": "quantize_tokens", "op": "int8_quantize", "rows": 16, "cols": 22016},
        # a matrix of odd sizes, offline
        {"name": "quantize_ragged", "op": "int8_quantize", "rows": 4097, "cols": 5001},
        # one token through the down projection of the large model, its activations in fp16
        _product("gemm_1", "int8_gemm", 1, 8192, 22016, False),
        # sixteen users through a square projection, after a norm that left integers
        _product("gemm_16", "int8_gemm", 16, 8192, 8192, True),
        # a short prompt through a matrix of odd sizes
        _product("gemm_ragged", "int8_gemm", 77, 5001, 4999, False),
        # a long prompt through a square projection
        _product("gemm_prompt", "int8_gemm", 4096, 8192, 8192, True),
        # one token through gate and up
        _product("glu_1", "int8_glu", 1, 11008, 4096, True),
        # a prompt through gate and up
        _product("glu_prompt", "int8_glu", 2048, 13824, 5120, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rms_norm", "rms_norm", "int8_quantize", "int8_gemm", "int8_gemm", "int8_glu", "int8_glu"])
    if op in ("rms_norm", "int8_quantize"):
        rows = _log(rng, 1, 8192)
        cols = min(_log(rng, 64, 24576), 4096 * 8192 // rows)
        if op == "int8_quantize":
            return {"op": op, "rows": rows, "cols": cols}
        case = _norm("", rows, cols, rng.choice(["fp16", "int8", "e4m3"]), rng.random() < 0.75)
    else:
        most = 4096 * 8192 * 8192 // (2 if op == "int8_glu" else 1)
        while True:
            case = _product("", op, _log(rng, 1, 8192), _log(rng, 64, 28000), _log(rng, 128, 24576), rng.random() < 0.5)
            if case["batch"] * case["rows"] * case["cols"] <= most:
                break
    del case["name"]
    return case


def work(case):
    op = case["op"]
    if op == "rms_norm":
        n = case["rows"] * case["cols"]
        out = {"fp16": 2 * n, "int8": n + 4 * case["rows"], "e4m3": n * (1 + 1 / 128)}[case["form"]]
        return {"bytes": 2 * n + (4 * n if case["residual"] else 0) + 2 * case["cols"] + out, "flops": 6 * n}
    if op == "int8_quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": 3 * n + 4 * case["rows"], "flops": 2 * n}
    b, r, c = case["batch"], case["rows"], case["cols"]
    x = b * c + 4 * b if case["stored"] else 2 * b * c
    m = 2 if op == "int8_glu" else 1
    return {"bytes": m * (r * c + 4 * r) + x + 2 * b * r, "flops": 2 * m * b * r * c}


# --------------------------------------------------------------------------------------------------- the inputs
def _int8(v):
    """(codes, scales) of float32 v: per row a scale max|v| / 127 and the nearest integers, columns padded to 128."""
    scale = v.abs().amax(dim=1) / 127
    q = torch.round(v / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]).to(torch.int8)
    return torch.nn.functional.pad(q, (0, -v.shape[1] % 128)), scale


def _e4m3(v):
    """(codes, scales) of float32 v: per row and block of 128 columns the smallest s with max|v| <= 448 * 2^s."""
    blocks = torch.nn.functional.pad(v, (0, -v.shape[1] % 128)).view(v.shape[0], -1, 128)
    m, e = torch.frexp(blocks.abs().amax(dim=-1))  # m * 2^e, 448 = 0.875 * 2^9
    s = torch.where(m > 0, e - 9 + (m > 0.875).int(), torch.zeros_like(e))
    q = torch.ldexp(blocks, -s[..., None]).to(torch.float8_e4m3fn)
    scale = torch.nn.functional.pad((s + 127).to(torch.uint8), (0, -s.shape[1] % 4), value=127)
    return q.view(v.shape[0], -1), scale.view(torch.float8_e8m0fnu)


def _activations(rows, cols, gen):
    """Activations inside a decoder: normal, a few channels far larger than the rest."""
    x = torch.randn(rows, cols, generator=gen, device=DEV)
    loud = torch.rand(cols, generator=gen, device=DEV) < 0.002
    return (x * torch.where(loud, 20.0, 1.0)).half()


def _matrix(rows, cols, gen):
    return _int8((torch.randn(rows, cols, generator=gen, device=DEV) * 0.02).half().float())


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    if op == "int8_quantize":
        return {"op": op, "x": _activations(case["rows"], case["cols"], gen)}
    if op == "rms_norm":
        rows, cols = case["rows"], case["cols"]
        s = {"op": op, "form": case["form"], "x": _activations(rows, cols, gen), "residual": None}
        if case["residual"]:
            s["residual"] = _activations(rows, cols, gen)
        s["weight"] = (1 + 0.2 * torch.randn(cols, generator=gen, device=DEV)).half()
        return s
    s = {"op": op, "cols": case["cols"], "scale": None, "x": _activations(case["batch"], case["cols"], gen)}
    if case["stored"]:
        s["x"], s["scale"] = _int8(s["x"].float())
    s["w"] = [_matrix(case["rows"], case["cols"], gen) for _ in range(2 if op == "int8_glu" else 1)]
    return s


# --------------------------------------------------------------------------------------------------- one pass
def _values(q, scale, cols):
    """What integers with a scale for each row stand for, in fp16."""
    return torch.mul(q[:, :cols], scale[:, None], out=torch.empty(q.shape[0], cols, dtype=torch.float16, device=DEV))


def _own(s):
    import non_uniform_weight_amd as nw
    op = s["op"]
    if op == "int8_quantize":
        return _values(*nw.int8_quantize(s["x"]), s["x"].shape[1])
    if op == "int8_gemm":
        return nw.int8_gemm(*s["w"][0], s["x"], x_scale=s["scale"])
    if op == "int8_glu":
        return nw.int8_glu(*s["w"][0], *s["w"][1], s["x"], x_scale=s["scale"])
    call = {"fp16": nw.rms_norm, "int8": nw.rms_norm_int8, "e4m3": nw.rms_norm_fp8}[s["form"]]
    got = call(s["x"], s["weight"], EPS, residual=s["residual"])
    if s["form"] == "fp16":
        return got
    if s["form"] == "int8":
        return _values(*got[:2], s["x"].shape[1]), got[1], *got[2:]
    return got[0].view(torch.float8_e4m3fn), got[1].view(torch.float8_e8m0fnu), *got[2:]


def run(s):
    op = s["op"]
    if own:
        return _own(s)
    if op == "int8_quantize":
        return _values(*_int8(s["x"].float()), s["x"].shape[1])
    if op == "rms_norm":
        total = () if s["residual"] is None else ((s["x"].float() + s["residual"].float()).half(),)
        v = (total[0] if total else s["x"]).float()
        y = v * torch.rsqrt(v.square().mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
        if s["form"] == "fp16":
            return (y.half(), *total) if total else y.half()
        if s["form"] == "int8":
            q, scale = _int8(y)
            return _values(q, scale, y.shape[1]), scale, *total
        return *_e4m3(y), *total
    q, scale = (s["x"], s["scale"]) if s["scale"] is not None else _int8(s["x"].float())
    y = [(q.float() @ wq.float().t()) * scale[:, None] * ws for wq, ws in s["w"]]
    if op == "int8_gemm":
        return y[0].half()
    return (y[0] / (1 + torch.exp(-y[0])) * y[1]).half()


# --------------------------------------------------------------------------------------------------- 64 bits
def _steps_64(v):
    """v in multiples of a 127th of its row's largest magnitude, in 64 bits, and those steps."""
    step = v.abs().max(dim=1, keepdim=True).values / 127
    return torch.round(v / step.clamp(min=1e-300)), step


def exact(case, seed):
    s = prepare(case, seed)
    op, x = case["op"], s["x"].double()
    if op == "int8_quantize":
        q, step = _steps_64(x)
        return q * step
    if op == "rms_norm":
        total = ()
        if case["residual"]:
            total = ((x + s["residual"].double()),)
            x = total[0].half().double()  # the sum is held in fp16, and the norm is that of what is held
        y = x / torch.sqrt((x * x).sum(dim=1, keepdim=True) / case["cols"] + EPS) * s["weight"].double()
        if case["form"] == "fp16":
            return (y, *total) if total else y
        if case["form"] == "int8":
            q, step = _steps_64(y)
            return q * step, step[:, 0], *total
        b = torch.nn.functional.pad(y, (0, -case["cols"] % 128)).view(case["rows"], -1, 128)
        f = torch.exp2(torch.ceil(torch.log2(b.abs().amax(dim=2, keepdim=True).clamp(min=2.0 ** -100) / 448)))
        b = b / f
        grid = torch.exp2(torch.floor(torch.log2(b.abs().clamp(min=2.0 ** -6))) - 3)
        return (torch.round(b / grid) * grid).flatten(1), None, *total
    if case["stored"]:
        x = x * s["scale"].double()[:, None]
    else:
        q, step = _steps_64(x)
        x = torch.nn.functional.pad(q * step, (0, -case["cols"] % 128))
    y = [x @ (wq.double() * ws.double()[:, None]).t() for wq, ws in s["w"]]
    return y[0] if op == "int8_gemm" else y[0] * torch.sigmoid(y[0]) * y[1]
