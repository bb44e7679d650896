"""Cases that measure the mixture-of-experts and the 8-bit floating point operators.

Five operators: the router (moe_route), the experts' products for given choices (moe_experts), both together
(moe_layer), the quantiser to e4m3 with a power-of-two scale for each block of 128 columns (fp8_quantize) and the
product with such weights (fp8_gemm).  `own` chooses between their plain form in torch and this package's calls.
"""
import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------------------------------- the cases
def _moe(name, tokens, experts, topk, hidden, inter, bits, density, sigmoid=False, op="moe_layer"):
    return {"name": name, "op": op, "tokens": tokens, "experts": experts, "topk": topk, "hidden": hidden,
            "inter": inter, "bits": bits, "density": density, "sigmoid": sigmoid}


def listed():
    return [
        # one token of one user through a small router: nothing but latency
        {"name": "route_1_of_8", "op": "moe_route", "tokens": 1, "experts": 8, "topk": 2, "hidden": 4096, "sigmoid": False},
        # sixteen users, many experts, sigmoid scores and a balancing bias
        {"name": "route_16_of_256", "op": "moe_route", "tokens": 16, "experts": 256, "topk": 8, "hidden": 8192, "sigmoid": True},
        # one token, many small experts: the common decoding step of a sparse model
        _moe("layer_1_small_experts", 1, 64, 6, 2048, 1280, 3, 0.0045),
        # one token, few large experts (the MLP shape 11008x4096)
        _moe("layer_1_large_experts", 1, 8, 2, 4096, 11008, 3, 0.0045),
        # eight users, four bits, no outliers
        _moe("layer_8_4bit", 8, 128, 8, 2048, 768, 4, 0.0),
        # sixteen users over many experts: the largest step
        _moe("layer_16_many_experts", 16, 128, 8, 4096, 1536, 3, 0.0045, sigmoid=True),
        # choices made elsewhere; a batch with padded rows and dropped choices
        _moe("experts_5_padded_2bit", 5, 32, 3, 2560, 1792, 2, 0.0005, op="moe_experts"),
        _moe("experts_16_of_8_4bit", 16, 8, 2, 4096, 3584, 4, 0.0045, op="moe_experts"),
        # the offline step on one matrix of the weights, and a ragged batch of activations
        {"name": "quantize_weights", "op": "fp8_quantize", "rows": 13824, "cols": 5120},
        {"name": "quantize_ragged", "op": "fp8_quantize", "rows": 333, "cols": 5001},
        # one token through the widest projection of the large model
        {"name": "gemm_1", "op": "fp8_gemm", "batch": 1, "rows": 8192, "cols": 22016},
        # a prompt of a few thousand tokens through a square projection
        {"name": "gemm_prompt", "op": "fp8_gemm", "batch": 4096, "rows": 8192, "cols": 8192},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["moe_route", "moe_layer", "moe_layer", "moe_experts", "fp8_quantize", "fp8_gemm", "fp8_gemm"])
    if op == "fp8_quantize":
        rows = _log(rng, 1, 16384)
        return {"op": op, "rows": rows, "cols": min(_log(rng, 64, 24576), 13824 * 5120 // rows)}
    if op == "fp8_gemm":
        while True:
            c = {"op": op, "batch": _log(rng, 1, 8192), "rows": _log(rng, 64, 28000), "cols": _log(rng, 128, 24576)}
            if c["batch"] * c["rows"] * c["cols"] <= 4096 * 8192 * 8192:
                return c
    tokens, experts = _log(rng, 1, 16), _log(rng, 4, 256)
    topk = rng.randint(1, min(8, experts))
    if op == "moe_route":
        return {"op": op, "tokens": tokens, "experts": experts, "topk": topk,
                "hidden": 256 * _log(rng, 2, 32), "sigmoid": rng.random() < 0.5}
    while True:
        hidden, inter = 256 * _log(rng, 3, 32), 256 * _log(rng, 2, 56)
        active = min(experts, tokens * topk)
        if active * hidden * inter <= 80 * 4096 * 1536 and experts * hidden * inter <= 128 * 4096 * 1536:
            c = _moe("", tokens, experts, topk, hidden, inter, rng.choice([2, 3, 4]), rng.choice([0.0, 0.0005, 0.0045]),
                     rng.random() < 0.5, op)
            del c["name"]
            return c


def work(case):
    op = case["op"]
    if op == "fp8_quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n + n * (1 + 1 / 128), "flops": 2 * n}
    if op == "fp8_gemm":
        b, r, c = case["batch"], case["rows"], case["cols"]
        return {"bytes": r * c * (1 + 1 / 128) + 2 * b * (r + c), "flops": 2 * b * r * c}
    t, e, k, h = case["tokens"], case["experts"], case["topk"], case["hidden"]
    route = {"bytes": 2 * h * (t + e) + 8 * t * k, "flops": 2 * t * e * h}
    if op == "moe_route":
        return route
    i, b = case["inter"], case["bits"]
    used = e * (1 - (1 - k / e) ** t)  # experts that t tokens choose, on average
    one = 3 * h * i * b / 8 + (2 * i + h) * 2 ** b * 2 + case["density"] * 3 * h * i * 4
    if case["density"]:
        one += 4 * (2 * i + h)
    got = {"bytes": used * one + 4 * t * h, "flops": 6 * t * k * h * i}
    if op == "moe_layer":
        got = {m: got[m] + route[m] for m in got}
    return got


# --------------------------------------------------------------------------------------------------- the inputs
def _pack(codes, bits):
    """The library's stored form of uint8 codes [..., rows, cols] (rows in tiles of 64, columns in groups of 256)."""
    lead, (rows, cols) = codes.shape[:-2], codes.shape[-2:]
    pairs = codes.view(*lead, rows, cols // 2, 2)
    pairs = pairs[..., 0] | (pairs[..., 1] << bits)
    if bits == 4:
        text = pairs
    elif bits == 2:
        pairs = pairs.view(*lead, rows, cols // 4, 2)
        text = pairs[..., 0] | (pairs[..., 1] << 4)
    else:
        pairs = pairs.view(*lead, rows, cols // 32, 16)
        rest = pairs[..., 12:]
        top = torch.cat([(rest >> (2 * k)) & 3 for k in range(3)], dim=-1)
        text = pairs[..., :12] | (top << 6)
    text = text.reshape(*lead, rows // 64, 64, cols // 256, 2 * bits, 16)
    n = len(lead)
    return text.permute(*range(n), n, n + 2, n + 3, n + 1, n + 4).contiguous().view(-1)


def _experts(case, rows, cols, gen):
    """One projection of every expert: codes, tables and outliers as k-means and the split leave them."""
    e, bits = case["experts"], case["bits"]
    # a row's codes are bell-shaped: byte values are dealt to the 2^bits centroids by the normal's quantiles
    edges = torch.linspace(-2.2, 2.2, 2 ** bits - 1, dtype=torch.float64)
    share = 0.5 * (1 + torch.erf(edges / math.sqrt(2)))
    deal = torch.bucketize((torch.arange(256) + 0.5) / 256, share).to(torch.uint8).to(DEV)
    drawn = torch.randint(0, 256, (e * rows * cols,), generator=gen, device=DEV, dtype=torch.uint8)
    codes = torch.cat([deal[part.int()] for part in drawn.split(1 << 28)]).view(e, rows, cols)
    lut = (torch.randn(e, rows, 2 ** bits, generator=gen, device=DEV) * 0.02).sort(dim=-1).values.half()
    made = {"codes": codes, "packed": _pack(codes, bits), "lut": lut}
    nnz = int(case["density"] * e * rows * cols)
    if nnz:
        at = torch.randint(0, e * rows * cols, (nnz,), generator=gen, device=DEV).sort().values
        row = at // cols
        made["row_ptr"] = torch.searchsorted(row, torch.arange(e * rows + 1, device=DEV)).int()
        made["col"] = (at % cols).to(torch.int32).to(torch.int16)
        made["val"] = (torch.randn(nnz, generator=gen, device=DEV) * 0.2).half()
        made["row"] = row
    return made


def _block_exponents(x):
    """Per row and block of 128 columns (the last may be short): the smallest s with max|x| <= 448 * 2^s."""
    padded = torch.nn.functional.pad(x, (0, -x.shape[1] % 128))
    blocks = padded.view(x.shape[0], -1, 128)
    top = blocks.abs().amax(dim=-1)
    m, e = torch.frexp(top)  # top = m * 2^e, 448 = 0.875 * 2^9
    s = torch.where(top > 0, e - 9 + (m > 0.875).int(), torch.zeros_like(e))
    return blocks, s


def _to_fp8(x):
    """(e4m3 codes as bytes, scale bytes) of float32 x: the stored form of 8-bit weights and activations."""
    blocks, s = _block_exponents(x)
    q = torch.ldexp(blocks, -s[..., None]).to(torch.float8_e4m3fn)
    scale = torch.nn.functional.pad((s + 127).to(torch.uint8), (0, -s.shape[1] % 4), value=127)
    return q.view(torch.uint8).view(x.shape[0], -1), scale


def _activations(rows, cols, gen):
    """Activations as a decoder's norm hands them on: normal, a few channels far larger than the rest."""
    x = torch.randn(rows, cols, generator=gen, device=DEV)
    loud = torch.rand(cols, generator=gen, device=DEV) < 0.002
    return (x * torch.where(loud, 20.0, 1.0)).half()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    s = {"op": op}
    if op == "fp8_quantize":
        s["x"] = _activations(case["rows"], case["cols"], gen)
        return s
    if op == "fp8_gemm":
        w = torch.randn(case["rows"], case["cols"], generator=gen, device=DEV) * 0.02
        s["wq"], s["wscale"] = _to_fp8(w.half().float())
        s["x"] = _activations(case["batch"], case["cols"], gen)
        return s
    t, e, k, h = case["tokens"], case["experts"], case["topk"], case["hidden"]
    s["x"] = torch.randn(t, h, generator=gen, device=DEV).half()
    s["topk"], s["sigmoid"] = k, case["sigmoid"]
    if op != "moe_experts":
        s["router"] = (torch.randn(e, h, generator=gen, device=DEV) / math.sqrt(h)).half()
        # the balancing bias goes with sigmoid scores, as does a factor on the weights
        s["bias"] = torch.randn(e, generator=gen, device=DEV) * 0.05 if case["sigmoid"] else None
        s["scale"] = 2.5 if case["sigmoid"] else 1.0
    if op == "moe_route":
        return s
    i = case["inter"]
    s["bits"] = case["bits"]
    s["gate"], s["up"] = _experts(case, i, h, gen), _experts(case, i, h, gen)
    s["down"] = _experts(case, h, i, gen)
    if op == "moe_experts":
        s["ids"] = torch.rand(t, e, generator=gen, device=DEV).argsort(dim=1)[:, :k].int()
        s["weights"] = torch.rand(t, k, generator=gen, device=DEV) + 0.1
        if t > 2:  # a padded row, and one choice that another GPU's expert answers
            s["ids"][-1] = -1
            s["ids"][0, k - 1] = -1
        s["ids"], s["weights"] = s["ids"].contiguous(), s["weights"].contiguous()
    return s


# --------------------------------------------------------------------------------------------------- one pass
def _route(s):
    logits = s["x"].double() @ s["router"].double().t()
    score = torch.sigmoid(logits) if s["sigmoid"] else torch.softmax(logits, dim=1)
    choice = score if s["bias"] is None else score + s["bias"].double()
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :s["topk"]]
    kept = score.gather(1, ids)
    return ids.int(), (s["scale"] * kept / kept.sum(dim=1, keepdim=True)).float()


def _weights(p, used, place):
    """The used experts' matrices [U, rows, cols] in 32 bits."""
    lut, codes = p["lut"][used].float(), p["codes"][used]
    w = lut.gather(2, codes.flatten(2).long())
    if "val" in p:
        rows, cols = codes.shape[1:]
        slot = place[p["row"] // rows]
        kept = slot >= 0
        at = (slot[kept] * rows + p["row"][kept] % rows) * cols + (p["col"][kept].long() & 0xFFFF)
        w.view(-1).index_add_(0, at, p["val"][kept].float())
    return w


def _experts_plain(s, ids, weights):
    experts = s["gate"]["lut"].shape[0]
    ids = ids.long()
    used = ids[ids >= 0].unique()
    place = torch.full((experts,), -1, device=DEV, dtype=torch.long)
    place[used] = torch.arange(used.numel(), device=DEV)
    x = s["x"].float().t().contiguous()
    g = torch.matmul(_weights(s["gate"], used, place), x)
    u = torch.matmul(_weights(s["up"], used, place), x)
    h = g / (1 + torch.exp(-g)) * u
    out = torch.matmul(_weights(s["down"], used, place), h)  # [U, hidden, T]
    share = (weights[None] * (ids[None] == used[:, None, None])).sum(dim=2)  # [U, T]
    return (out * share[:, None, :]).sum(dim=0).t().half()


def run(s):
    op = s["op"]
    if own:
        import non_uniform_weight_amd as nw
        if op == "fp8_quantize":
            q, scale = nw.fp8_quantize(s["x"])
            return {"q": q.view(torch.float8_e4m3fn), "scale": scale}
        if op == "fp8_gemm":
            return nw.fp8_gemm(s["wq"], s["wscale"], s["x"])
        if op == "moe_route":
            ids, weights = nw.moe_route(s["x"], s["router"], s["topk"], bias=s["bias"], sigmoid=s["sigmoid"],
                                        scale=s["scale"])
            return {"ids": ids, "weights": weights}
        if op == "moe_experts":
            return nw.moe_experts(s["x"], s["ids"], s["weights"], s["gate"], s["up"], s["down"], s["bits"])
        y, ids, weights = nw.moe_layer(s["x"], s["router"], s["topk"], s["gate"], s["up"], s["down"], s["bits"],
                                       bias=s["bias"], sigmoid=s["sigmoid"], scale=s["scale"])
        return {"y": y, "ids": ids, "weights": weights}
    if op == "fp8_quantize":
        q, scale = _to_fp8(s["x"].float())
        return {"q": q.view(torch.float8_e4m3fn), "scale": scale}
    if op == "fp8_gemm":
        rows = s["wq"].shape[0]
        blocks, e = _block_exponents(s["x"].float())
        x = torch.ldexp(torch.ldexp(blocks, -e[..., None]).to(torch.float8_e4m3fn).float(), e[..., None])
        w = s["wq"].view(torch.float8_e4m3fn).float().view(rows, -1, 128)
        w = torch.ldexp(w, s["wscale"][:, :w.shape[1], None].int() - 127)
        return (x.flatten(1) @ w.flatten(1).t()).half()
    if op == "moe_experts":
        return _experts_plain(s, s["ids"], s["weights"])
    ids, weights = _route(s)
    if op == "moe_route":
        return {"ids": ids, "weights": weights}
    return {"y": _experts_plain(s, ids, weights), "ids": ids, "weights": weights}


# --------------------------------------------------------------------------------------------------- 64 bits
def _e4m3_64(v):
    """v rounded to the nearest e4m3 value, ties to even, in 64 bits (|v| <= 448)."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _blocks_64(x):
    """e4m3 values and scales (a factor for each block) of x, from the definition."""
    b = torch.nn.functional.pad(x.double(), (0, -x.shape[1] % 128)).view(x.shape[0], -1, 128)
    top = b.abs().amax(dim=2, keepdim=True)
    s = torch.where(top > 0, torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)), torch.zeros_like(top))
    s = torch.where(top > 448 * torch.exp2(s), s + 1, s)
    s = torch.where((top > 0) & (top <= 448 * torch.exp2(s - 1)), s - 1, s)
    f = torch.exp2(s)
    return _e4m3_64(b / f), f


def _matrix_64(p, e, rows, cols):
    w = torch.take_along_dim(p["lut"][e].double(), p["codes"][e].view(rows, cols).long(), dim=1)
    if "val" in p:
        lo, hi = int(p["row_ptr"][e * rows]), int(p["row_ptr"][(e + 1) * rows])
        where = (p["row"][lo:hi] - e * rows, p["col"][lo:hi].long() & 0xFFFF)
        w.index_put_(where, p["val"][lo:hi].double(), accumulate=True)
    return w


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "fp8_quantize":
        q, _ = _blocks_64(s["x"])
        return {"q": q.flatten(1), "scale": None}
    if op == "fp8_gemm":
        q, f = _blocks_64(s["x"])
        w = s["wq"].view(torch.float8_e4m3fn).double().view(case["rows"], -1, 128)
        w = w * torch.exp2(s["wscale"][:, :w.shape[1], None].double() - 127)
        return (q * f).flatten(1) @ w.flatten(1).t()
    x = s["x"].double()
    if op != "moe_experts":
        logits = torch.matmul(x[:, None, :], s["router"].double().t()[None]).squeeze(1)
        if case["sigmoid"]:
            score = 1 / (1 + torch.exp(-logits))
        else:
            score = torch.exp(logits - logits.logsumexp(dim=1, keepdim=True))
        rank = score if s["bias"] is None else score + s["bias"].double()
        ids = rank.topk(case["topk"], dim=1).indices
        weights = score.gather(1, ids)
        weights = s["scale"] * weights / weights.sum(dim=1, keepdim=True)
        if op == "moe_route":
            return {"ids": None, "weights": weights}
    else:
        ids, weights = s["ids"].long(), s["weights"].double()
    h, i = case["hidden"], case["inter"]
    y = torch.zeros_like(x)
    for e in sorted(set(ids.flatten().tolist()) - {-1}):
        share = torch.where(ids == e, weights, torch.zeros_like(weights)).sum(dim=1)
        rows = (ids == e).any(dim=1).nonzero().flatten()
        a, b = x[rows] @ _matrix_64(s["gate"], e, i, h).t(), x[rows] @ _matrix_64(s["up"], e, i, h).t()
        y[rows] += share[rows, None] * ((a * torch.sigmoid(a) * b) @ _matrix_64(s["down"], e, h, i).t())
    return y if op == "moe_experts" else {"y": y, "ids": None, "weights": weights}
