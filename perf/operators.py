"""The 8-bit operators of the library on an MI355X: quantization in blocks of 128, the norm that feeds it and
its gradient, the block-scaled product and the product grouped by expert.

`run` makes one pass through one operator: in its plain form (elementary torch operations in fp32), or, where
`own` is true, through the calls a user makes of the library.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BLOCK = 128                       # columns (and, for a weight, rows) that share one scale
FLOOR = 2.0 ** -100               # the least magnitude a scale is made for
FORMATS = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}


# ---------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------

def listed():
    return [
        # a decoded token's activation, quantized by itself: launch latency
        {"name": "quantize_token", "op": "quantize", "rows": 1, "cols": 4096, "bf16": True, "block_rows": 1,
         "fmt": "e4m3"},
        # a frozen 28672 x 8192 up-projection put into 8-bit storage when a model is loaded
        {"name": "quantize_weight", "op": "quantize", "rows": 28672, "cols": 8192, "bf16": False, "block_rows": 128,
         "fmt": "e4m3"},
        # the norm before an attention projection for one decoded token: residual added, 8-bit output only
        {"name": "norm_token", "op": "norm", "rows": 1, "width": 4096, "residual": True, "bf16_out": False,
         "fp8_out": True, "rstd": False},
        # the same norm over a training batch: bf16 output for the adapter, 8-bit output for the frozen product
        {"name": "norm_batch", "op": "norm", "rows": 16384, "width": 8192, "residual": True, "bf16_out": True,
         "fp8_out": True, "rstd": True},
        # the norm's gradient in a short ragged batch of a 14B-shaped model
        {"name": "norm_grad_ragged", "op": "norm_grad", "rows": 1999, "width": 5120, "residual": True},
        # the norm's gradient over a training batch, joined with the residual stream's own gradient
        {"name": "norm_grad_batch", "op": "norm_grad", "rows": 16384, "width": 8192, "residual": True},
        # one decoded token through the 28672 x 8192 projection: every weight byte read once
        {"name": "matmul_token", "op": "matmul", "m": 1, "rows": 28672, "cols": 8192, "transpose": False, "rank": 0,
         "fmt": "e4m3"},
        # an attention projection over 2048 tokens with a rank-16 adapter's term
        {"name": "matmul_layer", "op": "matmul", "m": 2048, "rows": 4096, "cols": 4096, "transpose": False,
         "rank": 16, "fmt": "e4m3"},
        # the input gradient of an 11008 x 4096 projection for a ragged batch, gradients in e5m2
        {"name": "matmul_input_grad", "op": "matmul", "m": 4099, "rows": 11008, "cols": 4096, "transpose": True,
         "rank": 64, "fmt": "e5m2"},
        # the largest layer: 16384 tokens through the 28672 x 8192 projection with a rank-64 adapter's term
        {"name": "matmul_large", "op": "matmul", "m": 16384, "rows": 28672, "cols": 8192, "transpose": False,
         "rank": 64, "fmt": "e4m3"},
        # a few decoded tokens over 64 small experts: most experts get one row or none
        {"name": "grouped_tokens", "op": "grouped", "experts": 64, "m": 48, "spare": 0, "rows": 1536, "cols": 4096,
         "transpose": False, "rank": 0, "fmt": "e4m3", "routing": 3},
        # a training batch over 8 large experts with rank-16 adapters, ragged, one expert empty, padded rows behind
        {"name": "grouped_batch", "op": "grouped", "experts": 8, "m": 8205, "spare": 51, "rows": 11008, "cols": 4096,
         "transpose": False, "rank": 16, "fmt": "e4m3", "routing": 5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    return max(lo, _log(rng, lo, hi) // 16 * 16)


def draw(rng):
    op = rng.choice(["quantize", "norm", "norm_grad", "matmul", "matmul", "grouped", "grouped"])
    if op == "quantize":
        bf16 = rng.random() < 0.6
        return {"op": op, "rows": _log(rng, 1, 16384), "cols": _size(rng, 128, 12288), "bf16": bf16,
                "block_rows": 1 if bf16 else rng.choice([1, 128]), "fmt": rng.choice(["e4m3", "e5m2"])}
    if op == "norm":
        bf16_out = rng.random() < 0.6
        return {"op": op, "rows": _log(rng, 1, 16384), "width": _size(rng, 128, 8192), "residual": rng.random() < 0.7,
                "bf16_out": bf16_out, "fp8_out": not bf16_out or rng.random() < 0.6, "rstd": rng.random() < 0.5}
    if op == "norm_grad":
        return {"op": op, "rows": _log(rng, 1, 16384), "width": _size(rng, 128, 8192), "residual": rng.random() < 0.7}
    transpose = rng.random() < 0.4
    case = {"op": op, "transpose": transpose, "rank": rng.choice([0, 0, 16, 64, 128]),
            "fmt": rng.choice(["e4m3", "e5m2"]) if transpose else "e4m3"}
    if op == "matmul":
        return {**case, "m": _log(rng, 1, 16384), "rows": _size(rng, 512, 11008), "cols": _size(rng, 512, 11008)}
    experts = _log(rng, 2, 64)
    rows, cols = _size(rng, 512, 8192), _size(rng, 512, 8192)
    experts = max(2, min(experts, 400_000_000 // (rows * cols)))
    return {**case, "experts": experts, "m": _log(rng, 1, 8192), "spare": rng.choice([0, 0, 1, 37]), "rows": rows,
            "cols": cols, "routing": rng.randrange(1 << 20)}


def _counts(case):
    """Rows of each expert: unequal odds, one expert without any."""
    rng = random.Random(case["routing"])
    odds = [math.exp(rng.gauss(0.0, 0.7)) for _ in range(case["experts"])]
    odds[rng.randrange(case["experts"])] = 0.0
    got = [0] * case["experts"]
    for e in rng.choices(range(case["experts"]), odds, k=case["m"]):
        got[e] += 1
    return got


# ---------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------

def _normal(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device=DEV) * scale


def _activations(g, rows, width):
    """Hidden states: unit scale, with a few channels many times larger, as the residual stream has them."""
    x = _normal(g, rows, width)
    big = torch.randint(0, width, (max(1, width // 256),), generator=g, device=DEV)
    x[:, big] *= 20.0
    return x.to(torch.bfloat16)


def _gradients(g, rows, width):
    """Gradients: small, of sizes that differ from token to token."""
    x = _normal(g, rows, width, scale=1e-4)
    return (x * torch.exp(_normal(g, rows, 1))).to(torch.bfloat16)


def _weight(g, *shape):
    """A frozen weight: 0.02 wide, one value of a thousand 20 times larger."""
    w = _normal(g, *shape, scale=0.02)
    w[torch.rand(*shape, generator=g, device=DEV) < 1e-3] *= 20.0
    return w


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]
    s = {"op": op, "case": dict(case)}
    if op == "quantize":
        x = _activations(g, case["rows"], case["cols"]) if case["bf16"] else _weight(g, case["rows"], case["cols"])
        return {**s, "x": x}
    if op in ("norm", "norm_grad"):
        rows, width = case["rows"], case["width"]
        s["eps"] = 1e-6
        s["w"] = (1.0 + _normal(g, width, scale=0.1)).to(torch.bfloat16)
        x = _activations(g, rows, width)
        if op == "norm":
            return {**s, "x": x, "residual": _activations(g, rows, width) if case["residual"] else None}
        rstd = torch.rsqrt(x.float().square().mean(1) + s["eps"])
        return {**s, "h": x, "rstd": rstd, "dy": _gradients(g, rows, width),
                "dh": _gradients(g, rows, width) if case["residual"] else None}
    K, N = (case["rows"], case["cols"]) if case["transpose"] else (case["cols"], case["rows"])
    m = case["m"] + case.get("spare", 0)
    a = _gradients(g, m, K) if case["fmt"] == "e5m2" else _activations(g, m, K)
    s["a"], s["a_scales"] = _quantize(a, 1, case["fmt"])
    r = case["rank"]
    s["a2"] = s["b2"] = None
    if op == "matmul":
        s["w"], s["w_scales"] = _quantize(_weight(g, case["rows"], case["cols"]), BLOCK, "e4m3")
        if r:
            s["b2"] = _normal(g, N, r, scale=0.02).to(torch.bfloat16)
    else:
        E = case["experts"]
        made = [_quantize(_weight(g, case["rows"], case["cols"]), BLOCK, "e4m3") for _ in range(E)]
        s["w"] = torch.stack([w.view(torch.uint8) for w, _ in made]).view(torch.float8_e4m3fn)
        s["w_scales"] = torch.stack([x for _, x in made])
        counts = _counts(case)
        ends = torch.tensor([0] + counts, dtype=torch.int64).cumsum(0)
        s["offsets"] = ends.to(torch.int32).to(DEV)
        s["most"] = max(counts)
        s["out"] = torch.full((m, N), 1e-4, dtype=torch.bfloat16, device=DEV)
        if r:
            s["b2"] = _normal(g, E, N, r, scale=0.02).to(torch.bfloat16)
    if r:
        a2 = _normal(g, m, r)
        s["a2"] = (a2 * a.float().square().mean(1, keepdim=True).sqrt()).to(torch.bfloat16)
    return s


# ---------------------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------------------

def _blocks(x, block_rows):
    """x [R][C] as [ceil(R / block_rows)][block_rows][ceil(C / 128)][128], zeros behind its ends."""
    R, C = x.shape
    rb, cb = -(-R // block_rows), -(-C // BLOCK)
    x = torch.nn.functional.pad(x, (0, cb * BLOCK - C, 0, rb * block_rows - R))
    return x.view(rb, block_rows, cb, BLOCK)


def _quantize(x, block_rows, fmt):
    dtype, most = FORMATS[fmt]
    b = _blocks(x.float(), block_rows)
    amax = b.abs().amax((1, 3)).clamp_min(FLOOR)
    scales = amax / most
    codes = (b * (most / amax)[:, None, :, None]).to(dtype)
    rb, br, cb, _ = b.shape
    return codes.view(rb * br, cb * BLOCK)[:x.shape[0], :x.shape[1]].contiguous(), scales


def _spread(scales, block_rows, rows, cols):
    """One scale for each value of [rows][cols]."""
    return scales.repeat_interleave(block_rows, -2)[..., :rows, :].repeat_interleave(BLOCK, -1)[..., :cols]


def _values(codes, scales, block_rows):
    return codes.float() * _spread(scales, block_rows, codes.shape[-2], codes.shape[-1])


def _norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = (h + s["residual"].float()).to(torch.bfloat16).float()
    rstd = torch.rsqrt(h.square().mean(1, keepdim=True) + s["eps"])
    y = h * rstd * s["w"].float()
    c = s["case"]
    codes, scales = _quantize(y, 1, "e4m3") if c["fp8_out"] else (None, None)
    return {"y": y.to(torch.bfloat16) if c["bf16_out"] else None,
            "h": h.to(torch.bfloat16) if c["residual"] else None, "codes": codes, "scales": scales,
            "rstd": rstd[:, 0] if c["rstd"] else None}


def _norm_grad(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xhat = s["h"].float() * rstd
    gw = dy * s["w"].float()
    dx = rstd * (gw - xhat * (gw * xhat).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(torch.bfloat16), "dw": (dy * xhat).sum(0)}


def _matmul(s):
    w = _values(s["w"], s["w_scales"], BLOCK)
    y = _values(s["a"], s["a_scales"], 1) @ (w if s["case"]["transpose"] else w.t())
    if s["a2"] is not None:
        y = y + s["a2"].float() @ s["b2"].float().t()
    return y.to(torch.bfloat16)


def _grouped(s):
    """One batched product over the experts, each one's rows padded to the longest."""
    E, m, most = s["w"].shape[0], s["case"]["m"], s["most"]
    at = torch.arange(m, device=DEV)
    expert = torch.searchsorted(s["offsets"][1:], at, right=True)
    place = at - s["offsets"][expert]

    def padded(x):
        p = torch.zeros(E, most, x.shape[1], device=DEV)
        p[expert, place] = x[:m]
        return p

    w = _values(s["w"], s["w_scales"], BLOCK)
    y = padded(_values(s["a"], s["a_scales"], 1)) @ (w if s["case"]["transpose"] else w.transpose(1, 2))
    if s["a2"] is not None:
        y = y + padded(s["a2"].float()) @ s["b2"].float().transpose(1, 2)
    s["out"][:m] = y[expert, place].to(torch.bfloat16)
    return s["out"]


def run(s):
    op, c = s["op"], s["case"]
    if own:
        import quantized_lora_fine_amd as nf4
        if op == "quantize":
            return nf4.fp8_quantize(s["x"], c["block_rows"], FORMATS[c["fmt"]][0])
        if op == "norm":
            y, h, codes, scales, rstd = nf4.rmsnorm_fwd(s["x"], s["w"], s["eps"], residual=s["residual"],
                                                        want_y=c["bf16_out"], want_fp8=c["fp8_out"],
                                                        want_rstd=c["rstd"])
            return {"y": y, "h": h, "codes": codes, "scales": scales, "rstd": rstd}
        if op == "norm_grad":
            dx, dw = nf4.rmsnorm_bwd(s["dy"], s["h"], s["w"], s["rstd"], dH=s["dh"])
            return {"dx": dx, "dw": dw}
        if op == "matmul":
            return nf4.fp8_matmul(s["a"], s["a_scales"], s["w"], s["w_scales"], c["transpose"], s["a2"], s["b2"])
        return nf4.fp8_matmul_grouped(s["a"], s["a_scales"], s["w"], s["w_scales"], s["offsets"], c["transpose"],
                                      s["a2"], s["b2"], out=s["out"])
    if op == "quantize":
        return _quantize(s["x"], c["block_rows"], c["fmt"])
    return {"norm": _norm, "norm_grad": _norm_grad, "matmul": _matmul, "grouped": _grouped}[op](s)


# ---------------------------------------------------------------------------------------------------------
# what a pass cannot do without, and its outputs in 64 bits
# ---------------------------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["cols"]
        blocks = -(-case["rows"] // case["block_rows"]) * -(-case["cols"] // BLOCK)
        return {"bytes": n * ((2 if case["bf16"] else 4) + 1) + 4 * blocks, "flops": 2 * n}
    if op == "norm":
        n = case["rows"] * case["width"]
        each = 2 + (4 if case["residual"] else 0) + (2 if case["bf16_out"] else 0) + (1 if case["fp8_out"] else 0)
        scales = 4 * case["rows"] * -(-case["width"] // BLOCK) if case["fp8_out"] else 0
        return {"bytes": n * each + 2 * case["width"] + scales + (4 * case["rows"] if case["rstd"] else 0),
                "flops": 6 * n}
    if op == "norm_grad":
        n = case["rows"] * case["width"]
        return {"bytes": n * (8 if case["residual"] else 6) + 4 * case["rows"] + 6 * case["width"], "flops": 10 * n}
    m, rows, cols, r = case["m"], case["rows"], case["cols"], case["rank"]
    K, N = (rows, cols) if case["transpose"] else (cols, rows)
    used = sum(n > 0 for n in _counts(case)) if op == "grouped" else 1
    a = m * K + 4 * m * -(-K // BLOCK) + 2 * m * r
    w = used * (rows * cols + 4 * -(-rows // BLOCK) * -(-cols // BLOCK) + 2 * N * r)
    return {"bytes": a + w + 2 * m * N, "flops": 2 * m * N * (K + r)}


def _exact_scales(x, block_rows):
    """The largest magnitude of each block, spread over the block's values, and by block."""
    R, C = x.shape
    by_col = torch.stack([p.abs().amax(1) for p in x.split(BLOCK, 1)], 1)
    by_block = torch.stack([p.amax(0) for p in by_col.split(block_rows, 0)], 0).clamp_min(FLOOR)
    i = torch.arange(R, device=x.device) // block_rows
    j = torch.arange(C, device=x.device) // BLOCK
    return by_block, by_block[i][:, j]


def _exact_codes(x, block_rows, fmt):
    """(values of the codes, scales) by the format's definition: the nearest value of the 8-bit grid, ties to even."""
    most = FORMATS[fmt][1]
    mantissa, lowest = (3, -6) if fmt == "e4m3" else (2, -14)
    amax, each = _exact_scales(x, block_rows)
    v = x * (most / each.float()).double()
    v = v.float().double()  # the product is an fp32 value
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(lowest) - mantissa)
    return torch.round(v / step) * step, amax / most


def _exact_values(codes, scales, block_rows):
    i = torch.arange(codes.shape[0], device=codes.device) // block_rows
    j = torch.arange(codes.shape[1], device=codes.device) // BLOCK
    return codes.double() * scales.double()[i][:, j]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "quantize":
        return _exact_codes(s["x"].double(), case["block_rows"], case["fmt"])
    if op == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).float().to(torch.bfloat16).double()
        rstd = 1.0 / torch.sqrt((h * h).sum(1) / h.shape[1] + s["eps"])
        y = h * rstd[:, None] * s["w"].double()
        codes, scales = _exact_codes(y, 1, "e4m3") if case["fp8_out"] else (None, None)
        return {"y": y if case["bf16_out"] else None, "h": h if case["residual"] else None, "codes": codes,
                "scales": scales, "rstd": rstd if case["rstd"] else None}
    if op == "norm_grad":
        dy, h, w, r = s["dy"].double(), s["h"].double(), s["w"].double(), s["rstd"].double()[:, None]
        u = dy * w
        dot = (u * h).sum(1, keepdim=True)
        dx = r * u - h * r.pow(3) * dot / h.shape[1]
        return {"dx": dx if s["dh"] is None else dx + s["dh"].double(), "dw": (dy * h * r).sum(0)}
    a = _exact_values(s["a"], s["a_scales"], 1)
    if op == "matmul":
        w = _exact_values(s["w"], s["w_scales"], BLOCK)
        y = torch.matmul(a, w if case["transpose"] else w.t())
        return y if s["a2"] is None else y + torch.matmul(s["a2"].double(), s["b2"].double().t())
    y, at = s["out"].double(), 0
    for e, n in enumerate(_counts(case)):
        w = _exact_values(s["w"][e], s["w_scales"][e], BLOCK)
        part = torch.matmul(a[at:at + n], w if case["transpose"] else w.t())
        if s["a2"] is not None:
            part = part + torch.matmul(s["a2"][at:at + n].double(), s["b2"][e].double().t())
        y[at:at + n] = part
        at += n
    return y
