"""The operators around a shared projection on an MI355X: rows sorted by id, low-rank adapters of many requests and
their gradients (from bf16 inputs or from 8-bit activation checkpoints), the layer norm and its gradient.

`run` makes one pass through one operator: in its plain form (elementary torch operations in fp32), or, where
`own` is true, through the calls a user makes of the library.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BLOCK = 128                       # columns of a row that share one scale
FLOOR = 2.0 ** -100               # the least magnitude a scale is made for
FORMATS = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}


# ---------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------

def listed():
    return [
        # the rows of a decode step sorted by adapter, a few without one: launch latency
        {"name": "route_tokens", "op": "route", "m": 61, "spare": 3, "n": 48, "runs": False, "routing": 11},
        # a large batch's token copies sorted by expert
        {"name": "route_batch", "op": "route", "m": 131000, "spare": 72, "n": 256, "runs": False, "routing": 12},
        # the norm before a projection for one decoded token: residual added, 8-bit output only
        {"name": "layernorm_token", "op": "norm", "rows": 1, "width": 4096, "residual": True, "bias": True,
         "bf16_out": False, "fp8_out": True, "stats": False},
        # the same norm over a training batch: bf16 output for the adapters, 8-bit output for the frozen product
        {"name": "layernorm_batch", "op": "norm", "rows": 16384, "width": 8192, "residual": True, "bias": True,
         "bf16_out": True, "fp8_out": True, "stats": True},
        # the norm's gradient in a short ragged batch of a 14B-shaped model
        {"name": "layernorm_grad_ragged", "op": "norm_grad", "rows": 1999, "width": 5120, "residual": True,
         "bias": True},
        # the norm's gradient over a training batch, joined with the residual stream's own gradient
        {"name": "layernorm_grad_batch", "op": "norm_grad", "rows": 16384, "width": 8192, "residual": True,
         "bias": True},
        # one decoded token with its own adapter beside an attention projection
        {"name": "adapters_token", "op": "adapters", "m": 1, "spare": 0, "n": 8, "h": 4096, "o": 4096, "rank": 16,
         "runs": False, "ordered": False, "routing": 21},
        # a decode step of 61 requests over a pool of 48 adapters, three requests without one, beside an
        # up-projection
        {"name": "adapters_decode", "op": "adapters", "m": 61, "spare": 3, "n": 48, "h": 4096, "o": 11008,
         "rank": 32, "runs": False, "ordered": True, "routing": 22},
        # prompts of several requests in one batch, in the order of their arrival
        {"name": "adapters_prefill", "op": "adapters", "m": 7977, "spare": 23, "n": 12, "h": 4096, "o": 11008,
         "rank": 16, "runs": True, "ordered": True, "routing": 23},
        # the gradients of three adapters that are trained in one short batch
        {"name": "adapters_grad_ragged", "op": "adapters_grad", "m": 501, "spare": 10, "n": 3, "h": 4096, "o": 4096,
         "rank": 8, "runs": True, "ordered": True, "x": "bf16", "routing": 31},
        # eight adapters trained side by side on a down-projection, rows sorted by adapter
        {"name": "adapters_grad_batch", "op": "adapters_grad", "m": 8192, "spare": 0, "n": 8, "h": 11008, "o": 4096,
         "rank": 64, "runs": True, "ordered": False, "x": "bf16", "routing": 32},
        # the largest layer, 8192 -> 28672 at 16384 tokens with one adapter: gradients from an 8-bit checkpoint
        {"name": "adapters_grad_checkpoint", "op": "adapters_grad", "m": 16384, "spare": 0, "n": 1, "h": 8192,
         "o": 28672, "rank": 64, "runs": True, "ordered": False, "x": "e4m3", "routing": 33},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    return max(lo, _log(rng, lo, hi) // 16 * 16)


def draw(rng):
    op = rng.choice(["route", "norm", "norm_grad", "adapters", "adapters", "adapters_grad", "adapters_grad"])
    if op == "route":
        return {"op": op, "m": _log(rng, 24, 131072), "spare": rng.choice([0, 0, 1, 50]), "n": _log(rng, 4, 512),
                "runs": rng.random() < 0.3, "routing": rng.randrange(1 << 20)}
    if op == "norm":
        bf16_out = rng.random() < 0.6
        return {"op": op, "rows": _log(rng, 1, 16384), "width": _size(rng, 128, 8192), "residual": rng.random() < 0.7,
                "bias": rng.random() < 0.7, "bf16_out": bf16_out, "fp8_out": not bf16_out or rng.random() < 0.6,
                "stats": rng.random() < 0.5}
    if op == "norm_grad":
        return {"op": op, "rows": _log(rng, 1, 16384), "width": _size(rng, 128, 8192), "residual": rng.random() < 0.7,
                "bias": rng.random() < 0.7}
    m = _log(rng, 1, 12288)
    case = {"op": op, "m": m, "spare": rng.choice([0, 0, 1, 37]), "n": _log(rng, 1, 64), "h": _size(rng, 256, 8192),
            "o": _size(rng, 256, 8192), "rank": rng.choice([8, 16, 16, 32, 64, 64, 128]), "runs": rng.random() < 0.6,
            "ordered": rng.random() < 0.6, "routing": rng.randrange(1 << 20)}
    if op == "adapters_grad":
        case["x"] = rng.choice(["bf16", "bf16", "e4m3", "e4m3", "e5m2"])
    return case


def _ids(case):
    """The id of each row, -1 for a row without one: requests of many tokens one after another (`runs`), or every
    row its own draw. Unequal odds; with more than two ids one of them has no row."""
    rng = random.Random(case["routing"])
    n, m = case["n"], case["m"]
    odds = [math.exp(rng.gauss(0.0, 0.5)) for _ in range(n)]
    if n > 2:
        odds[rng.randrange(n)] = 0.0
    if case["runs"]:
        cuts = sorted(rng.randrange(m + 1) for _ in range(min(m, 2 * n) - 1))
        ids = []
        for a, b in zip([0] + cuts, cuts + [m]):
            ids += rng.choices(range(n), odds) * (b - a)
    else:
        ids = rng.choices(range(n), odds, k=m)
    if not case.get("ordered", True):
        return sorted(ids) + [-1] * case["spare"]
    for _ in range(case["spare"]):
        ids.insert(rng.randrange(len(ids) + 1), -1)
    return ids


def _counts(case):
    got = [0] * case["n"]
    for i in _ids(case):
        if i >= 0:
            got[i] += 1
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


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]
    s = {"op": op, "case": dict(case)}
    if op == "route":
        ids = _ids({**case, "routing": case["routing"] * 1009 + int(seed)})
        return {**s, "ids": torch.tensor(ids, dtype=torch.int32).to(DEV)}
    if op in ("norm", "norm_grad"):
        rows, width = case["rows"], case["width"]
        s["eps"] = 1e-5
        s["w"] = (1.0 + _normal(g, width, scale=0.1)).to(torch.bfloat16)
        x = (_activations(g, rows, width).float() + _normal(g, rows, 1, scale=0.5)).to(torch.bfloat16)
        if op == "norm":
            s["b"] = _normal(g, width, scale=0.1).to(torch.bfloat16) if case["bias"] else None
            return {**s, "x": x, "residual": _activations(g, rows, width) if case["residual"] else None}
        mean = x.double().mean(1, keepdim=True)
        rstd = torch.rsqrt((x.double() - mean).square().mean(1) + s["eps"])
        return {**s, "h": x, "mean": mean[:, 0].float(), "rstd": rstd.float(), "dy": _gradients(g, rows, width),
                "dh": _gradients(g, rows, width) if case["residual"] else None}
    n, h, o, r = case["n"], case["h"], case["o"], case["rank"]
    ids = torch.tensor(_ids(case), dtype=torch.int64)
    rows = len(ids)
    s["most"], s["listed"] = max(_counts(case)), case["m"]
    key = torch.where(ids < 0, n, ids)
    counts = torch.bincount(key, minlength=n + 1)[:n]
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32).to(DEV)
    s["order"] = torch.sort(key, stable=True)[1].to(torch.int32).to(DEV) if case["ordered"] else None
    s["l1"] = _normal(g, n, h, r, scale=h ** -0.5).to(torch.bfloat16)
    s["l2"] = _normal(g, n, r, o, scale=0.02).to(torch.bfloat16)
    s["s"] = 0.5 + 2.0 * torch.rand(n, generator=g, device=DEV)
    x = _activations(g, rows, h)
    if op == "adapters":
        s["x"] = x
        s["base"] = _normal(g, rows, o).to(torch.bfloat16)
        s["t"] = torch.full((rows, r), 0.25, device=DEV)
        s["out"] = torch.full((rows, o), 0.25, dtype=torch.bfloat16, device=DEV)
        return s
    s["x_scales"] = None
    if case["x"] != "bf16":
        x, s["x_scales"] = _quantize(x, case["x"])
    s["x"] = x
    s["dy"] = _gradients(g, rows, o)
    s["t"] = _normal(g, rows, r)
    s["base"] = _gradients(g, rows, h)
    s["out"] = torch.full((rows, h), 1e-4, dtype=torch.bfloat16, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------------------

def _quantize(x, fmt):
    dtype, most = FORMATS[fmt]
    R, C = x.shape
    cb = -(-C // BLOCK)
    b = torch.nn.functional.pad(x.float(), (0, cb * BLOCK - C)).view(R, cb, BLOCK)
    amax = b.abs().amax(2).clamp_min(FLOOR)
    codes = (b * (most / amax)[:, :, None]).to(dtype)
    return codes.view(R, cb * BLOCK)[:, :C].contiguous(), amax / most


def _values(codes, scales):
    return codes.float() * scales.repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def _route(s):
    n = s["case"]["n"]
    ids = s["ids"]
    key = torch.where((ids < 0) | (ids >= n), n, ids)
    key, order = torch.sort(key, stable=True)
    ends = torch.arange(n + 1, device=DEV, dtype=torch.int32)
    return {"order": order.to(torch.int32), "offsets": torch.searchsorted(key, ends).to(torch.int32)}


def _norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = (h + s["residual"].float()).to(torch.bfloat16).float()
    mean = h.mean(1, keepdim=True)
    d = h - mean
    rstd = torch.rsqrt(d.square().mean(1, keepdim=True) + s["eps"])
    y = d * rstd * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    c = s["case"]
    codes, scales = _quantize(y, "e4m3") if c["fp8_out"] else (None, None)
    return {"y": y.to(torch.bfloat16) if c["bf16_out"] else None,
            "h": h.to(torch.bfloat16) if c["residual"] else None, "codes": codes, "scales": scales,
            "mean": mean[:, 0] if c["stats"] else None, "rstd": rstd[:, 0] if c["stats"] else None}


def _norm_grad(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xhat = (s["h"].float() - s["mean"][:, None]) * rstd
    u = dy * s["w"].float()
    dx = rstd * (u - u.mean(1, keepdim=True) - xhat * (u * xhat).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(torch.bfloat16), "dw": (dy * xhat).sum(0), "db": dy.sum(0) if s["case"]["bias"] else None}


def _places(s):
    """For every listed row: its number, its adapter, and its place among that adapter's rows."""
    at = torch.arange(s["listed"], device=DEV)
    adapter = torch.searchsorted(s["offsets"][1:], at, right=True)
    return at if s["order"] is None else s["order"][:s["listed"]].long(), adapter, at - s["offsets"][adapter]


def _adapters(s):
    """Batched products over the adapters, each one's rows padded to the longest."""
    n, h, r = s["l1"].shape
    rows, adapter, place = _places(s)
    x = torch.zeros(n, s["most"], h, device=DEV)
    x[adapter, place] = s["x"][rows].float()
    t = x @ s["l1"].float()
    delta = (t @ s["l2"].float()) * s["s"][:, None, None]
    s["t"][rows] = t[adapter, place]
    s["out"][rows] = (s["base"][rows].float() + delta[adapter, place]).to(torch.bfloat16)
    return {"y": s["out"], "t": s["t"]}


def _adapters_grad(s):
    n, h, r = s["l1"].shape
    rows, adapter, place = _places(s)
    xv = s["x"].float() if s["x_scales"] is None else _values(s["x"], s["x_scales"])

    def padded(v):
        p = torch.zeros(n, s["most"], v.shape[1], device=DEV)
        p[adapter, place] = v[rows].float()
        return p

    x, dy, t = padded(xv), padded(s["dy"]), padded(s["t"])
    g = (dy @ s["l2"].float().transpose(1, 2)) * s["s"][:, None, None]
    dl2 = (t.transpose(1, 2) @ dy) * s["s"][:, None, None]
    dl1 = x.transpose(1, 2) @ g
    dx = g @ s["l1"].float().transpose(1, 2)
    s["out"][rows] = (s["base"][rows].float() + dx[adapter, place]).to(torch.bfloat16)
    return {"dx": s["out"], "dl1": dl1, "dl2": dl2}


def run(s):
    op, c = s["op"], s["case"]
    if own:
        import quantized_lora_fine_amd as nf4
        if op == "route":
            order, offsets = nf4.route(s["ids"], c["n"])
            return {"order": order, "offsets": offsets}
        if op == "norm":
            y, h, codes, scales, mean, rstd = nf4.layernorm_fwd(s["x"], s["w"], s["b"], s["eps"],
                                                                residual=s["residual"], want_y=c["bf16_out"],
                                                                want_fp8=c["fp8_out"], want_stats=c["stats"])
            return {"y": y, "h": h, "codes": codes, "scales": scales, "mean": mean, "rstd": rstd}
        if op == "norm_grad":
            dx, dw, db = nf4.layernorm_bwd(s["dy"], s["h"], s["w"], s["mean"], s["rstd"], dH=s["dh"],
                                           want_db=c["bias"])
            return {"dx": dx, "dw": dw, "db": db}
        if op == "adapters":
            y, t = nf4.adapters_fwd(s["x"], s["l1"], s["l2"], s["s"], s["offsets"], order=s["order"], base=s["base"],
                                    out=s["out"], T_out=s["t"])
            return {"y": y, "t": t}
        dx, dl1, dl2 = nf4.adapters_bwd(s["dy"], s["x"], s["t"], s["l1"], s["l2"], s["s"], s["offsets"],
                                        order=s["order"], x_scales=s["x_scales"], base=s["base"], dX=s["out"])
        return {"dx": dx, "dl1": dl1, "dl2": dl2}
    return {"route": _route, "norm": _norm, "norm_grad": _norm_grad, "adapters": _adapters,
            "adapters_grad": _adapters_grad}[op](s)


# ---------------------------------------------------------------------------------------------------------
# what a pass cannot do without, and its outputs in 64 bits
# ---------------------------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "route":
        m = case["m"] + case["spare"]
        return {"bytes": 8 * m + 4 * (case["n"] + 1), "flops": 0}
    if op == "norm":
        n = case["rows"] * case["width"]
        each = 2 + (4 if case["residual"] else 0) + (2 if case["bf16_out"] else 0) + (1 if case["fp8_out"] else 0)
        scales = 4 * case["rows"] * -(-case["width"] // BLOCK) if case["fp8_out"] else 0
        return {"bytes": n * each + 2 * case["width"] * (1 + case["bias"]) + scales + 8 * case["rows"] * case["stats"],
                "flops": 9 * n}
    if op == "norm_grad":
        n = case["rows"] * case["width"]
        return {"bytes": n * (8 if case["residual"] else 6) + 8 * case["rows"]
                + case["width"] * (6 + 4 * case["bias"]), "flops": 13 * n}
    m, h, o, r = case["m"], case["h"], case["o"], case["rank"]
    used = sum(c > 0 for c in _counts(case))
    lists = 4 * (case["n"] + 1) + (4 * m if case["ordered"] else 0) + 4 * used
    if op == "adapters":
        return {"bytes": m * (2 * h + 4 * o + 4 * r) + 2 * used * r * (h + o) + lists, "flops": 2 * m * r * (h + o)}
    x = 2 * h if case["x"] == "bf16" else h + 4 * -(-h // BLOCK)
    return {"bytes": m * (x + 2 * o + 4 * r + 4 * h) + 2 * used * r * (h + o) + 4 * case["n"] * r * (h + o) + lists,
            "flops": 4 * m * r * (h + o)}


def _exact_codes(y):
    """(values of the e4m3 codes, scales) by the format's definition: the nearest value of the 8-bit grid, ties to
    even."""
    C = y.shape[1]
    amax = torch.stack([p.abs().amax(1) for p in y.split(BLOCK, 1)], 1).clamp_min(FLOOR)
    each = amax[:, torch.arange(C, device=y.device) // BLOCK]
    v = (y * (448.0 / each.float()).double()).float().double()
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(-6) - 3)
    return torch.round(v / step) * step, amax / 448.0


def _exact_route(s, n):
    ids = s["ids"].tolist()
    rows = [[] for _ in range(n + 1)]
    for m, i in enumerate(ids):
        rows[i if 0 <= i < n else n].append(m)
    offsets = [0]
    for r in rows[:n]:
        offsets.append(offsets[-1] + len(r))
    return {"order": torch.tensor([m for r in rows for m in r], dtype=torch.int32),
            "offsets": torch.tensor(offsets, dtype=torch.int32)}


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "route":
        return _exact_route(s, case["n"])
    if op == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).float().to(torch.bfloat16).double()
        mean = h.sum(1) / h.shape[1]
        d = h - mean[:, None]
        rstd = 1.0 / torch.sqrt((d * d).sum(1) / h.shape[1] + s["eps"])
        y = d * rstd[:, None] * s["w"].double()
        if s["b"] is not None:
            y = y + s["b"].double()
        codes, scales = _exact_codes(y) if case["fp8_out"] else (None, None)
        return {"y": y if case["bf16_out"] else None, "h": h if case["residual"] else None, "codes": codes,
                "scales": scales, "mean": mean if case["stats"] else None, "rstd": rstd if case["stats"] else None}
    if op == "norm_grad":
        dy, w = s["dy"].double(), s["w"].double()
        mean, rstd = s["mean"].double()[:, None], s["rstd"].double()[:, None]
        xhat, u = (s["h"].double() - mean) * rstd, dy * w
        H = u.shape[1]
        dx = rstd * (u - u.sum(1, keepdim=True) / H) - rstd * xhat * ((u * xhat).sum(1, keepdim=True) / H)
        return {"dx": dx if s["dh"] is None else dx + s["dh"].double(), "dw": (dy * xhat).sum(0),
                "db": dy.sum(0) if case["bias"] else None}
    of = {}
    ids = _ids(case)
    for m, i in enumerate(ids):
        of.setdefault(i, []).append(m)
    of.pop(-1, None)
    n, h, r = s["l1"].shape
    o = s["l2"].shape[2]
    out = s["out"].double()
    if op == "adapters":
        t_all = s["t"].double()
        for a, rows in of.items():
            rows = torch.tensor(rows, device=DEV)
            t = torch.matmul(s["x"][rows].double(), s["l1"][a].double())
            t_all[rows] = t
            out[rows] = s["base"][rows].double() + s["s"][a].double() * torch.matmul(t, s["l2"][a].double())
        return {"y": out, "t": t_all}
    dl1 = torch.zeros(n, h, r, dtype=torch.float64, device=DEV)
    dl2 = torch.zeros(n, r, o, dtype=torch.float64, device=DEV)
    j = torch.arange(h, device=DEV) // BLOCK
    for a, rows in of.items():
        rows = torch.tensor(rows, device=DEV)
        x = s["x"][rows].double()
        if s["x_scales"] is not None:
            x = x * s["x_scales"][rows].double()[:, j]
        dy = s["dy"][rows].double() * s["s"][a].double()
        g = torch.matmul(dy, s["l2"][a].double().t().contiguous())
        dl2[a] = torch.matmul(s["t"][rows].double().t().contiguous(), dy)
        dl1[a] = torch.matmul(x.t().contiguous(), g)
        out[rows] = s["base"][rows].double() + torch.matmul(g, s["l1"][a].double().t().contiguous())
    return {"dx": out, "dl1": dl1, "dl2": dl2}
