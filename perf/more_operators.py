"""The measured cases of three operators around the MoE layer: the root-mean-square norm with the
residual's addition and an 8-bit output, routing to experts from given logits, and the product of a
few rows with 4-bit weights that have a scale and a zero point per group.

Each case runs in a plain form (elementary torch operations) or, with `own` set, through the
library's own entry points, on the same inputs; `exact` is the definition in 64 bits.

Norm.  h = x + r, y = h / sqrt(mean(h^2) + eps) * g; besides y, or in its place, e4m3 codes with one
fp32 scale per row and 128 columns (max|y| / 448).
Routing.  Scores s = sigmoid(l) or softmax(l); choice by s + b, the best groups of experts first
where there are groups (by the sum of their two best, or by the best), then the k best experts,
ties to the lower index; weights s, divided by their sum if asked for, times a scale.
4-bit weights.  W[j][i] = scale[i / group][j] (code[j][i] - zero[i / group][j]), codes packed two to
a byte along i, element 2i in the low nibble.  One matrix, or one per expert with the experts of
each row given; then silu(gate) * up (gate rows first), or the weighted sum over a row's experts.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
COLUMNS = 128  # of an 8-bit scale
EPS = 1e-6


def listed():
    return [
        # one decode step's token between the attention and the experts
        dict(name="norm-1x4096", op="norm", rows=1, cols=4096, dtype="bf16", residual=True, want="out"),
        # the same for a batch, into the 8-bit rows that the quantised experts take
        dict(name="norm-16x4096-fp8", op="norm", rows=16, cols=4096, dtype="bf16", residual=True, want="fp8"),
        # odd rows in 32 bits, no residual
        dict(name="norm-333x2050-f32", op="norm", rows=333, cols=2050, dtype="f32", residual=False, want="out"),
        # a prompt: the router reads the 16-bit rows, the quantised experts the 8-bit ones
        dict(name="norm-16384x4096-both", op="norm", rows=16384, cols=4096, dtype="bf16", residual=True, want="both"),
        # one token over 256 experts in 8 groups: latency
        dict(name="route-1x256-sigmoid", op="route", tokens=1, experts=256, top=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, group_score="top2", renormalise=True, dtype="f32"),
        # a prompt over 128 experts, 16-bit logits
        dict(name="route-8192x128-softmax", op="route", tokens=8192, experts=128, top=4, score="softmax", bias=False,
             groups=1, top_groups=1, group_score="max", renormalise=True, dtype="bf16"),
        # a long prompt over 256 experts in 8 groups
        dict(name="route-16384x256-sigmoid", op="route", tokens=16384, experts=256, top=8, score="sigmoid", bias=True,
             groups=8, top_groups=4, group_score="top2", renormalise=True, dtype="f32"),
        # a single token, a small matrix: launch latency
        dict(name="int4-1x512x256-g32", op="int4", tokens=1, n=512, k=256, group=32, experts=0, top=1, x="bf16",
             swiglu=False, weighted=False),
        # a dense expert's up projection for one token
        dict(name="int4-1x14336x4096-g128", op="int4", tokens=1, n=14336, k=4096, group=128, experts=0, top=1, x="bf16",
             swiglu=False, weighted=False),
        # its down projection for sixteen sequences, 8-bit rows
        dict(name="int4-16x4096x14336-g64-fp8", op="int4", tokens=16, n=4096, k=14336, group=64, experts=0, top=1, x="fp8",
             swiglu=False, weighted=False),
        # gate and up of 8 large experts for a few sequences
        dict(name="int4-8-of-8x28672x4096-g128", op="int4", tokens=8, n=28672, k=4096, group=128, experts=8, top=2, x="bf16",
             swiglu=True, weighted=False),
        # down of 64 experts and the sum over each token's six
        dict(name="int4-16-of-64x4096x1536-g32", op="int4", tokens=16, n=4096, k=1536, group=32, experts=64, top=6, x="bf16",
             swiglu=False, weighted=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "norm", "route", "route", "int4", "int4", "int4"])
    if op == "norm":
        cols, kind = log(64, 16384), rng.choice(["bf16", "bf16", "f32"])
        return dict(op=op, rows=log(1, min(16384, (67_000_000 if kind == "bf16" else 33_000_000) // cols)), cols=cols, dtype=kind,
                    residual=rng.random() < 0.7, want=rng.choice(["out", "fp8", "both"]))
    if op == "route":
        experts, groups = rng.choice([(8, 1), (16, 1), (16, 4), (37, 1), (60, 1), (64, 8), (96, 6), (128, 1), (160, 8), (256, 8), (256, 1)])
        top_groups = rng.randint(1, groups)
        return dict(op=op, tokens=log(1, 16384), experts=experts, top=rng.randint(1, min(8, top_groups * (experts // groups))),
                    score=rng.choice(["sigmoid", "softmax"]), bias=rng.random() < 0.6, groups=groups, top_groups=top_groups,
                    group_score=rng.choice(["top2", "max"]), renormalise=rng.random() < 0.8, dtype=rng.choice(["bf16", "f32"]))
    group = rng.choice([32, 64, 128])
    experts = rng.choice([0, 0, 4, 8, 16, 64, 128])
    kind = rng.choice(["plain", "swiglu", "weighted"]) if experts else rng.choice(["plain", "swiglu"])
    k = group * log(1, 14336 // group)
    n = 32 * log(1, max(1, min(28672, 900_000_000 // (k * max(experts, 1))) // 32))
    return dict(op=op, tokens=rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 9, 12, 16]), n=n, k=k, group=group, experts=experts,
                top=rng.randint(1, min(experts, 8)) if experts else 1, x="bf16" if kind == "weighted" else rng.choice(["bf16", "fp8"]),
                swiglu=kind == "swiglu", weighted=kind == "weighted")


# ------------------------------------------------------------------ inputs
def _normal(shape, std, g, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "norm":
        kind, shape = TYPES[case["dtype"]], (case["rows"], case["cols"])
        # a residual stream with a few large channels and a block's output to be added to it
        wide = torch.where(torch.rand(case["cols"], generator=g, device="cuda") < 0.01, 20.0, 1.0)
        r = (_normal(shape, 2.0, g) * wide).to(kind) if case["residual"] else None
        x = _normal(shape, 1.0, g, kind)
        return dict(case=case, x=x, residual=r, weight=(1 + _normal((case["cols"],), 0.2, g)).to(kind))
    if case["op"] == "route":
        t, e = case["tokens"], case["experts"]
        logits = (_normal((t, e), 1.5, g) + _normal((e,), 0.5, g)).to(TYPES[case["dtype"]])
        std = 0.1 if case["score"] == "sigmoid" else 0.01
        return dict(case=case, logits=logits, bias=_normal((e,), std, g) if case["bias"] else None)
    return _prepare_int4(case, g)


def _prepare_int4(case, g):
    t, n, k, e, top = (case[i] for i in ("tokens", "n", "k", "experts", "top"))
    lead = (e,) if e else ()
    s = dict(case=case)
    s["codes"] = torch.randint(0, 256, (*lead, n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    s["zeros"] = torch.randint(6, 10, (*lead, k // case["group"], n), generator=g, device="cuda", dtype=torch.uint8)
    s["scales"] = torch.rand((*lead, k // case["group"], n), generator=g, device="cuda") * 0.004 + 0.002
    rows = (t, top) if case["weighted"] else (t,)
    x = _normal((*rows, k), 1.0, g, torch.bfloat16)
    if case["x"] == "fp8":  # as the norm leaves them
        codes, scales = _to_fp8(x.float())
        s["x"], s["x_scales"] = codes, scales
    else:
        s["x"], s["x_scales"] = x, None
    s["ids"], s["w"] = None, None
    if e:  # distinct experts of each row, some of them favoured
        score = torch.rand((t, e), generator=g, device="cuda") + 0.5 * torch.rand((e,), generator=g, device="cuda")
        s["ids"] = torch.sort(score, dim=-1, descending=True, stable=True).indices[:, :top].to(torch.int32).contiguous()
        if case["weighted"]:
            w = torch.rand((t, top), generator=g, device="cuda") + 0.1
            s["w"] = w / w.sum(-1, keepdim=True)
    return s


# ------------------------------------------------------------- plain forms
def _columns(v):
    """[rows][cols] as [rows][blocks of 128], the last one filled up with zeros."""
    rows, cols = v.shape
    blocks = -(-cols // COLUMNS)
    if blocks * COLUMNS == cols:
        return v.view(rows, blocks, COLUMNS)
    p = torch.zeros((rows, blocks * COLUMNS), dtype=v.dtype, device=v.device)
    p[:, :cols] = v
    return p.view(rows, blocks, COLUMNS)


def _to_fp8(y):
    """Codes (e4m3) and scales of y's rows (fp32)."""
    v = _columns(y)
    scale = v.abs().amax(-1) / 448
    q = torch.where(scale[..., None] > 0, v / scale[..., None], 0.0).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(y.shape[0], -1)[:, :y.shape[1]].contiguous(), scale


def _plain_norm(s):
    case, kind = s["case"], s["x"].dtype
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    out = {"sum": h.to(kind)} if s["residual"] is not None else {}
    if case["want"] != "fp8":
        out["out"] = y.to(kind)
    if case["want"] != "out":
        out["codes"], out["scales"] = _to_fp8(y)
    return out


def _choose(case, s, bias):
    """Experts by score s (64 bits) and bias: the best groups, then the best of these."""
    c = s if bias is None else s + bias.double()
    if case["groups"] > 1:
        per = c.view(c.shape[0], case["groups"], -1)
        best = torch.sort(per, dim=-1, descending=True).values
        value = best[..., :2].sum(-1) if case["group_score"] == "top2" else best[..., 0]
        order = torch.sort(value, dim=-1, descending=True, stable=True).indices[:, :case["top_groups"]]
        kept = torch.zeros(value.shape, dtype=torch.bool, device=c.device).scatter_(1, order, True)
        c = torch.where(kept[..., None], per, -math.inf).view(c.shape)
    return torch.sort(c, dim=-1, descending=True, stable=True).indices[:, :case["top"]]


def _plain_route(s):
    # in 64 bits: two experts' scores may differ by less than 32 bits tell
    case, l = s["case"], s["logits"].double()
    if case["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-l))
    else:
        p = torch.exp(l - l.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
    ids = _choose(case, p, s["bias"])
    w = torch.gather(p, 1, ids)
    if case["renormalise"]:
        w = w / w.sum(-1, keepdim=True)
    return dict(ids=ids.to(torch.int32), w=(w * 2.5).float())


def _weights(s, dtype, pick=slice(None)):
    q = s["codes"][pick]
    q = torch.stack([q & 15, q >> 4], -1).flatten(-2).to(dtype)
    group = s["case"]["group"]
    q = q.unflatten(-1, (-1, group))
    z, scale = s["zeros"][pick].to(dtype).transpose(-1, -2), s["scales"][pick].to(dtype).transpose(-1, -2)
    return q.sub_(z[..., None]).mul_(scale[..., None]).flatten(-2)


def _rows(s, dtype):
    x = s["x"].to(dtype)
    if s["x_scales"] is not None:
        x = x * s["x_scales"].to(dtype).repeat_interleave(COLUMNS, -1)[:, :x.shape[-1]]
    return x


def _plain_int4(s):
    case, x = s["case"], _rows(s, torch.float32)
    w = _weights(s, torch.float32)
    if not case["experts"]:
        y = x @ w.T
    else:  # every expert on every row, then the chosen ones
        t, top = case["tokens"], case["top"]
        every = x.reshape(-1, case["k"]) @ w.transpose(-1, -2)
        at = torch.arange(t * top, device=x.device).view(t, top)
        y = every[s["ids"].long(), at if case["weighted"] else at // top]
    if case["swiglu"]:
        a, b = y.chunk(2, -1)
        y = a / (1 + torch.exp(-a)) * b
    if case["weighted"]:
        y = (y * s["w"][..., None]).sum(1)
    return y.to(torch.bfloat16)


# ------------------------------------------------------------------- calls
def run(state):
    case = state["case"]
    if not own:
        return {"norm": _plain_norm, "route": _plain_route, "int4": _plain_int4}[case["op"]](state)
    import mixture_experts_router_gb300 as cb
    if case["op"] == "norm":
        r = cb.rms_norm(state["x"], state["weight"], eps=EPS, residual=state["residual"], want=case["want"])
        out = {"sum": r.sum} if state["residual"] is not None else {}
        if case["want"] != "fp8":
            out["out"] = r.out
        if case["want"] != "out":
            out["codes"], out["scales"] = r.fp8.codes, r.fp8.scales
        return out
    if case["op"] == "route":
        ids, w = cb.route(state["logits"], case["top"], score=case["score"], bias=state["bias"], groups=case["groups"],
                          top_groups=case["top_groups"], group_score=case["group_score"], renormalise=case["renormalise"],
                          scale=2.5)
        return dict(ids=ids, w=w)
    x = state["x"] if state["x_scales"] is None else cb.Fp8Rows(state["x"], state["x_scales"])
    return cb.int4_matmul_few(x, cb.Int4Matrix(state["codes"], state["scales"], state["zeros"]), ids=state["ids"],
                              weights=state["w"], swiglu=case["swiglu"])


def work(case):
    if case["op"] == "norm":
        n, size = case["rows"] * case["cols"], 2 if case["dtype"] == "bf16" else 4
        blocks = case["rows"] * -(-case["cols"] // COLUMNS)
        each = size * (1 + 2 * case["residual"] + (case["want"] != "fp8")) + (case["want"] != "out")
        return dict(bytes=n * each + case["cols"] * size + 4 * blocks * (case["want"] != "out"), flops=8 * n)
    if case["op"] == "route":
        t, e = case["tokens"], case["experts"]
        return dict(bytes=t * (e * (2 if case["dtype"] == "bf16" else 4) + 8 * case["top"]) + 4 * e * case["bias"], flops=6 * t * e)
    t, n, k, e, top = (case[i] for i in ("tokens", "n", "k", "experts", "top"))
    used = e * (1 - (1 - top / e) ** t) if e else 1  # distinct experts of t rows
    x = t * (top if case["weighted"] else 1) * k * (2 if case["x"] == "bf16" else 1 + 4 / COLUMNS)
    y = t * (1 if case["weighted"] else top) * (n // 2 if case["swiglu"] else n) * 2
    return dict(bytes=used * n * (k / 2 + 5 * k / case["group"]) + x + y, flops=2 * t * top * n * k)


# -------------------------------------------------------- exact, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "route": _exact_route, "int4": _exact_int4}[case["op"]](s)


def _e4m3_64(v):
    """Nearest e4m3 values of v in 64 bits: 8 steps to a power of two, of 2^-9 below 2^-6."""
    e = torch.frexp(v.abs().clamp_min(2.0 ** -6)).exponent.double() - 1
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_norm(s):
    case, h = s["case"], s["x"].double()
    if s["residual"] is not None:
        h = h + s["residual"].double()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"].double()
    out = {"sum": h} if s["residual"] is not None else {}
    if case["want"] != "fp8":
        out["out"] = y
    if case["want"] != "out":
        v = _columns(y)
        scale = v.abs().amax(-1) / 448
        out["codes"] = _e4m3_64(v / scale[..., None].clamp_min(1e-300)).view(y.shape[0], -1)[:, :case["cols"]]
        out["scales"] = scale
    return out


def _exact_route(s):
    case, l = s["case"], s["logits"].double()
    p = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, -1)
    w = torch.gather(p, 1, _choose(case, p, s["bias"]))
    w = w / w.sum(-1, keepdim=True) if case["renormalise"] else w
    return dict(ids=None, w=w * 2.5)


def _exact_int4(s):
    case, x = s["case"], _rows(s, torch.float64)
    if not case["experts"]:
        y = x @ _weights(s, torch.float64).T
    else:
        t, top = s["ids"].shape
        n = case["n"]
        y = torch.zeros((t, top, n), dtype=torch.float64, device=x.device)
        for e in sorted(set(s["ids"].flatten().tolist())):
            r, slot = torch.nonzero(s["ids"] == e, as_tuple=True)
            y[r, slot] = (x[r, slot] if case["weighted"] else x[r]) @ _weights(s, torch.float64, e).T
    if case["swiglu"]:
        a, b = y.chunk(2, -1)
        y = a * torch.sigmoid(a) * b
    if case["weighted"]:
        y = torch.einsum("tsn,ts->tn", y, s["w"].double())
    return y
