"""The operators' measured cases: quantisation to 4-bit floating point with block scales, the
product of two such matrices (one matrix, or one per expert), and the MoE layer for a few tokens.

Each case runs in a plain form (elementary torch operations) or, with `own` set, through the
library's own entry points, on the same inputs; `exact` is the definition in 64 bits.

Formats.  A row of 4-bit elements (e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) is packed
two to a byte, element 2i in the low nibble.  "mx": a power-of-two scale byte (2^(b - 127)) for
every 32 elements of a row; "nv": an e4m3 scale byte for every 16 elements and one fp32 scale of
the whole matrix.  Scale bytes are stored in tiles of 128 rows x 4 blocks:
[ceil(rows/128)][ceil(blocks/4)][row % 32][row / 32 % 4][block % 4].
"""
import math

import torch

own = False

BLOCK = {"mx": 32, "nv": 16}
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
WEIGHT_STD = 0.02


def listed():
    return [
        # one decode step's activations on their way into a 4-bit product
        dict(name="quantise-16x4096-nv", op="quantise", fmt="nv", rows=16, cols=4096, dtype="bf16"),
        # an expert's gate and up weights, quantised when a checkpoint is loaded
        dict(name="quantise-28672x4096-mx", op="quantise", fmt="mx", rows=28672, cols=4096, dtype="bf16"),
        # a dense (shared) expert's up projection for a single token
        dict(name="product-1x14336x4096-nv", op="product", fmt="nv", m=1, n=14336, k=4096, groups=0, out="bf16"),
        # its down projection for a decode batch
        dict(name="product-64x4096x14336-mx", op="product", fmt="mx", m=64, n=4096, k=14336, groups=0, out="bf16"),
        # a ragged slice with an odd number of blocks, fp32 result
        dict(name="product-333x1000x1184-nv", op="product", fmt="nv", m=333, n=1000, k=1184, groups=0, out="f32"),
        # a prefill batch through the up projection
        dict(name="product-4096x14336x4096-nv", op="product", fmt="nv", m=4096, n=14336, k=4096, groups=0, out="bf16"),
        # 64 experts' products over a skewed routing: rows of expert e padded to tiles of 128
        dict(name="experts-64-6144x1536x4096-mx", op="product", fmt="mx", m=6144, n=1536, k=4096, groups=64, out="bf16"),
        # the smallest layer: launch latency
        dict(name="layer-1-tiny-bf16", op="layer", tokens=1, d=256, f=512, experts=8, top=2, weights="bf16"),
        # one token of a layer of 8 large experts
        dict(name="layer-1-8x14336-bf16", op="layer", tokens=1, d=4096, f=14336, experts=8, top=2, weights="bf16"),
        # a few sequences decoding together: most experts are read
        dict(name="layer-8-8x14336-bf16", op="layer", tokens=8, d=4096, f=14336, experts=8, top=2, weights="bf16"),
        # three sequences over 128 small experts
        dict(name="layer-3-128x768-bf16", op="layer", tokens=3, d=2048, f=768, experts=128, top=4, weights="bf16"),
        # quantised experts, a small decode batch
        dict(name="layer-16-64x1536-int8", op="layer", tokens=16, d=4096, f=1536, experts=64, top=6, weights="int8"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["quantise", "product", "product", "layer", "layer"])
    if op == "quantise":
        cols = 32 * log(1, 448)
        return dict(op=op, fmt=rng.choice(["mx", "nv"]), rows=log(1, min(100000, 117000000 // cols)), cols=cols,
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "product":
        groups = rng.choice([0, 0, 0, rng.randint(2, 96)])
        n, k = log(8, 14336), 32 * log(1, 448)
        if groups:
            n, k = log(8, 3000), 32 * log(1, 128)
        m = log(1, max(2, min(8192, 200_000_000_000 // (n * k))))
        return dict(op=op, fmt=rng.choice(["mx", "nv"]), m=m, n=n, k=k, groups=groups,
                    out=rng.choice(["bf16", "bf16", "f32"]))
    experts = rng.choice([1, 4, 8, 16, 37, 64, 128, 256])
    d = 256 * rng.randint(1, 16)
    f = 256 * log(1, max(1, min(56, 1_400_000_000 // (3 * 256 * d * experts))))
    return dict(op=op, tokens=rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 9, 12, 16]), d=d, f=f, experts=experts,
                top=rng.randint(1, min(experts, 8)), weights=rng.choice(["bf16", "bf16", "int8", "int4", "fp8"]))


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, std, g, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _group_rows(case):
    """Rows of each expert, in proportion to 1/(e + 3): the last experts have few or none."""
    w = [1.0 / (e + 3) for e in range(case["groups"])]
    rows = [int(case["m"] * v / sum(w)) for v in w]
    rows[0] += case["m"] - sum(rows)
    return rows


def _matrix(x, fmt, g):
    """x quantised by its definition, as the program that holds such a matrix has it."""
    scale = (x.float().abs().amax() / (6.0 * 448.0)).reshape(1).clamp_min(1e-30) if fmt == "nv" else None
    q = _quantise(x, fmt, scale)
    return dict(codes=_pack(q["codes"]), scales=_tile(q["bytes"]), scale=scale, rows=x.shape[0], cols=x.shape[1])


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "quantise":
        # activations with a few large channels, as norms leave them
        x = _normal((case["rows"], case["cols"]), 1.0, g)
        x = (x * torch.where(torch.rand(case["cols"], generator=g, device="cuda") < 0.01, 8.0, 1.0)).to(TYPES[case["dtype"]])
        scale = (x.float().abs().amax() / (6.0 * 448.0)).reshape(1) if case["fmt"] == "nv" else None
        return dict(case=case, x=x, scale=scale)
    if case["op"] == "product":
        tiles = None
        m, b = case["m"], case["n"]
        if case["groups"]:
            counts = _group_rows(case)
            ends = torch.tensor([0] + [(c + 127) // 128 for c in counts]).cumsum(0)
            tiles = ends.to(torch.int32).cuda()
            m, b = int(ends[-1]) * 128, case["n"] * case["groups"]
        x = _normal((m, case["k"]), 1.0, g, torch.bfloat16)
        if case["groups"]:  # rows past an expert's own are padding
            for start, c in zip(ends.tolist(), counts):
                x[start * 128 + c:start * 128 + (c + 127) // 128 * 128] = 0
        a = _matrix(x, case["fmt"], g)
        del x
        if case["groups"]:  # each expert's matrix starts a tile of its own
            n = case["n"]
            parts = [_matrix(_normal((n, case["k"]), WEIGHT_STD, g, torch.bfloat16), case["fmt"], g) for _ in range(case["groups"])]
            w = dict(codes=torch.cat([p["codes"] for p in parts]).view(case["groups"], n, -1),
                     scales=torch.stack([p["scales"] for p in parts]), rows=n, cols=case["k"],
                     scale=torch.cat([p["scale"] for p in parts]) if case["fmt"] == "nv" else None)
        else:
            w = _matrix(_normal((b, case["k"]), WEIGHT_STD, g, torch.bfloat16), case["fmt"], g)
        return dict(case=case, a=a, w=w, tiles=tiles)
    return _prepare_layer(case, g)


def _prepare_layer(case, g):
    d, f, e, kind = case["d"], case["f"], case["experts"], case["weights"]
    s = dict(case=case, x=_normal((case["tokens"], d), 1.0, g, torch.bfloat16),
             wr=_normal((e, d), WEIGHT_STD, g, torch.bfloat16), bias=_normal((e,), 0.1, g))
    for name, rows, cols in (("gate", f, d), ("up", f, d), ("down", d, f)):
        if kind == "bf16":
            w = torch.empty((e, rows, cols), device="cuda", dtype=torch.bfloat16)
            w.normal_(0.0, WEIGHT_STD, generator=g)
        elif kind == "int8":
            w = torch.randn((e, rows, cols), generator=g, device="cuda").mul_(40).round_().clamp_(-127, 127).to(torch.int8)
        elif kind == "int4":
            z = torch.randint(6, 10, (e, rows), generator=g, device="cuda", dtype=torch.uint8)
            q = torch.randn((e, rows, cols), generator=g, device="cuda").mul_(2.5).round_().clamp_(-6, 6)
            q = q.add_(z[..., None]).to(torch.uint8)
            w = q[..., 0::2] | (q[..., 1::2] << 4)
            s["z_" + name] = z
            del q
        else:
            w = torch.randn((e, rows, cols), generator=g, device="cuda").mul_(32).clamp_(-448, 448).to(torch.float8_e4m3fn)
        s["w_" + name] = w
        if kind != "bf16":
            lo, hi = (0.006, 0.010) if kind == "int4" else (0.5e-3, 1.0e-3)
            s["s_" + name] = torch.rand((e, rows), generator=g, device="cuda") * (hi - lo) + lo
    if own:  # the layer handle that a serving program keeps
        import mixture_experts_router_gb300 as cb
        s["layer"] = cb.MoELayer(16, d, f, e, case["top"], s["wr"], s["w_gate"], s["w_up"], s["w_down"],
                                 router_bias=s["bias"], s_gate=s.get("s_gate"), s_up=s.get("s_up"),
                                 s_down=s.get("s_down"), z_gate=s.get("z_gate"), z_up=s.get("z_up"),
                                 z_down=s.get("z_down"), wdtype=kind)
    return s


# ------------------------------------------------------------- plain forms
def _two_to(e):
    """2^e in 64 bits, from the bits (a device's pow and exp2 need not be exact)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _quantise(x, fmt, scale):
    """Signed 4-bit codes (0..15) and scale bytes of x's rows, with the values that they stand for.
    The comparisons with the borders between two values are made in 64 bits, where they are exact."""
    b = BLOCK[fmt]
    v = x.double().view(x.shape[0], -1, b)
    top = v.abs().amax(-1)
    if fmt == "mx":
        # the largest element's exponent less 2, e2m1's own largest
        byte = torch.where(top > 0, torch.frexp(top).exponent - 1 - 2 + 127, 0).clamp(0, 254)
        unit = _two_to(byte - 127)
    else:
        t = (top / (6.0 * scale.double())).clamp_max(448.0)
        e = (torch.frexp(t).exponent - 1).clamp_min(-6)
        steps = torch.round(t * _two_to(3 - e))  # 8..16 steps of 2^(e - 3), fewer below 2^-6
        unit = (steps * _two_to(e - 3)).clamp_max(448.0)
        e = (torch.frexp(unit).exponent - 1).clamp_min(-6)
        byte = torch.where(unit >= 2.0 ** -6, (e + 7) * 8 - 8, 0) + (unit * _two_to(3 - e)).int()
        unit = unit * scale.double()
    w = torch.where(unit[..., None] > 0, v.abs() / unit[..., None], 0.0)
    code = (w > 0.25).to(torch.uint8) + (w >= 0.75) + (w > 1.25) + (w >= 1.75) + (w > 2.5) + (w >= 3.5) + (w > 5.0)
    code = code + 8 * (v < 0)
    return dict(codes=code.to(torch.uint8).view(x.shape), bytes=byte.to(torch.uint8))


def _pack(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def _tile(scales):
    """Scale bytes [rows][blocks] in their stored order."""
    r, c = (scales.shape[0] + 127) // 128, (scales.shape[1] + 3) // 4
    p = torch.zeros((r * 128, c * 4), dtype=torch.uint8, device=scales.device)
    p[:scales.shape[0], :scales.shape[1]] = scales
    return p.view(r, 4, 32, c, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _untile(scales, rows, blocks):
    r, c = (rows + 127) // 128, (blocks + 3) // 4
    lead = scales.shape[:-1]
    p = scales.view(*lead, r, c, 32, 4, 4)
    order = list(range(len(lead))) + [len(lead) + i for i in (0, 3, 2, 1, 4)]
    return p.permute(order).reshape(*lead, r * 128, c * 4)[..., :rows, :blocks]


def _scale_values(b, fmt, dtype):
    b = b.to(torch.int32)
    if fmt == "mx":
        return _two_to(b - 127).to(dtype)
    return torch.where(b < 8, b.double() * 2.0 ** -9, (8 + (b & 7)) * _two_to((b >> 3) - 10)).to(dtype)


def _element_values(packed, dtype):
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=dtype, device=packed.device)
    return torch.stack([table[(packed & 15).int()], table[(packed >> 4).int()]], -1).flatten(-2)


def _values(m, fmt, dtype=torch.float32):
    """A stored matrix's values without its own scale (exact in 32 bits)."""
    v = _element_values(m["codes"], dtype)
    b = BLOCK[fmt]
    s = _scale_values(_untile(m["scales"], m["rows"], m["cols"] // b), fmt, dtype)
    return (v.unflatten(-1, (-1, b)) * s[..., None]).flatten(-2)


def _plain_quantise(s):
    fmt = s["case"]["fmt"]
    q = _quantise(s["x"], fmt, s["scale"])
    v = _element_values(_pack(q["codes"]), torch.float32).view(*q["bytes"].shape, BLOCK[fmt])
    v = v * _scale_values(q["bytes"], fmt, torch.float32)[..., None]
    v = v * s["scale"] if fmt == "nv" else v
    return v.view(s["x"].shape).to(s["x"].dtype)


def _plain_product(s):
    case, a, w = s["case"], s["a"], s["w"]
    x, y = _values(a, case["fmt"]), _values(w, case["fmt"])
    if s["tiles"] is None:
        out = x @ y.T
        out = out * (a["scale"] * w["scale"]) if case["fmt"] == "nv" else out
    else:  # each tile of 128 rows by its expert's matrix
        tile = torch.arange(x.shape[0] // 128, device=x.device)
        e = torch.searchsorted(s["tiles"][1:], tile, right=True).clamp_max(case["groups"] - 1)
        out = x.view(-1, 128, x.shape[1]) @ y[e].transpose(1, 2)
        out = out * (a["scale"] * w["scale"][e])[:, None, None] if case["fmt"] == "nv" else out
        out = out.view(x.shape[0], -1)
    return out.to(TYPES[case["out"]])


def _weights(s, name, dtype, pick=slice(None)):
    w, kind = s["w_" + name][pick], s["case"]["weights"]
    if kind == "bf16":
        return w.to(dtype)
    if kind == "int4":
        w = torch.stack([w & 15, w >> 4], -1).flatten(-2).to(dtype) - s["z_" + name][pick][..., None].to(dtype)
    return w.to(dtype) * s["s_" + name][pick][..., None].to(dtype)


def _plain_layer(s):
    x, k = s["x"].float(), s["case"]["top"]
    logits = x @ s["wr"].float().T + s["bias"]
    best, ids = torch.sort(logits, dim=-1, descending=True, stable=True)  # ties: the lower expert first
    gate = torch.exp(best[:, :k] - best[:, :1])
    gate = gate / gate.sum(-1, keepdim=True)
    share = torch.zeros_like(logits).scatter_(1, ids[:, :k], gate)
    g = x @ _weights(s, "gate", torch.float32).transpose(1, 2)
    u = x @ _weights(s, "up", torch.float32).transpose(1, 2)
    y = (g / (1 + torch.exp(-g)) * u) @ _weights(s, "down", torch.float32).transpose(1, 2)
    return (y * share.T[..., None]).sum(0).to(torch.bfloat16)


# ------------------------------------------------------------------- calls
def _fp4(cb, m, fmt):
    return cb.Fp4Matrix(fmt, m["rows"], m["cols"], m["codes"], m["scales"], m["scale"])


def run(state):
    case = state["case"]
    if not own:
        return {"quantise": _plain_quantise, "product": _plain_product, "layer": _plain_layer}[case["op"]](state)
    import mixture_experts_router_gb300 as cb
    if case["op"] == "quantise":
        q = cb.fp4_quantize(state["x"], case["fmt"], tensor_scale=state["scale"])
        return cb.fp4_dequantize(q, state["x"].dtype)
    if case["op"] == "product":
        return cb.fp4_matmul(_fp4(cb, state["a"], case["fmt"]), _fp4(cb, state["w"], case["fmt"]),
                             dtype=TYPES[case["out"]], tile_offsets=state["tiles"])
    out = torch.empty_like(state["x"])
    return state["layer"].forward_few(state["x"], out)


def work(case):
    if case["op"] == "quantise":
        n, size = case["rows"] * case["cols"], 2 if case["dtype"] == "bf16" else 4
        return dict(bytes=n * (2 * size + 0.5 + 1 / BLOCK[case["fmt"]]), flops=2 * n)
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        per = 0.5 + 1 / BLOCK[case["fmt"]]
        mats = 1
        if case["groups"]:
            m, mats = sum(_group_rows(case)), sum(c > 0 for c in _group_rows(case))
        return dict(bytes=(m + n * mats) * k * per + m * n * (2 if case["out"] == "bf16" else 4), flops=2 * m * n * k)
    t, d, f, e, k = (case[i] for i in ("tokens", "d", "f", "experts", "top"))
    used = e * (1 - (1 - k / e) ** t)  # distinct experts of t tokens
    size = {"bf16": 2, "int8": 1, "fp8": 1, "int4": 0.5}[case["weights"]]
    return dict(bytes=used * 3 * d * f * size + e * d * 2 + t * d * 4, flops=6 * t * k * d * f + 2 * t * e * d)


# -------------------------------------------------------- exact, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantise":
        return _exact_quantise(s)
    if case["op"] == "product":
        return _exact_product(s)
    return _exact_layer(s)


def _power(e):
    return torch.tensor([2.0 ** i for i in range(-160, 161)], dtype=torch.float64, device=e.device)[e.long() + 160]


def _exact_quantise(s):
    """Nearest values, ties to the even code: steps of 1/2 below 2, of 1 below 4, of 2 up to 6."""
    x, fmt = s["x"].double(), s["case"]["fmt"]
    v = x.view(x.shape[0], -1, BLOCK[fmt])
    top = v.abs().amax(-1, keepdim=True)
    if fmt == "mx":
        unit = _power(torch.frexp(top.clamp_min(2.0 ** -125)).exponent - 3)
    else:
        g = s["scale"].double()
        t = top / (6 * g)
        step = _power(torch.frexp(t.clamp_min(2.0 ** -6)).exponent - 4)
        unit = (torch.round(t / step) * step).clamp_max(448.0) * g
    r = torch.where(unit > 0, v.abs() / unit, 0.0)
    step = torch.where(r < 2, 0.5, torch.where(r < 4, 1.0, 2.0))
    return ((torch.round(r / step) * step).clamp_max(6.0) * unit * torch.sign(v)).view(x.shape)


def _decode64(m, fmt):
    """Values in 64 bits, element by element from the bits."""
    c = torch.stack([m["codes"] & 15, m["codes"] >> 4], -1).flatten(-2).long()
    e, half = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e == 0, half / 2, _power(e - 1) * (1 + half / 2)) * (1 - 2 * (c >> 3)).double()
    b, rows = BLOCK[fmt], m["rows"]
    n = m["cols"] // b
    r, k = torch.arange(rows, device=c.device)[:, None], torch.arange(n, device=c.device)[None]
    at = ((r // 128 * ((n + 3) // 4) + k // 4) * 32 + r % 32) * 16 + r // 32 % 4 * 4 + k % 4
    q = m["scales"][..., at].long()
    if fmt == "mx":
        q = _power(q - 127)
    else:
        q = torch.where(q < 8, (q & 7).double() / 8 * 2.0 ** -6, (1 + (q & 7).double() / 8) * _power((q >> 3) - 7))
    return v * q.repeat_interleave(b, -1)


def _exact_product(s):
    fmt, a, w = s["case"]["fmt"], s["a"], s["w"]
    x = _decode64(a, fmt)
    x = x * a["scale"].double() if fmt == "nv" else x
    if s["tiles"] is None:
        y = _decode64(w, fmt)
        return x @ (y * w["scale"].double() if fmt == "nv" else y).T
    out = torch.zeros((x.shape[0], w["rows"]), dtype=torch.float64, device=x.device)
    ends = s["tiles"].tolist()
    for e in range(s["case"]["groups"]):
        lo, hi = ends[e] * 128, ends[e + 1] * 128
        if hi > lo:
            y = _decode64(dict(w, codes=w["codes"][e], scales=w["scales"][e]), fmt)
            out[lo:hi] = x[lo:hi] @ (y * w["scale"][e].double() if fmt == "nv" else y).T
    return out


def _exact_layer(s):
    x, k = s["x"].double(), s["case"]["top"]
    logits = x @ s["wr"].double().T + s["bias"].double()
    out = torch.zeros_like(x)
    ids = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :k]
    gate = torch.softmax(torch.gather(logits, 1, ids), -1)
    for e in sorted(set(ids.flatten().tolist())):
        t, slot = torch.nonzero(ids == e, as_tuple=True)
        g = x[t] @ _weights(s, "gate", torch.float64, e).T
        h = g * torch.sigmoid(g) * (x[t] @ _weights(s, "up", torch.float64, e).T)
        out[t] += gate[t, slot][:, None] * (h @ _weights(s, "down", torch.float64, e).T)
    return out
