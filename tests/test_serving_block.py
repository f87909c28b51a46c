"""examples/serving_block.py against plain 64-bit arithmetic on the values that its 4-bit matrices
stand for.  The quantised activations are recomputed from the program's own intermediate values, so
the tolerances count only roundings: half a bf16 step of the result, and for the routed experts the
layer's own tolerance (mean relative error 5e-3, as in the layer's tests)."""
import os
import sys

import pytest
import torch

import mixture_experts_router_gb300 as cb

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
BF16 = torch.finfo(torch.bfloat16).eps / 2


def values(m, e=None):
    """What a 4-bit matrix stands for, in 64 bits (the reading back is tested on its own)."""
    if e is not None:
        n = m.scales.numel() // m.groups
        m = cb.Fp4Matrix(m.format, m.rows, m.cols, m.codes[e], m.scales.view(m.groups, n)[e],
                         None if m.tensor_scale is None else m.tensor_scale[e:e + 1])
    return cb.fp4_dequantize(m, torch.float32).double()


def quantised(x, like, scale):
    return values(cb.fp4_quantize(x, like.format, scale))


def dense64(dense, x):
    import serving_block as sb
    gu = quantised(x, dense, dense.act_scale) @ values(dense.up).T
    # H as the program has it: its products are tested on their own, here they feed the second one
    h = sb.swiglu(cb.fp4_matmul(cb.fp4_quantize(x, dense.format, dense.act_scale), dense.up))
    g, u = gu.chunk(2, -1)
    want_h = g * torch.sigmoid(g) * u
    assert (h.double() - want_h).norm() <= 3 * BF16 * want_h.norm()   # gate, up and h each rounded to bf16
    return quantised(h, dense, dense.act_scale) @ values(dense.down).T


def routed64(x, w_router, w_gate, w_up, w_down, k):
    x = x.double()
    logits = x @ w_router.double().T
    best, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    gate = torch.softmax(best[:, :k], -1)
    out = torch.zeros_like(x)
    for e in range(w_gate.shape[0]):
        t, slot = torch.nonzero(ids[:, :k] == e, as_tuple=True)
        if len(t):
            g = x[t] @ w_gate[e].double().T
            h = g * torch.sigmoid(g) * (x[t] @ w_up[e].double().T)
            out[t] += gate[t, slot][:, None] * (h @ w_down[e].double().T)
    return out, ids[:, :k], gate


@pytest.mark.parametrize("format", ["mx", "nv"])
def test_block_decodes_and_runs_prompts(format):
    import serving_block as sb
    block, routed, _ = sb.random_block(d=1024, f=512, E=16, top_k=4, dense_f=768, prompt_tokens=200, format=format)
    x = torch.randn(200, 1024, device="cuda").bfloat16()
    for got, rows in [(block.prompt(x), 200)] + [(block.decode(x[:n]), n) for n in (1, 3, 16)] + [(block.decode(x[7:10]), slice(7, 10))]:
        part = x[rows] if isinstance(rows, slice) else x[:rows]
        want = routed64(part, *routed, 4)[0] + dense64(block.dense, part)
        err = (got.double() - want).abs().sum() / want.abs().sum()
        assert err <= 5e-3, (rows, float(err))
    assert block.layer.last_error() == cb.CB_OK


@pytest.mark.parametrize("format", ["mx", "nv"])
def test_routed_experts_in_4_bits(format):
    import serving_block as sb
    d, f, E, k, T = 512, 256, 12, 3, 150
    block, routed, _ = sb.random_block(d=d, f=f, E=E, top_k=k, dense_f=256, prompt_tokens=T, format=format, seed=3)
    x = torch.randn(T, d, device="cuda").bfloat16()
    block.prompt(x)
    experts = sb.Fp4Experts(*routed[1:], format=format)
    got = experts(x, block.layer).double()
    _, ids, gate = routed64(x, *routed, k)
    scale = torch.full((1,), 32.0 / 448.0, device="cuda") if format == "nv" else None
    xq = quantised(x, experts, scale)
    want = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, slot = torch.nonzero(ids == e, as_tuple=True)
        if len(t):
            gu = (xq[t] @ values(experts.up, e).T).float().bfloat16()
            want[t] += gate[t, slot][:, None] * (quantised(sb.swiglu(gu), experts, scale) @ values(experts.down, e).T)
    # a value next to a border may go to the other 4-bit neighbour after the product's rounding
    assert (got - want).abs().sum() / want.abs().sum() <= 5e-3
