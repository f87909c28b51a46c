"""examples/serving_block.py's routed block against plain 64-bit arithmetic on the values that its matrices stand
for.  Everything before the experts is recomputed from the program's own rows, so the tolerance of a decode step
counts the roundings of h and of the result (half a bf16 step each, h's spread over f terms); the handle's own
tolerance holds for prompts (mean relative error 5e-3, as in the layer's tests)."""
import os
import sys

import pytest
import torch

import mixture_experts_router_gb300 as cb

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def values(m, e):
    q = torch.stack([m.codes[e] & 15, m.codes[e] >> 4], -1).flatten(-2).double()
    up = lambda t: t[e].double().T.repeat_interleave(m.group, -1)  # noqa: E731
    return (q - up(m.zeros)) * up(m.scales)


def experts64(x, ids, w, gate_up, down):
    """gate_up(e), down(e): matrices in 64 bits."""
    out = torch.zeros_like(x)
    for e in sorted(set(ids.flatten().tolist())):
        t, slot = torch.nonzero(ids == e, as_tuple=True)
        g, u = (x[t] @ gate_up(e).T).chunk(2, -1)
        out[t] += w[t, slot].double()[:, None] * ((g * torch.sigmoid(g) * u) @ down(e).T)
    return out


@pytest.mark.parametrize("group", [32, 64, 128])
def test_block(group):
    import serving_block as sb
    block, (_, wg, wu, wd) = sb.random_routed_block(d=1024, f=512, E=32, top_k=4, prompt_tokens=120, group=group, seed=group)
    x, res = torch.randn(120, 1024, device="cuda").bfloat16(), torch.randn(120, 1024, device="cuda").bfloat16()
    for n in (1, 3, 16, 3):      # the last from a graph that is there already
        part = slice(0, n) if n != 3 else slice(5, 8)
        got, new = block.decode(x[part], res[part])
        r = cb.rms_norm(x[part], block.norm, residual=res[part], want="both")
        ids, w = cb.route(r.out @ block.router_t, **block.how)
        rows = r.fp8.codes.double() * r.fp8.scales.double().repeat_interleave(128, -1)
        want = experts64(rows, ids, w, lambda e: values(block.up, e), lambda e: values(block.down, e))
        assert torch.equal(new, r.sum)
        assert (got.double() - want).norm() <= 2 * torch.finfo(torch.bfloat16).eps / 2 * want.norm()
    for n in (120, 77):
        got, new = block.prompt(x[:n], res[:n])
        r = cb.rms_norm(x[:n], block.norm, residual=res[:n])
        rows = torch.cat([r.out, r.out.new_zeros((120 - n, 1024))])      # the same product as the program's
        ids, w = (t[:n] for t in cb.route(rows @ block.router_t, **block.how))
        want = experts64(r.out.double(), ids, w, lambda e: torch.cat([wg[e], wu[e]]).double(), lambda e: wd[e].double())
        assert torch.equal(new, r.sum)
        assert (got.double() - want).abs().sum() <= 5e-3 * want.abs().sum()
    assert block.layer.last_error() == cb.CB_OK
    # 4-bit weights stand for the 16-bit ones to within a step of their group (a value and the zero point are rounded)
    for m, e, w16 in ((block.up, 3, torch.cat([wg[3], wu[3]])), (block.down, 5, wd[5])):
        step = m.scales[e].T.repeat_interleave(m.group, -1).double()
        assert ((values(m, e) - w16.double()).abs() <= step * 1.01).all()
