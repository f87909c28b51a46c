"""The layer on a routing that the caller has (cb_moe_forward_routed and its few-token form).

On the routing that the handle's own router chose the result has to be the router's own, bit for bit: the same
GEMMs over the same rows.  On another routing it is compared with 64 bits with the layer's own tolerance (mean
relative error 5e-3, as in the layer's tests)."""
import pytest
import torch

import gpu_harness
import mixture_experts_router_gb300 as cb
import synth
from mixture_experts_router_gb300 import build as cbuild


def test_refusals_before_cuda():
    cbuild.build()
    for f in (cb.cb_moe_forward_routed, cb.cb_moe_forward_routed_f32out):
        assert f(None, 16, 32, 48, 64) == cb.CB_ERR_INVALID_ARG
    for f in (cb.cb_moe_forward_few_routed, cb.cb_moe_forward_few_routed_f32out):
        assert f(None, 16, 1, 32, 48, 64) == cb.CB_ERR_INVALID_ARG
        assert f(None, 16, 17, 32, 48, 64) == cb.CB_ERR_INVALID_ARG


def weights(E, d, f, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = lambda *s: torch.empty(s, device="cuda").normal_(0, 0.02, generator=g).bfloat16()  # noqa: E731
    return g, (w(E, d), w(E, f, d), w(E, f, d), w(E, d, f))


def layer64(x, ids, w, w_gate, w_up, w_down):
    x, out = x.double(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    for e in range(w_gate.shape[0]):
        t, slot = torch.nonzero(ids == e, as_tuple=True)
        if len(t):
            g = x[t] @ w_gate[e].double().T
            h = g * torch.sigmoid(g) * (x[t] @ w_up[e].double().T)
            out[t] += w[t, slot].double()[:, None] * (h @ w_down[e].double().T)
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,f,E,k,kw", [
    (1, 256, 256, 1, 1, {}), (64, 256, 512, 8, 2, {}), (1000, 512, 256, 16, 4, {}), (333, 256, 256, 64, 6, {}),
    (5000, 256, 256, 128, 8, {}), (9000, 256, 256, 8, 8, {}), (100, 256, 512, 8, 2, dict(wdtype="int8")),
    (300, 256, 512, 20, 3, dict(wdtype="fp8")), (40, 512, 256, 8, 2, dict(wdtype="int4")), (70, 256, 256, 12, 1, dict(router="hash", hash_dims=3)),
    (200, 256, 256, 24, 3, dict(router="raw"))])
def test_the_routers_own_routing_gives_its_result(T, d, f, E, k, kw):
    layer = synth.make_layer(synth.Shape(name="given", T=T, d=d, f=f, E=E, k=k, **kw))
    gl = gpu_harness.GpuLayer(layer, flags=cb.CB_FLAG_GUARDS)
    try:
        gl.run()
        r = gl.routing()
        ids, w = torch.from_numpy(r["ids"]).cuda(), torch.from_numpy(r["w"]).cuda()
        out, out32 = torch.empty_like(gl.out), torch.empty_like(gl.out32)
        for _ in range(2):   # the second from a replayed graph
            for stream in (None, torch.cuda.Stream()):
                out.fill_(7), out32.fill_(7)
                torch.cuda.synchronize()
                gl.m.forward(gl.x, out, routing=(ids, w), stream=stream)
                gl.m.forward(gl.x, out32, f32out=True, routing=(ids, w), stream=stream)
                torch.cuda.synchronize()
                assert torch.equal(out, gl.out) and torch.equal(out32, gl.out32)
        again = gl.routing()
        for name in ("ids", "w", "counts", "offsets", "tok", "inv", "tile_offsets"):
            assert (again[name] == r[name]).all(), name
        n = min(T, 16)
        few, given = torch.empty_like(gl.out32[:n]), torch.empty_like(gl.out32[:n])
        gl.m.forward_few(gl.x[:n], few, f32out=True)
        gl.m.forward(gl.x, out)       # its own router again, after a given routing
        gl.m.forward_few(gl.x[:n], given, f32out=True, routing=(ids[:n], w[:n]))
        torch.cuda.synchronize()
        assert torch.equal(out, gl.out)
        same = (ids[:n] == torch.from_numpy(gl.routing()["ids"]).cuda()[:n]).all()
        assert same and (few - given).abs().max() <= 1e-4 * few.abs().max()   # the weights' last bits: the logits' sums have another order
        assert gl.m.last_error() == cb.CB_OK and gl.m.check_guards() == cb.CB_OK
    finally:
        gl.close()


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(50, 16, 4), (700, 64, 6)])
def test_routing_in_groups_through_the_layer(T, E, k):
    d, f = 512, 256
    g, (wr, wg, wu, wd) = weights(E, d, f, 3)
    layer = cb.MoELayer(T, d, f, E, k, wr, wg, wu, wd)
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    bias = torch.randn(E, generator=g, device="cuda") * 0.05
    out = torch.empty(T, d, dtype=torch.float32, device="cuda")
    s = torch.cuda.current_stream()
    for n in (T, 16, 3, 1):
        ids, w = cb.route(x[:n].float() @ wr.float().T, k, bias=bias, groups=8, top_groups=3, scale=2.5)
        if n == T:
            layer.forward(x, out, f32out=True, routing=(ids, w), stream=s)
        else:
            layer.forward_few(x[:n], out[:n], f32out=True, routing=(ids, w))
        want = layer64(x[:n], ids.long(), w, wg, wu, wd)
        assert (out[:n].double() - want).abs().sum() <= 5e-3 * want.abs().sum()
    # a captured step: routing and layer in one graph, on other tokens
    few, held = x[:4].clone(), torch.empty(4, d, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        r = cb.route(few.float() @ wr.float().T, k, bias=bias, groups=8, top_groups=3)
        layer.forward_few(few, held, routing=r)
    few.copy_(x[20:24])
    graph.replay()
    now = torch.empty_like(held)
    layer.forward_few(few, now, routing=cb.route(few.float() @ wr.float().T, k, bias=bias, groups=8, top_groups=3))
    assert torch.equal(held, now) and layer.last_error() == cb.CB_OK
    layer.close()


@pytest.mark.gpu
def test_routings_that_are_none():
    T, d, f, E, k = 40, 256, 256, 8, 3
    g, (wr, wg, wu, wd) = weights(E, d, f, 5)
    layer = cb.MoELayer(T, d, f, E, k, wr, wg, wu, wd, flags=cb.CB_FLAG_GUARDS)
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(-1)[:, :k].to(torch.int32).contiguous()
    w = torch.rand(T, k, generator=g, device="cuda")
    good = torch.empty(T, d, dtype=torch.float32, device="cuda")
    layer.forward(x, good, f32out=True, routing=(ids, w))
    assert layer.last_error() == cb.CB_OK
    bad = ids.clone()
    bad[2, 1], bad[3, 0], bad[5, 2], bad[7] = 8, -1, bad[5, 0], 1 << 30
    rows = [2, 3, 5, 7]
    rest = [t for t in range(T) if t not in rows]
    out = torch.empty_like(good)
    layer.forward(x, out, f32out=True, routing=(bad, w))
    assert layer.last_error() == cb.CB_ERR_DEVICE
    assert out[rows].isnan().all() and not out[rest].isnan().any()
    assert torch.allclose(out[rest], good[rest], rtol=1e-5, atol=1e-6)
    few, fine = torch.empty(16, d, dtype=torch.float32, device="cuda"), torch.empty(16, d, dtype=torch.float32, device="cuda")
    layer.forward_few(x[:16], fine, f32out=True, routing=(ids[:16].contiguous(), w[:16]))
    assert layer.last_error() == cb.CB_OK
    layer.forward_few(x[:16], few, f32out=True, routing=(bad[:16].contiguous(), w[:16]))
    assert layer.last_error() == cb.CB_ERR_DEVICE
    rest = [t for t in rest if t < 16]
    assert few[rows].isnan().all() and torch.allclose(few[rest], fine[rest], rtol=1e-5, atol=1e-6)
    assert layer.check_guards() == cb.CB_OK
    for r in ((ids.long(), w), (ids, w.double()), (ids[:3], w[:3]), (ids.cpu(), w), (ids[:, :2], w[:, :2])):
        with pytest.raises(ValueError):
            layer.forward(x, out, f32out=True, routing=r)
        with pytest.raises(ValueError):
            layer.forward_few(x[:16], few, f32out=True, routing=r)
    with pytest.raises(cb.CbMoeError):      # a result over the routing
        buf = torch.empty(T * d, dtype=torch.float32, device="cuda")
        layer.forward(x, buf.view(T, d), f32out=True, routing=(ids, buf[:T * k].view(T, k)))
    layer.close()


@pytest.mark.gpu
def test_captured_with_another_routing():
    """A captured forward reads the routing that is there when the graph runs."""
    T, d, f, E, k = 90, 256, 256, 12, 2
    g, (wr, wg, wu, wd) = weights(E, d, f, 7)
    layer = cb.MoELayer(T, d, f, E, k, wr, wg, wu, wd)
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    new = lambda: (torch.rand(T, E, generator=g, device="cuda").argsort(-1)[:, :k].to(torch.int32).contiguous(),  # noqa: E731
                   torch.rand(T, k, generator=g, device="cuda"))
    ids, w = new()
    out, want = torch.empty(T, d, dtype=torch.bfloat16, device="cuda"), torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x, out, stream=torch.cuda.current_stream(), routing=(ids, w))
    for _ in range(3):
        for t, v in zip((ids, w), new()):
            t.copy_(v)
        graph.replay()
        layer.forward(x, want, stream=torch.cuda.current_stream(), routing=(ids, w))
        assert torch.equal(out, want)
    assert layer.last_error() == cb.CB_OK
    layer.close()
