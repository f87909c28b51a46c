"""The layer for a few tokens (cb_moe_forward_few) against its formulas in 64 bits.

The tolerance of an output element is derived, element by element, from the roundings that the
layer makes:
  * fp32 sums: a dot product over K is a chain of at most K / 16 additions (the MMA's K) plus the
    joins of 16 warps, each off by at most 2^-23 of the sum of the terms' magnitudes (the MMA may
    truncate where an addition rounds): c(K) = (K / 16 + 32) 2^-23;
  * SiLU's fp32 evaluation: 2^-18 relative (fast exponential and divide);
  * H rounded to bf16: half a step, 2^-8 relative;
  * the gate's weights: 1e-5 (as everywhere in the layer's tests);
  * the output rounded to bf16: half a step.
"""
import os

import numpy as np
import pytest
import torch

import mixture_experts_router_gb300 as cb
import oracle
import synth
from mixture_experts_router_gb300 import build as cbuild

BF16 = torch.finfo(torch.bfloat16).eps / 2


# ------------------------------------------------------------------ no GPU
def test_refusals_before_any_cuda_call():
    cbuild.build()
    assert cb.cb_moe_forward_few(None, 16, 1, 32, 0) == cb.CB_ERR_INVALID_ARG
    assert cb.cb_moe_forward_few_f32out(None, 16, 1, 32, 0) == cb.CB_ERR_INVALID_ARG
    assert cb.CB_MOE_MAX_FEW == 16


# ----------------------------------------------------------------- helpers
def weights64(layer, name, e):
    """Expert e's dequantised matrix in 64 bits."""
    w, kind = getattr(layer, "w" + name)[e], layer.shape.wdtype
    if kind == "bf16":
        return synth.bf16_bits_to_f32(w).astype(np.float64)
    if kind == "int4":
        v = synth.unpack_int4(w).astype(np.float64) - getattr(layer, "z" + name)[e].astype(np.float64)[:, None]
    elif kind == "fp8":
        v = torch.from_numpy(w.copy()).view(torch.float8_e4m3fn).double().numpy()
    else:
        v = w.astype(np.float64)
    return v * getattr(layer, "s" + name)[e].astype(np.float64)[:, None]


def reference(layer, ids, w):
    """Outputs in 64 bits with H rounded to bf16's nearest, and the bound of each."""
    s = layer.shape
    x = synth.bf16_bits_to_f32(layer.x).astype(np.float64)
    n = x.shape[0]
    out, tol = np.zeros((n, s.d)), np.zeros((n, s.d))
    cd, cf = (s.d / 16 + 32) * 2.0 ** -23, (s.f / 16 + 32) * 2.0 ** -23
    for e in sorted(set(ids.ravel().tolist())):
        wg, wu, wd = (weights64(layer, m, e) for m in ("g", "u", "d"))
        for t, slot in zip(*np.nonzero(ids == e)):
            g, u = wg @ x[t], wu @ x[t]
            dg, du = cd * (np.abs(wg) @ np.abs(x[t])), cd * (np.abs(wu) @ np.abs(x[t]))
            sig = 1 / (1 + np.exp(-g))
            h = g * sig * u
            # |SiLU'| <= 1.1; the rounding of h once more for its being off
            dh = (1.1 * dg * (np.abs(u) + du) + np.abs(g * sig) * (du + 2.0 ** -18 * np.abs(u)))
            dh = dh + BF16 * (np.abs(h) + dh)
            y = wd @ h
            dy = np.abs(wd) @ dh + cf * (np.abs(wd) @ (np.abs(h) + dh))
            out[t] += w[t, slot] * y
            tol[t] += np.abs(w[t, slot]) * dy + 1e-5 * np.abs(y) + cf * np.abs(w[t, slot] * y)
    return out, tol


class Run:
    """A handle of `T` tokens on a synthetic layer of n tokens."""

    def __init__(self, shape, T=None, flags=0):
        import gpu_harness as gh
        self.layer = synth.make_layer(shape)
        s = shape
        w = {n: gh.to_dev(getattr(self.layer, n)) for n in ("wr", "bias", "wg", "wu", "wd", "sg", "su", "sd", "wh", "zg", "zu", "zd")}
        self.m = cb.MoELayer(s.T if T is None else T, s.d, s.f, s.E, s.k, w["wr"], w["wg"], w["wu"], w["wd"],
                             router_bias=w["bias"], s_gate=w["sg"], s_up=w["su"], s_down=w["sd"], flags=flags,
                             router=s.router, w_hash=w["wh"], z_gate=w["zg"], z_up=w["zu"], z_down=w["zd"],
                             wdtype=s.wdtype)
        self.x = gh.to_dev(self.layer.x)

    def few(self, f32=False, x=None):
        x = self.x if x is None else x
        out = torch.full(x.shape, 7.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        self.m.forward_few(x, out, f32out=f32)
        torch.cuda.synchronize()
        assert self.m.last_error() == cb.CB_OK
        return out


def check(r):
    """Both output types of r against the reference, but for tokens at a near tie of the router."""
    o = oracle.Oracle(r.layer)
    ids, w, gap_k, _ = o.route()
    keep = (r.layer.shape.router == "hash") | (gap_k >= 1e-5) | (gap_k == 0)
    assert keep.all(), "pick a seed without near ties"
    ref, tol = reference(r.layer, ids, w)
    f32 = r.few(f32=True).double().cpu().numpy()
    b16 = r.few().double().cpu().numpy()
    assert np.all(np.abs(f32 - ref) <= tol + 2.0 ** -24 * np.abs(ref)), np.max(np.abs(f32 - ref) / (tol + 1e-30))
    assert np.all(np.abs(b16 - ref) <= tol + BF16 * (np.abs(ref) + tol)), np.max(np.abs(b16 - ref) / (tol + BF16 * np.abs(ref) + 1e-30))
    return f32


# ------------------------------------------------------------------- tests
@pytest.mark.gpu
@pytest.mark.parametrize("wdtype", ["bf16", "int8", "int4", "fp8"])
@pytest.mark.parametrize("n,d,f,E,k", [
    (1, 256, 256, 1, 1), (1, 256, 512, 8, 2), (2, 512, 256, 5, 5), (3, 768, 1280, 16, 3), (7, 1024, 256, 64, 6),
    (8, 256, 768, 3, 2), (9, 512, 512, 37, 4), (16, 256, 256, 256, 16), (16, 1280, 512, 4, 2), (5, 4608, 256, 8, 2),
])
def test_matches_the_formulas(wdtype, n, d, f, E, k):
    check(Run(synth.custom_shape("few", n, d, f, E, k, wdtype=wdtype, seed=11 + n + E)))


@pytest.mark.gpu
@pytest.mark.parametrize("wdtype", ["bf16", "int4"])
@pytest.mark.parametrize("n", [8, 9, 16])
def test_all_tokens_of_many_choose_the_same_experts(wdtype, n):
    """More than 8 tokens at experts that are few of many: each expert is taken in parts."""
    shape = synth.custom_shape("few", n, 512, 512, 48, 4, wdtype=wdtype, seed=14)
    r = Run(shape)
    bias = np.zeros(48, np.float32)
    bias[[3, 17, 18, 40]] = [50, 40, 30, 20]
    r.layer.bias = bias
    w = {m: torch.from_numpy(getattr(r.layer, m)).cuda() for m in ("wr", "wg", "wu", "wd")}
    if wdtype == "bf16":
        w = {m: t.view(torch.bfloat16) for m, t in w.items()}
    else:
        w["wr"] = w["wr"].view(torch.bfloat16)
    opt = {m: torch.from_numpy(getattr(r.layer, m)).cuda() if getattr(r.layer, m) is not None else None
           for m in ("sg", "su", "sd", "zg", "zu", "zd")}
    r.m = cb.MoELayer(n, 512, 512, 48, 4, w["wr"], w["wg"], w["wu"], w["wd"], router_bias=torch.from_numpy(bias).cuda(),
                      s_gate=opt["sg"], s_up=opt["su"], s_down=opt["sd"], z_gate=opt["zg"], z_up=opt["zu"],
                      z_down=opt["zd"], wdtype=wdtype)
    check(r)


@pytest.mark.gpu
@pytest.mark.parametrize("router", ["raw", "hash"])
@pytest.mark.parametrize("n,E,k", [(1, 8, 2), (11, 20, 3)])
def test_other_routers(router, n, E, k):
    check(Run(synth.with_router(synth.custom_shape("few", n, 512, 512, E, k, seed=3), router)))


@pytest.mark.gpu
@pytest.mark.parametrize("wdtype", ["bf16", "int8"])
def test_one_large_layer(wdtype):
    """Many tiles per block, several turns of the 16 warps per row."""
    check(Run(synth.custom_shape("few", 4, 4096, 7168, 8, 2, wdtype=wdtype, seed=5)))


@pytest.mark.gpu
def test_int8_rows_in_blocks_of_64(monkeypatch):
    monkeypatch.setenv("CB_MOE_INT8", "smem")
    check(Run(synth.custom_shape("few", 6, 512, 768, 8, 2, wdtype="int8", seed=9)))


@pytest.mark.gpu
@pytest.mark.parametrize("wdtype", ["bf16", "int4"])
def test_on_a_handle_of_another_size_between_its_forwards(wdtype):
    """The handle's full forward and its routing are not disturbed, nor the few tokens' result."""
    shape = synth.custom_shape("few", 200, 512, 512, 8, 2, wdtype=wdtype, seed=21)
    r = Run(shape, flags=cb.CB_FLAG_GUARDS)
    full = torch.empty((200, 512), dtype=torch.bfloat16, device="cuda")
    again = torch.empty_like(full)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    r.m.forward(r.x, full, stream=side)
    few = torch.empty((16, 512), dtype=torch.bfloat16, device="cuda")
    r.m.forward_few(r.x[:16], few)               # waits for the forward on the other stream
    r.m.forward(r.x, again, stream=side)
    torch.cuda.synchronize()
    assert r.m.last_error() == cb.CB_OK and r.m.check_guards() == cb.CB_OK
    assert torch.equal(full, again)
    # both are within the tolerance of the same values; here: of each other's, in norm
    assert (few.double() - full[:16].double()).norm() <= 2 * BF16 * full[:16].double().norm()


@pytest.mark.gpu
@pytest.mark.parametrize("wdtype", ["bf16", "int8", "int4", "fp8"])
@pytest.mark.parametrize("n", [6, 14])
def test_long_streams_repeat_bit_for_bit(wdtype, n):
    """Hundreds of stages per block, two n-tiles and one: every run gives the first one's bits."""
    r = Run(synth.custom_shape("few", n, 2048, 1536, 24, 6, wdtype=wdtype, seed=31))
    want = check(r)
    for _ in range(200):
        out = torch.empty(r.x.shape, dtype=torch.float32, device="cuda")
        r.m.forward_few(r.x, out, f32out=True)
        assert np.array_equal(out.double().cpu().numpy(), want)
    assert r.m.last_error() == cb.CB_OK


@pytest.mark.gpu
def test_repeats_bit_for_bit_and_in_a_graph():
    r = Run(synth.custom_shape("few", 13, 768, 1024, 16, 4, seed=2), T=16)
    want = r.few()
    for _ in range(5):
        assert torch.equal(r.few(), want)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=stream):
        r.m.forward_few(r.x, out, stream=stream)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.gpu
def test_a_token_keeps_to_itself():
    """NaN and infinities in one token leave every other token's bits alone, whoever shares its experts."""
    r = Run(synth.custom_shape("few", 10, 512, 512, 4, 2, seed=8))
    want = r.few(f32=True)
    for bad in (float("nan"), float("inf")):
        x = r.x.clone()
        x[3, 17] = bad
        got = r.few(f32=True, x=x)
        others = [t for t in range(10) if t != 3]
        assert torch.equal(got[others], want[others])
        assert not torch.isfinite(got[3]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("router,n", [("softmax", 6), ("softmax", 4), ("hash", 4)])
def test_a_barrier_that_is_not_met_is_reported(router, n):
    """The handle's test flag makes the grid barriers wait for a block that does not exist, for
    1 ms: the first one, or (launches of few logits, or of the hash router's, have no first) the
    one before the down products, with copies already on their way.  The call ends, the status
    says why, and the handle's barrier words are whole again: the next call ends the same way."""
    shape = synth.with_router(synth.custom_shape("few", n, 512, 1024, 8, 2, seed=6), router)
    r = Run(shape, flags=cb.CB_FLAG_TEST_STALL_DISPATCH | cb.CB_FLAG_GUARDS)
    out = torch.empty(r.x.shape, dtype=torch.bfloat16, device="cuda")
    for _ in range(2):
        r.m.forward_few(r.x, out)
        assert r.m.last_error() == cb.CB_ERR_TIMEOUT
        assert r.m.last_error() == cb.CB_OK and r.m.check_guards() == cb.CB_OK


@pytest.mark.gpu
def test_zero_and_refused_sizes():
    r = Run(synth.custom_shape("few", 17, 256, 256, 4, 2, seed=4))
    out = torch.empty((17, 256), dtype=torch.bfloat16, device="cuda")
    h, x = r.m.handle, r.x.data_ptr()
    assert cb.cb_moe_forward_few(h, x, 0, out.data_ptr()) == cb.CB_OK
    assert cb.cb_moe_forward_few(h, x, -1, out.data_ptr()) == cb.CB_ERR_INVALID_ARG
    assert cb.cb_moe_forward_few(h, x, 17, out.data_ptr()) == cb.CB_ERR_UNSUPPORTED
    assert cb.cb_moe_forward_few(h, x, 1, x) == cb.CB_ERR_INVALID_ARG           # x is out
    assert cb.cb_moe_forward_few(h, x, 1, 0) == cb.CB_ERR_INVALID_ARG
    assert cb.cb_moe_forward_few(h, x + 2, 1, out.data_ptr()) == cb.CB_ERR_ALIGNMENT
    empty = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    assert r.m.forward_few(empty, empty.clone()).shape == (0, 256)
    with pytest.raises(cb.CbMoeError):
        r.m.forward_few(r.x, out)
    with pytest.raises(ValueError):
        r.m.forward_few(r.x[:2], out[:3])
    with pytest.raises(ValueError):
        r.m.forward_few(r.x[:2], out[:2].float())
    with pytest.raises(ValueError):
        r.m.forward_few(r.x[:4, ::2], out[:4, ::2])
    os.environ["CB_MOE_INJECT_FAULT"] = "launch"
    try:
        assert cb.cb_moe_forward_few(h, x, 1, out.data_ptr()) == cb.CB_ERR_CUDA
    finally:
        del os.environ["CB_MOE_INJECT_FAULT"]
    torch.cuda.synchronize()
    assert r.m.last_error() == cb.CB_OK


@pytest.mark.gpu
@pytest.mark.parametrize("wdtype", ["bf16", "int8", "int4", "fp8"])
@pytest.mark.parametrize("n", [3, 14])
def test_every_run_reads_its_own_intermediate_values(wdtype, n):
    """Runs in turn on two inputs without a pause between them: a block that read another block's H
    before it was written would find the other input's there."""
    r = Run(synth.custom_shape("few", n, 512, 2048, 16, 4, wdtype=wdtype, seed=17))
    xs = [r.x, (r.x.view(torch.bfloat16).float() * -0.5).bfloat16().view(r.x.dtype)]
    want = [r.few(f32=True, x=x) for x in xs]
    assert not torch.equal(*want)
    outs = [torch.empty_like(want[0]) for _ in range(200)]
    for i, out in enumerate(outs):
        r.m.forward_few(xs[i % 2], out, f32out=True)
    torch.cuda.synchronize()
    assert all(torch.equal(out, want[i % 2]) for i, out in enumerate(outs))
    assert r.m.last_error() == cb.CB_OK


@pytest.mark.gpu
@pytest.mark.parametrize("wdtype", ["bf16", "int8", "int4", "fp8"])
@pytest.mark.parametrize("n", [3, 14])
def test_a_launch_that_gave_up_leaves_nothing_behind(wdtype, n):
    """Rows of several rings' length, so that the weights' copies are ahead when the barrier's wait
    runs out: the launch sees them land, and other launches right after it are right."""
    shape = synth.custom_shape("few", n, 512, 4096, 8, 2, wdtype=wdtype, seed=23)
    stalled, r = Run(shape, flags=cb.CB_FLAG_TEST_STALL_DISPATCH | cb.CB_FLAG_GUARDS), Run(shape)
    want = r.few(f32=True)
    out, lost = torch.empty_like(want), torch.empty_like(want)
    for _ in range(3):
        stalled.m.forward_few(stalled.x, lost, f32out=True)
        r.m.forward_few(r.x, out, f32out=True)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and r.m.last_error() == cb.CB_OK
        assert stalled.m.last_error() == cb.CB_ERR_TIMEOUT and stalled.m.check_guards() == cb.CB_OK
