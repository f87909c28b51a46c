"""What MoELayer's calls and examples/serving_block.py refuse before anything reaches the library, and
that they run where the caller says.  Most of it needs no GPU: the handle is a stand-in."""
import os
import sys
import types

import pytest
import torch

import mixture_experts_router_gb300 as cb

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


class Reached(Exception):
    """The call got as far as the library."""


def layer(T, d, device=0):
    """A MoELayer that stands for a handle of T tokens; nothing is on a GPU."""
    m = cb.MoELayer.__new__(cb.MoELayer)
    m.handle, m.cfg = None, cb.cb_moe_config_t(T, d, 256, 4, 2, cb.CB_W_BF16, device, 0, 0, 0)
    return m


@pytest.fixture
def calls(monkeypatch):
    """The library's forwards, replaced by a record of what reached them."""
    got = []
    for name in ("cb_moe_forward", "cb_moe_forward_f32out", "cb_moe_forward_few", "cb_moe_forward_few_f32out"):
        monkeypatch.setattr(cb, name, lambda *a, name=name: got.append((name,) + a) or cb.CB_OK)
    return got


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


# ---------------------------------------------------------------- forward
def test_forward_refuses_tensors_that_it_would_run_past(calls):
    m = layer(20, 256)
    ok, f32 = bf16(20, 256), torch.zeros(20, 256)
    m.forward(ok, ok.clone())
    m.forward(bf16(33, 256), bf16(33, 256))                              # the first 20 rows
    m.forward(torch.zeros(20 * 256, dtype=torch.int16), ok)              # bits, any shape
    m.forward(ok, f32, f32out=True)
    assert len(calls) == 4
    short, gaps = bf16(19, 256), bf16(20, 512)[:, ::2]
    for x, out, kind in ((short, ok, False), (ok, short, False), (ok, ok.clone(), True), (gaps, ok, False), (ok, gaps, False),
                         (bf16(1, 256).expand(20, 256), ok, False)):
        with pytest.raises(ValueError):
            m.forward(x, out, f32out=kind)
    assert len(calls) == 4


# ------------------------------------------------------------ forward_few
class On:
    """A tensor said to be on a CUDA device: what the call asks of one."""

    def __init__(self, t, device=0):
        self.t, self.device = t, f"cuda:{device}"
        self.shape, self.dtype, self.index = t.shape, t.dtype, device

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.index


def test_forward_few_refuses_other_types(calls):
    """float16 has bf16's size, and its bits would be read as bf16's."""
    m, x = layer(20, 256), On(bf16(3, 256))
    stream = types.SimpleNamespace(cuda_stream=5)
    m.forward_few(x, On(bf16(3, 256)), stream=stream)
    m.forward_few(On(torch.zeros(3, 256, dtype=torch.int16)), On(torch.zeros(3, 256, dtype=torch.int16)), stream=stream)
    m.forward_few(x, On(torch.zeros(3, 256)), stream=stream, f32out=True)
    assert len(calls) == 3
    for a, b, f32 in ((torch.float16, torch.bfloat16, False), (torch.bfloat16, torch.float16, False),
                      (torch.bfloat16, torch.float32, False), (torch.bfloat16, torch.int32, True),
                      (torch.bfloat16, torch.bfloat16, True), (torch.uint8, torch.bfloat16, False)):
        with pytest.raises(ValueError):
            m.forward_few(On(torch.zeros(3, 256, dtype=a)), On(torch.zeros(3, 256, dtype=b)), stream=stream, f32out=f32)
    assert len(calls) == 3


def test_forward_few_refuses_other_devices(calls):
    """A host tensor's address, or another GPU's, never reaches the kernel."""
    x = bf16(3, 256)
    stream = types.SimpleNamespace(cuda_stream=5)
    layer(20, 256, device=1).forward_few(On(x, 1), On(x.clone(), 1), stream=stream)
    assert len(calls) == 1
    for a, b in ((x, x.clone()), (On(x), x.clone()), (x, On(x)), (On(x, 1), On(x)), (On(x), On(x, 1))):
        with pytest.raises(ValueError):
            layer(20, 256).forward_few(a, b, stream=stream)
    assert len(calls) == 1


def test_forward_few_runs_on_the_current_stream(calls, monkeypatch):
    """As the 4-bit calls beside it do: its input was written there."""
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 100 + device, raising=False)
    x = bf16(3, 256)
    layer(20, 256).forward_few(On(x), On(x.clone()))
    layer(20, 256, device=1).forward_few(On(x, 1), On(x.clone(), 1))
    layer(20, 256).forward_few(On(x), On(x.clone()), stream=types.SimpleNamespace(cuda_stream=5))
    assert [c[-1] for c in calls] == [100, 101, 5]


@pytest.mark.gpu
def test_forward_few_follows_its_input_on_a_side_stream():
    import gpu_harness as gh
    import synth
    s = synth.custom_shape("few", 5, 512, 512, 8, 2, seed=2)
    lay = synth.make_layer(s)
    m = cb.MoELayer(s.T, s.d, s.f, s.E, s.k, *(gh.to_dev(getattr(lay, n)) for n in ("wr", "wg", "wu", "wd")))
    x = gh.to_dev(lay.x)
    want, y, out = torch.empty_like(x), torch.zeros_like(x), torch.empty_like(x)
    m.forward_few(x, want)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda._sleep(20_000_000)                # y is written some 10 ms from now
        y.copy_(x)
        m.forward_few(y, out)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# ---------------------------------------------------------------- example
def test_serving_block_takes_prompts_up_to_its_handles_tokens(calls, monkeypatch):
    import serving_block as sb
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=5))
    block = sb.ServingBlock.__new__(sb.ServingBlock)
    block.layer, block.d, block.dense = layer(20, 256), 256, lambda x: torch.zeros(x.shape[0], 256)
    for n in (20, 7, 0):
        assert block.prompt(bf16(n, 256)).shape == (n, 256)
    assert [c[0] for c in calls] == ["cb_moe_forward_f32out"] * 3
    with pytest.raises(ValueError):
        block.prompt(bf16(21, 256))


def test_fp4_experts_refuse_rows_that_were_not_routed():
    import serving_block as sb
    for n in (19, 21):
        with pytest.raises(ValueError):
            sb.Fp4Experts.__call__(None, bf16(n, 256), layer(20, 256))


class Runtime:
    """The CUDA runtime's copies, recorded."""

    def __init__(self):
        self.streams = []

    def cudaMemcpy(self, dst, src, n, kind):
        self.streams.append("legacy")
        return 0

    def cudaMemcpyAsync(self, dst, src, n, kind, stream):
        self.streams.append(stream)
        return 0


def test_copies_of_the_routing_run_where_they_are_used(monkeypatch):
    import serving_block as sb
    rt = Runtime()
    monkeypatch.setattr(cb, "_cudart", rt)
    cb.copy_from_device(torch.zeros(4), 64, 16)
    cb.copy_from_device(torch.zeros(4), 64, 16, stream=types.SimpleNamespace(cuda_stream=9))
    cb.copy_from_device(torch.zeros(4), 64, 0, stream=types.SimpleNamespace(cuda_stream=9))
    assert rt.streams == ["legacy", 9]
    # the example, up to its first use of what it copied
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=7))
    m = layer(20, 256)
    m.routing = lambda: types.SimpleNamespace(ids=64, w=64, inv=64, offsets=64, tile_offsets=64)
    monkeypatch.setattr(torch.Tensor, "long", lambda t: (_ for _ in ()).throw(Reached()))
    with pytest.raises(Reached):
        sb.Fp4Experts.__call__(None, bf16(20, 256), m)
    assert rt.streams[2:] == [7] * 5


@pytest.mark.gpu
def test_fp4_experts_on_a_side_stream():
    """The routing that a forward on a side stream is still to write."""
    import serving_block as sb
    block, routed, _ = sb.random_block(d=512, f=256, E=12, top_k=3, dense_f=256, prompt_tokens=90, seed=3)
    experts = sb.Fp4Experts(*routed[1:])
    x, other = (torch.randn(90, 512, device="cuda").bfloat16() for _ in range(2))
    block.prompt(x)
    want = experts(x, block.layer)
    block.prompt(other)                              # another routing in the meantime
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda._sleep(20_000_000)
        block.prompt(x)
        got = experts(x, block.layer)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.gpu
def test_prompts_of_several_lengths():
    """A short prompt is the full one whose other rows are zeros (the routed experts' part: k = 2, so
    that the order of a token's additions does not matter)."""
    import serving_block as sb
    block, _, _ = sb.random_block(d=512, f=256, E=8, top_k=2, dense_f=256, prompt_tokens=100)
    block.dense = lambda x: torch.zeros(x.shape, device="cuda")
    x = torch.randn(100, 512, device="cuda").bfloat16()
    for n in (1, 37, 99):
        padded = torch.cat([x[:n], torch.zeros_like(x[n:])])
        got, want = block.prompt(x[:n]), block.prompt(padded)[:n]
        assert torch.equal(got, want) and got.abs().max() > 0
    assert block.layer.last_error() == cb.CB_OK
