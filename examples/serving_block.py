"""One MoE block as a serving program runs it: the routed experts of a layer handle, and beside
them a dense expert that every token takes, its weights kept in 4-bit floating point.

* decode: up to 16 tokens, `MoELayer.forward_few` on the handle that also runs prompts, and the
  dense expert by `fp4_quantize` and `fp4_matmul`, all in one CUDA graph;
* prompt: the handle's ordinary forward, and the same dense expert with more rows;
* routed experts in 4 bits: `fp4_matmul` over the handle's own dispatch (the 128-row tiles of
  its routing), one matrix per expert;
* a whole block with the residual's addition and the norm (`rms_norm`), routing in groups with a
  balance bias (`route`), prompts on the handle with that routing, decode steps on 4-bit integer
  weights in groups (`int4_matmul_few`), again in one CUDA graph.

    python examples/serving_block.py        # runs both on a GB300 and prints their times
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import mixture_experts_router_gb300 as cb  # noqa: E402


def swiglu(gu):
    """SiLU(gate) * up of [tokens][2 f] (gate columns first), in fp32, rounded to bf16."""
    g, u = gu.float().chunk(2, dim=-1)
    return (torch.nn.functional.silu(g) * u).bfloat16()


class DenseExpert:
    """SwiGLU feed-forward with both weight matrices and the activations in 4-bit floats."""

    def __init__(self, w_gate, w_up, w_down, format="mx"):
        self.format = format
        self.up = self._weights(torch.cat([w_gate, w_up]))     # [2 f][d]
        self.down = self._weights(w_down)                      # [d][f]
        # format "nv" has one scale per matrix, for activations fixed ahead of time
        # (their largest block scale, 448, then stands for magnitudes up to 32 * 6)
        self.act_scale = torch.full((1,), 32.0 / 448.0, device=w_down.device) if format == "nv" else None

    def _weights(self, w):
        scale = (w.float().abs().amax() / (6 * 448)).reshape(1) if self.format == "nv" else None
        return cb.fp4_quantize(w.contiguous(), self.format, tensor_scale=scale)

    def __call__(self, x):
        h = swiglu(cb.fp4_matmul(cb.fp4_quantize(x, self.format, self.act_scale), self.up))
        return cb.fp4_matmul(cb.fp4_quantize(h, self.format, self.act_scale), self.down, dtype=torch.float32)


class ServingBlock:
    def __init__(self, prompt_tokens, w_router, w_gate, w_up, w_down, dense, top_k):
        """Routed experts [E][f][d], [E][f][d], [E][d][f] in bf16; dense: a DenseExpert."""
        E, f, d = w_gate.shape
        self.layer = cb.MoELayer(prompt_tokens, d, f, E, top_k, w_router, w_gate, w_up, w_down)
        self.dense, self.d, self.graphs = dense, d, {}

    def prompt(self, x):
        """Up to prompt_tokens tokens: the handle's forward takes exactly that many, so a shorter
        prompt is padded with rows of zeros, whose results are dropped."""
        n, T = x.shape[0], self.layer.cfg.n_tokens
        if n > T:
            raise ValueError(f"a prompt of {n} tokens for a handle of {T}")
        rows = x if n == T else torch.cat([x, x.new_zeros((T - n, self.d))])
        out = torch.empty((T, self.d), dtype=torch.float32, device=x.device)
        self.layer.forward(rows, out, stream=torch.cuda.current_stream(), f32out=True)
        return (out[:n] + self.dense(x)).bfloat16()

    def _decode(self, x):
        out = torch.empty(x.shape, dtype=torch.float32, device=x.device)
        self.layer.forward_few(x, out, stream=torch.cuda.current_stream(), f32out=True)
        return (out + self.dense(x)).bfloat16()

    def decode(self, x):
        """One step for x.shape[0] <= 16 tokens, replayed from a graph per token count."""
        n = x.shape[0]
        if n not in self.graphs:
            static = x.clone()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                self._decode(static)                     # warm-up outside the capture
            torch.cuda.current_stream().wait_stream(side)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                out = self._decode(static)
            self.graphs[n] = (g, static, out)
        g, static, out = self.graphs[n]
        static.copy_(x)
        g.replay()
        return out.clone()


class Fp4Experts:
    """The routed experts themselves in 4-bit floats, over a handle's dispatch: x's rows gathered
    into 128-row tiles per expert, two products with one matrix per expert, the weighted sum."""

    def __init__(self, w_gate, w_up, w_down, format="mx"):
        self.format = format
        self.up = self._stack([torch.cat([g, u]) for g, u in zip(w_gate, w_up)])
        self.down = self._stack(list(w_down))

    def _stack(self, weights):
        scales = [(w.float().abs().amax() / (6 * 448)).reshape(1) if self.format == "nv" else None for w in weights]
        ms = [cb.fp4_quantize(w.contiguous(), self.format, tensor_scale=s) for w, s in zip(weights, scales)]
        return cb.Fp4Matrix(self.format, ms[0].rows, ms[0].cols, torch.stack([m.codes for m in ms]),
                            torch.cat([m.scales for m in ms]), torch.cat(scales) if self.format == "nv" else None)

    def __call__(self, x, layer):
        """x as in layer's last forward, whose routing is used."""
        T, k, E = layer.cfg.n_tokens, layer.cfg.top_k, layer.cfg.n_experts
        if x.shape[0] != T:
            raise ValueError(f"{x.shape[0]} rows for the routing of {T} tokens")
        v, grab, here = layer.routing(), {}, torch.cuda.current_stream()
        for name, n, dtype in (("ids", T * k, torch.int32), ("w", T * k, torch.float32), ("inv", T * k, torch.int32),
                               ("offsets", E + 1, torch.int32), ("tile_offsets", E + 1, torch.int32)):
            grab[name] = torch.empty(n, dtype=dtype, device=x.device)
            cb.copy_from_device(grab[name], getattr(v, name), 4 * n, stream=here)
        ids, tiles = grab["ids"].long(), grab["tile_offsets"]
        rows = 128 * ((T * k + 127 * E) // 128 + 1)       # room for every expert's padding
        at = 128 * tiles[ids].long() + grab["inv"].long() - grab["offsets"][ids].long()   # row of each (token, slot)
        a = torch.zeros((rows, x.shape[1]), dtype=torch.bfloat16, device=x.device)
        a[at] = x.repeat_interleave(k, 0)
        scale = torch.full((1,), 32.0 / 448.0, device=x.device) if self.format == "nv" else None
        q = lambda t: cb.fp4_quantize(t, self.format, scale)  # noqa: E731
        gu = torch.zeros((rows, self.up.rows), dtype=torch.bfloat16, device=x.device)  # rows past the tiles stay zero
        h = swiglu(cb.fp4_matmul(q(a), self.up, out=gu, tile_offsets=tiles))
        y = cb.fp4_matmul(q(h), self.down, dtype=torch.float32, tile_offsets=tiles)
        return (y[at] * grab["w"][:, None]).view(T, k, -1).sum(1)


def int4_groups(w, group=128):
    """w [..][rows][cols] as an Int4Matrix: per group of a row the 16 steps from its least to its largest value."""
    v = w.float().unflatten(-1, (-1, group))
    low, high = v.amin(-1).clamp_max(0), v.amax(-1).clamp_min(0)
    scale = ((high - low) / 15).clamp_min(1e-12)
    zero = (-low / scale).round().clamp(0, 15)
    q = ((v / scale[..., None]).round() + zero[..., None]).clamp(0, 15).to(torch.uint8).flatten(-2)
    codes = q[..., 0::2] | (q[..., 1::2] << 4)
    return cb.Int4Matrix(codes.contiguous(), scale.transpose(-1, -2).contiguous(),
                         zero.to(torch.uint8).transpose(-1, -2).contiguous())


class RoutedBlock:
    """x + residual, norm, routing, routed experts.  Prompts of exactly `prompt_tokens` (shorter ones
    padded) run on a handle with 16-bit weights, decode steps of up to 16 tokens on 4-bit ones."""

    def __init__(self, prompt_tokens, norm, w_router, balance, w_gate, w_up, w_down, top_k, groups, top_groups, scale, group=128):
        E, f, d = w_gate.shape
        self.layer = cb.MoELayer(prompt_tokens, d, f, E, top_k, w_router, w_gate, w_up, w_down)
        self.up, self.down = int4_groups(torch.cat([w_gate, w_up], 1), group), int4_groups(w_down, group)
        self.norm, self.router_t, self.balance = norm, w_router.t().contiguous(), balance
        self.how = dict(top_k=top_k, score="sigmoid", bias=balance, groups=groups, top_groups=top_groups, scale=scale)
        self.graphs = {}

    def prompt(self, x, residual):
        """(the experts' sum, the new residual), both bf16."""
        n, T = x.shape[0], self.layer.cfg.n_tokens
        if n > T:
            raise ValueError(f"a prompt of {n} tokens for a handle of {T}")
        r = cb.rms_norm(x, self.norm, residual=residual)
        rows = r.out if n == T else torch.cat([r.out, r.out.new_zeros((T - n, x.shape[1]))])
        out = torch.empty_like(rows)
        self.layer.forward(rows, out, stream=torch.cuda.current_stream(), routing=cb.route(rows @ self.router_t, **self.how))
        return out[:n], r.sum

    def _decode(self, x, residual):
        r = cb.rms_norm(x, self.norm, residual=residual, want="both")
        ids, w = cb.route(r.out @ self.router_t, **self.how)
        h = cb.int4_matmul_few(r.fp8, self.up, ids=ids, swiglu=True)     # a row per (token, expert)
        return cb.int4_matmul_few(h, self.down, ids=ids, weights=w), r.sum

    def decode(self, x, residual):
        """One step, replayed from a graph per token count."""
        n = x.shape[0]
        if n not in self.graphs:
            held = x.clone(), residual.clone()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                self._decode(*held)                      # warm-up outside the capture
            torch.cuda.current_stream().wait_stream(side)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                out = self._decode(*held)
            self.graphs[n] = (g, held, out)
        g, held, out = self.graphs[n]
        held[0].copy_(x), held[1].copy_(residual)
        g.replay()
        return tuple(t.clone() for t in out)


def random_routed_block(d=2048, f=768, E=64, top_k=6, groups=8, top_groups=4, prompt_tokens=256, group=128, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = lambda *s: torch.empty(s, device="cuda").normal_(0, 0.02, generator=g).bfloat16()  # noqa: E731
    norm = (1 + torch.empty(d, device="cuda").normal_(0, 0.1, generator=g)).bfloat16()
    balance = torch.empty(E, device="cuda").normal_(0, 0.05, generator=g)
    weights = w(E, d), w(E, f, d), w(E, f, d), w(E, d, f)
    return RoutedBlock(prompt_tokens, norm, weights[0], balance, *weights[1:], top_k, groups, top_groups, 2.5, group), weights


def random_block(d=2048, f=768, E=16, top_k=4, dense_f=1536, prompt_tokens=256, format="mx", seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = lambda *s: torch.empty(s, device="cuda").normal_(0, 0.02, generator=g).bfloat16()  # noqa: E731
    routed = w(E, d), w(E, f, d), w(E, f, d), w(E, d, f)
    dense = w(dense_f, d), w(dense_f, d), w(d, dense_f)
    return ServingBlock(prompt_tokens, *routed, DenseExpert(*dense, format=format), top_k), routed, dense


def main():
    block, routed, _ = random_block(4096, 1536, 64, 6, 14336, 2048)
    x = torch.randn(2048, 4096, device="cuda").bfloat16()

    def time(f, n=20):
        f()
        torch.cuda.synchronize()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(n):
            f()
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b) / n * 1e3

    print(f"prompt of 2048 tokens: {time(lambda: block.prompt(x)):.0f} us")
    for n in (1, 4, 16):
        print(f"decode, {n} tokens: {time(lambda: block.decode(x[:n])):.0f} us")
    quant, _ = random_routed_block(4096, 1536, 64, 6, prompt_tokens=2048)
    res = torch.randn(2048, 4096, device="cuda").bfloat16()
    print(f"norm, routing and experts, prompt of 2048 tokens: {time(lambda: quant.prompt(x, res)):.0f} us")
    for n in (1, 4, 16):
        print(f"norm, routing and 4-bit experts, decode, {n} tokens: {time(lambda: quant.decode(x[:n], res[:n])):.0f} us")
    experts = Fp4Experts(*routed[1:])
    print(f"routed experts in 4 bits, 2048 tokens: {time(lambda: experts(x, block.layer)):.0f} us")


if __name__ == "__main__":
    main()
