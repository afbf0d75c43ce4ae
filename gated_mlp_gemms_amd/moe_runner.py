"""Device buffers for one mixture-of-experts layer and the calls of its training step and its inference
forward, as ``runner.py`` holds them for the MLP. Every operator runs in the library's kernels; torch only adds ``dout``
to the router's part of dx and copies the columns of a router whose number of experts is not a multiple of a 16-byte
row's (8, fp32 4).

    out = x + sum over a token's k experts of weight (act(x W_gate^T) x W_up^T) W_down^T

(the residual stream x goes into the combine; where x is a norm of it, the stream is a tensor of its own). As a command it times one layer::

    python -m gated_mlp_gemms_amd.moe_runner --tokens 4096 --width 2048 --hidden 1376 --experts 32 --choices 4
"""
from __future__ import annotations

import torch

from . import GATED_ACTS
from .moe import (linear_bwd, linear_fwd, linear_workspace_bytes, make_linear_desc, moe_combine, moe_combine_bwd,
                  moe_gather, moe_route, moe_route_bwd, moe_sort, moe_sort_workspace_bytes)


class MoeRunner:
    """``tokens`` rows of ``width`` through ``experts`` experts of ``hidden`` units, ``choices`` a token.
    ``tensors``: x, dout [tokens, width]; router [experts, width]; w_gate, w_up (gated) or w1
    [experts, hidden, width]; w_down or w2 [experts, width, hidden]; optional b_gate, b_up or b1, b_down or b2; optional
    residual [tokens, width], added to the output in x's place: its gradient is dout, which dx then leaves out.
    ``train`` False holds no more than ``forward_infer`` needs."""

    def __init__(self, *, act, dtype, tokens, width, hidden, experts, choices, tensors, score="softmax", renorm=True,
                 train=True, device="cuda"):
        dt = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}.get(dtype, dtype)
        dev = torch.device(device)
        t = {k: v.to(dev) for k, v in tensors.items()}
        gated = act in GATED_ACTS
        T, d, h, E, k = int(tokens), int(width), int(hidden), int(experts), int(choices)
        n = T * k
        self.train, self.score, self.renorm, self.experts, self.dtype = train, score, renorm, E, dt
        self.x, self.router, self.residual = t["x"], t["router"], t.get("residual", t["x"])
        self.w1, self.w_up, self.w2 = t["w_gate" if gated else "w1"], t.get("w_up"), t["w_down" if gated else "w2"]
        self.b1, self.b_up, self.b2 = t.get("b_gate" if gated else "b1"), t.get("b_up"), t.get("b_down" if gated else "b2")

        def new(*shape, of=dt):
            return torch.empty(*shape, dtype=of, device=dev)

        i32, f32 = torch.int32, torch.float32
        self.logits, self.ids, self.weights = new(T, E), new(T, k, of=i32), new(T, k, of=f32)
        # The logits have the layer's type, as every tensor of a linear layer does: of 16 bits, a score is off by half a
        # step of that type, so near ties between experts may fall either way. moe_route takes fp32 scores from
        # wherever a program has them.
        # A linear layer's rows are 16-byte aligned: for another number of experts the router's product has
        # columns of zero weights behind, which its logits leave out
        q = 4 if dt == torch.float32 else 8
        Er = (E + q - 1) // q * q
        self.wide_router, self.wide_logits = self.router, self.logits
        if Er != E:
            self.wide_router, self.wide_logits = new(Er, d).zero_(), new(T, Er)
        self.offsets, self.row_of, self.slot_of = new(E + 1, of=i32), new(n, of=i32), new(n, of=i32)
        self.xs, self.a, self.ys, self.out = new(n, d), new(n, h), new(n, d), new(T, d)
        self.r_desc = make_linear_desc(T, d, Er, dtype=dt)
        self.up_desc = make_linear_desc(n, d, h, act=act, dtype=dt, experts=E)
        self.down_desc = make_linear_desc(n, h, d, dtype=dt, experts=E)
        phases = ("fwd", "bwd") if train else ("fwd",)
        need = max(linear_workspace_bytes(q, p) for q in (self.r_desc, self.up_desc, self.down_desc) for p in phases)
        # the calls follow one another on one stream: they share a workspace
        self.ws = new(max(need, moe_sort_workspace_bytes(n, E)), of=torch.uint8)
        if train:
            self.dout = t["dout"]
            self.preact = new(n, 2 * h if gated else h)
            self.dys, self.dweights, self.da, self.dxs = new(n, d), new(T, k, of=f32), new(n, h), new(n, d)
            self.dlogits, self.dx_router, self.dx = new(T, E), new(T, d), new(T, d)
            self.ones = new(T, k, of=f32).fill_(1.0)   # the weights of the experts' rows in dx
            like = lambda v: torch.empty_like(v) if v is not None else None   # noqa: E731
            self.wide_dlogits = self.dlogits
            self.d_router, self.dw1, self.dw_up, self.dw2 = like(self.router), like(self.w1), like(self.w_up), like(self.w2)
            self.wide_d_router = self.d_router
            if Er != E:
                self.wide_dlogits, self.wide_d_router = new(T, Er).zero_(), new(Er, d)
            self.db1, self.db_up, self.db2 = like(self.b1), like(self.b_up), like(self.b2)

    def _forward(self, preact):
        if self.wide_router is not self.router:
            self.wide_router[: self.experts].copy_(self.router)
        linear_fwd(self.r_desc, self.x, self.wide_router, self.wide_logits, workspace=self.ws)
        if self.wide_logits is not self.logits:
            self.logits.copy_(self.wide_logits[:, : self.experts])
        moe_route(self.logits, self.ids, self.weights, score=self.score, renorm=self.renorm)
        moe_sort(self.ids, self.experts, self.offsets, self.row_of, self.slot_of, workspace=self.ws)
        moe_gather(self.x, self.slot_of, self.offsets, self.xs)
        linear_fwd(self.up_desc, self.xs, self.w1, self.a, w_up=self.w_up, bias=self.b1, bias_up=self.b_up,
                   offsets=self.offsets, preact=preact, workspace=self.ws)
        linear_fwd(self.down_desc, self.a, self.w2, self.ys, bias=self.b2, offsets=self.offsets, workspace=self.ws)
        moe_combine(self.ys, self.weights, self.row_of, self.offsets, self.out, residual=self.residual)
        return self.out

    def forward(self):
        return self._forward(self.preact)

    def forward_infer(self):
        return self._forward(None)

    def backward(self):
        """Every gradient of :meth:`forward` against ``dout``; ``dx`` is the sum of the experts' rows', the router's
        and, where x is the residual, dout."""
        moe_combine_bwd(self.dout, self.ys, self.weights, self.row_of, self.slot_of, self.offsets, self.dys, self.dweights)
        linear_bwd(self.down_desc, self.dys, self.a, self.w2, offsets=self.offsets, dx=self.da, dw=self.dw2,
                   dbias=self.db2, workspace=self.ws)
        linear_bwd(self.up_desc, self.da, self.xs, self.w1, w_up=self.w_up, preact=self.preact, offsets=self.offsets,
                   dx=self.dxs, dw=self.dw1, dw_up=self.dw_up, dbias=self.db1, dbias_up=self.db_up, workspace=self.ws)
        moe_route_bwd(self.logits, self.ids, self.dweights, self.dlogits, score=self.score, renorm=self.renorm)
        if self.wide_dlogits is not self.dlogits:
            self.wide_dlogits[:, : self.experts].copy_(self.dlogits)
        linear_bwd(self.r_desc, self.wide_dlogits, self.x, self.wide_router, dx=self.dx_router, dw=self.wide_d_router,
                   workspace=self.ws)
        if self.wide_d_router is not self.d_router:
            self.d_router.copy_(self.wide_d_router[: self.experts])
        # summed in fp32 and rounded once; the router's part has been rounded, and with dout's once more
        rest = self.dx_router
        if self.residual is self.x:
            rest = torch.add(self.dx_router, self.dout, out=self.dx)
        moe_combine(self.dxs, self.ones, self.row_of, self.offsets, self.dx, residual=rest)

    def step(self):
        self.forward()
        self.backward()

    def grads(self) -> dict:
        g = {"dx": self.dx, "d_router": self.d_router, "dw1": self.dw1, "dw_up": self.dw_up, "dw2": self.dw2,
             "db1": self.db1, "db_up": self.db_up, "db2": self.db2}
        return {k: v for k, v in g.items() if v is not None}


def moe_tensors(*, act, dtype, tokens, width, hidden, experts, seed=0, device="cuda", bias=False) -> dict:
    """Seeded synthetic inputs and weights of a :class:`MoeRunner`."""
    gen = torch.Generator(device=device).manual_seed(seed)
    dt = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}.get(dtype, dtype)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, device=device, generator=gen) * scale).to(dt)

    up, down = ("w_gate", "w_down") if act in GATED_ACTS else ("w1", "w2")
    t = {"x": normal(tokens, width), "dout": normal(tokens, width), "router": normal(experts, width, scale=width ** -0.5),
         up: normal(experts, hidden, width, scale=width ** -0.5), down: normal(experts, width, hidden, scale=hidden ** -0.5)}
    if act in GATED_ACTS:
        t["w_up"] = normal(experts, hidden, width, scale=width ** -0.5)
    if bias:
        b1, b2 = ("b_gate", "b_down") if act in GATED_ACTS else ("b1", "b2")
        t.update({b1: normal(experts, hidden, scale=0.1), b2: normal(experts, width, scale=0.1)})
        if act in GATED_ACTS:
            t["b_up"] = normal(experts, hidden, scale=0.1)
    return t


def _time(f, n):
    for _ in range(3):
        f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(n):
        f()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) / n


def main(argv=None):
    import argparse

    p = argparse.ArgumentParser(prog="python -m gated_mlp_gemms_amd.moe_runner", description="time one layer of experts")
    for name, v in (("tokens", 4096), ("width", 2048), ("hidden", 1376), ("experts", 32), ("choices", 4), ("steps", 20),
                    ("decode-tokens", 16)):
        p.add_argument(f"--{name}", type=int, default=v)
    p.add_argument("--act", default="swiglu")
    p.add_argument("--dtype", default="bf16", choices=("bf16", "f16", "f32"))
    p.add_argument("--score", default="softmax", choices=("softmax", "sigmoid"))
    o = p.parse_args(argv)
    size = dict(act=o.act, dtype=o.dtype, width=o.width, hidden=o.hidden, experts=o.experts)
    t = moe_tensors(tokens=o.tokens, **size)
    r = MoeRunner(tokens=o.tokens, choices=o.choices, tensors=t, score=o.score, **size)
    ms = _time(r.step, o.steps)
    mats = 3 if o.act in GATED_ACTS else 2
    flops = 6.0 * o.tokens * o.choices * mats * o.width * o.hidden
    print(f"training step, {o.tokens} tokens: {ms:.3f} ms, {o.tokens / ms * 1e3:.0f} tokens/s, "
          f"{flops / ms / 1e9:.0f} TFLOP/s of the experts' products")
    few = {**t, "x": t["x"][: o.decode_tokens].contiguous()}
    d = MoeRunner(tokens=few["x"].shape[0], choices=o.choices, tensors=few, score=o.score, train=False, **size)
    d.forward_infer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.forward_infer()
    ms = _time(graph.replay, o.steps)
    print(f"inference forward in a graph, {few['x'].shape[0]} tokens: {ms * 1e3:.1f} us")


if __name__ == "__main__":
    main()
