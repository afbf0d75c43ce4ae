"""Device buffers for one mixture-of-experts layer and the calls of its training step and its inference
forward, as ``runner.py`` holds them for the MLP. Every operator runs in the library's kernels; torch only adds ``dout``
to the router's part of dx and copies the columns of a router whose number of experts is not a multiple of a 16-byte
row's (8, fp32 4).

    out = x + sum over a token's k experts of weight (act(x W_gate^T) x W_up^T) W_down^T

(the residual stream x goes into the combine; where x is a norm of it, the stream is a tensor of its own, or with ``norm``
the runner takes the norm itself: the experts' and the router's x is then norm(x)). ``balance`` adds that much of the
router's balance loss to what is trained on; with ``mx4`` the inference forward's experts are microscaled 4-bit.
As a command it times one layer::

    python -m gated_mlp_gemms_amd.moe_runner --tokens 4096 --width 2048 --hidden 1376 --experts 32 --choices 4
"""
from __future__ import annotations

import torch

from . import GATED_ACTS
from .moe import (linear_bwd, linear_fwd, linear_workspace_bytes, make_linear_desc, moe_balance, moe_balance_bwd,
                  moe_balance_workspace_bytes, moe_combine, moe_combine_bwd, moe_gather, moe_route, moe_route_bwd, moe_sort,
                  moe_sort_workspace_bytes)
from .mx4 import mx4_linear_fwd, mx4_linear_workspace_bytes, mx4_quantize, mx4_shapes
from .norm import norm_bwd, norm_fwd, norm_workspace_bytes


class MoeRunner:
    """``tokens`` rows of ``width`` through ``experts`` experts of ``hidden`` units, ``choices`` a token.
    ``tensors``: x, dout [tokens, width]; router [experts, width]; w_gate, w_up (gated) or w1
    [experts, hidden, width]; w_down or w2 [experts, width, hidden]; optional b_gate, b_up or b1, b_down or b2; optional
    residual [tokens, width], added to the output in x's place: its gradient is dout, which dx then leaves out.
    ``train`` False holds no more than ``forward_infer`` needs.
    ``norm`` "layer" or "rms": the layer works on norm(x) (tensors norm_weight, optional norm_bias [width]; ``eps`` the
    norm's), x being the residual stream. ``balance`` above 0: ``forward`` leaves the balance loss in ``loss`` [1] and the
    experts' loads in ``counts`` and ``shares``, and the gradients are those of the layer's loss plus ``balance`` times it; optional
    mask [tokens] (bool): the tokens that it counts. ``mx4`` (``train`` False): the experts work on 4-bit
    blocks of their weights, made here and by :meth:`quantize_weights` from the weights, which stay held beside them, and
    their inputs are rounded to blocks; width and hidden are multiples of 32."""

    def __init__(self, *, act, dtype, tokens, width, hidden, experts, choices, tensors, score="softmax", renorm=True,
                 train=True, device="cuda", norm=None, balance=0.0, mx4=False, eps=1e-5):
        if norm is not None and "residual" in tensors:
            raise ValueError("with a norm the residual stream is x itself")
        if norm not in (None, "layer", "rms"):
            raise ValueError(f'norm must be None, "layer" or "rms", not {norm!r}')
        if mx4 and train:
            raise ValueError("4-bit experts are for inference: train must be False")
        dt = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}.get(dtype, dtype)
        dev = torch.device(device)
        t = {k: v.to(dev) for k, v in tensors.items()}
        gated = act in GATED_ACTS
        T, d, h, E, k = int(tokens), int(width), int(hidden), int(experts), int(choices)
        n = T * k
        self.train, self.score, self.renorm, self.experts, self.dtype = train, score, renorm, E, dt
        self.x, self.router, self.residual = t["x"], t["router"], t.get("residual", t["x"])
        self.norm, self.eps, self.mx4 = norm, float(eps), mx4
        self.balance, self.mask = float(balance) if train else 0.0, t.get("mask")
        self.w1, self.w_up, self.w2 = t["w_gate" if gated else "w1"], t.get("w_up"), t["w_down" if gated else "w2"]
        self.b1, self.b_up, self.b2 = t.get("b_gate" if gated else "b1"), t.get("b_up"), t.get("b_down" if gated else "b2")

        def new(*shape, of=dt):
            return torch.empty(*shape, dtype=of, device=dev)

        i32, f32, u8 = torch.int32, torch.float32, torch.uint8
        if norm is not None:   # the stream is normed into a tensor of its own, which the layer then works on
            self.stream, self.x = self.x, new(T, d)
            self.norm_weight, self.norm_bias = t["norm_weight"], t.get("norm_bias")
            self.mean, self.rstd = (new(T, of=f32) if train and v else None for v in (norm == "layer", True))
        if self.balance:
            self.counts, self.shares, self.loss = new(E + 1, of=i32), new(E, of=f32), new(1, of=f32)
            self.dloss = new(1, of=f32).fill_(self.balance)
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
        need = max(need, moe_sort_workspace_bytes(n, E))
        if self.balance:
            need = max(need, moe_balance_workspace_bytes(T, E))
        if mx4:
            need = max(need, *(mx4_linear_workspace_bytes(q) for q in (self.up_desc, self.down_desc)))

            def blocks(rows, K, batch=None):
                return [new(*s, of=u8) for s in mx4_shapes(rows, K, batch)]

            self.xs4, self.a4 = blocks(n, d), blocks(n, h)
            self.w1_4, self.w2_4 = blocks(h, d, E), blocks(d, h, E)
            self.w_up_4 = blocks(h, d, E) if gated else (None, None)
            self.quantize_weights()
        if norm is not None and train:
            need = max(need, norm_workspace_bytes(T, d))
        # the calls follow one another on one stream: they share a workspace
        self.ws = new(need, of=u8)
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
            self.d_norm_weight = self.d_norm_bias = None
            if norm is not None:
                self.d_stream = new(T, d)
                self.d_norm_weight, self.d_norm_bias = like(self.norm_weight), like(self.norm_bias)

    def quantize_weights(self):
        """The experts' 4-bit blocks from their weights (``mx4``): again after the weights have changed."""
        for w, blocks in ((self.w1, self.w1_4), (self.w_up, self.w_up_4), (self.w2, self.w2_4)):
            if w is not None:
                mx4_quantize(w, *blocks)

    def _experts(self, preact):
        if self.mx4:
            mx4_quantize(self.xs, *self.xs4)
            mx4_linear_fwd(self.up_desc, *self.xs4, *self.w1_4, self.a, w_up=self.w_up_4[0], w_up_scales=self.w_up_4[1],
                           bias=self.b1, bias_up=self.b_up, offsets=self.offsets, workspace=self.ws)
            mx4_quantize(self.a, *self.a4)
            mx4_linear_fwd(self.down_desc, *self.a4, *self.w2_4, self.ys, bias=self.b2, offsets=self.offsets,
                           workspace=self.ws)
            return
        linear_fwd(self.up_desc, self.xs, self.w1, self.a, w_up=self.w_up, bias=self.b1, bias_up=self.b_up,
                   offsets=self.offsets, preact=preact, workspace=self.ws)
        linear_fwd(self.down_desc, self.a, self.w2, self.ys, bias=self.b2, offsets=self.offsets, workspace=self.ws)

    def _forward(self, train):
        preact = self.preact if train else None
        if self.norm is not None:
            norm_fwd(self.stream, self.x, weight=self.norm_weight, bias=self.norm_bias, mean=self.mean if train else None,
                     rstd=self.rstd if train else None, kind=self.norm, eps=self.eps)
        if self.wide_router is not self.router:
            self.wide_router[: self.experts].copy_(self.router)
        linear_fwd(self.r_desc, self.x, self.wide_router, self.wide_logits, workspace=self.ws)
        if self.wide_logits is not self.logits:
            self.logits.copy_(self.wide_logits[:, : self.experts])
        moe_route(self.logits, self.ids, self.weights, score=self.score, renorm=self.renorm)
        if train and self.balance:
            moe_balance(self.logits, self.ids, self.counts, self.shares, self.loss, mask=self.mask, score=self.score,
                        workspace=self.ws)
        moe_sort(self.ids, self.experts, self.offsets, self.row_of, self.slot_of, workspace=self.ws)
        moe_gather(self.x, self.slot_of, self.offsets, self.xs)
        self._experts(preact)
        moe_combine(self.ys, self.weights, self.row_of, self.offsets, self.out, residual=self.residual)
        return self.out

    def forward(self):
        return self._forward(True)

    def forward_infer(self):
        """The output alone: the balance loss with its loads, the norm's statistics and the pre-activation stay as
        :meth:`forward` left them."""
        return self._forward(False)

    def backward(self):
        """Every gradient of :meth:`forward` against ``dout`` (and ``balance`` times the balance loss); ``dx`` is the sum
        of the experts' rows', the router's and, where x is the residual, dout; with a norm it is norm(x)'s, and ``d_stream``
        x's."""
        moe_combine_bwd(self.dout, self.ys, self.weights, self.row_of, self.slot_of, self.offsets, self.dys, self.dweights)
        linear_bwd(self.down_desc, self.dys, self.a, self.w2, offsets=self.offsets, dx=self.da, dw=self.dw2,
                   dbias=self.db2, workspace=self.ws)
        linear_bwd(self.up_desc, self.da, self.xs, self.w1, w_up=self.w_up, preact=self.preact, offsets=self.offsets,
                   dx=self.dxs, dw=self.dw1, dw_up=self.dw_up, dbias=self.db1, dbias_up=self.db_up, workspace=self.ws)
        if self.balance:
            moe_balance_bwd(self.logits, self.ids, self.counts, self.dlogits, mask=self.mask, dloss=self.dloss,
                            dweights=self.dweights, score=self.score, renorm=self.renorm)
        else:
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
        if self.norm is not None:   # dx is norm(x)'s; the stream's own gradient is dout besides
            norm_bwd(self.dx, self.stream, self.rstd, self.d_stream, mean=self.mean, weight=self.norm_weight,
                     dresidual=self.dout, dweight=self.d_norm_weight, dbias=self.d_norm_bias, kind=self.norm,
                     workspace=self.ws)

    def step(self):
        self.forward()
        self.backward()

    def grads(self) -> dict:
        g = {"dx": self.dx if self.norm is None else self.d_stream, "d_norm_weight": self.d_norm_weight,
             "d_norm_bias": self.d_norm_bias, "d_router": self.d_router, "dw1": self.dw1, "dw_up": self.dw_up, "dw2": self.dw2,
             "db1": self.db1, "db_up": self.db_up, "db2": self.db2}
        return {k: v for k, v in g.items() if v is not None}


def moe_tensors(*, act, dtype, tokens, width, hidden, experts, seed=0, device="cuda", bias=False, norm=None) -> dict:
    """Seeded synthetic inputs and weights of a :class:`MoeRunner`, with ``norm`` those of its norm, too."""
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
    if norm is not None:
        t["norm_weight"] = (1 + 0.1 * torch.randn(width, device=device, generator=gen)).to(dt)
        if norm == "layer":
            t["norm_bias"] = normal(width, scale=0.1)
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
    p.add_argument("--norm", default=None, choices=("layer", "rms"), help="norm the residual stream in front of the layer")
    p.add_argument("--balance", type=float, default=0.0, help="how much of the balance loss the training step adds")
    p.add_argument("--mx4", action="store_true", help="4-bit experts in the inference forward")
    o = p.parse_args(argv)
    size = dict(act=o.act, dtype=o.dtype, width=o.width, hidden=o.hidden, experts=o.experts, norm=o.norm)
    t = moe_tensors(tokens=o.tokens, **size)
    r = MoeRunner(tokens=o.tokens, choices=o.choices, tensors=t, score=o.score, balance=o.balance, **size)
    ms = _time(r.step, o.steps)
    mats = 3 if o.act in GATED_ACTS else 2
    flops = 6.0 * o.tokens * o.choices * mats * o.width * o.hidden
    print(f"training step, {o.tokens} tokens: {ms:.3f} ms, {o.tokens / ms * 1e3:.0f} tokens/s, "
          f"{flops / ms / 1e9:.0f} TFLOP/s of the experts' products")
    few = {**t, "x": t["x"][: o.decode_tokens].contiguous()}
    d = MoeRunner(tokens=few["x"].shape[0], choices=o.choices, tensors=few, score=o.score, train=False, mx4=o.mx4, **size)
    d.forward_infer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.forward_infer()
    ms = _time(graph.replay, o.steps)
    print(f"inference forward in a graph, {few['x'].shape[0]} tokens: {ms * 1e3:.1f} us")


if __name__ == "__main__":
    main()
