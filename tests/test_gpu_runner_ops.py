"""GPU tests of the layer's runner with its norm, the router's balance loss and 4-bit experts, as one run of the operators
together."""
import pytest
import torch

import moe_reference as R
import mx4_reference as X
import norm_reference as N
from gated_mlp_gemms_amd.moe_runner import MoeRunner, main, moe_tensors
from gpu_helpers import announce

pytestmark = pytest.mark.gpu
COEF = 0.75


def leaves(t, ids, kind, score, mask, coef):
    """The layer's output, balance loss and leaves in float64 on the CPU, from the formulas."""
    leaf = {k: v.double().cpu().requires_grad_() for k, v in t.items() if k not in ("dout", "mask")}
    h, E = leaf["x"], t["router"].shape[0]
    c = h - h.mean(dim=1, keepdim=True) if kind == "layer" else h
    x = c / (c.square().mean(dim=1, keepdim=True) + 1e-5).sqrt() * leaf["norm_weight"]
    if kind == "layer":
        x = x + leaf["norm_bias"]
    z = x @ leaf["router"].T
    p = torch.softmax(z, 1) if score == "softmax" else torch.sigmoid(z)
    w = p.gather(1, ids)
    w = w / w.sum(1, keepdim=True)
    out = h
    for j in range(ids.shape[1]):
        e = ids[:, j]
        g, u = ((leaf[n][e] @ x[:, :, None])[:, :, 0] for n in ("w_gate", "w_up"))
        out = out + w[:, j:j + 1] * (leaf["w_down"][e] @ (torch.nn.functional.silu(g) * u)[:, :, None])[:, :, 0]
    live = torch.ones(len(h), dtype=torch.bool) if mask is None else mask.cpu()
    f = torch.bincount(ids[live].reshape(-1), minlength=E).double() / (int(live.sum()) * ids.shape[1])
    q = p / p.sum(1, keepdim=True)
    loss = E * (f * q[live].mean(0)).sum()
    return leaf, out, loss


@pytest.mark.parametrize("kind,score,masked,experts", [("layer", "softmax", False, 8), ("rms", "sigmoid", True, 8),
                                                       ("rms", "softmax", True, 7), ("layer", "sigmoid", False, 7)])
def test_training_step_against_double(kind, score, masked, experts):
    """fp32: norm, router, balance loss, experts and every gradient, against autograd of the formulas in float64. The bound is
    that of the runner with a norm outside it, of two norms (the forward's and the backward's sums over a row) more."""
    size = dict(act="swiglu", dtype="f32", tokens=45, width=32, hidden=40, experts=experts)
    announce(f"runner {kind} {score} {experts} experts, mask {masked}")
    t = moe_tensors(seed=11, norm=kind, **size)
    if masked:
        t["mask"] = torch.arange(45, device="cuda") % 3 > 0
    r = MoeRunner(choices=3, tensors=t, score=score, norm=kind, balance=COEF, **size)
    r.step()
    leaf, out, loss = leaves(t, r.ids.long().cpu(), kind, score, t.get("mask"), COEF)
    R.check("loss", r.loss.cpu(), loss.detach()[None], torch.full((1,), 100 * R.U32 * loss.item(), dtype=torch.float64))
    ((out * t["dout"].double().cpu()).sum() + COEF * loss).backward()
    names = {"dx": "x", "d_norm_weight": "norm_weight", "d_norm_bias": "norm_bias", "d_router": "router", "dw1": "w_gate",
             "dw_up": "w_up", "dw2": "w_down"}
    grads = r.grads()
    assert sorted(grads) == sorted(k for k, n in names.items() if n in leaf)
    for k, a, b in [("out", r.out, out.detach())] + [(k, grads[k], leaf[names[k]].grad) for k in grads]:
        R.check(k, a.cpu(), b, torch.full_like(b, 3200 * R.U32 * b.abs().max().item()))
    infer = MoeRunner(choices=3, tensors=t, score=score, norm=kind, balance=COEF, train=False, **size)
    assert torch.equal(infer.forward_infer(), r.out)


def test_balance_gradient_against_differences():
    """The router's gradient of the balance loss alone (dout 0), against central differences of the loss in float64: the steps
    of 1e-4 are off by their square times a third derivative, both far below the bound."""
    size = dict(act="swiglu", dtype="f32", tokens=30, width=32, hidden=32, experts=5)
    t = moe_tensors(seed=12, norm="rms", **size)
    t["dout"].zero_()
    r = MoeRunner(choices=2, tensors=t, norm="rms", balance=COEF, **size)
    r.step()
    ids = r.ids.long().cpu()

    def loss(router):
        with torch.no_grad():
            return COEF * leaves({**t, "router": router}, ids, "rms", "softmax", None, COEF)[2].item()

    scale = r.grads()["d_router"].abs().max().item()
    assert scale > 0
    for e, c in [(0, 0), (1, 7), (2, 31), (4, 16)]:
        d = torch.zeros_like(t["router"], dtype=torch.float64)
        d[e, c] = 1e-4
        diff = (loss(t["router"].double() + d) - loss(t["router"].double() - d)) / 2e-4
        assert abs(r.grads()["d_router"][e, c].item() - diff) <= 3200 * R.U32 * scale + 1e-7 * scale


@pytest.mark.parametrize("act,tokens,experts,bias", [("swiglu", 1, 8, False), ("swiglu", 60, 8, True), ("relu_sq", 60, 7, True)])
@pytest.mark.parametrize("dtype", list(R.DT))
def test_inference_with_4bit_experts(act, tokens, experts, bias, dtype):
    """Stage by stage from the runner's own buffers: blocks equal the formula's, products within their bounds; and again from
    a replayed graph, the same bits."""
    announce(f"runner with 4-bit experts {act} {tokens} tokens {dtype}")
    size = dict(act=act, dtype=dtype, tokens=tokens, width=96, hidden=160, experts=experts)
    t = moe_tensors(seed=13, norm="rms", bias=bias, **size)
    r = MoeRunner(choices=3, tensors=t, norm="rms", train=False, mx4=True, **size)
    out = r.forward_infer().clone()
    dt, gated = R.DT[dtype], act in R.GATED
    y = N.norm_fwd(t["x"], t["norm_weight"], None, "rms", 1e-5)
    R.check("norm", r.x, y[0], y[3] + R.half_step(dt) * (y[0].abs() + y[3]) + R.floor_of(dt))
    off = r.offsets.cpu()
    token = r.slot_of.long() // 3
    assert torch.equal(r.xs, r.x[token])
    for (codes, scales), x in ((r.xs4, r.xs), (r.a4, r.a), (r.w1_4, r.w1), (r.w2_4, r.w2)):
        code, scale = X.unpack(codes, scales)
        rc, rs = X.encode(x)
        assert torch.equal(code, rc) and torch.equal(scale[..., : rs.shape[-1]], rs)
    xq, aq, w1, w2 = (X.rounded(v) for v in (r.xs, r.a, r.w1, r.w2))
    w_up = X.rounded(r.w_up) if gated else None
    ref, pre, mag = R.linear(act, xq, w1, w_up, r.b1, r.b_up, None, off)
    R.check("a", r.a, ref, R.linear_bound(act, dt, 96, ref, pre, mag, 160))
    ref, pre, mag = R.linear("none", aq, w2, None, r.b2, None, None, off)
    R.check("ys", r.ys, ref, R.linear_bound("none", dt, 160, ref, pre, mag, 96))
    ys = r.ys.double()[r.row_of.long()].reshape(tokens, 3, 96)
    w = r.weights.double()[:, :, None]
    ref = t["x"].double() + (w * ys).sum(1)
    R.check("out", out, ref, R.half_step(dt) * ref.abs() + 16 * R.U32 * (t["x"].double().abs() + (w * ys).abs().sum(1)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.forward_infer()
    for _ in range(3):
        r.out.zero_()
        graph.replay()
        assert torch.equal(r.out, out)
    # other weights, the blocks made anew
    r.w1.mul_(0.5)
    r.quantize_weights()
    r.out.zero_()
    graph.replay()
    code, scale = X.unpack(*r.w1_4)
    rc, rs = X.encode(r.w1)
    assert torch.equal(code, rc) and torch.equal(scale[..., : rs.shape[-1]], rs)


def test_training_step_in_a_graph():
    """bf16: the step's replays, with eager steps of a second runner between them, equal the eager step."""
    size = dict(act="swiglu", dtype="bf16", tokens=300, width=256, hidden=136, experts=8)
    t = moe_tensors(seed=14, norm="layer", **size)
    a, b = (MoeRunner(choices=2, tensors=t, norm="layer", balance=COEF, **size) for _ in range(2))
    a.step()
    want = {**{k: v.clone() for k, v in a.grads().items()}, "loss": a.loss.clone(), "out": a.out.clone()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step()
    for _ in range(3):
        for v in a.grads().values():
            v.zero_()
        a.loss.zero_()
        graph.replay()
        b.step()
        torch.cuda.synchronize()
        for r in (a, b):
            got = {**r.grads(), "loss": r.loss, "out": r.out}
            for k, v in want.items():
                assert torch.equal(got[k], v), k


def test_refusals():
    size = dict(act="swiglu", dtype="bf16", tokens=4, width=64, hidden=64, experts=4)
    t = moe_tensors(norm="rms", **size)
    for more, text in ((dict(norm="group"), "norm must be"), (dict(norm="rms", tensors={**t, "residual": t["x"]}), "residual"),
                       (dict(mx4=True), "inference")):
        with pytest.raises(ValueError, match=text):
            MoeRunner(choices=2, **{"tensors": t, **size, **more})


def test_command(capsys):
    main(["--tokens", "64", "--width", "64", "--hidden", "96", "--experts", "4", "--choices", "2", "--steps", "2",
          "--decode-tokens", "3", "--norm", "layer", "--balance", "0.01", "--mx4"])
    text = capsys.readouterr().out
    assert "training step, 64 tokens" in text and "in a graph, 3 tokens" in text
